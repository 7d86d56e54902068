"""Helper of test_gpu_recurrence_rings.py: runs the recurrence over ragged items of which a block
takes tile after tile, with whichever libgsr.so GSR_LIBRARY selects, and saves every output to the
.npz named on the command line."""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gaussian_splatting_tile_bin_gb300 as gsr  # noqa: E402

SHAPES = [(20, 2500, 128, torch.bfloat16, False), (15, 2500, 66, torch.float16, True), (30, 1500, 64, torch.float32, True)]


def outputs():
    ctx = gsr.Context(0)
    res = {}
    for n, (b, tokens, c, dtype, reverse) in enumerate(SHAPES):
        g = torch.Generator().manual_seed(n)
        x, f, o, dout = (torch.randn(b, tokens, c, generator=g).to(dtype).cuda() for _ in range(4))
        lengths = torch.randint(1, tokens, (b,), generator=g, dtype=torch.int32).cuda()
        for run in range(3):
            out, final, states = gsr.gated_recurrence_forward(ctx, x, f, o, lengths=lengths, reverse=reverse)
            grads = gsr.gated_recurrence_backward(ctx, dout, x, f, o, states, lengths=lengths, reverse=reverse)
            for name, t in zip(("out", "final", "dx", "df", "do", "di"), (out, final, *grads)):
                res[f"{n}.{run}.{name}"] = t.float().cpu().numpy()
    ctx.synchronize()
    ctx.close()
    return res


if __name__ == "__main__":
    np.savez(sys.argv[1], **outputs())
