"""Helper of test_gpu_recurrence_lanes.py: runs the recurrence over ragged items whose last lanes
have no channels, through loads and through bulk copies, with whichever libgsr.so GSR_LIBRARY
selects, and saves every output to the .npz named on the command line."""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gaussian_splatting_tile_bin_gb300 as gsr  # noqa: E402

SHAPES = [(3, 700, 33, torch.bfloat16, False), (4, 600, 77, torch.float32, True), (3, 500, 250, torch.bfloat16, True),
          (3, 900, 40, torch.float16, False), (5, 300, 5, torch.float32, False)]


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
