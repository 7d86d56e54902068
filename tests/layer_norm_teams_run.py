"""Helper of test_gpu_layer_norm_teams.py: runs the layer norm over rows that warps of one block
share, of one team to eight, with whichever libgsr.so GSR_LIBRARY selects, and saves every output
to the .npz named on the command line."""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gaussian_splatting_tile_bin_gb300 as gsr  # noqa: E402

SHAPES = [(6000, 520, torch.bfloat16), (3001, 1280, torch.float32), (2000, 2049, torch.float16), (900, 4096, torch.bfloat16),
          (700, 8191, torch.float32)]


def outputs():
    ctx = gsr.Context(0)
    res = {}
    for n, (rows, c, dtype) in enumerate(SHAPES):
        g = torch.Generator().manual_seed(n)
        x, r, dout, dt = (torch.randn(rows, c, generator=g).to(dtype).cuda() for _ in range(4))
        w, b = (torch.randn(c, generator=g).cuda() for _ in range(2))
        for run in range(3):
            out, total, mean, rstd = gsr.layer_norm_forward(ctx, x, w, b, residual=r)
            grads = gsr.layer_norm_backward(ctx, dout, total, w, mean, rstd, dl_dtotal=dt)
            for name, t in zip(("out", "mean", "rstd", "dx", "dw", "db"), (out, mean, rstd, *grads)):
                res[f"{n}.{run}.{name}"] = t.float().cpu().numpy()
    ctx.synchronize()
    ctx.close()
    return res


if __name__ == "__main__":
    np.savez(sys.argv[1], **outputs())
