"""Fits a small image-to-Gaussians decoder through the rasterizer.

Feature maps of a few views go through a group norm with SiLU; their patches
become keys and values with rotary positions (view, row, column); Gaussian tokens
attend to all of them, a linear head turns each token into a 3-D Gaussian, and
the Gaussians are projected, binned and composited.  The image's gradient goes
back the same way into every parameter.

    python examples/image_decoder.py --steps 60
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import gaussian_splatting_tile_bin_gb300 as gsr  # noqa: E402
import gen  # noqa: E402


class NormAct(torch.autograd.Function):
    @staticmethod
    def forward(fn, ctx, x, groups, weight, bias):
        out, mean, rstd = gsr.group_norm_forward(ctx, x, groups, weight, bias, activation="silu")
        fn.save_for_backward(x, weight, bias, mean, rstd)
        fn.ctx, fn.groups = ctx, groups
        return out

    @staticmethod
    def backward(fn, dout):
        x, weight, bias, mean, rstd = fn.saved_tensors
        dx, dw, db = gsr.group_norm_backward(fn.ctx, dout.contiguous(), x, fn.groups, weight, bias, mean, rstd)
        return None, dx, None, dw, db


class Rotary(torch.autograd.Function):
    @staticmethod
    def forward(fn, ctx, x, positions, frequencies, sections):
        fn.ctx, fn.args = ctx, (positions, frequencies, sections)
        return gsr.rotary_forward(ctx, x, positions, frequencies, sections)

    @staticmethod
    def backward(fn, dout):
        return None, gsr.rotary_backward(fn.ctx, dout.contiguous(), *fn.args), None, None, None


class CrossAttention(torch.autograd.Function):
    @staticmethod
    def forward(fn, ctx, q, k, v, key_mask):
        out, lse = gsr.cross_attention_forward(ctx, q, k, v, key_mask=key_mask)
        fn.save_for_backward(q, k, v, out, lse, key_mask)
        fn.ctx = ctx
        return out

    @staticmethod
    def backward(fn, dout):
        q, k, v, out, lse, key_mask = fn.saved_tensors
        grads = gsr.cross_attention_backward(fn.ctx, q, k, v, out, lse, dout.contiguous(), key_mask=key_mask)
        return (None, *grads, None)


class Render(torch.autograd.Function):
    """Gaussians [n, 14] to an image [side * side, 3]."""

    @staticmethod
    def forward(fn, ctx, gaussians, camera, side):
        splats, depths = gsr.project_forward(ctx, gaussians, camera)
        bins = gsr.bin_splats(ctx, splats, depths, side, side)
        out, final_t, last = gsr.rasterize_forward(ctx, splats, bins)
        fn.ctx, fn.camera, fn.bins = ctx, camera, bins
        fn.save_for_backward(gaussians, splats, final_t, last)
        return out[:, :3]

    @staticmethod
    def backward(fn, dimage):
        gaussians, splats, final_t, last = fn.saved_tensors
        dout = torch.zeros((dimage.shape[0], 4), device=dimage.device)
        dout[:, :3] = dimage
        dsplats = gsr.rasterize_backward(fn.ctx, splats, fn.bins, dout, final_t, last)
        return None, gsr.project_backward(fn.ctx, gaussians, fn.camera, dsplats), None, None


class Decoder(torch.nn.Module):
    def __init__(self, ctx, views, grid, channels=64, tokens=1024, q_heads=4, kv_heads=2, dim=64, seed=0):
        super().__init__()
        self.ctx, self.shape = ctx, (tokens, q_heads, kv_heads, dim)
        gen_ = torch.Generator().manual_seed(seed)

        def parameter(*shape, scale):
            return torch.nn.Parameter((torch.randn(shape, generator=gen_) * scale).cuda())

        self.norm_weight = torch.nn.Parameter(torch.ones(channels, device="cuda"))
        self.norm_bias = torch.nn.Parameter(torch.zeros(channels, device="cuda"))
        self.to_k = parameter(channels, kv_heads * dim, scale=channels ** -0.5)
        self.to_v = parameter(channels, kv_heads * dim, scale=channels ** -0.5)
        self.queries = parameter(1, tokens, q_heads * dim, scale=1.0)
        self.head = parameter(q_heads * dim, 14, scale=0.02)
        # The Gaussians the head's output is added to: a cloud in the middle of the scene.
        base = torch.zeros(tokens, 14)
        base[:, :3] = torch.rand((tokens, 3), generator=gen_) * 2 - 1
        base[:, 3:6] = -3.0
        base[:, 6] = 1.0
        base[:, 11:] = 0.5
        self.register_buffer("base", base.cuda())
        # Positions: (view, row, column) of a patch; a query's own place in the cloud.
        self.sections = [8, 12, 12]
        self.register_buffer("frequencies", gsr.rotary_frequencies(self.sections))
        view, row, col = torch.meshgrid(torch.arange(views), torch.arange(grid), torch.arange(grid), indexing="ij")
        keys = torch.stack([view, row, col], dim=-1).reshape(-1, 3)
        self.register_buffer("key_positions", keys.to(torch.int32).cuda())
        self.register_buffer("query_positions", ((base[:, :3] + 1) * grid / 2).contiguous().cuda())

    def forward(self, features, key_mask):
        """features [views, rows, columns, channels] bf16 to Gaussians [tokens, 14]."""
        tokens, q_heads, kv_heads, dim = self.shape
        x = NormAct.apply(self.ctx, features, 8, self.norm_weight, self.norm_bias)
        x = x.reshape(1, -1, features.shape[-1])
        k = (x @ self.to_k.to(x.dtype)).view(1, -1, kv_heads, dim)
        v = (x @ self.to_v.to(x.dtype)).view(1, -1, kv_heads, dim)
        q = self.queries.to(x.dtype).view(1, tokens, q_heads, dim)
        k = Rotary.apply(self.ctx, k, self.key_positions, self.frequencies, self.sections)
        q = Rotary.apply(self.ctx, q, self.query_positions, self.frequencies, self.sections)
        out = CrossAttention.apply(self.ctx, q, k, v, key_mask)
        return self.base + out.reshape(tokens, -1).float() @ self.head


def train(steps=60, views=3, grid=16, side=128, seed=0, log=print):
    """Returns the losses of `steps` Adam steps towards one view of a synthetic scene."""
    ctx = gsr.Context(0)
    scene = gen.lego_scene(n=4000, seed=seed)
    camera = scene.camera.copy()
    camera[12:16] *= side / 800                     # fx, fy, cx, cy of an 800 x 800 image
    with torch.no_grad():
        target = Render.apply(ctx, torch.from_numpy(scene.gaussians).cuda(), camera, side)
    generator = torch.Generator().manual_seed(seed)
    features = torch.randn((views, grid, grid, 64), generator=generator).to(torch.bfloat16).cuda()
    key_mask = torch.ones((1, views * grid * grid), dtype=torch.bool, device="cuda")
    key_mask[:, ::grid] = False                     # the first column of every view lies off the object
    model = Decoder(ctx, views, grid, seed=seed)
    optimizer = torch.optim.Adam(model.parameters(), lr=1e-2)
    losses = []
    for step in range(steps):
        optimizer.zero_grad()
        image = Render.apply(ctx, model(features, key_mask), camera, side)
        loss = ((image - target) ** 2).mean()
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step}: loss {losses[-1]:.5f}")
    ctx.synchronize()                               # raises if a kernel gave up on the way
    ctx.close()
    return losses


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=60)
    train(parser.parse_args().steps)
