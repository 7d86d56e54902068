"""The example decoder with token layers: it runs, and its gradients are the operators'."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import image_decoder
    return image_decoder


def test_training_runs(example):
    losses = example.train(steps=3, log=lambda line: None, layers=2)
    assert len(losses) == 3 and all(torch.isfinite(torch.tensor(losses)))


def test_every_parameter_gets_a_gradient(example):
    import gen
    import gaussian_splatting_tile_bin_gb300 as gsr
    ctx = gsr.Context(0)
    model = example.Decoder(ctx, views=2, grid=8, tokens=200, layers=2)
    features = torch.randn(2, 8, 8, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    camera = gen.lego_scene(n=1).camera.copy()
    camera[12:16] *= 64 / 800
    mask = torch.ones(1, 128, dtype=torch.bool, device="cuda")
    example.Render.apply(ctx, model(features, mask), camera, 64).square().sum().backward()
    names = [name for name, _ in model.named_parameters()]
    assert sum(name.startswith("layers.") for name in names) == 8
    for name, parameter in model.named_parameters():
        assert torch.isfinite(parameter.grad).all(), name
        assert parameter.grad.abs().sum() > 0, name
    ctx.close()


def test_a_layers_gradient(example):
    """A layer in float against autograd through plain operations in 64 bits: within 128 roundings
    of the largest value for each of its six steps, none of which spreads an error by more than
    8 times."""
    import gaussian_splatting_tile_bin_gb300 as gsr
    torch.backends.cuda.matmul.allow_tf32 = False
    ctx = gsr.Context(0)
    c, n = 32, 90
    layer = example.TokenLayer(ctx, c, torch.Generator().manual_seed(2))
    g = torch.Generator().manual_seed(3)
    x, residual, d0, d1 = (torch.randn(1, n, c, generator=g) for _ in range(4))
    dev = [t.cuda().requires_grad_() for t in (x, residual)]
    y, total = layer(*dev)
    ((y * d0.cuda()).sum() + (total * d1.cuda()).sum()).backward()

    wide = [t.double().requires_grad_() for t in (x, residual)]
    p = {k: v.detach().cpu().double().requires_grad_() for k, v in layer.named_parameters()}
    s = wide[0] + wide[1]
    hat = (s - s.mean(-1, keepdim=True)) / torch.sqrt(s.var(-1, correction=0, keepdim=True) + 1e-5)
    parts = (hat * p["norm_weight"] + p["norm_bias"]) @ p["to_parts"]
    sides = []
    for k, order in ((0, range(n)), (3, range(n - 1, -1, -1))):
        v, f, o = (parts[0, :, (k + i) * c:(k + i + 1) * c] for i in range(3))
        h, hs = torch.zeros(c, dtype=torch.float64), {}
        for t in order:
            a = torch.sigmoid(f[t])
            h = a * h + (1 - a) * v[t]
            hs[t] = h
        sides.append(torch.stack([hs[t] for t in range(n)]) * torch.nn.functional.silu(o))
    want = torch.cat(sides, dim=1)[None] @ p["back"]
    ((want * d0).sum() + (s * d1).sum()).backward()
    pairs = [(y, want), (total, s)] + [(a.grad, b.grad) for a, b in zip(dev, wide)]
    pairs += [(v.grad, p[k].grad) for k, v in layer.named_parameters()]
    for got, value in pairs:
        error = (got.detach().cpu().double() - value.detach()).abs().max() / value.detach().abs().max()
        assert error <= 6 * 8 * 128 * 2.0 ** -24, float(error)
    ctx.close()
