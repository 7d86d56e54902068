"""The example decoder: its operators and the rasterizer in one training step."""
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


def test_training_lowers_the_loss(example):
    losses = example.train(steps=25, log=lambda line: None)
    assert all(torch.isfinite(torch.tensor(losses)))
    assert losses[-1] < 0.8 * losses[0]


def test_every_parameter_gets_a_gradient(example):
    import gen
    import gaussian_splatting_tile_bin_gb300 as gsr
    ctx = gsr.Context(0)
    model = example.Decoder(ctx, views=2, grid=8, tokens=200)
    features = torch.randn(2, 8, 8, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    camera = gen.lego_scene(n=1).camera.copy()
    camera[12:16] *= 64 / 800
    mask = torch.ones(1, 128, dtype=torch.bool, device="cuda")
    image = example.Render.apply(ctx, model(features, mask), camera, 64)
    image.square().sum().backward()
    for name, parameter in model.named_parameters():
        assert torch.isfinite(parameter.grad).all(), name
        assert parameter.grad.abs().sum() > 0, name
    ctx.close()
