"""Blocks of the recurrence that take tile after tile of many ragged items, through the rings of
copies and through loads, give each item the bits that it has alone, where a block takes one."""
import pytest
import torch

from test_gpu_gated_recurrence import BF16, F16, F32, _dev, _inputs, ctx, gsr  # noqa: F401
from test_gpu_token_layers import _held_up

pytestmark = pytest.mark.gpu


def _step(gsr, ctx, t, items, lengths, reverse):  # noqa: F811
    at = {k: None if v is None else v[items] for k, v in t.items()}
    how = dict(lengths=lengths[items], reverse=reverse)
    out, final, states = gsr.gated_recurrence_forward(ctx, at["x"], at["forget"], at["gate"], initial=at["initial"], **how)
    grads = gsr.gated_recurrence_backward(ctx, at["dout"], at["x"], at["forget"], at["gate"], states,
                                          dl_dfinal=at["dfinal"], **how)
    return [out, final] + [g for g in grads if g is not None]


@pytest.mark.parametrize("dtype,c", [(BF16, 128), (F16, 136), (BF16, 130), (F16, 33), (F32, 64), (F32, 33)])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("reverse", [False, True])
def test_many_tiles_of_a_block(gsr, ctx, dtype, c, gate, reverse):  # noqa: F811
    b, n = 40, 2600
    t = {k: _dev(v) for k, v in _inputs(b, n, c, dtype, c, gate).items()}
    some = [n, 0, 1, 127, 128, 129, 1024, 1025, 2559, 2560, 2561, 17]
    lengths = torch.tensor([some[i % len(some)] if i % 3 else (577 * i) % (n + 1) for i in range(b)], dtype=torch.int32,
                           device="cuda")
    together = _step(gsr, ctx, t, slice(0, b), lengths, reverse)
    for i in range(0, b, 3):
        for whole, alone in zip(together, _step(gsr, ctx, t, slice(i, i + 1), lengths, reverse)):
            assert torch.equal(whole[i:i + 1], alone)
    for i in range(1, len(some)):
        for whole, alone in zip(together, _step(gsr, ctx, t, slice(i, i + 1), lengths, reverse)):
            assert torch.equal(whole[i:i + 1], alone)


def test_warps_that_are_held_up_change_no_bit(gsr, tmp_path):  # noqa: F811
    _held_up(tmp_path, "recurrence.cu", "recurrence_rings_run")
