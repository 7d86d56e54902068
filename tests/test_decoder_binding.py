"""The binding's checks of the decoder's operators that need no GPU: tensors without
storage stand in for another device's."""
import types

import pytest
import torch


def _elsewhere(*shape, dtype=torch.bfloat16, device="cuda:1"):
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        return torch.empty(*shape, dtype=dtype, device=device)


def test_tensors_of_another_device_are_refused():
    """The kernels run on the context's device: another's pointers would fault there."""
    import __graft_entry__
    __graft_entry__._build_module().build()
    import gaussian_splatting_tile_bin_gb300 as gsr
    ctx = types.SimpleNamespace(device=0, _h=None)
    x, stats = _elsewhere(2, 5, 16), _elsewhere(2, 4, dtype=torch.float32)
    q, lse = _elsewhere(2, 5, 2, 16), _elsewhere(2, 2, 5, dtype=torch.float32)
    positions, freq = _elsewhere(5, 1, dtype=torch.float32), _elsewhere(8, dtype=torch.float32)
    for call in (lambda: gsr.group_norm_forward(ctx, x, 4),
                 lambda: gsr.group_norm_backward(ctx, x, x, 4, None, None, stats, stats),
                 lambda: gsr.rotary_forward(ctx, q, positions, freq, [8]),
                 lambda: gsr.rotary_backward(ctx, q, positions, freq, [8]),
                 lambda: gsr.cross_attention_forward(ctx, q, q, q),
                 lambda: gsr.cross_attention_backward(ctx, q, q, q, q, lse, q)):
        with pytest.raises(ValueError, match="is on cuda:1, the context on cuda:0"):
            call()
