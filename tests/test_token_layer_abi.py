"""The token layers' C ABI and binding without a GPU: packed layouts, calls without a
context, tensors of the CPU and of another device."""
import ctypes
import os
import subprocess
import types

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    return ctypes.CDLL(__graft_entry__._build_module().build())


def test_packed_layouts_match_the_header(tmp_path, lib):
    from gaussian_splatting_tile_bin_gb300 import _abi
    src = tmp_path / "layout.c"
    src.write_text(r'''
#include <stdio.h>
#include <stddef.h>
#include "gsr.h"
int main(void) {
    printf("%zu %zu %zu %zu %d\n", sizeof(gsr_layer_norm), offsetof(gsr_layer_norm, eps), sizeof(gsr_recurrence),
           offsetof(gsr_recurrence, lengths), GSR_RECURRENCE_BLOCK);
    return 0;
}
''')
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)], text=True).split()]
    assert got == [_abi.LAYER_NORM.size, 20, _abi.RECURRENCE.size, _abi.RECURRENCE.size - 8, _abi.RECURRENCE_BLOCK]


@pytest.mark.parametrize("name,pointers", [("gsr_layer_norm_forward", 11), ("gsr_layer_norm_backward", 12),
                                           ("gsr_gated_recurrence_forward", 10), ("gsr_gated_recurrence_backward", 13)])
def test_null_context(lib, name, pointers):
    call = getattr(lib, name)
    call.argtypes = [ctypes.c_void_p] * pointers
    assert call(*[None] * pointers) == 1


def test_cpu_tensors_are_refused_before_any_call(lib):
    import gaussian_splatting_tile_bin_gb300 as gsr
    x = torch.zeros(2, 4, 8)
    for call in (lambda: gsr.layer_norm_forward(None, x), lambda: gsr.layer_norm_backward(None, x, x, None, x, x),
                 lambda: gsr.gated_recurrence_forward(None, x, x),
                 lambda: gsr.gated_recurrence_backward(None, x, x, x, None, x)):
        with pytest.raises(ValueError, match="must be"):
            call()


def test_tensors_of_another_device_are_refused(lib):
    import gaussian_splatting_tile_bin_gb300 as gsr
    from torch._subclasses.fake_tensor import FakeTensorMode
    ctx = types.SimpleNamespace(device=0, _h=None)
    with FakeTensorMode():
        x = torch.empty(2, 5, 16, dtype=torch.bfloat16, device="cuda:1")
        stats = torch.empty(2, 5, device="cuda:1")
    for call in (lambda: gsr.layer_norm_forward(ctx, x), lambda: gsr.layer_norm_backward(ctx, x, x, None, stats, stats),
                 lambda: gsr.gated_recurrence_forward(ctx, x, x),
                 lambda: gsr.gated_recurrence_backward(ctx, x, x, x, None, stats)):
        with pytest.raises(ValueError, match="is on cuda:1, the context on cuda:0"):
            call()
