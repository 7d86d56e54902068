"""The decoder operators' C ABI without a GPU: the binding's packed layouts are
the header's, and calls without a context fail cleanly."""
import ctypes
import os
import struct
import subprocess

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
    printf("%zu %zu %zu %zu\n", sizeof(gsr_group_norm), sizeof(gsr_heads), sizeof(gsr_rotary), sizeof(gsr_attention));
    printf("%zu %zu %zu\n", offsetof(gsr_group_norm, positions), offsetof(gsr_group_norm, activation),
           offsetof(gsr_group_norm, eps));
    printf("%zu %zu %zu\n", offsetof(gsr_rotary, sections), offsetof(gsr_rotary, positions_int),
           offsetof(gsr_rotary, positions_batch_stride));
    printf("%zu %zu %zu\n", offsetof(gsr_attention, scale), offsetof(gsr_attention, kv_lengths),
           offsetof(gsr_attention, key_mask));
    printf("%d %d %d %d\n", GSR_MAX_AXES, GSR_F32, GSR_BF16, GSR_F16);
    return 0;
}
''')
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = [[int(v) for v in line.split()] for line in subprocess.check_output([str(exe)], text=True).splitlines()]
    assert got[0] == [t.size for t in (_abi.GROUP_NORM, _abi.HEADS, _abi.ROTARY, _abi.ATTENTION)]

    assert got[1] == [struct_offset("@4i", "q"), struct_offset("@4iq", "i"), struct_offset("@4iqi", "f")]
    assert got[2] == [struct_offset("@7i", "i"), struct_offset("@11i", "i"), struct_offset("@12i", "q")]
    assert got[3] == [struct_offset("@7i", "f"), struct_offset("@7if", "P"), struct_offset("@7ifP", "P")]
    assert got[4] == [_abi.MAX_AXES] + [_abi.DTYPES[t] for t in (torch.float32, torch.bfloat16, torch.float16)]


def struct_offset(before, field):
    """Offset of a field behind others in a native layout."""
    return struct.calcsize(before + field) - struct.calcsize("@" + field)


@pytest.mark.parametrize("name,pointers", [("gsr_group_norm_forward", 9), ("gsr_group_norm_backward", 12),
                                           ("gsr_rotary_forward", 7), ("gsr_rotary_backward", 7),
                                           ("gsr_cross_attention_forward", 8), ("gsr_cross_attention_backward", 12)])
def test_null_context(lib, name, pointers):
    call = getattr(lib, name)
    call.argtypes = [ctypes.c_void_p] * pointers
    assert call(*[None] * pointers) == 1


def test_cpu_tensors_are_refused_before_any_call(lib):
    import gaussian_splatting_tile_bin_gb300 as gsr
    x = torch.zeros(2, 4, 2, 8)
    for call in (lambda: gsr.group_norm_forward(None, x, 2), lambda: gsr.rotary_forward(None, x, x, x, [4]),
                 lambda: gsr.cross_attention_forward(None, x.bfloat16(), x, x),
                 lambda: gsr.cross_attention_forward(None, x, x, x)):
        with pytest.raises(ValueError, match="must be"):
            call()
