"""The decoder operators' host code on the CPU, against a runtime that runs nothing
(fake_runtime.cpp): which uses of the workspace streams, events and captures order,
and what happens to memory that a captured graph holds."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
OK, INVALID_ARG, CUDA, OOM = 0, 1, 2, 3
ONE, TWO, THREE, FOUR = (ctypes.c_void_p(0x100 * i) for i in (1, 2, 3, 4))
AT = 1 << 30    # where the arrays would lie; nothing reads them


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    import __graft_entry__
    build = __graft_entry__._build_module()
    build.build()
    objects = [os.path.join(build.BUILD, os.path.basename(s) + ".o") for s in build.sources()]
    if not all(os.path.exists(o) for o in objects):
        build.build(force=True)
    out = str(tmp_path_factory.mktemp("fake") / "libgsr_fake.so")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    # -Bsymbolic: the fake runtime's functions, whatever else the process has loaded
    subprocess.check_call(["g++", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", f"-I{cuda}/include", "-o", out,
                           os.path.join(HERE, "fake_runtime.cpp"), *objects, "-ldl"])
    fake = ctypes.CDLL(out)
    for name in ("fake_new_stream", "fake_begin_capture", "fake_end_capture"):
        getattr(fake, name).argtypes = [ctypes.c_void_p]
    fake.fake_edge.argtypes = [ctypes.c_void_p] * 2
    for name, pointers in (("group_norm_forward", 9), ("group_norm_backward", 12), ("rotary_forward", 7),
                           ("cross_attention_forward", 8), ("cross_attention_backward", 12)):
        getattr(fake, "gsr_" + name).argtypes = [ctypes.c_void_p] * pointers
    fake.gsr_destroy.argtypes = [ctypes.c_void_p]
    fake.gsr_last_error.argtypes = [ctypes.c_void_p]
    fake.gsr_last_error.restype = ctypes.c_char_p
    return fake


@pytest.fixture
def ctx(lib):
    lib.fake_reset()
    handle = ctypes.c_void_p()
    assert lib.gsr_create(ctypes.byref(handle), 0) == OK
    yield handle
    lib.fake_reset()


def _heads(tokens, heads, dim=64):
    from gaussian_splatting_tile_bin_gb300 import _abi
    return _abi.HEADS.pack(AT, tokens * heads * dim, heads * dim, dim)


def attention(lib, ctx, stream, tokens=200, keys=700, mask=False, backward=False):
    from gaussian_splatting_tile_bin_gb300 import _abi
    desc = _abi.ATTENTION.pack(2, 2, tokens, keys, 4, 2, 64, 0.125, 0, AT if mask else 0)
    q, k = _heads(tokens, 4), _heads(keys, 2)
    if backward:
        return lib.gsr_cross_attention_backward(ctx, desc, q, k, k, q, AT, q, q, k, k, stream)
    return lib.gsr_cross_attention_forward(ctx, desc, q, k, k, q, AT, stream)


def norm(lib, ctx, stream, channels=64, backward=False):
    from gaussian_splatting_tile_bin_gb300 import _abi
    desc = _abi.GROUP_NORM.pack(1, 2, channels, 8, 200000, 1, 1e-5)
    if backward:
        return lib.gsr_group_norm_backward(ctx, desc, AT, AT, AT, AT, AT, AT, AT, AT, AT, stream)
    return lib.gsr_group_norm_forward(ctx, desc, AT, AT, AT, AT, AT, AT, stream)


def test_eager_streams_are_ordered(lib, ctx):
    for call in (attention, norm):
        for stream in (ONE, TWO, ONE, THREE):
            assert call(lib, ctx, stream) == OK
            assert call(lib, ctx, stream, backward=True) == OK
    assert lib.fake_conflicts() == 0 and lib.fake_launches() > 20


@pytest.mark.parametrize("call", [attention, norm])
def test_growth_keeps_what_a_graph_holds(lib, ctx, call):
    assert call(lib, ctx, ONE) == OK
    lib.fake_begin_capture(ONE)
    assert call(lib, ctx, ONE) == OK
    lib.fake_end_capture(ONE)
    size = {attention: dict(tokens=3000, keys=9000, mask=True), norm: dict(channels=2048)}[call]
    assert call(lib, ctx, ONE, **size) == OK
    assert lib.fake_freed_while_held() == 0
    # A second graph takes the grown workspace, and the next growth keeps both.
    lib.fake_begin_capture(TWO)
    assert call(lib, ctx, TWO, **size) == OK
    lib.fake_end_capture(TWO)
    assert attention(lib, ctx, ONE, tokens=6000, keys=40000, mask=True, backward=True) == OK
    assert lib.fake_freed_while_held() == 0 and lib.fake_allocations() == 3
    lib.gsr_destroy(ctx)
    assert lib.fake_live() == 0


def test_growth_frees_what_no_graph_holds(lib, ctx):
    for keys in (500, 5000, 50000):
        assert attention(lib, ctx, ONE, keys=keys, mask=True) == OK
        assert lib.fake_allocations() == 1


def test_growth_during_a_capture_is_refused(lib, ctx):
    assert attention(lib, ctx, ONE) == OK
    lib.fake_begin_capture(ONE)
    assert attention(lib, ctx, ONE, keys=50000, mask=True) == CUDA
    assert b"capture" in lib.gsr_last_error(ctx)


@pytest.mark.parametrize("call", [attention, norm])
def test_streams_of_one_capture_are_ordered(lib, ctx, call):
    """Branches that the caller forks and joins share the workspace one after the other."""
    for stream in (ONE, TWO):
        assert call(lib, ctx, stream) == OK
        assert call(lib, ctx, stream, backward=True) == OK
    for _ in range(2):
        lib.fake_begin_capture(ONE)
        assert lib.fake_edge(ONE, TWO) == OK and lib.fake_edge(ONE, THREE) == OK
        for stream in (ONE, TWO, THREE, ONE, TWO):
            assert call(lib, ctx, stream) == OK
        assert call(lib, ctx, THREE, backward=True) == OK
        assert lib.fake_edge(TWO, ONE) == OK and lib.fake_edge(THREE, ONE) == OK
        lib.fake_end_capture(ONE)
        # Outside the capture the live streams go on as before it.
        assert call(lib, ctx, TWO) == OK and call(lib, ctx, ONE) == OK
    assert lib.fake_conflicts() == 0 and lib.fake_pulled_in() == 0


def test_captures_side_by_side(lib, ctx):
    """Captures that know nothing of each other, with live calls between theirs."""
    for stream in (ONE, TWO, THREE, FOUR):
        assert attention(lib, ctx, stream) == OK
    lib.fake_begin_capture(ONE)
    lib.fake_begin_capture(TWO)
    assert lib.fake_edge(ONE, THREE) == OK
    for stream in (ONE, FOUR, TWO, THREE, FOUR, TWO, ONE):
        assert attention(lib, ctx, stream) == OK
    assert lib.fake_edge(THREE, ONE) == OK
    lib.fake_end_capture(ONE)
    lib.fake_end_capture(TWO)
    assert attention(lib, ctx, ONE) == OK
    assert lib.fake_conflicts() == 0 and lib.fake_pulled_in() == 0


@pytest.mark.parametrize("call", [attention, norm])
def test_a_handle_that_another_stream_has_taken(lib, ctx, call):
    """A stream destroyed with work queued, whose handle the next stream gets."""
    for _ in range(2):
        assert call(lib, ctx, ONE) == OK
        lib.fake_new_stream(ONE)
    assert call(lib, ctx, ONE) == OK
    assert lib.fake_conflicts() == 0


def _uses():
    yield lambda lib, ctx, stream: attention(lib, ctx, stream, mask=True)
    yield lambda lib, ctx, stream: attention(lib, ctx, stream, mask=True, backward=True)
    yield lambda lib, ctx, stream: attention(lib, ctx, stream, tokens=2, keys=20000)
    yield lambda lib, ctx, stream: norm(lib, ctx, stream)
    yield lambda lib, ctx, stream: norm(lib, ctx, stream, backward=True)


@pytest.mark.parametrize("call", list(_uses()))
@pytest.mark.parametrize("fail", ["fake_fail_launch", "fake_fail_map", "fake_fail_number"])
def test_a_failed_call_leaves_its_mark(lib, ctx, call, fail):
    """A call that fails after some of its launches: what it launched is ordered before the next use."""
    assert call(lib, ctx, ONE) == OK
    failed = 0
    for n in range(1, 12):
        getattr(lib, fail)(n)
        rc = call(lib, ctx, ONE if n % 2 else TWO)
        getattr(lib, fail)(0)
        failed += rc != OK
        assert rc in (OK, CUDA) and (rc == OK or lib.gsr_last_error(ctx))
        assert call(lib, ctx, TWO if n % 2 else ONE) == OK
    assert lib.fake_conflicts() == 0
    if fail == "fake_fail_launch":
        assert failed >= 2


def rotary(lib, ctx, stream):
    from gaussian_splatting_tile_bin_gb300 import _abi
    desc = _abi.ROTARY.pack(2, 2, 200, 4, 64, 0, 1, 16, 0, 0, 0, 0, 0)
    return lib.gsr_rotary_forward(ctx, desc, _heads(200, 4), AT, AT, _heads(200, 4), stream)


def test_a_wait_that_ran_out_is_reported(lib, ctx):
    """By the next call of any decoder operator, or by gsr_synchronize; once."""
    lib.gsr_synchronize.argtypes = [ctypes.c_void_p] * 2
    assert lib.gsr_synchronize(None, None) == INVALID_ARG
    assert lib.gsr_synchronize(ctx, None) == OK      # nothing has run yet
    assert attention(lib, ctx, ONE) == OK
    for call in (lambda: lib.gsr_synchronize(ctx, ONE), lambda: attention(lib, ctx, ONE),
                 lambda: attention(lib, ctx, ONE, tokens=1), lambda: attention(lib, ctx, ONE, backward=True),
                 lambda: norm(lib, ctx, ONE), lambda: norm(lib, ctx, ONE, backward=True),
                 lambda: rotary(lib, ctx, ONE)):
        assert call() == OK
        lib.fake_set_status()
        launches = lib.fake_launches()
        assert call() == CUDA and b"gave up waiting" in lib.gsr_last_error(ctx)
        assert lib.fake_launches() == launches
        assert call() == OK
    lib.fake_set_status()                            # by the last call of a program
    assert lib.gsr_synchronize(ctx, ONE) == CUDA
    assert lib.gsr_synchronize(ctx, ONE) == OK


@pytest.mark.parametrize("call", [attention, norm])
def test_a_stream_whose_number_is_not_had(lib, ctx, call):
    """The call's own use is marked all the same, and the stream before it is not taken for its."""
    assert call(lib, ctx, ONE) == OK
    lib.fake_fail_number(2)              # asked before and after a call's launches
    assert call(lib, ctx, TWO) == CUDA
    assert call(lib, ctx, ONE) == OK
    assert lib.fake_conflicts() == 0
