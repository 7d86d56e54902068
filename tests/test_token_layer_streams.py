"""The token layers' host code on the CPU, against the runtime that runs nothing: how
their uses of the workspace are ordered beside the other decoder operators', what a failed
call leaves, and where a wait that ran out is reported."""
import ctypes

import pytest

from test_decoder_streams import AT, CUDA, INVALID_ARG, OK, ONE, THREE, TWO, attention, ctx, lib  # noqa: F401


@pytest.fixture(autouse=True)
def _signatures(lib):  # noqa: F811
    for name, pointers in (("layer_norm_forward", 11), ("layer_norm_backward", 12), ("gated_recurrence_forward", 10),
                           ("gated_recurrence_backward", 13)):
        getattr(lib, "gsr_" + name).argtypes = [ctypes.c_void_p] * pointers
    lib.gsr_synchronize.argtypes = [ctypes.c_void_p] * 2


def _rows(tokens, channels, at=AT):
    from gaussian_splatting_tile_bin_gb300 import _abi
    return _abi.HEADS.pack(at, tokens * channels, channels, 0)


def norm(lib, ctx, stream, channels=256, tokens=500, backward=False):  # noqa: F811
    from gaussian_splatting_tile_bin_gb300 import _abi
    desc, x, y = _abi.LAYER_NORM.pack(1, 2, tokens, 1, channels, 1e-5), _rows(tokens, channels), _rows(tokens, channels, 2 * AT)
    if backward:
        return lib.gsr_layer_norm_backward(ctx, desc, x, x, AT, AT, AT, x, x, AT, AT, stream)
    return lib.gsr_layer_norm_forward(ctx, desc, x, x, AT, AT, x, y, AT, AT, stream)


def recurrence(lib, ctx, stream, tokens=1000, channels=256, backward=False):  # noqa: F811
    from gaussian_splatting_tile_bin_gb300 import _abi
    desc, x = _abi.RECURRENCE.pack(1, 2, tokens, channels, 1, 0), _rows(tokens, channels)
    if backward:
        return lib.gsr_gated_recurrence_backward(ctx, desc, x, x, x, x, AT, AT, x, x, x, AT, stream)
    return lib.gsr_gated_recurrence_forward(ctx, desc, x, x, x, AT, x, AT, AT, stream)


def _uses():
    yield lambda lib, ctx, stream: norm(lib, ctx, stream, backward=True)
    yield lambda lib, ctx, stream: recurrence(lib, ctx, stream)
    yield lambda lib, ctx, stream: recurrence(lib, ctx, stream, backward=True)


def test_streams_are_ordered(lib, ctx):  # noqa: F811
    for stream in (ONE, TWO, ONE, THREE, TWO):
        assert attention(lib, ctx, stream) == OK
        assert norm(lib, ctx, stream) == OK
        for use in _uses():
            assert use(lib, ctx, stream) == OK
    assert lib.fake_conflicts() == 0 and lib.fake_launches() > 20


@pytest.mark.parametrize("call", list(_uses()))
def test_streams_of_one_capture_are_ordered(lib, ctx, call):  # noqa: F811
    for stream in (ONE, TWO):
        assert call(lib, ctx, stream) == OK
    for _ in range(2):
        lib.fake_begin_capture(ONE)
        assert lib.fake_edge(ONE, TWO) == OK and lib.fake_edge(ONE, THREE) == OK
        for stream in (ONE, TWO, THREE, ONE, TWO):
            assert call(lib, ctx, stream) == OK
        assert lib.fake_edge(TWO, ONE) == OK and lib.fake_edge(THREE, ONE) == OK
        lib.fake_end_capture(ONE)
        assert call(lib, ctx, TWO) == OK and call(lib, ctx, ONE) == OK
    assert lib.fake_conflicts() == 0 and lib.fake_pulled_in() == 0


@pytest.mark.parametrize("call", list(_uses()))
@pytest.mark.parametrize("fail", ["fake_fail_launch", "fake_fail_map", "fake_fail_number"])
def test_a_failed_call_leaves_its_mark(lib, ctx, call, fail):  # noqa: F811
    assert call(lib, ctx, ONE) == OK
    failed = 0
    for n in range(1, 8):
        getattr(lib, fail)(n)
        rc = call(lib, ctx, ONE if n % 2 else TWO)
        getattr(lib, fail)(0)
        failed += rc != OK
        assert rc in (OK, CUDA) and (rc == OK or lib.gsr_last_error(ctx))
        assert call(lib, ctx, TWO if n % 2 else ONE) == OK
    assert lib.fake_conflicts() == 0
    if fail == "fake_fail_launch":
        assert failed >= 2


def test_growth_during_a_capture_is_refused_and_kept_behind_it(lib, ctx):  # noqa: F811
    assert recurrence(lib, ctx, ONE) == OK
    lib.fake_begin_capture(ONE)
    assert recurrence(lib, ctx, ONE) == OK
    assert recurrence(lib, ctx, ONE, tokens=1 << 20) == CUDA and b"capture" in lib.gsr_last_error(ctx)
    lib.fake_end_capture(ONE)
    assert recurrence(lib, ctx, ONE, tokens=1 << 20) == OK
    assert lib.fake_freed_while_held() == 0 and lib.fake_allocations() == 2
    lib.gsr_destroy(ctx)
    assert lib.fake_live() == 0


def test_few_tokens_and_forward_norms_take_no_workspace(lib, ctx):  # noqa: F811
    for stream in (ONE, TWO):
        assert norm(lib, ctx, stream) == OK and recurrence(lib, ctx, stream, tokens=1) == OK
    assert lib.fake_allocations() == 0 and lib.fake_launches() == 4


def test_rows_of_two_blocks_have_a_status_word(lib, ctx):  # noqa: F811
    """Rows that two blocks share wait for each other: forward, and without gradients of parameters,
    too the word that reports a wait is made, before a capture."""
    from gaussian_splatting_tile_bin_gb300 import _abi
    x = _rows(40, 9000)
    call = lambda: lib.gsr_layer_norm_backward(ctx, _abi.LAYER_NORM.pack(1, 2, 40, 1, 9000, 1e-5), x, x, AT, AT, AT, x, x,  # noqa: E731
                                               None, None, ONE)
    assert norm(lib, ctx, ONE, 256) == OK
    launches = lib.fake_launches()
    lib.fake_begin_capture(ONE)
    for use in (call, lambda: norm(lib, ctx, ONE, 9000)):
        assert use() == CUDA and b"capture" in lib.gsr_last_error(ctx) and lib.fake_launches() == launches
    lib.fake_end_capture(ONE)
    assert call() == OK and norm(lib, ctx, ONE, 9000) == OK and lib.fake_launches() == launches + 2
    lib.fake_begin_capture(ONE)
    assert call() == OK and norm(lib, ctx, ONE, 9000) == OK
    lib.fake_end_capture(ONE)
    lib.fake_set_status()
    assert norm(lib, ctx, ONE, 9000) == CUDA and b"gave up waiting" in lib.gsr_last_error(ctx)
    for stream in (ONE, TWO, THREE, ONE):
        assert norm(lib, ctx, stream, 9000, backward=True) == OK
    assert lib.fake_conflicts() == 0


def test_a_wait_that_ran_out_is_reported(lib, ctx):  # noqa: F811
    assert recurrence(lib, ctx, ONE) == OK
    for call in (lambda: norm(lib, ctx, ONE), lambda: norm(lib, ctx, ONE, backward=True), lambda: recurrence(lib, ctx, ONE),
                 lambda: recurrence(lib, ctx, ONE, tokens=1), lambda: recurrence(lib, ctx, ONE, backward=True)):
        assert call() == OK
        lib.fake_set_status()
        launches = lib.fake_launches()
        assert call() == CUDA and b"gave up waiting" in lib.gsr_last_error(ctx)
        assert lib.fake_launches() == launches
        assert call() == OK
    lib.fake_set_status()
    assert lib.gsr_synchronize(ctx, ONE) == CUDA and lib.gsr_synchronize(ctx, ONE) == OK


@pytest.mark.parametrize("sizes", [(1, -1, 1, 1, 8), (1, 1, 1, -1, 8), (1, 1, 1, 1, 0), (1, 1, 1, 1, 16385), (3, 1, 1, 1, 8),
                                   (1, 1, 1, 1025, 8), (1, 1 << 14, 1 << 15, 1, 8), (1, 1 << 13, 1 << 13, 32, 8)])
def test_layer_norm_sizes_are_refused(lib, ctx, sizes):  # noqa: F811
    from gaussian_splatting_tile_bin_gb300 import _abi
    x, y, desc = _rows(4, 8), _rows(4, 8, 2 * AT), _abi.LAYER_NORM.pack(*sizes, 1e-5)
    launches = lib.fake_launches()
    assert lib.gsr_layer_norm_forward(ctx, desc, x, x, AT, AT, x, y, AT, AT, ONE) == INVALID_ARG
    assert lib.gsr_layer_norm_backward(ctx, desc, x, x, AT, AT, AT, x, x, AT, AT, ONE) == INVALID_ARG
    assert lib.fake_launches() == launches


def test_layer_norm_arrays_are_refused(lib, ctx):  # noqa: F811
    from gaussian_splatting_tile_bin_gb300 import _abi
    x, y, odd = _rows(4, 8), _rows(4, 8, 2 * AT), _rows(4, 8, AT + 1)
    negative, shared = _abi.HEADS.pack(AT, 32, -8, 0), _abi.HEADS.pack(AT, 0, 8, 0)
    good = [_abi.LAYER_NORM.pack(1, 2, 4, 1, 8, 1e-5), x, x, AT, AT, x, y, AT, AT]
    assert lib.gsr_layer_norm_forward(ctx, *good, ONE) == OK
    for i, bad in ((0, None), (1, None), (1, odd), (1, negative), (2, None), (2, odd), (3, AT + 2), (4, AT + 2), (5, None),
                   (5, shared), (6, None), (6, x), (6, shared), (7, None), (8, None), (8, AT + 1)):
        args = list(good)
        args[i] = bad
        assert lib.gsr_layer_norm_forward(ctx, *args, ONE) == INVALID_ARG, i
        assert lib.gsr_last_error(ctx)
    assert lib.gsr_layer_norm_forward(ctx, *[shared if i == 2 else v for i, v in enumerate(good)], ONE) == OK
    good = [good[0], x, x, AT, AT, AT, x, y, AT, AT]
    assert lib.gsr_layer_norm_backward(ctx, *good, ONE) == OK
    for i, bad in ((0, None), (1, None), (2, odd), (4, None), (5, AT + 1), (6, odd), (7, None), (7, shared), (8, AT + 1)):
        args = list(good)
        args[i] = bad
        assert lib.gsr_layer_norm_backward(ctx, *args, ONE) == INVALID_ARG, i


@pytest.mark.parametrize("sizes", [(1, -1, 4, 8), (1, 1, -4, 8), (1, 1, 4, 0), (1, 1, 4, 65537), (3, 1, 4, 8),
                                   (1, 65537, 1, 8), (1, 1, (1 << 24) + 1, 8), (1, 1 << 14, 1 << 15, 8),
                                   (1, 65536, 4096, 65536)])
def test_recurrence_sizes_are_refused(lib, ctx, sizes):  # noqa: F811
    from gaussian_splatting_tile_bin_gb300 import _abi
    x, desc = _rows(4, 8), _abi.RECURRENCE.pack(*sizes, 0, 0)
    launches = lib.fake_launches()
    assert lib.gsr_gated_recurrence_forward(ctx, desc, x, x, x, AT, x, AT, AT, ONE) == INVALID_ARG
    assert lib.gsr_gated_recurrence_backward(ctx, desc, x, x, x, x, AT, AT, x, x, x, AT, ONE) == INVALID_ARG
    assert lib.fake_launches() == launches


def test_recurrence_arrays_are_refused(lib, ctx):  # noqa: F811
    from gaussian_splatting_tile_bin_gb300 import _abi
    x, odd = _rows(400, 8), _rows(400, 8, AT + 1)
    shared, far = _abi.HEADS.pack(AT, 0, 8, 0), _abi.HEADS.pack(AT, 1 << 38, 1 << 31, 0)
    good = [_abi.RECURRENCE.pack(1, 2, 400, 8, 0, 0), x, x, x, AT, x, AT, AT]
    assert lib.gsr_gated_recurrence_forward(ctx, *good, ONE) == OK
    for i, bad in ((0, None), (0, _abi.RECURRENCE.pack(1, 2, 400, 8, 0, AT + 2)), (1, None), (1, odd), (1, far), (2, None),
                   (2, odd), (3, odd), (4, AT + 2), (5, None), (5, shared), (6, None), (6, AT + 1), (7, AT + 2)):
        args = list(good)
        args[i] = bad
        assert lib.gsr_gated_recurrence_forward(ctx, *args, ONE) == INVALID_ARG, i
        assert lib.gsr_last_error(ctx)
    for i, fine in ((1, shared), (3, None), (4, None), (7, None)):
        assert lib.gsr_gated_recurrence_forward(ctx, *[fine if k == i else v for k, v in enumerate(good)], ONE) == OK
    good = [good[0], x, x, x, x, AT, AT, x, x, x, AT]
    assert lib.gsr_gated_recurrence_backward(ctx, *good, ONE) == OK
    for i, bad in ((0, None), (1, None), (2, odd), (3, None), (4, None), (4, odd), (5, None), (5, AT + 1), (6, AT + 1), (7, None),
                   (7, shared), (8, None), (9, None), (9, shared), (10, AT + 2)):
        args = list(good)
        args[i] = bad
        assert lib.gsr_gated_recurrence_backward(ctx, *args, ONE) == INVALID_ARG, i
