"""The gated recurrence's gradients where a gate shuts something out: states, values and gradients
orders of magnitude apart, within bounds that are relative to each gate."""
import pytest

from test_gpu_gated_recurrence import BF16, F16, F32, _run, ctx, gsr  # noqa: F401
from test_gpu_recurrence_gates import _inputs, _single_steps
import recurrence_gate_reference as ref

pytestmark = pytest.mark.gpu


def _compare(gsr, ctx, t, lengths=None, reverse=False):  # noqa: F811
    b, n, _ = t["x"].shape
    wide = {k: None if v is None else v.double() for k, v in t.items()}
    want = ref.recurrence(wide["x"], wide["forget"], wide["gate"], wide["initial"], lengths or [n] * b, reverse, t["x"].dtype,
                          dout=wide["dout"], dfinal=wide["dfinal"])
    got = _run(gsr, ctx, t, lengths, reverse)
    for name, value in want.items():
        ref.check(got[name], value, name)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("n", [1, 2, 8, 9, 63, 64, 65, 130, 600])
def test_open_and_shut_gates(gsr, ctx, dtype, reverse, n):  # noqa: F811
    for c, gate in ((40, True), (66, True), (33, True), (64, False)):
        _compare(gsr, ctx, _inputs(2, n, c, dtype, 200 * n + c, gate), [n, max(n - 7, 0)], reverse)


@pytest.mark.parametrize("n", [1, 8, 17, 65, 140])
@pytest.mark.parametrize("last", [False, True])
def test_single_steps(gsr, ctx, n, last):  # noqa: F811
    """Among them a state of 0 or next to nothing that an open gate keeps from a large value."""
    _compare(gsr, ctx, _single_steps(n, last))
