"""Lanes of the recurrence's working warps that come apart, where only those with a channel
store, are together again before the warp's next instruction on tensor memory."""
import pytest

from test_gpu_token_layers import _held_up, gsr  # noqa: F401

pytestmark = pytest.mark.gpu


def test_lanes_that_are_held_up_change_no_bit(gsr, tmp_path):  # noqa: F811
    _held_up(tmp_path, "recurrence.cu", "recurrence_lanes_run")
