"""Warps of a block that share a row of the layer norm, and hand each other their sums through two
copies in turn, give the same bits when they are held up."""
import pytest

from test_gpu_token_layers import _held_up, gsr  # noqa: F401

pytestmark = pytest.mark.gpu


def test_warps_of_a_team_are_held_up(gsr, tmp_path):  # noqa: F811
    _held_up(tmp_path, "layernorm.cu", "layer_norm_teams_run")
