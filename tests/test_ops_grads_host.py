"""Host-only checks of clipping by a given sum of squares: the norm does not go where it is read."""
import pytest

from sharded_optimizer_step_zero_amd import ops
from test_ops_host import P, refused


@pytest.mark.parametrize("table, pieces", [(P, 1), (P, 100000), (0, 0)])
def test_the_norm_does_not_go_where_the_sum_of_squares_is(table, pieces):
    assert "same" in refused(ops.zs_grads_clip, table, pieces, 1.0, 3 * P, 3 * P, 0, 0, 0)
