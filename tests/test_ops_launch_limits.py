"""Sizes whose kernels could not be launched are argument errors, found before anything is
enqueued.  (No accepted call is made here: the addresses are not real.)"""
import pytest

from sharded_optimizer_step_zero_amd import ops

from test_ops_host import NORM, change, refused, xent_args


@pytest.mark.parametrize("rows, width", [(1 << 22, 16384), (1 << 22, 8200), (1 << 23, 4104), (0x7fffffff, 65536)])
def test_norm_of_too_many_workgroups(rows, width):
    """2^32 threads and more: 1024 a row above 8192 columns, 512 above 4096."""
    args = change(NORM, _1=width, _3=width, _6=width, _8=width, _12=rows, _13=width)
    assert "many rows" in refused(ops.zs_norm_forward, *args)


@pytest.mark.parametrize("tokens", [1 << 26, 0x7fffffff - 512])
def test_xent_of_too_many_tokens(tokens):
    """The statistics' join has 64 threads a token."""
    args = change(xent_args(0), _7=tokens, _13=1 << 60)
    assert "many rows" in refused(ops.zs_xent_forward, *args)
