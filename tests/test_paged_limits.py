"""Limits of the paged cache's entry points at their edges (no GPU needed): the
last size that is taken and the first that is not."""
import pytest

from test_paged_refusals import attn_args, lib  # noqa: F401
from w4_weight_only_b200 import _abi


def test_prefix_below_2_30(lib):
    """Positions are prefix + own, each below 2^30."""
    assert lib.w4a_attn_shared(*attn_args(P_=1 << 30)) == _abi.ERR_SHAPE
    assert lib.w4a_attn_shared(*attn_args(P_=(1 << 30) - 1)) != _abi.ERR_SHAPE


def test_table_below_2_30(lib):
    assert lib.w4a_attn_shared(*attn_args(width=1 << 26, batch=1)) == _abi.ERR_SHAPE
    assert lib.w4a_attn_shared(*attn_args(width=(1 << 26) - 1, batch=1)) != _abi.ERR_SHAPE


@pytest.mark.parametrize("prefix,fits", [(0, True), (4096, False)])
def test_tables_that_fit_only_without_the_prefix(lib, prefix, fits):
    """4,096 tables of 8,170 pages of 64 over 64 KV heads: 2,144,338,432 tiles of
    64 keys (with ten a table besides) by themselves, 2,161,119,744 with a
    prefix of 4,096 read ahead of each; 2^31 - 1 is the most."""
    big = dict(batch=4096, nq=64, nkv=64, page=64, width=8170, rows=1 << 20)
    assert (lib.w4a_attn_shared(*attn_args(**big, P_=prefix)) != _abi.ERR_SHAPE) == fits
