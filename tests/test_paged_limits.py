"""Limits of the paged cache's entry points at their edges (no GPU needed): the
last size that is taken and the first that is not."""
from test_paged_refusals import attn_args, lib  # noqa: F401
from w4_weight_only_b200 import _abi


def test_prefix_below_2_30(lib):
    """Positions are prefix + own, each below 2^30."""
    assert lib.w4a_attn_shared(*attn_args(P_=1 << 30)) == _abi.ERR_SHAPE
    assert lib.w4a_attn_shared(*attn_args(P_=(1 << 30) - 1)) != _abi.ERR_SHAPE
