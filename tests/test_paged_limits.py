"""Limits of the paged cache's entry points at their edges (no GPU needed): the
last size that is taken and the first that is not."""
import pytest

from test_paged_refusals import P, attn_args, lib, prep_args  # noqa: F401
from w4_weight_only_b200 import _abi, config


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


PAGES = 4 * 2 * 16 * 64 * 2  # bytes of K (or V): 4 pages of 16 rows, 2 KV heads of 64


@pytest.mark.parametrize("kw", [
    dict(q=P(0x100000 + 3 * 800 * 4 + 768 * 4 - 16)),          # the last row's end
    dict(q=P(0x100000 - 4 * 8 * 64 * 2 + 16)),                 # q_out ends in the first row
    dict(k=P(0x300000 + PAGES - 16)), dict(k=P(0x300000)),     # K and V
    dict(k=P(0x100000 + 16)), dict(v=P(0x200000)), dict(v=P(0x400000)), dict(k=P(0x410000))])
def test_prep_overlaps(lib, kw):
    """qkv: 4 rows of 768 floats, 800 apart; an output on an input or on another output."""
    a = dict(qkv=P(0x100000), ld=800, rows=4, q=P(0x200000), k=P(0x280000), v=P(0x300000), qg=P(0x400000), kg=P(0x410000),
             pos=P(0x420000), slots=P(0x430000), ws=P(0x440000), ws_bytes=256)
    a.update(kw)
    assert lib.w4a_qk_prep_paged(*prep_args(config.tiny().to_c(), **a)) == _abi.ERR_ARG
