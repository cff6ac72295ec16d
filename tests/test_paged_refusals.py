"""Argument checks of the paged cache's entry points (no GPU needed): each
refusal leaves before any launch."""
import ctypes as C

import pytest

from w4_weight_only_b200 import _abi, config

P = C.c_void_p


@pytest.fixture(scope="module")
def lib(built_lib):
    return _abi.lib()


def plan_args(**kw):
    a = dict(n_new=P(0x1000), lens=P(0x2000), state=P(0x3000), queue=P(0x10000), n_queue=64, table=P(0x20000), batch=4,
             width=8, page=16, prefix=0, lens_out=P(0x4000), state_out=P(0x5000), row_start=P(0x6000), slots=P(0x7000),
             pos=P(0x8000), max_rows=16, ws=P(0x9000), ws_bytes=256, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(n_new=None), "ARG"), (dict(state=None), "ARG"), (dict(slots=None), "ARG"), (dict(ws=None), "ARG"),
    (dict(batch=0), "SHAPE"), (dict(batch=4097), "SHAPE"), (dict(width=0), "SHAPE"), (dict(prefix=-1), "SHAPE"),
    (dict(max_rows=-1), "SHAPE"), (dict(max_rows=(1 << 30) + 1), "SHAPE"), (dict(page=8), "SHAPE"), (dict(page=48), "SHAPE"), (dict(page=512), "SHAPE"),
    (dict(n_queue=0), "SHAPE"), (dict(n_queue=1 << 27, page=16), "SHAPE"), (dict(ws=P(0x9008)), "ALIGN"),
    (dict(ws_bytes=255), "WORKSPACE"),
    (dict(lens_out=P(0x2000)), "ARG"), (dict(state_out=P(0x3004)), "ARG"), (dict(slots=P(0x8000)), "ARG"),
    (dict(table=P(0x10000)), "ARG")])
def test_plan_refusals(lib, kw, code):
    assert lib.w4a_paged_plan(*plan_args(**kw)) == getattr(_abi, "ERR_" + code)


def prep_args(c, **kw):
    a = dict(cfg=C.byref(c), full=1, qkv=P(0x1000), ld=768, rows=2, qg=P(0x1000), kg=P(0x1000), pos=P(0x1000),
             slots=P(0x1000), q=P(0x1000), k=P(0x1000), v=P(0x1000), n_pages=4, page=16, ws=P(0x1000), ws_bytes=256,
             stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(cfg=None), "ARG"), (dict(qkv=None), "ARG"), (dict(k=None), "ARG"), (dict(rows=0), "SHAPE"),
    (dict(ld=764), "SHAPE"), (dict(ld=770), "SHAPE"), (dict(page=17), "SHAPE"), (dict(n_pages=0), "SHAPE"),
    (dict(qkv=P(0x1004)), "ALIGN"), (dict(q=P(0x1002)), "ALIGN"), (dict(v=P(0x1008)), "ALIGN"),
    (dict(ws_bytes=0), "WORKSPACE"), (dict(rows=(1 << 30) + 1), "SHAPE")])
def test_prep_refusals(lib, kw, code):
    assert lib.w4a_qk_prep_paged(*prep_args(config.tiny().to_c(), **kw)) == getattr(_abi, "ERR_" + code)


@pytest.mark.parametrize("nq,nkv,hd,code", [(8, 2, 96, "UNSUPPORTED"), (8, 3, 64, "SHAPE"), (34, 2, 64, "SHAPE"),
                                            (0, 1, 64, "SHAPE"), (512, 32, 128, "SHAPE")])
def test_prep_head_refusals(lib, nq, nkv, hd, code):
    c = config.tiny()
    c.n_heads, c.n_kv_heads, c.head_dim = nq, nkv, hd
    assert lib.w4a_qk_prep_paged(*prep_args(c.to_c(), ld=1 << 20)) == getattr(_abi, "ERR_" + code)


def attn_args(**kw):
    a = dict(q=P(0x100000), rows=2, batch=2, nq=8, nkv=2, hd=64, k=P(0x1000), v=P(0x1000), n_pages=4, page=16,
             row_start=P(0x1000), lens=P(0x1000), table=P(0x1000), width=2, ptab=P(0x1000), P_=5, window=0, max_new=1,
             out=P(0x200000), ws=P(0x1000), ws_bytes=0, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), "ARG"), (dict(lens=None), "ARG"), (dict(ptab=None), "ARG"), (dict(rows=0), "SHAPE"),
    (dict(rows=(1 << 20) + 1), "SHAPE"), (dict(batch=0), "SHAPE"), (dict(nq=34), "SHAPE"), (dict(hd=32), "UNSUPPORTED"),
    (dict(page=24), "SHAPE"), (dict(P_=-1), "SHAPE"), (dict(window=-1), "SHAPE"), (dict(max_new=0), "SHAPE"),
    (dict(width=0), "SHAPE"), (dict(width=1 << 26), "SHAPE"), (dict(width=1 << 25, batch=128), "SHAPE"), (dict(k=P(0x1008)), "ALIGN"), (dict(out=P(0x100000)), "ARG")])
def test_attn_refusals(lib, kw, code):
    assert lib.w4a_attn_shared(*attn_args(**kw)) == getattr(_abi, "ERR_" + code)


def test_attn_refuses_tables_that_fit_only_without_the_prefix(lib):
    """4,096 tables of 8,182 pages of 64 over 64 KV heads: 2^31 tiles of 64 keys
    with a prefix of 4,096 ahead of each."""
    big = dict(batch=4096, nq=64, nkv=64, page=64, width=8182, rows=1 << 20)
    assert lib.w4a_attn_shared(*attn_args(**big, P_=4096)) == _abi.ERR_SHAPE


def test_sizes(lib):
    out = C.c_size_t(0)
    c = config.tiny().to_c()
    assert lib.w4a_paged_kv_bytes(C.byref(c), 10, 32, C.byref(out)) == 0 and out.value == 4 * 2 * 10 * 2 * 32 * 64 * 2
    k, v = C.c_size_t(0), C.c_size_t(0)
    assert lib.w4a_paged_kv_layer(C.byref(c), 10, 32, 3, C.byref(k), C.byref(v)) == 0
    one = 10 * 2 * 32 * 64 * 2
    assert (k.value, v.value) == (6 * one, 7 * one)
    assert lib.w4a_paged_kv_layer(C.byref(c), 10, 32, 4, C.byref(k), C.byref(v)) == _abi.ERR_ARG
    assert lib.w4a_paged_kv_bytes(C.byref(c), 10, 20, C.byref(out)) == _abi.ERR_SHAPE
    assert lib.w4a_paged_kv_bytes(C.byref(c), 1 << 30, 16, C.byref(out)) == _abi.ERR_SHAPE
    assert lib.w4a_attn_shared_workspace_bytes(16, 16, 40, 8, 128, 1, C.byref(out)) == 0 and out.value >= 256
    assert lib.w4a_attn_shared_workspace_bytes(16, 16, 40, 7, 128, 1, C.byref(out)) == _abi.ERR_SHAPE
