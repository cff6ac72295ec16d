"""The paged KV cache against the float64 oracle: plans (exact), QK-norm /
rotation / append, attention behind a shared prefix, and the three together.

Tolerances.  A bf16 rounding is off by at most 2^-8 of its value.
prep: one rounding of the result; before it fp32 arithmetic (about ten
roundings of 2^-24, a sum of squares of up to 5,120 terms in a tree of depth
< 40, an angle reduced in fp64 and rounded to fp32 at |angle| <= pi) stays
below 2^-18 of |x1| + |x2|.
attention: one rounding of the result and one of each softmax weight (2^-8 of
sum p|v| at most); fp32 scores of |s| < 2^5 are off by < hd 2^-24 sum|q k| /
sqrt(hd) < 2^-12, which moves a weight by less than 2^-11 of itself.
"""
import numpy as np
import pytest
import torch

from oracle import paged as op
from w4_weight_only_b200 import config as wc
from helpers import np64, oracle_config

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api(built_lib, cuda):
    from w4_weight_only_b200 import api
    return api


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ---------------------------------------------------------------------------
# plans
# ---------------------------------------------------------------------------
def plan_case(seed, batch, page, max_len, max_new, ended=0.1, spare=0):
    """Lengths, new tokens, a shuffled free queue that wraps, tables."""
    rng = np.random.default_rng(seed)
    lens = [int(x) for x in rng.integers(0, max_len + 1, batch)]
    new = [-1 if rng.random() < ended else int(rng.integers(0, max_new + 1)) for _ in range(batch)]
    held = [-(-n // page) for n in lens]
    take = sum(-(-(n + max(k, 0)) // page) - h for n, k, h in zip(lens, new, held) if k >= 0)
    freed = sum(h for h, k in zip(held, new) if k < 0)
    N = max(1, sum(held) + max(0, take - freed) + spare)
    ids = [int(x) for x in rng.permutation(N)]
    width = max(1, max(-(-(n + max(k, 0)) // page) for n, k in zip(lens, new)))
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-7] * (width - h))
        at += h
    head = int(rng.integers(0, N))
    queue = [-9] * N
    for i, p in enumerate(ids[at:]):
        queue[(head + i) % N] = p
    return new, lens, [head, N - at], queue, table


def run_plan(api, new, lens, state, queue, table, page, prefix, max_rows, ws=None):
    t, q = i32(table), i32(queue)
    p = api.paged_plan(i32(new), i32(lens), i32(state), q, t, page, max_rows, prefix_len=prefix, ws=ws)
    return [x.tolist() for x in (p.lens, p.state, p.row_start, p.slots, p.pos, t, q)]


@pytest.mark.parametrize("seed,batch,page,max_len,max_new,spare,pad", [
    (0, 1, 16, 0, 1, 0, 0), (1, 1, 64, 100, 1, 0, 3), (2, 16, 64, 500, 1, 5, 0), (3, 33, 16, 70, 9, 0, 1),
    (4, 511, 32, 90, 40, 0, 100), (5, 513, 16, 40, 2, 3, 0), (6, 4096, 16, 64, 3, 0, 17), (7, 5, 256, 1000, 9000, 0, 0),
    (8, 64, 128, 300, 700, 0, 5000)])
def test_plan_equals_oracle(api, seed, batch, page, max_len, max_new, spare, pad):
    """Pages just suffice (spare = 0: those freed by the same call are taken too)."""
    case = plan_case(seed, batch, page, max_len, max_new, spare=spare)
    rows = sum(max(k, 0) for k in case[0]) + pad
    ref = op.plan(*case, page, 777, rows)
    ws = api.zeros_workspace(256)
    got = run_plan(api, *case, page, 777, rows, ws)
    api.check(ws)
    for name, a, b in zip(("lens", "state", "row_start", "slots", "pos", "table", "queue"), got, ref):
        assert a == list(b), name


def test_plan_all_or_nothing(api):
    """Too few pages, rows or columns, or a count out of range: nothing changes and the check reports it."""
    from w4_weight_only_b200 import _abi
    page = 16
    new, lens, state, queue, table = plan_case(11, 40, page, 100, 30)
    rows = sum(max(k, 0) for k in new)

    def fails(msg, n=new, l=lens, s=state, r=rows, t=table):
        ws = api.zeros_workspace(256)
        got = run_plan(api, n, l, s, queue, t, page, 0, r, ws)
        assert got[0] == l and got[1] == s and got[2] == [0] * 41 and got[3] == [-1] * r == got[4], msg
        assert got[5] == t and got[6] == queue, msg
        with pytest.raises(_abi.W4AError) as e:
            api.check(ws)
        assert e.value.code == _abi.ERR_KERNEL, msg

    fails("rows", r=rows - 1)
    fails("pages", s=[state[0], state[1] - 1])
    fails("width", t=[r[:-1] for r in table])
    fails("n_new", n=[-2] + new[1:])
    fails("lens", l=[-1] + lens[1:])
    fails("head", s=[len(queue), 1])
    fails("count", s=[0, len(queue) + 1])


def test_plan_of_nothing(api):
    """No new tokens, no rows; and a step that only ends sequences."""
    assert run_plan(api, [0, 0], [5, 0], [1, 1], [9, 2, 9], [[0], [1]], 16, 3, 0)[:3] == [[5, 0], [1, 1], [0, 0, 0]]
    got = run_plan(api, [-1, 0], [5, 17], [1, 0], [9, 9, 9], [[0, 9], [1, 2]], 16, 3, 2)
    assert got == [[0, 17], [1, 1], [0, 0, 0], [-1, -1], [-1, -1], [[0, 9], [1, 2]], [9, 0, 9]]


# ---------------------------------------------------------------------------
# QK-norm, rotation, append
# ---------------------------------------------------------------------------
def shape_config(nq, nkv, hd):
    return wc.Config(d_model=512, n_layers=4, n_heads=nq, n_kv_heads=nkv, head_dim=hd, ffn=512, vocab=16, window=64)


@pytest.mark.parametrize("nq,nkv,hd,page,rows,full,start", [
    (8, 2, 64, 16, 1, True, 0), (8, 2, 64, 16, 37, False, 5), (40, 8, 128, 64, 3, True, 131071),
    (40, 8, 128, 128, 65, False, 4000), (16, 1, 128, 32, 9, True, 70), (4, 4, 64, 256, 130, True, 1 << 20),
    (128, 16, 128, 16, 2, False, 9)])
def test_prep_against_oracle(api, nq, nkv, hd, page, rows, full, start):
    cfg = shape_config(nq, nkv, hd)
    g = gen(rows)
    width, pad = cfg.qkv_dim, 3
    wide = torch.randn((rows + pad, width + 8), generator=g, device="cuda") * 3  # strided rows
    y = wide[:, :width]
    if rows > 2:
        y[1] *= 1e-4   # the norm's eps counts
        y[2] = 0.0
    qg = 1 + 0.2 * torch.randn(nq * hd, generator=g, device="cuda")
    kg = 1 + 0.2 * torch.randn(nkv * hd, generator=g, device="cuda")
    n_pages = -(-rows // page) + 2
    slots = [int(x) for x in np.random.default_rng(rows).permutation(n_pages * page)[:rows]]
    at = i32(slots)
    live = list(range(rows + pad))
    slots, pos = slots + [-1] * pad, [start + i for i in range(rows)] + [-1] * pad
    if rows > 5:
        slots[4] = -1  # a hole
        live.remove(4)
    live = [r for r in live if r < rows]
    k = torch.full((n_pages, nkv, page, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    v, q = torch.full_like(k, 5.0), torch.full((rows + pad, nq, hd), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = api.zeros_workspace(256)
    api.qk_prep_paged(cfg, full, y, qg, kg, i32(pos), i32(slots), k, v, ws=ws, q_out=q)
    api.check(ws)
    rq, rk, rv, qs, ks = op.prep(oracle_config(cfg), np64(y), np64(qg), np64(kg), np.maximum(pos, 0), full)
    flat = lambda t: np64(t).transpose(0, 2, 1, 3).reshape(-1, nkv, hd)
    K, V, Q = flat(k), flat(v), np64(q)
    s = [slots[r] for r in live]
    assert np.all(np.abs(Q[live] - rq[live]) <= 2.0 ** -8 * np.abs(rq[live]) + 2.0 ** -18 * qs[live])
    assert np.all(np.abs(K[s] - rk[live]) <= 2.0 ** -8 * np.abs(rk[live]) + 2.0 ** -18 * ks[live])
    assert np.array_equal(V[s], np64(torch.from_numpy(rv[live]).to(torch.bfloat16)))
    rest = np.setdiff1d(np.arange(n_pages * page), s)
    dead = np.setdiff1d(np.arange(rows + pad), live)
    assert np.all(K[rest] == 7) and np.all(V[rest] == 5) and np.all(Q[dead] == 3)  # left as they were


def test_prep_reports_bad_slots(api):
    """A slot outside the cache or a negative position: skipped, reported."""
    from w4_weight_only_b200 import _abi
    cfg = shape_config(8, 2, 64)
    for slot, pos in ((64, 0), (-2, 0), (3, -1), (2 ** 31 - 1, 0)):
        k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
        v, q = torch.zeros_like(k), torch.zeros((2, 8, 64), dtype=torch.bfloat16, device="cuda")
        ws = api.zeros_workspace(256)
        y = torch.ones((2, cfg.qkv_dim), device="cuda")
        api.qk_prep_paged(cfg, True, y, torch.ones(512, device="cuda"), torch.ones(128, device="cuda"), i32([pos, 1]),
                          i32([slot, 5]), k, v, ws=ws, q_out=q)
        with pytest.raises(_abi.W4AError) as e:
            api.check(ws)
        assert e.value.code == _abi.ERR_KERNEL
        assert not q[0].any() and q[1].all() and int((v != 0).sum()) == 2 * 64


# ---------------------------------------------------------------------------
# attention behind a shared prefix
# ---------------------------------------------------------------------------
def attn_case(seed, nq, nkv, hd, page, P, lens, new, pad=0, junk=None, q_scale=1.5):
    """Pages in random order; rows of pages that no sequence holds are junk."""
    rng, g = np.random.default_rng(seed), gen(seed)
    np_, held = -(-P // page), [-(-n // page) for n in lens]
    n_pages = np_ + sum(held) + 2
    ids = [int(x) for x in rng.permutation(n_pages)]
    ptab, at, width = ids[:np_], np_, max(1, max(held)) + 1
    table = []
    for h in held:
        table.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    k = torch.randn((n_pages, nkv, page, hd), generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn((n_pages, nkv, page, hd), generator=g, device="cuda").to(torch.bfloat16)
    if junk is not None:
        for p in ids[at:]:
            k[p], v[p] = junk, junk
        if P % page:
            k[ptab[-1], :, P % page:], v[ptab[-1], :, P % page:] = junk, junk
        for b, n in enumerate(lens):
            if n % page:
                k[table[b][n // page], :, n % page:], v[table[b][n // page], :, n % page:] = junk, junk
    start = np.concatenate([[0], np.cumsum(new)]).tolist()
    q = (torch.randn((start[-1] + pad, nq, hd), generator=g, device="cuda") * q_scale).to(torch.bfloat16)
    return dict(q=q, k=k, v=v, start=start, lens=lens, table=table, ptab=ptab, P=P)


def run_attn(api, c, window=0, max_new=None, out=None, ws=None):
    mn = max_new or max(1, max(b - a for a, b in zip(c["start"], c["start"][1:])))
    if ws is None:
        ws = api.attn_shared_workspace(c["q"].shape[0], len(c["lens"]), c["q"].shape[1], c["k"].shape[1],
                                       c["q"].shape[2], mn)
    out = api.attn_shared(c["q"], c["k"], c["v"], i32(c["start"]), i32(c["lens"]), i32(c["table"]),
                          i32(c["ptab"]) if c["P"] else None, c["P"], window=window, max_new=mn, ws=ws, out=out)
    api.check(ws)
    return out


def close(c, out, window):
    ref, size = op.attend(np64(c["q"]), np64(c["k"]), np64(c["v"]), c["start"], c["lens"], c["table"], c["ptab"],
                          c["P"], window)
    n = c["start"][-1]
    err = np.abs(np64(out)[:n] - ref[:n]) - (2.0 ** -8 * np.abs(ref[:n]) + (2.0 ** -8 + 2.0 ** -11) * size[:n])
    worst = np.unravel_index(np.nanargmax(err), err.shape) if np.isfinite(err).any() else None
    assert np.all(err <= 0), (worst, np64(out)[:n][worst] if worst else None, ref[:n][worst] if worst else None)


ATTN = [
    # nq, nkv, hd, page, P, lens, new, window
    (8, 2, 64, 16, 0, [1], [1], 0),
    (8, 2, 64, 16, 100, [1, 17, 40], [1, 1, 1], 0),
    (8, 2, 64, 64, 129, [5, 64, 65], [5, 1, 3], 0),
    (8, 2, 64, 256, 300, [257, 1, 600], [1, 1, 2], 64),
    (40, 8, 128, 16, 1, [1], [1], 0),
    (40, 8, 128, 64, 1000, [1] * 16, [1] * 16, 0),
    (40, 8, 128, 64, 130, [70, 1, 128, 129, 300], [1, 0, 1, 1, 1], 0),
    (40, 8, 128, 64, 700, [10, 90, 500, 640, 900], [1] * 5, 512),
    (40, 8, 128, 128, 257, [30] * 30, [1] * 30, 0),
    (40, 8, 128, 32, 515, [9, 20, 41], [9, 7, 2], 0),
    (40, 8, 128, 32, 90, [33, 160], [20, 60], 0),
    (40, 8, 128, 64, 0, [300], [300], 0),
    (40, 8, 128, 64, 200, [150, 260], [130, 101], 96),
    (8, 8, 64, 16, 260, [3, 1], [2, 1], 0),
    (16, 1, 128, 64, 333, [100, 129], [1, 2], 0),
    (16, 1, 64, 16, 65, [200], [150], 33),
    (6, 2, 128, 16, 640, [50, 0, 70], [1, 0, 1], 0),
    (7, 1, 64, 32, 64, [64], [64], 1),
]


@pytest.mark.parametrize("i", range(len(ATTN)))
def test_attention_against_oracle(api, i):
    """Values in rows that nothing sees are NaN: none may reach an output."""
    nq, nkv, hd, page, P, lens, new, window = ATTN[i]
    c = attn_case(i, nq, nkv, hd, page, P, lens, new, pad=2, junk=float("nan"))
    out = torch.full_like(c["q"], 9.0)
    run_attn(api, c, window, out=out)
    close(c, out, window)
    assert torch.all(out[c["start"][-1]:] == 9.0)  # rows behind the last sequence
    again = run_attn(api, c, window, out=torch.empty_like(out))
    assert torch.equal(again[:c["start"][-1]], out[:c["start"][-1]])
