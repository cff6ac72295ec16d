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
    # packed rows of 128, 129, 256, 257 (one tile, a tile and a rest, a pair, a pair and a rest)
    (8, 2, 64, 64, 200, [70, 40], [32, 33], 0),
    (16, 1, 128, 64, 150, [16, 17], [16, 17], 0),
    (1, 1, 128, 16, 70, [256, 300, 257], [256, 129, 257], 0),
    # 48 and 49 packed rows, 32 and 33, among single rows: both kernels in one call
    (16, 1, 64, 32, 100, [50, 9, 1, 300, 2], [3, 2, 1, 4, 1], 0),
    (1, 1, 64, 16, 90, [80, 130, 1, 64, 200, 90], [48, 49, 1, 32, 33, 17], 70),
    # many keys, few rows: runs that cut a segment several times
    (40, 8, 128, 64, 9, [9000], [1], 0),
    (16, 2, 64, 128, 5000, [3, 700], [1, 4], 0),
    # a window that hides the whole prefix from some sequences, all of it from all
    (40, 8, 128, 64, 300, [10, 400, 100], [1, 1, 1], 64),
    (40, 8, 128, 32, 300, [100, 400], [1, 1], 50),
    (8, 2, 64, 16, 1000, [200] * 40, [1] * 40, 130),
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


@pytest.mark.parametrize("many", [False, True])
def test_attention_of_a_large_batch(api, many):
    """300 sequences of 0 to 2 rows; with `many`, some of 30 to 40 among them."""
    rng = np.random.default_rng(int(many))
    new = [int(n) for n in rng.integers(0, 3, 300)]
    if many:
        for b in rng.integers(0, 300, 12):
            new[b] = int(rng.integers(30, 41))
    lens = [n + int(rng.integers(0, 150)) for n in new]
    c = attn_case(300, 8, 2, 64, 16, 77, lens, new, pad=5, junk=float("inf"))
    out = torch.full_like(c["q"], 9.0)
    run_attn(api, c, 0, out=out)
    close(c, out, 0)
    assert torch.all(out[c["start"][-1]:] == 9.0)


def test_calls_on_two_streams_at_once(api):
    """Two attentions in flight, each with its own workspace and stream: the
    same bits as one after the other."""
    c = [attn_case(50 + i, 40, 8, 128, 64, 3000, [500] * 16, [1 + 2 * i] * 16) for i in range(2)]
    ref = [run_attn(api, x) for x in c]
    streams = [torch.cuda.Stream() for _ in c]
    args = [(x["q"], x["k"], x["v"], i32(x["start"]), i32(x["lens"]), i32(x["table"]), i32(x["ptab"]), 3000) for x in c]
    ws = [api.attn_shared_workspace(x["q"].shape[0], 16, 40, 8, 128, 1 + 2 * i) for i, x in enumerate(c)]
    outs = [torch.empty_like(x["q"]) for x in c]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                api.attn_shared(*args[i], max_new=1 + 2 * i, ws=ws[i], out=outs[i])
    torch.cuda.synchronize()
    for i in range(2):
        api.check(ws[i])
        assert torch.equal(outs[i], ref[i])


@pytest.mark.parametrize("P,new,more", [
    (8192, [1300, 743, 855, 824], 200), (1000, [1300, 700, 900], 0), (0, [4000], 0), (8192, [1] * 16, 1500),
    (4097, [9, 7, 8, 5] * 6, 900)])
def test_inputs_that_no_cache_holds(api, P, new, more):
    """The first call, every input in memory only, gives the bits of the second."""
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for seed in range(2):
        c = attn_case(seed, 40, 8, 128, 64, P, [n + more for n in new], new)
        flush.zero_()
        first = run_attn(api, c)
        assert torch.isfinite(first).all()
        assert torch.equal(first, run_attn(api, c))


def test_attention_with_rising_scores(api):
    """Scores that grow along the keys to 2^100 of the first one's weight: every
    reference has to move, in the prefix and in the own positions, for few rows
    and for many.  sum|q k| stays below 2^10, so an fp32 score is off by less
    than 128 2^-24 2^10 / sqrt(128), a weight by less than 2^-9 of itself."""
    for new, P in (([1, 1, 1], 700), ([3, 9, 2], 1100), ([60, 130, 1], 900)):
        lens = [n + 200 for n in new]
        c = attn_case(len(new), 40, 8, 128, 32, P, lens, new)
        c["q"] = c["q"] * 0 + 1
        flat = lambda x: x.transpose(1, 2).reshape(-1, 8, 128)
        k = flat(c["k"]).clone()
        for ids, n, base in [(c["ptab"], P, 0)] + [(c["table"][b], m, P) for b, m in enumerate(lens)]:
            i = torch.arange(n, device="cuda")
            at = i32(ids).long()[i // 32] * 32 + i % 32
            k[at] = (k[at].float() * 0.1 + (0.0025 * (i + base) * (1 + (i % 7 == 0)))[:, None, None]).to(torch.bfloat16)
        c["k"] = k.view(-1, 32, 8, 128).transpose(1, 2).contiguous()
        out = run_attn(api, c)
        ref, size = op.attend(np64(c["q"]), np64(c["k"]), np64(c["v"]), c["start"], lens, c["table"], c["ptab"], P, 0)
        assert np.all(np.abs(np64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -9) * size)


def test_the_widest_window_is_none(api):
    for P, lens, new in ((2000, [300, 77], [1, 1]), (700, [500, 90], [300, 20]), (5000, [40, 700], [9, 8])):
        c = attn_case(len(lens), 40, 8, 128, 64, P, lens, new)
        assert torch.equal(run_attn(api, c, 2 ** 31 - 1), run_attn(api, c, 0))


def test_attention_one_workspace_for_many_shapes(api):
    """A workspace of the largest call serves the others, in any order, twice."""
    cases = [attn_case(i, *ATTN[i][:7]) for i in (5, 8, 10, 12, 5)]
    news = [max(b - a for a, b in zip(c["start"], c["start"][1:])) for c in cases]
    size = max(api.attn_shared_workspace(c["q"].shape[0], len(c["lens"]), 40, 8, 128, n).numel()
               for c, n in zip(cases, news))
    ws, outs = api.zeros_workspace(size), []
    for _ in range(2):
        outs.append([run_attn(api, c, ATTN[i][7], ws=ws) for c, i in zip(cases, (5, 8, 10, 12, 5))])
    for a, b, c, i in zip(*outs, cases, (5, 8, 10, 12, 5)):
        assert torch.equal(a, b)
        close(c, a, ATTN[i][7])


def test_attention_reports_numbers_that_do_not_fit(api):
    """Rows beyond max_new, lengths beyond the table or below the rows, rows
    outside the call: the sequence is skipped and reported, the others are as
    without it.  A page id outside the cache is reported."""
    from w4_weight_only_b200 import _abi
    for hurt in ("new", "len", "short", "start", "page", "prefix page"):
        c = attn_case(3, 40, 8, 128, 64, 200, [100, 70, 300], [1, 3, 2])
        good = run_attn(api, c)
        start, lens, table, ptab, mn = list(c["start"]), list(c["lens"]), [list(r) for r in c["table"]], list(c["ptab"]), 3
        if hurt == "new":
            mn = 2
        elif hurt == "len":
            lens[1] = len(table[1]) * 64 + 1
        elif hurt == "short":
            lens[1] = 2
        elif hurt == "start":
            start[3] = 7
        elif hurt == "page":
            table[1][1] = c["k"].shape[0]
        else:
            ptab[0] = -1
        out = torch.full_like(c["q"], 9.0)
        ws = api.attn_shared_workspace(6, 3, 40, 8, 128, 3)
        api.attn_shared(c["q"], c["k"], c["v"], i32(start), i32(lens), i32(table), i32(ptab), 200, max_new=mn, ws=ws,
                        out=out)
        with pytest.raises(_abi.W4AError) as e:
            api.check(ws)
        assert e.value.code == _abi.ERR_KERNEL, hurt
        if hurt in ("new", "len", "short"):
            assert torch.equal(out[:1], good[:1]) and torch.equal(out[4:], good[4:]) and torch.all(out[1:4] == 9.0), hurt
        elif hurt == "start":
            assert torch.equal(out[:4], good[:4]) and torch.all(out[4:] == 9.0)


def test_pages_past_32_bits(api):
    """Pages whose elements lie beyond 2^31: the same bits as in a small cache."""
    c = attn_case(7, 40, 8, 128, 64, 300, [130, 70], [2, 1])
    good = run_attn(api, c)
    n, far = c["k"].shape[0], 40000
    big = dict(c)
    for x in ("k", "v"):
        big[x] = torch.zeros((far + n, 8, 64, 128), dtype=torch.bfloat16, device="cuda")
        big[x][far:] = c[x]
    big["table"] = [[p + far if p >= 0 else p for p in r] for r in c["table"]]
    big["ptab"] = [p + far for p in c["ptab"]]
    assert torch.equal(run_attn(api, big), good)
    cfg = shape_config(40, 8, 128)
    y = torch.randn((3, cfg.qkv_dim), generator=gen(1), device="cuda")
    qg, kg = torch.ones(5120, device="cuda"), torch.ones(1024, device="cuda")
    k0, v0 = torch.zeros_like(c["k"]), torch.zeros_like(c["k"])
    slots = [5, 64 * (n - 1) + 63, 64]
    api.qk_prep_paged(cfg, True, y, qg, kg, i32([4, 5, 6]), i32(slots), k0, v0)
    ws = api.zeros_workspace(256)
    api.qk_prep_paged(cfg, True, y, qg, kg, i32([4, 5, 6]), i32([s + 64 * far for s in slots]), big["k"], big["v"], ws=ws)
    api.check(ws)
    for s in slots:
        assert torch.equal(big["k"][far + s // 64, :, s % 64], k0[s // 64, :, s % 64])
        assert torch.equal(big["v"][far + s // 64, :, s % 64], v0[s // 64, :, s % 64])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
class Serving:
    """A layer of the small decoder on the paged cache: W4 QKV weights, the
    prefix filled as a sequence of its own, then steps of a batch behind it."""

    def __init__(self, api, cfg, n_pages, page, batch, seed):
        g = gen(seed)
        self.api, self.cfg, self.page, self.B = api, cfg, page, batch
        self.lin = api.quantize_linear(torch.randn((cfg.qkv_dim, cfg.d_model), generator=g, device="cuda") * 0.05)
        self.qg = 1 + 0.2 * torch.randn(cfg.q_dim, generator=g, device="cuda")
        self.kg = 1 + 0.2 * torch.randn(cfg.kv_dim, generator=g, device="cuda")
        self.kv = api.PagedKVCache(cfg, n_pages, page)
        self.k, self.v = self.kv.layer_views(3)
        self.queue, self.state = self.kv.free_queue()
        self.ws = api.zeros_workspace(256)

    def step(self, x, new, lens, table, max_rows, max_new, prefix=None, P=0, window=0, aws=None):
        """x bf16 [rows, d] -> (plan, q, attention output)."""
        api, cfg = self.api, self.cfg
        p = api.paged_plan(new, lens, self.state, self.queue, table, self.page, max_rows, prefix_len=P, ws=self.ws)
        y = torch.cat([api.gemv(self.lin, x[i:i + 16]) for i in range(0, len(x), 16)])
        q = api.qk_prep_paged(cfg, True, y, self.qg, self.kg, p.pos, p.slots, self.k, self.v, ws=self.ws)
        o = api.attn_shared(q, self.k, self.v, p.row_start, p.lens, table, prefix, P, window=window, max_new=max_new,
                            ws=aws)
        return p, q, o


def test_a_batch_behind_a_shared_prefix(api):
    """The prefix as a sequence, then a batch that grows, ends and is refilled
    behind it: attention against the oracle on the device's own q and pages,
    and against w4a_attn_decode on a private, linear copy of each history."""
    cfg, page, P, B = wc.tiny(), 16, 85, 3
    S = Serving(api, cfg, 40, page, B, 5)
    g = gen(6)
    x = lambda n: (torch.randn((n, cfg.d_model), generator=g, device="cuda")).to(torch.bfloat16)
    ptab = torch.full((1, 8), -1, dtype=torch.int32, device="cuda")
    p, q, o = S.step(x(P), i32([P]), i32([0]), ptab, P, P)
    S.state = p.state
    c = dict(q=q, k=S.k, v=S.v, start=[0, P], lens=[P], table=ptab.tolist(), ptab=[0], P=0)
    close(c, o, 0)
    prefix = ptab[0, :6].contiguous()
    lens, table = i32([0] * B), torch.full((B, 6), -1, dtype=torch.int32, device="cuda")
    kept = set(prefix.tolist())
    for new in ([5, 20, 1], [1, 1, 1], [4, 0, 2], [1, -1, 1], [1, 7, 1], [-1, 1, -1], [9, 1, 3]):
        rows = sum(max(n, 0) for n in new)
        p, q, o = S.step(x(rows + 2), i32(new), lens, table, rows + 2, max(new), prefix, P)
        api.check(S.ws)
        lens, S.state = p.lens, p.state
        c = dict(q=q, k=S.k, v=S.v, start=p.row_start.tolist(), lens=lens.tolist(), table=table.tolist(),
                 ptab=prefix.tolist(), P=P)
        close(c, o, 0)
        # no page belongs to two
        held = [t[j] for t, n in zip(c["table"], c["lens"]) for j in range(-(-n // page))]
        head, count = S.state.tolist()
        free = [S.queue.tolist()[(head + i) % 40] for i in range(count)]
        assert sorted(held + free + list(kept)) == list(range(40))
        # the last row of each sequence through the linear cache's attention
        for b, n in enumerate(c["lens"]):
            if n == 0 or new[b] < 1:
                continue
            i = torch.arange(P + n, device="cuda")
            pages = torch.where(i < P, prefix[(i // page).clamp(max=5)], table[b][((i - P) // page).clamp(min=0)]).long()
            at = torch.where(i < P, i % page, (i - P) % page)
            kc = torch.zeros((1, 2, 256, 64), dtype=torch.bfloat16, device="cuda")
            vc = torch.zeros_like(kc)
            api.kv_write_region(kc, vc, 1, 2, 64, 256, 0, 0, S.k[pages, :, at].transpose(0, 1).contiguous(),
                                S.v[pages, :, at].transpose(0, 1).contiguous())
            r = c["start"][b + 1] - 1
            ref = api.attn_decode(q[r:r + 1].contiguous(), kc, vc, 2, 256, i32([P + n - 1])).float()
            # two roundings of the result and the weights' (2^-8 of sum p|v|, here <= max|v|)
            assert torch.all((o[r].float() - ref[0]).abs() <= 2.0 ** -7 * ref[0].abs() + 2.0 ** -7 * vc.abs().max())


def test_a_step_captured_and_replayed(api):
    """A decode step in a CUDA graph on a side stream, replayed with other
    lengths and tokens: the same bits as the calls made one by one."""
    cfg, page, P, B = wc.tiny(), 16, 40, 4
    S = Serving(api, cfg, 64, page, B, 8)
    ptab = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    g = gen(9)
    x = lambda n: (torch.randn((n, cfg.d_model), generator=g, device="cuda")).to(torch.bfloat16)
    p, _, _ = S.step(x(P), i32([P]), i32([0]), ptab, P, P)
    S.state = p.state
    prefix = ptab[0, :3].contiguous()
    table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    p, _, _ = S.step(x(30), i32([10, 3, 16, 1]), i32([0] * B), table, 30, 16, prefix, P)
    lens, state = p.lens, p.state
    aws = api.attn_shared_workspace(B, B, cfg.n_heads, cfg.n_kv_heads, cfg.head_dim, 1)
    xs, ones = x(B), i32([1] * B)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    snap = lambda: [t.clone() for t in (S.kv.mem, S.queue, table)]
    keep = snap()
    S.state = state
    with torch.cuda.stream(side):
        S.step(xs, ones, lens, table, B, 1, prefix, P, aws=aws)  # warm up
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            gp, gq, go = S.step(xs, ones, lens, table, B, 1, prefix, P, aws=aws)
    torch.cuda.synchronize()
    for t, s in zip((S.kv.mem, S.queue, table), keep):
        t.copy_(s)
    for _ in range(20):  # crosses page borders
        new_x = x(B)
        keep = snap()
        ep, eq, eo = S.step(new_x, ones, lens.clone(), table, B, 1, prefix, P)
        after = snap()
        for t, s in zip((S.kv.mem, S.queue, table), keep):
            t.copy_(s)
        xs.copy_(new_x)
        graph.replay()
        torch.cuda.synchronize()
        api.check(aws)
        assert torch.equal(go, eo) and torch.equal(gq, eq) and torch.equal(gp.lens, ep.lens)
        for a, b in zip(snap(), after):
            assert torch.equal(a, b)
        lens.copy_(gp.lens)
        state.copy_(gp.state)


def test_binding_refuses(api):
    """Types, shapes, devices and layouts that the binding does not take."""
    c = attn_case(1, 8, 2, 64, 16, 20, [9], [1])
    a = dict(q=c["q"], k_pages=c["k"], v_pages=c["v"], row_start=i32([0, 1]), lens=i32([9]), table=i32(c["table"]),
             prefix_table=i32(c["ptab"]), prefix_len=20)
    api.attn_shared(**a)
    for bad, err in ((dict(q=c["q"].half()), TypeError), (dict(q=c["q"][:, ::2]), ValueError),
                     (dict(lens=i32([9]).long()), TypeError), (dict(row_start=i32([0, 1, 1])), ValueError),
                     (dict(v_pages=c["v"][:-1]), ValueError), (dict(k_pages=c["k"].transpose(1, 2)), ValueError),
                     (dict(table=i32(c["table"]).cpu()), ValueError), (dict(prefix_len=33), ValueError),
                     (dict(table=i32(c["table"])[0]), ValueError), (dict(out=c["q"]), RuntimeError)):
        with pytest.raises(err):
            api.attn_shared(**{**a, **bad})
    cfg = shape_config(8, 2, 64)
    y, qg, kg = torch.ones((2, cfg.qkv_dim), device="cuda"), torch.ones(512, device="cuda"), torch.ones(128, device="cuda")
    p = dict(cfg=cfg, full=True, qkv=y, q_gain=qg, k_gain=kg, pos=i32([0, 1]), slots=i32([0, 1]), k_pages=c["k"],
             v_pages=c["v"])
    api.qk_prep_paged(**p)
    for bad, err in ((dict(qkv=y.half()), TypeError), (dict(qkv=y[:, 1:]), ValueError), (dict(qkv=y.cpu()), ValueError),
                     (dict(q_gain=qg[:-1]), ValueError), (dict(slots=i32([0])), ValueError),
                     (dict(k_pages=c["k"][0]), ValueError)):
        with pytest.raises(err):
            api.qk_prep_paged(**{**p, **bad})
    n = dict(n_new=i32([1]), lens=i32([0]), state=i32([0, 2]), queue=i32([0, 1]), table=i32([[0]]), page_size=16, max_rows=1)
    api.paged_plan(**n)
    for bad, err in ((dict(lens=i32([0, 0])), ValueError), (dict(state=i32([0])), ValueError),
                     (dict(table=i32([0])), ValueError), (dict(queue=i32([0, 1]).float()), TypeError),
                     (dict(state=n["lens"].new_zeros(2).cpu()), ValueError)):
        with pytest.raises(err):
            api.paged_plan(**{**n, **bad})
