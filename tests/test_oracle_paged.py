"""The paged oracle against the decoder's own oracle: one sequence's pages read
position by position give the linear cache's attention, and prep the same
rotation; the plan keeps every page in one place."""
import numpy as np

from oracle import model as om
from oracle import paged as op


def test_attend_equals_the_linear_cache():
    cfg = om.tiny_config()
    rng = np.random.default_rng(0)
    P, n, page = 21, 14, 16
    K, V = rng.standard_normal((2, cfg.n_kv_heads, P + n, cfg.head_dim))
    k, v = np.full((5, cfg.n_kv_heads, page, cfg.head_dim), np.nan), np.full((5, cfg.n_kv_heads, page, cfg.head_dim), np.nan)
    ptab, tab = [3, 0], [4]
    for p in range(P + n):
        pg, i = (ptab[p // page], p % page) if p < P else (tab[(p - P) // page], (p - P) % page)
        k[pg, :, i], v[pg, :, i] = K[:, p], V[:, p]
    q = rng.standard_normal((2, cfg.n_heads, cfg.head_dim))
    for window in (0, 64, 9):
        out, _ = op.attend(q, k, v, [0, 2], [n], [tab], ptab, P, window)
        for r in range(2):
            pos = P + n - 2 + r
            lo = max(0, pos - window + 1) if window else 0
            for h in range(cfg.n_heads):
                c = h // (cfg.n_heads // cfg.n_kv_heads)
                ref = om.attend(q[r, h], K[c, lo:pos + 1], V[c, lo:pos + 1], 1 / np.sqrt(cfg.head_dim))
                assert np.allclose(out[r, h], ref, rtol=1e-12, atol=1e-14)


def test_prep_equals_qk_prep():
    cfg = om.tiny_config()
    rng = np.random.default_rng(1)
    y = rng.standard_normal((3, cfg.qkv_dim))
    qg, kg = rng.standard_normal(cfg.q_dim), rng.standard_normal(cfg.kv_dim)
    for full in (False, True):
        q, k, v, _, _ = op.prep(cfg, y, qg, kg, [0, 7, 90000], full)
        for r, pos in enumerate((0, 7, 90000)):
            rq, rk = om.qk_prep(cfg, y[r, :cfg.q_dim], y[r, cfg.q_dim:cfg.q_dim + cfg.kv_dim], qg, kg, pos, full)
            assert np.allclose(q[r], np.reshape(rq, q[r].shape), rtol=1e-10, atol=1e-12)
            assert np.allclose(k[r], np.reshape(rk, k[r].shape), rtol=1e-10, atol=1e-12)
            assert np.array_equal(v[r].ravel(), y[r, cfg.q_dim + cfg.kv_dim:])


def test_plan_keeps_pages_apart():
    rng = np.random.default_rng(2)
    B, page, W, N = 6, 4, 9, 40
    lens, state, queue, table = [0] * B, [0, N], list(range(N)), [[-1] * W for _ in range(B)]
    for _ in range(60):
        new = [int(rng.integers(-1, 6)) for _ in range(B)]
        got = op.plan(new, lens, state, queue, table, page, 10, 64)
        if got is None:  # does not fit: end the longest
            new = [-1 if n == max(lens) else 0 for n in lens]
            got = op.plan(new, lens, state, queue, table, page, 10, 64)
        lens, state, start, slots, pos, table, queue = got
        held = [t[j] for t, n in zip(table, lens) for j in range(-(-n // page))]
        free = [queue[(state[0] + i) % N] for i in range(state[1])]
        assert sorted(held + free) == list(range(N))
        rows = slots[:start[-1]]
        assert len(set(rows)) == len(rows) and all(s == -1 for s in slots[start[-1]:])


def test_plan_refuses_what_does_not_fit():
    assert op.plan([5], [0], [0, 1], [0], [[-1, -1]], 4, 0, 9) is None      # one page for five positions
    assert op.plan([5], [0], [0, 2], [0, 1], [[-1]], 4, 0, 9) is None       # a table of one page
    assert op.plan([5], [0], [0, 2], [0, 1], [[-1, -1]], 4, 0, 4) is None   # four rows
    assert op.plan([5], [0], [0, 2], [0, 1], [[-1, -1]], 4, 0, 5) is not None
