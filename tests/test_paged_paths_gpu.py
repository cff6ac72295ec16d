"""Attention behind a shared prefix against the float64 oracle, one case or
more for each way in which the host cuts a call (paged_paths.PATHS), and at the
sizes of prompts and turns.

Tolerance: as in test_paged_gpu.py (one rounding of the result, one of each
weight, the scores'), and the sums in fp32: N visible keys add at most N 2^-24
of sum p |v| in the numerator and as much in the sum of the weights.
"""
import numpy as np
import pytest
import torch

from oracle import paged as op
from helpers import np64, oracle_config
from paged_paths import PATHS
from test_paged_gpu import api, attn_case, gen, i32, run_attn, shape_config  # noqa: F401

pytestmark = pytest.mark.gpu


def sampled(c, most):
    """At most about `most` rows: the first and last of each sequence and those
    around the borders of row tiles, then a spread of the others."""
    n, g = c["start"][-1], c["q"].shape[1] // c["k"].shape[1]
    if n <= most:
        return list(range(n))
    keep = {r for s in c["start"] for r in (s - 1, s)}
    keep |= {x * 256 // g + d for x in (1, 2, 3, n * g // 256) for d in (-1, 0, 1)}
    keep = sorted(r for r in keep if 0 <= r < n)
    if len(keep) > most:
        keep = keep[:: -(-len(keep) // most)]
    return sorted(set(keep) | set(range(0, n, -(-n // max(1, most - len(keep))))))


def close_rows(c, out, window, rows):
    """Those rows against the oracle, each as a sequence of one row."""
    lens, table = [], []
    for r in rows:
        b = max(s for s in range(len(c["lens"])) if c["start"][s] <= r < c["start"][s + 1])
        lens.append(c["lens"][b] - (c["start"][b + 1] - 1 - r))
        table.append(c["table"][b])
    ref, size = op.attend(np64(c["q"][rows]), np64(c["k"]), np64(c["v"]), list(range(len(rows) + 1)), lens, table,
                          c["ptab"], c["P"], window)
    n = np.array([c["P"] + x if not window else min(window, c["P"] + x) for x in lens])[:, None, None]
    err = np.abs(np64(out[rows]) - ref) - (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -11 + 2 * n * 2.0 ** -24) * size)
    assert np.all(err <= 0), (np.unravel_index(np.nanargmax(err), err.shape), np.nanmax(err))


@pytest.mark.parametrize("name", PATHS)
def test_path(api, name):
    """Rows of pages that nothing sees hold NaN."""
    (nq, nkv, hd, page, P, lens, new, window), pad, _ = PATHS[name]
    c = attn_case(len(name), nq, nkv, hd, page, P, lens, new, pad=pad, junk=float("nan"))
    n, out = c["start"][-1], torch.full_like(c["q"], 9.0)
    run_attn(api, c, window, out=out)
    assert torch.isfinite(out).all() and torch.all(out[n:] == 9.0)
    close_rows(c, out, window, sampled(c, 60))
    again = run_attn(api, c, window, out=torch.empty_like(out))
    assert torch.equal(again[:n], out[:n])


@pytest.mark.parametrize("P,new,more,window", [
    (8192, [1300, 743, 855, 824], 200, 0), (8192, [1300, 743, 855, 824], 200, 4096), (1000, [1300, 700, 900], 0, 0),
    (0, [4000], 0, 0), (0, [8192], 0, 0), (0, [8192], 0, 4096), (4097, [9, 7, 8, 5] * 6, 900, 0),
    (4097, [9, 7, 8, 5] * 6, 900, 2000), (32768, [1] * 64, 900, 0), (6001, [1] * 16, 5900, 4096)])
def test_sizes_of_use(api, P, new, more, window):
    """Prompts, turns, drafts and decodes of the 32B shape: up to 40 rows of each."""
    c = attn_case(len(new) + window, 40, 8, 128, 64, P, [n + (more * (i + 1)) // len(new) for i, n in enumerate(new)], new)
    out = run_attn(api, c, window)
    assert torch.isfinite(out).all()
    close_rows(c, out, window, sampled(c, 40 if P < 32768 else 12))


@pytest.mark.parametrize("P,lens,new", [
    (5000, [201, 100, 300], [1, 1, 1]), (3000, [150] * 64, [1] * 64), (4500, [200] * 4, [100] * 4),
    (4500, [300, 200], [40, 9])])
def test_rising_scores_over_a_prefix_of_its_own(api, P, lens, new):
    """Scores that grow along the keys to 2^100 of the first one's weight, over
    a prefix that has pieces of its own: references differ between the pieces
    as far as within them.  sum|q k| stays below 2^10, as in the test beside
    the shorter prefixes; weights off by less than 2^-9 of themselves."""
    c = attn_case(len(new), 40, 8, 128, 32, P, lens, new)
    c["q"] = c["q"] * 0 + 1
    flat = lambda x: x.transpose(1, 2).reshape(-1, 8, 128)
    k = flat(c["k"]).clone()
    top = P + max(lens)
    for ids, n, base in [(c["ptab"], P, 0)] + [(c["table"][b], m, P) for b, m in enumerate(lens)]:
        i = torch.arange(n, device="cuda")
        at = i32(ids).long()[i // 32] * 32 + i % 32
        k[at] = (k[at].float() * 0.1 + (3.4 * (i + base) / top * (1 + (i % 7 == 0)))[:, None, None]).to(torch.bfloat16)
    c["k"] = k.view(-1, 32, 8, 128).transpose(1, 2).contiguous()
    out = run_attn(api, c)
    rows = sampled(c, 40)
    one = [(c["table"][b], m - (c["start"][b + 1] - 1 - r)) for r in rows for b, m in enumerate(lens)
           if c["start"][b] <= r < c["start"][b + 1]]
    ref, size = op.attend(np64(c["q"][rows]), np64(c["k"]), np64(c["v"]), list(range(len(rows) + 1)),
                          [m for _, m in one], [t for t, _ in one], c["ptab"], P, 0)
    assert np.all(np.abs(np64(out[rows]) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -9) * size)


@pytest.mark.parametrize("nq,nkv,hd,batch,most,longest", [
    (8, 2, 64, 4096, 1, 40),       # the most sequences
    (1, 1, 64, 4096, 256, 256),    # the most rows: 2^20
    (1024, 64, 64, 3, 2, 300),     # the most heads, 16 to a KV head
    (64, 64, 128, 2, 130, 200)])
def test_largest_calls(api, nq, nkv, hd, batch, most, longest):
    rng = np.random.default_rng(batch)
    whole = most == 256
    new = [most if whole else int(rng.integers(0, most + 1)) for _ in range(batch)]
    lens = [n if whole else n + int(rng.integers(0, longest - most + 1)) for n in new]
    new[0], lens[0] = most, longest
    c = attn_case(batch, nq, nkv, hd, 16, 21, lens, new)
    assert not whole or c["q"].shape[0] == 1 << 20
    out = run_attn(api, c)
    assert torch.isfinite(out).all()
    n = c["start"][-1]
    close_rows(c, out, 0, sorted({0, n - 1} | {int(r) for r in rng.integers(0, n, 20)}))


@pytest.mark.parametrize("nq,nkv,hd", [(160, 20, 128), (320, 40, 64)])
def test_the_widest_rows(api, nq, nkv, hd):
    """QKV rows of 25,600 values, the most: append and attention."""
    cfg = shape_config(nq, nkv, hd)
    assert cfg.qkv_dim == 25600
    g, rows, page = gen(1), 5, 16
    y = torch.randn((rows, cfg.qkv_dim), generator=g, device="cuda")
    qg, kg = 1 + 0.2 * torch.randn(nq * hd, generator=g, device="cuda"), torch.ones(nkv * hd, device="cuda")
    k = torch.zeros((2, nkv, page, hd), dtype=torch.bfloat16, device="cuda")
    v, slots, pos = torch.zeros_like(k), [3, 17, 4, 31, 0], [0, 1, 2, 3, 4]
    ws = api.zeros_workspace(256)
    q = api.qk_prep_paged(cfg, True, y, qg, kg, i32(pos), i32(slots), k, v, ws=ws)
    api.check(ws)
    rq, rk, rv, qs, ks = op.prep(oracle_config(cfg), np64(y), np64(qg), np64(kg), pos, True)
    K, V = (np64(t).transpose(0, 2, 1, 3).reshape(-1, nkv, hd)[slots] for t in (k, v))
    # (the bounds of test_paged_gpu.py; a sum of squares of up to 20,480 terms in a tree)
    assert np.all(np.abs(np64(q) - rq) <= 2.0 ** -8 * np.abs(rq) + 2.0 ** -18 * qs)
    assert np.all(np.abs(K - rk) <= 2.0 ** -8 * np.abs(rk) + 2.0 ** -18 * ks)
    assert np.array_equal(V, np64(torch.from_numpy(rv).to(torch.bfloat16)))
