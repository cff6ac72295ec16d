"""Attention behind a shared prefix with a NaN or an infinity among what a row
sees: the output is what the softmax's formula gives, however the keys were
cut into pieces, and nothing else changes.

q or K: an infinite or NaN score makes every output of its (row, head) NaN, a
score of -inf takes its key out.  V: the column of every row that sees it is
not finite (a row of the call that does not see it may get it there too).
All other outputs keep their bits: a masked or finite weight does not depend
on the values of other rows.
"""
import numpy as np
import pytest
import torch

from oracle import paged as op
from helpers import np64
from test_paged_gpu import api, attn_case, run_attn  # noqa: F401

pytestmark = pytest.mark.gpu

CUTS = {
    # nq, nkv, hd, page, P, lens, new, window
    "whole segments": (40, 8, 128, 64, 0, [30] * 64, [1] * 64, 0),
    "a segment in pieces": (40, 8, 128, 64, 0, [300], [1], 0),
    "a segment in pieces, 48 rows": (8, 2, 64, 16, 0, [900, 70], [12, 3], 0),
    "prefix ahead": (40, 8, 128, 64, 100, [70, 300], [1, 1], 0),
    "prefix pass, one tile of rows": (40, 8, 128, 64, 1000, [1] * 16, [1] * 16, 0),
    "prefix pass, a pair and a rest": (40, 8, 128, 64, 1500, [30] * 64, [1] * 64, 0),
    "prefix pass, window": (40, 8, 128, 64, 1000, [40 * i + 1 for i in range(20)], [1] * 20, 700),
    "prefix with few rows": (40, 8, 128, 64, 5000, [1, 70, 300], [1] * 3, 0),
    "prefix with few rows, window": (16, 2, 64, 32, 5000, [5, 300], [1, 1], 2000),
    "own tiles in pieces": (40, 8, 128, 64, 0, [300], [300], 0),
    "own tiles in pieces behind a prefix pass": (40, 8, 128, 64, 4500, [160] * 4, [60] * 4, 0),
    "joined with the prefix at the tile's end": (40, 8, 128, 64, 4500, [200] * 4, [100] * 4, 0),
    "finished at the tile's end": (40, 8, 128, 64, 0, [300] * 4, [300] * 4, 0),
    "one visible key": (8, 2, 64, 16, 20, [9, 40], [3, 30], 1),
}
BAD = {"nan": float("nan"), "inf": float("inf")}


def place(c, b, pos):
    """(page, row) of position pos of sequence b."""
    page = c["k"].shape[2]
    ids, at = (c["ptab"], pos) if pos < c["P"] else (c["table"][b], pos - c["P"])
    return ids[at // page], at % page


def where(c, r):
    """(sequence, position) of row r."""
    b = max(s for s in range(len(c["lens"])) if c["start"][s] <= r < c["start"][s + 1])
    return b, c["P"] + c["lens"][b] - (c["start"][b + 1] - r)


def seeing(c, b, pos, window):
    """Rows that see position pos (an own position: of sequence b)."""
    at = [(r, *where(c, r)) for r in range(c["start"][-1])]
    return [r for r, s, p in at if (pos < c["P"] or s == b) and pos <= p and (window == 0 or p - pos < window)]


def attend_rows(c, rows, window):
    """The oracle's (out, size) of some rows, each as a sequence of one row."""
    at = [where(c, r) for r in rows]
    with np.errstate(invalid="ignore"):
        return op.attend(np64(c["q"][rows]), np64(c["k"]), np64(c["v"]), list(range(len(rows) + 1)),
                         [p + 1 - c["P"] for _, p in at], [c["table"][b] for b, _ in at], c["ptab"], c["P"], window)


@pytest.mark.parametrize("cut", CUTS)
def test_queries(api, cut):
    nq, nkv, hd, page, P, lens, new, window = CUTS[cut]
    c = attn_case(7, nq, nkv, hd, page, P, lens, new)
    base = run_attn(api, c, window)
    assert torch.isfinite(base).all()
    R = c["q"].shape[0]
    for bad in BAD.values():
        for r, h in {(0, 1), (R // 2, nq - 1), (R - 1, nq // 2)}:
            hurt = dict(c, q=c["q"].clone())
            hurt["q"][r, h, hd - 3] = bad
            out = run_attn(api, hurt, window)
            assert torch.isnan(out[r, h]).all(), (bad, r, h, out[r, h, :4])
            out[r, h] = base[r, h]
            assert torch.equal(out, base), (bad, r, h)


@pytest.mark.parametrize("cut", CUTS)
def test_keys_and_values(api, cut):
    nq, nkv, hd, page, P, lens, new, window = CUTS[cut]
    g, kvh, dim = nq // nkv, nkv - 1, 11
    c = attn_case(8, nq, nkv, hd, page, P, lens, new)
    base = run_attn(api, c, window)
    assert torch.isfinite(base).all()
    b = len(lens) - 1
    last = P + lens[b] - 1
    lowest = max(0, last - window + 1) if window else 0
    for pos in sorted({last, lowest, (lowest + last) // 2, max(0, P - 1), 2 * P // 3}):
        rows = seeing(c, b, pos, window)
        if not rows:
            continue
        pg, at = place(c, b, pos)
        heads = slice(kvh * g, (kvh + 1) * g)
        mine = torch.zeros_like(base, dtype=torch.bool)
        mine[torch.tensor(rows, device="cuda"), heads] = True
        for name, bad in BAD.items():
            hurt = dict(c, k=c["k"].clone())
            hurt["k"][pg, kvh, at, dim] = bad
            out = run_attn(api, hurt, window)
            assert torch.equal(out[~mine], base[~mine]), (name, pos)
            got = out[rows][:, heads]
            if name == "nan":
                assert torch.isnan(got).all(), pos
            else:  # +inf scores give NaN, -inf scores leave the other keys
                some = rows[:: max(1, len(rows) // 12)]
                want, size = (x[:, heads] for x in attend_rows(hurt, some, window))
                o, ok = np64(out[some][:, heads]), np.isfinite(want)
                assert np.array_equal(np.isnan(o), ~ok), pos
                assert np.all(np.abs(o - want)[ok] <= (2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -11) * size)[ok])
                # (a row that sees nothing else has no weight left either)
                only = torch.tensor([[window == 1 or where(c, r)[1] == 0] for r in rows], device="cuda")
                assert torch.equal(torch.isnan(got).all(-1), (c["q"][rows][:, heads, dim] >= 0) | only), pos
            hurt = dict(c, v=c["v"].clone())
            hurt["v"][pg, kvh, at, dim] = bad
            out = run_attn(api, hurt, window)
            assert not torch.isfinite(out[rows][:, heads, dim]).any(), (name, pos)
            out[:, heads, dim] = base[:, heads, dim]
            assert torch.equal(out, base), (name, pos)
