"""The paged KV cache in float64, position by position (test infrastructure):
the plan of a step, QK-norm and rotation into pages, attention behind a shared
prefix.  Written from the definitions in include/w4a.h, apart from the CUDA
package."""
from __future__ import annotations

import math

import numpy as np

from . import model as om


def plan(n_new, lens, state, queue, table, page, prefix_len, max_rows):
    """One step's plan with plain lists; returns (lens, state, row_start,
    slots, pos, table, queue), or None where the step does not fit."""
    queue, table = list(queue), [list(r) for r in table]
    (head, count), N = state, len(queue)
    if sum(max(n, 0) for n in n_new) > max_rows:
        return None
    for b, n in enumerate(n_new):
        if n < 0:
            for j in range(-(-lens[b] // page)):
                queue[(head + count) % N] = table[b][j]
                count += 1
    out, start, slots, pos = [], [0], [], []
    for b, n in enumerate(n_new):
        for i in range(lens[b], lens[b] + max(n, 0)):
            if i % page == 0:
                if count == 0 or i // page >= len(table[b]):
                    return None
                table[b][i // page] = queue[head]
                head, count = (head + 1) % N, count - 1
            slots.append(table[b][i // page] * page + i % page)
            pos.append(prefix_len + i)
        out.append(lens[b] + n if n >= 0 else 0)
        start.append(start[-1] + max(n, 0))
    pad = [-1] * (max_rows - len(slots))
    return out, [head, count], start, slots + pad, pos + pad, table, queue


def prep(cfg: om.OracleConfig, qkv, q_gain, k_gain, pos, full):
    """(q [rows, nq, hd], k, v [rows, nkv, hd], size) of rows with pos >= 0;
    size: |x1| + |x2| of each rotated pair before the rotation, times the
    attention factor (the scale that rounding errors of the pair go by)."""
    y = np.asarray(qkv, dtype=np.float64)
    inv, ms = om.layer_rope(cfg, full)
    h2 = cfg.head_dim // 2
    ang = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(inv)[None, :]
    c, s = np.cos(ang)[:, None, :], np.sin(ang)[:, None, :]

    def form(x, gain, heads):
        x = om.rmsnorm(x, gain, cfg.eps).reshape(len(y), heads, cfg.head_dim)
        a, b = x[..., :h2], x[..., h2:]
        size = np.concatenate([np.abs(a) + np.abs(b)] * 2, -1) * ms
        return np.concatenate([a * c - b * s, b * c + a * s], -1) * ms, size

    q, qs = form(y[:, :cfg.q_dim], q_gain, cfg.n_heads)
    k, ks = form(y[:, cfg.q_dim:cfg.q_dim + cfg.kv_dim], k_gain, cfg.n_kv_heads)
    return q, k, y[:, cfg.q_dim + cfg.kv_dim:].reshape(len(y), cfg.n_kv_heads, cfg.head_dim), qs, ks


def attend(q, k_pages, v_pages, row_start, lens, table, prefix_table, P, window):
    """(out, size) [rows, nq, hd] float64; size = sum of p |v| (the scale of
    the weights' rounding).  k_pages, v_pages: float64 [n_pages, nkv, page,
    hd]; positions that no row sees are never read.  Rows behind the last
    sequence are NaN."""
    q = np.asarray(q, dtype=np.float64)
    R, nq, hd = q.shape
    nkv, page = k_pages.shape[1], k_pages.shape[2]
    out, size = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    for b, n in enumerate(lens):
        r0, r1 = row_start[b], row_start[b + 1]
        for r in range(r0, r1):
            p = P + n - (r1 - r0) + (r - r0)
            j = np.arange(max(0, p - window + 1) if window else 0, p + 1)
            pre, mine = j[j < P], j[j >= P] - P
            pg = np.concatenate([np.asarray(prefix_table, dtype=np.int64)[pre // page],
                                 np.asarray(table[b], dtype=np.int64)[mine // page]])
            at = np.concatenate([pre % page, mine % page])
            for c in range(nkv):
                K, V = k_pages[pg, c, at], v_pages[pg, c, at]
                h = slice(c * (nq // nkv), (c + 1) * (nq // nkv))
                w = om.softmax(q[r, h] @ K.T / math.sqrt(hd))
                out[r, h], size[r, h] = w @ V, w @ np.abs(V)
    return out, size
