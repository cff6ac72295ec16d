"""What is timed of the paged KV cache: the block tables and slot maps of a
step (plan), the QK-norm, rotation and append into the pages (prep), and the
attention of a batch that shares a prefix (attn), each in plain torch
operations and as the calls of this package.

A case names its operator ("op") and the sizes; request lengths follow from
the case alone, values from the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda"
THETA, YARN_FACTOR, YARN_CTX, BETA_FAST, BETA_SLOW, EPS = 500000.0, 8.0, 8192, 32.0, 1.0, 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a small batch: a token each, a page now and then
        dict(name="plan_decode_16", op="plan", batch=16, page=64, max_len=8192, prompt=0, prefix=8192),
        # a busy server's step: decodes, idle slots, ended requests, admitted prompts
        dict(name="plan_admit_1024", op="plan", batch=1024, page=16, max_len=2048, prompt=1024, prefix=777),
        # the QKV rows of one decode step, the 32B shape, a full-attention layer (YaRN)
        dict(name="prep_decode_16", op="prep", rows=16, pad=0, nq=40, nkv=8, hd=128, page=64, full=True, start=9000),
        # a prompt chunk of the 32B shape, a sliding-window layer
        dict(name="prep_prompt_8192", op="prep", rows=8192, pad=0, nq=40, nkv=8, hd=128, page=64, full=False, start=0),
        # the small decoder, an odd number of rows, padding rows behind them
        dict(name="prep_odd_1231", op="prep", rows=1231, pad=49, nq=8, nkv=2, hd=64, page=16, full=True, start=60000),
        # the small decoder: three short sequences behind a short shared prompt
        dict(name="attn_small_3", op="attn", batch=3, nq=8, nkv=2, hd=64, page=16, prefix=100, max_len=40, new=1,
             window=0),
        # decode, 32B shape: 16 sequences behind one 8K prompt
        dict(name="attn_decode_16", op="attn", batch=16, nq=40, nkv=8, hd=128, page=64, prefix=8192, max_len=2048,
             new=1, window=0),
        # the same on a sliding-window layer: the window ends inside the prefix, or behind it
        dict(name="attn_window_16", op="attn", batch=16, nq=40, nkv=8, hd=128, page=64, prefix=6001, max_len=6000,
             new=1, window=4096),
        # decode of a large batch behind a long shared document
        dict(name="attn_decode_64", op="attn", batch=64, nq=40, nkv=8, hd=128, page=128, prefix=32768, max_len=1024,
             new=1, window=0),
        # a few drafted tokens a sequence, checked together; small pages, odd lengths
        dict(name="attn_draft_24", op="attn", batch=24, nq=40, nkv=8, hd=128, page=16, prefix=4097, max_len=1500,
             new=9, window=0),
        # user turns of about a thousand tokens each behind the shared prompt
        dict(name="attn_turns_4", op="attn", batch=4, nq=40, nkv=8, hd=128, page=64, prefix=8192, max_len=1500,
             new=1300, window=0),
        # one whole prompt, no prefix yet
        dict(name="attn_prompt_8192", op="attn", batch=1, nq=40, nkv=8, hd=128, page=64, prefix=0, max_len=8192,
             new=8192, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "prep", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        return dict(op="plan", batch=_log(rng, 1, 1024), page=page, max_len=_log(rng, 16, 2048),
                    prompt=rng.choice([0, _log(rng, 2, 1024)]), prefix=_log(rng, 1, 9000) - 1)
    shape = rng.choice([dict(nq=40, nkv=8, hd=128), dict(nq=40, nkv=8, hd=128), dict(nq=8, nkv=2, hd=64),
                        dict(nq=16, nkv=2, hd=128), dict(nq=8, nkv=8, hd=64)])
    if op == "prep":
        return dict(op="prep", rows=_log(rng, 1, 8192), pad=rng.choice([0, rng.randrange(1, 64)]), page=page,
                    full=rng.random() < 0.5, start=_log(rng, 1, 100000) - 1, **shape)
    window = rng.choice([0, 0, 64, 512, 4096])
    if rng.random() < 0.25:   # prompts and turns
        batch, new, prefix = rng.randrange(1, 5), _log(rng, 32, 1300), _log(rng, 1, 8192) - 1
        max_len = new + _log(rng, 1, 1000)
    else:                     # single tokens, a few drafted ones
        batch, new, prefix = _log(rng, 1, 64), rng.choice([1, 1, 1, rng.randrange(2, 10)]), _log(rng, 1, 16384) - 1
        max_len = max(new, _log(rng, 1, 4096))
    return dict(op="attn", batch=batch, page=page, prefix=prefix, max_len=max_len, new=new, window=window, **shape)


def _rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _plan_lengths(case):
    """(lens, n_new) of the batch: single tokens; with prompts also idle, ended and admitted sequences."""
    rng = _rng(case)
    lens, new = [], []
    for _ in range(case["batch"]):
        n, k = rng.randrange(0, case["max_len"] + 1), 1
        if case["prompt"]:
            r = rng.random()
            if r < 0.15:
                k = 0
            elif r < 0.25:
                k = -1
            elif r < 0.35:
                n, k = 0, rng.randrange(1, case["prompt"] + 1)
        lens.append(n)
        new.append(k)
    return lens, new


def _attn_lengths(case):
    """(lens, n_new): own positions after the append, and how many of them are this step's rows."""
    rng = _rng(case)
    lens, new = [], []
    for b in range(case["batch"]):
        k = case["new"] if b == 0 else rng.randrange((case["new"] + 1) // 2, case["new"] + 1)
        n = case["max_len"] if b == 0 else rng.randrange(min(case["max_len"], max(k, case["max_len"] // 8)),
                                                         case["max_len"] + 1)
        lens.append(n)
        new.append(k)
    return lens, new


def _pages(n, page):
    return (n + page - 1) // page


def work(case):
    if case["op"] == "plan":
        lens, new = _plan_lengths(case)
        B, page = case["batch"], case["page"]
        rows = sum(max(k, 0) for k in new)
        moved = sum(_pages(n, page) if k < 0 else _pages(n + k, page) - _pages(n, page) for n, k in zip(lens, new))
        return {"bytes": 4.0 * (2 * B + 2 + 2 * moved + B + 2 + B + 1 + 2 * rows), "flops": 0.0}
    if case["op"] == "prep":
        width = (case["nq"] + 2 * case["nkv"]) * case["hd"]
        return {"bytes": float(case["rows"] * (6 * width + 8) + 4 * (case["nq"] + case["nkv"]) * case["hd"]),
                "flops": 10.0 * case["rows"] * width}
    lens, new = _attn_lengths(case)
    P, W, nq, nkv, hd = case["prefix"], case["window"], case["nq"], case["nkv"], case["hd"]
    pairs, own_keys, first = 0, 0, P
    for n, k in zip(lens, new):
        p0 = P + n - k                       # position of the sequence's first row
        lo = max(0, p0 - W + 1) if W else 0
        first = min(first, lo)
        own_keys += P + n - max(P, lo)
        pairs += sum(min(p + 1, W) if W else p + 1 for p in range(p0, P + n))
    rows = sum(new)
    return {"bytes": float(4 * hd * nkv * (P - first + own_keys) + 4 * rows * nq * hd), "flops": 4.0 * hd * nq * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _plan_inputs(case, seed):
    lens, new = _plan_lengths(case)
    page = case["page"]
    rng = random.Random(seed)
    held = [_pages(n, page) for n in lens]
    width = max(1, max(_pages(n + max(k, 0), page) for n, k in zip(lens, new)))
    n_pages = sum(held) + sum(_pages(n + max(k, 0), page) for n, k in zip(lens, new)) + 7
    ids = list(range(n_pages))
    rng.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    free = ids[at:]
    head = rng.randrange(n_pages)            # the queue wraps
    queue = [0] * n_pages
    for i, p in enumerate(free):
        queue[(head + i) % n_pages] = p
    rows = max(1, sum(max(k, 0) for k in new))
    return dict(lens=_i32(lens), new=_i32(new), state=_i32([head, len(free)]), queue=_i32(queue), table=_i32(table),
                page=page, prefix=case["prefix"], rows=rows)


def _prep_inputs(case, seed):
    g, rng = _gen(seed), random.Random(seed)
    nq, nkv, hd, page, rows, pad = (case[k] for k in ("nq", "nkv", "hd", "page", "rows", "pad"))
    n_pages = _pages(rows, page) + 3
    slots = rng.sample(range(n_pages * page), rows) + [-1] * pad
    pos = [case["start"] + i for i in range(rows)] + [-1] * pad
    y = torch.randn((rows + pad, (nq + 2 * nkv) * hd), generator=g, device=DEV) * 0.7
    return dict(y=y, q_gain=1 + 0.1 * torch.randn(nq * hd, generator=g, device=DEV),
                k_gain=1 + 0.1 * torch.randn(nkv * hd, generator=g, device=DEV), slots=_i32(slots), pos=_i32(pos),
                k=torch.zeros((n_pages, nkv, page, hd), dtype=torch.bfloat16, device=DEV),
                v=torch.zeros((n_pages, nkv, page, hd), dtype=torch.bfloat16, device=DEV),
                q=torch.zeros((rows + pad, nq, hd), dtype=torch.bfloat16, device=DEV),
                nq=nq, nkv=nkv, hd=hd, page=page, full=case["full"])


def _attn_inputs(case, seed):
    g, rng = _gen(seed), random.Random(seed)
    nq, nkv, hd, page, P = (case[k] for k in ("nq", "nkv", "hd", "page", "prefix"))
    lens, new = _attn_lengths(case)
    used = _pages(P, page) + sum(_pages(n, page) for n in lens)
    ids = list(range(used + 2))
    rng.shuffle(ids)
    prefix_table, at = ids[:_pages(P, page)], _pages(P, page)
    width = max(1, max(_pages(n, page) for n in lens))
    table = []
    for n in lens:
        h = _pages(n, page)
        table.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    start = [0]
    for k in new:
        start.append(start[-1] + k)
    shape = (used + 2, nkv, page, hd)
    # keys after their norm and rotation, values, and queries whose scores spread over a few units
    k = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    v = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    q = (torch.randn((start[-1], nq, hd), generator=g, device=DEV) * 1.5).to(torch.bfloat16)
    return dict(q=q, k=k, v=v, table=_i32(table), prefix_table=_i32(prefix_table or [0]), lens=_i32(lens),
                row_start=_i32(start), host_lens=lens, host_start=start, nq=nq, nkv=nkv, hd=hd, page=page, prefix=P,
                window=case["window"], new=case["new"])


def _inputs(case, seed):
    return {"plan": _plan_inputs, "prep": _prep_inputs, "attn": _attn_inputs}[case["op"]](case, seed)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["op"] = case["op"]
    if own:
        from w4_weight_only_b200 import api, config
        if case["op"] == "plan":
            s["ws"] = api.zeros_workspace(256)
        elif case["op"] == "prep":
            s["cfg"] = config.Config(d_model=512, n_layers=4, n_heads=s["nq"], n_kv_heads=s["nkv"], head_dim=s["hd"],
                                     ffn=512, vocab=16, window=64)
            s["ws"] = api.zeros_workspace(256)
        else:
            s["ws"] = api.attn_shared_workspace(s["q"].shape[0], len(s["host_lens"]), s["nq"], s["nkv"], s["hd"],
                                                s["new"])
            s["out"] = torch.empty_like(s["q"])
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plan_plain(s):
    lens, new, table, queue, page = s["lens"].long(), s["new"].long(), s["table"], s["queue"], s["page"]
    B, width = table.shape
    N = queue.numel()
    head, count = s["state"][0].long(), s["state"][1].long()
    live = new >= 0
    add = new.clamp(min=0)
    zero = torch.zeros_like(lens)
    held = (lens + page - 1) // page
    lens2 = torch.where(live, lens + add, zero)
    take = torch.where(live, (lens2 + page - 1) // page - held, zero)
    freed = torch.where(live, zero, held)
    take0, freed0 = torch.cumsum(take, 0) - take, torch.cumsum(freed, 0) - freed
    j = torch.arange(width, device=DEV)
    # ended sequences' pages to the queue's end (entries that are not freed go to a spare place)
    mine = j[None, :] < freed[:, None]
    spot = torch.where(mine, (head + count + freed0[:, None] + j[None, :]) % N, torch.full_like(mine, N, dtype=torch.long))
    grown = torch.cat([queue, queue.new_zeros(1)])
    grown[spot.reshape(-1)] = table.reshape(-1)
    queue.copy_(grown[:N])
    k = j[None, :] - held[:, None]
    fresh = (k >= 0) & (k < take[:, None])
    page_id = queue[(head + take0[:, None] + k.clamp(min=0)) % N]
    table.copy_(torch.where(fresh, page_id, table))
    row_start = torch.zeros(B + 1, dtype=torch.long, device=DEV)
    row_start[1:] = torch.cumsum(add, 0)
    r = torch.arange(s["rows"], device=DEV)
    seq = torch.searchsorted(row_start[1:].contiguous(), r, right=True).clamp(max=B - 1)
    at = lens[seq] + r - row_start[seq]
    inside = r < row_start[B]
    at = torch.where(inside, at, torch.zeros_like(at))
    slots = torch.where(inside, table[seq, at // page].long() * page + at % page, torch.full_like(at, -1))
    pos = torch.where(inside, at + s["prefix"], torch.full_like(at, -1))
    state = torch.stack([(head + take.sum()) % N, count + freed.sum() - take.sum()])
    return (lens2.int(), state.int(), row_start.int(), slots.int(), pos.int(), table, queue)


def _frequencies(hd, full):
    """Inverse frequencies (float64 list) and attention factor of a layer: plain rotation, or YaRN on full layers."""
    f = [THETA ** (-2.0 * i / hd) for i in range(hd // 2)]
    if not full:
        return f, 1.0
    lo = math.floor(hd * math.log(YARN_CTX / (BETA_FAST * 2 * math.pi)) / (2 * math.log(THETA)))
    hi = math.ceil(hd * math.log(YARN_CTX / (BETA_SLOW * 2 * math.pi)) / (2 * math.log(THETA)))
    lo, hi = max(lo, 0), min(hi, hd - 1)
    out = []
    for i, x in enumerate(f):
        r = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
        out.append(x / YARN_FACTOR * r + x * (1.0 - r))
    return out, 0.1 * math.log(YARN_FACTOR) + 1.0


def _prep_plain(s):
    nq, nkv, hd, page = s["nq"], s["nkv"], s["hd"], s["page"]
    y, M = s["y"], s["y"].shape[0]
    f, factor = _frequencies(hd, s["full"])
    angle = s["pos"].double()[:, None] * torch.tensor(f, dtype=torch.float64, device=DEV)[None, :]
    cos, sin = (torch.cos(angle) * factor).float()[:, None, :], (torch.sin(angle) * factor).float()[:, None, :]

    def norm_rotate(x, gain, heads):
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain
        x = x.view(M, heads, hd)
        a, b = x[..., :hd // 2], x[..., hd // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(torch.bfloat16)

    q = norm_rotate(y[:, :nq * hd], s["q_gain"], nq)
    k = norm_rotate(y[:, nq * hd:(nq + nkv) * hd], s["k_gain"], nkv)
    v = y[:, (nq + nkv) * hd:].reshape(M, nkv, hd).to(torch.bfloat16)
    rows = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"][rows].long()
    s["q"][rows] = q[rows]
    s["k"][at // page, :, at % page] = k[rows]
    s["v"][at // page, :, at % page] = v[rows]
    return s["q"], s["k"], s["v"]


def _rows_of(pages, table, n, dtype):
    """The first n positions of a page list, [n_kv, n, hd]."""
    page = pages.shape[2]
    x = pages[table[:_pages(n, page)].long()].to(dtype)
    return x.transpose(0, 1).reshape(pages.shape[1], -1, pages.shape[3])[:, :n]


def _attn_plain(s):
    nq, nkv, hd, P, W = s["nq"], s["nkv"], s["hd"], s["prefix"], s["window"]
    g, scale = nq // nkv, 1.0 / math.sqrt(hd)
    kp, vp = (_rows_of(s[x], s["prefix_table"], P, torch.float32) for x in ("k", "v"))
    out = torch.empty_like(s["q"])
    for b, n in enumerate(s["host_lens"]):
        r0, r1 = s["host_start"][b], s["host_start"][b + 1]
        ko, vo = (_rows_of(s[x], s["table"][b], n, torch.float32) for x in ("k", "v"))
        for c0 in range(r0, r1, 1024):
            c1 = min(r1, c0 + 1024)
            q = s["q"][c0:c1].float().view(c1 - c0, nkv, g, hd).permute(1, 2, 0, 3).reshape(nkv, -1, hd)
            sc = torch.cat([q @ kp.transpose(1, 2), q @ ko.transpose(1, 2)], -1) * scale
            p = P + n - (r1 - r0) + torch.arange(c0 - r0, c1 - r0, device=DEV)
            key = torch.arange(P + n, device=DEV)
            hidden = key[None, :] > p[:, None]
            if W:
                hidden |= key[None, :] <= p[:, None] - W
            sc.masked_fill_(hidden.repeat(g, 1)[None], float("-inf"))
            e = torch.exp(sc - sc.amax(-1, keepdim=True))
            o = (e[..., :P] @ vp + e[..., P:] @ vo) / e.sum(-1, keepdim=True)
            out[c0:c1] = o.view(nkv, g, c1 - c0, hd).permute(2, 0, 1, 3).reshape(c1 - c0, nq, hd).to(out.dtype)
    return out


def run(state):
    s = state
    if not own:
        return {"plan": _plan_plain, "prep": _prep_plain, "attn": _attn_plain}[s["op"]](s)
    from w4_weight_only_b200 import api
    if s["op"] == "plan":
        p = api.paged_plan(s["new"], s["lens"], s["state"], s["queue"], s["table"], s["page"], s["rows"],
                           prefix_len=s["prefix"], ws=s["ws"])
        return (p.lens, p.state, p.row_start, p.slots, p.pos, s["table"], s["queue"])
    if s["op"] == "prep":
        q = api.qk_prep_paged(s["cfg"], s["full"], s["y"], s["q_gain"], s["k_gain"], s["pos"], s["slots"], s["k"],
                              s["v"], ws=s["ws"], q_out=s["q"])
        return q, s["k"], s["v"]
    return api.attn_shared(s["q"], s["k"], s["v"], s["row_start"], s["lens"], s["table"], s["prefix_table"],
                           s["prefix"], window=s["window"], max_new=s["new"], ws=s["ws"], out=s["out"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _plan_exact(s):
    page, queue, N = s["page"], s["queue"].tolist(), s["queue"].numel()
    table, lens, new = s["table"].tolist(), s["lens"].tolist(), s["new"].tolist()
    head, count = s["state"].tolist()
    for b, k in enumerate(new):              # ended sequences give their pages back
        if k < 0:
            for j in range(_pages(lens[b], page)):
                queue[(head + count) % N] = table[b][j]
                count += 1
    out_lens, start, slots, pos = [], [0], [], []
    for b, k in enumerate(new):
        n = lens[b]
        for i in range(max(k, 0)):
            if (n + i) % page == 0:          # the position opens a page
                table[b][(n + i) // page] = queue[head]
                head, count = (head + 1) % N, count - 1
            slots.append(table[b][(n + i) // page] * page + (n + i) % page)
            pos.append(s["prefix"] + n + i)
        out_lens.append(n + k if k >= 0 else 0)
        start.append(start[-1] + max(k, 0))
    pad = [-1] * (s["rows"] - len(slots))
    return tuple(_i32(x) for x in (out_lens, [head, count], start, slots + pad, pos + pad, table, queue))


def _prep_exact(s):
    nq, nkv, hd, page = s["nq"], s["nkv"], s["hd"], s["page"]
    f, factor = _frequencies(hd, s["full"])
    turn = torch.polar(torch.full((hd // 2,), factor, dtype=torch.float64, device=DEV)[None, :].expand(len(s["pos"]), -1),
                       s["pos"].double()[:, None] * torch.tensor(f, dtype=torch.float64, device=DEV))
    y = s["y"].double()
    q, k, v = torch.split(y, [nq * hd, nkv * hd, nkv * hd], 1)

    def form(x, gain, heads):
        x = (x / torch.sqrt(x.square().mean(1, keepdim=True) + EPS) * gain.double()).view(-1, heads, 2, hd // 2)
        z = torch.complex(x[:, :, 0], x[:, :, 1]) * turn[:, None]
        return torch.cat([z.real, z.imag], -1)

    q, k, v = form(q, s["q_gain"], nq), form(k, s["k_gain"], nkv), v.reshape(-1, nkv, hd)
    kk, vv, qq = (s[x].double() for x in ("k", "v", "q"))
    live = s["slots"] >= 0
    at = s["slots"][live].long()
    qq[live] = q[live]
    flat = lambda t: t.transpose(1, 2).reshape(-1, nkv, hd)
    kf, vf = flat(kk), flat(vv)
    kf[at], vf[at] = k[live], v[live]
    back = lambda t: t.view(-1, page, nkv, hd).transpose(1, 2)
    return qq, back(kf), back(vf)


def _attn_exact(s):
    nq, nkv, hd, P, W, page = s["nq"], s["nkv"], s["hd"], s["prefix"], s["window"], s["page"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["host_lens"]):
        r0, r1 = s["host_start"][b], s["host_start"][b + 1]
        # every position's page and place in it
        i, j = torch.arange(P, device=DEV), torch.arange(n, device=DEV)
        pg = torch.cat([s["prefix_table"][i // page], s["table"][b][j // page]]).long()
        at = torch.cat([i % page, j % page])
        p = torch.arange(P + n - (r1 - r0), P + n, device=DEV)
        for c in range(nkv):
            k, v = s["k"][pg, c, at].double(), s["v"][pg, c, at].double()
            for h in range(c * (nq // nkv), (c + 1) * (nq // nkv)):
                for t in range(0, r1 - r0, 2048):
                    pt = p[t:t + 2048]
                    z = s["q"][r0 + t:r0 + t + len(pt), h].double() @ k.T / math.sqrt(hd)
                    seen = torch.arange(P + n, device=DEV)[None] <= pt[:, None]
                    if W:
                        seen &= torch.arange(P + n, device=DEV)[None] > pt[:, None] - W
                    z = torch.where(seen, z, torch.full_like(z, float("-inf")))
                    out[r0 + t:r0 + t + len(pt), h] = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)) @ v
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    return {"plan": _plan_exact, "prep": _prep_exact, "attn": _attn_exact}[case["op"]](s)
