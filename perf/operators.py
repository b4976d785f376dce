"""The paged-cache operators as a serving loop calls them, and their plain forms.

``kvc_page_plan`` (block tables, slot maps and positions of a step's new
tokens), ``kvc_page_write`` (rows of K and V into their pages) and
``kvc_paged_attention`` (a chunk of new tokens, down to one, over the paged
cache).  ``listed()`` gives the cases that are measured, ``draw()`` more of
the same ranges; ``run()`` makes one pass, with the library's calls where
``own`` is true and with elementary torch operations in 32 bits where it is
not.
"""
from __future__ import annotations

import math
import random

import torch

own = False

# status of a request in the plan
OK, NO_PAGES, ROW_FULL, INVALID, TOO_MANY = 0, 1, 2, 3, 4


# ------------------------------------------------------------------- cases
def _plan(name, R, new, kv, page, **kw):
    c = {"name": name, "op": "plan", "R": R, "new": new, "kv": kv, "page": page, "ragged": False,
         "released": 0, "short": False}
    c.update(kw)
    return c


def _write(name, R, T, layers, heads, d, page, dtype="bf16", **kw):
    c = {"name": name, "op": "write", "R": R, "T": T, "layers": layers, "heads": heads, "d": d,
         "page": page, "dtype": dtype, "packed": False, "skipped": False}
    c.update(kw)
    return c


def _attend(name, R, new, kv, q_heads, heads, d, page, dtype="bf16", **kw):
    c = {"name": name, "op": "attend", "R": R, "new": new, "kv": kv, "q_heads": q_heads,
         "heads": heads, "d": d, "page": page, "dtype": dtype, "ragged": False, "causal": True,
         "window": 0}
    c.update(kw)
    return c


def listed():
    return [
        # one decoding step of sixteen agents, each 10,240 tokens into its trajectory
        _plan("plan_step", 16, 1, 10240, 64),
        # a busy server: a thousand requests, prompts of all lengths admitted, some finished
        _plan("plan_admit", 1024, 1024, 2048, 16, ragged=True, released=100),
        # the step's keys and values of one layer
        _write("write_step", 16, 1, 1, 8, 128, 64, packed=True),
        # sixteen agents' 128-token prefixes, one layer, in the projection's token-major layout
        _write("write_prefix", 16, 128, 1, 8, 128, 64, packed=True),
        # two corrected trajectories of 10,240 tokens, all layers, leave the chain for the pool
        _write("write_context", 2, 10240, 32, 8, 128, 128),
        # one short request decodes alone: latency
        _attend("attend_one", 1, 1, 777, 32, 8, 128, 16),
        # sixteen agents decode over 10,240-token trajectories
        _attend("attend_step", 16, 1, 10240, 32, 8, 128, 64),
        # one very long request decodes: the work is along one axis
        _attend("attend_long", 1, 1, 131072, 32, 8, 128, 128),
        # sixteen agents' 128-token prefixes over the shared context
        _attend("attend_prefix", 16, 128, 10368, 32, 8, 128, 64),
        # dense prefill of two 8,192-token contexts
        _attend("attend_prefill", 2, 8192, 8192, 32, 8, 128, 128),
        # ragged chunks of a 9,000-token vision-language trajectory: 7 query heads on each KV
        # head, pages that do not divide a tile, a sliding window
        _attend("attend_ragged", 5, 700, 9000, 28, 4, 128, 48, ragged=True, window=4096),
        # fp32 caches of small heads, ragged
        _attend("attend_f32", 6, 65, 2000, 8, 2, 64, 20, dtype="f32", ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["plan", "write", "attend", "attend", "attend"])
    limits = {k: max(_cost(c) for c in listed() if c["op"] == k) for k in ("plan", "write", "attend")}
    page = rng.choice([8, 16, 16, 17, 20, 32, 48, 64, 64, 100, 128, 256])
    while True:
        if kind == "plan":
            R = _log_int(rng, 1, 1024)
            c = _plan("", R, _log_int(rng, 1, 4096), _log_int(rng, 1, 16384), page, ragged=True,
                      released=rng.randint(0, R // 4), short=rng.random() < 0.3)
        elif kind == "write":
            dtype = rng.choice(["bf16", "bf16", "f32"])
            c = _write("", _log_int(rng, 1, 64), _log_int(rng, 1, 10240), rng.choice([1, 1, 4, 28, 32]),
                       rng.choice([1, 2, 4, 8]), rng.choice([64, 128] if dtype == "bf16" else [32, 64, 80]),
                       page, dtype=dtype, packed=rng.random() < 0.5, skipped=rng.random() < 0.5)
        elif rng.random() < 0.2:
            c = _attend("", _log_int(rng, 1, 16), _log_int(rng, 1, 300), _log_int(rng, 1, 5000),
                        0, rng.choice([1, 2, 4]), rng.choice([32, 64, 80, 128]), page, dtype="f32",
                        ragged=True, causal=rng.random() < 0.8)
            c["q_heads"] = c["heads"] * rng.choice([1, 2, 4])
        else:
            c = _attend("", _log_int(rng, 1, 64), rng.choice([1, _log_int(rng, 1, 8192)]),
                        _log_int(rng, 1, 131072), 0, rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128]),
                        page, ragged=rng.random() < 0.7, causal=rng.random() < 0.9)
            c["q_heads"] = c["heads"] * rng.choice([1, 2, 4, 4, 7, 8])
            if c["causal"] and rng.random() < 0.25:
                c["window"] = _log_int(rng, 16, 8192)
        if c["op"] == "attend":
            c["kv"] = max(c["kv"], c["new"])
        if _cost(c) <= limits[c["op"]]:
            break
    del c["name"]
    return c


def _cost(c):
    """Seconds, roughly, of the plain form's dense arithmetic or traffic."""
    if c["op"] == "plan":
        return float(c["R"] * (c["new"] + (c["new"] + c["kv"]) // c["page"]))
    if c["op"] == "write":
        return float(c["R"] * c["T"] * c["layers"] * c["heads"] * c["d"] * _size(c))
    pairs = c["R"] * c["q_heads"] * c["new"] * c["kv"]
    rows = c["R"] * c["heads"] * c["kv"]
    return pairs * c["d"] * 4 / 4e13 + pairs * 24 / 4e12 + rows * c["d"] * 24 / 4e12


def _size(c):
    return 2 if c["dtype"] == "bf16" else 4


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _lengths(c):
    """(new tokens, cached tokens before the step) of every request.  They are the
    case's own: the seed changes values and pages, not the amount of work."""
    rng = random.Random(7 * c["R"] + 3 * c["new"] + c["kv"])
    new, kv = [], []
    for r in range(c["R"]):
        n = rng.randint(1, c["new"]) if c["ragged"] else c["new"]
        t = rng.randint(1, c["kv"]) if c["ragged"] else c["kv"]
        if c["op"] == "attend":                # kv counts the new tokens
            t = max(t, n) - n
        new.append(n)
        kv.append(t)
    if c["op"] == "plan":
        for r in rng.sample(range(c["R"]), c["released"]):
            new[r] = -1
    return new, kv


def _pages(n, page):
    return -(-n // page)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    make = {"plan": _prepare_plan, "write": _prepare_write, "attend": _prepare_attend}[case["op"]]
    s = make(case, g)
    s["case"] = case
    if own:
        _handles(case, s)
    return s


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _table(counts, width, perm):
    """[R, width] table of the first pages of ``perm``, ``counts[r]`` to a row, -1 beyond."""
    cnt = torch.tensor(counts, device="cuda")
    first = torch.cumsum(cnt, 0) - cnt
    col = torch.arange(width, device="cuda")
    idx = (first[:, None] + col).clamp(max=perm.numel() - 1)
    return torch.where(col < cnt[:, None], perm[idx], perm.new_full((), -1)).to(torch.int32)


def _prepare_plan(c, g):
    B, R = c["page"], c["R"]
    new, kv = _lengths(c)
    held = [_pages(t, B) for t in kv]
    need = [_pages(t + max(n, 0), B) - _pages(t, B) for n, t in zip(new, kv)]
    back = sum(h for h, n in zip(held, new) if n < 0)
    spare = max(0, sum(need) - back) + (-(sum(need) // 3) if c["short"] else 8)
    n_free = max(0, spare)
    P = sum(held) + n_free
    width = max(_pages(t + max(n, 0), B) for n, t in zip(new, kv))
    perm = torch.randperm(P, generator=g, device="cuda")
    free = torch.full((P,), -1, dtype=torch.int32, device="cuda")
    free[:n_free] = perm[sum(held):].to(torch.int32)
    total = sum(max(n, 0) for n in new)
    e = lambda n, t: torch.empty(n, dtype=t, device="cuda")  # noqa: E731
    return {"P": P, "width": width, "tokens": total, "new": _i32(new), "kv": _i32(kv),
            "table": _table(held, width, perm), "free": free, "n_free": _i32([n_free]),
            "out": {"kv_lens": e(R, torch.int32), "n_free": e(1, torch.int32),
                    "q_start": e(R + 1, torch.int32), "slots": e(total, torch.int64),
                    "positions": e(total, torch.int32), "status": e(R, torch.int32)}}


def _prepare_write(c, g):
    R, T, L, H, d, B = (c[k] for k in ("R", "T", "layers", "heads", "d", "page"))
    P = R * _pages(T, B) + 3
    dt = _dtype(c)
    rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=dt)  # noqa: E731
    # a projection leaves [tokens, heads, d] rows, the chain leaves [R, L, H, T, d] caches
    src = [rnd(R, L, T, H, d).permute(0, 1, 3, 2, 4) if c["packed"] else rnd(R, L, H, T, d)
           for _ in "KV"]
    perm = torch.randperm(P, generator=g, device="cuda")
    t = torch.arange(T, device="cuda")
    page = perm[(torch.arange(R, device="cuda")[:, None] * _pages(T, B) + t // B)]
    slots = page * B + t % B
    if c["skipped"]:
        hole = torch.rand((R, T), generator=g, device="cuda") < 0.2
        slots = torch.where(hole, torch.full_like(slots, -1), slots)
    pool = [torch.zeros((P, L, H, B, d), dtype=dt, device="cuda") for _ in "KV"]
    return {"P": P, "src": src, "slots": slots.contiguous(), "pool": pool}


def _prepare_attend(c, g):
    R, H, d, B = (c[k] for k in ("R", "heads", "d", "page"))
    new, before = _lengths(c)
    kv = [n + t for n, t in zip(new, before)]
    width = _pages(max(kv), B)
    P = sum(_pages(t, B) for t in kv) + 2
    dt = _dtype(c)
    rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=dt)  # noqa: E731
    perm = torch.randperm(P, generator=g, device="cuda")
    pool = [rnd(P, 2, H, B, d) for _ in "KV"]
    N = sum(new)
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    return {"P": P, "width": width, "tokens": N, "max_new": max(new), "max_kv": max(kv), "layer": 1,
            "q": 2 * rnd(N, c["q_heads"], d), "pool": pool, "scale": 1.0 / math.sqrt(d),
            "table": _table([_pages(t, B) for t in kv], width, perm), "q_start": _i32(start),
            "kv": _i32(kv), "out": torch.empty((N, c["q_heads"], d), dtype=dt, device="cuda"),
            "lse": torch.empty((N, c["q_heads"]), dtype=torch.float32, device="cuda")}


def _handles(c, s):
    """The descriptors and the workspace that a program keeps beside its buffers."""
    from agent_shared_context_gb300 import kvc
    s["kvc"] = kvc
    s["dev_status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if c["op"] == "plan":
        s["pg"] = kvc.paged(s["P"], c["page"], 1, 1, 64, "bf16", c["R"], s["width"])
    elif c["op"] == "write":
        s["pg"] = kvc.paged(s["P"], c["page"], c["layers"], c["heads"], c["d"], c["dtype"], c["R"], 1)
    else:
        s["pg"] = kvc.paged(s["P"], c["page"], 2, c["heads"], c["d"], c["dtype"], c["R"], s["width"])
        s["att"] = kvc.attn_params(s["q"], s["out"], s["layer"], scale=s["scale"], causal=c["causal"],
                                   window=c["window"])
        n = kvc.kvc_paged_attention_workspace(s["pg"], s["att"])
        s["workspace"] = torch.zeros(max(n, 256), dtype=torch.uint8, device="cuda")


# -------------------------------------------------------------------- runs
def run(s):
    c = s["case"]
    if own:
        return {"plan": _own_plan, "write": _own_write, "attend": _own_attend}[c["op"]](c, s)
    return {"plan": _plain_plan, "write": _plain_write, "attend": _plain_attend}[c["op"]](c, s)


def _own_plan(c, s):
    o = s["out"]
    s["kvc"].kvc_page_plan(s["pg"], s["new"], s["kv"], o["kv_lens"], s["table"], s["free"], s["n_free"],
                           o["n_free"], o["q_start"], o["slots"], o["positions"], o["status"])
    return dict(o, table=s["table"], free=s["free"])


def _own_write(c, s):
    s["kvc"].kvc_page_write(s["pg"], s["src"][0], s["src"][1], s["slots"], s["pool"][0], s["pool"][1])
    return s["pool"]


def _own_attend(c, s):
    s["kvc"].kvc_paged_attention(s["pg"], s["att"], s["q"], s["pool"][0], s["pool"][1], s["table"],
                                 s["q_start"], s["kv"], s["out"], s["workspace"], s["dev_status"],
                                 lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_plan(c, s):
    """Every step of the plan over all requests, blocks and tokens at once."""
    B, P, width, N, R = c["page"], s["P"], s["width"], s["tokens"], c["R"]
    new, kv, table, free = s["new"].long(), s["kv"].long(), s["table"].long(), s["free"].long()
    F = s["n_free"].long()
    bad = (new < -1) | (kv < 0) | (kv > width * B)
    gone = (new == -1) & ~bad
    n = torch.where(bad | gone, 0, new)
    end = torch.cumsum(n, 0)
    full = ~bad & (kv + n > width * B)
    many = ~bad & ~full & (n > 0) & (end > N)
    held = (kv + B - 1) // B
    need = torch.where(bad | gone | full | many, 0, (kv + n + B - 1) // B - held)
    back = torch.where(gone, held, 0)
    back_end = torch.cumsum(back, 0)
    avail = F + back_end[-1:]
    need_end = torch.cumsum(need, 0)
    short = (need > 0) & (need_end > avail)
    zero = torch.zeros_like(n)
    status = torch.where(bad, INVALID, torch.where(full, ROW_FULL, torch.where(many, TOO_MANY,
                         torch.where(short, NO_PAGES, zero))))
    need = torch.where(short, 0, need)
    taken = torch.cumsum(need, 0)
    kv_out = torch.where(gone, 0, torch.where(status == OK, kv + n, kv))
    n_free = avail - taken[-1:]
    # the stack once the released pages are on it
    col = torch.arange(width, device=kv.device)
    put = torch.where(gone[:, None] & (col < held[:, None]), F + (back_end - back)[:, None] + col, P)
    stack = torch.cat([torch.where(torch.arange(P, device=kv.device) < F, free, -1),
                       free.new_full((1,), -1)]).scatter(0, put.clamp(max=P).reshape(-1),
                                                         table.reshape(-1))
    k = col - held[:, None]
    pop = avail - 1 - ((taken - need)[:, None] + k)
    fresh = (k >= 0) & (k < need[:, None])
    table = torch.where(fresh, stack[pop.clamp(0, P)], table)
    at = torch.arange(P, device=kv.device)
    free = torch.where((at >= F) & (at < n_free), stack[:P], free)
    start = torch.cat([zero[:1], end]).clamp(max=N)
    tok = torch.arange(N, device=kv.device)
    r = torch.searchsorted(end, tok, right=True).clamp(max=R - 1)
    pos = kv[r] + tok - (end - n)[r]
    live = (tok < end[-1]) & (status[r] == OK)
    slot = table[r, (pos // B).clamp(max=width - 1)] * B + pos % B
    i32 = torch.int32
    return {"kv_lens": kv_out.to(i32), "n_free": n_free.to(i32), "q_start": start.to(i32),
            "slots": torch.where(live, slot, -1), "positions": torch.where(live, pos, -1).to(i32),
            "status": status.to(i32), "table": table.to(i32), "free": free.to(i32)}


def _plain_write(c, s):
    """Rows by advanced indexing; skipped rows go to a page of their own behind the pool."""
    B, P = c["page"], s["P"]
    slots = s["slots"].reshape(-1)
    if c["skipped"]:
        keep = slots >= 0
        slots = slots[keep]
    for pool, src in zip(s["pool"], s["src"]):
        rows = src.permute(0, 3, 1, 2, 4).reshape(-1, *src.shape[1:3], src.shape[4])
        rows = rows[keep] if c["skipped"] else rows
        pool[slots // B, :, :, slots % B] = rows
    return s["pool"]


def _plain_attend(c, s):
    """Softmax over the padded batch: gathered keys, all scores, one mask."""
    B, H, d, layer = c["page"], c["heads"], c["d"], s["layer"]
    G, nq, nk = c["q_heads"] // H, s["max_new"], s["max_kv"]
    start, kv = s["q_start"].long(), s["kv"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(nq, device=kv.device)
    j = torch.arange(nk, device=kv.device)
    R = kv.numel()
    page = s["table"].long()[:, j // B].clamp(min=0)
    live = j < kv[:, None]                                                  # [R, nk]
    k, v = (torch.where(live[:, None, :, None], p[:, layer].transpose(1, 2)[page, (j % B)[None]]
                        .permute(0, 2, 1, 3).float(), 0.0) for p in s["pool"])  # [R, H, nk, d]
    rows = (start[:-1, None] + i).clamp(max=s["tokens"] - 1)
    q = s["q"].float()[rows].view(R, nq, H, G, d).permute(0, 2, 3, 1, 4).reshape(R, H, G * nq, d)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(R, H, G, nq, nk)
    pos = (kv - n)[:, None] + i                                             # [R, nq]
    see = live[:, None, :].expand(R, nq, nk)
    if c["causal"]:
        see = see & (j <= pos[:, :, None])
    if c["window"]:
        see = see & (j > pos[:, :, None] - c["window"])
    x.masked_fill_(~see[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(R, H, G * nq, nk), v).view(R, H, G, nq, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + total.log()).squeeze(-1)
    tok = torch.arange(s["tokens"], device=kv.device)
    r = torch.searchsorted(start, tok, right=True) - 1
    t = tok - start[r]
    out = o[r, :, :, t].reshape(-1, H * G, d).to(_dtype(c))
    return {"out": out, "lse": lse[r, :, :, t].reshape(-1, H * G)}


# ------------------------------------------------------- exact values, work
def exact(case, seed):
    """The outputs in 64 bits.  A plan is whole numbers and has none."""
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    c = case
    B = c["page"]
    if c["op"] == "write":
        if c["R"] * c["T"] * c["layers"] * c["heads"] * c["d"] > 1 << 30:
            return None
        outs = []
        for pool, src in zip(s["pool"], s["src"]):
            flat = pool.double().permute(0, 3, 1, 2, 4).flatten(0, 1)
            for r in range(c["R"]):
                keep = (s["slots"][r] >= 0).nonzero()[:, 0]
                flat.index_copy_(0, s["slots"][r][keep], src[r].double().permute(2, 0, 1, 3)[keep])
            outs.append(flat.unflatten(0, (-1, B)).permute(0, 2, 3, 1, 4))
        return outs
    new, before = _lengths(c)
    if sum(n * (n + t) for n, t in zip(new, before)) * c["q_heads"] * c["d"] > 2.5e12:
        return None
    G = c["q_heads"] // c["heads"]
    out = torch.zeros((s["tokens"], c["q_heads"], c["d"]), dtype=torch.float64, device="cuda")
    lse = torch.full((s["tokens"], c["q_heads"]), -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for r, (n, t) in enumerate(zip(new, before)):
        pages = s["table"][r, :_pages(n + t, B)].long()
        j = torch.arange(n + t, device="cuda")
        for h in range(c["heads"]):
            k, v = (p[pages, s["layer"], h].reshape(-1, c["d"])[:n + t].double() for p in s["pool"])
            for a in range(0, n, 1024):
                b = min(n, a + 1024)
                pos = t + torch.arange(a, b, device="cuda")[:, None]
                dark = torch.zeros((b - a, n + t), dtype=torch.bool, device="cuda")
                if c["causal"]:
                    dark |= j > pos
                if c["window"]:
                    dark |= j <= pos - c["window"]
                for e in range(h * G, h * G + G):
                    x = (s["q"][first + a:first + b, e].double() @ k.T) * s["scale"]
                    x[dark] = -math.inf
                    z = torch.logsumexp(x, -1)
                    lse[first + a:first + b, e] = z
                    p = torch.exp(x - z[:, None])
                    out[first + a:first + b, e] = torch.nan_to_num(p, nan=0.0) @ v
        first += n
    return {"out": out, "lse": lse}


def work(case):
    c = case
    if c["op"] == "write":
        rows = 2 * c["R"] * c["T"] * c["layers"] * c["heads"]
        share = 0.8 if c["skipped"] else 1.0
        return {"bytes": int(share * rows * c["d"] * _size(c) * 2 + 8 * c["R"] * c["T"]), "flops": 0}
    new, before = _lengths(c)
    B = c["page"]
    if c["op"] == "plan":
        tokens = sum(max(n, 0) for n in new)
        fresh = sum(_pages(t + n, B) - _pages(t, B) for n, t in zip(new, before) if n > 0)
        back = sum(_pages(t, B) for n, t in zip(new, before) if n < 0)
        return {"bytes": 12 * tokens + 8 * max(fresh, back) + 24 * c["R"], "flops": 0}
    pairs, keys = 0, 0
    for n, t in zip(new, before):
        lo, w = 0, c["window"]
        if not c["causal"]:
            pairs += n * (n + t)
        elif not w:
            pairs += n * t + n * (n + 1) // 2
        else:
            pairs += sum(min(w, t + i + 1) for i in range(n))
            lo = max(0, t + 1 - w)
        keys += n + t - lo
    tokens, e = sum(new), _size(c)
    return {"bytes": 2 * keys * c["heads"] * c["d"] * e + tokens * c["q_heads"] * (2 * c["d"] * e + 4),
            "flops": 4 * pairs * c["q_heads"] * c["d"]}
