"""Paged caches in plain float64 NumPy with explicit loops.

``page_plan`` walks the requests and keeps the free pages as a Python list,
``page_write`` copies row by row, ``paged_attention`` forms every row's scores
and softmax on its own.  No code is shared with the library.
"""
from __future__ import annotations

import math

import numpy as np

PLAN_OK, PLAN_NO_PAGES, PLAN_ROW_FULL, PLAN_INVALID, PLAN_TOKENS = range(5)


def page_plan(page_size, new_lens, kv_lens, block_table, free_pages, n_free, max_tokens):
    """Returns kv_lens, block_table, free_pages, n_free, q_start, slots,
    positions and status after a plan of the step."""
    B = page_size
    table = np.array(block_table, dtype=np.int64)
    R, width = table.shape
    blocks = lambda n: -(-n // B)  # noqa: E731
    invalid = [n < -1 or c < 0 or c > width * B for n, c in zip(new_lens, kv_lens)]
    stack = [int(p) for p in free_pages[:n_free]]
    for r in range(R):
        if not invalid[r] and new_lens[r] == -1:
            stack.extend(int(table[r, b]) for b in range(blocks(int(kv_lens[r]))))
    kv = [int(c) for c in kv_lens]
    status = [PLAN_OK] * R
    q_start, tokens = [0], 0
    slots = np.full(max_tokens, -1, dtype=np.int64)
    positions = np.full(max_tokens, -1, dtype=np.int64)
    dry = False
    for r in range(R):
        n, c = int(new_lens[r]), int(kv_lens[r])
        first = tokens
        if invalid[r]:
            status[r] = PLAN_INVALID
        elif n == -1:
            kv[r] = 0
        else:
            tokens += n
            need = blocks(c + n) - blocks(c)
            if c + n > width * B:
                status[r] = PLAN_ROW_FULL
            elif n > 0 and tokens > max_tokens:
                status[r] = PLAN_TOKENS
            elif need > 0 and (dry or need > len(stack)):
                status[r] = PLAN_NO_PAGES
                dry = True
            else:
                for b in range(blocks(c), blocks(c + n)):
                    table[r, b] = stack.pop()
                for t in range(n):
                    p = c + t
                    slots[first + t] = table[r, p // B] * B + p % B
                    positions[first + t] = p
                kv[r] = c + n
        q_start.append(min(tokens, max_tokens))
    out_free = np.array(free_pages, dtype=np.int64)
    for i in range(n_free, len(stack)):
        out_free[i] = stack[i]
    return dict(kv_lens=np.array(kv), block_table=table, free_pages=out_free, n_free=len(stack),
                q_start=np.array(q_start), slots=slots, positions=positions,
                status=np.array(status))


def page_write(src, slots, pool, layer=0):
    """Rows of src [n, nl, H, T, d] into a copy of pool [P, L, H, B, d]."""
    out = np.array(pool)
    P, _, _, B, _ = out.shape
    n, nl, _, T, _ = src.shape
    for r in range(n):
        for t in range(T):
            s = int(slots[r, t])
            if 0 <= s < P * B:
                out[s // B, layer:layer + nl, :, s % B, :] = src[r, :, :, t, :]
    return out


def paged_attention(q, pool_K, pool_V, block_table, q_start, kv_lens, scale, layer=0, causal=True,
                    window=0):
    """(out [N, Hq, d], lse [N, Hq], mass [N, Hq, d], reach [N, Hq]) in float64.

    mass = sum_j p_j |v_j| and reach = max_j scale sum_i |q_i k_ij| over the
    keys in sight are what rounding errors are proportional to.  Rows of no
    request are NaN."""
    q = np.asarray(q, dtype=np.float64)
    N, Hq, d = q.shape
    H, B = pool_K.shape[2], pool_K.shape[3]
    G = Hq // H
    out = np.full((N, Hq, d), np.nan)
    lse = np.full((N, Hq), np.nan)
    mass = np.full((N, Hq, d), np.nan)
    reach = np.zeros((N, Hq))
    for r in range(len(kv_lens)):
        kv, a, b = int(kv_lens[r]), int(q_start[r]), int(q_start[r + 1])
        pages = [int(p) for p in block_table[r][:-(-kv // B)]]
        for h in range(H):
            rows = lambda pool: (np.concatenate([pool[p, layer, h] for p in pages])[:kv]  # noqa: E731
                                 if pages else np.zeros((0, d))).astype(np.float64)
            K, V = rows(pool_K), rows(pool_V)
            for i in range(b - a):
                pos = kv - (b - a) + i
                hi = min(kv, pos + 1) if causal else kv
                lo = max(0, pos - window + 1) if window else 0
                for e in range(h * G, h * G + G):
                    if hi <= lo:
                        out[a + i, e] = mass[a + i, e] = 0.0
                        lse[a + i, e] = -math.inf
                        continue
                    x = scale * (K[lo:hi] @ q[a + i, e])
                    top = x.max()
                    p = np.exp(x - top)
                    lse[a + i, e] = top + math.log(p.sum())
                    p /= p.sum()
                    out[a + i, e] = p @ V[lo:hi]
                    mass[a + i, e] = p @ np.abs(V[lo:hi])
                    reach[a + i, e] = scale * (np.abs(K[lo:hi]) @ np.abs(q[a + i, e])).max()
    return out, lse, mass, reach
