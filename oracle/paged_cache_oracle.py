"""Plain CPU implementation of the paged-cache operators (test infrastructure): Python
integers for the step plan and the moves, fp64 for the attention. Shares no code with
the CUDA path."""
from __future__ import annotations

import math

import torch


def plan(lens, new, held, nfree, free, table, parents, page, n, words):
    """The step plan on Python lists. Returns a dict of the call's outputs; `table` and
    `free` are new lists. parents None with words > 0 is a chain."""
    R, width, pages = len(lens), len(table[0]), len(free)
    table, free = [list(row) for row in table], list(free)
    top = nfree
    for r in range(R):                                   # returns, in request order
        if new[r] < 0 and 0 <= held[r] <= width:
            for j in range(held[r]):
                if top < pages:
                    free[top] = table[r][j]
                top += 1
    top = min(top, pages)
    starts, row = [], 0
    for r in range(R):
        starts.append(min(row, n))
        row += max(new[r], 0)
    starts.append(min(row, n))
    granted, held_out = [0] * R, list(held)
    asked, taken = 0, 0
    row = 0
    valid = [False] * R
    for r in range(R):
        T = new[r]
        if T < 0:
            held_out[r] = 0
            continue
        row += T
        want = -(-(lens[r] + T) // page)
        if not (0 <= held[r] <= width) or lens[r] < 0 or want > width or lens[r] > held[r] * page \
                or (words and T > 32 * words) or (T > 0 and row > n):
            continue
        valid[r] = True
        need = max(0, want - held[r])
        asked += need
        if need and asked > top:
            continue
        for j in range(need):
            table[r][held[r] + j] = free[top - 1 - (asked - need + j)]
        if need:
            taken = asked
        held_out[r] = held[r] + need
        granted[r] = T
    slots, positions, mask = [-1] * n, [0] * n, [[0] * words for _ in range(n)]
    for r in range(R):
        for t in range(starts[r + 1] - starts[r]):
            i = starts[r] + t
            depth = t
            if words and valid[r]:
                node, depth, bits = t, -1, 0
                while node >= 0:
                    bits |= 1 << node
                    depth += 1
                    up = node - 1 if parents is None else parents[starts[r] + node]
                    if up >= node or up < -1:
                        break
                    node = up
                for w in range(words):
                    x = (bits >> (32 * w)) & 0xffffffff
                    mask[i][w] = x - (1 << 32) if x >> 31 else x
            positions[i] = lens[r] + depth
            if granted[r] > 0:
                place = lens[r] + t
                slots[i] = table[r][place // page] * page + place % page
    return dict(table=table, free_pages=free, held=held_out, nfree=[top - taken], starts=starts, granted=granted,
                slots=slots, positions=positions, mask=mask)


def visible(mask_row, t, T):
    """Which of a request's T new tokens its token t sees (mask_row: words, or None)."""
    if mask_row is None:
        return [j <= t for j in range(T)]
    return [bool((int(mask_row[j // 32]) >> (j % 32)) & 1) for j in range(T)]


def tree_attention(q, k_cache, v_cache, table, lens, starts, counts, mask, scale):
    """o, lse and the weighted mean of |v| (for error bounds) of every existing row, fp64
    on the CPU; other rows are NaN. Only visible tokens are ever touched."""
    n, Hq, d = q.shape
    page, Hkv = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hkv
    o = torch.full((n, Hq, d), math.nan, dtype=torch.float64)
    a = torch.zeros(n, Hq, d, dtype=torch.float64)
    lse = torch.full((n, Hq), math.nan, dtype=torch.float64)
    smax = torch.zeros(n, Hq, dtype=torch.float64)
    for r, (L, T) in enumerate(zip(lens, counts)):
        for t in range(T):
            i = starts[r] + t
            see = list(range(L)) + [L + j for j, x in enumerate(visible(None if mask is None else mask[i], t, T)) if x]
            if not see:
                o[i] = 0
                lse[i] = -math.inf
                continue
            at = torch.tensor(see)
            ids, off = torch.tensor(table[r])[at // page].long(), at % page
            k = k_cache[ids, off].double().repeat_interleave(G, 1)          # [keys, Hq, d]
            v = v_cache[ids, off].double().repeat_interleave(G, 1)
            s = torch.einsum("hd,khd->hk", q[i].double(), k) * scale
            lse[i] = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[i][:, None])
            o[i] = torch.einsum("hk,khd->hd", p, v)
            a[i] = torch.einsum("hk,khd->hd", p, v.abs())
            smax[i] = (torch.einsum("hd,khd->hk", q[i].double().abs(), k.abs()) * scale).amax(1)
    return o, lse, a, smax


def accept(cache, table, lens, accepted, taken):
    """A copy of cache [..., pages, page, H, d] with each request's accepted rows moved."""
    out = cache.clone()
    page = cache.shape[-3]
    for r, L in enumerate(lens):
        for i in range(taken[r]):
            s, t = L + accepted[r][i], L + i
            out[..., table[r][t // page], t % page, :, :] = cache[..., table[r][s // page], s % page, :, :]
    return out
