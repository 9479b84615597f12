"""Plain 64-bit references of the paged key-value cache's operators: the step's plan (one sequence after the other, on
lists), rotary positions, and attention of one sequence and head at a time."""
from __future__ import annotations

import math

import numpy as np

HALF_STEP = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}    # relative, of one rounding
TINY = {"bfloat16": 2.0 ** -134, "float16": 2.0 ** -25}       # half a subnormal step
ERR_CAPACITY, ERR_PAGE = 0x4, 0x20


def pages(n, page):
    return -(-n // page)


def plan(page, cached, new, table, free, count, rows):
    """fp4moe_kv_plan's outputs as lists, and the error bits."""
    B, columns, num_pages = len(cached), len(table[0]) if table else 0, len(free)
    table, free, err = [list(r) for r in table], list(free), 0
    limit = min(columns * page, 2 ** 31 - 1 - page)
    c, a, first, refused = [], [], [0], []
    for b in range(B):
        x = min(max(cached[b], 0), limit)
        err |= ERR_PAGE * (x != cached[b])
        y = x + new[b]
        err |= ERR_PAGE * (y < 0)
        c.append(x)
        a.append(max(y, 0))
        first.append(first[-1] + max(new[b], 0))
        refused.append(y > limit or (new[b] > 0 and first[-1] > rows))
        err |= ERR_CAPACITY * refused[-1]
    F = min(max(count, 0), num_pages)
    err |= ERR_PAGE * (F != count)
    stack = free[:F]
    for b in range(B):
        if a[b] < c[b]:
            stack += table[b][pages(a[b], page):pages(c[b], page)]
    err |= ERR_PAGE * (len(stack) > num_pages)
    stack, closed = stack[:num_pages], False
    for b in range(B):
        need = 0 if refused[b] or a[b] <= c[b] else pages(a[b], page) - pages(c[b], page)
        if need and (closed or need > len(stack)):
            closed = refused[b] = True
            err |= ERR_CAPACITY
        elif need:
            for j in range(pages(c[b], page), pages(a[b], page)):
                table[b][j] = stack.pop()
    position, slot = [0] * rows, [-1] * rows
    for b in range(B):
        for i in range(max(new[b], 0)):
            t = first[b] + i
            if t >= rows:
                break
            position[t] = min(c[b] + i, 2 ** 31 - 1)
            if not refused[b]:
                p = table[b][position[t] // page]
                if 0 <= p < num_pages:
                    slot[t] = p * page + position[t] % page
                else:
                    err |= ERR_PAGE
    kv_len = [c[b] if refused[b] else a[b] for b in range(B)]
    return {"table": table, "free": stack + free[len(stack):], "count": [len(stack)], "kv_len": kv_len,
            "q_offset": [min(f, rows) for f in first], "position": position, "slot": slot}, err


def rotate(x, position, inv_freq, first, interleaved, amplitude):
    """fp64 x [T, heads, D] turned, and for each element the magnitude |x| + |y| that its roundings go by."""
    half = len(inv_freq)
    ang = position.astype(np.float64)[:, None] * inv_freq[None, :]
    cos, sin = np.cos(ang)[:, None] * amplitude, np.sin(ang)[:, None] * amplitude
    i = np.arange(half)
    p, q = (first + 2 * i, first + 2 * i + 1) if interleaved else (first + i, first + i + half)
    out, mag = x.copy(), np.zeros_like(x)
    u, v = x[..., p], x[..., q]
    out[..., p], out[..., q] = u * cos - v * sin, v * cos + u * sin
    mag[..., p] = mag[..., q] = np.abs(u) + np.abs(v)
    return out, mag


def attention(q, k, v, slots, first, new, kv, scale, causal, window):
    """fp64 (out, lse, the sum of weighted |v|, the largest sum of |q k| scale of a row) of packed rows.

    q [T, H, D]; k, v [slots, Hk, D]; slots[b]: the slot of each key of sequence b (a torch tensor; -1: zeros)."""
    import torch
    T, H, D = q.shape
    G = H // k.shape[1]
    q = q.double()
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=q.device)
    top = torch.zeros(T, H, dtype=torch.float64, device=q.device)
    for b in range(len(new)):
        n, L = new[b], len(slots[b])
        if n == 0 or L == 0:
            continue
        j = torch.arange(L, device=q.device)
        pos = kv[b] - n + torch.arange(n, device=q.device)
        see = (j[None] <= pos[:, None]) if causal else torch.ones(n, L, dtype=torch.bool, device=q.device)
        if window:
            see &= j[None] > pos[:, None] - window
        hole = (slots[b] < 0)[:, None, None]
        kb, vb = (torch.where(hole, 0.0, x[slots[b].clamp(min=0)].double()) for x in (k, v))
        for h in range(H):
            qh = q[first[b]:first[b] + n, h]
            s = torch.where(see, qh @ kb[:, h // G].t() * scale, -math.inf)
            any_key = see.any(1)
            m = s.amax(1, keepdim=True)
            e = torch.where(see, torch.exp(s - m), 0.0)
            l = e.sum(1, keepdim=True)
            # keys that a row does not see must not reach it: 0 * inf is left out, key by key where v is not finite
            vf = torch.where(torch.isfinite(vb[:, h // G]), vb[:, h // G], 0.0)
            o = e @ vf
            for jj in torch.nonzero(~torch.isfinite(vb[:, h // G]).all(1)).flatten().tolist():
                bad = torch.where(torch.isfinite(vb[jj, h // G]), 0.0, vb[jj, h // G])
                o = torch.where(see[:, jj:jj + 1], o + e[:, jj:jj + 1] * bad, o)
            rows = slice(first[b], first[b] + n)
            out[rows, h] = torch.where(any_key[:, None], o / l, 0.0)
            mag[rows, h] = torch.where(any_key[:, None], (e @ vf.abs()) / l, 0.0)
            lse[rows, h] = torch.where(any_key, (m + torch.log(l))[:, 0], -math.inf)
            top[rows, h] = torch.where(see, qh.abs() @ kb[:, h // G].abs().t() * scale, 0.0).amax(1)
    return out, lse, mag, top
