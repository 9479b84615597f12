"""Cases that time the attention half of a decoder block over a paged key-value cache, with their plain forms.

Three operators, one kind of case each:
  plan  page tables, positions and cache slots of a step's new tokens, from the lengths of its sequences
  rope  rotary positions of a step's q and k, and its k and v written into the paged cache
  attn  attention of each sequence's new tokens over its pages of the cache

The cache is [pages, page size, kv heads, head dim]; a slot is page * page size + place in the page. Sequence b's j-th
page is page_table[b, j]. New tokens of a step are packed: those of sequence b are rows q_offset[b] .. q_offset[b + 1].

The lengths of a case's sequences follow from the case, the rest of its inputs from the seed. The plain forms are
elementary torch operations in fp32 (angles in fp64), rounded once at the end.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
WORKSPACE = 64 << 20  # bytes that the attention call asks for, at any size


def _plan(name, B, page, cached, new, kind):
    return {"name": name, "op": "plan", "B": B, "page": page, "cached": cached, "new": new, "kind": kind}


def _rope(name, T, heads, kv_heads, D, rot, dtype, interleaved=False, first=0, far=8192, factor=1.0):
    return {"name": name, "op": "rope", "T": T, "heads": heads, "kv_heads": kv_heads, "D": D, "rot": rot, "first": first,
            "dtype": dtype, "interleaved": interleaved, "far": far, "factor": factor, "page": 64}


def _attn(name, B, new, kv, heads, kv_heads, D, dtype, page=64, window=0, causal=True, ragged=True):
    return {"name": name, "op": "attn", "B": B, "new": new, "kv": kv, "heads": heads, "kv_heads": kv_heads, "D": D,
            "dtype": dtype, "page": page, "window": window, "causal": causal, "ragged": ragged}


def listed():
    return [
        _plan("plan_decode", 64, 16, 8192, 1, "decode"),       # a decode batch of 64: one new token each
        _plan("plan_mixed", 512, 64, 16384, 512, "mixed"),     # chunks of prompts, decodes, finished and cut back sequences
        _rope("rope_token", 1, 32, 8, 128, 128, "bf16", far=131072),           # one sequence's next token, far out
        _rope("rope_prefill", 8192, 32, 8, 128, 128, "bf16"),                  # a prefill batch of 8192 tokens
        _rope("rope_odd_fp16", 1000, 12, 4, 96, 40, "fp16", True, 8, 131072, 8.0),  # part of the head, pairs side by side, scaled
        _attn("attn_token", 1, 1, 4096, 32, 8, 128, "bf16"),                   # one sequence's next token
        _attn("attn_decode", 64, 1, 8192, 32, 8, 128, "bf16"),                 # a ragged decode batch of 64
        _attn("attn_long", 4, 1, 131072, 32, 8, 128, "bf16", ragged=False),    # four sequences with long caches
        _attn("attn_verify", 16, 4, 8192, 64, 8, 64, "bf16", page=16),         # four proposed tokens for each of 16 sequences
        _attn("attn_chunk", 8, 512, 4096, 32, 8, 128, "bf16"),                 # prompt chunks behind ragged prefixes
        _attn("attn_prefill", 1, 8192, 8192, 32, 8, 128, "bf16", ragged=False),  # a whole prompt of 8192 tokens
        _attn("attn_odd_fp16", 5, 333, 2500, 6, 2, 80, "fp16", page=48, window=1000),  # odd everything, a sliding window
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "attn", "attn", "attn"])
    if op == "plan":
        B = _log_int(rng, 1, 1024)
        kind = rng.choice(["decode", "mixed"])
        new = 1 if kind == "decode" else _log_int(rng, 1, max(1, min(8192, 100000 // B)))
        cached = _log_int(rng, 1, min(32768, 16384 * 512 // B))
        return {"op": op, "B": B, "page": rng.choice([1, 16, 16, 48, 64, 64, 100, 128]), "cached": cached, "new": new,
                "kind": kind}
    kv_heads = rng.choice([1, 2, 4, 8, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "rope":
        D = rng.choice([32, 64, 80, 96, 128, 128, 128, 256])
        rot = rng.choice([D, D, D // 2, D // 4 + 2])
        first = rng.choice([0, 0, D - rot])
        T = _log_int(rng, 1, min(8192, 8192 * 48 * 128 // ((heads + 2 * kv_heads) * D)))
        return {"op": op, "T": T, "heads": heads, "kv_heads": kv_heads, "D": D, "rot": rot, "first": first, "dtype": dtype,
                "interleaved": rng.random() < 0.5, "far": _log_int(rng, 1024, 1000000),
                "factor": rng.choice([1.0, 1.0, 4.0, 32.0]), "page": rng.choice([1, 16, 48, 64, 128])}
    kind = rng.choice(["decode", "decode", "verify", "chunk", "chunk"])
    D = rng.choice([64, 64, 80, 96, 128, 128, 128, 128] + ([160, 256] if kind == "decode" else []))
    new = {"decode": 1, "verify": rng.randint(2, 8), "chunk": _log_int(rng, 16, 2048)}[kind]
    top = 131072 if kind == "decode" else 16384
    kv = _log_int(rng, max(1, new), top)
    B = _log_int(rng, 1, 128)
    most = min(4 * 131072 * 8 * 128 // (kv * kv_heads * D), 8192 * 8192 * 32 // (2 * heads * new * kv))
    causal = rng.random() < 0.85
    window = _log_int(rng, 16, 4096) if causal and rng.random() < 0.25 else 0
    return {"op": op, "B": max(1, min(B, most)), "new": new, "kv": kv, "heads": heads, "kv_heads": kv_heads, "D": D,
            "dtype": dtype, "page": rng.choice([1, 16, 16, 32, 48, 64, 64, 128, 256]), "window": window, "causal": causal,
            "ragged": rng.random() < 0.75}


# ------------------------------------------------------------------ what follows from the case alone
def _spread(B, lo, hi, ragged=True, shift=0.0):
    """B lengths in [lo, hi], spread evenly and out of order; the first is hi."""
    if not ragged:
        return [hi] * B
    return [hi] + [lo + int((hi - lo) * ((b * 0.6180339887498949 + shift) % 1.0)) for b in range(1, B)]


def _plan_lengths(c):
    """(cached lengths, new lengths) of a plan: in a mixed one, of each four sequences one decodes, one takes a chunk
    (or starts), one is finished and one gives back a few tokens."""
    B = c["B"]
    cached = _spread(B, c["cached"] // 8, c["cached"])
    if c["kind"] == "decode":
        return cached, [1] * B
    chunk = _spread(B, (c["new"] + 1) // 2, c["new"], shift=0.37)
    new = [(chunk[b], 1, -cached[b], -min(cached[b], 3))[b % 4] for b in range(B)]
    cached = [0 if b % 8 == 4 else cached[b] for b in range(B)]  # every second chunk is a sequence's first
    return cached, new


def _attn_lengths(c):
    """(new lengths, lengths with them) of the sequences."""
    new = _spread(c["B"], (c["new"] + 1) // 2, c["new"], c["ragged"], 0.37)
    kv = _spread(c["B"], max(c["kv"] // 4, 1), c["kv"], c["ragged"])
    return new, [max(n, k) if c["causal"] else k for n, k in zip(new, kv)]


def _pages(length, page):
    return -(-length // page)


def _visible(c, n, kv):
    """(number of visible (row, key) pairs of one head, number of keys that any row sees) of one sequence."""
    if not c["causal"]:
        return n * kv, kv
    w = c["window"] or kv
    pairs = sum(min(p + 1, w) for p in range(kv - n, kv))
    return pairs, kv - max(0, kv - n + 1 - w)


def work(case):
    c = case
    if c["op"] == "plan":  # both lengths in, length and offset out, pages taken or given back, positions and slots
        cached, new = _plan_lengths(c)
        moved = sum(abs(_pages(a + n, c["page"]) - _pages(a, c["page"])) for a, n in zip(cached, new))
        return {"bytes": 16 * c["B"] + 8 * moved + 8 * sum(max(n, 0) for n in new), "flops": 0}
    if c["op"] == "rope":
        n = c["T"] * (c["heads"] + 2 * c["kv_heads"]) * c["D"]
        return {"bytes": 4 * n + 8 * c["T"], "flops": 3 * c["T"] * (c["heads"] + c["kv_heads"]) * c["rot"]}
    new, kv = _attn_lengths(c)
    seen = [_visible(c, n, k) for n, k in zip(new, kv)]
    rows = sum(new) * c["heads"]
    bytes_ = rows * c["D"] * 4 + 4 * rows + sum(k for _, k in seen) * c["kv_heads"] * c["D"] * 4
    bytes_ += sum(4 * _pages(k, c["page"]) for k in kv)
    return {"bytes": bytes_, "flops": 4 * c["D"] * c["heads"] * sum(p for p, _ in seen)}


# ------------------------------------------------------------------ the cases' inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(gen, counts, columns, spare):
    """(page table [B, columns], the pages left over, number of pages): pages in random order, -1 behind a row's own."""
    total = sum(counts)
    order = torch.randperm(total + spare, device="cuda", generator=gen).to(torch.int32)
    first = torch.tensor([0] + counts, device="cuda").cumsum(0)[:-1]
    j = torch.arange(columns, device="cuda")[None, :]
    has = j < torch.tensor(counts, device="cuda")[:, None]
    table = torch.where(has, order[(first[:, None] + j).clamp(max=total + spare - 1)], torch.full_like(order[:1], -1))
    return table.contiguous(), order[total:].contiguous(), total + spare


def _inv_freq(rot, factor):
    """fp64 radians per position; slow pairs slowed by `factor`, in between a ramp (long contexts)."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = 10000.0 ** (-2.0 * i / rot)
    turns = 4096.0 * f / (2.0 * math.pi)  # in the length that the frequencies were made for
    keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * keep + f / factor * (1.0 - keep)


def prepare(case, seed):
    c = dict(case)
    gen = _generator(seed)
    s = {"case": c, "err": torch.zeros(4, dtype=torch.int32, device="cuda")}  # the kernels' error word
    if c["op"] == "plan":
        cached, new = _plan_lengths(c)
        counts = [_pages(a, c["page"]) for a in cached]
        columns = max(_pages(max(a, a + n), c["page"]) for a, n in zip(cached, new)) + 1
        need = sum(max(0, _pages(a + n, c["page"]) - k) for a, n, k in zip(cached, new, counts))
        s["table"], left, pages = _tables(gen, counts, columns, need + 64)
        s["free"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        s["free"][:left.numel()] = left
        s["free_count"], s["free_count_out"] = _ints([left.numel()]), _ints([0])
        s["cached"], s["new"] = _ints(cached), _ints(new)
        s["kv_len"], s["q_offset"] = torch.empty_like(s["cached"]), _ints([0] * (c["B"] + 1))
        room = max(64, _pages(sum(max(n, 0) for n in new), 64) * 64)  # the step's rows, as a captured graph pads them
        s["position"], s["slot"] = _ints([0] * room), _ints([0] * room)
        return s
    dtype = DTYPES[c["dtype"]]
    Hq, Hk, D, page = c["heads"], c["kv_heads"], c["D"], c["page"]
    if c["op"] == "rope":
        T = c["T"]
        s["qkv"] = torch.randn(T, (Hq + 2 * Hk) * D, device="cuda", generator=gen).to(dtype)  # a projection's rows
        pages = _pages(T, page) + 8
        shape = (pages, page, Hk, D)
        s["k_cache"], s["v_cache"] = (torch.zeros(shape, dtype=dtype, device="cuda") for _ in range(2))
        s["slot"] = torch.randperm(pages * page, device="cuda", generator=gen)[:T].to(torch.int32)
        s["position"] = torch.randint(0, c["far"], (T,), device="cuda", generator=gen).to(torch.int32)
        s["inv_freq"] = _inv_freq(c["rot"], c["factor"])
        s["amplitude"] = 1.0 + 0.1 * math.log(c["factor"])
        s["q_out"] = torch.empty(T, Hq, D, dtype=dtype, device="cuda")
        return s
    new, kv = _attn_lengths(c)
    counts = [_pages(k, page) for k in kv]
    s["table"], _, pages = _tables(gen, counts, max(counts), 8)
    shape = (pages, page, Hk, D)
    channel = torch.exp(0.3 * torch.randn(Hk, D, device="cuda", generator=gen)).to(dtype)  # keys differ between channels
    s["k_cache"] = torch.randn(shape, device="cuda", dtype=dtype, generator=gen).mul_(channel)
    s["v_cache"] = torch.randn(shape, device="cuda", dtype=dtype, generator=gen)
    T = sum(new)
    s["q"] = (1.5 * torch.randn(T, Hq, D, device="cuda", generator=gen)).to(dtype)
    s["kv_len"] = _ints(kv)
    s["q_offset"] = _ints([sum(new[:b]) for b in range(c["B"] + 1)])
    s["new_max"], s["kv_max"] = max(new), max(kv)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(T, Hq, dtype=torch.float32, device="cuda")
    s["ws"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _plain_plan(s):
    c, B = s["case"], s["case"]["B"]
    page = c["page"]
    old, new, table = s["cached"].long(), s["new"].long(), s["table"]
    after = old + new
    p_old, p_new = (old + page - 1) // page, (after + page - 1) // page
    need, freed = (p_new - p_old).clamp(min=0), (p_old - p_new).clamp(min=0)
    at_need, at_freed = need.cumsum(0) - need, freed.cumsum(0) - freed
    top = s["free_count"].long() + freed.sum()  # pages on the stack once those given back are on it
    n = s["free"].numel()
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    back = (j >= p_new[:, None]) & (j < p_old[:, None])
    to = torch.where(back, s["free_count"].long() + at_freed[:, None] + j - p_new[:, None], torch.full_like(j, n))
    stack = torch.cat([s["free"], s["free"][:1]]).index_put((to,), table)[:n]
    take = (j >= p_old[:, None]) & (j < p_new[:, None])
    k = at_need[:, None] + j - p_old[:, None]
    table = torch.where(take, stack[(top - 1 - k).clamp(0, n - 1)], table)
    left = top - need.sum()
    free = torch.where(torch.arange(n, device=table.device) < left, stack, s["free"])
    tokens = new.clamp(min=0)
    q_offset = torch.cat([tokens.new_zeros(1), tokens.cumsum(0)])
    t = torch.arange(s["slot"].numel(), device=table.device)
    b = torch.searchsorted(q_offset[1:].contiguous(), t, right=True).clamp(max=B - 1)
    fine = t < q_offset[B]
    position = torch.where(fine, old[b] + t - q_offset[b], torch.zeros_like(t))
    slot = table[b, position // page].long() * page + position % page
    i32 = torch.int32
    return {"table": table, "free": free, "free_count": left.to(i32), "kv_len": after.to(i32), "q_offset": q_offset.to(i32),
            "position": position.to(i32), "slot": torch.where(fine, slot, torch.full_like(slot, -1)).to(i32)}


def _split_qkv(s):
    c = s["case"]
    Hq, Hk, D = c["heads"], c["kv_heads"], c["D"]
    qkv = s["qkv"].view(c["T"], Hq + 2 * Hk, D)
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]


def _plain_rotate(s, x):
    c = s["case"]
    rot, first = c["rot"], c["first"]
    a = s["position"].double()[:, None] * s["inv_freq"]
    cos, sin = ((f(a) * s["amplitude"]).to(torch.float32)[:, None, :] for f in (torch.cos, torch.sin))
    y = x.to(torch.float32)
    r = y[..., first:first + rot]
    u, v = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :rot // 2], r[..., rot // 2:])
    u, v = u * cos - v * sin, v * cos + u * sin
    r = torch.stack([u, v], -1).flatten(-2) if c["interleaved"] else torch.cat([u, v], -1)
    return torch.cat([y[..., :first], r, y[..., first + rot:]], -1).to(x.dtype)


def _plain_rope(s):
    q, k, v = _split_qkv(s)
    slot = s["slot"].long()
    page = s["case"]["page"]
    s["k_cache"][slot // page, slot % page] = _plain_rotate(s, k)
    s["v_cache"][slot // page, slot % page] = v
    return {"q": _plain_rotate(s, q), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attention(s):
    c = s["case"]
    B, Hk, D, N, L, page = c["B"], c["kv_heads"], c["D"], s["new_max"], s["kv_max"], c["page"]
    dev, T = s["q"].device, s["q"].shape[0]
    first, length = s["q_offset"].long(), s["kv_len"].long()
    n = first[1:] - first[:-1]
    i, j = torch.arange(N, device=dev), torch.arange(L, device=dev)
    q = s["q"][(first[:-1, None] + i).clamp(max=T - 1)].to(torch.float32)  # padded to the longest chunk
    q = q.view(B, N, Hk, -1, D).permute(0, 2, 3, 1, 4)
    G = q.shape[2]
    at = s["table"].long().clamp(min=0)[:, j // page], j % page
    k = s["k_cache"][at].to(torch.float32).permute(0, 2, 3, 1)
    seen = torch.full((B, N), L, device=dev) if not c["causal"] else (length - n)[:, None] + i + 1
    seen = torch.minimum(seen, length[:, None])[..., None]
    mask = j < seen
    if c["window"]:
        mask = mask & (j >= seen - c["window"])
    mask = mask[:, None, None]
    x = (q.flatten(2, 3) @ k).view(B, Hk, G, N, L).mul_(D ** -0.5).masked_fill_(~mask, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    v = s["v_cache"][at].to(torch.float32).permute(0, 2, 1, 3)
    o = (x.flatten(2, 3) @ v).view(B, Hk, G, N, D) / torch.where(total == 0, torch.ones_like(total), total)
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(first[1:].contiguous(), t, right=True)
    rows = lambda y: y.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, t - first[b]]  # noqa: E731
    return {"out": rows(o).to(s["q"].dtype), "lse": rows(m + torch.log(total))[..., 0]}


# ------------------------------------------------------------------ one pass
def _run_own(s):
    from block_scaled_fp4_top_gb300 import api

    c = s["case"]
    if c["op"] == "plan":
        api.fp4moe_kv_plan(c["page"], s["cached"], s["new"], s["table"], s["free"], s["free_count"], s["kv_len"],
                           s["free_count_out"], s["q_offset"], s["position"], s["slot"], s["err"])
        return {"table": s["table"], "free": s["free"], "free_count": s["free_count_out"], "kv_len": s["kv_len"],
                "q_offset": s["q_offset"], "position": s["position"], "slot": s["slot"]}
    if c["op"] == "rope":
        q, k, v = _split_qkv(s)
        api.fp4moe_rope_cache(q, k, v, s["position"], s["slot"], s["inv_freq"], s["q_out"], s["k_cache"], s["v_cache"],
                              s["err"], first=c["first"], interleaved=c["interleaved"], amplitude=s["amplitude"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    api.fp4moe_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_len"], s["q_offset"],
                               c["D"] ** -0.5, s["out"], s["lse"], s["ws"], s["err"], causal=c["causal"],
                               window=c["window"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plain_plan, "rope": _plain_rope, "attn": _plain_attention}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_plan(s):
    """One sequence after the other, on lists."""
    c = s["case"]
    page, B = c["page"], c["B"]
    table, free = s["table"].tolist(), s["free"].tolist()
    cached, new = s["cached"].tolist(), s["new"].tolist()
    stack = free[:s["free_count"].item()]
    for b in range(B):  # all pages given back, then all taken
        stack += table[b][_pages(cached[b] + min(new[b], 0), page):_pages(cached[b], page)]
    position, slot, q_offset = [], [], [0]
    for b in range(B):
        for j in range(_pages(cached[b], page), _pages(cached[b] + new[b], page)):
            table[b][j] = stack.pop()
        for p in range(cached[b], cached[b] + new[b]):
            position.append(p)
            slot.append(table[b][p // page] * page + p % page)
        q_offset.append(len(position))
    pad = s["slot"].numel() - len(slot)
    return {"table": _ints(table), "free": _ints(stack + free[len(stack):]), "free_count": _ints([len(stack)]),
            "kv_len": _ints([a + n for a, n in zip(cached, new)]), "q_offset": _ints(q_offset),
            "position": _ints(position + [0] * pad), "slot": _ints(slot + [-1] * pad)}


def _exact_rope(s):
    """Every pair as a complex number, turned by multiplication; places by flat index."""
    c = s["case"]
    half, first = c["rot"] // 2, c["first"]
    p = torch.arange(half, device="cuda")
    at = (first + 2 * p, first + 2 * p + 1) if c["interleaved"] else (first + p, first + p + half)
    turn = torch.polar(torch.full((c["T"], half), float(s["amplitude"]), dtype=torch.float64, device="cuda"),
                       s["position"].double()[:, None] * s["inv_freq"][None, :])
    row = s["qkv"].double().view(c["T"], -1, c["D"])
    turned = c["heads"] + c["kv_heads"]
    z = torch.complex(row[:, :turned][..., at[0]], row[:, :turned][..., at[1]]) * turn[:, None]
    row = row.clone()
    row[:, :turned, at[0]], row[:, :turned, at[1]] = z.real, z.imag
    caches = []
    for x, old in ((row[:, c["heads"]:turned], s["k_cache"]), (row[:, turned:], s["v_cache"])):
        flat = old.double().flatten(0, 1).clone()
        flat.index_copy_(0, s["slot"].long(), x)
        caches.append(flat.view(old.shape))
    return {"q": row[:, :c["heads"]], "k_cache": caches[0], "v_cache": caches[1]}


def _exact_attention(s):
    """One sequence and one kv head at a time, by its own keys only."""
    c = s["case"]
    new, kv = _attn_lengths(c)
    G, page = c["heads"] // c["kv_heads"], c["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    t = 0
    for b in range(c["B"]):
        n, L = new[b], kv[b]
        key = torch.arange(L, device="cuda")
        slot = s["table"][b].long()[key // page] * page + key % page
        last = torch.arange(L - n, L, device="cuda") if c["causal"] else torch.full((n,), L - 1, device="cuda")
        hidden = key[None, :] > last[:, None]
        if c["window"]:
            hidden = hidden | (key[None, :] <= last[:, None] - c["window"])
        for h in range(c["kv_heads"]):
            k = s["k_cache"].flatten(0, 1)[slot, h].double()
            v = s["v_cache"].flatten(0, 1)[slot, h].double()
            for g in range(h * G, h * G + G):
                z = s["q"][t:t + n, g].double() @ k.t() / math.sqrt(c["D"])
                z = z.masked_fill(hidden, -math.inf)
                lse[t:t + n, g] = torch.logsumexp(z, 1)
                out[t:t + n, g] = torch.softmax(z, 1) @ v
        t += n
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "rope": _exact_rope, "attn": _exact_attention}[case["op"]](s)
