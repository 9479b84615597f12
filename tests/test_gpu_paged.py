"""GPU: the paged key-value cache's plan, rotary positions and attention against their 64-bit definitions.

Tolerances are sums of the roundings that the definitions allow:
* a plan is whole numbers: equal;
* a turned element: its angle is off by 2^-31 turns, what cosine and sine of it add is 2^-22, the products and their sum
  2^-23, all against (|x| + |y|) amplitude, and half a step of its type at the end;
* a score: fp32 additions of exact products, at worst 2^-22 of the running magnitude for each MMA of 16 dims, so
  ds = scale sum|q k| (D / 16 + 2) 2^-22, and 2^-23 of its own size in the exponent; the weights are off by that, by 2^-21
  of the exponential and by half a step of the cache's type in front of the product with v; sums over n keys by
  (n / 16 + 64) 2^-22. All against sum p|v| / sum p, and half a step of the output.
"""
import math

import numpy as np
import pytest

import paged_ref as ref
from dense_ref import Guarded
from helpers import ensure_built
from paged_ref import HALF_STEP, TINY

pytestmark = pytest.mark.gpu
DTYPES = ["bfloat16", "float16"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def ints(v, shape=None):
    import torch
    t = torch.tensor(v, dtype=torch.int32, device="cuda")
    return t.reshape(shape) if shape else t


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------------- plan
def run_plan(page, cached, new, table, free, count, rows, in_place=False, err0=0):
    import torch
    from block_scaled_fp4_top_gb300 import api
    B, columns = len(cached), len(table[0]) if table else 4
    i32 = torch.int32
    bufs = {"cached": Guarded((B,), i32, ints(cached)), "new": Guarded((B,), i32, ints(new)),
            "table": Guarded((B, columns), i32, ints(table, (B, columns))), "free": Guarded((len(free),), i32, ints(free)),
            "count_in": Guarded((1,), i32, ints([count])), "kv_len": Guarded((B,), i32), "count": Guarded((1,), i32),
            "q_offset": Guarded((B + 1,), i32), "position": Guarded((rows,), i32), "slot": Guarded((rows,), i32)}
    err = ints([err0, 0, 0, 0])
    if in_place:
        bufs["kv_len"], bufs["count"] = bufs["cached"], bufs["count_in"]
    t = {n: b.t for n, b in bufs.items()}
    call = lambda: api.fp4moe_kv_plan(page, t["cached"], t["new"], t["table"], t["free"], t["count_in"], t["kv_len"],  # noqa: E731
                                      t["count"], t["q_offset"], t["position"], t["slot"], err)
    call()
    torch.cuda.synchronize()
    want, bits = ref.plan(page, cached, new, table, free, count, rows)
    for n, w in want.items():
        assert t[n].flatten().tolist() == np.array(w, dtype=np.int64).reshape(-1).tolist(), n
    assert err.tolist() == [err0 | bits, 0, 0, 0]
    for b in bufs.values():
        b.check()
    if not in_place:
        assert t["cached"].tolist() == cached and t["count_in"].tolist() == [count] and t["new"].tolist() == new
        call()  # from the same state: the same
        torch.cuda.synchronize()
        for n, w in want.items():
            assert t[n].flatten().tolist() == np.array(w, dtype=np.int64).reshape(-1).tolist(), n
    return bits


def state(rng, B, page, most, columns, spare):
    """cached lengths, a table of random pages and the stack of the others."""
    cached = [int(rng.integers(0, most + 1)) for _ in range(B)]
    n = sum(ref.pages(c, page) for c in cached)
    order = rng.permutation(n + spare).tolist()
    table, at = [], 0
    for c in cached:
        k = ref.pages(c, page)
        table.append(order[at:at + k] + [-7] * (columns - k))
        at += k
    return cached, table, order[at:] + [-3] * n, spare


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page,most,new,rows", [(1, 16, 40, 1, 64), (3, 1, 9, 5, 64), (64, 16, 500, 1, 64),
                                                  (33, 5, 60, 70, 1500), (100, 7, 200, 300, 20000), (1000, 64, 900, 4, 3000),
                                                  (2049, 16, 90, 30, 70000), (8192, 4, 21, 3, 9000)])
def test_plan(B, page, most, new, rows, in_place):
    rng = np.random.default_rng(B + page)
    columns = ref.pages(most + new, page) + 1
    cached, table, free, count = state(rng, B, page, most, columns, B * ref.pages(new, page) + B + 3)
    fresh = [int(rng.choice([0, 1, int(rng.integers(0, new + 1)), -c, -int(rng.integers(0, c + 1))])) for c in cached]
    while sum(max(n, 0) for n in fresh) > rows:
        fresh[int(np.argmax(fresh))] = 0
    assert run_plan(page, cached, fresh, table, free, count, rows, in_place) == 0


def test_plan_of_nothing():
    assert run_plan(16, [], [], [], [1, 0], 2, 64) == 0
    assert run_plan(16, [0, 0], [0, 0], [[-1], [-1]], [1, 0], 2, 0) == 0
    assert run_plan(16, [5], [-5], [[0]], [1, -1], 1, 3) == 0


def test_plan_refuses_sequences_without_room():
    free = list(range(40))
    table = [[-1] * 6 for _ in range(5)]
    # pool of 3 pages: the second sequence does not fit, and so none after it that needs a page; one that needs none does
    assert run_plan(4, [0, 0, 0, 0, 0], [8, 9, 1, 0, 4], table, free, 3, 64) == ref.ERR_CAPACITY
    table[3][0] = 9
    assert run_plan(4, [0, 0, 0, 2, 0], [8, 9, 1, 2, 4], table, free, 3, 64) == ref.ERR_CAPACITY
    # more than the table's columns; the others are served
    assert run_plan(4, [0, 0, 0, 0, 0], [4, 25, 1, 0, 4], table, free, 30, 64) == ref.ERR_CAPACITY
    # rows cut at 16: the third has 9 rows from 12 on
    assert run_plan(4, [0, 0, 0, 0, 0], [8, 4, 9, 1, 0], table, free, 30, 16) == ref.ERR_CAPACITY
    # pages given back in the same step are there to take
    table[0] = [31, 32, 33, 34, -1, -1]
    assert run_plan(4, [16, 0, 0, 0, 0], [-16, 12, 4, 0, 0], table, free, 0, 64, err0=0x8) == 0


def test_plan_of_lengths_and_pages_out_of_range():
    free = list(range(8))
    table = [[5, 6, -1], [7, 99, -1], [-2, -1, -1]]
    assert run_plan(4, [-3, 0, 0], [2, 0, 0], table, free, 4, 64) == ref.ERR_PAGE
    assert run_plan(4, [13, 0, 0], [0, 0, 0], table, free, 4, 64) == ref.ERR_PAGE
    assert run_plan(4, [3, 0, 0], [-4, 0, 0], table, free, 4, 64) == ref.ERR_PAGE
    assert run_plan(4, [0, 6, 2], [0, 2, 1], table, free, 4, 64) == ref.ERR_PAGE       # pages 99 and -2
    assert run_plan(4, [0, 0, 0], [1, 0, 0], table, free, 9, 64) == ref.ERR_PAGE
    assert run_plan(4, [0, 0, 0], [0, 0, 0], table, free, -1, 64) == ref.ERR_PAGE
    assert run_plan(4, [8, 0, 0], [-8, 0, 5], table, free, 7, 64) == ref.ERR_PAGE      # a page for a full stack
    big = 2 ** 31 - 1
    assert run_plan(4, [big, 0, 0], [big, -big - 1, 0], table, free, 4, 64) == ref.ERR_PAGE | ref.ERR_CAPACITY


# ------------------------------------------------------------------------- rotary positions
def cache(pages, page, Hk, D, dtype, order="tokens", seed=None):
    """Two caches with a canary in every element; order "heads": [pages][heads][tokens][dims] in memory."""
    import torch
    shape = (pages, page, Hk, D) if order == "tokens" else (pages, Hk, page, D)
    out = []
    for i in range(2):
        if seed is None:
            t = torch.full(shape, 123.0, dtype=dtype, device="cuda")
        else:
            t = torch.randn(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed + i)).to(dtype)
        out.append(t if order == "tokens" else t.transpose(1, 2))
    return out


def check_rope(T, H, Hk, D, rot, dtype="bfloat16", first=0, interleaved=False, amplitude=1.0, far=100000, page=16,
               order="tokens", in_place=False, pad=(), packed=True, with_q=True, with_kv=True, seed=0):
    import torch
    from block_scaled_fp4_top_gb300 import api
    dt = getattr(torch, dtype)
    rng = np.random.default_rng(seed + T)
    gen = torch.Generator("cuda").manual_seed(seed)
    width = (H + 2 * Hk) * D + (0 if packed else 24)
    rows = Guarded((T, width), dt, torch.randn(T, width, device="cuda", generator=gen))
    before = rows.t.clone()
    q, k, v = (rows.t[:, a * D:b * D].unflatten(1, (-1, D)) for a, b in ((0, H), (H, H + Hk), (H + Hk, H + 2 * Hk)))
    pages = ref.pages(T, page) + 2
    kc, vc = cache(pages, page, Hk, D, dt, order)
    slot = rng.permutation(pages * page)[:T]
    position = rng.integers(-5, far, T)
    position[0] = far
    slot[list(pad)] = -1
    inv = torch.from_numpy(10000.0 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))).cuda()
    qo = Guarded((T, H, D), dt)
    err = ints([0])
    dst = q if in_place else qo.t
    api.fp4moe_rope_cache(q if with_q else None, k if with_kv else None, v if with_kv else None, ints(position.tolist()),
                          ints(slot.tolist()), inv, dst if with_q else None, kc, vc, err, first=first,
                          interleaved=interleaved, amplitude=amplitude)
    torch.cuda.synchronize()
    rows.check()
    qo.check()
    assert err.tolist() == [0]
    x = f64(before)[:, :(H + 2 * Hk) * D].reshape(T, -1, D)
    want, mag = ref.rotate(x[:, :H + Hk], position, inv.cpu().numpy(), first, interleaved, amplitude)
    rel = 2 * math.pi * 2.0 ** -31 + 2.0 ** -22 + 2.0 ** -23
    live = slot >= 0

    def near(got, a, b):
        w, bound = want[:, a:b], mag[:, a:b] * abs(amplitude) * rel
        bound = bound + np.where(mag[:, a:b] > 0, (np.abs(w) + bound) * HALF_STEP[dtype] + TINY[dtype], 0.0)  # copies are exact
        assert (np.abs(got - w) <= bound)[live].all(), np.abs(got - w).max()

    if with_q:
        near(f64(dst), 0, H)
        left = before[:, :H * D].view(T, H, D) if in_place else torch.full_like(qo.raw[:1], 0xA5)
        for t in pad:  # left as it was
            assert torch.equal(dst[t], left[t]) if in_place else (dst[t].contiguous().view(torch.uint8) == left).all()
    flat = [c.reshape(pages * page, Hk, D) for c in (kc, vc)]
    used = torch.from_numpy(slot[live]).cuda()
    if with_kv:
        got = np.zeros((T, Hk, D))
        got[live] = f64(flat[0][used])
        near(got, H, H + Hk)
        assert torch.equal(flat[1][used], before[:, (H + Hk) * D:(H + 2 * Hk) * D].view(T, Hk, D)[torch.from_numpy(live).cuda()])
    rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    if with_kv:
        rest[used] = False
    for f in flat:
        assert (f[rest] == 123.0).all(), "a slot that is not the step's was written"
    if not in_place:
        assert torch.equal(rows.t, before)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,first", [(128, 128, 0), (64, 64, 0), (96, 40, 8), (80, 22, 58), (256, 256, 0), (256, 64, 192),
                                         (128, 2, 0), (128, 2, 125), (8, 8, 0), (16, 6, 3), (72, 48, 16), (128, 0, 0),
                                         (192, 64, 128), (40, 34, 5)])
def test_rope_parts_of_the_head(D, rot, first, interleaved, dtype):
    check_rope(5, 6, 2, D, rot, dtype, first, interleaved, amplitude=1.25)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 64, 333, 3000])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_rows(T, interleaved):
    check_rope(T, 32, 8, 128, 128, interleaved=interleaved, pad=(T // 2,) if T > 1 else ())


@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 1), (8, 8), (20, 4), (71, 1), (64, 8)])
def test_rope_heads(H, Hk):
    check_rope(9, H, Hk, 64, 64, "float16")
    check_rope(9, H, Hk, 80, 30, "float16", 2)


@pytest.mark.parametrize("opts", [dict(order="heads"), dict(in_place=True), dict(in_place=True, interleaved=True, pad=(0, 6)),
                                  dict(pad=(0, 3, 6)), dict(packed=False), dict(with_q=False), dict(with_kv=False), dict(page=1),
                                  dict(page=48, order="heads"), dict(amplitude=-0.5), dict(far=2 ** 31 - 1),
                                  dict(pad=tuple(range(7)))])
@pytest.mark.parametrize("rot,first", [(128, 0), (38, 3)])
def test_rope_options(opts, rot, first):
    check_rope(7, 12, 4, 128, rot, first=first, **opts)


def test_rope_slots_out_of_the_cache():
    import torch
    from block_scaled_fp4_top_gb300 import api
    T, H, Hk, D = 6, 4, 2, 64
    q, k, v = (torch.randn(T, h, D, device="cuda").bfloat16() for h in (H, Hk, Hk))
    kc, vc = cache(3, 5, Hk, D, torch.bfloat16)
    inv = api.rope_inv_freq(D)
    err, out = ints([0]), torch.full_like(q, 7.0)
    api.fp4moe_rope_cache(q, k, v, ints([1] * T), ints([15, -2, 14, -2 ** 31, 2 ** 31 - 1, -1]), inv, out, kc, vc, err)
    torch.cuda.synchronize()
    assert err.tolist() == [ref.ERR_PAGE]
    flat = kc.view(15, Hk, D)
    assert (flat[:14] == 123.0).all() and (vc.view(15, Hk, D)[:14] == 123.0).all() and not (flat[14] == 123.0).any()
    assert (out[5] == 7.0).all() and not (out[:5] == 7.0).any()


@pytest.mark.parametrize("rot,first", [(64, 0), (30, 1)])
def test_rope_keeps_what_it_does_not_turn(rot, first):
    """Payloads of NaN, infinities and negative zeros outside the turned part come through as they are."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    T, D = 3, 64
    q, k, v = (torch.randint(-2 ** 15, 2 ** 15, (T, 2, D), device="cuda", dtype=torch.int16).view(torch.bfloat16) for _ in range(3))
    kc, vc = cache(1, 4, 2, D, torch.bfloat16)
    out, inv = torch.empty_like(q), api.rope_inv_freq(rot)
    api.fp4moe_rope_cache(q, k, v, ints([5, 6, 7]), ints([2, 0, 1]), inv, out, kc, vc, ints([0]), first=first)
    rest = [d for d in range(D) if d < first or d >= first + rot]
    bits = lambda t: t.view(torch.int16)  # noqa: E731
    at = [2, 0, 1]
    assert torch.equal(bits(vc)[0, at], bits(v))
    if rest:
        assert torch.equal(bits(out)[..., rest], bits(q)[..., rest]) and torch.equal(bits(kc)[0, at][..., rest], bits(k)[..., rest])


def test_rope_inv_freq():
    import torch
    from block_scaled_fp4_top_gb300 import api
    f = api.rope_inv_freq(64, 500000.0, device="cpu")
    i = np.arange(32)
    np.testing.assert_allclose(f.numpy(), 500000.0 ** (-2.0 * i / 64), rtol=1e-14)
    np.testing.assert_allclose(api.rope_inv_freq(64, 500000.0, 4.0, device="cpu").numpy(), f.numpy() / 4, rtol=1e-14)
    s = api.rope_inv_freq(64, 500000.0, 8.0, 8192, 1.0, 4.0, device="cpu").numpy()
    turns = 8192 * f.numpy() / (2 * np.pi)
    assert (s[turns >= 4] == f.numpy()[turns >= 4]).all()
    np.testing.assert_allclose(s[turns <= 1], f.numpy()[turns <= 1] / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and (s[mid] < f.numpy()[mid]).all() and (s[mid] > f.numpy()[mid] / 8).all()
    assert api.rope_inv_freq(0).shape == (0,)
    assert torch.equal(api.rope_inv_freq(64, 500000.0).cpu(), f)


# ------------------------------------------------------------------------- attention
def attention_case(new, kv, H, Hk, D, dtype="bfloat16", page=16, columns=None, order="tokens", seed=0, spread=1.0, spare=3,
                   hole=()):
    """Packed q, caches whose unused places hold NaN, a table of random pages (rows past their own: an invalid page)."""
    import torch
    dt = getattr(torch, dtype)
    rng = np.random.default_rng(seed + sum(kv) + D)
    counts = [ref.pages(max(L, 0), page) for L in kv]
    columns = max(counts + [1]) if columns is None else columns
    total = sum(counts) + spare
    order_p = rng.permutation(total).tolist()
    table, at = np.full((len(kv), columns), 2 ** 31 - 1, dtype=np.int64), 0
    kc, vc = cache(total, page, Hk, D, dt, order, seed=seed + 11)
    slots = []
    used = torch.zeros(total * page, dtype=torch.bool, device="cuda")
    for b, L in enumerate(kv):
        mine = order_p[at:at + counts[b]]
        at += counts[b]
        table[b, :len(mine)] = mine[:columns]
        L = min(max(L, 0), columns * page)
        j = np.arange(L)
        s = torch.from_numpy(np.array(mine + [0], dtype=np.int64)[j // page] * page + j % page).cuda()
        used[s] = True
        slots.append(s)
    for b, j in hole:
        table[b, j] = -1 if (b + j) % 2 else total
        slots[b][j * page:(j + 1) * page] = -1
    for c in (kc, vc):  # keys that nobody sees
        c.masked_fill_(~used.view(total, page)[:, :, None, None], float("nan"))
    gen = torch.Generator("cuda").manual_seed(seed + 5)
    q = (spread * torch.randn(sum(new), H, D, device="cuda", generator=gen)).to(dt)
    flat = [c.reshape(total * page, Hk, D) for c in (kc, vc)]
    return q, kc, vc, flat, ints(table.tolist(), (len(kv), columns)), slots


def compare(out, lse, want, kv, D, dtype, what=""):
    o, z, mag, top = (t.cpu().numpy() for t in want)
    n = max(list(kv) + [1])
    ds = top * (D / 16 + 2) * 2.0 ** -22 + top * 2.0 ** -23
    rel = (2 * ds + 2.0 ** -20 + (n / 16 + 64) * 2.0 ** -22)[..., None]
    bound = mag * (rel + HALF_STEP[dtype] * (1 + rel)) + TINY[dtype]
    bound = bound + (np.abs(o) + bound) * HALF_STEP[dtype]
    got = f64(out)
    fine = np.isfinite(o)
    assert (np.isfinite(got) == fine).all() and (np.isnan(got) == np.isnan(o)).all(), what
    with np.errstate(invalid="ignore"):
        err = np.where(fine, np.abs(got - o), 0.0)
    over = err > np.where(fine, bound, np.inf)
    assert not over.any(), (what, int(over.sum()), np.argwhere(over)[:4].tolist(), err.max(), np.abs(o[fine]).max())
    if lse is not None:
        g = lse.cpu().numpy().astype(np.float64)
        fine = np.isfinite(z)
        assert (np.isneginf(g) == np.isneginf(z)).all() and (np.isfinite(g) == fine).all(), what
        with np.errstate(invalid="ignore"):
            err = np.where(fine, np.abs(g - z), 0.0)
        assert (err <= np.where(fine, ds + rel[..., 0] + np.abs(z) * 2.0 ** -22, np.inf)).all(), (what, err.max())


def run_attention(q, kc, vc, table, kv, first, scale, causal, window, with_lse=True, out=None, rows=None, err_want=0):
    import torch
    from block_scaled_fp4_top_gb300 import api
    T, H, D = q.shape
    out = Guarded((T, H, D), q.dtype) if out is None else out
    lse = Guarded((T, H), torch.float32) if with_lse else None
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    err = ints([0])
    args = (q, kc, vc, table, ints(list(kv)), ints(list(first)), scale, out.t, lse.t if lse else None, ws, err)
    api.fp4moe_paged_attention(*args, causal=causal, window=window)
    torch.cuda.synchronize()
    got = out.t.clone(), lse.t.clone() if lse else None
    api.fp4moe_paged_attention(*args, causal=causal, window=window)   # on the workspace as the first call left it
    torch.cuda.synchronize()
    assert torch.equal(out.t.view(torch.int16), got[0].view(torch.int16)), "not deterministic"
    if lse:
        assert torch.equal(lse.t.view(torch.int32), got[1].view(torch.int32))
        lse.check()
    out.check()
    assert err.tolist() == [err_want]
    assert not ws[:4096].any(), "counters not left at zero"
    return got


def check_attention(new, kv, H, Hk, D, dtype="bfloat16", page=16, causal=True, window=0, scale=None, tile=None, **kw):
    if tile:
        from block_scaled_fp4_top_gb300 import api
        assert api.fp4moe_paged_attention_plan(len(new), sum(new), H, Hk, D) == tile
    q, kc, vc, flat, table, slots = attention_case(new, kv, H, Hk, D, dtype, page, **kw)
    scale = D ** -0.5 if scale is None else scale
    first = [sum(new[:b]) for b in range(len(new) + 1)]
    out, lse = run_attention(q, kc, vc, table, kv, first, scale, causal, window,
                             err_want=ref.ERR_PAGE if kw.get("hole") else 0)
    want = ref.attention(q, *flat, slots, first, new, kv, scale, causal, window)
    compare(out, lse, want, kv, D, dtype)
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [8, 24, 64, 72, 80, 96, 128, 136, 160, 256])
def test_attention_head_dims(D, dtype):
    check_attention([1, 1, 1], [1, 150, 400], 8, 2, D, dtype)
    check_attention([7, 1, 30], [7, 150, 401], 8, 2, D, dtype)


@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (6, 2), (7, 1), (16, 2), (16, 1), (17, 1), (48, 2), (128, 1), (600, 2)])
@pytest.mark.parametrize("new", [[1, 1], [5, 3], [40, 1]])
def test_attention_head_groups(H, Hk, new):
    check_attention(new, [200, 43], H, Hk, 64)


@pytest.mark.parametrize("page", [1, 3, 7, 16, 48, 64, 100, 128, 200, 1000])
@pytest.mark.parametrize("order", ["tokens", "heads"])
def test_attention_pages(page, order):
    check_attention([1, 20, 3], [333, 257, 128], 8, 2, 128, page=page, order=order)


@pytest.mark.parametrize("new,kv", [([1], [1]), ([1], [127]), ([1], [128]), ([1], [129]), ([1], [5000]), ([300], [300]), ([129], [1000]),
                                    ([0, 1, 0, 2, 0], [0, 3, 50, 70, 0]), ([0, 0], [9, 0]), ([1] * 200, [37] * 200),
                                    ([1] * 5, [1, 9000, 3, 2, 1]), ([2, 2], [0, 1]), ([5, 9], [3, 0])])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_lengths(new, kv, D):
    """Lengths from none on; more new tokens than keys, whose first rows see nothing."""
    out = check_attention(new, kv, 8, 2, D)
    first = np.cumsum([0] + new)
    for b, (n, L) in enumerate(zip(new, kv)):
        if L < n:
            assert (out[first[b]:first[b] + n - L] == 0).all()


@pytest.mark.parametrize("window", [1, 2, 15, 16, 100, 129, 5000])
@pytest.mark.parametrize("new,kv", [([1, 1], [700, 90]), ([60, 200], [700, 200])])
def test_attention_window(window, new, kv):
    check_attention(new, kv, 8, 4, 64, window=window)


@pytest.mark.parametrize("new,kv", [([1, 1], [700, 0]), ([60, 300], [130, 17]), ([5], [4000])])
@pytest.mark.parametrize("D", [80, 128])
def test_attention_of_every_key(new, kv, D):
    check_attention(new, kv, 8, 4, D, "float16", causal=False)


@pytest.mark.parametrize("dtype,spread,scale", [("bfloat16", 30.0, None), ("float16", 8.0, None), ("bfloat16", 1.0, 1e-4),
                                                ("bfloat16", 1.0, 3.0), ("float16", 0.0, None)])
@pytest.mark.parametrize("new", [[1, 1], [40, 3]])
def test_attention_spread_of_the_scores(dtype, spread, scale, new):
    check_attention(new, [900, 77], 4, 2, 128, dtype, spread=spread, scale=scale)


# The same for the larger tiles, which these sizes take.
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [8, 16, 24, 48, 64, 72, 80, 96, 112, 120, 128])
@pytest.mark.parametrize("page", [5, 16])
def test_tiles_head_dims(D, dtype, page):
    check_attention([70, 1, 30], [70, 150, 401], 16, 8, D, dtype, page, tile=256)


@pytest.mark.parametrize("H,Hk", [(8, 8), (24, 8), (20, 4), (56, 8), (16, 1), (17, 1), (33, 1), (128, 1), (130, 1), (256, 2), (600, 2)])
@pytest.mark.parametrize("new", [[129, 3], [64, 64, 65], [0, 1000, 0]])
def test_tiles_head_groups(H, Hk, new):
    new = [n if H // Hk < 60 else n // 4 for n in new]
    check_attention(new, [n + 77 for n in new], H, Hk, 64, tile=256)


@pytest.mark.parametrize("page", [1, 2, 3, 8, 16, 24, 48, 64, 100, 128, 136, 256, 1000])
@pytest.mark.parametrize("order", ["tokens", "heads"])
@pytest.mark.parametrize("D", [64, 128])
def test_tiles_pages(page, order, D):
    check_attention([100, 20, 3], [733, 257, 128], 16, 4, D, page=page, order=order, tile=256)


@pytest.mark.parametrize("new,kv", [([128], [128]), ([129], [129]), ([300], [300]), ([65], [1000]), ([257], [5000]), ([90, 1, 0, 90], [90, 5000, 50, 91]),
                                    ([200, 7], [3, 0]), ([60, 60, 60], [1, 20000, 59]), ([40] * 40, list(range(40, 80))), ([1] * 30 + [500], [100] * 30 + [500])])
@pytest.mark.parametrize("D", [64, 128])
def test_tiles_lengths(new, kv, D):
    out = check_attention(new, kv, 32, 8, D, tile=256)
    first = np.cumsum([0] + new)
    for b, (n, L) in enumerate(zip(new, kv)):
        if L < n:
            assert (out[first[b]:first[b] + n - L] == 0).all()


@pytest.mark.parametrize("window", [1, 2, 64, 100, 128, 129, 300, 5000])
@pytest.mark.parametrize("new,kv", [([60, 200], [700, 200]), ([1, 300], [3000, 1500])])
def test_tiles_window(window, new, kv):
    check_attention(new, kv, 16, 8, 64, window=window, tile=256)


@pytest.mark.parametrize("new,kv", [([100, 64], [700, 0]), ([60, 300], [130, 17]), ([130], [4000])])
@pytest.mark.parametrize("D,page", [(80, 16), (128, 7)])
def test_tiles_of_every_key(new, kv, D, page):
    check_attention(new, kv, 16, 8, D, "float16", page, causal=False, tile=256)


@pytest.mark.parametrize("dtype,spread,scale", [("bfloat16", 30.0, None), ("float16", 8.0, None), ("bfloat16", 1.0, 1e-4),
                                                ("bfloat16", 1.0, 3.0), ("float16", 0.0, None)])
@pytest.mark.parametrize("D", [64, 128])
def test_tiles_spread_of_the_scores(dtype, spread, scale, D):
    check_attention([140, 3], [1900, 77], 16, 8, D, dtype, spread=spread, scale=scale, tile=256)


def test_tiles_scores_that_rise():
    """Every step's maximum far above the steps' before: the sums so far are rescaled each time, in every row."""
    import torch
    for D in (64, 128):
        new, kv = [130], [1500]
        q, kc, vc, flat, table, slots = attention_case(new, kv, 16, 8, D)
        q.copy_(torch.ones_like(q) + 0.1 * q)
        rise = torch.linspace(-4.0, 4.0, 1500, device="cuda")[:, None, None]
        for b, f in ((kc, flat[0]),):
            s = slots[0]
            b[s // 16, s % 16] = (rise + 0.05 * f[s].float()).bfloat16()
        flat = [c.reshape(-1, 8, D) for c in (kc, vc)]
        out, lse = run_attention(q, kc, vc, table, kv, [0, 130], 1.0, True, 0)
        want = ref.attention(q, *flat, slots, [0], new, kv, 1.0, True, 0)
        compare(out, lse, want, kv, D, "bfloat16")


@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (128, 7)])
@pytest.mark.parametrize("new", [[130], [200, 31]])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_tiles_keep_hidden_keys_out(D, page, new, bad):
    import torch
    kv, H, Hk = [380, 300][:len(new)], 16, 8
    first = [0] + np.cumsum(new).tolist()
    for where, window in (("v", 0), ("v", 70), ("k", 0)):
        q, kc, vc, flat, table, slots = attention_case(new, kv, H, Hk, D, page=page)
        j = kv[0] - 1 - new[0] // 2                     # a middle new token's own key
        s = int(slots[0][j])
        (vc if where == "v" else kc)[s // page, s % page, 1, 3] = bad
        flat = [c.reshape(-1, Hk, D) for c in (kc, vc)]
        out, lse = run_attention(q, kc, vc, table, kv, first, D ** -0.5, True, window)
        want = ref.attention(q, *flat, slots, first[:-1], new, kv, D ** -0.5, True, window)
        i = torch.arange(sum(new), device="cuda")
        pos = i + kv[0] - new[0]
        sees = (i < new[0]) & (pos >= j) & ((pos - window < j) if window else True)
        clean = [0, 1] + list(range(4, H))
        assert torch.isfinite(out[~sees]).all() and torch.isfinite(out[:, clean]).all()
        if where == "v":
            assert not torch.isfinite(out[sees][:, 2:4, 3]).any()
            compare(out, lse, want, kv, D, "bfloat16")
        else:
            compare(out[~sees], lse[~sees], [t[~sees] for t in want], kv, D, "bfloat16")
            compare(out[:, clean], lse[:, clean], [t[:, clean] for t in want], kv, D, "bfloat16")


@pytest.mark.parametrize("D,page", [(64, 16), (64, 5), (128, 16)])
def test_tiles_keep_hidden_keys_out_of_many_short_sequences(D, page):
    """Units of one step each, so that loads run several units ahead of the rows that are made again."""
    import torch
    B, n, H, Hk = 300, 40, 16, 8
    new = kv = [n] * B
    q, kc, vc, flat, table, slots = attention_case(new, kv, H, Hk, D, page=page)
    for b in range(B):
        s = int(slots[b][20 + b % 19])
        vc[s // page, s % page, b % Hk, 5] = (float("nan"), float("inf"))[b % 2]
    flat = [c.reshape(-1, Hk, D) for c in (kc, vc)]
    first = [n * b for b in range(B + 1)]
    out, lse = run_attention(q, kc, vc, table, kv, first, D ** -0.5, True, 0)
    want = ref.attention(q, *flat, slots, first[:-1], new, kv, D ** -0.5, True, 0)
    compare(out, lse, want, [n], D, "bfloat16")


@pytest.mark.parametrize("page", [16, 7])
def test_tiles_pages_out_of_the_cache(page):
    check_attention([100, 30, 2], [300, 60, 40], 16, 8, 64, page=page, hole=[(0, 2), (1, 0), (2, 1)], tile=256)


@pytest.mark.parametrize("H,Hk,D", [(32, 8, 128), (24, 8, 64), (12, 4, 80)])
def test_tiles_strides(H, Hk, D):
    """q as a slice of a projection's rows, out into a wider matrix; rows past the last sequence stay as they were."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    new, kv = [130, 70], [290, 140]
    q, kc, vc, flat, table, slots = attention_case(new, kv, H, Hk, D)
    wide = torch.randn(210, (H + 4) * D, device="cuda").bfloat16()
    wide[:200, D:(H + 1) * D] = q.flatten(1)
    out = torch.full((210, H + 2, D), 9.0, device="cuda", dtype=torch.bfloat16)
    ws, err = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda"), ints([0])
    api.fp4moe_paged_attention(wide[:, D:(H + 1) * D].unflatten(1, (H, D)), kc, vc, table, ints(kv), ints([0, 130, 200]), D ** -0.5,
                               out[:, 1:H + 1], None, ws, err)
    torch.cuda.synchronize()
    want = ref.attention(q, *flat, slots, [0, 130], new, kv, D ** -0.5, True, 0)
    compare(out[:200, 1:H + 1], None, want, kv, D, "bfloat16")
    assert (out[:, 0] == 9.0).all() and (out[:, H + 1] == 9.0).all() and (out[200:] == 9.0).all() and err.tolist() == [0]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [[1], [3], [50]])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_keeps_hidden_keys_out(D, new, bad):
    """A value that only later rows see does not reach earlier ones; those that see it get what the formula gives."""
    import torch
    kv, H, Hk, page = [180], 4, 2, 16
    for where in ("v", "k"):
        q, kc, vc, flat, table, slots = attention_case(new, kv, H, Hk, D, page=page)
        j = kv[0] - 1 - new[0] // 2                     # the middle new token's own key
        s = int(slots[0][j])
        (vc if where == "v" else kc)[s // page, s % page, 1, 3] = bad
        flat = [c.reshape(-1, Hk, D) for c in (kc, vc)]
        out, lse = run_attention(q, kc, vc, table, kv, [0, new[0]], D ** -0.5, True, 0)
        want = ref.attention(q, *flat, slots, [0], new, kv, D ** -0.5, True, 0)
        before = torch.arange(new[0], device="cuda") + kv[0] - new[0] < j
        sees = ~before
        assert torch.isfinite(out[before]).all() and torch.isfinite(out[:, :H // 2]).all()
        if where == "v":
            assert not torch.isfinite(out[sees][:, H // 2:, 3]).any()
            compare(out, lse, want, kv, D, "bfloat16")
        else:
            compare(out[before], lse[before], [t[before] for t in want], kv, D, "bfloat16")
            compare(out[:, :H // 2], lse[:, :H // 2], [t[:, :H // 2] for t in want], kv, D, "bfloat16")


def test_attention_scores_of_minus_infinity():
    """-infinity as a score takes no weight; a row that sees nothing else is 0 / 0, unlike one that sees no key."""
    import torch
    q, kc, vc, flat, table, slots = attention_case([2, 1], [20, 1], 2, 1, 64)
    q[:, :, 0] = 1.0
    kc[int(slots[0][4]) // 16, int(slots[0][4]) % 16, 0, 0] = -float("inf")
    kc[int(slots[1][0]) // 16, int(slots[1][0]) % 16, 0, 0] = -float("inf")
    out, lse = run_attention(q, kc, vc, table, [20, 1], [0, 2, 3], 0.125, True, 0)
    assert torch.isfinite(out[:2]).all() and torch.isfinite(lse[:2]).all()
    assert torch.isnan(out[2]).all() and torch.isneginf(lse[2]).all()
    flat = [c.reshape(-1, 1, 64) for c in (kc, vc)]
    want = ref.attention(q[:2], *flat, slots[:1], [0], [2], [20], 0.125, True, 0)
    o, z, mag, top = want
    assert torch.allclose(out[:2].double(), o, atol=2e-2) and torch.allclose(lse[:2].double(), z, atol=1e-4)


def test_attention_pages_out_of_the_cache():
    """They read as zeros, with an error; and so do lengths past the table's columns, whose keys are missing."""
    import torch
    check_attention([1, 30, 2], [100, 60, 40], 8, 2, 64, hole=[(0, 2), (1, 0), (2, 1)])
    q, kc, vc, flat, table, slots = attention_case([2, 3], [90, 40], 4, 2, 64, columns=4)
    out, lse = run_attention(q, kc, vc, table, [90, 40], [0, 2, 5], 0.125, True, 0, err_want=ref.ERR_PAGE)
    want = ref.attention(q, *flat, slots, [0, 2], [2, 3], [90, 40], 0.125, True, 0)
    compare(out, lse, want, [90, 40], 64, "bfloat16")
    out, lse = run_attention(q, kc, vc, table, [-5, 40], [0, 2, 5], 0.125, True, 0, err_want=ref.ERR_PAGE)
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all()


def test_attention_offsets_out_of_range():
    """Offsets out of order or past T are cut to the rows there are; rows past the last sequence stay as they were."""
    import torch
    q, kc, vc, flat, table, slots = attention_case([4, 6], [50, 60], 4, 2, 64)
    for first, new in (([0, 4, 7], [4, 3]), ([2, 4, 4], [2, 0]), ([0, 4, 99], [4, 6]), ([-3, 4, 1], [4, 0]), ([0, 0, 0], [0, 0])):
        out = Guarded((10, 4, 64), torch.bfloat16)
        out.t.fill_(9.0)
        got, _ = run_attention(q, kc, vc, table, [50, 60], first, 0.125, True, 0, out=out)
        starts = [max(0, min(first[0], 10)), max(0, min(first[1], 10))]
        want = ref.attention(q, *flat, slots, starts, new, [50, 60], 0.125, True, 0)
        rows = torch.zeros(10, dtype=torch.bool, device="cuda")
        for s, n in zip(starts, new):
            rows[s:s + n] = True
        compare(got[rows], None, [t[rows] for t in want], [50, 60], 64, "bfloat16", str(first))
        assert (got[~rows] == 9.0).all()


def test_attention_strides():
    """q as a slice of a projection's rows, out into a wider matrix."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    q, kc, vc, flat, table, slots = attention_case([3, 2], [90, 40], 4, 2, 64)
    wide = torch.randn(5, 8 * 64, device="cuda").bfloat16()
    wide[:, 64:5 * 64] = q.flatten(1)
    out = torch.full((5, 6, 64), 9.0, device="cuda", dtype=torch.bfloat16)
    ws, err = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda"), ints([0])
    api.fp4moe_paged_attention(wide[:, 64:5 * 64].unflatten(1, (4, 64)), kc, vc, table, ints([90, 40]), ints([0, 3, 5]), 0.125,
                               out[:, 1:5], None, ws, err)
    torch.cuda.synchronize()
    want = ref.attention(q, *flat, slots, [0, 3], [3, 2], [90, 40], 0.125, True, 0)
    compare(out[:, 1:5], None, want, [90, 40], 64, "bfloat16")
    assert (out[:, 0] == 9.0).all() and (out[:, 5] == 9.0).all()


@pytest.mark.parametrize("new", [[1, 1], [100, 100]])
def test_attention_offsets_past_32_bits(new):
    """Pages whose elements lie past 2^31 and 2^32 of the cache's."""
    import torch
    page, Hk, D = 64, 8, 128
    pages = 2 ** 32 // (page * Hk * D) + 40
    kc, vc = (torch.empty(pages, page, Hk, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kv = [500, 300]
    where = [[pages - 1 - i for i in range(8)], [2 ** 31 // (page * Hk * D) + 3 * i for i in range(5)]]
    gen = torch.Generator("cuda").manual_seed(1)
    for w in where:
        for p in w:
            for c in (kc, vc):
                c[p] = torch.randn(page, Hk, D, device="cuda", generator=gen).bfloat16()
    table = ints([w + [0] * (8 - len(w)) for w in where])
    slots = [torch.tensor([w[j // page] * page + j % page for j in range(L)], device="cuda") for w, L in zip(where, kv)]
    q = torch.randn(sum(new), 16, D, device="cuda", generator=gen).bfloat16()
    first = [0, new[0], sum(new)]
    out, lse = run_attention(q, kc, vc, table, kv, first, D ** -0.5, True, 0)
    want = ref.attention(q, kc.view(-1, Hk, D), vc.view(-1, Hk, D), slots, first, new, kv, D ** -0.5, True, 0)
    compare(out, lse, want, kv, D, "bfloat16")


def in_gaps(c, order, filler):
    """The same cache with `filler` between its heads."""
    import torch
    wide = torch.full((*c.shape[:3], c.shape[3] + 8), filler, device="cuda", dtype=c.dtype)
    if order == "heads":
        wide = torch.full((c.shape[0], c.shape[2], c.shape[1], c.shape[3] + 8), filler, device="cuda", dtype=c.dtype).transpose(1, 2)
    wide[..., :c.shape[3]] = c
    return wide[..., :c.shape[3]]


@pytest.mark.parametrize("D", [8, 24, 64, 72, 80, 120])
@pytest.mark.parametrize("page", [1, 5, 16])
@pytest.mark.parametrize("order", ["tokens", "heads"])
@pytest.mark.parametrize("new", [[1, 1], [140, 31]])
def test_attention_of_heads_apart(D, page, order, new):
    """What lies between a cache's heads is no part of any: NaN there reach no result. Nor does one head's reach another's."""
    import torch
    H, Hk, kv = 16, 8, [300, 140]
    q, kc, vc, flat, table, slots = attention_case(new, kv, H, Hk, D, page=page, order=order)
    first = [0, new[0], sum(new)]
    want = ref.attention(q, *flat, slots, first, new, kv, D ** -0.5, True, 0)
    kc, vc = (in_gaps(c, order, float("nan")) for c in (kc, vc))
    out, lse = run_attention(q, kc, vc, table, kv, first, D ** -0.5, True, 0)
    compare(out, lse, want, kv, D, "bfloat16")
    kc[:, :, 3] = float("nan")
    out, lse = run_attention(q, kc, vc, table, kv, first, D ** -0.5, True, 0)
    clean = [h for h in range(H) if h // 2 != 3]
    compare(out[:, clean], lse[:, clean], [t[:, clean] for t in want], kv, D, "bfloat16")


@pytest.mark.parametrize("D", [48, 80])
@pytest.mark.parametrize("page,order", [(16, "tokens"), (5, "tokens"), (5, "heads")])
def test_attention_after_another_call(D, page, order):
    """A call's bits do not depend on what the one before it, of values that are not finite, left behind."""
    import torch
    new, kv, H, Hk = [140, 31], [300, 140], 16, 8
    case = attention_case(new, kv, H, Hk, D, page=page, order=order)
    other = attention_case(new, kv, H, Hk, 64 if D < 64 else 128, page=page, order=order)
    got = []
    for left in (0.0, float("nan")):
        q, kc, vc, flat, table, slots = other
        vc[:] = left
        run_attention(q, kc, vc, table, kv, [0, 140, 171], 0.1, True, 0)
        q, kc, vc, flat, table, slots = case
        got.append(run_attention(q, kc, vc, table, kv, [0, 140, 171], D ** -0.5, True, 0)[0])
    want = ref.attention(case[0], *case[3], case[5], [0, 140], new, kv, D ** -0.5, True, 0)
    compare(got[0], None, want, kv, D, "bfloat16")
    assert torch.equal(got[0].view(torch.int16), got[1].view(torch.int16))


def test_attention_of_as_many_rows_as_32_bits_count():
    """One sequence of nearly 2^31 rows, of which the last ten see keys."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    T, D, L = 2 ** 31 - 64, 8, 10
    if torch.cuda.mem_get_info()[0] < 100 * 2 ** 30:
        pytest.skip("100 GB of memory")
    q, kc, vc, flat, table, slots = attention_case([L], [L], 1, 1, D)
    big = torch.zeros(T, 1, D, dtype=torch.bfloat16, device="cuda")
    big[T - L:] = q
    out = torch.full_like(big, 9.0)
    ws, err = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda"), ints([0])
    api.fp4moe_paged_attention(big, kc, vc, table, ints([L]), ints([0, T]), D ** -0.5, out, None, ws, err)
    torch.cuda.synchronize()
    want = ref.attention(q, *flat, slots, [0], [L], [L], D ** -0.5, True, 0)
    compare(out[T - L:], None, want, [L], D, "bfloat16")
    assert not any(c.any() for c in out[:T - L].view(-1).split(2 ** 30)) and err.tolist() == [0]


# The same for tiles of 32 rows, which these sizes take.
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [8, 16, 24, 48, 56, 64])
@pytest.mark.parametrize("page", [5, 16])
def test_tiles_of_32_head_dims(D, dtype, page):
    check_attention([7, 1, 9], [7, 150, 401], 16, 4, D, dtype, page, tile=32)


@pytest.mark.parametrize("H,Hk,new", [(1, 1, [17, 18]), (6, 2, [10, 7]), (7, 1, [3, 4]), (17, 1, [1, 1]), (31, 1, [1, 1]), (32, 1, [1, 1]),
                                      (33, 1, [1, 0, 1]), (71, 1, [2, 0]), (8, 1, [4] * 40), (16, 8, [16] * 30 + [5]), (600, 1, [1, 0])])
def test_tiles_of_32_head_groups(H, Hk, new):
    check_attention(new, [200 + 43 * b for b in range(len(new))], H, Hk, 64, tile=32)


@pytest.mark.parametrize("new,kv", [([5], [5]), ([5], [4]), ([8], [1]), ([8], [128]), ([8], [129]), ([8], [20000]), ([0, 20, 0], [0, 37, 9]),
                                    ([8] * 50, list(range(8, 58))), ([6, 8, 7, 8], [1, 9000, 3, 8])])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 3), (True, 100), (False, 0)])
def test_tiles_of_32_lengths(new, kv, causal, window):
    check_attention(new, kv, 32, 8, 64, causal=causal, window=window, tile=32)


@pytest.mark.parametrize("dtype,spread,scale", [("bfloat16", 30.0, None), ("float16", 8.0, None), ("bfloat16", 1.0, 1e-4),
                                                ("bfloat16", 1.0, 3.0), ("float16", 0.0, None)])
def test_tiles_of_32_spread_of_the_scores(dtype, spread, scale):
    check_attention([8, 7], [1900, 77], 32, 8, 64, dtype, spread=spread, scale=scale, tile=32)


@pytest.mark.parametrize("D,new", [(64, [3]), (64, [9]), (128, [3]), (256, [3])])
def test_attention_scores_that_rise(D, new):
    """Every group's maximum above the groups' before, by little and by much: a maximum that lags loses nothing."""
    import torch
    for top in (0.25, 4.0):
        kv = [1500]
        q, kc, vc, flat, table, slots = attention_case(new, kv, 8, 2, D)
        q.copy_(torch.ones_like(q) + 0.1 * q)
        rise = torch.linspace(-top, top, 1500, device="cuda")[:, None, None]
        s = slots[0]
        kc[s // 16, s % 16] = (rise + 0.05 * flat[0][s].float()).bfloat16()
        flat = [c.reshape(-1, 2, D) for c in (kc, vc)]
        out, lse = run_attention(q, kc, vc, table, kv, [0, new[0]], 1.0, True, 0)
        want = ref.attention(q, *flat, slots, [0], new, kv, 1.0, True, 0)
        compare(out, lse, want, kv, D, "bfloat16")
