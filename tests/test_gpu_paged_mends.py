"""GPU: the paged cache's calls after a call that gave up, with values that are not finite far inside long sequences, with
weights across the range of fp16, with lengths and positions at their limits. Against the 64-bit references of paged_ref.py,
with the tolerances that test_gpu_paged.py derives."""
import math
from fractions import Fraction

import numpy as np
import pytest

import paged_ref as ref
from helpers import ensure_built
from test_gpu_paged import attention_case, compare, ints, run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


# ------------------------------------------------------------------------- after a timeout
@pytest.mark.parametrize("D,new", [(128, [1, 1]), (64, [130, 3]), (256, [2, 1])])
def test_a_cache_after_a_call_that_gave_up(D, new):
    """Counters of joins that were left counting do not reach the calls after the word has been read and cleared."""
    import torch
    from block_scaled_fp4_top_gb300 import _lib, api
    H, Hk, B = 8, 2, len(new)
    cache = api.PagedKvCache(400, 16, Hk, D, B, 3000, 3000)
    inv = api.rope_inv_freq(D)
    gen = torch.Generator("cuda").manual_seed(D)
    for lengths in ([2800, 150], new):
        T = sum(lengths)
        cache.plan(ints(lengths))
        q, k, v = (torch.randn(T, h, D, device="cuda", generator=gen).bfloat16() for h in (H, Hk, Hk))
        cache.append(q, k, v, inv, q)
    out = torch.empty_like(q)

    def attend(q, out):
        out.fill_(5.0)
        cache.attend(q, D ** -0.5, out)
        torch.cuda.synchronize()
        return out

    want = attend(-q, torch.empty_like(q))
    attend(q, out)                                            # its parts lie in the workspace now
    assert cache.read_error() == 0 and not cache.ws[:4096].any()
    cache.ws[256:4096].view(torch.int32).fill_(1)             # what a call that gives up may leave
    cache.err[0] = _lib.ERR_TIMEOUT
    assert (attend(-q, out) == 5.0).all()                     # skipped
    assert cache.read_error(clear=False) == _lib.ERR_TIMEOUT
    assert (attend(-q, out) == 5.0).all()                     # still
    assert cache.read_error() == _lib.ERR_TIMEOUT
    for _ in range(3):
        assert torch.equal(attend(-q, out).view(torch.int16), want.view(torch.int16))
        assert cache.read_error() == 0 and not cache.ws[:4096].any()


# ------------------------------------------------------------------------- values that are not finite
def put(cache, slots, page, key, head, dims, value):
    s = int(slots[key])
    for d in dims:
        cache[s // page, s % page, head, d] = value


def check_values(new, kv, H, Hk, D, bad, dtype="bfloat16", page=16, window=0, order="tokens"):
    """bad: (sequence, key, kv head, dims, value) of v. Infinite or NaN for the rows that see them, and for no others; the
    call does not give up (run_attention holds the error word to 0)."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    assert api.fp4moe_paged_attention_plan(len(new), sum(new), H, Hk, D) == 256
    q, kc, vc, flat, table, slots = attention_case(new, kv, H, Hk, D, dtype, page, order=order)
    for b, key, head, dims, value in bad:
        put(vc, slots[b], page, key, head, dims, value)
    flat = [c.reshape(-1, Hk, D) for c in (kc, vc)]
    first = [sum(new[:b]) for b in range(len(new) + 1)]
    out, lse = run_attention(q, kc, vc, table, kv, first, D ** -0.5, True, window)
    want = ref.attention(q, *flat, slots, first[:-1], new, kv, D ** -0.5, True, window)
    assert torch.isinf(want[0]).any() or torch.isnan(want[0]).any()
    compare(out, lse, want, kv, D, dtype)


NAN, INF = float("nan"), float("inf")


def test_one_value_late_in_a_long_prompt():
    """The rows of its unit see up to 16384 keys; the other sequences are served as well."""
    check_values([4096, 40, 1], [16384, 900, 50], 1, 1, 128, [(0, 16384 - 77, 0, (3, 90), INF), (0, 13000, 0, (4,), NAN)])


@pytest.mark.parametrize("D,prefix", [(128, 131072), (64, 32768)])
def test_new_values_behind_a_long_prefix(D, prefix):
    """Every new key has some: as many as a unit can have that only some of its rows see."""
    bad = [(0, prefix + i, i % 2, (i % D, (7 * i + 1) % D), (NAN, INF, -INF)[i % 3]) for i in range(0, 300)]
    check_values([300, 5], [prefix + 300, 70], 4, 2, D, bad)


@pytest.mark.parametrize("window", [0, 300])
def test_no_value_is_finite(window):
    """Every key of every unit, one query head a kv head, so that most keys of a unit are seen by some of its rows only."""
    bad = [(0, j, h, [slice(None)], -INF if j % 97 == 0 else INF) for j in range(900) for h in range(2)]
    check_values([600, 5], [900, 70], 2, 2, 128, bad, window=window)


@pytest.mark.parametrize("page,order", [(16, "tokens"), (7, "tokens"), (7, "heads")])
@pytest.mark.parametrize("D,dtype", [(128, "bfloat16"), (64, "float16"), (72, "bfloat16"), (8, "bfloat16"), (40, "float16"), (120, "bfloat16")])
def test_values_at_both_ends_of_a_window(D, dtype, page, order):
    """Keys that enter and that leave the window within a unit, one that all its rows see, both signs of one dim, whole rows."""
    bad = [(0, 3000, 0, (0,), INF), (0, 3100, 0, (0, 5), -INF), (0, 3499, 1, range(D), NAN), (0, 2400, 1, (D - 1,), INF),
           (0, 2010, 1, (1,), -INF), (0, 2700, 0, (9 % D,), NAN), (1, 0, 0, (2,), INF), (1, 449, 1, (3,), INF), (1, 300, 1, range(8), -INF)]
    check_values([600, 450], [3500, 450], 6, 2, D, bad, dtype, page, 1000, order)
    check_values([600, 450], [3500, 450], 6, 2, D, bad, dtype, page, 40, order)


@pytest.mark.parametrize("D", [128, 24])
def test_infinite_keys_with_infinite_values(D):
    """A score of -infinity has weight 0, and 0 times infinity is NaN in its dims only; one of infinity makes the row NaN."""
    import torch
    new, kv, H, Hk, page = [300], [700], 4, 2, 16
    q, kc, vc, flat, table, slots = attention_case(new, kv, H, Hk, D, "bfloat16", page)
    for key in (450, 690):
        put(kc, slots[0], page, key, 0, [0], INF)
        put(vc, slots[0], page, key, 0, [1, 2], -INF)
    put(vc, slots[0], page, 600, 1, [5], NAN)
    flat = [c.reshape(-1, Hk, D) for c in (kc, vc)]
    out, lse = run_attention(q, kc, vc, table, kv, [0, 300], D ** -0.5, True, 0)
    with np.errstate(invalid="ignore"):
        want = ref.attention(q, *flat, slots, [0], new, kv, D ** -0.5, True, 0)
        nan = torch.isnan(want[0])
        assert (nan.all(2).sum() > 0) and (nan.any(2) & ~nan.all(2)).sum() > 0
        compare(out, lse, want, kv, D, "bfloat16")
    clean = torch.isfinite(want[3])                             # rows whose scores are finite: their tolerances are too
    compare(out[clean][:, None], lse[clean][:, None], [t[clean][:, None] for t in want], kv, D, "bfloat16")


# ------------------------------------------------------------------------- weights across fp16's range
@pytest.mark.parametrize("gap", [10.0, 14.0, 18.0])
@pytest.mark.parametrize("D,new,tile", [(64, 1, 16), (128, 2, 16), (256, 1, 16), (64, 20, 32), (64, 40, 256), (128, 33, 256)])
@pytest.mark.parametrize("where", ["first", "late"])
def test_one_key_above_very_many(D, new, tile, gap, where):
    """A key e^gap times as heavy as each of 131071 others, whose value is 0: the result is the others' share, from 0.86 down
    to 0.002. A weight is rounded by half a step of fp16, or, where it is below 2^-21 of the row's largest, by 2^-32 of that: n
    keys by n 2^-32 max|v| / sum of weights (at least 1) beside the tolerance of compare. The sequences share their pages,
    and there are as many as the GPU has work for, so that no row's keys are divided and every one meets the heavy key."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    n, page, H, B = 131072, 64, 8, 20
    q, kc, vc, flat, table, slots = attention_case([new], [n], H, H, D, "float16", page, spread=0.02)
    q = (0.02 * torch.randn(B * new, H, D, device="cuda", generator=torch.Generator("cuda").manual_seed(3))).half()
    assert api.fp4moe_paged_attention_plan(B, B * new, H, H, D) == tile
    s = slots[0]
    q[..., 0] = 1.0
    kc[s // page, s % page, :, 0] = 0.0
    vc[s // page, s % page] = (1.0 + vc[s // page, s % page] / 8).clamp(0.25, 1.75)
    at = 0 if where == "first" else n - new - 5
    put(kc, s, page, at, slice(None), [0], gap)
    put(vc, s, page, at, slice(None), [slice(None)], 0.0)
    flat = [c.reshape(-1, H, D) for c in (kc, vc)]
    first, kv, new = [new * b for b in range(B + 1)], [n] * B, [new] * B
    out, lse = run_attention(q, kc, vc, table.expand(B, -1).contiguous(), kv, first, 1.0, True, 0)
    o, z, mag, top = ref.attention(q, *flat, slots * B, first[:-1], new, kv, 1.0, True, 0)
    small = n * 2.0 ** -32 * 1.75 / ref.HALF_STEP["float16"]     # (compare takes half a step of mag)
    compare(out, lse, (o, z, mag + small, top), kv, D, "float16")


# ------------------------------------------------------------------------- steps of fewer rows, and of some of the tensors
def test_a_step_of_fewer_rows_than_tokens():
    """A plan that knows the step's rows leaves out the sequence that does not fit, and says so; the others are served."""
    import torch
    from block_scaled_fp4_top_gb300 import _lib, api
    H, Hk, D = 4, 2, 64
    cache = api.PagedKvCache(40, 16, Hk, D, 3, 200, 100)
    inv = api.rope_inv_freq(D)
    gen = torch.Generator("cuda").manual_seed(1)
    q, k, v = (torch.randn(24, h, D, device="cuda", generator=gen).bfloat16() for h in (H, Hk, Hk))
    cache.plan(ints([20, 6, 0]), rows=24)
    cache.append(q, k, v, inv, q)
    assert cache.read_error() == _lib.ERR_CAPACITY
    assert cache.kv_len.tolist() == [20, 0, 0] and cache.q_offset.tolist() == [0, 20, 24, 24]
    assert (cache.slot[:20] >= 0).all() and (cache.slot[20:] == -1).all()
    out = torch.empty_like(q)
    cache.attend(q, 0.125, out)
    torch.cuda.synchronize()
    assert cache.read_error() == 0
    slots = [torch.tensor([int(cache.page_table[0, j // 16]) * 16 + j % 16 for j in range(20)], device="cuda")]
    flat = [c[0].flatten(0, 1) for c in (cache.k, cache.v)]
    want = ref.attention(q[:20], *flat, slots, [0], [20], [20], 0.125, True, 0)
    compare(out[:20], None, want, [20], D, "bfloat16")
    assert (out[20:] == 0).all()                              # rows of a sequence without keys
    cache.plan(ints([1, 6, 0]), rows=7)                       # its tokens again, where there is room
    cache.append(q[:7], k[:7], v[:7], inv, q[:7])
    torch.cuda.synchronize()
    assert cache.read_error() == 0 and cache.kv_len.tolist() == [21, 6, 0]


def test_q_and_k_of_a_step_apart():
    """The forms of the calls that take q alone, or k and v alone, and attention to every key, through the class."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    H, Hk, D, new = 4, 2, 64, [30, 9]
    T = sum(new)
    gen = torch.Generator("cuda").manual_seed(2)
    q, k, v = (torch.randn(T, h, D, device="cuda", generator=gen).bfloat16() for h in (H, Hk, Hk))
    inv = api.rope_inv_freq(D)
    caches, turned = [], []
    for apart in (False, True):
        cache = api.PagedKvCache(20, 16, Hk, D, 2, 64, 64)
        cache.plan(ints(new), rows=T)
        qt = torch.empty_like(q)
        if apart:
            cache.append(None, k, v, inv, None)
            cache.append(q, None, None, inv, qt)
        else:
            cache.append(q, k, v, inv, qt)
        caches.append(cache)
        turned.append(qt)
    assert torch.equal(turned[0], turned[1])
    for a, b in ((caches[0].k, caches[1].k), (caches[0].v, caches[1].v)):
        assert torch.equal(a[0], b[0])
    cache, out, lse = caches[1], torch.empty_like(q), torch.empty(T, H, device="cuda")
    cache.attend(turned[1], 0.125, out, lse, causal=False)
    torch.cuda.synchronize()
    assert cache.read_error() == 0
    slots = [torch.tensor([int(cache.page_table[b, j // 16]) * 16 + j % 16 for j in range(n)], device="cuda") for b, n in enumerate(new)]
    flat = [c[0].flatten(0, 1) for c in (cache.k, cache.v)]
    compare(out, lse, ref.attention(turned[1], *flat, slots, [0, 30], new, new, 0.125, False, 0), new, D, "bfloat16")
    with pytest.raises(api.Fp4MoeError):
        cache.append(None, None, None, inv, None)
    with pytest.raises(api.Fp4MoeError):
        cache.append(q, k, None, inv, q)


# ------------------------------------------------------------------------- angles of far positions
PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494")


@pytest.mark.parametrize("position", [2 ** 31 - 1, 2 ** 31 - 12345, 2 ** 28 + 3, 2 ** 24 + 1, 1000003, -7])
@pytest.mark.parametrize("quarter", [0, 1, 2, 3])
@pytest.mark.parametrize("near", [1.0, 1e-3, 500.0])
def test_rope_angles(position, quarter, near):
    """Angles next to a multiple of a quarter turn, where a cosine or sine is as small as the angle's own error and a bf16
    value shows it: off by at most 2^-25 turns + position |inv_freq| 2^-55. Beside that the sine of an fp32 angle is off by
    2^-22 of itself, and half a step of bf16. Next to whole turns fp32 holds the fraction of a turn to 2^-24 of itself, and
    what is left of 2^-25 is the cut to 32 bits, 2^-32, and that of the step, position 2^-63."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    half = 64
    rng = np.random.default_rng(quarter)
    turns = abs(position) * near / (2 * math.pi)
    freq = np.array([2 * math.pi * (math.floor(turns * (1 + i / half)) + quarter / 4 + rng.normal() * 2.0 ** -27) / abs(position)
                     for i in range(half)])
    x = torch.zeros(1, 1, 2 * half, device="cuda", dtype=torch.bfloat16)
    x[..., :half] = 1.0                                                     # (1, 0) -> (cos, sin)
    out = torch.empty_like(x)
    cache = torch.zeros(1, 1, 1, 2 * half, device="cuda", dtype=torch.bfloat16)
    err = ints([0])
    api.fp4moe_rope_cache(x, None, None, ints([position]), ints([0]), torch.from_numpy(freq).cuda(), out, cache, cache.clone(), err)
    torch.cuda.synchronize()
    assert err.tolist() == [0]
    got = out.double().cpu().numpy().reshape(2, half)
    for i in range(half):
        angle = position * Fraction(float(freq[i])) / (2 * PI)              # in turns
        nearest = round(angle * 4)
        a = float((angle - Fraction(nearest, 4)) * 2 * PI)                  # from the quarter, in radians
        s, c = math.sin(a), math.cos(a)
        want = [(c, s), (-s, c), (-c, -s), (s, -c)][nearest % 4]
        step = abs(position) * freq[i] * 2.0 ** -55
        for part in range(2):
            w = want[part]
            left = 2.0 ** -32 + abs(position) * 2.0 ** -63 if nearest % 4 == 0 and part == 1 else 2.0 ** -25
            # (a cosine next to 1 is off by the square of the angle's error)
            tol = 2 * math.pi * (left + step) + abs(w) * (2.0 ** -22 + ref.HALF_STEP["bfloat16"])
            assert abs(got[part][i] - w) <= tol, (i, part, got[part][i], w, tol, freq[i])
