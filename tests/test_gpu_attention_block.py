"""GPU: the paged cache's calls as they are used together: PagedKvCache over several steps (chunks, decodes, proposed tokens
given back, finished and new sequences), the example's attention half in front of its feed-forward half, streams, graphs.

The reference keeps every sequence's history of turned keys and values on its own and knows nothing of pages."""
import os
import sys

import numpy as np
import pytest

import paged_ref as ref
import synthgen as sg
from helpers import ROOT, ensure_built
from test_gpu_paged import compare, f64, ints

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


class History:
    """What a sequence's cache should hold, as the 16-bit values that the call wrote."""

    def __init__(self, B, Hk, D):
        import torch
        self.k, self.v = ([torch.empty(0, Hk, D, device="cuda") for _ in range(B)] for _ in range(2))

    def step(self, new, k, v):
        import torch
        t = 0
        for b, n in enumerate(new):
            for rows, x in ((self.k, k), (self.v, v)):
                rows[b] = torch.cat([rows[b], x[t:t + n].float()]) if n >= 0 else rows[b][:len(rows[b]) + n]
            t += max(n, 0)

    def attention(self, q, new, scale, window=0):
        """(reference, lengths) over the histories."""
        import torch
        first = np.cumsum([0] + [max(n, 0) for n in new]).tolist()
        lengths = [len(x) for x in self.k]
        k, v = torch.cat(self.k), torch.cat(self.v)
        starts = np.cumsum([0] + lengths).tolist()
        slots = [torch.arange(starts[b], starts[b + 1], device="cuda") for b in range(len(lengths))]
        return ref.attention(q, k, v, slots, first, [max(n, 0) for n in new], lengths, scale, True, window), lengths


STEPS = [[40, 7, 0, 130], [1, 1, 5, 1], [4, 4, 4, 4], [-3, -1, -2, 0], [1, 1, 1, 1], [-43, 1, 90, 1], [33, 1, 1, -137], [1, 1, 1, 12]]


def lengths_stay_positive():
    have = [0] * 4
    for s in STEPS:
        have = [a + b for a, b in zip(have, s)]
        assert min(have) >= 0, s


def cache_rows(cache, layer, kv_len):
    """k and v of each sequence as they lie in the cache now."""
    import torch
    page = cache.page_size
    out = []
    for x in (cache.k[layer], cache.v[layer]):
        flat = x.flatten(0, 1)
        out.append([flat[torch.tensor([int(cache.page_table[b, j // page]) * page + j % page for j in range(L)], dtype=torch.long,
                                      device="cuda")] for b, L in enumerate(kv_len)])
    return out


@pytest.mark.parametrize("page", [1, 16, 24])
@pytest.mark.parametrize("D,dtype,window", [(64, "bfloat16", 0), (128, "float16", 0), (80, "bfloat16", 50)])
def test_a_cache_over_many_steps(page, D, dtype, window):
    import torch
    from block_scaled_fp4_top_gb300 import api
    lengths_stay_positive()
    H, Hk, B, layers = 6, 2, 4, 2
    dt = getattr(torch, dtype)
    cache = api.PagedKvCache(400 // page + 24, page, Hk, D, B, 260, 200, layers, dt)
    inv = api.rope_inv_freq(D, device="cuda")
    hist = [History(B, Hk, D) for _ in range(layers)]
    gen = torch.Generator("cuda").manual_seed(page + D)
    for new in STEPS:
        T = sum(max(n, 0) for n in new)
        cache.plan(ints(new))
        if T == 0:
            for layer in range(layers):
                hist[layer].step(new, torch.empty(0, Hk, D, device="cuda"), torch.empty(0, Hk, D, device="cuda"))
            continue
        pos = cache.position[:T].cpu().numpy()
        for layer in range(layers):
            qkv = torch.randn(T, H + 2 * Hk, D, device="cuda", generator=gen).to(dt)
            q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
            want_k, mag = ref.rotate(f64(k), pos, inv.cpu().numpy(), 0, False, 1.0)
            qt, out = torch.empty_like(q.contiguous()), torch.empty(T, H, D, dtype=dt, device="cuda")
            lse = torch.empty(T, H, device="cuda")
            cache.append(q, k, v, inv, qt, layer=layer)
            cache.attend(qt, D ** -0.5, out, lse, window, layer)
            torch.cuda.synchronize()
            assert cache.read_error() == 0
            # the new keys by definition (half a step), then their stored values go into the history
            kv_len = cache.kv_len.tolist()
            rows_k, rows_v = cache_rows(cache, layer, kv_len)
            new_k = torch.cat([rows_k[b][len(rows_k[b]) - max(n, 0):] for b, n in enumerate(new)])
            new_v = torch.cat([rows_v[b][len(rows_v[b]) - max(n, 0):] for b, n in enumerate(new)])
            # cosine, sine, products: 2^-21 of |x| + |y|; then one rounding: half a step of the value, but no less than half a
            # step of the subnormals (TINY): fp16 values below 2^-14 lie 2^-24 apart, more than 2^-10 of themselves
            rel = mag * 2.0 ** -21
            bound = (np.abs(want_k) + rel) * ref.HALF_STEP[dtype] + ref.TINY[dtype] + rel
            assert (np.abs(f64(new_k) - want_k) <= bound).all()
            assert torch.equal(new_v, v)
            hist[layer].step(new, new_k, new_v)
            for b in range(B):  # nothing else of any sequence has changed
                assert torch.equal(rows_k[b].float(), hist[layer].k[b]) and torch.equal(rows_v[b].float(), hist[layer].v[b])
            want, lengths = hist[layer].attention(qt, new, D ** -0.5, window)
            assert lengths == kv_len
            compare(out, lse, want, lengths, D, dtype)
    used = sum(ref.pages(L, page) for L in cache.kv_len.tolist())
    assert int(cache.free_count) == cache.free_pages.numel() - used
    left = cache.free_pages[:int(cache.free_count)].tolist()
    held = [int(cache.page_table[b, j]) for b, L in enumerate(cache.kv_len.tolist()) for j in range(ref.pages(L, page))]
    assert sorted(left + held) == list(range(cache.free_pages.numel()))        # every page once


def test_one_decode_graph_serves_every_step():
    """A captured step replayed as lengths grow past pages and past what they were at capture; padded rows stay out."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    B, H, Hk, D, page, rows = 3, 8, 2, 128, 16, 5
    prompt = [30, 1, 200]
    inv = api.rope_inv_freq(D)
    gen = torch.Generator("cuda").manual_seed(2)
    pq = torch.randn(sum(prompt), H + 2 * Hk, D, device="cuda", generator=gen).bfloat16()
    steps = [torch.randn(rows, H + 2 * Hk, D, device="cuda", generator=gen).bfloat16() for _ in range(40)]
    outs = []
    for captured in (False, True):
        cache = api.PagedKvCache(60, page, Hk, D, B, 300, 300)
        new, x = ints(prompt), steps[0].clone()
        q = torch.empty(300, H, D, dtype=torch.bfloat16, device="cuda")
        out = torch.full((rows, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        cache.plan(new)
        cache.append(pq[:, :H], pq[:, H:H + Hk], pq[:, H + Hk:], inv, q[:sum(prompt)])
        new.fill_(1)

        def step():
            cache.plan(new)
            cache.append(x[:, :H], x[:, H:H + Hk], x[:, H + Hk:], inv, q[:rows])
            cache.attend(q[:rows], D ** -0.5, out)

        got = []
        if captured:
            lens, state = cache.kv_len.clone(), (cache.free_count.clone(), cache.free_pages.clone(), cache.page_table.clone())
            step()
            torch.cuda.synchronize()
            cache.kv_len.copy_(lens)
            for t, s in zip((cache.free_count, cache.free_pages, cache.page_table), state):
                t.copy_(s)
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                step()
        for x_t in steps:
            x.copy_(x_t)
            graph.replay() if captured else step()
            got.append(out.clone())
        torch.cuda.synchronize()
        assert cache.read_error() == 0 and cache.kv_len.tolist() == [p + 40 for p in prompt]
        assert (out[B:] == 7.0).all()                                      # rows without a sequence
        outs.append(got)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_two_graphs_share_a_workspace():
    """Two captured attentions of different sizes on one workspace, replayed in turn, and an eager one in between."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    from test_gpu_paged import attention_case
    ws, err = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda"), ints([0])
    jobs = []
    for new, kv, D in (([1, 1], [3000, 17], 128), ([200, 3], [900, 2000], 64), ([4], [5000], 80)):
        q, kc, vc, flat, table, slots = attention_case(new, kv, 8, 2, D)
        first = [sum(new[:b]) for b in range(len(new) + 1)]
        out = torch.empty_like(q)
        args = (q, kc, vc, table, ints(kv), ints(first), D ** -0.5, out, None, ws, err)
        api.fp4moe_paged_attention(*args)
        torch.cuda.synchronize()
        jobs.append((args, out, out.clone()))
    graphs = []
    for args, _, _ in jobs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.fp4moe_paged_attention(*args)
        graphs.append(g)
    for _ in range(5):
        for (_, out, want), g in zip(jobs, graphs):
            out.zero_()
            g.replay()
        jobs[2][1].zero_()
        api.fp4moe_paged_attention(*jobs[2][0])
        torch.cuda.synchronize()
        for _, out, want in jobs:
            assert torch.equal(out, want)
    assert err.tolist() == [0]


def test_two_streams_with_workspaces_of_their_own():
    import torch
    from block_scaled_fp4_top_gb300 import api
    from test_gpu_paged import attention_case
    q, kc, vc, flat, table, slots = attention_case([60, 9, 1], [700, 300, 900], 8, 2, 64)
    bufs = []
    for _ in range(2):
        bufs.append((torch.empty_like(q), torch.zeros(64 << 20, dtype=torch.uint8, device="cuda"), ints([0]), torch.cuda.Stream()))
    kv, first = ints([700, 300, 900]), ints([0, 60, 69, 70])
    torch.cuda.synchronize()
    for _ in range(10):
        for out, ws, err, s in bufs:
            api.fp4moe_paged_attention(q, kc, vc, table, kv, first, 0.125, out, None, ws, err, stream=s)
    torch.cuda.synchronize()
    want = ref.attention(q, *flat, slots, [0, 60, 69], [60, 9, 1], [700, 300, 900], 0.125, True, 0)
    for out, _, err, _ in bufs:
        assert err.tolist() == [0]
        compare(out, None, want, [900], 64, "bfloat16")
    assert torch.equal(bufs[0][0], bufs[1][0])


def test_a_call_that_finds_a_timeout_skips_its_work():
    """As the 4-bit product does; the word is cleared with fp4moe_read_error."""
    import torch
    from block_scaled_fp4_top_gb300 import _lib, api
    from test_gpu_paged import attention_case
    for new in ([1, 1], [60, 70]):
        q, kc, vc, flat, table, slots = attention_case(new, [200, 100], 8, 2, 64)
        ws, err = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda"), ints([_lib.ERR_TIMEOUT, 0, 0, 0])
        out = torch.full_like(q, 5.0)
        args = (q, kc, vc, table, ints([200, 100]), ints([0, new[0], sum(new)]), 0.125, out, None, ws, err)
        api.fp4moe_paged_attention(*args)
        torch.cuda.synchronize()
        assert (out == 5.0).all() and api.fp4moe_read_error(err) == _lib.ERR_TIMEOUT
        api.fp4moe_paged_attention(*args)
        torch.cuda.synchronize()
        want = ref.attention(q, *flat, slots, [0, new[0]], new, [200, 100], 0.125, True, 0)
        compare(out, None, want, [200], 64, "bfloat16")
        assert err.tolist() == [0, 0, 0, 0]


def test_the_example_block_with_its_attention_half():
    """Prompts and decode steps through norm, projection, cache and attention, then projection, norm and experts."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    from dense_ref import rms_norm
    from decoder_block import make_attention, make_block
    wl = sg.TINY_SHARED
    heads, kv_heads, D, B = 4, 2, 64, wl.T
    cache = api.PagedKvCache(8 * B, 16, kv_heads, D, B, 100, 9 * B)
    attn = make_attention(wl, heads, kv_heads, D, cache, 9 * B)
    block, _ = make_block(wl, heads * D)
    gen = torch.Generator("cuda").manual_seed(4)
    hist = History(B, kv_heads, D)
    inv = attn.inv_freq.cpu().numpy()
    for new in ([1 + b % 9 for b in range(B)], [1] * B, [1] * B):
        T = sum(new)
        h = torch.randn(T, wl.H, device="cuda", generator=gen).bfloat16()
        cache.plan(ints(new))
        o = attn.forward(h)
        torch.cuda.synchronize()
        n = rms_norm(f64(h), f64(attn.gamma), attn.eps)
        assert (np.abs(f64(attn.n[:T]) - n) <= np.abs(n) * (2.0 ** -8 + 2.0 ** -20)).all()
        raw = torch.empty(T, (heads + 2 * kv_heads) * D, dtype=torch.bfloat16, device="cuda")
        attn.proj.forward(attn.n[:T].contiguous(), raw)
        raw = f64(raw).reshape(T, heads + 2 * kv_heads, D)
        turned, mag = ref.rotate(raw[:, :heads + kv_heads], cache.position[:T].cpu().numpy(), inv, 0, False, 1.0)
        got = attn.qkv[:T]
        rows_k, rows_v = cache_rows(cache, 0, cache.kv_len.tolist())
        new_k, new_v = (torch.cat([r[b][len(r[b]) - n_b:] for b, n_b in enumerate(new)]) for r in (rows_k, rows_v))
        bound = np.abs(turned) * 2.0 ** -8 + mag * 2.0 ** -20
        assert (np.abs(f64(got[:, :heads]) - turned[:, :heads]) <= bound[:, :heads]).all()      # q, turned in place
        assert (np.abs(f64(new_k) - turned[:, heads:]) <= bound[:, heads:]).all()
        assert (f64(new_v) == raw[:, heads + kv_heads:]).all()
        hist.step(new, new_k, new_v)
        want, lengths = hist.attention(got[:, :heads], new, attn.scale)
        compare(o.view(T, heads, D), None, want, lengths, D, "bfloat16")
        if T == B:  # a decode step, through the experts as well
            h0, y = h.clone(), block.forward(o, h)
            torch.cuda.synchronize()
            assert torch.isfinite(y).all() and not torch.equal(h, h0)
        assert attn.read_error() | block.read_error() == 0


def test_the_example_runs():
    import subprocess
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decoder_block.py"), "--tiny"], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "graph replay equals eager: True" in r.stdout and r.stdout.count("error word 0x0") == 2, r.stdout
