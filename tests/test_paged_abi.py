"""The paged key-value cache's calls on the CPU: every refusal of the C calls and of the binding. No call here reaches
a CUDA API: each fails validation first, or has nothing to do."""
import ctypes

import pytest
import torch

from helpers import ensure_built

P, Q = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000)    # aligned, never dereferenced
BAD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    from block_scaled_fp4_top_gb300 import _lib
    return _lib.load()


def kv(**k):
    from block_scaled_fp4_top_gb300 import _lib
    d = dict(dtype=0, kv_heads=2, head_dim=64, page_size=16, num_pages=8, page_stride=2048, token_stride=128, head_stride=64) | k
    return _lib.KvCache(*[d[n] for n, _ in _lib.KvCache._fields_])


BAD_CACHES = [(dict(dtype=2), "UNSUPPORTED"), (dict(dtype=-1), "UNSUPPORTED"), (dict(head_dim=4), "UNSUPPORTED"),
              (dict(head_dim=100), "UNSUPPORTED"), (dict(head_dim=264), "UNSUPPORTED"), (dict(head_dim=0), "UNSUPPORTED"),
              (dict(kv_heads=0), "INVALID_ARG"), (dict(kv_heads=65536), "INVALID_ARG"), (dict(page_size=0), "INVALID_ARG"),
              (dict(num_pages=0), "INVALID_ARG"), (dict(page_size=65536, num_pages=32768), "INVALID_ARG"),
              (dict(page_stride=2044), "INVALID_ARG"), (dict(token_stride=-128), "INVALID_ARG"), (dict(head_stride=2 ** 40), "INVALID_ARG")]


def test_sizes_of_the_binding_are_the_headers(lib):
    import os
    import re
    from block_scaled_fp4_top_gb300 import _lib
    from helpers import ROOT
    with open(os.path.join(ROOT, "include", "fp4moe.h")) as f:
        text = f.read()
    assert int(re.search(r"FP4MOE_KV_MAX_SEQS (\d+)", text)[1]) == _lib.KV_MAX_SEQS
    assert int(re.search(r"FP4MOE_ATTENTION_WORKSPACE_BYTES \((\d+)u << 20\)", text)[1]) << 20 == _lib.ATTENTION_WORKSPACE_BYTES
    assert int(re.search(r"FP4MOE_ERR_PAGE\s+(0x[0-9a-f]+)u", text)[1], 16) == _lib.ERR_PAGE


def test_plan_refusals(lib):
    from block_scaled_fp4_top_gb300 import _lib
    names = ("cached", "new", "table", "free", "count", "kv_len", "count_out", "offset", "position", "slot", "err")

    def f(B=4, page=16, pages=8, columns=4, rows=64, **k):
        a = {n: P for n in names} | k
        return lib.fp4moe_kv_plan(B, page, pages, a["cached"], a["new"], a["table"], columns, a["free"], a["count"], a["kv_len"],
                                  a["count_out"], a["offset"], rows, a["position"], a["slot"], a["err"], None)

    for bad in (dict(B=-1), dict(page=0), dict(pages=0), dict(columns=-1), dict(rows=-1), dict(page=2 ** 16, pages=2 ** 15)):
        assert f(**bad) == _lib.INVALID_ARG, bad
    assert f(B=8193) == _lib.UNSUPPORTED
    for n in names:
        assert f(**{n: None}) == _lib.INVALID_ARG, n
        assert f(**{n: BAD}) == _lib.MISALIGNED, n


def test_rope_refusals(lib):
    from block_scaled_fp4_top_gb300 import _lib
    ptrs = ("q", "k", "v", "position", "slot", "inv", "qo", "kc", "vc", "err")

    def f(cache=None, T=4, H=6, qs=384, ks=128, vs=128, first=0, rot=64, amp=1.0, qos=384, **p):
        a = {n: P for n in ptrs} | {"vc": Q} | p
        return lib.fp4moe_rope_cache(kv(**(cache or {})), T, H, a["q"], qs, a["k"], ks, a["v"], vs, a["position"], a["slot"], first,
                                     rot, 0, a["inv"], amp, a["qo"], qos, a["kc"], a["vc"], a["err"], None)

    for c, want in BAD_CACHES:
        assert f(c) == getattr(_lib, want), c
    assert lib.fp4moe_rope_cache(None, 0, 0, *[P, 0] * 3, P, P, 0, 0, 0, P, 1.0, P, 0, P, P, P, None) == _lib.INVALID_ARG
    for bad in (dict(T=-1), dict(H=-1), dict(H=65532), dict(T=2 ** 31 - 1), dict(first=-2), dict(first=2), dict(rot=-2), dict(rot=3),
                dict(rot=66), dict(first=2 ** 31 - 1, rot=2), dict(amp=float("nan")), dict(amp=float("inf")), dict(qs=376), dict(qs=388),
                dict(qos=376), dict(ks=120), dict(vs=132), dict(qs=-384, T=1), dict(qs=2 ** 40)):
        assert f(**bad) == _lib.INVALID_ARG, bad
    for n in ptrs:  # q and q_out, and k, v and the caches, are given together
        assert f(**{n: None}) == _lib.INVALID_ARG, n
        assert f(**{n: BAD}) == _lib.MISALIGNED, n
    assert f(vc=P) == _lib.INVALID_ARG                          # two results, one buffer
    assert f(q=None, qo=None) == _lib.INVALID_ARG               # heads of no q
    assert f(q=None, qo=None, H=0, k=None, v=None, kc=None, vc=None) == _lib.OK   # nothing to do
    assert f(T=0) == _lib.OK and f(T=0, q=None, k=None, err=None) == _lib.OK


def test_attention_refusals(lib):
    from block_scaled_fp4_top_gb300 import _lib
    ptrs = ("kc", "vc", "q", "table", "kv_len", "offset", "out", "ws", "err")

    def f(cache=None, B=2, T=4, H=6, qs=384, columns=4, scale=0.125, causal=1, window=0, os=384, lse=P, **p):
        a = {n: P for n in ptrs} | {"out": Q} | p
        return lib.fp4moe_paged_attention(kv(**(cache or {})), a["kc"], a["vc"], B, T, H, a["q"], qs, a["table"], columns, a["kv_len"],
                                          a["offset"], scale, causal, window, a["out"], os, lse, a["ws"], a["err"], None)

    for c, want in BAD_CACHES:
        assert f(c) == getattr(_lib, want), c
    for bad in (dict(B=-1), dict(T=-1), dict(columns=-1), dict(window=-1), dict(H=0), dict(H=5), dict(T=2 ** 30), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(causal=0, window=3), dict(qs=380),
                dict(qs=376), dict(os=376), dict(os=2 ** 40), dict(out=P)):
        assert f(**bad) == _lib.INVALID_ARG, bad
    assert f(scale=3.4e38) == _lib.INVALID_ARG
    assert f(B=8193) == _lib.UNSUPPORTED and f(columns=2 ** 27 - 63) == _lib.UNSUPPORTED
    for n in ptrs:
        assert f(**{n: None}) == _lib.INVALID_ARG, n
        assert f(**{n: BAD}) == _lib.MISALIGNED, n
    assert f(lse=BAD) == _lib.MISALIGNED
    assert f(T=0, q=None, out=None) == _lib.OK and f(B=0, table=None) == _lib.OK


def test_attention_plan(lib):
    """Which kernel takes what: the sizes that the GPU tests use for each do take it."""
    from block_scaled_fp4_top_gb300 import _lib, api
    plan = api.fp4moe_paged_attention_plan
    for B, T, H, Hk, D, want in ((1, 1, 32, 8, 128, 16), (64, 64, 32, 8, 128, 16), (16, 64, 64, 8, 64, 32), (16, 65, 64, 8, 64, 256), (16, 32, 64, 8, 64, 16),
                                 (1, 8, 32, 8, 64, 32), (1, 24, 32, 8, 64, 32), (1, 25, 32, 8, 64, 256), (8, 2048, 32, 8, 128, 256),
                                 (1, 8, 32, 8, 128, 16), (4, 32, 32, 8, 128, 256), (1, 8192, 32, 8, 136, 16), (1, 8192, 32, 8, 256, 16),
                                 (0, 0, 8, 8, 64, 16), (1, 2**31 // 64 - 1, 64, 1, 64, 256), (8192, 8192, 1, 1, 8, 16)):
        assert plan(B, T, H, Hk, D) == want, (B, T, H, Hk, D)
    p = lib.fp4moe_paged_attention_plan
    assert p(kv(), 1, 1, 3, None) == _lib.INVALID_ARG and p(kv(), -1, 1, 2, None) == _lib.INVALID_ARG
    assert p(kv(), 1, -1, 2, None) == _lib.INVALID_ARG and p(kv(), 8193, 1, 2, None) == _lib.UNSUPPORTED
    assert p(None, 1, 1, 2, None) == _lib.INVALID_ARG and p(kv(), 1, 1, 2, None) == _lib.OK      # outputs optional
    for c, want in BAD_CACHES:
        assert p(kv(**c), 1, 1, 2, None) == getattr(_lib, want), c


def test_binding_refuses_wrong_shapes_and_types():
    """The C calls see pointers only, so the binding holds every tensor to its shape and type; and every tensor here is on
    the host, which is refused before any call too."""
    from block_scaled_fp4_top_gb300 import api
    E = api.Fp4MoeError
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    h = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d)  # noqa: E731
    good = dict(cached=i(3), new=i(3), table=i(3, 4), free=i(9), count=i(1), kv_len=i(3), count_out=i(1), offset=i(4), position=i(8),
                slot=i(8), err=i(4))
    for bad in [{}, dict(new=i(2)), dict(table=i(2, 4)), dict(table=i(12)), dict(offset=i(3)), dict(position=i(7)),
                dict(new=torch.zeros(3)), dict(table=i(4, 3).t()), dict(count=i(2)), dict(err=h(1)), dict(kv_len=i(3).long())]:
        a = good | bad
        with pytest.raises(E):
            api.fp4moe_kv_plan(16, a["cached"], a["new"], a["table"], a["free"], a["count"], a["kv_len"], a["count_out"],
                               a["offset"], a["position"], a["slot"], a["err"])
    good = dict(q=h(5, 6, 64), k=h(5, 2, 64), v=h(5, 2, 64), position=i(5), slot=i(5), inv=torch.zeros(32, dtype=torch.float64),
                qo=h(5, 6, 64), kc=h(8, 16, 2, 64), vc=h(8, 16, 2, 64), err=i(1))
    for bad in [{}, dict(q=h(4, 6, 64)), dict(q=h(5, 6, 32)), dict(q=h(5, 6, 64, d=torch.float16)), dict(qo=h(5, 5, 64)), dict(qo=None),
                dict(k=h(5, 3, 64)), dict(k=None), dict(v=h(5, 64)), dict(inv=torch.zeros(32)), dict(kc=h(8, 16, 2, 64, d=torch.float32)),
                dict(vc=h(8, 16, 64, 2).transpose(2, 3)), dict(vc=h(8, 2, 16, 64).transpose(1, 2)), dict(kc=h(8, 16, 128)),
                dict(q=h(5, 64, 6).transpose(1, 2)), dict(q=h(5, 6, 68)[..., :64]), dict(position=i(4))]:
        a = good | bad
        with pytest.raises(E):
            api.fp4moe_rope_cache(a["q"], a["k"], a["v"], a["position"], a["slot"], a["inv"], a["qo"], a["kc"], a["vc"], a["err"])
    good = dict(q=h(5, 6, 64), kc=h(8, 16, 2, 64), vc=h(8, 16, 2, 64), table=i(2, 4), kv_len=i(2), offset=i(3), out=h(5, 6, 64),
                lse=torch.zeros(5, 6), ws=torch.zeros(64 << 20, dtype=torch.uint8), err=i(1))
    for bad in [{}, dict(q=h(5, 6, 32)), dict(out=h(5, 4, 64)), dict(out=h(4, 6, 64)), dict(table=i(3, 4)), dict(offset=i(2)),
                dict(lse=torch.zeros(6, 5)), dict(ws=torch.zeros(100, dtype=torch.uint8)), dict(kc=h(8, 16, 64)), dict(kv_len=i(2).long())]:
        a = good | bad
        with pytest.raises(E):
            api.fp4moe_paged_attention(a["q"], a["kc"], a["vc"], a["table"], a["kv_len"], a["offset"], 0.125, a["out"], a["lse"],
                                       a["ws"], a["err"])
    for bad in (dict(rot_dim=3), dict(rot_dim=-2), dict(rot_dim=4, base=0.0), dict(rot_dim=4, factor=0.0), dict(rot_dim=4, slow=32.0)):
        with pytest.raises(E):
            api.rope_inv_freq(**bad)
