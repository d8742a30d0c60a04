"""Argument checks and sizes of the paged 8-bit cache's entry points, without a GPU.

Every call below is refused, or is empty, before any CUDA call.
"""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def kq():
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    import quantized_decode_gemv_block_gb300 as m
    m.load_library()
    return m


FAKE = 1 << 20  # never dereferenced


def cache_c(kq, **kw):
    a = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, n_pages=10, page_size=32, n_kv=2, head_dim=64)
    a.update(kw)
    return kq.KV8CacheC(*[a[f[0]] for f in kq.KV8CacheC._fields_])


def test_cache_sizes(kq):
    L = kq.lib()
    assert L.kq_kv8_bytes(10, 32, 4, 128) == 10 * 32 * 4 * 128
    assert L.kq_kv8_bytes(1 << 20, 128, 8, 128) == (1 << 20) * 128 * 8 * 128  # passes 32 bits
    for bad in ((-1, 32, 4, 128), (10, 24, 4, 128), (10, 32, 0, 128), (10, 32, 4, 96), (1 << 27, 16, 1, 64)):
        assert L.kq_kv8_bytes(*bad) == 0
    # slots of 512 positions plus one per request, query rows of up to 32 tokens, D sums and two statistics
    assert L.kq_attention_kv8_workspace_size(3, 1000, 1, 16, 4, 128) == (1000 // 512 + 3) * 4 * 4 * 130 * 4
    assert L.kq_attention_kv8_workspace_size(3, 1000, 500, 16, 4, 128) == (1000 // 512 + 3) * 4 * 4 * 32 * 130 * 4
    for bad in ((-1, 10, 1, 4, 4, 64), (4097, 10, 1, 4, 4, 64), (1, -1, 1, 4, 4, 64), (1, 10, 1, 6, 4, 64), (1, 10, 1, 4, 4, 80),
                (1, 10, -1, 4, 4, 64), (1, 10, 1, 130, 2, 64)):
        assert L.kq_attention_kv8_workspace_size(*bad) == 0


def test_pages_refusals(kq):
    L = kq.lib()
    good = dict(ctx=FAKE, new=FAKE, B=4, P=32, table=FAKE, width=8, free=FAKE, cap=100, nf=FAKE, nfo=FAKE + 4, cu=FAKE, pos=FAKE,
                slot=FAKE, T=16, status=FAKE)

    def plan(**kw):
        a = dict(good, **kw)
        return L.kq_pages_plan(a["ctx"], a["new"], a["B"], a["P"], a["table"], a["width"], a["free"], a["cap"], a["nf"],
                               a["nfo"], a["cu"], a["pos"], a["slot"], a["T"], a["status"], None)

    def release(**kw):
        a = dict(good, **kw)
        return L.kq_pages_release(a["ctx"], a["new"], a["B"], a["P"], a["table"], a["width"], a["free"], a["cap"], a["nf"],
                                  a["nfo"], a["status"], None)
    for f in (plan, release):
        for kw in (dict(B=-1), dict(B=4097), dict(P=0), dict(P=24), dict(P=256), dict(width=-1), dict(width=1 << 26), dict(cap=-1),
                   dict(nf=None), dict(nfo=None), dict(nfo=FAKE), dict(status=None), dict(ctx=None), dict(new=None), dict(table=None),
                   dict(free=None), dict(ctx=FAKE + 2), dict(table=FAKE + 1)):
            assert f(**kw) == kq.KQ_ERR_ARG, (f, kw)
            assert L.kq_last_error().decode() != ""
    for kw in (dict(T=-1), dict(cu=None), dict(pos=None), dict(slot=None), dict(slot=FAKE + 2)):
        assert plan(**kw) == kq.KQ_ERR_ARG, kw


def test_rope_refusals(kq):
    L = kq.lib()
    good = dict(xd=kq.BF16, yd=kq.BF16, q=FAKE, qs=512, qo=FAKE + 65536, qos=512, nq=4, k=FAKE, ks=256, ko=FAKE + 65536, kos=256, nk=2,
                T=3, D=128, rot=128, fr=FAKE, ax=None, pos=FAKE, na=1, fl=0)

    def rope(**kw):
        a = dict(good, **kw)
        return L.kq_rope(a["xd"], a["yd"], a["q"], a["qs"], a["qo"], a["qos"], a["nq"], a["k"], a["ks"], a["ko"], a["kos"],
                         a["nk"], a["T"], a["D"], a["rot"], a["fr"], a["ax"], a["pos"], a["na"], a["fl"], None)
    assert rope(xd=9) == kq.KQ_ERR_UNSUPPORTED and rope(yd=0) == kq.KQ_ERR_UNSUPPORTED
    for kw in (dict(fl=4), dict(T=-1), dict(nq=-1), dict(D=0), dict(rot=130), dict(rot=7), dict(na=0), dict(na=256), dict(qs=511),
               dict(kos=255), dict(q=None), dict(ko=None), dict(fr=None), dict(pos=None), dict(q=FAKE + 1),
               dict(qo=FAKE, yd=kq.F32), dict(qo=FAKE, qos=1024)):
        assert rope(**kw) == kq.KQ_ERR_ARG, kw
    assert rope(T=0) == 0 and rope(nq=0, nk=0, q=None, k=None) == 0


def test_append_and_attention_refusals(kq):
    L = kq.lib()
    c = cache_c(kq)

    def append(cache=c, xd=kq.BF16, k=FAKE, ks=128, v=FAKE, vs=128, slot=FAKE, T=3):
        return L.kq_kv8_append(ctypes.addressof(cache) if cache is not None else None, xd, k, ks, v, vs, slot, T, None)
    assert append(cache=None) == kq.KQ_ERR_ARG
    for kw in (dict(page_size=48), dict(head_dim=80), dict(n_kv=0), dict(n_pages=-1), dict(n_pages=1 << 27), dict(k=None),
               dict(v_scale=None), dict(v=FAKE + 8), dict(k_scale=FAKE + 2)):
        assert append(cache=cache_c(kq, **kw)) == kq.KQ_ERR_ARG, kw
    assert append(xd=5) == kq.KQ_ERR_UNSUPPORTED
    for kw in (dict(T=-1), dict(ks=120), dict(vs=130), dict(k=None), dict(slot=None), dict(k=FAKE + 8), dict(slot=FAKE + 2)):
        assert append(**kw) == kq.KQ_ERR_ARG, kw
    assert append(T=0) == 0

    good = dict(qd=kq.BF16, q=FAKE, qs=256, od=kq.BF16, o=FAKE, os=256, nq=4, ctx=FAKE, new=FAKE, B=2, T=3, mn=2, ml=100, tl=200,
                table=FAKE, width=4, mask=None, ws=FAKE, wsn=1 << 30)

    def attn(cache=c, **kw):
        a = dict(good, **kw)
        return L.kq_attention_kv8(ctypes.addressof(cache), a["qd"], a["q"], a["qs"], a["od"], a["o"], a["os"], a["nq"], a["ctx"], a["new"],
                                  a["B"], a["T"], a["mn"], a["ml"], a["tl"], a["table"], a["width"], a["mask"], 0.1, a["ws"], a["wsn"], None)
    assert attn(qd=7) == kq.KQ_ERR_UNSUPPORTED and attn(od=0) == kq.KQ_ERR_UNSUPPORTED
    for kw in (dict(nq=3), dict(nq=0), dict(nq=130, qs=65536, os=65536), dict(B=-1), dict(B=4097), dict(T=-1), dict(T=(1 << 20) + 1),
               dict(mn=-1), dict(ml=-1), dict(ml=1 << 29), dict(tl=-1), dict(width=-1), dict(qs=255), dict(os=260), dict(q=None), dict(o=None),
               dict(ctx=None), dict(new=None), dict(table=None), dict(q=FAKE + 8), dict(mask=FAKE, mn=33), dict(mask=FAKE + 2)):
        assert attn(**kw) == kq.KQ_ERR_ARG, kw
    assert attn(cache=cache_c(kq, head_dim=96)) == kq.KQ_ERR_ARG
    need = L.kq_attention_kv8_workspace_size(2, 200, 2, 4, 2, 64)
    assert attn(ws=None) == kq.KQ_ERR_WORKSPACE and attn(wsn=need - 1) == kq.KQ_ERR_WORKSPACE and attn(ws=FAKE + 64) == kq.KQ_ERR_WORKSPACE
    assert attn(T=0) == 0 and attn(B=0) == 0


def test_binding_refuses_wrong_tensors(kq):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    cache = kq.KV8Cache(2, 16, 2, 64, device="cpu")
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(kq.KQError):
        kq.KV8Cache(2, 24, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        kq.KV8Cache(2, 16, 2, 64, k=torch.zeros((2, 2, 1023), dtype=torch.int8), v=cache.v, k_scale=cache.k_scale, v_scale=cache.v_scale)
    with pytest.raises(TypeError):
        kq.kv8_append(cache, k.half(), k.half(), i(3), stream=0)
    with pytest.raises(ValueError):
        kq.kv8_append(cache, k, k[:2], i(3), stream=0)
    with pytest.raises(ValueError):
        kq.kv8_append(cache, k, k, i(2), stream=0)
    with pytest.raises(ValueError):
        kq.kv8_append(cache, k.transpose(0, 1).contiguous().transpose(0, 1), k, i(3), stream=0)  # heads apart
    with pytest.raises(ValueError):
        kq.pages_plan(i(2).long(), i(2), i(2, 4), i(9), i(1), 16, 8, out=kq.PagesPlan(2, 8, "cpu"), stream=0)
    with pytest.raises(ValueError):
        kq.rope(k, k[:2], i(3), torch.zeros(32), stream=0)
    with pytest.raises(ValueError):
        kq.rope(k, None, i(2), torch.zeros(32), stream=0)
    with pytest.raises(ValueError):
        kq.rope(None, None, i(2), torch.zeros(32), stream=0)
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kq.attention_kv8(q, cache, i(2, 1), i(1), i(2), 1, 16, stream=0)
    with pytest.raises(ValueError):
        kq.attention_kv8(q, cache, i(2, 1), i(2), i(2), 1, 16, out=q[:2], stream=0)
    with pytest.raises(kq.KQError):
        kq.attention_kv8(torch.zeros((3, 3, 64), dtype=torch.bfloat16), cache, i(2, 1), i(2), i(2), 1, 16, stream=0)


def test_tensors_in_host_memory_are_refused_where_there_is_a_gpu(kq, monkeypatch):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    cache = kq.KV8Cache(2, 16, 2, 64, device="cpu")
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    for call in (lambda: kq.kv8_append(cache, x, x, i(3), stream=0),
                 lambda: kq.attention_kv8(x, cache, i(2, 1), i(2), i(2), 1, 16, stream=0),
                 lambda: kq.rope(x, None, i(3), torch.zeros(32), stream=0),
                 lambda: kq.pages_plan(i(2), i(2), i(2, 4), i(9), i(1), 16, 8, stream=0),
                 lambda: kq.pages_release(i(2), i(2).bool(), i(2, 4), i(9), i(1), i(1), 16, stream=0)):
        with pytest.raises(ValueError, match="must be on the GPU"):
            call()


def test_calls_of_more_tokens_than_the_kernels_count(kq):
    """Above 2^30 an int index that moves by a grid of threads could pass 2^31."""
    L, big = kq.lib(), (1 << 30) + 1
    c = cache_c(kq)
    assert L.kq_pages_plan(FAKE, FAKE, 4, 32, FAKE, 8, FAKE, 100, FAKE, FAKE + 4, FAKE, FAKE, FAKE, big, FAKE, None) == kq.KQ_ERR_ARG
    assert L.kq_pages_plan(FAKE, FAKE, 4, 32, FAKE, 8, FAKE, big, FAKE, FAKE + 4, FAKE, FAKE, FAKE, 16, FAKE, None) == kq.KQ_ERR_ARG
    assert L.kq_pages_release(FAKE, FAKE, 4, 32, FAKE, 8, FAKE, big, FAKE, FAKE + 4, FAKE, None) == kq.KQ_ERR_ARG
    assert L.kq_rope(kq.BF16, kq.BF16, FAKE, 1, FAKE, 1, 1, None, 0, None, 0, 0, big, 1, 0, None, None, None, 1, 0, None) == kq.KQ_ERR_ARG
    assert L.kq_kv8_append(ctypes.addressof(c), kq.BF16, FAKE, 128, FAKE, 128, FAKE, big, None) == kq.KQ_ERR_ARG


def test_rope_positions_of_several_axes_have_a_row_of_tokens_each(kq):
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="axes, tokens"):
        kq.rope(x, None, torch.zeros((2, 4), dtype=torch.int32), torch.zeros(32), stream=0)
