"""The paged 8-bit cache: append (exact) and attention against 64-bit forms, masks, bounds, invariance, capture.

Attention's tolerance per element, base = sum_p w_p |v_p|, mag = largest sum_d |scale q_d k_pd|:
 - fp32 output: q in two fp16 parts (2^-22 of each product), fp32 sums of D <= 128 products (below 2^-18 of their magnitudes
   even if every addition erred alike), so a score is off by under mag 2^-17; a weight by that plus 2^-21 (exp2, two parts),
   the sum and its norm together by twice that: base (2 mag 2^-17 + 2^-19), and 2^-23 of the result;
 - bf16 output: fp16 q and weights, half a step of 2^-11 each in place of 2^-22: scores off by mag 2^-12 for fp32 q and
   nothing for bf16 q (exact in fp16), weights by 2^-12: base (2 mag (2^-12 or 0 + 2^-17) + 2^-11), and 2^-8 of the result.
"""
import numpy as np
import pytest
import torch

import kv8_plain as plain
import quantized_decode_gemv_block_gb300 as kq

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    yield
    assert kq.device_errors() == 0


def dev(a, dtype=np.int32):
    return torch.tensor(np.asarray(a, dtype), device="cuda")


# ---------------------------------------------------------------- append

def codes(cache, which):
    raw = (cache.k if which == "k" else cache.v).cpu().numpy().reshape(cache.n_pages, cache.n_kv, -1)
    return plain.codes_of(raw, cache.page_size, cache.head_dim, which)


def check_pages(cache, x, which, page_tokens):
    """page_tokens: {page: rows of x, from its offset 0}. Codes and scales equal coding each page at once."""
    c, s = codes(cache, which), (cache.k_scale if which == "k" else cache.v_scale).cpu().numpy()
    x = x.double().cpu().numpy()
    for page, rows in page_tokens.items():
        for h in range(cache.n_kv):
            want, ws = plain.quantize_page(x[rows, h])
            if want is None:
                assert np.isnan(s[page, h]), (which, page, h)
                continue
            assert s[page, h] == ws, (which, page, h, s[page, h], ws)
            assert np.array_equal(c[page, h, :len(rows)], want), (which, page, h)


def values(T, n_kv, D, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((2, T, n_kv, D), generator=g, device="cuda") * torch.exp2(torch.randint(-3, 6, (2, T, n_kv, 1), generator=g, device="cuda").float())
    x[:, T // 2, 0] = 0
    return x.to(DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("P,D,n_kv", [(16, 64, 1), (32, 128, 2), (64, 64, 3), (128, 128, 1)])
@pytest.mark.parametrize("group", ["all", "one", "odd"])
def test_the_cache_does_not_depend_on_how_tokens_are_grouped(dtype, P, D, n_kv, group):
    T = 2 * P + 5
    k, v = values(T, n_kv, D, dtype, P + D)
    pages = [3, 0, 4]
    cache = kq.KV8Cache(6, P, n_kv, D)
    cache.k.fill_(77)
    cache.v.fill_(-77)
    cache.k_scale.fill_(1e9)  # what another request left
    cache.v_scale.fill_(float("nan"))
    slot = np.array([pages[t // P] * P + t % P for t in range(T)], np.int32)
    sizes = {"all": [T], "one": [1] * T, "odd": [3, 1, 7, P - 2, 2, T]}[group]
    t = 0
    for n in sizes:
        n = min(n, T - t)
        if n:
            kq.kv8_append(cache, k[t:t + n], v[t:t + n], dev(slot[t:t + n]))
        t += n
    at = {pages[i]: list(range(i * P, min(T, (i + 1) * P))) for i in range(3)}
    check_pages(cache, k, "k", at)
    check_pages(cache, v, "v", at)
    assert (cache.k[[1, 2, 5]] == 77).all() and (cache.v_scale[[1, 2, 5]].isnan()).all()  # other pages untouched


def test_many_requests_in_one_call_with_skipped_tokens_and_strides():
    P, D, n_kv, B = 32, 128, 4, 40
    rng = np.random.default_rng(0)
    rows = torch.randn((200, 3 * n_kv * D), device="cuda")  # fused rows: k and v are views
    k, v = rows[:, n_kv * D:2 * n_kv * D].unflatten(1, (n_kv, D)), rows[:, 2 * n_kv * D:].unflatten(1, (n_kv, D))
    cache = kq.KV8Cache(100, P, n_kv, D)
    slot, at, t, free = np.full(200, -1, np.int32), {}, 0, list(rng.permutation(100))
    while t < 200 and free:
        n = min(int(rng.integers(1, 50)), 200 - t)
        for i in range(n):
            if i % P == 0:
                page = free.pop()
                at[page] = []
            slot[t + i] = page * P + i % P
            at[page].append(t + i)
        t += n + int(rng.integers(0, 3))  # tokens between requests are skipped
    kq.kv8_append(cache, k, v, dev(slot))
    check_pages(cache, k, "k", at)
    check_pages(cache, v, "v", at)


@pytest.mark.parametrize("P,D,n_kv,dtype", [(16, 64, 3, "f32"), (32, 128, 8, "bf16"), (64, 128, 2, "f32"), (128, 128, 4, "bf16")])
def test_prompts_and_tokens_of_several_requests(P, D, n_kv, dtype):
    """Calls of several thousand tokens, whose CTAs take many tokens each, over pages that hold tokens already."""
    rng = np.random.default_rng(P)
    lens, more = rng.integers(1, 700, 20), rng.integers(1, 300, 20)
    nb = -(-(lens + more) // P)
    k, v = values(int((lens + more).sum()), n_kv, D, dtype, P)
    cache, pages = kq.KV8Cache(int(nb.sum()) + 2, P, n_kv, D), rng.permutation(int(nb.sum()) + 2)
    first = np.concatenate([[0], np.cumsum(nb)])
    rows, at, t = [[], []], {}, 0
    for r in range(20):
        for i in range(lens[r] + more[r]):
            page = int(pages[first[r] + i // P])
            at.setdefault(page, []).append(t)
            rows[int(i >= lens[r])].append((t, page * P + i % P))
            t += 1
    for part in rows:
        sel = torch.tensor([a for a, _ in part], device="cuda")
        kq.kv8_append(cache, k[sel], v[sel], dev([b for _, b in part]))
    check_pages(cache, k, "k", at)
    check_pages(cache, v, "v", at)


def test_borders_tiny_and_zero_values():
    P, D = 16, 64
    x = torch.zeros((16, 1, D), device="cuda")
    rows = [0.0, 1.0, -1.0, 2.0, -2.0, 1.9999999, 0.5, -0.015625, 0.015625, 0.0156249, -1e-30, 1e-30, -1e-45, 1e-45, 127.0 / 64, -3e-39]
    for i, r in enumerate(rows):
        x[i, 0, i::7] = r
    for scale in (1.0, 2.0 ** -119, 2.0 ** -149, 2.0 ** 120, 0.0):
        y = (x.double() * scale).float()
        cache = kq.KV8Cache(1, P, 1, D)
        kq.kv8_append(cache, y, -y, dev(range(16)))
        check_pages(cache, y, "k", {0: list(range(16))})
        check_pages(cache, -y, "v", {0: list(range(16))})
        for t in range(16):  # and one token at a time
            kq.kv8_append(cache, y[t:t + 1], -y[t:t + 1], dev([t]))
        check_pages(cache, y, "k", {0: list(range(16))})
        check_pages(cache, -y, "v", {0: list(range(16))})


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_break_their_page_and_head_alone(bad):
    P, D = 32, 64
    k, v = values(3 * P, 2, D, "f32", 5)
    k[P + 3, 1, 17] = bad
    v[2 * P, 0, 0] = bad
    cache = kq.KV8Cache(3, P, 2, D)
    kq.kv8_append(cache, k, v, dev(range(3 * P)))
    at = {i: list(range(i * P, i * P + P)) for i in range(3)}
    check_pages(cache, k, "k", at)
    check_pages(cache, v, "v", at)
    kq.kv8_append(cache, k[:1], v[:1], dev([P + 5]))
    assert cache.k_scale[1, 1].isnan()  # stays broken
    kq.kv8_append(cache, k[:P], v[:P], dev(range(P, 2 * P)))
    check_pages(cache, k, "k", {1: list(range(P))})  # until it is begun again


def test_slots_beyond_the_cache_are_skipped_and_reported():
    P, D = 16, 64
    cache = kq.KV8Cache(2, P, 1, D)
    cache.k.fill_(5)
    cache.v.fill_(5)
    x = torch.ones((3, 1, D), device="cuda")
    assert kq.device_errors() == 0
    kq.kv8_append(cache, x, x, dev([32, -1, 2 ** 31 - 1]))
    assert kq.device_errors() == 2 and (cache.k == 5).all() and (cache.v == 5).all() and (cache.k_scale == 0).all()


# ---------------------------------------------------------------- attention

def make(lens, P, D, n_q, n_kv, x, seed, spread=2, spare=2):
    """A filled cache with scattered pages, and q: (cache, codes, table, ctx, new, q)."""
    rng = np.random.default_rng(seed)
    ctx, new = np.array([c for c, _ in lens], np.int64), np.array([n for _, n in lens], np.int64)
    nb = -(-(ctx + new) // P)
    pages = int(nb.sum()) + spare
    perm = rng.permutation(pages)
    table = np.zeros((len(lens), max(1, int(nb.max()))), np.int32)
    at = 0
    for r, n in enumerate(nb):
        table[r, :n] = perm[at:at + n]
        at += n
    kc, vc = (np.clip(np.floor(rng.standard_normal((pages, n_kv, P, D)) * 40), -128, 127).astype(np.int8) for _ in range(2))
    ks, vs = (np.exp2(rng.integers(-5 - spread, -4, (pages, n_kv))).astype(np.float32) for _ in range(2))
    cache = kq.KV8Cache(pages, P, n_kv, D, k=dev(plain.stored(kc, P, D, "k"), np.int8), v=dev(plain.stored(vc, P, D, "v"), np.int8),
                        k_scale=dev(ks, np.float32), v_scale=dev(vs, np.float32))
    q = torch.tensor(rng.standard_normal((int(new.sum()), n_q, D)), device="cuda").to(DT[x])
    return cache, (kc, ks, vc, vs), table, ctx, new, q


def run(cache, table, ctx, new, q, y, mask=None, scale=None, **kw):
    o = kq.attention_kv8(q, cache, dev(table), dev(ctx), dev(new), int(max(new)), int(max(ctx + new)), scale=scale,
                         mask=None if mask is None else dev(np.asarray(mask, np.uint32).view(np.int32)), out_dtype=DT[y], **kw)
    torch.cuda.synchronize()
    return o


def check(o, q, parts, table, ctx, new, P, n_kv, scale, mask=None):
    ref, base, mag = plain.attention(q.double().cpu().numpy(), *parts, table, ctx, new, P, n_kv, scale, mask)
    if o.dtype == torch.float32:
        tol = base * (2 * mag * 2.0 ** -17 + 2.0 ** -19) + np.abs(ref) * 2.0 ** -23
    else:
        dq = 2.0 ** -12 if q.dtype == torch.float32 else 0.0
        tol = base * (2 * mag * (dq + 2.0 ** -17) + 2.0 ** -11) + np.abs(ref) * 2.0 ** -8
    err = np.abs(o.double().cpu().numpy() - ref)
    assert np.isfinite(err).all() and (err <= tol).all(), (err / np.maximum(tol, 1e-30)).max()


def attn_case(lens, P, D, n_q, n_kv, x, y, seed=0):
    cache, parts, table, ctx, new, q = make(lens, P, D, n_q, n_kv, x, seed)
    o = run(cache, table, ctx, new, q, y)
    check(o, q, parts, table, ctx, new, P, n_kv, D ** -0.5)


# one token and no context; page, group, tile and segment borders and their neighbours; empty requests among others
BORDERS = [(0, 1), (14, 1), (15, 1), (16, 1), (0, 0), (62, 1), (63, 1), (64, 1), (100, 0), (127, 1), (255, 1), (256, 1), (300, 1), (511, 1), (515, 1)]


@pytest.mark.parametrize("x,y", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("P,D", [(16, 64), (16, 128), (32, 128), (64, 64), (128, 128)])
def test_single_tokens(x, y, P, D):
    attn_case(BORDERS, P, D, 8, 2, x, y, seed=P + D)


@pytest.mark.parametrize("n_q,n_kv", [(1, 1), (5, 1), (12, 2), (16, 2), (40, 1), (64, 1)])
@pytest.mark.parametrize("y", ["bf16", "f32"])
def test_head_groups(n_q, n_kv, y):
    attn_case([(33, 1), (290, 1)], 32, 64, n_q, n_kv, "bf16", y)


@pytest.mark.parametrize("x,y", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("P,D,n_q,n_kv", [(16, 128, 8, 2), (64, 64, 4, 4), (32, 64, 20, 4)])
def test_windows_and_prompts(x, y, P, D, n_q, n_kv):
    attn_case([(0, 2), (254, 5), (700, 32), (3, 17), (0, 33), (250, 70), (0, 300), (61, 0), (400, 31)], P, D, n_q, n_kv, x, y)


def test_a_context_of_more_than_128_tiles():
    attn_case([(33100, 1), (32767, 1), (70, 1)], 128, 64, 2, 1, "bf16", "f32")


@pytest.mark.parametrize("x,y", [("bf16", "bf16"), ("f32", "f32")])
def test_windows_of_more_than_32_tokens_over_long_contexts(x, y):
    """Cut along the context too where their blocks of rows are few; next to requests that are cut otherwise."""
    attn_case([(5000, 33), (4055, 40), (4056, 40), (9000, 64), (6000, 1), (4500, 300), (7, 35)], 32, 64, 4, 2, x, y)
    attn_case([(12000, 50), (3, 3)], 16, 128, 1, 1, x, y)


@pytest.mark.parametrize("B", [1000, 4096])
def test_many_requests(B):
    rng = np.random.default_rng(B)
    attn_case([(int(c), int(n)) for c, n in zip(rng.integers(0, 60, B), rng.integers(0, 3, B))], 16, 64, 4, 1, "bf16", "f32")


@pytest.mark.parametrize("y", ["bf16", "f32"])
def test_tree_masks_and_rows_that_see_nothing(y):
    P, D, n_q, n_kv = 16, 64, 4, 2
    cache, parts, table, ctx, new, q = make([(0, 4), (100, 32), (250, 12), (0, 1), (40, 1)], P, D, n_q, n_kv, "f32", 3)
    rng = np.random.default_rng(1)
    mask = rng.integers(0, 1 << 32, int(new.sum()), dtype=np.uint64).astype(np.uint32)
    mask[0] = 0           # nothing at all
    mask[1] = 1 << 31     # bits past the window are no tokens
    mask[48] = 0          # nothing, alone in its request
    mask[49] = 0          # its context alone
    o = run(cache, table, ctx, new, q, y, mask=mask)
    assert (o[0] == 0).all() and (o[1] == 0).all() and (o[48] == 0).all()
    m = mask.copy()
    t = 0
    for n in new:  # the 64-bit form reads the window's bits alone
        m[t:t + n] &= np.uint32((1 << int(n)) - 1)
        t += n
    check(o, q, parts, table, ctx, new, P, n_kv, D ** -0.5, m)


def test_strided_rows_and_padding_rows():
    P, D, n_q, n_kv = 32, 128, 4, 2
    cache, parts, table, ctx, new, q = make([(20, 2), (300, 3)], P, D, n_q, n_kv, "bf16", 4)
    rows = torch.zeros((8, (n_q + 3) * D), dtype=torch.bfloat16, device="cuda")
    rows[:5, D:D + n_q * D] = q.flatten(1)
    out = torch.full((8, 2 * n_q * D), 7.0, device="cuda")
    view = out[:, n_q * D:].unflatten(1, (n_q, D))
    run(cache, table, ctx, new, rows[:, D:D + n_q * D].unflatten(1, (n_q, D)), "f32", out=view)
    check(view[:5], q, parts, table, ctx, new, P, n_kv, D ** -0.5)
    assert (view[5:] == 7).all() and (out[:, :n_q * D] == 7).all()


def test_scales_and_queries_of_any_size():
    """Pages whose scales differ by 2^40 and query rows from 1e-20 to 1e20, scores of +-30 and single spikes."""
    P, D, n_q, n_kv = 16, 64, 2, 1
    cache, parts, table, ctx, new, q = make([(200, 1), (90, 2)], P, D, n_q, n_kv, "f32", 5)
    kc, ks, vc, vs = parts
    vs[:] = np.exp2(np.random.default_rng(2).integers(-20, 21, vs.shape))
    cache.v_scale.copy_(torch.tensor(vs))
    big = torch.tensor([1e20, 1e-20, 3e10], device="cuda")[:, None, None]
    for y in ("f32", "bf16"):
        qq = q * big
        scales = (4e-20, 5e19, 1e-10)
        for i, s in enumerate(scales):
            o = run(cache, table, ctx, new, qq, y, scale=s)
            ref = slice(i, i + 1)
            full = plain.attention(qq.double().cpu().numpy(), *parts, table, ctx, new, P, n_kv, s)
            r, base, mag = (a[ref] for a in full)
            tol = base * (2 * mag * (2.0 ** -17 if y == "f32" else 2.0 ** -12 + 2.0 ** -17) + 2.0 ** (-19 if y == "f32" else -11))
            tol += np.abs(r) * 2.0 ** (-23 if y == "f32" else -8)
            assert (np.abs(o[ref].double().cpu().numpy() - r) <= tol).all(), (y, i)


def test_a_broken_page_reaches_the_rows_that_see_it_alone():
    P, D, n_q, n_kv = 16, 64, 4, 2
    for key in ("k_scale", "v_scale"):
        cache, parts, table, ctx, new, q = make([(30, 10), (50, 1), (300, 2)], P, D, n_q, n_kv, "bf16", 6)
        clean = run(cache, table, ctx, new, q, "f32")
        getattr(cache, key)[int(table[0, 2]), 1] = float("nan")  # positions 32.. of request 0, kv head 1
        o = run(cache, table, ctx, new, q, "f32")
        hit = torch.zeros(o.shape, dtype=torch.bool, device="cuda")
        hit[2:10, 2:] = True
        assert o[hit].isnan().all() and torch.equal(o[~hit], clean[~hit]), key


def test_non_finite_queries_reach_their_own_rows_alone():
    P, D, n_q, n_kv = 16, 64, 4, 2
    cache, parts, table, ctx, new, q = make([(30, 3), (300, 1)], P, D, n_q, n_kv, "f32", 7)
    clean = run(cache, table, ctx, new, q, "f32")
    q = q.clone()
    q[1, 2, 5] = float("nan")
    q[3, 0, 0] = float("inf")
    o = run(cache, table, ctx, new, q, "f32")
    hit = torch.zeros(o.shape, dtype=torch.bool, device="cuda")
    hit[1, 2] = hit[3, 0] = True
    assert not o[hit].isfinite().any() and torch.equal(o[~hit], clean[~hit])


def test_page_ids_and_lengths_out_of_bounds_are_reported():
    P, D, n_q, n_kv = 16, 64, 2, 1
    cache, parts, table, ctx, new, q = make([(40, 1), (70, 1), (300, 1)], P, D, n_q, n_kv, "bf16", 8)
    clean = run(cache, table, ctx, new, q, "f32")
    assert kq.device_errors() == 0
    for bad in (-1, cache.n_pages, 2 ** 31 - 1):
        t = table.copy()
        t[1, 2] = bad
        o = run(cache, t, ctx, new, q, "f32")
        assert kq.device_errors() == 2 and o[1].isnan().all() and torch.equal(o[[0, 2]], clean[[0, 2]])
    for c, n in ((-1, 1), (40, -1), (10 ** 6, 1), (2 ** 31 - 1, 1), (40, 2 ** 31 - 1), (40, 2)):
        cc, nn = ctx.copy(), new.copy()
        cc[0], nn[0] = c, n
        out = torch.full_like(clean, 3.0)
        kq.attention_kv8(q, cache, dev(table), dev(cc), dev(nn), 1, 301, total_len=1000, out=out)
        assert kq.device_errors() == 2, (c, n)
    out = torch.full_like(clean, 3.0)  # more tokens than rows: nothing is done
    kq.attention_kv8(q[:2], cache, dev(table), dev(ctx), dev(new), 1, 301, out=out[:2])
    assert kq.device_errors() == 2 and (out == 3).all()
    out = torch.full_like(clean, 3.0)  # a total below the truth: the request that finds no room is left out
    kq.attention_kv8(q, cache, dev(table), dev(ctx), dev(np.array([1, 1, 1])), 1, 301, total_len=0, out=out)
    assert kq.device_errors() in (0, 2) and torch.equal(out[:2], clean[:2])


def test_a_row_does_not_depend_on_the_batch_or_on_the_window():
    P, D, n_q, n_kv = 32, 128, 8, 2
    lens = [(500, 6), (9, 1), (1000, 32), (0, 3), (2000, 1)]
    cache, parts, table, ctx, new, q = make(lens, P, D, n_q, n_kv, "bf16", 9)
    for y in ("f32", "bf16"):
        o = run(cache, table, ctx, new, q, y)
        t = 0
        for r, n in enumerate(new):
            for m in {1, min(int(n), 2), min(int(n), 4), int(n)}:  # the request alone, with a window of its first m tokens
                a = run(cache, table[r:r + 1], ctx[r:r + 1], np.array([m]), q[t:t + m], y)
                assert torch.equal(a, o[t:t + m]), (r, m)
            t += n


def test_other_stream_capture_and_replay_with_other_lengths():
    P, D, n_q, n_kv = 16, 64, 4, 2
    cache, parts, table, ctx, new, q = make([(600, 1), (50, 1)], P, D, n_q, n_kv, "bf16", 10)
    td, cd, nd = dev(table), dev(ctx), dev(new)
    out = torch.empty((2, n_q, D), device="cuda")
    ws = torch.empty(kq.attention_kv8_workspace_size(2, 1300, 1, n_q, n_kv, D), dtype=torch.uint8, device="cuda")
    call = lambda: kq.attention_kv8(q, cache, td, cd, nd, 1, 620, total_len=1300, out=out, workspace=ws)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    check(out, q, parts, table, ctx, new, P, n_kv, D ** -0.5)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for c in ([5, 49], [600, 0], [256, 255], [255, 17]):
        cd.copy_(dev(c))
        out.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        check(out, q, parts, table, np.array(c), new, P, n_kv, D ** -0.5)


def test_offsets_beyond_32_bits():
    """Pages whose code offsets pass 2^32 bytes: 2^31 slots' worth of one head at D = 128 would take 256 GB, so a
    cache of 40 million tokens (5 GB of k and of v) with its pages at the end."""
    P, D, n_q, n_kv = 128, 128, 4, 1
    n_pages = 40_000_000 // P
    k, v = (torch.empty((n_pages, n_kv, P * D), dtype=torch.int8, device="cuda") for _ in range(2))
    cache = kq.KV8Cache(n_pages, P, n_kv, D, k=k, v=v)
    x = torch.randn((2, 300, n_kv, D), device="cuda").to(torch.bfloat16)
    pages = np.array([[n_pages - 1, n_pages - 200, n_pages - 3]], np.int32)
    slot = (pages[0, np.arange(300) // P].astype(np.int64) * P + np.arange(300) % P).astype(np.int32)
    kq.kv8_append(cache, x[0], x[1], dev(slot))
    for t, which in ((k, "k"), (v, "v")):
        got = plain.codes_of(t[pages[0].astype(np.int64)].cpu().numpy(), P, D, which)
        src = x[0 if which == "k" else 1].double().cpu().numpy()
        for i in range(3):
            rows = src[i * P:min(300, (i + 1) * P), 0]
            assert np.array_equal(got[i, 0, :len(rows)], plain.quantize_page(rows)[0])
    q = torch.randn((1, n_q, D), device="cuda")
    o = run(cache, pages, np.array([299]), np.array([1]), q, "f32")
    sub = pages[0].astype(np.int64)
    parts = (plain.codes_of(k[sub].cpu().numpy(), P, D, "k"), cache.k_scale[sub].cpu().numpy(),
             plain.codes_of(v[sub].cpu().numpy(), P, D, "v"), cache.v_scale[sub].cpu().numpy())
    check(o, q, parts, np.array([[0, 1, 2]]), np.array([299]), np.array([1]), P, n_kv, D ** -0.5)


@pytest.mark.parametrize("handle", [False, True])
def test_memory_of_calls_on_a_given_stream(handle, monkeypatch):
    """What a call allocates itself comes from its stream's pool: what the current stream asks for next is elsewhere."""
    P, D, n_q, n_kv = 16, 64, 4, 2
    cache, parts, table, ctx, new, q = make([(1300, 1), (50, 1)], P, D, n_q, n_kv, "bf16", 12)
    td, cd, nd = dev(table), dev(ctx), dev(new)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    real, seen = kq.lib(), []

    class Spy:
        def __getattr__(self, name):
            def call(*args):
                if name == "kq_attention_kv8":
                    seen.append((args[5], args[-3]))  # o, workspace
                return getattr(real, name)(*args)
            return call

    monkeypatch.setattr(kq, "lib", Spy)
    stream = s.cuda_stream if handle else s
    o = kq.attention_kv8(q, cache, td, cd, nd, 1, 1400, total_len=1400, out_dtype=torch.float32, stream=stream)
    need = kq.attention_kv8_workspace_size(2, 1400, 1, n_q, n_kv, D)
    other = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    assert seen[0][0] == o.data_ptr() and seen[0][1] != other.data_ptr()
    table2, free, n_free, pos, freq = td.clone(), dev([1, 2, 3]), dev([3]), dev([0, 0]), torch.ones(8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    plan = kq.pages_plan(cd, nd, table2, free, n_free, P, 2, stream=stream)
    turned, _ = kq.rope(q, None, pos, freq, stream=stream)
    s.synchronize()
    check(o, q, parts, table, ctx, new, P, n_kv, D ** -0.5)
    assert plan.pos.tolist() == [1300, 50] and plan.status.item() == 0
    assert torch.equal(turned, q)


@pytest.mark.parametrize("x,y", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("D", [64, 128])
def test_few_heads_are_cut_finer(x, y, D):
    """Segments of 256 positions up to 16384, twice as long beyond; more than 64 segments for windows of over 32 tokens."""
    attn_case([(255, 1), (256, 1), (511, 2), (513, 5), (16383, 1), (16384, 2), (16640, 20)], 16, D, 4, 2, x, y)
    attn_case([(40000, 40), (5, 2), (4063, 33), (4062, 33), (9000, 100)], 128, D, 2, 1, x, y)


def test_segments_of_a_prompt_end_inside_pages_and_windows_of_page_ids():
    """Lengths whose shares are odd multiples of 128 positions."""
    attn_case([(4100, 33), (6700, 47), (7300, 64), (11111, 130)], 64, 64, 6, 3, "bf16", "f32")
    attn_case([(5003, 60), (8200, 35)], 32, 128, 24, 12, "bf16", "bf16")


@pytest.mark.parametrize("n_q,n_kv,D", [(4, 1, 64), (8, 2, 128), (3, 3, 64)])
def test_windows_over_every_cut_give_the_bits_of_single_tokens(n_q, n_kv, D):
    """Windows whose tokens stand before and after the positions where segments, their size or the warps that join
    them change."""
    P, n = 16, 4
    ends = [256, 512, 1024, 2048, 4096, 8192, 16384, 32768, 65536]
    lens = [(e - 2, n) for e in ends]
    cache, parts, table, ctx, new, q = make(lens, P, D, n_q, n_kv, "f32", 21)
    for y in ("f32", "bf16"):
        o = run(cache, table, ctx, new, q, y)
        for i in range(n):
            a = run(cache, table, ctx + i, np.ones_like(new), q.view(len(ends), n, n_q, D)[:, i].contiguous(), y)
            same = (a == o.view(len(ends), n, n_q, D)[:, i]).flatten(1).all(1)
            assert same.all(), (i, [e for e, s in zip(ends, same.tolist()) if not s])
