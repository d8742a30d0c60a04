"""Rows of one call that go to one page with skipped rows between them, or with slots left out: codes and scales equal coding
the page's values at once, whichever row raises the scale."""
import numpy as np
import pytest
import torch

import kv8_plain as plain
import quantized_decode_gemv_block_gb300 as kq
from test_gpu_kv8 import DT, codes, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    yield
    assert kq.device_errors() == 0


def values(T, n_kv, D, dtype, seed):
    """Values whose size changes from row to row, up and down by up to 2^9."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((2, T, n_kv, D), generator=g, device="cuda") * torch.exp2(torch.randint(-4, 6, (2, T, n_kv, 1), generator=g, device="cuda").float())
    return x.to(DT[dtype])


def check(cache, k, v, held):
    """held: {page: {offset: (call's k and v, row)}}."""
    for which, scale in (("k", cache.k_scale.cpu().numpy()), ("v", cache.v_scale.cpu().numpy())):
        c = codes(cache, which)
        x = [t.double().cpu().numpy() for t in (k if which == "k" else v)]
        for page, slots in held.items():
            at = sorted(slots)
            for h in range(cache.n_kv):
                want, ws = plain.quantize_page(np.stack([x[slots[o][0]][slots[o][1], h] for o in at]))
                assert scale[page, h] == ws, (which, page, h)
                assert np.array_equal(c[page, h, at], want), (which, page, h)


def run(P, D, n_kv, dtype, calls, n_pages=7):
    """calls: lists of slots, run in turn from an empty cache, three times."""
    ks, vs = zip(*(values(len(s), n_kv, D, dtype, 7 * i + P) for i, s in enumerate(calls)))
    held = {}
    for i, slots in enumerate(calls):
        rows = [(row, s) for row, s in enumerate(slots) if 0 <= s < n_pages * P]
        held.update({s // P: {} for _, s in rows if s % P == 0})  # begun afresh
        for row, s in rows:
            held[s // P][s % P] = (i, row)
    for _ in range(3):
        cache = kq.KV8Cache(n_pages, P, n_kv, D)
        cache.k.fill_(99)
        cache.v.fill_(-99)
        cache.k_scale.fill_(float("nan"))
        cache.v_scale.fill_(3e4)
        for k, v, s in zip(ks, vs, calls):
            kq.kv8_append(cache, k, v, dev(s))
        check(cache, ks, vs, held)


S = -1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("P,D,n_kv", [(16, 64, 1), (16, 64, 9), (32, 128, 2), (64, 128, 1), (128, 64, 3), (128, 128, 2)])
def test_skipped_rows_and_left_out_slots_in_a_page(dtype, P, D, n_kv):
    base = 2 * P
    begun = [base, base + 1, base + 2]
    for later in ([base + 3, S, base + 5], [base + 3, base + 5], [S, base + 3, S, S, base + 4, S], [base + 4, S, base + P - 1],
                  [base + 3] + [S] * 40 + [base + 6], [S, S, base + 3, base + 4, base + 5, S, base + 6, base + 9, base + 10],
                  [base + o for o in range(3, P, 2)], [base + 4, S, 0, S, 1, 5, S, S, 7],
                  [base + 3] + [S] * 700 + [base + 5] + [S] * 3000 + [base + 6, S, 3 * P, S, 3 * P + 2]):
        run(P, D, n_kv, dtype, [begun, later])
    # pages that begin in the call
    run(P, D, n_kv, dtype, [[0, S, 1, 3, S, S, 6, P, S, P + 1]])
    run(P, D, n_kv, dtype, [[S] * 5 + [x for o in range(P) for x in (o, S)] + [x for o in range(P) for x in (3 * P + o, S, S)]])


@pytest.mark.parametrize("P,D,n_kv,dtype", [(16, 64, 8, "bf16"), (16, 64, 8, "f32"), (64, 128, 8, "bf16"), (128, 128, 2, "bf16"), (128, 128, 2, "f32")])
def test_many_pages_whose_rows_are_scattered(P, D, n_kv, dtype):
    """Calls whose CTAs take many rows each; every second page has skipped rows and left-out slots, some of them past what a CTA
    loads at first."""
    rng = np.random.default_rng(P)
    n_pages, first, second = 24000 // P, [], []
    for page in rng.permutation(n_pages):
        begun = int(rng.integers(0, P // 2))
        first += [int(page) * P + o for o in range(begun)]
        offs = range(begun, P) if page % 2 else sorted(rng.choice(np.arange(begun, P), int(rng.integers(1, P - begun + 1)), replace=False))
        if not begun:
            offs = sorted({0, *offs})
        for o in offs:
            if page % 2 == 0 and rng.random() < 0.1:
                second += [S] * int(rng.choice([1, 2, 30, 200]))
            second.append(int(page) * P + int(o))
    run(P, D, n_kv, dtype, [first, second], n_pages)


def test_slots_beyond_the_cache_between_the_rows_of_a_page():
    P, n = 16, 7
    for bad in ([n * P], [2 ** 31 - 1, S], [S, n * P + 3]):
        run(P, 64, 2, "f32", [[0, 1], [2, *bad, 4, *bad, *bad, 5]], n)
        assert kq.device_errors() == 2


@pytest.mark.parametrize("P,D,rows", [(16, 64, [9, 5, 7, S, 6, 9, 5]), (32, 128, [40, 39, 38, S, 33, S, 34]), (16, 64, [5, S, 4, 0, 1, S, 3])])
def test_rows_that_are_not_in_order(P, D, rows):
    """Outside what the call promises, yet of one page and behind one another: as if appended one by one."""
    n_kv, begun = 2, [0, 1, 2, 3, P, P + 1]
    k, v = values(len(rows), n_kv, D, "f32", 3)
    k0, v0 = values(len(begun), n_kv, D, "f32", 4)
    got, want = (kq.KV8Cache(3, P, n_kv, D) for _ in range(2))
    for c in (got, want):
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            t.zero_()
        kq.kv8_append(c, k0, v0, dev(begun))
    kq.kv8_append(got, k, v, dev(rows))
    for i, s in enumerate(rows):
        kq.kv8_append(want, k[i:i + 1], v[i:i + 1], dev([s]))
    for a, b in ((got.k, want.k), (got.v, want.v), (got.k_scale, want.k_scale), (got.v_scale, want.v_scale)):
        assert torch.equal(a, b)
