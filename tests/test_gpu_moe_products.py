"""The experts' products (kq_moe_gate_up, kq_moe_down) against 64-bit forms on the oracle's weights.

Tolerance of a product: the library's contract, d = 1e-4 sum_k |w_k x_k|. act = silu(g) u: |silu'| <= 1.1, so
1.1 d_g |u| + (|silu(g)| + 1.1 d_g) d_u, expf, the division and the products 8 units of 2^-24, and the rounding to bf16 (8 significant
bits: neighbours of 1 are 2^-7 apart, so at most 2^-8 of the value). y: the
weights' sum of the products' d, one rounding per choice and one for add, and the rounding to y's type.
"""
import numpy as np
import pytest
import torch

import quantized_decode_gemv_block_gb300 as kq
from moe_plain import bf16, dev, experts, product

pytestmark = pytest.mark.gpu
TOL, U = 1e-4, 2.0 ** -24
FORMATS = ["q4_k", "q8_0", "q5_k", "q6_k", "affine4"]


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    import oracle
    oracle.build()
    assert torch.cuda.is_available()
    yield
    assert kq.device_errors() == 0


def some_ids(T, k, E, seed=0, none=0.0, twice=False):
    rng = np.random.default_rng(seed + T + E)
    ids = np.stack([rng.integers(0, E, k) if twice else rng.permutation(E)[:k] for _ in range(T)]) if T else np.zeros((0, k))
    ids = ids.astype(np.int32)
    ids[rng.random((T, k)) < none] = -1
    return ids


def gate_up(fmt, w, wp, x, ids, F, **kw):
    T, k = ids.shape
    E, K = wp.shape[0], wp.shape[2]
    plan = kq.moe_plan(dev(ids), E)
    act = kw.pop("act", None)
    if act is None:
        act = torch.full((T * k, F), 77.0, dtype=torch.bfloat16, device="cuda")
    out = kq.moe_gate_up(fmt, w, x, plan, F, K, act=act, **kw)
    e = ids.reshape(-1)
    y, b = product(wp, x.repeat_interleave(k, 0), e)
    g, u, dg, du = y[:, :F], y[:, F:], TOL * b[:, :F], TOL * b[:, F:]
    with np.errstate(over="ignore"):
        silu = g / (1 + np.exp(-g))
    ref = silu * u
    tol = 1.1 * dg * np.abs(u) + (np.abs(silu) + 1.1 * dg) * du + 8 * U * np.abs(ref)
    tol += (np.abs(ref) + tol) * 2.0 ** -8 + 2.0 ** -126
    got = out.double().cpu().numpy()
    assert (np.abs(got - ref) <= tol)[e >= 0].all(), (np.abs(got - ref) - tol)[e >= 0].max()
    assert (got[e < 0] == 77.0).all()  # left as they were
    return out


def down(fmt, w, wp, act, ids, weights, H, add=None, dtype=torch.float32, **kw):
    T, k = ids.shape
    E, K = wp.shape[0], wp.shape[2]
    plan = kq.moe_plan(dev(ids), E)
    a0 = None if add is None else add.double().cpu().numpy()
    out = kq.moe_down(fmt, w, act, plan, dev(ids), weights, H, K, add=add, out_dtype=dtype, **kw)
    e = ids.reshape(-1)
    y, b = product(wp, act, e)
    c = np.abs(weights.double().cpu().numpy())
    y, b = y.reshape(T, k, H), b.reshape(T, k, H)
    ref = (y * weights.double().cpu().numpy()[..., None]).sum(1)
    size = (np.abs(y) * c[..., None]).sum(1)
    if add is not None:
        ref, size = ref + a0, size + np.abs(a0)
    tol = TOL * (b * c[..., None]).sum(1) + (k + 1) * U * size + np.abs(ref) * torch.finfo(dtype).eps / 2 + 2.0 ** -126
    got = out.double().cpu().numpy()
    assert (np.abs(got - ref) <= tol).all(), (np.abs(got - ref) - tol).max()
    return out


def some_weights(T, k, seed=0):
    return torch.rand((T, k), generator=torch.Generator(device="cuda").manual_seed(seed + T), device="cuda")


def both(fmt, T, k, E, H, F, none=0.0, twice=False, seed=0):
    ids = some_ids(T, k, E, seed, none, twice)
    w1, p1 = experts(fmt, E, 2 * F, H, seed)
    act = gate_up(fmt, w1, p1, bf16(T, H, seed=seed), ids, F)
    w2, p2 = experts(fmt, E, H, F, seed + 1)
    act = torch.where(torch.tensor(ids.reshape(-1) < 0, device="cuda")[:, None], float("nan"), act)  # read by nobody
    down(fmt, w2, p2, act, ids, some_weights(T, k), H)
    return ids


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 40])
def test_formats_and_token_counts(fmt, T):
    both(fmt, T, 2, 4, 512, 256)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("K", [256, 768, 2304, 2560, 2816, 5120, 5376, 10496])
def test_lengths(fmt, K):
    """One, several and too many units for one CTA: two, four and eight CTAs share K."""
    E, T, k, N = 2, 5, 1, 40
    ids = some_ids(T, k, E)
    w, p = experts(fmt, E, 2 * N, K)
    gate_up(fmt, w, p, bf16(T, K), ids, N)
    w, p = experts(fmt, E, N, K)
    down(fmt, w, p, bf16(T * k, K), ids, some_weights(T, k), N)


@pytest.mark.parametrize("fmt", FORMATS)
def test_the_longest_rows(fmt):
    E, T, k, N, K = 1, 17, 1, 24, 20480
    ids = some_ids(T, k, E)
    w, p = experts(fmt, E, 2 * N, K)
    gate_up(fmt, w, p, bf16(T, K), ids, N)


@pytest.mark.parametrize("T,k", [(1, 32), (40, 3)])
def test_the_most_experts(T, k):
    E, N, K = 1024, 8, 256
    ids = some_ids(T, k, E)
    w, p = experts("q4_k", E, 2 * N, K)
    gate_up("q4_k", w, p, bf16(T, K), ids, N)


@pytest.mark.parametrize("fmt", ["q4_k", "q6_k", "affine4"])
@pytest.mark.parametrize("N", [8, 24, 56, 136])
def test_rows_that_end_inside_a_tile(fmt, N):
    E, T, k, K = 8, 6, 3, 512
    ids = some_ids(T, k, E)
    w, p = experts(fmt, E, 2 * N, K)
    gate_up(fmt, w, p, bf16(T, K), ids, N)
    w, p = experts(fmt, E, N, K)
    down(fmt, w, p, bf16(T * k, K), ids, some_weights(T, k), N)


@pytest.mark.parametrize("N", [1, 3, 7, 17, 33])
def test_odd_rows(N):
    E, T, k, K = 3, 5, 2, 256
    ids = some_ids(T, k, E)
    w, p = experts("q4_k", E, 2 * N, K)
    gate_up("q4_k", w, p, bf16(T, K), ids, N)
    w, p = experts("q4_k", E, N, K)
    down("q4_k", w, p, bf16(T * k, K), ids, some_weights(T, k), N)


@pytest.mark.parametrize("kw", [dict(E=1, k=1), dict(E=60, k=4), dict(E=16, k=16), dict(E=8, k=2, none=0.3), dict(E=8, k=2, none=1.0),
                                dict(E=5, k=4, twice=True), dict(E=1, k=6, twice=True)])
def test_shares_of_experts(kw):
    both("q4_k", 21, H=256, F=256, **kw)


def test_one_expert_takes_all_and_others_none():
    T, E, K, N = 90, 30, 512, 64
    ids = np.full((T, 1), 11, np.int32)
    w, p = experts("q4_k", E, 2 * N, K)
    gate_up("q4_k", w, p, bf16(T, K), ids, N)


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_pair_has_the_bits_it_has_alone(fmt):
    """In windows of up to 32 tokens of an expert, whatever the others are."""
    T, k, E, H, F = 30, 2, 4, 768, 256
    ids = some_ids(T, k, E)
    w1, p1 = experts(fmt, E, 2 * F, H)
    w2, p2 = experts(fmt, E, H, F, 1)
    x, weights = bf16(T, H), some_weights(T, k)
    act = gate_up(fmt, w1, p1, x, ids, F)
    y = down(fmt, w2, p2, act, ids, weights, H)
    for t in (0, 13, 29):
        a = gate_up(fmt, w1, p1, x[t:t + 1], ids[t:t + 1], F)
        assert torch.equal(a, act[t * k:(t + 1) * k])
        assert torch.equal(down(fmt, w2, p2, a, ids[t:t + 1], weights[t:t + 1], H)[0], y[t])
    one = some_ids(T, k, E, seed=9)
    one[4] = ids[4]
    assert torch.equal(gate_up(fmt, w1, p1, x, one, F)[8:10], act[8:10])


def many_ids(counts, seed=0):
    """Ids of one choice per token: counts[e] tokens for expert e, in a random order."""
    ids = np.concatenate([np.full(n, e, np.int32) for e, n in enumerate(counts)])
    return np.random.default_rng(seed).permutation(ids)[:, None].copy()


@pytest.mark.parametrize("counts", [(33,), (64,), (65,), (255,), (256,), (257,), (513, 1), (40, 0, 31, 300, 32, 33, 0), (100, 150, 200, 250),
                                    (700, 3, 3, 3), (48,) * 16])
@pytest.mark.parametrize("K", [256, 768, 1280])
def test_many_rows_of_an_expert(counts, K):
    """Q4_K calls of many rows per expert (KQ_MOE_TC_ROWS on average) run on the tensor cores, experts of few rows or none among them."""
    E, F, H = len(counts), 128, 256
    ids = many_ids(counts)
    w, p = experts("q4_k", E, 2 * F, K)
    gate_up("q4_k", w, p, bf16(len(ids), K), ids, F)
    w, p = experts("q4_k", E, H, K)
    down("q4_k", w, p, bf16(len(ids), K), ids, some_weights(len(ids), 1), H)


@pytest.mark.parametrize("N", [1, 8, 40, 63, 64, 65, 127, 128, 129, 200, 320])
def test_many_rows_of_odd_matrices(N):
    E, K = 3, 512
    ids = many_ids((70, 90, 130))
    w, p = experts("q4_k", E, 2 * N, K)
    gate_up("q4_k", w, p, bf16(len(ids), K), ids, N)
    w, p = experts("q4_k", E, N, K)
    down("q4_k", w, p, bf16(len(ids), K), ids, some_weights(len(ids), 1), N)


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_rows_several_choices_and_empty_slots(fmt):
    ids = both(fmt, 150, 3, 8, 512, 256, none=0.1)
    assert (ids < 0).any()


def test_many_rows_keep_a_pairs_bits():
    """A row's bits on the tensor cores, whatever rows stand before, behind and beside it in its expert's tiles."""
    E, F, H, K = 3, 128, 256, 768
    w1, p1 = experts("q4_k", E, 2 * F, K)
    w2, p2 = experts("q4_k", E, H, K, 1)
    x = bf16(700, K)
    outs = []
    for order in (np.arange(700), np.random.default_rng(2).permutation(700), np.arange(150)):
        ids = (np.arange(700) * 7 % 13 % E).astype(np.int32)[order][:, None].copy()
        rows = x[torch.tensor(order, device="cuda")].contiguous()
        a = gate_up("q4_k", w1, p1, rows, ids, F)
        y = down("q4_k", w2, p2, rows, ids, torch.ones((len(order), 1), device="cuda"), H)
        back = torch.tensor(np.argsort(order), device="cuda")
        outs.append((a[back], y[back]))
    for a, y in outs[1:]:
        n = len(a)
        assert torch.equal(a, outs[0][0][:n]) and torch.equal(y, outs[0][1][:n])


def test_many_rows_of_the_most_experts():
    E, N, K, T, k = 1024, 8, 256, 5700, 8
    ids = some_ids(T, k, E)
    assert T * k >= 44 * E
    w, p = experts("q4_k", E, 2 * N, K)
    gate_up("q4_k", w, p, bf16(T, K), ids, N)


def test_a_long_run_of_tiles():
    """More tiles than the tensor-core product works out ahead (64 per pair of SMs): the same rows again and again, against few of them."""
    F, K, n, T = 256, 256, 97, 700_000
    w, p = experts("q4_k", 1, 2 * F, K)
    x = bf16(n, K)
    few = gate_up("q4_k", w, p, x, np.zeros((n, 1), np.int32), F)
    rows = torch.arange(T, device="cuda") % n
    out = kq.moe_gate_up("q4_k", w, x[rows], kq.moe_plan(torch.zeros((T, 1), dtype=torch.int32, device="cuda"), 1), F, K)
    assert torch.equal(out, few[rows])


def test_many_rows_of_long_k():
    E, F = 2, 64
    ids = many_ids((60, 45))
    w, p = experts("q4_k", E, 2 * F, 5376)
    gate_up("q4_k", w, p, bf16(len(ids), 5376), ids, F)


def test_many_rows_with_special_values():
    """Rows of zeros, of tiny and of huge values, and of NaN and infinity beside plain ones."""
    E, F, K = 2, 128, 512
    ids = many_ids((80, 60))
    w, p = experts("q4_k", E, 2 * F, K)
    x = bf16(len(ids), K)
    x[3] = 0
    x[5] *= 1e-30
    x[9] *= 1e15
    x[11, 200:] *= 1e-6
    clean = gate_up("q4_k", w, p, x, ids, F)
    x[20, 7], x[21, 300] = float("nan"), float("inf")
    out = kq.moe_gate_up("q4_k", w, x, kq.moe_plan(dev(ids), E), F, K)
    keep = [t for t in range(len(ids)) if t not in (20, 21)]
    assert torch.equal(out[keep], clean[keep]) and out[20].isnan().all() and not out[21].isfinite().all()


@pytest.mark.parametrize("dmin,m,bits", [(16.2, 63, 0), (20.0, 51, 0), (20.0, 52, 4), (16.25, 63, 4), (1000.0, 1, 0), (1000.0, 2, 4), (60000.0, 0, 0)])
@pytest.mark.parametrize("at", [(0, 0, 0), (1, 130, 1), (0, 199, 2)])
def test_many_rows_of_large_mins(dmin, m, bits, at):
    """Mins of a block up to what 64 dmin m in fp16 allows are computed, larger ones reported; calls of few rows take them all."""
    import oracle
    E, H, K = 2, 200, 768
    ids = many_ids((60, 45))
    w, p = experts("q4_k", E, H, K)
    block = w.view(E, H, K // 256, 144)[at]
    block[2:4] = torch.tensor([dmin], dtype=torch.float16).view(torch.uint8).cuda()
    block[8:12] = m  # of sub-blocks 0 to 3; 0 of 4 to 7
    block[12:16] &= 0x0F
    e = at[0]
    p[e] = oracle.dequant(2, w.view(E, -1)[e].cpu().numpy(), H, K).reshape(H, K)
    ones = torch.ones((len(ids), 1), device="cuda")
    x = bf16(len(ids), K)
    down("q4_k", w, p, x[:40], ids[:40], ones[:40], H)
    assert kq.device_errors() == 0
    if bits:
        kq.moe_down("q4_k", w, x, kq.moe_plan(dev(ids), E), dev(ids), ones, H, K)
    else:
        down("q4_k", w, p, x, ids, ones, H)
    assert kq.device_errors() == bits


def test_many_rows_in_a_plan_out_of_bounds():
    E, F, K = 4, 64, 256
    ids = many_ids((50, 60, 70, 40))
    w, p = experts("q4_k", E, 2 * F, K)
    x = bf16(len(ids), K)
    good = kq.moe_plan(dev(ids), E)
    want = gate_up("q4_k", w, p, x, ids, F)
    assert kq.device_errors() == 0
    for change in ("order", "offsets", "negative"):
        order, off = good.order.clone(), good.offsets.clone()
        if change == "order":
            order[0], order[77] = len(ids), -5
        elif change == "offsets":
            off[E] = len(ids) + 1
        else:
            off[0] = -1
        act = torch.full((len(ids), F), 3.0, dtype=torch.bfloat16, device="cuda")
        kq.moe_gate_up("q4_k", w, x, kq.MoePlan(off, order), F, K, act=act)
        assert kq.device_errors() == 2, change
        same = (act == want).all(1)
        assert (same | (act == 3.0).all(1)).all() and not same.all() and same.any()


@pytest.mark.parametrize("last", [10, 179, 0, -1])
def test_many_rows_in_a_plan_whose_last_offset_falls(last):
    """Only the last expert is left out: the others' rows are computed, also those behind the last offset. The workspace holds zeros
    beforehand, which read as rows' tags name pair 0: a place that nobody has written to changes row 0."""
    E, F, H, K = 4, 64, 200, 256
    ids = many_ids((50, 60, 70, 40))
    T = len(ids)
    w1, p1 = experts("q4_k", E, 2 * F, K)
    w2, p2 = experts("q4_k", E, H, K, 1)
    x, ones = bf16(T, K), torch.ones((T, 1), device="cuda")
    good = kq.moe_plan(dev(ids), E)
    act = gate_up("q4_k", w1, p1, x, ids, F)
    y = down("q4_k", w2, p2, x, ids, ones, H)
    assert kq.device_errors() == 0
    off = good.offsets.clone()
    off[E] = last
    plan = kq.MoePlan(off, good.order)
    rest = torch.from_numpy(ids[:, 0] < 3).cuda()
    for mark in (3.0, 5.0):
        ws = torch.zeros(kq.moe_gate_up_workspace_size("q4_k", T, 1, E, F, K), dtype=torch.uint8, device="cuda")
        out = torch.full((T, F), mark, dtype=torch.bfloat16, device="cuda")
        kq.moe_gate_up("q4_k", w1, x, plan, F, K, act=out, workspace=ws)
        assert kq.device_errors() == 2
        assert torch.equal(out[rest], act[rest]) and (out[~rest] == mark).all()
    ws = torch.zeros(kq.moe_down_workspace_size("q4_k", T, 1, E, H, K), dtype=torch.uint8, device="cuda")
    out = kq.moe_down("q4_k", w2, x, plan, dev(ids), ones, H, K, workspace=ws)
    assert kq.device_errors() == 2
    assert torch.equal(out[rest], y[rest]) and not out[~rest].any()


def test_many_rows_in_twice_as_many_places_as_the_order_fills():
    """Places behind the last expert's rows have no pair, and are no error."""
    E, F, K = 2, 64, 256
    ids = many_ids((70, 60))
    both = np.concatenate((ids, np.full_like(ids, -1)))
    w, p = experts("q4_k", E, 2 * F, K)
    gate_up("q4_k", w, p, bf16(len(both), K), both, F)
    assert kq.device_errors() == 0


def test_many_rows_twice_give_the_same_bits_on_two_streams():
    E, F, K = 6, 256, 512
    ids = many_ids((90, 33, 500, 10, 64, 200))
    w, p = experts("q4_k", E, 2 * F, K)
    x, plan = bf16(len(ids), K), kq.moe_plan(dev(ids), E)
    want = gate_up("q4_k", w, p, x, ids, F)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(4):
        got += [kq.moe_gate_up("q4_k", w, x, plan, F, K, stream=s) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) for a in got)


def test_products_agree_with_gemv():
    E, H, K, T = 3, 520, 2560, 4
    ids = np.array([[0], [2], [1], [2]], np.int32)
    w, p = experts("q4_k", E, H, K)
    x = bf16(T, K)
    y = down("q4_k", w, p, x, ids, torch.ones((T, 1), device="cuda"), H)
    size = kq.row_bytes("q4_k", K) * H
    for t in range(T):
        e = int(ids[t, 0])
        g = kq.gemv("q4_k", w[e * size:(e + 1) * size], x[t:t + 1], H, K)
        b = np.abs(x[t].double().cpu().numpy()) @ np.abs(p[e]).T
        assert (np.abs((g[0] - y[t]).double().cpu().numpy()) <= 2 * TOL * b).all()


def test_added_rows_types_strides_and_in_place():
    T, k, E, H, K = 13, 2, 4, 264, 512
    ids = some_ids(T, k, E, none=0.2)
    w, p = experts("q4_k", E, H, K)
    act, weights = bf16(T * k, K), some_weights(T, k)
    wide = torch.randn((T, H + 9), device="cuda")
    add = wide[:, 5:5 + H]
    y = down("q4_k", w, p, act, ids, weights, H, add=add)
    yb = down("q4_k", w, p, act, ids, weights, H, add=add, dtype=torch.bfloat16)
    assert torch.equal(yb, y.to(torch.bfloat16))
    out = torch.full((T, H + 3), 9.0, device="cuda")
    down("q4_k", w, p, act, ids, weights, H, add=add, y=out[:, 1:1 + H])
    assert torch.equal(out[:, 1:1 + H], y) and (out[:, 0] == 9.0).all() and (out[:, 1 + H:] == 9.0).all()
    plan = kq.moe_plan(dev(ids), E)
    kq.moe_down("q4_k", w, act, plan, dev(ids), weights, H, K, add=add, y=add)
    assert torch.equal(add, y)
    x = bf16(T, K + 24)[:, 8:8 + K]
    w, p = experts("q4_k", E, 2 * 40, K)
    gate_up("q4_k", w, p, x, ids, 40)


def test_tokens_without_experts_get_what_is_added():
    T, k, E, H, K = 4, 2, 3, 64, 256
    ids = np.full((T, k), -1, np.int32)
    w, p = experts("q4_k", E, H, K)
    act = torch.full((T * k, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    add = torch.randn((T, H), device="cuda")
    plan = kq.moe_plan(dev(ids), E)
    y = kq.moe_down("q4_k", w, act, plan, dev(ids), torch.full((T, k), float("nan"), device="cuda"), H, K, add=add)
    assert torch.equal(y, add)
    assert not kq.moe_down("q4_k", w, act, plan, dev(ids), some_weights(T, k), H, K).any()


def test_a_nan_stays_in_its_token():
    T, k, E, H, K = 20, 1, 2, 96, 512
    ids = np.zeros((T, k), np.int32)
    w, p = experts("q4_k", E, 2 * H, K)
    x = bf16(T, K)
    clean = gate_up("q4_k", w, p, x, ids, H)
    x[7, 100] = float("nan")
    x[9, 3] = float("inf")
    out = kq.moe_gate_up("q4_k", w, x, kq.moe_plan(dev(ids), E), H, K)
    keep = [t for t in range(T) if t not in (7, 9)]
    assert torch.equal(out[keep], clean[keep]) and out[7].isnan().all() and not out[9].isfinite().all()


def test_plans_out_of_bounds_are_left_out_and_reported():
    T, k, E, F, K = 6, 2, 4, 32, 256
    ids = some_ids(T, k, E)
    w, p = experts("q4_k", E, 2 * F, K)
    x = bf16(T, K)
    good = kq.moe_plan(dev(ids), E)
    want = gate_up("q4_k", w, p, x, ids, F)
    assert kq.device_errors() == 0
    for change in ("order", "offsets", "falling", "negative"):
        order, off = good.order.clone(), good.offsets.clone()
        if change == "order":
            order[0], order[3] = T * k, -5
        elif change == "offsets":
            off[E] = T * k + 1
        elif change == "falling":
            off[2] = 0 if off[1] > 0 else -1
        else:
            off[0] = -1
        act = torch.full((T * k, F), 3.0, dtype=torch.bfloat16, device="cuda")
        kq.moe_gate_up("q4_k", w, x, kq.MoePlan(off, order), F, K, act=act)
        assert kq.device_errors() == 2, change
        same = (act == want).all(1)
        if change == "falling":  # expert 1 is left out; expert 2 has the pairs that its offsets name, the others' too
            last = good.order[good.offsets[3]:good.offsets[4]].long()
            assert same[last].all()
        else:
            assert (same | (act == 3.0).all(1)).all() and not same.all()


def test_captured_and_replayed_with_other_choices():
    T, k, E, H, F = 24, 2, 8, 512, 256
    w1, p1 = experts("q4_k", E, 2 * F, H)
    w2, p2 = experts("q6_k", E, H, F, 1)
    x, ids, weights = bf16(T, H), dev(some_ids(T, k, E)), some_weights(T, k)

    def step():
        plan = kq.moe_plan(ids, E)
        act = kq.moe_gate_up("q4_k", w1, x, plan, F, H)
        return kq.moe_down("q6_k", w2, act, plan, ids, weights, H, F)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for seed in (5, 6):
        new = some_ids(T, k, E, seed=seed, none=0.1)
        ids.copy_(dev(new))
        x.copy_(bf16(T, H, seed=seed))
        graph.replay()
        a = gate_up("q4_k", w1, p1, x, new, F)
        a = torch.where(ids.flatten()[:, None] < 0, 0, a)
        assert torch.equal(down("q6_k", w2, p2, a, new, weights, H), y)


def test_two_streams_at_once():
    T, k, E, H, F = 40, 2, 8, 512, 256
    w, p = experts("q4_k", E, 2 * F, H)
    calls = [(bf16(T, H, seed=i), some_ids(T, k, E, seed=i)) for i in range(2)]
    plans = [kq.moe_plan(dev(i), E) for _, i in calls]
    want = [gate_up("q4_k", w, p, x, i, F) for x, i in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[], []]
    for _ in range(5):
        for n, s in enumerate(streams):
            got[n].append(kq.moe_gate_up("q4_k", w, calls[n][0], plans[n], F, H, stream=s))
    torch.cuda.synchronize()
    for n in range(2):
        assert all(torch.equal(a, want[n]) for a in got[n])


def test_no_tokens():
    w, _ = experts("q4_k", 2, 32, 256)
    plan = kq.moe_plan(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 2)
    assert kq.moe_gate_up("q4_k", w, torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), plan, 16, 256).shape == (0, 16)
    y = kq.moe_down("q4_k", w, torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), plan,
                    torch.empty((0, 2), dtype=torch.int32, device="cuda"), torch.empty((0, 2), device="cuda"), 32, 256)
    assert y.shape == (0, 32)
