"""Routing to experts and the plan of their rows against plain forms in 64 bits.

Ids have to be equal: choices are those of 64-bit scores. Weights, u = 2^-24: a difference of logits rounds once and is off by
u |d|, which exp makes u |d| of its result; expf, the sum of up to 1024 positive terms (32 of a lane, 5 levels), the
division and the scale add 2 + 37 + 3: w (|d| + 42 + 42) u for scores divided by their sum, d the distance from the
largest logit (softmax) or the logit (sigmoid).
"""
import numpy as np
import pytest
import torch

import quantized_decode_gemv_block_gb300 as kq

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def best(c, n):
    """The n largest of c in falling order, ties to the lowest; those that cannot be chosen (-inf) left out."""
    order = sorted(range(len(c)), key=lambda i: (-c[i], i))
    return [i for i in order if c[i] > -np.inf][:n]


def plain(x, k, score, bias, G, g, group, renorm, scale):
    """(ids, weights, distances) token by token."""
    T, E = x.shape
    ids, weights, far = np.full((T, k), -1, np.int32), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        v = np.where(np.isnan(x[t]), -np.inf, np.minimum(x[t], np.finfo(np.float32).max))
        top = v.max()
        with np.errstate(over="ignore", invalid="ignore"):
            if score == "softmax":
                s = np.exp(v - top) if top > -np.inf else np.zeros(E)
                z = s.sum()
                s = s / z if z > 0 else s
            else:
                s = 1 / (1 + np.exp(-v))
        c = v.copy() if bias is None else np.where((v == -np.inf) | ~(bias > -np.inf), -np.inf, s + np.nan_to_num(bias, nan=0.0, posinf=np.inf))
        if G > 1:
            n = E // G
            cs = c if bias is not None or group == "max" else np.where(v == -np.inf, -np.inf, s)
            gs = []
            for i in range(G):
                two = sorted(cs[i * n:(i + 1) * n])[::-1][:2]
                gs.append(two[0] + (two[1] if len(two) > 1 and two[1] > -np.inf else 0.0) if group == "top2" else two[0])
            kept = best(gs, g)
            for i in range(G):
                if i not in kept:
                    c[i * n:(i + 1) * n] = -np.inf
        got = best(c, k)
        w = s[got]
        if renorm:
            if score == "softmax" and len(got):
                w = np.exp(v[got] - v[got].max())
            w = w / w.sum() if w.sum() > 0 else w
        ids[t, :len(got)], weights[t, :len(got)] = got, w * scale
        base = (v[got].max() if renorm and len(got) else top) if score == "softmax" else 0.0
        far[t, :len(got)] = np.abs(v[got] - base)
    return ids, weights, far


def run(x, k, score="softmax", bias=None, G=1, g=1, group="max", renorm=True, scale=1.0, **kw):
    ids, w = kq.moe_route(x, k, score=score, bias=bias, n_group=G, top_group=g, group_score=group, renorm=renorm, scale=scale, **kw)
    b = None if bias is None else bias.double().cpu().numpy()
    want, ww, far = plain(x.double().cpu().numpy(), k, score, b, G, g, group, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), want), np.argwhere(ids.cpu().numpy() != want)[:5]
    got = w.double().cpu().numpy()
    assert (np.abs(got - ww) <= ww * (far + 84) * U + 2.0 ** -126).all(), np.abs(got - ww).max()
    return ids, w


def logits(T, E, x="f32", seed=0, spread=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * T + E)
    return (spread * torch.randn((T, E), generator=g, device="cuda")).to(DT[x])


def some_bias(E, seed=0):
    return 0.1 * torch.randn((E,), generator=torch.Generator(device="cuda").manual_seed(seed + E), device="cuda")


@pytest.mark.parametrize("E", [1, 2, 3, 31, 32, 33, 60, 64, 128, 160, 256, 257, 512, 1000, 1024])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sizes_types_and_scores(E, x, score):
    for k in {1, min(E, 2), min(E, 8), min(E, 32)}:
        for bias in (None, some_bias(E)):
            run(logits(37, E, x), k, score, bias, renorm=k != 2, scale=1.0 if k != 8 else 2.5)


@pytest.mark.parametrize("G,per", [(2, 1), (2, 8), (3, 5), (4, 15), (8, 4), (8, 32), (16, 16), (32, 2), (32, 32), (5, 7)])
@pytest.mark.parametrize("group", ["max", "top2"])
def test_groups(G, per, group):
    E = G * per
    for g in {1, max(1, G // 2), G}:
        for bias in (None, some_bias(E)):
            for score in ("softmax", "sigmoid"):
                run(logits(23, E, "bf16" if g == 1 else "f32"), min(g * per, 6), score, bias, G, g, group)


def test_equal_logits_go_to_the_lowest_expert():
    x = torch.zeros((3, 96), device="cuda")
    x[1, 40:] = 1.0
    x[2, ::2] = -1.0
    for bias in (None, torch.zeros(96, device="cuda")):
        for score in ("softmax", "sigmoid"):
            ids, _ = run(x, 5, score, bias)
            assert ids.tolist() == [[0, 1, 2, 3, 4], [40, 41, 42, 43, 44], [1, 3, 5, 7, 9]]
            run(x, 5, score, bias, 8, 2, "top2")
            run(x, 5, score, bias, 8, 2, "max")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choices_that_fp32_cannot_order(score):
    """Biases that make sums of score and bias equal to a few units of 2^-30: the order is that of 64 bits."""
    T, E = 64, 64
    x = logits(T, E, "f32", seed=5)
    v = x[0].double()
    s = torch.softmax(v, -1) if score == "softmax" else torch.sigmoid(v)
    step = torch.randint(0, 5, (E,), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").double() * 2.0 ** -30
    bias = (1.0 - s + step).float()  # rounds to units of 2^-24 or finer: sums are within a few of them of 1
    x = x[:1].expand(T, E).contiguous()
    run(x, 8, score, bias)
    run(x, 8, score, bias, 8, 3, "top2")
    run(x, 8, score, bias, 8, 3, "max")


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [32, 64, 256, 1000])
def test_equals_at_the_border_and_a_larger_one_behind_them(E, score, x):
    """The k-th choice and the next ones have the same logit and bias; one behind them is their equal in fp32 and larger in 64 bits: sigmoids of
    17 and 18 are both 1 in fp32, and so are softmax scores of about 2^-30 beside a bias of 1."""
    rows = torch.zeros((6, E), device="cuda")
    low, high = (17.0, 18.0) if score == "sigmoid" else (1.0, 2.0)
    for t, at in enumerate(([0, 1], [0, 1, 2], [3, 4, 9, 10], [0, 30], [1, 2, 3, 4, 5, 6, 7], [0, 1])):
        rows[t, at] = low
        rows[t, E - 1 - t] = high
    rows[5, E - 2] = high  # two equals behind
    if score == "softmax":
        rows[:, 20] = 22.0
    bias = torch.zeros(E, device="cuda")
    if score == "softmax":
        bias += 1.0
        bias[20] = -1.0
    for k in (1, 2, 3, 5, 8):
        run(rows.to(DT[x]), k, score, bias)
        for G, g in ((4, 2), (8, 3)):
            if k <= E // G * g and E % G == 0:
                run(rows.to(DT[x]), k, score, bias, G, g, "top2")
                run(rows.to(DT[x]), k, score, bias, G, g, "max")


def test_groups_whose_two_best_cancel():
    """A sum of 1000 + s and -1000 + s' is off by units of 2^-14 in fp32, whatever it comes to; beside it a group whose sum is nearer than that."""
    T = 96
    g = torch.Generator(device="cuda").manual_seed(11)
    s = 0.3 + 0.3 * torch.rand((T, 8), generator=g, device="cuda", dtype=torch.float64)
    apart = (10 ** (-6 + 1.6 * torch.rand(T, generator=g, device="cuda", dtype=torch.float64))) * (torch.arange(T, device="cuda") % 2 * 2 - 1)
    s[:, 5] = s[:, 0] + s[:, 1] - s[:, 4] + apart
    x = torch.log(s / (1 - s)).float()
    bias = torch.tensor([1000.0, -1000.0, -float("inf"), -float("inf"), 0.0, 0.0, -float("inf"), -float("inf")], device="cuda")
    run(x, 2, "sigmoid", bias, 2, 1, "top2")
    run(x[:, [4, 5, 6, 7, 0, 1, 2, 3]].contiguous(), 2, "sigmoid", bias[[4, 5, 6, 7, 0, 1, 2, 3]].contiguous(), 2, 1, "top2")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_of_the_lowest_value(score):
    """A bias of fp32's lowest value puts an expert last without excluding it: the sum of two such choices is below fp32's range, and still above a
    group without any choice and below one with a single such choice."""
    x = logits(20, 16)
    low = torch.finfo(torch.float32).min
    for first, second in ((-float("inf"), low), (low, -float("inf"))):
        bias = some_bias(16)
        bias[:4], bias[4:8] = first, second
        for group in ("top2", "max"):
            run(x, 10, score, bias, 4, 3, group)
            run(x, 8, score, bias, 4, 2, group)
        one = bias.clone()
        one[:8] = low
        one[5:8] = -float("inf")
        run(x, 9, score, one, 4, 3, "top2")
    run(x, 16, score, torch.full((16,), low, device="cuda"), 4, 4, "top2")
    run(x, 4, score, torch.full((16,), low, device="cuda"), 4, 2, "top2")


def test_experts_that_cannot_be_chosen():
    """-inf and NaN logits, whole rows of them, +inf, and biases that exclude."""
    x = logits(9, 40)
    x[0] = -float("inf")
    x[1] = float("nan")
    x[2, 3:] = -float("inf")
    x[3, ::2] = -float("inf")
    x[4, 7] = float("inf")
    x[5, 7] = x[5, 30] = float("inf")
    x[6, 1:] = float("nan")
    bias = some_bias(40)
    bias[5], bias[6], bias[7] = -float("inf"), float("nan"), float("inf")
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            for renorm in (True, False):
                ids, w = run(x, 6, score, b, renorm=renorm)
                assert ids[0].tolist() == [-1] * 6 and not w[0].any() and not w.isnan().any()
                run(x, 6, score, b, 5, 2, "top2", renorm)
                run(x, 6, score, b, 5, 2, "max", renorm)


def test_large_logits():
    x = logits(20, 128, spread=60.0)
    for score in ("softmax", "sigmoid"):
        run(x.clamp(-80, 80), 8, score)
        run(x.clamp(-30, 30), 8, score, some_bias(128))
    ids, w = kq.moe_route(torch.full((2, 64), -200.0, device="cuda"), 4, score="sigmoid")
    assert ids.tolist() == [[0, 1, 2, 3]] * 2 and not w.any()  # every score is 0 in fp32, and so is their sum


def test_strided_logits_given_outputs_and_rows_alone():
    wide = logits(301, 200, "bf16")
    x, bias = wide[:, 40:168], some_bias(128)
    ids, w = torch.full((301, 8), 7, dtype=torch.int32, device="cuda"), torch.empty((301, 8), device="cuda")
    a = run(x, 8, "sigmoid", bias, 8, 4, "top2", ids=ids, weights=w)
    assert a[0] is ids and a[1] is w
    for t in (0, 150, 300):
        one = kq.moe_route(x[t:t + 1], 8, score="sigmoid", bias=bias, n_group=8, top_group=4, group_score="top2")
        assert torch.equal(one[0][0], ids[t]) and torch.equal(one[1][0], w[t])


def test_many_tokens():
    run(logits(2500, 64, "bf16"), 6, "softmax", None, 8, 3, "max", False, 16.0)


# ---------------------------------------------------------------- plan

def plain_plan(ids, E):
    flat = ids.reshape(-1)
    order = [p for e in range(E) for p in np.flatnonzero(flat == e)]
    n = np.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
    return np.concatenate(([0], np.cumsum(n))), np.array(order + [-1] * (len(flat) - len(order)), np.int64)


def check_plan(ids, E, **kw):
    plan = kq.moe_plan(torch.tensor(ids, dtype=torch.int32, device="cuda"), E, **kw)
    off, order = plain_plan(ids, E)
    assert np.array_equal(plan.offsets.cpu().numpy(), off) and np.array_equal(plan.order.cpu().numpy(), order)
    return plan


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 128), (3, 2, 5), (16, 8, 128), (33, 1, 1024), (100, 32, 60), (511, 8, 256), (512, 8, 256),
                                   (513, 8, 256), (1000, 6, 64), (4097, 4, 1024), (9000, 8, 8), (20000, 10, 512)])
def test_plan(T, k, E):
    rng = np.random.default_rng(T + k + E)
    ids = rng.integers(0, E, (T, k))
    check_plan(ids, E)
    ids[rng.random((T, k)) < 0.2] = -1
    check_plan(ids, E)


def test_plan_of_one_expert_of_none_and_of_ids_out_of_range():
    check_plan(np.full((3000, 4), 17), 64)
    check_plan(np.full((77, 4), -1), 64)
    check_plan(np.array([[0, 64, 5], [-7, 63, 2 ** 31 - 1], [-2 ** 31, 5, 5]]), 64)
    plan = check_plan(np.zeros((0, 4), np.int64), 9)
    assert plan.order.shape == (0,)


def test_plan_of_the_largest_batch():
    T, k, E = 1 << 20, 8, 300
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    plan = kq.moe_plan(ids, E)
    key = torch.where(ids.flatten() < 0, E, ids.flatten())
    want = torch.sort(key, dim=0, stable=True).indices
    live = int((key < E).sum())
    assert plan.offsets[-1].item() == live
    assert torch.equal(plan.order[:live].long(), want[:live]) and (plan.order[live:] == -1).all()
    assert torch.equal(plan.offsets[1:].long(), torch.bincount(key, minlength=E + 1)[:E].cumsum(0))


def test_route_and_plan_captured_and_replayed():
    x = logits(600, 128)
    out = kq.MoePlan(torch.empty(129, dtype=torch.int32, device="cuda"), torch.empty(4800, dtype=torch.int32, device="cuda"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kq.moe_plan(kq.moe_route(x, 8)[0], 128, out=out)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, w = kq.moe_route(x, 8)
        kq.moe_plan(ids, 128, out=out)
    for seed in (8, 9):
        x.copy_(logits(600, 128, seed=seed))
        graph.replay()
        want = kq.moe_route(x, 8)
        assert torch.equal(ids, want[0]) and torch.equal(w, want[1])
        plan = kq.moe_plan(ids, 128)
        assert torch.equal(plan.offsets, out.offsets) and torch.equal(plan.order, out.order)
