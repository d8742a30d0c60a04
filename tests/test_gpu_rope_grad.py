"""Gradients of kq.rope through autograd: against the formula (the rotation back) and against differences, which are exact for a
linear map but for rounding. Tolerances: see the rotary positions' tests."""
import numpy as np
import pytest
import torch

import quantized_decode_gemv_block_gb300 as kq
from test_gpu_rope import DT, check, freqs, plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def inputs(T, axes, pairs, seed=0):
    rng = np.random.default_rng(seed)
    pos, axis = rng.integers(0, 5000, (axes, T)).astype(np.int32), rng.integers(0, axes, pairs).astype(np.uint8)
    return pos, axis, torch.tensor(pos, device="cuda"), torch.tensor(axis, device="cuda"), torch.tensor(freqs(pairs), device="cuda")


@pytest.mark.parametrize("x,y", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("adjacent,inverse", [(False, False), (True, False), (False, True)])
def test_gradients_are_the_rotation_back(x, y, adjacent, inverse):
    T, pairs = 9, 24
    pos, axis, pd, ad, f = inputs(T, 2, pairs)
    q, k = (torch.randn((T, h, 64), device="cuda").to(DT[x]).requires_grad_() for h in (4, 2))
    gq, gk = (torch.randn((T, h, 64), device="cuda").to(DT[y]) for h in (4, 2))
    oq, ok = kq.rope(q, k, pd, f, pair_axis=ad, adjacent=adjacent, inverse=inverse, out_dtype=DT[y])
    with torch.no_grad():
        a, b = kq.rope(q, k, pd, f, pair_axis=ad, adjacent=adjacent, inverse=inverse, out_dtype=DT[y])
    assert torch.equal(a, oq) and torch.equal(b, ok) and not a.requires_grad and oq.dtype == DT[y]
    torch.autograd.backward((oq, ok), (gq, gk))
    for t, g in ((q, gq), (k, gk)):
        assert t.grad.dtype == DT[x]
        check(t.grad, *plain(g, pos, freqs(pairs), axis, adjacent, not inverse), (x, y))


@pytest.mark.parametrize("adjacent", [False, True])
def test_gradients_against_differences(adjacent):
    T, D = 5, 16
    _, _, pd, ad, f = inputs(T, 2, 6)
    q, g = torch.randn((T, 1, D), device="cuda").requires_grad_(), torch.randn((T, 1, D), device="cuda")
    kq.rope(q, None, pd, f, pair_axis=ad, adjacent=adjacent)[0].backward(g)
    with torch.no_grad():
        for e in range(T * D):
            d = torch.zeros(T * D, device="cuda")
            d[e] = 1.0
            hi, lo = (kq.rope(q + s * d.view_as(q), None, pd, f, pair_axis=ad, adjacent=adjacent)[0].double() for s in (1, -1))
            # each of a pair's two outputs is off by 2^-21 (|a| + |b|), values below 8, times |g| below 6
            assert abs((((hi - lo) / 2) * g.double()).sum().item() - q.grad.flatten()[e].item()) < 2 * 2.0 ** -21 * 16 * 6


def test_one_of_two_and_views_and_expanded_gradients():
    """q and k as views of one product's rows; gradients that autograd hands over expanded, transposed, or not at all."""
    T, D, pairs = 7, 32, 16
    pos, _, pd, _, f = inputs(T, 1, pairs)
    rows = torch.randn((T, 5 * D), device="cuda", requires_grad=True)
    q, k = rows[:, :3 * D].unflatten(1, (3, D)), rows[:, 3 * D:].unflatten(1, (2, D))
    oq, ok = kq.rope(q, k, pd[0], f)
    (oq.sum() + (ok.transpose(0, 1) * 2).sum()).backward()
    ones = torch.cat([torch.ones((T, 3, D)), torch.full((T, 2, D), 2.0)], 1)
    ref, base = plain(ones, pos, freqs(pairs), np.zeros(pairs, int), False, True)
    check(rows.grad.view(T, 5, D), ref, base, "fused rows")
    rows.grad = None
    oq, ok = kq.rope(q, k, pd[0], f)
    ok.sum().backward()  # nothing comes back for q
    assert (rows.grad[:, :3 * D] == 0).all() and rows.grad[:, 3 * D:].abs().sum() > 0
    qd = q.detach()
    oq, ok = kq.rope(qd, k, pd[0], f)  # k alone requires a gradient
    assert not oq.requires_grad
    assert torch.autograd.grad(ok.sum() + oq.sum(), rows)[0][:, :3 * D].abs().sum() == 0


def test_gradients_of_gradients():
    T, D = 4, 16
    _, _, pd, _, f = inputs(T, 1, 8)
    q = torch.randn((T, 1, D), device="cuda", requires_grad=True)
    g = torch.randn((T, 1, D), device="cuda", requires_grad=True)
    o, _ = kq.rope(q, None, pd[0], f)
    dq, = torch.autograd.grad(o, q, g, create_graph=True)
    w = torch.randn_like(dq)
    back, = torch.autograd.grad(dq, g, w)
    with torch.no_grad():
        assert torch.equal(back, kq.rope(w, None, pd[0], f)[0])


def test_other_streams_and_a_captured_step():
    T, D = 33, 64
    pos, _, pd, _, f = inputs(T, 1, 32)
    x, g = torch.randn((T, 2, D), device="cuda"), torch.randn((T, 2, D), device="cuda")
    ref, base = plain(g, pos, freqs(32), np.zeros(32, int), False, True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q = x.clone().requires_grad_()
        grad, = torch.autograd.grad(kq.rope(q, None, pd[0], f)[0], q, g)
    s.synchronize()
    check(grad, ref, base, "stream")
    del grad
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        grad, = torch.autograd.grad(kq.rope(q, None, pd[0], f)[0], q, g)
    g.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    check(grad, 2 * ref, 2 * base, "captured")
