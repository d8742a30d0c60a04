"""Rotary positions (kq_rope) against the formula in 64 bits, its inverse as its gradient, strides and ranges.

Tolerance per element: the angle is off by at most 2^-32 turn of truncation and 2^-27 half turns of rounding
(under 2^-24 rad together), sincospif by 2 units of 2^-24, each of the two products and the sum by a rounding of 2^-24:
under 2^-21 (|a| + |b|) in all, and the output's rounding of eps/2 of the result.
"""
import numpy as np
import pytest
import torch

import quantized_decode_gemv_block_gb300 as kq

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def plain(x, pos, freq, axis, adjacent, inverse):
    """(result, |a| + |b| of each element's pair) in 64 bits; angles in Python's own precision of pos * freq."""
    x = x.double().cpu().numpy()
    h = len(freq)
    ang = np.stack([pos[axis[i]].astype(np.longdouble) * np.longdouble(freq[i]) for i in range(h)], -1) if h else np.zeros((x.shape[0], 0))
    c, s = np.cos(ang).astype(np.float64)[:, None], np.sin(ang).astype(np.float64)[:, None] * (-1 if inverse else 1)
    m = np.arange(h) * 2 if adjacent else np.arange(h)
    n = m + (1 if adjacent else h)
    y, b = x.copy(), np.abs(x)
    y[..., m], y[..., n] = x[..., m] * c - x[..., n] * s, x[..., n] * c + x[..., m] * s
    b[..., m] = b[..., n] = np.abs(x[..., m]) + np.abs(x[..., n])
    return y, b


def check(out, ref, base, what):
    tol = base * 2.0 ** -21 + np.abs(ref) * torch.finfo(out.dtype).eps / 2
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (what, (err - tol).max())


def freqs(h, base=10000.0):
    return (base ** (-np.arange(h) / max(h, 1))).astype(np.float32)


def case(T, nq, nk, D, rot, axes, x, y, adjacent, inverse, far=5000, view=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + T)
    rng = np.random.default_rng(seed + T)
    w = (nq + nk) * D + view
    rows = torch.randn((T, w), generator=g, device="cuda").to(DT[x])
    q, k = rows[:, :nq * D].unflatten(1, (nq, D)), rows[:, nq * D:(nq + nk) * D].unflatten(1, (nk, D))
    if not view:
        q, k = q.contiguous(), k.contiguous()
    h = rot // 2
    pos = rng.integers(-far, far + 1, (axes, T)).astype(np.int32)
    axis = rng.integers(0, axes, h).astype(np.uint8)
    f = freqs(h)
    qo, ko = kq.rope(q if nq else None, k if nk else None, torch.tensor(pos, device="cuda"), torch.tensor(f, device="cuda"),
                     pair_axis=torch.tensor(axis, device="cuda") if axes > 1 else None, adjacent=adjacent, inverse=inverse, out_dtype=DT[y])
    for a, o in ((q, qo), (k, ko)):
        if o is not None:
            ref, base = plain(a, pos, f, axis if axes > 1 else np.zeros(h, int), adjacent, inverse)
            check(o, ref, base, (T, nq, nk, D, rot))


@pytest.mark.parametrize("x,y", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("T,nq,nk,D,rot,axes,view", [(1, 4, 1, 64, 64, 1, 0), (3, 32, 8, 128, 128, 3, 0), (17, 5, 1, 80, 80, 2, 16),
                                                     (9, 3, 3, 80, 20, 3, 0), (33, 8, 2, 96, 48, 1, 7), (5, 1, 0, 256, 64, 3, 8),
                                                     (4, 2, 1, 7, 4, 1, 0), (6, 2, 2, 64, 0, 1, 0), (700, 16, 4, 64, 32, 3, 256)])
def test_matches_the_formula(x, y, adjacent, T, nq, nk, D, rot, axes, view):
    case(T, nq, nk, D, rot, axes, x, y, adjacent, inverse=T % 2 == 0, view=view)


@pytest.mark.parametrize("D,rot", [(32, 32), (24, 20)])
def test_many_tokens(D, rot):
    """CTAs that take several tokens each, the last of them fewer."""
    case(5003, 2, 1, D, rot, 3, "bf16", "f32", True, False)


def test_rows_that_start_off_16_bytes():
    rows = torch.randn((11, 3 * 64 + 1), device="cuda")
    q = rows[:, 1:1 + 128].unflatten(1, (2, 64))
    pos = np.arange(11, dtype=np.int32)[None]
    o, _ = kq.rope(q, None, torch.tensor(pos, device="cuda"), torch.tensor(freqs(32), device="cuda"))
    check(o, *plain(q, pos, freqs(32), np.zeros(32, int), False, False), "off 16 bytes")


@pytest.mark.parametrize("x,y", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("T,nq,nk,D,rot,view", [(40, 3, 1, 64, 64, 2), (700, 6, 2, 80, 20, 0), (65, 2, 2, 96, 24, 6), (9, 1, 1, 12, 8, 0),
                                                (5, 2, 1, 132, 132, 0), (300, 3, 2, 80, 40, 0), (40, 3, 1, 64, 64, 4),
                                                (21, 1, 2, 72, 72, 12), (4, 1, 1, 88, 0, 0)])
def test_rows_and_halves_that_start_on_two_or_four_elements(x, y, adjacent, T, nq, nk, D, rot, view):
    case(T, nq, nk, D, rot, 2, x, y, adjacent, True, view=view)


@pytest.mark.parametrize("far", [2 ** 24, 2 ** 31 - 1])
def test_far_positions(far):
    case(40, 2, 1, 64, 64, 2, "f32", "f32", False, False, far=far)


def test_quarter_turns_and_extreme_frequencies():
    """pos * freq at and next to multiples of a quarter turn; frequencies of 0, above 1, negative and tiny."""
    f = np.array([np.pi / 2, np.pi / 4, np.pi, 1.0, 0.0, -0.7, 6.2831855, 1e-12, 3e-39, 100.5, -np.pi, 0.5, 2.0 ** -20, 1e-7, 0.1, 7.0], np.float32)
    pos = np.arange(-20, 21, dtype=np.int32)[None]
    x = torch.randn((41, 1, 32), device="cuda")
    o, _ = kq.rope(x, None, torch.tensor(pos, device="cuda"), torch.tensor(f, device="cuda"))
    check(o, *plain(x, pos, f, np.zeros(16, int), False, False), "quarter turns")


@pytest.mark.parametrize("adjacent", [False, True])
def test_in_place(adjacent):
    x = torch.randn((50, 3, 64), device="cuda").to(torch.bfloat16)
    pos, f = torch.arange(50, dtype=torch.int32, device="cuda"), torch.tensor(freqs(32), device="cuda")
    want, _ = kq.rope(x, None, pos, f, adjacent=adjacent)
    got, _ = kq.rope(x, None, pos, f, adjacent=adjacent, q_out=x)
    assert got is x and torch.equal(got, want)


@pytest.mark.parametrize("adjacent", [False, True])
def test_the_inverse_is_the_gradient(adjacent):
    """Against the formula's adjoint (<R x, g> = <x, R^-1 g>) and against differences, which are exact for a
    linear map but for fp32 rounding."""
    T, H, D = 7, 2, 32
    x, g = torch.randn((T, H, D), device="cuda"), torch.randn((T, H, D), device="cuda")
    pos, f = torch.randint(0, 9999, (T,), dtype=torch.int32, device="cuda"), torch.tensor(freqs(16), device="cuda")
    fwd = lambda v: kq.rope(v, None, pos, f, adjacent=adjacent)[0].double()  # noqa: E731
    grad = kq.rope(g, None, pos, f, adjacent=adjacent, inverse=True)[0].double()
    ref, base = plain(g, pos.cpu().numpy()[None], freqs(16), np.zeros(16, int), adjacent, True)
    check(grad.float(), ref, base, "adjoint formula")
    for e in range(0, T * H * D, 37):
        d = torch.zeros(T * H * D, device="cuda")
        d[e] = 1.0
        diff = ((fwd(x + d.view_as(x)) - fwd(x - d.view_as(x))) / 2 * g.double()).sum()
        # each of the pair's two outputs is off by 2^-21 (|a| + |b|) at magnitudes below 8, times |g| below 6
        assert abs(diff.item() - grad.flatten()[e].item()) < 2 * 2.0 ** -21 * 16 * 6


def test_an_axis_without_positions_turns_nothing():
    x = torch.randn((4, 1, 32), device="cuda")
    pos = torch.full((2, 4), 100, dtype=torch.int32, device="cuda")
    o, _ = kq.rope(x, None, pos, torch.ones(16, device="cuda"), pair_axis=torch.full((16,), 2, dtype=torch.uint8, device="cuda"))
    assert torch.equal(o, x)


def test_nothing_to_do():
    q, k = kq.rope(torch.zeros((0, 2, 64), device="cuda"), None, torch.zeros(0, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda"))
    assert q.shape == (0, 2, 64) and k is None
