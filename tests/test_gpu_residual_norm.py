"""The norms around a residual sum (kq_residual_norm) against the formula in 64 bits.

Tolerances, u = 2^-24: a sum of squares is off by at most 69 u of itself (32 terms of a thread, 5 levels of a warp, 32 warps), so
with the division, eps, rsqrtf (2 units) and two products rms(v) w is off by 41 u of itself; times gate and scale, 43 u. h' adds
its own rounding. x = h' f w: h' is off by e, f by |e| / |h'| (2-norms) + 39 u of itself, and two products round. Each output is
then rounded to its type, eps/2 of the result.
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


def rms(v, eps):
    return v / np.sqrt(np.mean(v * v, -1, keepdims=True) + eps)


def num(t):
    return None if t is None else t.double().cpu().numpy()


def plain(h, y, post, gate, scale, pre, eps, off):
    """(h', its error bound, x, its error bound) in 64 bits, without the outputs' rounding."""
    w = lambda t: 1.0 if t is True else num(t) + (1.0 if off else 0.0)  # noqa: E731
    z = np.zeros(1) if y is None else num(y) if post is None else rms(num(y), eps) * w(post)
    part = scale * z * (1.0 if gate is None else num(gate))
    s = part + (0.0 if h is None else num(h))
    e = 43 * U * np.abs(part) + U * np.abs(s)
    if pre is None:
        return s, e, None, None
    x = rms(s, eps) * w(pre)
    size = np.sqrt((s * s).sum(-1, keepdims=True))
    f = x / np.where(s == 0, 1, s)
    f = np.abs(np.where(s == 0, w(pre) / np.sqrt(np.mean(s * s, -1, keepdims=True) + eps), f))
    loss = np.sqrt((e * e).sum(-1, keepdims=True)) / np.where(size == 0, 1, size) + 41 * U
    return s, e, x, f * e + np.abs(x) * loss


def check(out, ref, tol, what):
    o = num(out)
    err = np.abs(o - ref)
    lim = tol + (np.abs(ref) + tol) * torch.finfo(out.dtype).eps / 2
    assert (err <= lim).all(), (what, (err - lim).max())


def make(T, H, y="f32", h="f32", w="f32", post=True, pre=True, gate="", seed=0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * T + H)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    wide = lambda dt: (3 * r(T, H + pad)).to(DT[dt])[:, :H]  # noqa: E731
    a = dict(h=wide(h) if h else None, y=wide(y) if y else None)
    a["post"] = (1 + 0.3 * r(H)).to(DT[w]) if post == True else post or None  # noqa: E712
    a["pre"] = (1 + 0.3 * r(H)).to(DT[w]) if pre == True else pre or None  # noqa: E712
    if gate:
        a["gate"] = r(H).to(DT[y]) if gate == "one" else wide(y)
    return a


def run(a, x="bf16", scale=1.0, eps=1e-6, off=False, **kw):
    ho, xo = kq.residual_norm(**a, scale=scale, eps=eps, unit_offset=off, x_dtype=DT[x], **kw)
    s, e, v, ev = plain(a["h"], a["y"], a["post"], a.get("gate"), scale, a["pre"], eps, off)
    check(ho, s, e, "h")
    if a["pre"] is None:
        assert xo is None
    else:
        check(xo, v, ev, "x")
    return ho, xo


@pytest.mark.parametrize("H", [1, 2, 7, 8, 9, 64, 255, 256, 257, 1000, 2048, 2049, 2560, 4096, 8192, 8200, 16384, 20001, 32768])
@pytest.mark.parametrize("y,h", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
def test_sizes_and_types(H, y, h):
    for T in (1, 5):
        run(make(T, H, y, h, w=y, gate="rows"), x=h, scale=0.5)


@pytest.mark.parametrize("T", [1, 2, 3, 31, 257, 1999])
@pytest.mark.parametrize("H", [96, 512, 2560])
def test_rows(T, H):
    run(make(T, H, "f32", "f32", "bf16"))


@pytest.mark.parametrize("kw", [dict(post=None), dict(pre=None), dict(post=None, pre=None), dict(gate="one"), dict(gate="rows"), dict(h=""),
                                dict(y="", post=None), dict(h="", pre=None), dict(post=None, gate="one", pre=None)])
@pytest.mark.parametrize("off", [False, True])
def test_parts_left_out(kw, off):
    run(make(6, 1000, **{**dict(w="bf16"), **kw}), off=off, scale=1.7)
    run(make(6, 1024, **{**dict(w="f32"), **kw}), off=off)


def test_norms_without_weights():
    a = make(9, 768)
    a["post"] = a["pre"] = True
    run(a)


@pytest.mark.parametrize("pad", [1, 3, 8, 40])
def test_strides_and_alignment_keep_the_bits(pad):
    """Views into wider rows: the same values give the same bits as contiguous ones."""
    a = make(11, 1024, "bf16", "f32", gate="rows", pad=pad)
    b = {k: (v.contiguous() if isinstance(v, torch.Tensor) else v) for k, v in a.items()}
    for p, q in zip(run(a), run(b)):
        assert torch.equal(p, q)
    big = torch.empty((11, 1024 + pad), device="cuda")
    xo = torch.full((11, 1024 + pad), 5.0, device="cuda", dtype=torch.bfloat16)
    ho, x = run(a, h_out=big[:, pad:], x_out=xo[:, :1024])
    for p, q in zip((ho, x), run(b)):
        assert torch.equal(p, q)
    assert (xo[:, 1024:] == 5.0).all()


def test_a_row_has_the_bits_it_has_alone():
    a = make(300, 2560, "f32", "f32")
    ho, xo = run(a)
    for t in (0, 17, 299):
        one = {k: (v[t:t + 1] if k in ("h", "y") else v) for k, v in a.items()}
        h1, x1 = run(one)
        assert torch.equal(h1[0], ho[t]) and torch.equal(x1[0], xo[t])


def test_in_place():
    a = make(50, 1544, "bf16", "f32")
    ho, xo = run(a)
    b = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in a.items()}
    h2, x2 = kq.residual_norm(**b, h_out=b["h"], x_out=b["y"])
    assert h2 is b["h"] and x2 is b["y"] and torch.equal(h2, ho) and torch.equal(x2, xo)


def test_rows_of_zeros_and_extreme_values():
    a = make(8, 512, "f32", "f32")
    a["h"][0] = a["y"][0] = 0.0
    a["y"][1] = 1e-30
    a["y"][2] = 1e18
    a["h"][3], a["y"][3] = 1e-20, 0.0
    a["y"][4, 5] = float("inf")
    a["y"][5, 6] = float("nan")
    ho, xo = kq.residual_norm(**a, eps=1e-6)
    keep = [0, 1, 2, 3, 6, 7]
    s, e, v, ev = plain(a["h"][keep], a["y"][keep], a["post"], None, 1.0, a["pre"], 1e-6, False)
    check(ho[keep], s, e, "h")
    check(xo[keep], v, ev + 2.0 ** -149, "x")
    assert xo[4].isnan().any() and xo[5].isnan().all()  # inf / inf; a NaN makes the row's mean NaN
    assert not ho[keep].isnan().any()


@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-38, 1e-33])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("H", [40, 1001, 4096, 32768])
def test_tiny_rows_under_hardly_any_eps(H, dt, eps):
    """Rows whose squares leave fp32, down to values that are subnormal themselves, beside plain ones. eps is the fp32 number that the call takes:
    1e-44 is none, the nearest, 7 2^-149, is 2 % below it, and under these rows eps counts in full."""
    eps = float(np.float32(eps))
    a = make(8, H, dt, dt)
    for t, size in enumerate((1e-15, 1e-17, 1e-20, 1e-25, 1e-34, 1e-38, 1e-42)):
        a["y"][t] = (a["y"][t].double() * size).to(DT[dt])
    for b, k in ((dict(a, h=None), "y"), (dict(a, y=None, h=a["y"], post=None), "h")):
        if dt == "bf16" and eps == 0.0:  # 1e-42 is none of bf16's numbers but 0, and 0 / 0 is what the formula gives
            assert not b[k][6].any() and kq.residual_norm(**b, eps=eps)[1][6].isnan().all()
            b[k] = b[k][[0, 1, 2, 3, 4, 5, 7]].contiguous()
        run(b, eps=eps)


def test_a_row_of_zeros_without_eps_is_nan():
    a = make(3, 1001, "f32", "f32")
    a["h"][1] = 0.0
    h, x = kq.residual_norm(a["h"], None, pre=a["pre"], eps=0.0)
    assert torch.equal(h, a["h"]) and x[1].isnan().all() and x[::2].isfinite().all()
    assert not kq.residual_norm(a["h"], None, pre=a["pre"], eps=1e-40)[1][1].any()


def test_eps_counts():
    a = make(4, 640)
    a["y"] *= 1e-4
    run(a, eps=1e-5)
    run(a, eps=0.5)


def test_captured_and_replayed_on_a_stream():
    a = make(64, 2048, "f32", "f32")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kq.residual_norm(**a)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ho, xo = kq.residual_norm(**a)
    for seed in (3, 4):
        b = make(64, 2048, "f32", "f32", seed=seed)
        for k, v in b.items():
            a[k].copy_(v)
        graph.replay()
        want = kq.residual_norm(**b)
        assert torch.equal(ho, want[0]) and torch.equal(xo, want[1])


def test_given_stream():
    a = make(700, 2560)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ho, xo = kq.residual_norm(**a, stream=s)
    s.synchronize()
    want = run(a)
    assert torch.equal(ho, want[0]) and torch.equal(xo, want[1])


def test_no_tokens():
    h, x = kq.residual_norm(torch.empty((0, 64), device="cuda"), torch.empty((0, 64), device="cuda"), pre=True)
    assert h.shape == x.shape == (0, 64)
