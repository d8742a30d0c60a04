"""Rotary positions (kq_rope) at frequencies that are not finite, and at large ones. Tolerances: see the rotary positions' tests."""
import numpy as np
import pytest
import torch

import quantized_decode_gemv_block_gb300 as kq
from test_gpu_rope import check, plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("pos", [0, 5, -7])
def test_a_frequency_that_is_not_finite_breaks_its_pairs_alone(adjacent, pos):
    """cos and sin of pos * inf and of pos * NaN are NaN, at position 0 too."""
    f = np.array([1.0, np.nan, 0.5, np.inf, 0.25, -np.inf, 0.1, 3e38], np.float32)
    x = torch.randn((3, 2, 20), device="cuda")
    p = np.full((1, 3), pos, np.int32)
    o, _ = kq.rope(x, None, torch.tensor(p, device="cuda"), torch.tensor(f, device="cuda"), adjacent=adjacent)
    pair = lambda i: (2 * i, 2 * i + 1) if adjacent else (i, i + 8)  # noqa: E731
    for i in range(8):
        got = o[..., pair(i)]
        assert got.isfinite().all() if np.isfinite(f[i]) else got.isnan().all(), i
    assert torch.equal(o[..., 16:], x[..., 16:])
    g = np.where(np.isfinite(f) & (f < 2), f, 0).astype(np.float32)
    ref, base = plain(x, p, g, np.zeros(8, int), adjacent, False)
    keep = [d for i in (0, 2, 4, 6) for d in pair(i)] + [16, 17, 18, 19]
    check(o[..., keep], ref[..., keep], base[..., keep], "finite pairs")


def test_an_axis_without_positions_turns_nothing_at_any_frequency():
    x = torch.randn((4, 1, 32), device="cuda")
    pos = torch.full((2, 4), 100, dtype=torch.int32, device="cuda")
    o, _ = kq.rope(x, None, pos, torch.full((16,), float("nan"), device="cuda"),
                   pair_axis=torch.full((16,), 2, dtype=torch.uint8, device="cuda"))
    assert torch.equal(o, x)


def test_large_frequencies_at_far_positions():
    """|pos * inv_freq| up to 2^38: the reference's products are exact in 64 bits of long double or in integers."""
    f = np.array([2.0, 100.5, 127.99999, 64.0, 33.333332, 1.5, 3.1415927, 0.99999994], np.float32)
    rng = np.random.default_rng(2)
    pos = rng.integers(-2 ** 31, 2 ** 31, (1, 40)).astype(np.int32)
    x = torch.randn((40, 1, 16), device="cuda")
    o, _ = kq.rope(x, None, torch.tensor(pos, device="cuda"), torch.tensor(f, device="cuda"))
    # angle modulo a turn in integers: freq = m 2^e exactly, 2^200 / (2 pi) to 200 bits
    inv_turn = _inverse_turn(200)
    ang = np.zeros((40, 8))
    for t in range(40):
        for i in range(8):
            m, e = np.frexp(f[i])
            num = int(pos[0, t]) * int(m * 2 ** 24)  # times 2^(e - 24)
            frac = (num * inv_turn) << int(e) >> 24  # turns times 2^200
            ang[t, i] = (frac % (1 << 200)) / 2.0 ** 200 * 2 * np.pi
    a, b = (x[:, 0, :8].double().cpu().numpy(), x[:, 0, 8:].double().cpu().numpy())
    ref = np.concatenate([a * np.cos(ang) - b * np.sin(ang), b * np.cos(ang) + a * np.sin(ang)], -1)[:, None]
    base = np.tile(np.abs(a) + np.abs(b), 2)[:, None]
    check(o, ref, base, "far")


def _inverse_turn(bits):
    """floor(2^bits / (2 pi)), pi by Machin's formula in integers."""
    one = 1 << (bits + 64)

    def arctan_inverse(n):
        term, total, k = one // n, 0, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total
    pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239))
    return (one << bits) // (2 * pi)
