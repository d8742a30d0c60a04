"""fp32 queries of the attention over the paged 8-bit cache, where the output is bf16: carried in 22 bits.

Two kinds of keys give a row nearly the same score, one through the dims whose query values lie almost half a step of
fp16 above a number that fp16 holds, the other through dims whose values lie as far below one. Scores of about 100 then move apart
by 0.1 if queries are rounded to fp16, and the output, values of +-1 weighted by the two kinds, by 0.05.

Tolerance per element, base = sum_p w_p |v_p|, mag = largest sum_d |scale q_d k_pd|: q in two fp16 parts (2^-22 of each
product) and fp32 sums of D <= 128 products (below 2^-18 of their magnitudes), so a score is off by under mag 2^-17; weights in fp16
(2^-12) twice, in the sum and its norm; the output's rounding: base (2 mag 2^-17 + 2^-11) + 2^-8 of the result.
"""
import numpy as np
import pytest
import torch

import kv8_plain as plain
import quantized_decode_gemv_block_gb300 as kq
from test_gpu_kv8 import dev, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    yield
    assert kq.device_errors() == 0


def two_kinds(lens, P, D, n_q, n_kv, seed):
    rng = np.random.default_rng(seed)
    ctx, new = np.array([c for c, _ in lens]), np.array([n for _, n in lens])
    nb = -(-(ctx + new) // P)
    pages = int(nb.sum())
    perm, at = rng.permutation(pages), 0
    table = np.zeros((len(lens), int(nb.max())), np.int32)
    for r, n in enumerate(nb):
        table[r, :n] = perm[at:at + n]
        at += n
    half = D // 2
    kind = rng.integers(0, 2, (pages, n_kv, P))
    # +100.5 on the kind's half of the dims; elsewhere +0.5 and -0.5 in turn
    kc = np.broadcast_to(np.where(np.arange(D) % 2, -1, 0), (pages, n_kv, P, D)).copy()
    vc = np.empty((pages, n_kv, P, D), np.int64)
    for a in (0, 1):
        kc[kind == a, a * half:(a + 1) * half] = 100
        vc[kind == a] = (63, -64)[a]
    ks = np.full((pages, n_kv), 2.0 ** -6, np.float32)
    q = np.empty((int(new.sum()), n_q, D), np.float32)
    q[..., :half] = 1 + 0.49 * 2.0 ** -10   # down to 1 in fp16
    q[..., half:] = 1 + 0.51 * 2.0 ** -10   # up to 1 + 2^-10
    q *= np.exp2(rng.integers(-3, 1, q.shape[:2] + (1,)))
    cache = kq.KV8Cache(pages, P, n_kv, D, k=dev(plain.stored(kc.astype(np.int8), P, D, "k"), np.int8),
                        v=dev(plain.stored(vc.astype(np.int8), P, D, "v"), np.int8), k_scale=dev(ks, np.float32), v_scale=dev(ks, np.float32))
    return cache, (kc.astype(np.int8), ks, vc.astype(np.int8), ks), table, ctx, new, torch.tensor(q, device="cuda")


@pytest.mark.parametrize("D,n_q,n_kv", [(64, 4, 2), (128, 4, 1)])
@pytest.mark.parametrize("lens", [[(40, 1), (700, 1)], [(0, 3), (90, 12), (300, 32)], [(50, 40), (10, 2)]], ids=["tokens", "windows", "prompt"])
def test_scores_of_fp32_queries_keep_22_bits_for_bf16_outputs(D, n_q, n_kv, lens):
    P = 32
    cache, parts, table, ctx, new, q = two_kinds(lens, P, D, n_q, n_kv, D)
    scale = 100 / (D / 2 * 100.5 / 64)
    o = run(cache, table, ctx, new, q, "bf16", scale=scale)
    ref, base, mag = plain.attention(q.double().cpu().numpy(), *parts, table, ctx, new, P, n_kv, scale)
    tol = base * (2 * mag * 2.0 ** -17 + 2.0 ** -11) + np.abs(ref) * 2.0 ** -8
    err = np.abs(o.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (err / tol).max()
