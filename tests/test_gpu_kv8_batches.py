"""Batches of every size up to 4096 requests, in processes of their own: the requests' shared memory passes 48 KB with the
kernels' own at sizes below the largest, and a call of more requests made before would have opened the way."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import kv8_plain as plain
import quantized_decode_gemv_block_gb300 as kq
from conftest import ROOT

pytestmark = pytest.mark.gpu


def dev(a, dtype=np.int32):
    return torch.tensor(np.asarray(a, dtype), device="cuda")


def plans():
    P = 16
    for B in (4000, 4051, 4052, 4053, 4094, 4095, 4096):
        rng = np.random.default_rng(B)
        ctx, new = rng.integers(0, 40, B), rng.integers(0, 3, B)
        held, want = -(-ctx // P), -(-(ctx + new) // P)
        pages = rng.permutation(int(want.sum()))
        table = np.full((B, 4), -1, np.int32)
        table[np.arange(4) < held[:, None]] = pages[:held.sum()]
        free, T = pages[held.sum():], int(new.sum())
        p = kq.pages_plan(dev(ctx), dev(new), td := dev(table), dev(free), dev([len(free)]), P, T)
        rest = list(free)
        for r in range(B):
            for b in range(held[r], want[r]):
                table[r, b] = rest.pop()
        cu = np.concatenate([[0], np.cumsum(new)])
        req = np.repeat(np.arange(B), new)
        pos = ctx[req] + np.arange(T) - cu[req]
        assert p.status.item() == 0 and p.n_free.item() == len(rest) and np.array_equal(td.cpu(), table), B
        assert np.array_equal(p.cu.cpu(), cu) and np.array_equal(p.slot.cpu(), table[req, pos // P] * P + pos % P), B


def releases():
    for B in (4000, 4095, 4096):
        done = torch.arange(B, device="cuda") % 3 == 0
        table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
        free, out = torch.full((B,), -5, dtype=torch.int32, device="cuda"), dev([0])
        st = kq.pages_release(torch.full((B,), 7, dtype=torch.int32, device="cuda"), done, table, free, dev([0]), out, 16)
        n = int(done.sum())
        assert st.item() == 0 and out.item() == n and torch.equal(free[:n], torch.arange(0, B, 3, dtype=torch.int32, device="cuda"))


def attentions(D):
    """Batches in which a few requests are joined from several segments; each of them equal to itself alone and near the
    64-bit form (tolerance: see the attention's tests, fp32 output)."""
    P, n_q, n_kv = 16, 4, 4
    lengths = [700, 1500, 513, 2100]
    rng = np.random.default_rng(D)
    for B in (1800, 1864, 1865, 1866, 1867, 1868, 1950, 1951, 1952, 1953, 2046, 2047, 2048, 4095, 4096):
        ctx, new = np.zeros(B, np.int64), np.ones(B, np.int64)
        long = np.sort(rng.permutation(B)[:4])
        ctx[long] = np.array(lengths) - 1
        nb = -(-(ctx + new) // P)
        pages = int(nb.sum())
        perm = rng.permutation(pages).astype(np.int32)
        table = np.zeros((B, int(nb.max())), np.int32)
        table[np.arange(table.shape[1]) < nb[:, None]] = perm
        kc, vc = (rng.integers(-128, 128, (pages, n_kv, P, D), dtype=np.int8) for _ in range(2))
        ks, vs = (np.exp2(rng.integers(-7, -4, (pages, n_kv))).astype(np.float32) for _ in range(2))
        cache = kq.KV8Cache(pages, P, n_kv, D, k=dev(plain.stored(kc, P, D, "k"), np.int8), v=dev(plain.stored(vc, P, D, "v"), np.int8),
                            k_scale=dev(ks, np.float32), v_scale=dev(vs, np.float32))
        q = torch.tensor(rng.standard_normal((B, n_q, D)), device="cuda").float()
        o = kq.attention_kv8(q, cache, dev(table), dev(ctx), dev(new), 1, 2100, total_len=int((ctx + new).sum()))
        for r in long:
            a = kq.attention_kv8(q[r:r + 1], cache, dev(table[r:r + 1]), dev(ctx[r:r + 1]), dev([1]), 1, 2100)
            assert torch.equal(a[0], o[r]), (B, r)
        some = np.concatenate([long, [0, B // 2, B - 1]])
        ref, base, mag = plain.attention(q[some].double().cpu().numpy(), kc, ks, vc, vs, table[some], ctx[some], new[some], P, n_kv, D ** -0.5)
        err = np.abs(o[some].double().cpu().numpy() - ref)
        assert (err <= base * (2 * mag * 2.0 ** -17 + 2.0 ** -19) + np.abs(ref) * 2.0 ** -23).all(), B


@pytest.mark.parametrize("call", ["plans()", "releases()", "attentions(64)", "attentions(128)"])
def test_every_batch_size_in_a_fresh_process(call):
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    tests = os.path.join(ROOT, "tests")
    code = f"import sys; sys.path[:0] = [{ROOT!r}, {tests!r}]; import test_gpu_kv8_batches as t; t.{call}; assert t.kq.device_errors() == 0"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
