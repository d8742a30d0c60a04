"""Calls of the paged cache from two host threads, each on its own stream with its own batch size."""
import threading

import numpy as np
import pytest
import torch

import quantized_decode_gemv_block_gb300 as kq
from test_gpu_kv8 import dev, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    yield
    assert kq.device_errors() == 0


def batch(B, new, y, seed):
    """A call of B requests, one of them joined from segments, and its output made by this thread alone."""
    P, D, n_q, n_kv = 16, 64, 4, 2
    lens = [(5 + i % 30, new) for i in range(B - 1)] + [(900, new)]
    cache, _, table, ctx, new_len, q = make(lens, P, D, n_q, n_kv, "bf16", seed)
    td, cd, nd = dev(table), dev(ctx), dev(new_len)
    ws = torch.empty(kq.attention_kv8_workspace_size(B, int((ctx + new_len).sum()), new, n_q, n_kv, D), dtype=torch.uint8, device="cuda")
    out = torch.empty(q.shape, dtype=y, device="cuda")

    def call():
        kq.attention_kv8(q, cache, td, cd, nd, new, 900 + new, total_len=int((ctx + new_len).sum()), out=out, workspace=ws)
    call()
    torch.cuda.synchronize()
    return call, out, out.clone()


def in_threads(work):
    """Runs the functions in threads of their own, on streams of their own; returns what they raised."""
    raised = []

    def body(f):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                f()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            raised.append(e)
    torch.cuda.synchronize()
    ts = [threading.Thread(target=body, args=(f,)) for f in work]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    return raised


@pytest.mark.parametrize("new,y", [(1, torch.float32), (6, torch.bfloat16), (40, torch.bfloat16)])
def test_batches_of_two_sizes_in_turn(new, y):
    """One thread with many requests, one with few, strictly in turn."""
    a, b = batch(300, new, y, 1), batch(8, new, y, 2)
    gate = threading.Barrier(2, timeout=60)

    def first():
        try:
            for _ in range(5):
                a[0]()
                gate.wait()  # the other's turn
                gate.wait()
        except Exception:
            gate.abort()
            raise

    def second():
        try:
            for _ in range(5):
                gate.wait()
                b[0]()
                gate.wait()
        except Exception:
            gate.abort()
            raise
    a[1].fill_(0)
    b[1].fill_(0)
    assert in_threads([first, second]) == []
    assert torch.equal(a[1], a[2]) and torch.equal(b[1], b[2])


def test_batches_of_two_sizes_at_once():
    """Free-running threads: attention with few and with thousands of requests (whose join takes more than 48 KB),
    plans of 4096 and 4095 requests."""
    a, b, c = batch(4096, 1, torch.float32, 3), batch(3, 1, torch.float32, 4), batch(2048, 1, torch.float32, 5)
    plans = []
    for B in (4096, 4095):
        ctx, new = dev(np.arange(B) % 16), dev(np.ones(B))
        table = torch.arange(2 * B, dtype=torch.int32, device="cuda").view(B, 2).contiguous()
        free, n = torch.arange(9000, dtype=torch.int32, device="cuda"), dev([9000])
        out = kq.PagesPlan(B, B)
        plans.append((lambda *x, t=table, o=out, B=B: kq.pages_plan(*x, 16, B, out=o), (ctx, new, table, free, n), out))

    def many(f):
        def loop():
            for _ in range(200):
                f()
        return loop
    for x in (a, b, c):
        x[1].fill_(0)
    assert in_threads([many(a[0]), many(b[0]), many(c[0])] + [many(lambda f=f, x=x: f(*x)) for f, x, _ in plans]) == []
    for x in (a, b, c):
        assert torch.equal(x[1], x[2])
    assert all(o.status.item() == 0 for _, _, o in plans)
