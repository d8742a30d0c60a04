"""Argument checks and sizes of the experts' entry points, without a GPU: every call is refused, or is empty, before any CUDA call."""
import pytest
import torch


@pytest.fixture(scope="module")
def kq():
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    import quantized_decode_gemv_block_gb300 as m
    m.load_library()
    return m


FAKE = 1 << 20  # never dereferenced


def test_route_refusals(kq):
    L = kq.lib()
    good = dict(xd=kq.BF16, x=FAKE, s=64, T=4, E=64, k=6, b=FAKE, G=8, g=2, sc=1.0, fl=7, ids=FAKE, w=FAKE)

    def call(**kw):
        a = dict(good, **kw)
        return L.kq_moe_route(a["xd"], a["x"], a["s"], a["T"], a["E"], a["k"], a["b"], a["G"], a["g"], a["sc"], a["fl"], a["ids"], a["w"], None)
    assert call(xd=0) == kq.KQ_ERR_UNSUPPORTED
    for kw in (dict(fl=8), dict(T=-1), dict(E=0), dict(E=1032, s=2000), dict(k=0), dict(k=33), dict(k=17), dict(T=1 << 21, k=8), dict(G=0),
               dict(G=7), dict(G=64), dict(g=0), dict(g=9), dict(s=63), dict(x=None), dict(ids=None), dict(w=None), dict(x=FAKE + 1),
               dict(b=FAKE + 2), dict(ids=FAKE + 1), dict(w=FAKE + 2)):
        assert call(**kw) == kq.KQ_ERR_ARG, kw
        assert L.kq_last_error().decode() != ""
    assert call(T=0, x=None, ids=None, w=None) == 0


def test_plan_refusals(kq):
    L = kq.lib()
    for a in ((FAKE, -1, 2, 8, FAKE, FAKE), (FAKE, 4, 0, 8, FAKE, FAKE), (FAKE, 4, 2, 0, FAKE, FAKE), (FAKE, 4, 2, 1025, FAKE, FAKE),
              (FAKE, 1 << 20, 9, 8, FAKE, FAKE), (None, 4, 2, 8, FAKE, FAKE), (FAKE, 4, 2, 8, None, FAKE), (FAKE, 4, 2, 8, FAKE, None),
              (FAKE + 2, 4, 2, 8, FAKE, FAKE), (FAKE, 4, 2, 8, FAKE + 1, FAKE), (FAKE, 4, 2, 8, FAKE, FAKE + 3)):
        assert L.kq_moe_plan(*a, None) == kq.KQ_ERR_ARG, a


def test_product_refusals_and_sizes(kq):
    L = kq.lib()
    good = dict(fmt=kq.Q4_K, w=FAKE, x=FAKE, xs=512, off=FAKE, ord=FAKE, ids=FAKE, wt=FAKE, T=4, k=2, E=8, N=64, K=512, act=FAKE, add=FAKE, ads=64,
                yd=kq.F32, y=FAKE + 65536, ys=64, ws=FAKE, wsn=1 << 40)

    def up(**kw):
        a = dict(good, **kw)
        return L.kq_moe_gate_up(a["fmt"], a["w"], a["x"], a["xs"], a["off"], a["ord"], a["T"], a["k"], a["E"], a["N"], a["K"], a["act"],
                                a["ws"], a["wsn"], None)

    def down(**kw):
        a = dict(good, **kw)
        return L.kq_moe_down(a["fmt"], a["w"], a["x"], a["off"], a["ord"], a["ids"], a["wt"], a["T"], a["k"], a["E"], a["N"], a["K"], a["add"],
                             a["ads"], a["yd"], a["y"], a["ys"], a["ws"], a["wsn"], None)
    for f in (up, down):
        assert f(fmt=9) == kq.KQ_ERR_UNSUPPORTED
        for kw in (dict(T=-1), dict(k=0), dict(k=33), dict(E=0), dict(E=1025), dict(N=0), dict(N=(1 << 20) + 1), dict(K=0), dict(K=500),
                   dict(K=20736, xs=20736), dict(E=1024, N=1 << 20, xs=512), dict(T=(1 << 22) + 1), dict(w=None), dict(x=None), dict(off=None),
                   dict(ord=None), dict(w=FAKE + 8), dict(x=FAKE + 8), dict(off=FAKE + 2), dict(ord=FAKE + 2)):
            assert f(**kw) == kq.KQ_ERR_ARG, (f, kw)
            assert L.kq_last_error().decode() != ""
        assert f(T=0, w=None, x=None) == 0
        # one row of one 210-byte block: the last row's aligned copy would pass the buffer's end
        assert f(fmt=kq.Q6_K, E=1, N=1, K=256, xs=256, ads=256, ys=256) == kq.KQ_ERR_UNSUPPORTED
    for kw in (dict(xs=511), dict(xs=516), dict(act=None), dict(act=FAKE + 8)):
        assert up(**kw) == kq.KQ_ERR_ARG, kw
    assert down(yd=5) == kq.KQ_ERR_UNSUPPORTED
    for kw in (dict(ys=63), dict(ads=63), dict(y=None), dict(ids=None), dict(wt=None), dict(y=FAKE + 2), dict(add=FAKE + 1),
               dict(add=FAKE + 65536, ads=65), dict(add=FAKE + 65536, yd=kq.BF16)):
        assert down(**kw) == kq.KQ_ERR_ARG, kw
    for kw in (dict(ws=None), dict(ws=FAKE + 16), dict(wsn=100)):
        assert down(**kw) == kq.KQ_ERR_WORKSPACE, kw
    assert kq.moe_down_workspace_size("q4_k", 4, 2, 8, 64, 512) >= 4 * 2 * 64 * 4
    for bad in ((99, 4, 2, 8, 64, 512), (kq.Q4_K, 4, 33, 8, 64, 512), (kq.Q4_K, 4, 2, 8, 64, 500), (kq.Q4_K, -1, 2, 8, 64, 512)):
        assert L.kq_moe_down_workspace_size(*bad) == 0 and L.kq_moe_gate_up_workspace_size(*bad) == 0


def test_the_bindings_limits_are_the_headers(kq):
    import os
    import re

    from conftest import ROOT
    text = open(os.path.join(ROOT, "include", "kq.h")).read()
    names = re.findall(r"\b(KQ_(?:MOE|NORM|ROUTE)_\w+) = (\d+)u?\b", text)
    assert len(names) == 10
    for name, value in names:
        assert getattr(kq, name) == int(value), name


def test_binding_refusals(kq):
    x = torch.zeros((4, 64))
    i32 = dict(dtype=torch.int32)
    for kw, match in ((dict(score="relu"), "softmax"), (dict(group_score="sum"), "top2"), (dict(bias=torch.zeros(63)), "bias"),
                      (dict(bias=torch.zeros(64).bfloat16()), "bias"), (dict(ids=torch.zeros((4, 7), **i32)), "ids"),
                      (dict(weights=torch.zeros((4, 8)).t()), "weights")):
        with pytest.raises(ValueError, match=match):
            kq.moe_route(x, 8, stream=0, **kw)
    with pytest.raises(ValueError, match="tokens, experts"):
        kq.moe_route(x[0], 8, stream=0)
    with pytest.raises(ValueError, match="gradient"):
        kq.moe_route(x.clone().requires_grad_(), 8, stream=0)
    ids = torch.zeros((4, 2), **i32)
    for bad in (ids.long(), ids[:, :1].expand(4, 2), ids.flatten()):
        with pytest.raises(ValueError):
            kq.moe_plan(bad, 8, stream=0)
    with pytest.raises(ValueError, match="offsets"):
        kq.MoePlan(torch.zeros(1, **i32), torch.zeros(8, **i32))
    with pytest.raises(ValueError, match="order"):
        kq.MoePlan(torch.zeros(9, **i32), torch.zeros(8))
    plan = kq.MoePlan(torch.zeros(9, **i32), torch.zeros(8, **i32))
    w = torch.zeros(8 * 64 * 288, dtype=torch.uint8)
    xb = torch.zeros((4, 512), dtype=torch.bfloat16)
    for a, match in (((w[1:], xb, plan, 32, 512), "blocks"), ((w, xb.float(), plan, 32, 512), "bf16"), ((w, xb, plan, 64, 512), "blocks"),
                     ((w, xb[:3], plan, 32, 512), "choices"), ((w, xb[:, :256], plan, 32, 512), "must be")):
        with pytest.raises(ValueError, match=match):
            kq.moe_gate_up("q4_k", *a, stream=0)
    wt, act = torch.zeros((4, 2)), torch.zeros((8, 512), dtype=torch.bfloat16)
    for a, kw, match in (((act[:7], plan, ids, wt), {}, "act"), ((act, plan, ids.long(), wt), {}, "ids"), ((act, plan, ids, wt.double()), {}, "weights"),
                         ((act, plan, ids[:3], wt[:3]), {}, "plan"), ((act, plan, ids, wt), dict(add=xb[:, :64]), "fp32"),
                         ((act, plan, ids, wt), dict(y=torch.zeros((4, 63))), "must be"),
                         ((act, plan, ids, wt), dict(y=torch.zeros((4, 64)), out_dtype=torch.bfloat16), "out_dtype")):
        with pytest.raises(ValueError, match=match):
            kq.moe_down("q4_k", w, *a, 64, 512, stream=0, **kw)
