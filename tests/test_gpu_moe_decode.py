"""The example with experts: norms, routing, plan and the experts' products in a row, beside the paged cache's operators."""
import os
import sys

import numpy as np
import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import moe_decode
    return moe_decode


def prompts(ex, n, seed=3):
    rng = np.random.default_rng(seed)
    return [rng.integers(0, ex.SMALL["vocab"], int(rng.integers(1, 60))).tolist() for _ in range(n)]


def test_a_request_gets_the_tokens_it_gets_alone(ex):
    import quantized_decode_gemv_block_gb300 as kq
    ps = prompts(ex, 6)
    dec = ex.MoEDecoder(slots=3)
    together = ex.generate(dec, ps, 7)
    assert dec.n_free.item() == 64 and sorted(dec.free.tolist()) == list(range(64))
    for p, want in zip(ps, together):
        assert ex.generate(ex.MoEDecoder(slots=1), [p], 7) == [want]
    assert kq.device_errors() == 0


def test_a_layers_experts_are_the_definition(ex):
    """What passed the experts of each layer in a step of two requests, against 64 bits on the oracle's weights: ids equal, the
    output within the products' 1e-4 of their terms, the activations' rounding to bf16 (2^-8 of each) under the down
    weights, and the routing weights' fp32."""
    import oracle
    d = ex.SMALL
    dec = ex.MoEDecoder(slots=2)
    rec = []
    dec.step({0: prompts(ex, 1)[0][:9], 1: [4, 5, 6]}, record=rec)
    assert len(rec) == d["n_layers"]
    h, f, E, k = d["hidden"], d["ffn"], d["experts"], d["choices"]
    deq = lambda fmt, w, n, m: np.asarray(oracle.dequant(fmt, np.ascontiguousarray(w.cpu().numpy()), n, m)).reshape(n, m)  # noqa: E731
    for lay, r in zip(dec.layers, rec):
        x, s = r["x"].double().cpu().numpy(), 1 / (1 + np.exp(-r["logits"].double().cpu().numpy()))
        choice = s + lay["bias"].double().cpu().numpy()
        top2 = np.sort(choice.reshape(len(x), d["groups"], -1), -1)[..., -2:].sum(-1)
        w1, w2 = lay["experts_gate_up"].view(E, 2 * f, -1), lay["experts_down"].view(E, h, -1)
        wg, wd = deq(2, lay["gate_up"], 2 * f, h), deq(2, lay["down"], h, f)
        for t in range(len(x)):
            kept = np.argsort(-top2[t], kind="stable")[:d["top_groups"]]
            c = np.where(np.isin(np.arange(E) // (E // d["groups"]), kept), choice[t], -np.inf)
            ids = np.argsort(-c, kind="stable")[:k]
            assert r["ids"][t].tolist() == ids.tolist()
            p = s[t, ids] / s[t, ids].sum() * d["route_scale"]

            def mlp(a, b, weight):
                g, u = (a[:f] @ x[t], a[f:] @ x[t])
                act = g / (1 + np.exp(-g)) * u
                err = 1e-4 * (np.abs(a[:f]) @ np.abs(x[t]) * (1.1 * np.abs(u)) + np.abs(a[f:]) @ np.abs(x[t]) * np.abs(g)) + np.abs(act) * 2.0 ** -8
                size = np.abs(b) @ np.abs(act)
                return weight * (b @ act), weight * (np.abs(b) @ err * 1.01 + 1e-4 * size + 2.0 ** -18 * size)
            parts = [mlp(wg, wd, 1.0)] + [mlp(deq(2, w1[e], 2 * f, h), deq(5, w2[e], h, f), q) for e, q in zip(ids, p)]
            ref, tol = sum(a for a, _ in parts), sum(b for _, b in parts)
            assert (np.abs(r["y"][t].double().cpu().numpy() - ref) <= tol).all()


def test_a_layer_captured_and_replayed(ex):
    """The run from the norm to the mixture's output as one graph, replayed with other rows, gives the bits of plain calls."""
    import quantized_decode_gemv_block_gb300 as kq
    dec = ex.MoEDecoder(slots=1)
    lay, d = dec.layers[0], ex.SMALL
    g = torch.Generator(device="cuda").manual_seed(5)
    h, y = (torch.randn((24, d["hidden"]), generator=g, device="cuda") for _ in range(2))

    def run():
        a, x = kq.residual_norm(h, y, post=lay["attn_out"], pre=lay["ffn_in"], eps=d["eps"])
        return kq.residual_norm(a, dec._experts(lay, x), post=lay["ffn_out"], pre=dec.norm_out, eps=d["eps"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(3):
        h.copy_(torch.randn(h.shape, generator=g, device="cuda"))
        y.copy_(torch.randn(y.shape, generator=g, device="cuda"))
        graph.replay()
        want = run()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_the_command_runs(ex, capsys, monkeypatch):
    monkeypatch.setattr(sys, "argv", ["moe_decode.py", "--requests", "3", "--tokens", "4"])
    ex.main()
    out = capsys.readouterr().out
    assert out.count("->") == 3 and "pages free at the end: 64" in out
