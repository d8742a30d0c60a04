"""The paged decoding example: the four operators together with the quantized products."""
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
    import paged_decode
    return paged_decode


def prompts(ex, n, seed=3):
    rng = np.random.default_rng(seed)
    return [rng.integers(0, ex.SMALL["vocab"], int(rng.integers(1, 60))).tolist() for _ in range(n)]


def test_a_request_gets_the_tokens_it_gets_alone(ex):
    import quantized_decode_gemv_block_gb300 as kq
    ps = prompts(ex, 7)
    dec = ex.PagedDecoder(slots=3)
    together = ex.generate(dec, ps, 9)
    assert dec.n_free.item() == 64 and sorted(dec.free.tolist()) == list(range(64))  # every page came back
    for p, want in zip(ps, together):
        assert ex.generate(ex.PagedDecoder(slots=1), [p], 9) == [want]
    assert kq.device_errors() == 0


def test_logits_are_near_a_decoder_without_a_cache(ex):
    """Against the same weights with fp32 attention over unquantized k and v of the whole sequence. A code is off by at
    most half a step, a step is at most 1/64 of its page's largest value (about 3.5 sigma): 1.6 % of sigma rms on k and v,
    which the softmax's average reduces and two layers at most double: 5 % of the logits' size bounds it."""
    import oracle
    d = ex.SMALL
    dec = ex.PagedDecoder(slots=1)
    seq = prompts(ex, 1, seed=8)[0] + [5, 6, 7, 8]
    first = len(seq) - 6
    got = []
    for i in range(0, first, 32):
        y = dec.step({0: seq[i:min(i + 32, first)]}, logits=True)[0]
    got.append(y)
    for t in seq[first:]:
        got.append(dec.step({0: [t]}, logits=True)[0])
    # the dense form
    deq = lambda fmt, w, n, k: torch.tensor(np.asarray(oracle.dequant(fmt, w.cpu().numpy(), n, k)), device="cuda").double()  # noqa: E731
    bf = lambda v: v.to(torch.bfloat16).double()  # noqa: E731
    norm = lambda v: bf(v * torch.rsqrt(v.square().mean(-1, keepdim=True) + d["eps"]))  # noqa: E731
    x = dec.embed[torch.tensor(seq, device="cuda")].double()
    T, hd = len(seq), d["head_dim"]
    pos = torch.arange(T, device="cuda").double()
    ang = pos[:, None] * dec.freq.double()
    cos, sin = ang.cos()[:, None], ang.sin()[:, None]

    def rot(v):
        a, b = v.chunk(2, -1)
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    for lay in dec.layers:
        w = {n: deq(2, lay[n], *dec.shapes[n]) for n in dec.shapes}
        qkv = norm(x) @ w["qkv"].T
        q, k, v = qkv.split([dec.q_dim, dec.kv_dim, dec.kv_dim], -1)
        q, k, v = rot(q.view(T, -1, hd)), rot(k.view(T, -1, hd)), v.view(T, -1, hd)
        k, v = (t.repeat_interleave(d["n_q"] // d["n_kv"], 1) for t in (k, v))
        s = torch.einsum("qhd,khd->hqk", q, k) * hd ** -0.5
        s = s.masked_fill(torch.ones((T, T), device="cuda").triu(1).bool(), -torch.inf).softmax(-1)
        x = x + bf(torch.einsum("hqk,khd->qhd", s, v).flatten(1)) @ w["o"].T
        gate, up = (norm(x) @ w["gate_up"].T).chunk(2, -1)
        x = x + bf(torch.nn.functional.silu(gate) * up) @ w["down"].T
    ref = (norm(x) @ deq(1, dec.head, d["vocab"], d["hidden"]).T)[first - 1:]
    err = (torch.stack(got).double() - ref).norm(dim=-1) / ref.norm(dim=-1)
    assert (err < 0.05).all(), err


def test_the_command_runs(ex, capsys, monkeypatch):
    monkeypatch.setattr(sys, "argv", ["paged_decode.py", "--requests", "3", "--tokens", "4"])
    ex.main()
    out = capsys.readouterr().out
    assert out.count("->") == 3 and "pages free at the end: 64" in out
