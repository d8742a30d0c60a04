"""Greedy decoding of several requests through a decoder whose feed-forward is a mixture of quantized experts.

The decoder of paged_decode.py (its pages, rotary positions, 8-bit cache and head) with experts in place of each layer's
feed-forward, and norms that keep a row's bits whatever the batch:

    kq.residual_norm   the block's output normed, added to the residual stream, and the sum normed for what follows
    kq.gemm            the router's logits
    kq.moe_route       the experts of each token and their weights (sigmoid scores, a bias for balance, groups)
    kq.moe_plan        the tokens of each expert
    kq.moe_gate_up     gate and up products of the chosen experts, silu(gate) * up
    kq.moe_down        down products, a token's experts under their weights, onto the shared expert's output

Up to 32 tokens per step a request gets the tokens it would get alone.

    python examples/moe_decode.py [--requests 5] [--tokens 12]
"""
from __future__ import annotations

import argparse

import torch

from paged_decode import PagedDecoder, generate, kq, weights_cuda

SMALL = dict(n_layers=2, hidden=512, n_q=8, n_kv=2, head_dim=64, ffn=256, vocab=2000, theta=10000.0, eps=1e-6, experts=16, choices=4,
             groups=4, top_groups=2, route_scale=2.0)


class MoEDecoder(PagedDecoder):
    """Experts in Q4_K (gate | up) and Q6_K (down), a shared expert beside them, the router in Q8_0."""

    def __init__(self, d=SMALL, seed=0, **kw):
        super().__init__(d, seed=seed, **kw)  # its gate_up and down become the shared expert's
        h, f, E = d["hidden"], d["ffn"], d["experts"]
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        tid = 1000
        for lay in self.layers:
            lay["router"] = kq.quantize("q8_0", weights_cuda(E, h, seed=seed, tensor_id=tid))
            lay["experts_gate_up"] = torch.cat([kq.quantize("q4_k", weights_cuda(2 * f, h, seed=seed, tensor_id=tid + 1 + 2 * e)) for e in range(E)])
            lay["experts_down"] = torch.cat([kq.quantize("q6_k", weights_cuda(h, f, seed=seed, tensor_id=tid + 2 + 2 * e)) for e in range(E)])
            lay["bias"] = 0.05 * torch.randn((E,), generator=g, device="cuda")
            for name in ("attn_in", "attn_out", "ffn_in", "ffn_out"):
                lay[name] = 1 + 0.1 * torch.randn((h,), generator=g, device="cuda")
            tid += 1 + 2 * E
        self.norm_out = 1 + 0.1 * torch.randn((h,), generator=g, device="cuda")

    def _experts(self, lay, x, record=None):
        """The mixture's output (fp32) for normed rows x (bf16)."""
        d = self.d
        logits = kq.gemm("q8_0", lay["router"], x, d["experts"], d["hidden"])
        ids, weights = kq.moe_route(logits, d["choices"], score="sigmoid", bias=lay["bias"], n_group=d["groups"], top_group=d["top_groups"],
                                    group_score="top2", scale=d["route_scale"])
        plan = kq.moe_plan(ids, d["experts"])
        act = kq.moe_gate_up("q4_k", lay["experts_gate_up"], x, plan, d["ffn"], d["hidden"])
        gate, up = self._product(lay, "gate_up", x).chunk(2, -1)
        shared = self._product(lay, "down", (torch.nn.functional.silu(gate) * up).to(torch.bfloat16))
        y = kq.moe_down("q6_k", lay["experts_down"], act, plan, ids, weights, d["hidden"], d["ffn"], add=shared, y=shared)
        if record is not None:
            record.append(dict(x=x, logits=logits, ids=ids, weights=weights, act=act, y=y))
        return y

    def step(self, new: dict[int, list[int]], logits: bool = False, record: list | None = None):
        """Runs the new tokens of the slots given; returns {slot: next token}, or {slot: logits} if asked. record: receives what
        passed each layer's experts."""
        d, B = self.d, self.table.shape[0]
        counts = [len(new.get(s, ())) for s in range(B)]
        tokens = [t for s in range(B) for t in new.get(s, ())]
        T = len(tokens)
        assert 0 < T <= self.max_tokens
        new_len = torch.tensor(counts, dtype=torch.int32, device="cuda")
        plan = kq.pages_plan(self.length, new_len, self.table, self.free, self.n_free, self.page_size, T)
        if plan.status.item():  # nothing was handed out: the decoder is as it was
            raise RuntimeError(f"pages_plan refused the step: status {plan.status.item()}")
        self.n_free = plan.n_free.clone()
        max_len = max(a + b for a, b in zip(self.lens, counts))
        h = self.embed[torch.tensor(tokens, device="cuda")]
        x = kq.residual_norm(h, None, pre=self.layers[0]["attn_in"], eps=d["eps"])[1]
        for i, (lay, cache) in enumerate(zip(self.layers, self.caches)):
            qkv = self._product(lay, "qkv", x)
            q = qkv[:, :self.q_dim].unflatten(1, (d["n_q"], -1))
            k = qkv[:, self.q_dim:self.q_dim + self.kv_dim].unflatten(1, (d["n_kv"], -1))
            v = qkv[:, self.q_dim + self.kv_dim:].unflatten(1, (d["n_kv"], -1))
            q, k = kq.rope(q, k, plan.pos, self.freq)
            kq.kv8_append(cache, k, v, plan.slot)
            o = kq.attention_kv8(q, cache, self.table, self.length, new_len, max(counts), max_len, out_dtype=torch.bfloat16)
            h, x = kq.residual_norm(h, self._product(lay, "o", o.flatten(1)), post=lay["attn_out"], pre=lay["ffn_in"], eps=d["eps"], h_out=h)
            after = self.layers[i + 1]["attn_in"] if i + 1 < len(self.layers) else self.norm_out
            h, x = kq.residual_norm(h, self._experts(lay, x, record), post=lay["ffn_out"], pre=after, eps=d["eps"], h_out=h)
        self.length += new_len
        self.lens = [a + b for a, b in zip(self.lens, counts)]
        live = [s for s in range(B) if counts[s]]
        hidden = x[torch.tensor([sum(counts[:s + 1]) - 1 for s in live], device="cuda")]
        if logits:
            y = kq.gemm("q8_0", self.head, hidden, d["vocab"], d["hidden"])
            return {s: y[i] for i, s in enumerate(live)}
        got = []
        for i in range(0, len(live), 16):
            got += kq.head_argmax(self.head, None, hidden[i:i + 16].contiguous(), d["vocab"], d["hidden"], all_rows=True)[0].tolist()
        return dict(zip(live, got))


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=5)
    ap.add_argument("--tokens", type=int, default=12)
    a = ap.parse_args()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, SMALL["vocab"], (3 + 17 * i % 41,), generator=g).tolist() for i in range(a.requests)]
    dec = MoEDecoder(slots=4)
    for p, o in zip(prompts, generate(dec, prompts, a.tokens)):
        print(f"prompt of {len(p)} tokens -> {o}")
    print(f"pages free at the end: {dec.n_free.item()}")


if __name__ == "__main__":
    main()
