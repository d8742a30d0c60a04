"""Greedy decoding of several requests over a paged 8-bit KV cache.

A small random decoder with block-quantized weights serves requests of uneven length together. One step
takes each request's new tokens (its prompt, then one token at a time) through

    kq.pages_plan     slots and block-table entries of the new tokens, from the lengths on the GPU
    per layer:
      kq.gemm         q, k, v of all new tokens
      kq.rope         positions into q and k
      kq.kv8_append   k and v into the layer's pages, 8 bits
      kq.attention_kv8  over each request's pages
      kq.gemm         the layer's other products
    kq.head_argmax    the next token of each request

and a request that ends gives its pages back (kq.pages_release). Up to 32 tokens per step every product
keeps a row's bits whatever the batch, and so do the four operators. Prompts enter in pieces of one page
that do not depend on the other requests (the pages' scales at the time of reading do depend on the
pieces), so a request gets the tokens it would get alone.

    python examples/paged_decode.py [--requests 5] [--tokens 12]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_decode_gemv_block_gb300 as kq  # noqa: E402
from quantized_decode_gemv_block_gb300.inputs import weights_cuda  # noqa: E402

SMALL = dict(n_layers=2, hidden=512, n_q=8, n_kv=2, head_dim=64, ffn=1024, vocab=2000, theta=10000.0, eps=1e-6)


class PagedDecoder:
    """A dense decoder (Q4_K layers, Q8_0 head) and its paged cache for up to `slots` requests."""

    def __init__(self, d=SMALL, slots=8, n_pages=64, page_size=16, max_blocks=16, max_tokens=32, seed=0):
        self.d, self.page_size, self.max_tokens = d, page_size, max_tokens
        h, hd = d["hidden"], d["head_dim"]
        self.q_dim, self.kv_dim = d["n_q"] * hd, d["n_kv"] * hd
        self.shapes = dict(qkv=(self.q_dim + 2 * self.kv_dim, h), o=(h, self.q_dim), gate_up=(2 * d["ffn"], h), down=(h, d["ffn"]))
        tid = 0
        self.layers = []
        for _ in range(d["n_layers"]):
            lay = {}
            for name, (n, k) in self.shapes.items():
                lay[name] = kq.quantize("q4_k", weights_cuda(n, k, seed=seed, tensor_id=tid))
                tid += 1
            self.layers.append(lay)
        self.head = kq.quantize("q8_0", weights_cuda(d["vocab"], h, seed=seed, tensor_id=tid))
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.embed = torch.randn((d["vocab"], h), generator=g, device="cuda")
        pairs = hd // 2
        self.freq = (d["theta"] ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / pairs)).float()
        # pages: one table and one free list for all layers, a cache for each
        self.caches = [kq.KV8Cache(n_pages, page_size, d["n_kv"], hd) for _ in range(d["n_layers"])]
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((slots, max_blocks), -1, **i32)
        self.free = torch.arange(n_pages - 1, -1, -1, **i32)
        self.n_free = torch.tensor([n_pages], **i32)
        self.length = torch.zeros(slots, **i32)  # cached tokens of each slot
        self.lens = [0] * slots                  # the same on the host, which knows what it submitted

    def _norm(self, x):
        # in 64 bits: the order of torch's sums depends on the number of rows
        x = x.double()
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + self.d["eps"])).to(torch.bfloat16)

    def _product(self, lay, name, x):
        n, k = self.shapes[name]
        return kq.gemm("q4_k", lay[name], x.contiguous(), n, k)

    def step(self, new: dict[int, list[int]], logits: bool = False):
        """Runs the new tokens of the slots given; returns {slot: next token}, or {slot: logits} if asked. A step for which
        there are no pages raises RuntimeError and changes nothing."""
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
        x = self.embed[torch.tensor(tokens, device="cuda")]
        for lay, cache in zip(self.layers, self.caches):
            qkv = self._product(lay, "qkv", self._norm(x))
            q = qkv[:, :self.q_dim].unflatten(1, (d["n_q"], -1))
            k = qkv[:, self.q_dim:self.q_dim + self.kv_dim].unflatten(1, (d["n_kv"], -1))
            v = qkv[:, self.q_dim + self.kv_dim:].unflatten(1, (d["n_kv"], -1))
            q, k = kq.rope(q, k, plan.pos, self.freq)
            kq.kv8_append(cache, k, v, plan.slot)
            o = kq.attention_kv8(q, cache, self.table, self.length, new_len, max(counts), max_len, out_dtype=torch.bfloat16)
            x = x + self._product(lay, "o", o.flatten(1))
            gu = self._product(lay, "gate_up", self._norm(x))
            gate, up = gu.chunk(2, -1)
            x = x + self._product(lay, "down", (torch.nn.functional.silu(gate) * up).to(torch.bfloat16))
        self.length += new_len
        self.lens = [a + b for a, b in zip(self.lens, counts)]
        live = [s for s in range(B) if counts[s]]
        last = torch.tensor([sum(counts[:s + 1]) - 1 for s in live], device="cuda")
        hidden = self._norm(x[last])
        if logits:
            y = kq.gemm("q8_0", self.head, hidden, d["vocab"], d["hidden"])
            return {s: y[i] for i, s in enumerate(live)}
        got = []
        for i in range(0, len(live), 16):
            got += kq.head_argmax(self.head, None, hidden[i:i + 16].contiguous(), d["vocab"], d["hidden"], all_rows=True)[0].tolist()
        return dict(zip(live, got))

    def release(self, slots):
        """Gives back the pages of requests that ended."""
        done = torch.zeros(self.table.shape[0], dtype=torch.bool, device="cuda")
        done[torch.tensor(list(slots), device="cuda")] = True
        out = torch.empty_like(self.n_free)
        kq.pages_release(self.length, done, self.table, self.free, self.n_free, out, self.page_size)
        self.n_free = out
        self.length[done] = 0
        for s in slots:
            self.lens[s] = 0


def generate(dec: PagedDecoder, prompts: list[list[int]], tokens: int) -> list[list[int]]:
    """Greedy continuations: requests enter as slots allow, each with a page of its prompt or one token per
    step, or none where the step has no room left for it."""
    out, where, todo, waiting = [[] for _ in prompts], {}, {}, list(range(len(prompts)))
    while waiting or where:
        for s in range(dec.table.shape[0]):
            if waiting and s not in where:
                where[s] = waiting.pop(0)
                todo[s] = list(prompts[where[s]])
        room, new = dec.max_tokens, {}
        for s in sorted(where, key=lambda s: len(todo[s])):  # decoding requests first
            n = min(len(todo[s]), dec.page_size)
            if n <= room:
                new[s] = todo[s][:n]
                room -= n
        got = dec.step(new)
        ended = []
        for s, piece in new.items():
            todo[s] = todo[s][len(piece):]
            if not todo[s]:
                out[where[s]].append(got[s])
                todo[s] = [got[s]]
                if len(out[where[s]]) == tokens:
                    ended.append(s)
        if ended:
            dec.release(ended)
            for s in ended:
                del where[s], todo[s]
    return out


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=5)
    ap.add_argument("--tokens", type=int, default=12)
    a = ap.parse_args()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, SMALL["vocab"], (3 + 17 * i % 41,), generator=g).tolist() for i in range(a.requests)]
    dec = PagedDecoder(slots=4)
    for p, o in zip(prompts, generate(dec, prompts, a.tokens)):
        print(f"prompt of {len(p)} tokens -> {o}")
    print(f"pages free at the end: {dec.n_free.item()}")


if __name__ == "__main__":
    main()
