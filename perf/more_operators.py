"""Measured cases of a mixture-of-experts block over block-quantized weights: norms with the residual, routing, the
plan of the experts' rows, and the experts' products.

A decoder layer with experts runs five operators in a row. `kq.residual_norm` closes the block before (its norm, gate and
residual scale) and norms the sum for the next; `kq.moe_route` chooses k experts for each token from the router's
logits; `kq.moe_plan` sorts the (token, choice) pairs by expert; `kq.moe_gate_up` multiplies each pair's row by its
expert's gate and up matrices and forms silu(g) * u; `kq.moe_down` multiplies by the expert's down matrix and adds a
token's choices up under their weights.

Weights stand in GGUF-style blocks (Q8_0, Q4_K, Q5_K, Q6_K, affine4 in groups of 32), E experts one behind another.

`own = False` computes the operators in plain torch; `own = True` calls this package.
"""
import math
import random

import torch

own = False

F32, BF16 = "f32", "bf16"
_T = {F32: torch.float32, BF16: torch.bfloat16}
_BLOCK = {"q8_0": (32, 34), "q4_k": (256, 144), "q5_k": (256, 176), "q6_k": (256, 210), "affine4": (32, 20)}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # closing an attention block and norming for the experts, eight decoding requests
        dict(name="norm_decode", op="norm", T=8, H=2560, y=F32, h=F32, x=BF16, w=F32, post=True, pre=True, gate="", scale=1.0, off=False),
        # a long prompt under a per-token gate (a modulated block) with a residual scale, weights stored around zero
        dict(name="norm_prompt_gated", op="norm", T=8192, H=4096, y=BF16, h=F32, x=BF16, w=BF16, post=True, pre=True, gate="rows", scale=0.5,
             off=True),
        # a decoding batch's choice of 8 of 128 experts, logits as a bf16 product gives them (equal logits happen)
        dict(name="route_decode", op="route", T=16, E=128, k=8, x=BF16, score="softmax", bias=False, G=1, g=1, group="max", renorm=True, scale=1.0,
             pad=0),
        # a prompt padded to its bucket: balanced sigmoid scores, 4 of 8 groups, 8 of 256 experts; padding tokens' logits are -inf
        dict(name="route_prompt_groups", op="route", T=8192, E=256, k=8, x=F32, score="sigmoid", bias=True, G=8, g=4, group="top2", renorm=True,
             scale=2.5, pad=123),
        # the plan of a decoding batch
        dict(name="plan_decode", op="plan", T=16, E=128, k=8, pad=0),
        # the plan of a padded prompt
        dict(name="plan_prompt", op="plan", T=8192, E=256, k=8, pad=123),
        # one token through 8 of 128 experts
        dict(name="gate_up_single", op="gate_up", fmt="q4_k", T=1, E=128, k=8, H=2048, F=768, pad=0),
        # an uneven decoding batch over fewer and wider experts in 8 bits, three slots of it empty
        dict(name="gate_up_batch_q8", op="gate_up", fmt="q8_0", T=37, E=60, k=4, H=2560, F=1280, pad=3),
        # a prompt
        dict(name="gate_up_prompt", op="gate_up", fmt="q4_k", T=2048, E=128, k=8, H=2048, F=768, pad=0),
        # one token, the down matrices in 6 bits as mixed files keep them
        dict(name="down_single_q6", op="down", fmt="q6_k", T=1, E=128, k=8, H=2048, F=768, add=False, y=F32, pad=0),
        # a decoding batch, added onto the shared expert's output
        dict(name="down_batch", op="down", fmt="q4_k", T=64, E=128, k=8, H=2048, F=768, add=True, y=F32, pad=0),
        # a prompt, bf16 out
        dict(name="down_prompt", op="down", fmt="q4_k", T=2048, E=128, k=8, H=2048, F=768, add=False, y=BF16, pad=0),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["norm", "route", "plan", "gate_up", "gate_up", "down", "down"])
    if op == "norm":
        H = rng.choice([_log(rng, 64, 16384), 8 * _log(rng, 32, 2048), 256 * _log(rng, 1, 64)])
        return dict(op=op, T=_log(rng, 1, min(65536, 23068672 // H)), H=H, y=rng.choice([F32, BF16]), h=rng.choice([F32, BF16]),
                    x=rng.choice([F32, BF16]), w=rng.choice([F32, BF16]), post=rng.random() < 0.5, pre=rng.random() < 0.8,
                    gate=rng.choice(["", "", "one", "rows"]), scale=rng.choice([1.0, 0.25, 1.7]), off=rng.random() < 0.3)
    T, pad = _log(rng, 1, 8192), rng.choice([0, 0, 1])
    if op in ("route", "plan"):
        G = rng.choice([1, 1, 4, 8])
        E = G * rng.choice([4, 8, 15, 16, 32]) if G > 1 else rng.choice([4, 8, 60, 64, 128, 160, 256, 512])
        g = max(1, G // 2)
        k = min(rng.choice([1, 2, 4, 6, 8, 10]), E // G * g)
        d = dict(op=op, T=T, E=E, k=k, pad=min(T - 1, pad * (T // 9 + 1)))
        if op == "plan":
            return d
        return dict(d, x=rng.choice([F32, BF16]), score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, G=G, g=g,
                    group=rng.choice(["max", "top2"]), renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))
    E = rng.choice([8, 16, 60, 64, 128])
    k = min(rng.choice([1, 2, 4, 6, 8]), E // 2)
    H, F = 256 * _log(rng, 2, 16), 256 * _log(rng, 1, 8)
    fmt = rng.choice(["q4_k", "q4_k", "q4_k", "q8_0", "q5_k", "q6_k", "affine4"])
    while E * H * F > (201326592 if fmt == "q4_k" else 134217728):  # 128 x 2048 x 768
        H, F = max(256, H // 512 * 256), max(256, F // 512 * 256)
    T = min(T, max(1, 25769803776 // (k * H * F)))  # 2048 x 8 x 2048 x 768
    d = dict(op=op, fmt=fmt, T=T, E=E, k=k, H=H, F=F, pad=min(T - 1, pad * (T // 9 + 1)))
    return d if op == "gate_up" else dict(d, add=rng.random() < 0.5, y=rng.choice([F32, F32, BF16]))


# ---------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _randint(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.uint8 if hi <= 256 else torch.int32)


def _half(v):
    """fp32 [...] -> its fp16 bytes [..., 2]."""
    return v.half().unsqueeze(-1).view(torch.uint8)


def _weights(g, fmt, E, N, K):
    """Blocks of E x N rows of K weights: codes over their whole range, scales that make weights of about N(0, 0.02)."""
    n, size = _BLOCK[fmt]
    shape = (E * N, K // n)
    u = 0.7 + 0.7 * torch.rand(shape, generator=g, device="cuda")
    if fmt == "q8_0":
        parts = [_half(u * (0.02 / 74)), _randint(g, 0, 256, *shape, 32)]
    elif fmt == "affine4":
        parts = [_half(u * (0.02 / 4.6)), _half(u * (-0.02 / 4.6 * 7.5)), _randint(g, 0, 256, *shape, 16)]
    elif fmt == "q6_k":
        scales = torch.randint(-96, 97, (*shape, 16), generator=g, device="cuda", dtype=torch.int8).view(torch.uint8)
        parts = [_randint(g, 0, 256, *shape, 192), scales, _half(u * (0.02 / 1030))]
    else:  # a sub-block's min is about half its codes' range below zero
        top = 15.0 if fmt == "q4_k" else 31.0
        sc = _randint(g, 24, 64, *shape, 8)
        m = (sc.to(torch.int16) + _randint(g, 0, 5, *shape, 8).to(torch.int16) - 2).clamp_(0, 63).to(torch.uint8)
        lo = sc[..., :4] | (sc[..., 4:] >> 4 << 6)
        hi = m[..., :4] | (m[..., 4:] >> 4 << 6)
        rest = (sc[..., 4:] & 15) | ((m[..., 4:] & 15) << 4)
        d = u * (0.02 / (44 * top * 0.3))
        parts = [_half(d), _half(d * top / 2), lo, hi, rest, _randint(g, 0, 256, *shape, 128 if fmt == "q4_k" else 160)]
    w = torch.cat(parts, -1)
    assert w.shape[-1] == size
    return w.view(E, N, K // n * size)


def _ids(case, g):
    """Distinct experts of every token, some more popular than others; -1 for padding tokens."""
    T, E, k = case["T"], case["E"], case["k"]
    z = _randn(g, T, E) + 0.4 * _randn(g, E)
    ids = torch.sort(z, dim=-1, descending=True).indices[:, :k].to(torch.int32)
    ids[T - case["pad"]:] = -1
    return ids.contiguous()


def _plan(ids, E):
    flat = ids.flatten().long()
    key = torch.where(flat < 0, E, flat)
    n = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat((n.new_zeros(1), torch.cumsum(n, 0)))
    order = torch.sort(key, dim=0, stable=True).indices
    order = torch.where(torch.arange(order.numel(), device="cuda") < offsets[-1], order, -1)
    return offsets.to(torch.int32), order.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 29)
    st = dict(case=case)
    op, T = case["op"], case["T"]
    if op == "norm":
        H = case["H"]
        st["y"], st["h"] = (3 * _randn(g, T, H)).to(_T[case["y"]]), _randn(g, T, H).to(_T[case["h"]])
        if case["gate"]:
            st["gate"] = (_randn(g, *((H,) if case["gate"] == "one" else (T, H)))).to(_T[case["y"]])
        mid = 0.0 if case["off"] else 1.0
        st["post"], st["pre"] = ((mid + 0.2 * _randn(g, H)).to(_T[case["w"]]) if case[n] else None for n in ("post", "pre"))
        return st
    E, k = case["E"], case["k"]
    if op == "route":
        x = 1.5 * _randn(g, T, E) + 0.5 * _randn(g, E)
        x[T - case["pad"]:] = -math.inf
        st["logits"] = x.to(_T[case["x"]])
        st["bias"] = 0.1 * _randn(g, E) if case["bias"] else None
        return st
    st["ids"] = _ids(case, g)
    if op == "plan":
        return st
    H, F = case["H"], case["F"]
    st["offsets"], st["order"] = _plan(st["ids"], E)
    n = st["offsets"].diff()
    st["live"] = n.nonzero().flatten()  # the experts that have rows, for the plain form alone
    st["most"], st["rows"] = int(n.max()), int(st["offsets"][-1])
    if op == "gate_up":
        st["w"] = _weights(g, case["fmt"], E, 2 * F, H)
        st["x"] = _randn(g, T, H).to(torch.bfloat16)
        st["act"] = torch.zeros((T * k, F), dtype=torch.bfloat16, device="cuda")  # padding tokens' rows stay as they are
    else:
        st["w"] = _weights(g, case["fmt"], E, H, F)
        z = _randn(g, T * k, F)
        st["act"] = (z * torch.sigmoid(z) * _randn(g, T * k, F)).to(torch.bfloat16)
        p = torch.softmax(_randn(g, T, k), -1)
        st["weights"] = torch.where(st["ids"] < 0, 0, p).contiguous()
        st["add"] = _randn(g, T, H) if case["add"] else None
    if own:
        import quantized_decode_gemv_block_gb300 as kq
        st["plan"] = kq.MoePlan(st["offsets"], st["order"])
        size = kq.moe_gate_up_workspace_size if op == "gate_up" else kq.moe_down_workspace_size
        n = size(case["fmt"], T, k, E, *((F, H) if op == "gate_up" else (H, F)))
        st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- plain forms

def _rms(v, w, off):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * (w.float() + 1 if off else w.float())


def _norm_plain(st):
    c = st["case"]
    z = st["y"].float()
    if c["post"]:
        z = _rms(z, st["post"], c["off"])
    if c["gate"]:
        z = z * st["gate"].float()
    h = st["h"].float() + c["scale"] * z
    return {"h": h.to(_T[c["h"]]), "x": _rms(h, st["pre"], c["off"]).to(_T[c["x"]]) if c["pre"] else None}


def _route_plain(st):
    """Scores and choices in 64 bits: near a border 32 would choose another expert."""
    c, x = st["case"], st["logits"].double()
    T, E, G, k = c["T"], c["E"], c["G"], c["k"]
    off = torch.isneginf(x)  # an expert that cannot be chosen
    if c["score"] == "softmax":
        top = x.amax(-1, keepdim=True).nan_to_num(neginf=0.0)
        s = torch.exp(x - top)
        s = s / s.sum(-1, keepdim=True).clamp(min=1e-300)
    else:
        s = 1 / (1 + torch.exp(-x))
    choice = (s + st["bias"].double() if c["bias"] else s).masked_fill(off, -math.inf)
    if G > 1:
        best = torch.sort(choice.view(T, G, E // G), dim=-1, descending=True).values
        two = best[..., 0] + torch.where(torch.isneginf(best[..., 1]), 0, best[..., 1]) if c["group"] == "top2" else best[..., 0]
        kept = torch.sort(two, dim=-1, descending=True, stable=True).indices[:, :c["g"]]
        out = torch.ones((T, G), dtype=torch.bool, device="cuda").scatter_(1, kept, False)
        choice = choice.masked_fill(out[:, :, None].expand(T, G, E // G).reshape(T, E), -math.inf)
    got = torch.sort(choice, dim=-1, descending=True, stable=True)
    none = torch.isneginf(got.values[:, :k])
    ids = got.indices[:, :k]
    p = s.gather(1, ids).masked_fill(none, 0)
    if c["renorm"]:
        p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
    return {"ids": ids.masked_fill(none, -1).to(torch.int32), "weights": (p * c["scale"]).float()}


def _plan_plain(st):
    offsets, order = _plan(st["ids"], st["case"]["E"])
    return {"offsets": offsets, "order": order}


def _f16(b):
    return b.contiguous().view(torch.float16).float()


def _plain_weights(fmt, w):
    """Blocks [..., bytes of a row] -> fp32 weights [..., K]."""
    n, size = _BLOCK[fmt]
    b = w.unflatten(-1, (-1, size))
    if fmt == "q8_0":
        v = _f16(b[..., :2]) * b[..., 2:].view(torch.int8).float()
    elif fmt == "affine4":
        q = torch.stack((b[..., 4:] & 15, b[..., 4:] >> 4), -1).flatten(-2).float()
        v = _f16(b[..., :2]) * q + _f16(b[..., 2:4])
    elif fmt == "q6_k":
        ql, qh = b[..., :128].unflatten(-1, (2, 1, 2, 32)), b[..., 128:192].unflatten(-1, (2, 1, 32))  # half, -, column, byte
        low = torch.cat((ql & 15, ql >> 4), -3).flatten(-3, -2)  # [..., 2, 4, 32]
        top = torch.cat((qh & 3, qh >> 2 & 3, qh >> 4 & 3, qh >> 6), -2)
        q = (low | top << 4).float().sub_(32).flatten(-3).unflatten(-1, (16, 16))
        v = (_f16(b[..., 208:]) * b[..., 192:208].view(torch.int8).float()).unsqueeze(-1).mul(q).flatten(-2)
    else:
        s0, s1, s2 = b[..., 4:8], b[..., 8:12], b[..., 12:16]
        sc = torch.cat((s0 & 63, s2 & 15 | s0 >> 6 << 4), -1).float()
        m = torch.cat((s1 & 63, s2 >> 4 | s1 >> 6 << 4), -1).float()
        qs = b[..., -128:].unflatten(-1, (4, 1, 32))
        q = torch.cat((qs & 15, qs >> 4), -2).flatten(-3, -2)  # [..., 8, 32]
        if fmt == "q5_k":
            bit = torch.arange(8, dtype=torch.uint8, device=b.device)[:, None]
            q = q | (b[..., 16:48].unsqueeze(-2) >> bit & 1) << 4
        v = (_f16(b[..., :2]) * sc).unsqueeze(-1) * q.float() - (_f16(b[..., 2:4]) * m).unsqueeze(-1)
        v = v.flatten(-2)
    return v.flatten(-2)


def _products_plain(st, rows):
    """Each pair's row (fp32, in the order of the plan) times its expert's matrix: the rows of an expert padded to the most that one has."""
    r = torch.arange(st["rows"], device="cuda")
    ends = st["offsets"][st["live"] + 1].long()
    e = torch.searchsorted(ends, r, right=True)
    at = r - st["offsets"].long()[st["live"]][e]
    x = torch.zeros((len(ends), st["most"], rows.shape[1]), device="cuda")
    x[e, at] = rows
    return torch.bmm(x, _plain_weights(st["case"]["fmt"], st["w"][st["live"]]).transpose(1, 2))[e, at]


def _gate_up_plain(st):
    pair = st["order"][:st["rows"]].long()
    y = _products_plain(st, st["x"].float()[pair // st["case"]["k"]])
    g, u = y.chunk(2, -1)
    st["act"][pair] = (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)
    return st["act"]


def _down_plain(st):
    c = st["case"]
    pair = st["order"][:st["rows"]].long()
    y = torch.zeros((c["T"] * c["k"], c["H"]), device="cuda")
    y[pair] = _products_plain(st, st["act"].float()[pair])
    y = (y.view(c["T"], c["k"], c["H"]) * st["weights"][..., None]).sum(1)
    return (y + st["add"] if c["add"] else y).to(_T[c["y"]])


# ---------------------------------------------------------------- one pass

def run(state):
    st, c = state, state["case"]
    if not own:
        return {"norm": _norm_plain, "route": _route_plain, "plan": _plan_plain, "gate_up": _gate_up_plain, "down": _down_plain}[c["op"]](st)
    import quantized_decode_gemv_block_gb300 as kq
    if c["op"] == "norm":
        h, x = kq.residual_norm(st["h"], st["y"], post=st["post"], gate=st.get("gate"), scale=c["scale"], pre=st["pre"], eps=1e-6,
                                unit_offset=c["off"], x_dtype=_T[c["x"]])
        return {"h": h, "x": x}
    if c["op"] == "route":
        ids, weights = kq.moe_route(st["logits"], c["k"], score=c["score"], bias=st["bias"], n_group=c["G"], top_group=c["g"],
                                    group_score=c["group"], renorm=c["renorm"], scale=c["scale"])
        return {"ids": ids, "weights": weights}
    if c["op"] == "plan":
        plan = kq.moe_plan(st["ids"], c["E"])
        return {"offsets": plan.offsets, "order": plan.order}
    if c["op"] == "gate_up":
        return kq.moe_gate_up(c["fmt"], st["w"], st["x"], st["plan"], c["F"], c["H"], act=st["act"], workspace=st["ws"])
    return kq.moe_down(c["fmt"], st["w"], st["act"], st["plan"], st["ids"], st["weights"], c["H"], c["F"], add=st["add"], out_dtype=_T[c["y"]],
                       workspace=st["ws"])


def work(case):
    op, T = case["op"], case["T"]
    b = {F32: 4, BF16: 2}
    if op == "norm":
        H, rows = case["H"], 1 if case["gate"] == "one" else T
        n = T * H * (b[case["y"]] + 2 * b[case["h"]] + (b[case["x"]] if case["pre"] else 0))
        n += (rows * H * b[case["y"]] if case["gate"] else 0) + H * b[case["w"]] * (case["post"] + case["pre"])
        return {"bytes": n, "flops": T * H * (3 + 4 * case["post"] + 4 * case["pre"])}
    E, k = case["E"], case["k"]
    if op == "route":
        return {"bytes": T * E * b[case["x"]] + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 4 * T * E}
    if op == "plan":
        return {"bytes": 8 * T * k + 4 * (E + 1), "flops": 0}
    H, F, live = case["H"], case["F"], T - case["pad"]
    n, size = _BLOCK[case["fmt"]]
    used = E * (1 - (1 - k / E) ** live)  # experts that have a row, on average
    blocks = used * H * F * (2 if op == "gate_up" else 1) * size / n
    if op == "gate_up":
        return {"bytes": int(blocks) + 2 * live * (H + k * F) + 4 * (live * k + E + 1), "flops": 4 * live * k * H * F}
    y = T * H * (b[case["y"]] + (4 if case["add"] else 0))
    return {"bytes": int(blocks) + 2 * live * k * F + y + 4 * (live * k + E + 1) + 8 * T * k, "flops": 2 * live * k * H * F}


# ---------------------------------------------------------------- in 64 bits, from the definitions

def _exact_norm(st, c):
    def rms(v, w):
        return v / torch.sqrt(torch.einsum("th,th->t", v, v) / c["H"] + 1e-6)[:, None] * (w.double() + (1.0 if c["off"] else 0.0))
    z = rms(st["y"].double(), st["post"]) if c["post"] else st["y"].double()
    h = st["h"].double() + c["scale"] * (z * st["gate"].double() if c["gate"] else z)
    return {"h": h, "x": rms(h, st["pre"]) if c["pre"] else None}


def _exact_route(st, c):
    """Token by token over the chosen experts' weights; the choices are whole numbers."""
    x = st["logits"].double()
    s = torch.softmax(x, -1).nan_to_num(0.0) if c["score"] == "softmax" else torch.sigmoid(x)
    ids = _route_plain(st)["ids"].long()
    p = torch.stack([torch.where(ids[:, j] < 0, 0, s[torch.arange(c["T"], device="cuda"), ids[:, j].clamp(min=0)]) for j in range(c["k"])], 1)
    if c["renorm"]:
        p = p / torch.where(p.sum(1) > 0, p.sum(1), 1)[:, None]
    return {"ids": None, "weights": p * c["scale"]}


def _exact_weights(fmt, w):
    """One expert's blocks [N, bytes] -> [N, K] in 64 bits, weight by weight of a block."""
    n, size = _BLOCK[fmt]
    b = w.view(w.shape[0], -1, size)
    i = torch.arange(n, device="cuda")
    f16 = lambda at: b[..., at:at + 2].contiguous().view(torch.float16).double()  # noqa: E731
    if fmt == "q8_0":
        v = b[..., 2 + i].view(torch.int8).double() * f16(0)
    elif fmt == "affine4":
        v = (b[..., 4 + i // 2].long() >> 4 * (i % 2) & 15).double() * f16(0) + f16(2)
    elif fmt == "q6_k":
        half, q, l = i // 128, i % 128 // 32, i % 32
        low = b[..., 64 * half + 32 * (q % 2) + l].long() >> 4 * (q // 2) & 15
        high = b[..., 128 + 32 * half + l].long() >> 2 * q & 3
        v = (low + 16 * high - 32).double() * b[..., 192 + i // 16].view(torch.int8).double() * f16(208)
    else:
        j, l = i // 32, i % 32
        a, z = b[..., 4 + j % 4].long(), b[..., 8 + j % 4].long()
        r = b[..., 12 + j % 4].long()
        sc = torch.where(j < 4, a & 63, r & 15 | a >> 6 << 4)
        m = torch.where(j < 4, z & 63, r >> 4 | z >> 6 << 4)
        q = b[..., size - 128 + 32 * (j // 2) + l].long() >> 4 * (j % 2) & 15
        if fmt == "q5_k":
            q = q + 16 * (b[..., 16 + l].long() >> j & 1)
        v = f16(0) * (sc * q).double() - f16(2) * m.double()
    return v.flatten(1)


def _exact_products(st, c):
    k, F = c["k"], c["F"]
    y = torch.zeros((c["T"] * k, 2 * F if c["op"] == "gate_up" else c["H"]), dtype=torch.float64, device="cuda")
    ends = st["offsets"].tolist()
    for e in range(c["E"]):
        if ends[e + 1] > ends[e]:
            pair = st["order"][ends[e]:ends[e + 1]].long()
            rows = st["x"][pair // k] if c["op"] == "gate_up" else st["act"][pair]
            y[pair] = torch.einsum("pk,nk->pn", rows.double(), _exact_weights(c["fmt"], st["w"][e]))
    if c["op"] == "gate_up":
        return torch.nn.functional.silu(y[:, :F]) * y[:, F:]
    out = torch.einsum("tkh,tk->th", y.view(c["T"], k, c["H"]), st["weights"].double())
    return out + st["add"].double() if c["add"] else out


def exact(case, seed):
    if case["op"] == "plan":  # whole numbers only: nothing is rounded
        return None
    st = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "gate_up": _exact_products, "down": _exact_products}[case["op"]](st, case)
