"""Measured cases of the paged 8-bit KV cache: page planning, rotary positions, cache append, attention.

A serving step over a paged cache runs four operators in a row. `kq.pages_plan` turns the
requests' lengths into block-table entries and one cache slot per new token; `kq.rope`
rotates q and k by positions of one or more axes; `kq.kv8_append` quantizes the new k and v
into the cache's pages; `kq.attention_kv8` attends over those pages.

The cache holds int8 codes c and one fp32 scale s for each (page, kv head), a power of two (or
0 while every value is 0); an element stands for (c + 1/2) s. A value x is coded as
floor(x / s) with s = 2^(floor(log2 max|x|) - 6) over the page's tokens, so that a page whose
scale grows is recoded by floor(c * s_old / s_new) to exactly what coding all of its tokens at
once gives. Codes are integers that follow exactly from the inputs.

Within a (page, kv head) the codes are stored in groups of 16 tokens, each in the order in which
a warp's matrix operands take them (see _k_plain and _v_plain, which undo it).

`own = False` computes the operators in plain torch; `own = True` calls this package.
"""
import math
import random

import torch

own = False

F32, BF16 = "f32", "bf16"
_T = {F32: torch.float32, BF16: torch.bfloat16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # rotary: eight decoding requests, one token each, far positions of one axis
        dict(name="rope_decode", op="rope", T=8, n_q=32, n_kv=8, D=128, rot=128, axes=1, adjacent=False,
             inverse=False, fused=False, x=BF16, y=BF16, far=1000000),
        # rotary straight from a qkv product's fp32 rows, an odd number of image and text tokens, half of each head rotated
        dict(name="rope_image_fused", op="rope", T=1999, n_q=16, n_kv=4, D=64, rot=32, axes=3, adjacent=False,
             inverse=False, fused=True, x=F32, y=BF16, far=20000),
        # the gradient of a long prompt's rotation (the inverse rotation), adjacent pairs, video positions
        dict(name="rope_prompt_gradient", op="rope", T=32768, n_q=32, n_kv=8, D=128, rot=128, axes=3, adjacent=True,
             inverse=True, fused=False, x=BF16, y=BF16, far=32768),
        # pages and slots of a decode step
        dict(name="pages_decode", op="pages", B=64, lens=11, ctx_lo=1, ctx_hi=8192, new_lo=1, new_hi=1, P=32, pad=0),
        # a server's whole queue: prompts, verify windows and idle requests, padded to a fixed token count
        dict(name="pages_queue", op="pages", B=4096, lens=12, ctx_lo=0, ctx_hi=4000, new_lo=0, new_hi=255, P=16, pad=777),
        # cache append of one token per request
        dict(name="append_decode", op="append", B=64, lens=13, ctx_lo=1, ctx_hi=4096, new_lo=1, new_hi=1, P=32,
             n_kv=8, D=128, x=BF16),
        # verify windows of uneven length, fp32 k and v as a qkv product gives them
        dict(name="append_verify", op="append", B=24, lens=14, ctx_lo=1, ctx_hi=2000, new_lo=1, new_hi=16, P=16,
             n_kv=4, D=64, x=F32),
        # long prompts filling fresh pages
        dict(name="append_prompt", op="append", B=8, lens=15, ctx_lo=0, ctx_hi=100, new_lo=3001, new_hi=4097, P=64,
             n_kv=8, D=128, x=BF16),
        # one request, one token, 4096 positions, 16 query heads on 4 kv heads
        dict(name="attn_single", op="attn", B=1, lens=16, ctx_lo=4095, ctx_hi=4095, new_lo=1, new_hi=1, P=32, n_q=16,
             n_kv=4, D=128, x=F32, y=BF16, tree=False),
        # verify windows with tree masks, fp32 in and out
        dict(name="attn_verify_tree", op="attn", B=16, lens=17, ctx_lo=1000, ctx_hi=9000, new_lo=5, new_hi=8, P=16,
             n_q=16, n_kv=4, D=64, x=F32, y=F32, tree=True),
        # a decoding batch of uneven context lengths
        dict(name="attn_batch", op="attn", B=64, lens=18, ctx_lo=1, ctx_hi=8191, new_lo=1, new_hi=1, P=32, n_q=32,
             n_kv=8, D=128, x=BF16, y=BF16, tree=False),
        # few requests with very long contexts
        dict(name="attn_long", op="attn", B=4, lens=19, ctx_lo=125001, ctx_hi=131071, new_lo=1, new_hi=1, P=64, n_q=32,
             n_kv=8, D=128, x=BF16, y=BF16, tree=False),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["rope", "pages", "append", "attn", "attn"])
    if op == "rope":
        n_kv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 96, 128, 256])
        n_q = n_kv * rng.choice([1, 2, 4, 8])
        T = _log(rng, 1, max(2, 167772160 // (max(40, n_q + 2 * n_kv) * max(D, 128)) // 2))
        return dict(op=op, T=T, n_q=n_q, n_kv=n_kv, D=D, rot=rng.choice([D, D // 2, D // 4]), axes=rng.choice([1, 2, 3]),
                    adjacent=rng.random() < 0.4, inverse=rng.random() < 0.3, fused=rng.random() < 0.4,
                    x=rng.choice([F32, BF16]), y=rng.choice([F32, BF16]), far=_log(rng, 1, 1 << 24))
    P = rng.choice([16, 32, 64, 128])
    if op == "pages":
        lo, hi = _log(rng, 1, 4000), _log(rng, 1, 255)
        return dict(op=op, B=_log(rng, 1, 4096), lens=rng.randrange(1 << 30), ctx_lo=rng.choice([0, lo // 2]), ctx_hi=lo,
                    new_lo=rng.choice([0, 1]), new_hi=hi, P=P, pad=rng.choice([0, 1, 777]))
    if op == "append":
        B, hi = _log(rng, 1, 64), _log(rng, 1, 4000)
        B = max(1, min(B, 30000 // hi))
        c = _log(rng, 1, 4096)
        return dict(op=op, B=B, lens=rng.randrange(1 << 30), ctx_lo=rng.choice([0, c // 2]), ctx_hi=c, new_lo=max(1, hi // 2),
                    new_hi=hi, P=P, n_kv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]), x=rng.choice([F32, BF16]))
    n_kv, D, new = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([1, 1, _log(rng, 2, 32), _log(rng, 33, 512)])
    n_q, B = n_kv * rng.choice([1, 2, 4, 5, 8]), _log(rng, 1, 64)
    c = _log(rng, 1, max(1, min(131072, 200000000 // (B * n_kv * D), 100000000 // (B * n_q * new) + 1)))
    return dict(op=op, B=B, lens=rng.randrange(1 << 30), ctx_lo=c // 2, ctx_hi=c, new_lo=max(1, new // 2), new_hi=new, P=P, n_q=n_q,
                n_kv=n_kv, D=D, x=rng.choice([F32, BF16]), y=rng.choice([F32, BF16, BF16]), tree=new <= 32 and rng.random() < 0.3)


def _lens(case):
    r = random.Random(case["lens"])
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    return ctx, new


def _blocks(n, P):
    return -(-n // P)


# ---------------------------------------------------------------- inputs

def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _codes(g, pages, n_kv, P, D):
    """Codes of pages that hold values of about N(0, 1), and their scales."""
    c = torch.empty((pages, n_kv, P * D), dtype=torch.int8, device="cuda")
    s = torch.tensor([1 / 64, 1 / 32, 1 / 16], device="cuda")[torch.randint(0, 3, (pages, n_kv), generator=g, device="cuda")]
    step = max(1, (1 << 26) // (n_kv * P * D))
    for i in range(0, pages, step):
        x = _randn(g, min(step, pages - i), n_kv, P * D)
        c[i:i + step] = torch.floor(x / s[i:i + step, :, None]).clamp_(-128, 127).to(torch.int8)
    return c, s


def _paged(case, g, extra):
    """Context and new lengths, and a block table of scattered pages for all of their positions."""
    ctx, new = _lens(case)
    nb = [_blocks(c + n, case["P"]) for c, n in zip(ctx, new)]
    pages = sum(nb) + extra
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    width = max(max(nb), 1)
    table = torch.zeros((case["B"], width), dtype=torch.int32, device="cuda")
    used = torch.arange(width, device="cuda")[None, :] < _ints(nb)[:, None]
    table[used] = perm[:sum(nb)]
    return ctx, new, pages, perm, table


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)
    st = dict(case=case)
    op = case["op"]
    if op == "rope":
        T, D, H = case["T"], case["D"], case["n_q"] + case["n_kv"]
        if case["fused"]:  # q | k | v rows of one product
            rows = _randn(g, T, (H + case["n_kv"]) * D).to(_T[case["x"]])
            st["q"] = rows[:, :case["n_q"] * D].view(T, case["n_q"], D)
            st["k"] = rows[:, case["n_q"] * D:H * D].view(T, case["n_kv"], D)
        else:
            st["q"] = _randn(g, T, case["n_q"], D).to(_T[case["x"]])
            st["k"] = _randn(g, T, case["n_kv"], D).to(_T[case["x"]])
        pairs = case["rot"] // 2
        start = torch.randint(0, case["far"] + 1, (case["axes"], 1), generator=g, device="cuda")
        step = torch.randint(0, 3, (case["axes"], T), generator=g, device="cuda")
        st["pos"] = (start + step.cumsum(1)).to(torch.int32)
        st["freq"] = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / pairs)).float()
        st["axis"] = (torch.arange(pairs, device="cuda") * case["axes"] // pairs).to(torch.uint8)
        return st
    if op == "pages":
        ctx, new = _lens(case)
        P = case["P"]
        width = max(_blocks(c + n, P) for c, n in zip(ctx, new)) + 1
        held = [_blocks(c, P) for c in ctx]
        need = sum(_blocks(c + n, P) for c, n in zip(ctx, new))
        perm = torch.randperm(need + 5, generator=g, device="cuda").to(torch.int32)
        st["table"] = torch.full((case["B"], width), -1, dtype=torch.int32, device="cuda")
        st["table"][torch.arange(width, device="cuda")[None, :] < _ints(held)[:, None]] = perm[:sum(held)]
        st["ctx"], st["new"] = _ints(ctx), _ints(new)
        st["free"] = torch.zeros(need + 5, dtype=torch.int32, device="cuda")
        st["free"][:need + 5 - sum(held)] = perm[sum(held):]
        st["n_free"] = _ints([need + 5 - sum(held)])
        st["T"] = sum(new) + case["pad"]
        return st
    ctx, new, pages, perm, table = _paged(case, g, 3)
    P, D, n_kv, T = case["P"], case["D"], case["n_kv"], sum(new)
    st["kc"], st["ks"] = _codes(g, pages, n_kv, P, D)
    st["vc"], st["vs"] = _codes(g, pages, n_kv, P, D)
    st["new"], st["ctx"], st["table"] = _ints(new), _ints(ctx), table
    req = torch.repeat_interleave(torch.arange(case["B"], device="cuda"), st["new"].long())
    cu = torch.cumsum(st["new"].long(), 0) - st["new"]
    pos = st["ctx"].long()[req] + torch.arange(T, device="cuda") - cu[req]
    if op == "append":
        st["slot"] = (table[req, pos // P] * P + pos % P).to(torch.int32)
        st["first"] = cu
        st["k"] = (_randn(g, T, n_kv, D) * torch.exp(0.7 * _randn(g, T, n_kv, 1))).to(_T[case["x"]])
        st["v"] = (_randn(g, T, n_kv, D) * torch.exp(0.7 * _randn(g, T, n_kv, 1))).to(_T[case["x"]])
    else:
        st["q"] = _randn(g, T, case["n_q"], D).to(_T[case["x"]])
        st["max_new"], st["max_len"], st["total_len"] = max(new), max(c + n for c, n in zip(ctx, new)), sum(ctx) + T
        if case["tree"]:
            w = torch.randint(0, 1 << 31, (T,), generator=g, device="cuda")
            own_bit = (torch.arange(T, device="cuda") - cu[req])
            st["mask"] = ((w | (1 << own_bit)) & ((2 << own_bit) - 1)).to(torch.int32)
    if own:
        import quantized_decode_gemv_block_gb300 as kq
        st["cache"] = kq.KV8Cache(pages, P, n_kv, D, k=st["kc"], v=st["vc"], k_scale=st["ks"], v_scale=st["vs"])
        if op == "attn":
            n = kq.attention_kv8_workspace_size(case["B"], st["total_len"], st["max_new"], case["n_q"], n_kv, D)
            st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- plain forms

def _rope_plain(st):
    c = st["case"]
    h = c["rot"] // 2
    ang = st["pos"].double()[st["axis"].long()].T * st["freq"].double()  # [T, pairs]
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    if c["inverse"]:
        sin = -sin
    out = []
    for x in (st["q"], st["k"]):
        x = x.float()
        a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if c["adjacent"] else (x[..., :h], x[..., h:2 * h])
        ra, rb = a * cos - b * sin, b * cos + a * sin
        r = torch.stack((ra, rb), -1).flatten(-2) if c["adjacent"] else torch.cat((ra, rb), -1)
        out.append(torch.cat((r, x[..., 2 * h:]), -1).to(_T[c["y"]]))
    return {"q": out[0], "k": out[1]}


def _pages_plain(st):
    P, T, B = st["case"]["P"], st["T"], st["case"]["B"]
    ctx, new, table = st["ctx"].long(), st["new"].long(), st["table"]
    have, want = (ctx + P - 1) // P, (ctx + new + P - 1) // P
    ends = torch.cumsum(want - have, 0)
    first = ends - (want - have)
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    fresh = (col >= have[:, None]) & (col < want[:, None])
    at = st["n_free"].long() - 1 - first[:, None] - (col - have[:, None])  # popped from the end of the free list
    table = torch.where(fresh, st["free"][at.clamp(0, st["free"].shape[0] - 1)], table)
    st["table"].copy_(table)
    cu = torch.cat((new.new_zeros(1), torch.cumsum(new, 0)))
    t = torch.arange(T, device="cuda")
    req = torch.searchsorted(cu, t, right=True) - 1
    live = req < B
    req = req.clamp(max=B - 1)
    pos = torch.where(live, ctx[req] + t - cu[req], 0)
    slot = torch.where(live, table[req, pos // P].long() * P + pos % P, -1)
    return {"table": st["table"], "cu": cu.to(torch.int32), "pos": pos.to(torch.int32), "slot": slot.to(torch.int32),
            "n_free": (st["n_free"] - ends[-1]).to(torch.int32)}


def _k_offsets(D):
    """Place of (token, dim) in a group of 16 tokens' K codes."""
    p, d = torch.arange(16, device="cuda")[:, None], torch.arange(D, device="cuda")[None, :]
    return d // 32 * 512 + (p // 4 * 2 + p % 2) * 64 + d // 4 % 4 * 16 + d // 16 % 2 * 8 + p // 2 % 2 * 4 + d % 4


def _v_offsets(D):
    p, d = torch.arange(16, device="cuda")[:, None], torch.arange(D, device="cuda")[None, :]
    return d // 32 * 512 + d % 8 * 64 + p // 4 * 16 + d // 16 % 2 * 8 + d // 8 % 2 * 4 + p % 4


def _append_plain(st):
    P, n_kv, D = st["case"]["P"], st["case"]["n_kv"], st["case"]["D"]
    slot = st["slot"].long()
    page, at = slot // P, slot % P
    head = torch.arange(n_kv, device="cuda")
    first = st["first"]
    for x, codes, scale, offs in ((st["k"], st["kc"], st["ks"], _k_offsets(D)), (st["v"], st["vc"], st["vs"], _v_offsets(D))):
        x = x.float()
        top = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")
        need = torch.where(top > 0, (torch.frexp(top).exponent + 120 << 23).view(torch.float32), 0)  # 2^(exponent - 7)
        old = scale[page[first]] * (at[first] > 0)[:, None]  # a page that starts here holds nothing yet
        grown = torch.maximum(old, need[page[first]])
        keep = torch.floor(codes[page[first]].float() * (old / torch.where(grown > 0, grown, 1))[..., None]).to(torch.int8)
        held = torch.where((at[first] > 0)[:, None, None], keep, codes[page[first]])
        codes[page[first]] = held
        now = scale.index_copy(0, page, need[page]).index_copy_(0, page[first], grown)
        scale.copy_(now)
        s = now[page]
        c = torch.where(s[..., None] > 0, torch.floor(x / torch.where(s > 0, s, 1)[..., None]), 0).to(torch.int8)
        flat = (page[:, None] * n_kv + head)[..., None] * (P * D) + (at // 16 * 16 * D)[:, None, None] + offs[at % 16][:, None, :]
        codes.view(-1)[flat.view(-1)] = c.view(-1)
    return {"k": st["kc"], "v": st["vc"], "k_scale": st["ks"], "v_scale": st["vs"]}


def _k_plain(c, P, D):
    """Codes [..., P*D] as stored -> [..., P, D]."""
    c = c.unflatten(-1, (P // 16, D // 32, 4, 2, 4, 2, 2, 4))  # group, d/32, p/4, p%2, d/4%4, d/16%2, p/2%2, d%4
    n = c.dim() - 8
    return c.permute(*range(n), n, n + 2, n + 6, n + 3, n + 1, n + 5, n + 4, n + 7).flatten(-8, -5).flatten(-4)


def _v_plain(c, P, D):
    c = c.unflatten(-1, (P // 16, D // 32, 8, 4, 2, 2, 4))  # group, d/32, d%8, p/4, d/16%2, d/8%2, p%4
    n = c.dim() - 7
    return c.permute(*range(n), n, n + 3, n + 6, n + 1, n + 4, n + 5, n + 2).flatten(-7, -5).flatten(-4)


def _attn_plain(st):
    c = st["case"]
    P, D, n_kv, B, L, M = c["P"], c["D"], c["n_kv"], c["B"], st["max_len"], st["max_new"]
    grp, T = c["n_q"] // n_kv, st["q"].shape[0]
    table = st["table"].long()
    nb = table.shape[1]
    kv = []
    for codes, scale, plain in ((st["kc"], st["ks"], _k_plain), (st["vc"], st["vs"], _v_plain)):
        x = plain(codes[table], P, D).float().add_(0.5).mul_(scale[table][..., None, None])  # [B, nb, n_kv, P, D]
        kv.append(x.transpose(1, 2).reshape(B, n_kv, nb * P, D)[:, :, :L])
    k, v = kv
    ctx, new = st["ctx"].long(), st["new"].long()
    cu = torch.cumsum(new, 0) - new
    i = torch.arange(M, device="cuda")
    tok = (cu[:, None] + i).clamp(max=T - 1)  # [B, M]
    q = st["q"].float()[tok].view(B, M, n_kv, grp, D).permute(0, 2, 1, 3, 4).reshape(B, n_kv, M * grp, D)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(1 / math.sqrt(D)).view(B, n_kv, M, grp, L)
    p = torch.arange(L, device="cuda")
    j = p[None, :] - ctx[:, None]  # index within the window of new tokens
    see = (j < 0)[:, None, :] | (j[:, None, :] <= i[None, :, None])
    if "mask" in st:
        bit = (st["mask"].long()[tok][:, :, None] >> j.clamp(0, 31)[:, None, :]) & 1
        see = (j < 0)[:, None, :] | ((bit == 1) & (j[:, None, :] < new[:, None, None]))
    s = s.masked_fill_(~see[:, None, :, None, :], -math.inf)
    s = torch.exp(s - s.amax(-1, keepdim=True).nan_to_num(neginf=0.0))
    den = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, n_kv, M * grp, L), v).view(B, n_kv, M, grp, D) / torch.where(den > 0, den, 1)
    o = o.permute(0, 2, 1, 3, 4).reshape(B * M, c["n_q"], D)
    t = torch.arange(T, device="cuda")
    req = torch.searchsorted(torch.cumsum(new, 0), t, right=True)
    return o[req * M + t - cu[req]].to(_T[c["y"]])


# ---------------------------------------------------------------- one pass

def run(state):
    st, c = state, state["case"]
    if not own:
        return {"rope": _rope_plain, "pages": _pages_plain, "append": _append_plain, "attn": _attn_plain}[c["op"]](st)
    import quantized_decode_gemv_block_gb300 as kq
    if c["op"] == "rope":
        q, k = kq.rope(st["q"], st["k"], st["pos"], st["freq"], pair_axis=st["axis"], adjacent=c["adjacent"],
                       inverse=c["inverse"], out_dtype=_T[c["y"]])
        return {"q": q, "k": k}
    if c["op"] == "pages":
        plan = kq.pages_plan(st["ctx"], st["new"], st["table"], st["free"], st["n_free"], c["P"], st["T"])
        return {"table": st["table"], "cu": plan.cu, "pos": plan.pos, "slot": plan.slot, "n_free": plan.n_free}
    if c["op"] == "append":
        kq.kv8_append(st["cache"], st["k"], st["v"], st["slot"])
        return {"k": st["kc"], "v": st["vc"], "k_scale": st["ks"], "v_scale": st["vs"]}
    return kq.attention_kv8(st["q"], st["cache"], st["table"], st["ctx"], st["new"], st["max_new"], st["max_len"],
                            total_len=st["total_len"], scale=1 / math.sqrt(c["D"]), mask=st.get("mask"), out_dtype=_T[c["y"]],
                            workspace=st["ws"])


def work(case):
    op = case["op"]
    b = {F32: 4, BF16: 2}
    if op == "rope":
        n = case["T"] * (case["n_q"] + case["n_kv"]) * case["D"]
        return {"bytes": n * (b[case["x"]] + b[case["y"]]) + 4 * case["axes"] * case["T"], "flops": 6 * n * case["rot"] // (2 * case["D"])}
    ctx, new = _lens(case)
    T, P = sum(new), case["P"]
    if op == "pages":
        fresh = sum(_blocks(c + n, P) - _blocks(c, P) for c, n in zip(ctx, new))
        started = sum(n > 0 and c % P > 0 for c, n in zip(ctx, new))
        return {"bytes": 4 * (3 * case["B"] + 2 + 2 * (T + case["pad"]) + 2 * fresh + started), "flops": 0}
    n_kv, D = case["n_kv"], case["D"]
    if op == "append":
        return {"bytes": 2 * T * n_kv * D * (b[case["x"]] + 1) + 4 * T, "flops": 4 * T * n_kv * D}
    seen = sum(c + n for c, n in zip(ctx, new))
    pages = sum(_blocks(c + n, P) for c, n in zip(ctx, new))
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
    return {"bytes": 2 * seen * n_kv * D + pages * (8 * n_kv + 4) + T * case["n_q"] * D * (b[case["x"]] + b[case["y"]]),
            "flops": 4 * D * case["n_q"] * pairs}


# ---------------------------------------------------------------- in 64 bits, from the definitions

def _exact_rope(st, c):
    h = c["rot"] // 2
    out = {}
    for name in ("q", "k"):
        x = st[name].double()
        y = x.clone()
        for i in range(h):
            m, n = (2 * i, 2 * i + 1) if c["adjacent"] else (i, i + h)
            a = st["pos"][int(st["axis"][i])].double() * st["freq"][i].double() * (-1.0 if c["inverse"] else 1.0)
            z = torch.complex(x[..., m], x[..., n]) * torch.polar(torch.ones_like(a), a)[:, None]
            y[..., m], y[..., n] = z.real, z.imag
        out[name] = y
    return out


def _exact_append(st, c):
    P, D = c["P"], c["D"]
    new, slot = st["new"].tolist(), st["slot"].tolist()
    out = {}
    for x, codes, scale, name, place in ((st["k"], "kc", "ks", "k", _k_offsets(D)), (st["v"], "vc", "vs", "v", _v_offsets(D))):
        x = x.double()
        codes, scale = st[codes].clone(), st[scale].double()
        place = torch.cat([place + g * 16 * D for g in range(P // 16)])  # [P, D]
        t = 0
        for n in new:
            end = t + n
            while t < end:
                page, at = divmod(slot[t], P)
                m = min(P - at, end - t)
                s_old = scale[page] if at else torch.zeros_like(scale[page])
                top = x[t:t + m].abs().amax((0, 2))
                s_new = torch.where(top > 0, ((top.view(torch.int64) >> 52) - 6 << 52).view(torch.float64), 0)
                s_new = torch.maximum(s_old, s_new)
                one = torch.where(s_new > 0, s_new, 1)[:, None]
                if at:
                    codes[page] = torch.floor(codes[page].double() * s_old[:, None] / one).to(torch.int8)
                q = torch.floor(x[t:t + m] / one).to(torch.int8)  # [m, n_kv, D]
                codes[page][:, place[at:at + m].reshape(-1)] = q.transpose(0, 1).reshape(q.shape[1], -1)
                scale[page] = s_new
                t += m
        out[name], out[name + "_scale"] = codes, scale
    return out


def _exact_attn(st, c):
    P, D, n_kv = c["P"], c["D"], c["n_kv"]
    grp = c["n_q"] // n_kv
    ko, vo = (torch.cat([f(D) + g * 16 * D for g in range(P // 16)]).reshape(-1) for f in (_k_offsets, _v_offsets))
    out = torch.zeros((st["q"].shape[0], c["n_q"], D), dtype=torch.float64, device="cuda")
    t = 0
    for r, (ctx, new) in enumerate(zip(st["ctx"].tolist(), st["new"].tolist())):
        L = ctx + new
        pages = st["table"][r, :_blocks(L, P)].long()
        for h in range(n_kv):
            k = ((st["kc"][pages, h][:, ko].double() + 0.5) * st["ks"][pages, h].double()[:, None]).reshape(-1, D)[:L]
            v = ((st["vc"][pages, h][:, vo].double() + 0.5) * st["vs"][pages, h].double()[:, None]).reshape(-1, D)[:L]
            q = st["q"][t:t + new, h * grp:(h + 1) * grp].double()
            s = torch.einsum("igd,ld->igl", q, k) / math.sqrt(D)
            see = torch.ones((new, new), dtype=torch.bool, device="cuda").tril()
            if "mask" in st:
                see = (st["mask"][t:t + new, None].long() >> torch.arange(new, device="cuda")) & 1 > 0
            s[:, :, ctx:] = s[:, :, ctx:].masked_fill(~see[:, None], -math.inf)
            out[t:t + new, h * grp:(h + 1) * grp] = torch.einsum("igl,ld->igd", torch.softmax(s, -1), v)
        t += new
    return out


def exact(case, seed):
    if case["op"] == "pages":  # whole numbers only: nothing is rounded
        return None
    st = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attn": _exact_attn}[case["op"]](st, case)
