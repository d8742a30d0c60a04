"""Inputs and 64-bit forms of the experts' products (test helpers)."""
import numpy as np
import torch

import oracle
from quantized_decode_gemv_block_gb300 import inputs

FMTS = {"q8_0": 1, "q4_k": 2, "affine4": 3, "q5_k": 4, "q6_k": 5}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def experts(fmt, E, N, K, seed=0):
    """(blocks on the GPU, [E, N, K] weights in 64 bits) of E matrices of normal weights."""
    blocks, plain = [], []
    for e in range(E):
        b = oracle.quantize(FMTS[fmt], inputs.weights(N, K, seed=seed, tensor_id=e))
        blocks.append(np.asarray(b).reshape(-1))
        plain.append(oracle.dequant(FMTS[fmt], b, N, K).reshape(N, K))
    return dev(np.concatenate(blocks)), np.stack(plain)


def bf16(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + sum(shape))
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def product(w, x, e):
    """(W_e x, sum |W_e x|) for each row of x, e its expert (-1: left out)."""
    x = x.double().cpu().numpy()
    y, b = np.zeros((len(x), w.shape[1])), np.zeros((len(x), w.shape[1]))
    for i in range(w.shape[0]):
        at = np.flatnonzero(e == i)
        if len(at):
            y[at], b[at] = x[at] @ w[i].T, np.abs(x[at]) @ np.abs(w[i]).T
    return y, b
