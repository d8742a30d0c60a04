"""Plain 64-bit forms of the paged 8-bit cache's operators, from their definitions (test helpers)."""
import numpy as np


def token_bytes(P, D, which):
    """Byte of (token, dim) within a (page, kv head): the layout that include/kq.h gives."""
    out = np.empty((P, D), np.int64)
    for o in range(P):
        b, p = divmod(o, 16)
        for d in range(D):
            if which == "k":
                x = d // 32 * 512 + (p // 4 * 2 + p % 2) * 64 + d // 4 % 4 * 16 + d // 16 % 2 * 8 + p // 2 % 2 * 4 + d % 4
            else:
                x = d // 32 * 512 + d % 8 * 64 + p // 4 * 16 + d // 16 % 2 * 8 + d // 8 % 2 * 4 + p % 4
            out[o, d] = 16 * b * D + x
    return out


def codes_of(raw, P, D, which):
    """(..., P*D) int8 as stored -> (..., P, D)."""
    return raw[..., token_bytes(P, D, which)]


def stored(codes, P, D, which):
    """(..., P, D) codes -> (..., P*D) as stored."""
    at = token_bytes(P, D, which).reshape(-1)
    out = np.zeros(codes.shape[:-2] + (P * D,), np.int8)
    out[..., at] = codes.reshape(codes.shape[:-2] + (P * D,))
    return out


def quantize_page(x):
    """(tokens, D) values of one (page, kv head) -> codes, scale."""
    x = np.asarray(x, np.float64)
    if not np.isfinite(x).all():
        return None, np.nan
    top = np.abs(x).max() if x.size else 0.0
    if top == 0:
        return np.zeros(x.shape, np.int8), 0.0
    s = max(2.0 ** (np.frexp(top)[1] - 1 - 6), 2.0 ** -126)
    return np.floor(x / s).astype(np.int8), s


def attention(q, kc, ks, vc, vs, table, ctx, new, P, n_kv, scale, mask=None):
    """o, sum_p w_p |v_p| and the largest sum |scale q k| over a token's heads; kc, vc: codes (pages, n_kv, P, D)."""
    T, n_q, D = q.shape
    grp = n_q // n_kv
    o, base, mag = np.zeros((T, n_q, D)), np.zeros((T, n_q, D)), np.zeros((T, n_q, 1))
    t = 0
    for r in range(len(ctx)):
        L = ctx[r] + new[r]
        pages = table[r, :-(-L // P)]
        for h in range(n_kv):
            k = ((kc[pages, h].astype(np.float64) + 0.5) * ks[pages, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:L]
            v = ((vc[pages, h].astype(np.float64) + 0.5) * vs[pages, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:L]
            for i in range(new[r]):
                see = np.arange(L) <= ctx[r] + i
                if mask is not None:
                    j = np.arange(L) - ctx[r]
                    see = (j < 0) | ((int(mask[t + i]) >> np.clip(j, 0, 31) & 1) == 1)
                if not see.any():
                    continue
                kk, vv = k[see], v[see]
                qq = q[t + i, h * grp:(h + 1) * grp].astype(np.float64)
                s = scale * qq @ kk.T
                w = np.exp(s - s.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                o[t + i, h * grp:(h + 1) * grp] = w @ vv
                base[t + i, h * grp:(h + 1) * grp] = w @ np.abs(vv)
                mag[t + i, h * grp:(h + 1) * grp, 0] = (abs(scale) * np.abs(qq) @ np.abs(kk).T).max(-1)
        t += new[r]
    return o, base, mag
