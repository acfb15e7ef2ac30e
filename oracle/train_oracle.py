"""fp64 restatements of the calls in include/usaf_train.h: the router's auxiliary losses and their
gradient, the dense router gradient products, and the 8-bit activation store. Plain numpy, nothing
shared with the CUDA path."""
import numpy as np


def _groups(T, group_offset):
    off = [0, T] if group_offset is None else [int(o) for o in group_offset]
    return [np.arange(off[g], off[g + 1]) for g in range(len(off) - 1)]


def softmax_lse(logits):
    """Row softmax and logsumexp; a row of nothing but -inf has zeros and 0."""
    l = np.asarray(logits, np.float64)
    dead = np.all(np.isneginf(l), axis=1)
    top = np.where(dead, 0.0, np.max(l, axis=1))
    with np.errstate(over="ignore", invalid="ignore"):
        ex = np.exp(l - top[:, None])
    s = ex.sum(1)
    s1 = np.where(dead, 1.0, s)
    return ex / s1[:, None], np.where(dead, 0.0, top + np.log(s1)), ~dead


def router_aux(logits, topk_idx, k, coef_balance, coef_z, token_mask=None, group_offset=None,
               d_loss=1.0):
    """dict of count [G,E], prob_sum [G,E], n_tok [G], loss [3] and dlogit [T,E]; the terms of
    dlogit's bracket besides (scale [T,E]: what a rounding error of the gradient is relative to)."""
    T, E = logits.shape
    p, lse, live = softmax_lse(logits)
    if token_mask is not None:
        live = live & (np.asarray(token_mask) != 0)
    idx = np.asarray(topk_idx).reshape(T, k)
    groups = _groups(T, group_offset)
    G = len(groups)
    count = np.zeros((G, E), np.int64)
    prob = np.zeros((G, E))
    n_tok = np.zeros(G, np.int64)
    sel = [g[live[g]] for g in groups]
    for g, t in enumerate(sel):
        n_tok[g] = t.size
        prob[g] = p[t].sum(0)
        np.add.at(count[g], idx[t].reshape(-1), 1)
    n = int(n_tok.sum())
    dl = np.zeros((T, E))
    scale = np.zeros((T, E))
    bal = z = 0.0
    for g, t in enumerate(sel):
        if not t.size:
            continue
        w = E / (k * n * t.size)
        bal += w * float(count[g] @ prob[g])
        z += float((lse[t] ** 2).sum()) / n
        pull = coef_balance * w * (count[g] - (p[t] @ count[g])[:, None])
        push = coef_z * 2.0 / n * lse[t][:, None]
        dl[t] = d_loss * p[t] * (pull + push)
        scale[t] = abs(d_loss) * p[t] * (coef_balance * w * count[g].max() + np.abs(push))
    loss = np.array([coef_balance * bal + coef_z * z, bal, z])
    return dict(count=count, prob_sum=prob, n_tok=n_tok, loss=loss, dlogit=dl, scale=scale)


def router_grad(dlogit, x, w_router, g_in=None, dx_in=None):
    d = np.asarray(dlogit, np.float64)
    g = d.T @ np.asarray(x, np.float64)
    dx = d @ np.asarray(w_router, np.float64)
    return (g if g_in is None else g + g_in), (dx if dx_in is None else dx + dx_in)


def act8_encode(v):
    """(codes, exponent bytes) of the rows of v in blocks of 16 along the last axis."""
    v = np.asarray(v, np.float64)
    rows, n = v.shape
    nb = -(-n // 16)
    code = np.zeros((rows, n), np.int8)
    byte = np.zeros((rows, nb), np.uint8)
    for b in range(nb):
        blk = v[:, 16 * b:16 * b + 16]
        amax = np.abs(blk).max(1)
        bad = ~np.isfinite(amax)
        safe = np.where(bad | (amax == 0), 1.0, amax)
        e = np.ceil(np.log2(safe / 127.0)).astype(np.int64)
        e += safe > 127.0 * np.exp2(e)            # log2 may be an ulp off at a power of two
        e -= safe <= 127.0 * np.exp2(e - 1)
        e = np.clip(e, -126, 121)
        with np.errstate(invalid="ignore"):
            c = np.clip(np.rint(blk / np.exp2(e)[:, None]), -127, 127)
        none = bad | (amax == 0)
        code[:, 16 * b:16 * b + 16] = np.where(none[:, None], 0, c).astype(np.int8)
        byte[:, b] = np.where(bad, 255, np.where(amax == 0, 0, e + 127))
    return code, byte


def act8_decode(code, byte):
    n = code.shape[1]
    b = np.repeat(byte.astype(np.int64), 16, axis=1)[:, :n]
    v = code.astype(np.float64) * np.where(b == 0, 0.0, np.exp2(b - 127.0))
    return np.where(b == 255, np.nan, v)


def act8_restore(x_code, x_exp, h_code, h_exp, topk_w, perm_tok, perm_slot, rows):
    """(x, x_perm, h, wa) of the first `rows` permuted rows."""
    x = act8_decode(x_code, x_exp)
    h = act8_decode(h_code[:, :rows], h_exp[:, :-(-rows // 16)])
    live = perm_slot[:rows] >= 0
    xp = np.where(live[None, :], x[perm_tok[:rows]].T, 0.0)
    I = h.shape[0] // 2
    w = np.where(live, np.asarray(topk_w, np.float64)[np.maximum(perm_slot[:rows], 0)], 0.0)
    return x, xp, h, w * h[:I] / (1.0 + np.exp(-h[:I])) * h[I:]
