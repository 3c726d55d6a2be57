"""Plain 64-bit references of the expert-layer operators, with bounds on the
fp32 arithmetic of the library's, for the tests."""
import numpy as np

U = 2.0 ** -24  # half a unit in the last place of fp32, relative
FLT_MAX = float(np.finfo(np.float32).max)


def e4m3_table():
    """Value of every e4m3 byte (NaN for 0x7f / 0xff)."""
    v = np.empty(256)
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[b] = np.nan if (e == 15 and m == 7) else (-x if s else x)
    return v


E4M3 = e4m3_table()


def route(logits, top_k, score="softmax", bias=None, renormalize=True, scale=1.0):
    """logits: float64 [T, E] (the stored values).  Returns weights (float64), experts,
    offsets, row_token, token_row and the relative bound of the fp32 weights."""
    T, E = logits.shape
    ok = ~np.isnan(logits) & (logits != -np.inf)
    l = np.where(ok, np.minimum(logits, FLT_MAX), -np.inf)
    key = l
    if bias is not None:
        with np.errstate(over="ignore"):
            key = 1.0 / (1.0 + np.exp(-l)) + bias.astype(np.float64)
        ok &= ~np.isnan(key) & (key != -np.inf)
        key = np.where(ok, key, -np.inf)
    weights = np.zeros((T, top_k))
    experts = np.full((T, top_k), -1, np.int32)
    spread = np.zeros(T)
    for t in range(T):
        order = np.argsort(-key[t], kind="stable")[:top_k]
        order = order[ok[t, order]]
        experts[t, :order.size] = order
        if not order.size:
            continue
        live = l[t] > -np.inf
        if score == "softmax":
            m = l[t][live].max()
            p = np.where(live, np.exp(l[t] - m), 0.0)
            total = p.sum()
            # the rounding of l - m is relative to it, and exp turns it into one of its value
            spread[t] = min(m - l[t][order].min(), 1e4)
        else:
            with np.errstate(over="ignore"):
                p = np.where(live, 1.0 / (1.0 + np.exp(-l[t])), 0.0)
            total = 1.0
        w = p[order]
        if renormalize:
            total = w.sum()
        weights[t, :order.size] = w / total * scale if total > 0 else 0.0
    rows = [(e, t, j) for t in range(T) for j, e in enumerate(experts[t]) if e >= 0]
    rows.sort(key=lambda r: (r[0], r[1]))
    counts = np.bincount([r[0] for r in rows], minlength=E) if rows else np.zeros(E, int)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    row_token = np.full(T * top_k, -1, np.int32)
    token_row = np.full((T, top_k), -1, np.int32)
    for r, (_, t, j) in enumerate(rows):
        row_token[r] = t
        token_row[t, j] = r
    # l - m: U * spread; exp: 2 units of 2^-23 on each side of the quotient; a sum of at
    # most E terms: E U; the division, the scale and the stored value: 1 U each
    bound = (U * (2 * spread + 8 + E + 4))[:, None]
    return weights, experts, offsets, row_token, token_row, bound


def _norm(v, dv, kind, gamma, beta, eps, K):
    """norm(v) and a bound on its fp32 value's error, from one of v's (dv).  A sum over the
    row in fp32 runs through at most 64 terms in a thread and 10 levels between threads."""
    c = 74 * U
    if kind == "layer":
        mu = v.mean(1, keepdims=True)
        dv = dv + c * np.abs(v).mean(1, keepdims=True) + dv.mean(1, keepdims=True) + U * (np.abs(v) + np.abs(mu))
        v = v - mu
    if kind != "none":
        ms = (v * v).mean(1, keepdims=True)
        dms = (2 * np.abs(v) * dv + dv * dv).mean(1, keepdims=True) + c * ms
        r = 1.0 / np.sqrt(ms + eps)
        dr = r * (0.5 * dms / (ms + eps) * 1.1 + 6 * U)
        v, dv = v * r, dv * r + np.abs(v) * dr + U * np.abs(v * r)
    if gamma is not None:
        v, dv = v * gamma, dv * np.abs(gamma) + U * np.abs(v * gamma)
    if beta is not None and kind == "layer":
        v = v + beta
        dv = dv + U * np.abs(v)
    return v, dv


def block_norm(x, residual=None, token_row=None, weights=None, post=("none", None, None, 1e-5),
               gate=None, token_gate=None, residual_scale=1.0, pre=("none", None, None, 1e-5)):
    """float64 (h, bound of h, y, bound of y); entries of token_row outside the rows skipped."""
    R, K = x.shape
    if token_row is not None:
        c = np.zeros((token_row.shape[0], K))
        d = np.zeros_like(c)
        for j in range(token_row.shape[1]):
            row = token_row[:, j]
            use = (row >= 0) & (row < R)
            term = np.where(use[:, None], x[np.where(use, row, 0)], 0.0) * np.where(use, weights[:, j], 0.0)[:, None]
            c += term
            d += U * (np.abs(term) + np.abs(c))
    else:
        c, d = x, np.zeros_like(x)
    v, d = _norm(c, d, *post, K)
    if gate is not None:
        v, d = v * gate, d * np.abs(gate) + U * np.abs(v * gate)
    if token_gate is not None:
        g = token_gate[:, None]
        v, d = v * g, d * np.abs(g) + U * np.abs(v * g)
    if residual is not None:
        a = residual * float(np.float32(residual_scale))
        v = v + a
        d = d + U * (np.abs(a) + np.abs(v))
    y, dy = _norm(v, d, *pre, K)
    return v, d, y, dy


def check_codes(values, scale, y, dy, top):
    """Codes (decoded, before the scale) and scales against y +- dy: the scale is max |y| /
    top, and every code the nearest of its grid, as far as y is known."""
    amax = np.abs(y).max(1)
    damax = dy.max(1)
    step = amax / top
    if top == 448.0:  # a zero or subnormal FP8 step is stored as 0
        step = np.where(step < 2.0 ** -126, 0.0, step)
    assert (np.abs(scale - step) <= damax / top + 2 * U * step + 1e-45).all()
    live = scale > 0
    s = np.where(live, scale, 1.0)[:, None].astype(np.float64)
    t = y / s
    # error of y, of the reciprocal and the product (3 U), the half-step of the grid
    slack = dy / s + 4 * U * np.abs(t)
    if top == 127.0:
        half = 0.5
        assert (np.abs(values) <= 127).all()
    else:
        mag = np.maximum(np.abs(t) + slack, 2.0 ** -6)
        half = 2.0 ** (np.floor(np.log2(mag)) - 4)
    # the largest value may lie a rounding above the top of the grid and saturates there
    assert (np.abs(values - np.clip(t, -top, top))[live] <= (half + slack)[live]).all()
    assert (values[~live] == 0).all()
