"""Plain fp64 NumPy forms of the training operators: layer norm, attention,
activations in 8 bits.  Each function also returns, where its result is a sum
of products that the kernels form from rounded factors, the sum of the
products' magnitudes, from which the tests derive their tolerances."""
import numpy as np

BLOCK = 128


# ---------------------------------------------------------------- layer norm
def layer_norm(x, w, b, eps):
    mean = x.mean(-1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(-1) + eps)
    return d * rstd[:, None] * w + b, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, w):
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - g.mean(-1, keepdims=True) - xh * (g * xh).mean(-1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


# ----------------------------------------------------------------- attention
def visible(nq, nk, causal, window):
    """[nq, nk] True where a query sees a key."""
    see = np.ones((nq, nk), bool)
    if causal:
        place = np.arange(nq)[:, None] + (nk - nq)
        j = np.arange(nk)[None, :]
        see = j <= place
        if window:
            see &= j > place - window
    return see


def _probabilities(q, k, see, scale):
    s = np.where(see, (q @ k.T) * scale, -np.inf)
    top = s.max(1, initial=-np.inf)
    top = np.where(np.isfinite(top), top, 0.0)
    e = np.exp(s - top[:, None])
    with np.errstate(divide="ignore"):
        lse = top + np.log(e.sum(1))
    return np.exp(s - np.where(np.isfinite(lse), lse, 0.0)[:, None]), lse


def attention(q, k, v, causal, window, scale):
    """One sequence, q [nq, heads, dim], k and v [nk, kv_heads, dim]:
    o, lse [heads, nq], and sum_j p_ij |v_j|."""
    nq, heads, _ = q.shape
    group = heads // k.shape[1]
    see = visible(nq, k.shape[0], causal, window)
    o, mag, lse = np.zeros(q.shape), np.zeros(q.shape), np.full((heads, nq), -np.inf)
    for h in range(heads):
        p, lse[h] = _probabilities(q[:, h], k[:, h // group], see, scale)
        o[:, h] = p @ v[:, h // group]
        mag[:, h] = p @ np.abs(v[:, h // group])
    return o, lse, mag


def attention_backward(do, q, k, v, o, causal, window, scale):
    """One sequence: (dq, dk, dv), the magnitudes of the products that are
    summed into each, and (for the fp32 differences inside ds) the
    magnitudes with |do||v| + |do||o| in the place of |do v - do o|."""
    nq, heads, _ = q.shape
    group = heads // k.shape[1]
    see = visible(nq, k.shape[0], causal, window)
    out = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)]
    mag = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)]
    wide = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)]
    for h in range(heads):
        kh, vh, qh, g = k[:, h // group], v[:, h // group], q[:, h], do[:, h]
        p, _ = _probabilities(qh, kh, see, scale)
        ds = p * (g @ vh.T - (g * o[:, h]).sum(1, keepdims=True)) * scale
        big = p * (np.abs(g) @ np.abs(vh).T + (np.abs(g) * np.abs(o[:, h])).sum(1, keepdims=True)) * scale
        out[0][:, h] = ds @ kh
        out[1][:, h // group] += ds.T @ qh
        out[2][:, h // group] += p.T @ g
        mag[0][:, h] = np.abs(ds) @ np.abs(kh)
        mag[1][:, h // group] += np.abs(ds).T @ np.abs(qh)
        mag[2][:, h // group] += p.T @ np.abs(g)
        wide[0][:, h] = big @ np.abs(kh)
        wide[1][:, h // group] += big.T @ np.abs(qh)
        wide[2][:, h // group] += p.T @ np.abs(g)
    return out, mag, wide


# --------------------------------------------------- activations in 8 bits
def e4m3_table():
    """The value of every e4m3 code (NaN for 0x7F and 0xFF)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v[(c & 0x7F) == 0x7F] = np.nan
    return np.where(c & 0x80, -v, v)


def act8_encode(x):
    """(codes, scale bytes [blocks, rows]) of x [rows, cols]: the nearest
    e4m3 value (ties to the even code) of x over the block's scale."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    codes = np.zeros((rows, cols), np.uint8)
    scales = np.zeros((blocks, rows), np.uint8)
    pos = e4m3_table()[:0x7F]                     # rising values of codes 0 .. 0x7E
    mid = (pos[1:] + pos[:-1]) / 2
    for b in range(blocks):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        for r in range(rows):
            if not np.isfinite(part[r]).all():
                scales[b, r] = 255
                continue
            a = np.abs(part[r]).max()
            e = -111
            while a > 448.0 * 2.0 ** e:
                e += 1
            scales[b, r] = e + 127
            u = np.abs(part[r]) * 2.0 ** -e
            lo = np.searchsorted(mid, u, side="left")         # codes whose upper midpoint is below u
            tie = (lo < len(mid)) & (mid[np.minimum(lo, len(mid) - 1)] == u)
            lo = lo + (tie & (lo % 2 == 1))
            codes[r, b * BLOCK:b * BLOCK + part.shape[1]] = lo | np.where(np.signbit(part[r]), 0x80, 0)
    return codes, scales


def act8_decode(codes, scales):
    """The values of codes [rows, cols] under scale bytes [blocks, rows]."""
    with np.errstate(invalid="ignore"):
        unit = np.where(scales == 255, np.inf, 2.0 ** (scales.astype(np.float64) - 127))
        return e4m3_table()[codes] * np.repeat(unit, BLOCK, 0)[:codes.shape[1]].T


def act8_weight_grad(dy, x):
    """dy^T x and the sum of the products' magnitudes."""
    return dy.T @ x, np.abs(dy).T @ np.abs(x)


# ------------------------------------------------------ products by expert
def expert_ranges(offsets, tokens):
    """[(first, end)] of each expert's tokens: offsets cut to the token axis
    and raised to the largest before them."""
    at = np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, tokens))
    return list(zip(at[:-1], at[1:]))


def expert_matmul(x, w, offsets, transpose=False):
    """x[t] w[e]^T (or x[t] w[e]) for the tokens of each expert, zeros for the
    others, and the sum of the products' magnitudes."""
    y = np.zeros((x.shape[0], w.shape[2 if transpose else 1]))
    mag = np.zeros_like(y)
    for e, (a, b) in enumerate(expert_ranges(offsets, x.shape[0])):
        m = w[e] if transpose else w[e].T
        y[a:b] = x[a:b] @ m
        mag[a:b] = np.abs(x[a:b]) @ np.abs(m)
    return y, mag


def expert_weight_grad(dy, x, offsets):
    """[experts, out, cols]: dy^T x over each expert's tokens, and the sum of
    the products' magnitudes."""
    parts = [(dy[a:b].T @ x[a:b], np.abs(dy[a:b]).T @ np.abs(x[a:b])) for a, b in expert_ranges(offsets, x.shape[0])]
    return np.stack([p for p, _ in parts]), np.stack([m for _, m in parts])
