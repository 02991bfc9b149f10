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


# ------------------------------------------------- weights in 8 bits
def _nearest_codes(u):
    """e4m3 codes nearest to u (|u| <= 448), ties to the even code."""
    pos = e4m3_table()[:0x7F]
    mid = (pos[1:] + pos[:-1]) / 2
    a = np.abs(u)
    lo = np.searchsorted(mid, a, side="left")
    tie = (lo < len(mid)) & (mid[np.minimum(lo, len(mid) - 1)] == a)
    return (lo + (tie & (lo % 2 == 1))) | np.where(np.signbit(u), 0x80, 0)


def _scale_exponent(top, largest):
    """The smallest whole e >= -111 with top 2^-e <= largest."""
    e = -111
    while top > largest * 2.0 ** e:
        e += 1
    return e


def act8_encode_weight(w):
    """(codes, scale bytes [column blocks, row blocks]) of w [out, cols]."""
    out, cols = w.shape
    codes = np.zeros(w.shape, np.uint8)
    scales = np.zeros((-(-cols // BLOCK), -(-out // BLOCK)), np.uint8)
    for k in range(scales.shape[0]):
        for o in range(scales.shape[1]):
            at = np.s_[o * BLOCK:(o + 1) * BLOCK, k * BLOCK:(k + 1) * BLOCK]
            if not np.isfinite(w[at]).all():
                scales[k, o] = 255
                continue
            e = _scale_exponent(np.abs(w[at]).max(), 448.0)
            scales[k, o] = e + 127
            codes[at] = _nearest_codes(w[at] * 2.0 ** -e)
    return codes, scales


def act8_decode_weight(codes, scales):
    """The values of codes [out, cols] under scale bytes [column blocks, row blocks]."""
    unit = np.where(scales == 255, np.inf, 2.0 ** (scales.astype(np.float64) - 127))
    with np.errstate(invalid="ignore"):
        return e4m3_table()[codes] * np.repeat(np.repeat(unit.T, BLOCK, 0)[:codes.shape[0]], BLOCK, 1)[:, :codes.shape[1]]


# --------------------------------------------- AdamW with states in 8 bits
def root_table():
    """The value of every code of a root."""
    c = np.arange(256)
    return np.where(c == 0, 0.0, (1 + (c & 15) / 16.0) * 2.0 ** ((c >> 4) - 8.0))


def adamw8_noise(n, seed, beta=0.0):
    """The number in [0, 1) that each element is rounded with.  beta: the larger
    of the two; above 31/32 the place in a byte's 1/256 is the call's, else its
    middle."""
    salt = seed * 0x9E3779B1 % 2 ** 32
    x = (np.arange(-(-n // 4), dtype=np.uint64) + np.uint64(salt)) % np.uint64(2 ** 32)
    for shift, factor in ((16, 0x7FEB352D), (15, 0x846CA68B)):
        x = (x ^ (x >> np.uint64(shift))) * np.uint64(factor) % np.uint64(2 ** 32)
    x ^= x >> np.uint64(16)
    b = np.stack([(x >> np.uint64(8 * k)) & np.uint64(255) for k in range(4)], 1).reshape(-1)[:n]
    return (b.astype(np.float64) + ((salt >> 21) / 2048 if beta > 31 / 32 else 0.5)) / 256


def _blocks(x):
    return [x[i:i + BLOCK] for i in range(0, len(x), BLOCK)]


def adamw8_decode(avg, root, avg_scale, root_scale):
    """(m, r) of flat codes and their blocks' scale bytes."""
    def unit(s):
        return np.repeat(np.where(s == 255, np.inf, 2.0 ** (s.astype(np.float64) - 127)), BLOCK)[:len(avg)]
    with np.errstate(invalid="ignore"):
        return e4m3_table()[avg] * unit(avg_scale), root_table()[root] * unit(root_scale)


def adamw8_codes(x, noise, table, largest, least, given=None):
    """(codes, scale bytes) of magnitudes x by the rounding rule: the largest
    code whose value is at most u, or the next where (u - value) / (next -
    value) + noise >= 1; at least `least` for what is not 0.  And how near each
    was to the other choice, as a part of the step.  given: scale bytes that a
    block takes where its largest is within 2^-20 of a scale's limit."""
    codes, scales, near = np.zeros(len(x), np.uint8), [], np.ones(len(x))
    for i, part in enumerate(_blocks(x)):
        if not np.isfinite(part).all():
            scales.append(255)
            continue
        top = part.max(initial=0.0)
        e = _scale_exponent(top, largest)
        if given is not None and abs(int(given[i]) - 127 - e) == 1:
            other = int(given[i]) - 127
            if abs(top / (largest * 2.0 ** min(e, other)) - 1) < 2.0 ** -20:
                e = other
        scales.append(e + 127)
        u = part * 2.0 ** -e
        lo = np.searchsorted(table, u, side="right") - 1
        up = np.minimum(lo + 1, len(table) - 1)
        step = np.where(up > lo, table[up] - table[lo], 1.0)
        frac = (u - table[lo]) / step
        z = noise[i * BLOCK:i * BLOCK + len(part)]
        c = np.where(frac + z >= 1, up, lo)
        codes[i * BLOCK:i * BLOCK + len(part)] = np.where(u > 0, np.maximum(c, least), 0)
        near[i * BLOCK:i * BLOCK + len(part)] = np.abs(frac + z - 1)
    return codes, np.array(scales, np.uint8), near


def adamw8_step(p, g, m, r, step, lr, beta1, beta2, eps, wd):
    """(p, m, r) after the step, before the states are rounded."""
    g = np.where(np.isfinite(g), np.clip(g, -2.0 ** 63, 2.0 ** 63), g)
    m = m + (1 - beta1) * (g - m)
    r = np.sqrt(r * r + (1 - beta2) * (g * g - r * r))
    size = lr * np.sqrt(1 - beta2 ** step) / (1 - beta1 ** step)
    return p * (1 - lr * wd) - size * m / (eps + r), m, r
