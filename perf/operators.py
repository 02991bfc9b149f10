"""Cases of the training operators around the Muon step, for measurement.

Three operators of a transformer block's training step, whose gradients are
what the optimizer consumes:

  layer_norm   forward (y, mean, rstd) and backward (dx, and the weight's and
               the bias's gradient, summed over all rows);
  attention    forward (o, lse) and the backward pass that recomputes the
               probabilities from lse; batched or packed documents, shared
               key/value heads, causal, sliding window;
  act8         activations kept in 8 bits for the backward pass (e4m3 codes,
               one power-of-two scale per token and 128 columns): store and
               restore, and the weight's gradient dW = dY^T X^ taken straight
               from the codes.

A case is a dict of plain values.  ``run`` computes the plain form (elementary
torch operations in 32 bits, rounded once at the end) or, where ``own`` is
true, calls the framework.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK = 128          # columns that share one scale
E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one micro-batch of a few tokens: the call's latency
        dict(name="ln_fwd_few", op="layer_norm", dir="forward", rows=8, cols=768, pad=0, dtype="bf16", wdtype="fp32"),
        # the norm of a 4096-wide model over 32 K tokens
        dict(name="ln_bwd_4096", op="layer_norm", dir="backward", rows=32768, cols=4096, pad=0, dtype="bf16",
             wdtype="fp32"),
        # an odd width inside wider rows (a slice of a larger activation), all in fp32
        dict(name="ln_bwd_ragged", op="layer_norm", dir="backward", rows=4099, cols=1023, pad=6, dtype="fp32",
             wdtype="fp32"),
        # one short sequence of a 12-head, 768-wide model: latency of the backward pass
        dict(name="attn_bwd_short", op="attention", dir="backward", batch=1, sq=61, sk=61, heads=12, kv_heads=12,
             dim=64, causal=True, window=0, docs=0, cut=0, fused=False, dtype="bf16"),
        # a batch of that model at its context length, q, k and v slices of one projection
        dict(name="attn_bwd_gpt2", op="attention", dir="backward", batch=8, sq=1024, sk=1024, heads=12, kv_heads=12,
             dim=64, causal=True, window=0, docs=0, cut=0, fused=True, dtype="bf16"),
        # 8 K context, 32 query heads on 8 key/value heads of 128
        dict(name="attn_fwd_8k", op="attention", dir="forward", batch=1, sq=8192, sk=8192, heads=32, kv_heads=8,
             dim=128, causal=True, window=0, docs=0, cut=0, fused=False, dtype="bf16"),
        dict(name="attn_bwd_8k", op="attention", dir="backward", batch=1, sq=8192, sk=8192, heads=32, kv_heads=8,
             dim=128, causal=True, window=0, docs=0, cut=0, fused=False, dtype="bf16"),
        # documents of uneven lengths packed into one row of tokens, 16 heads, fp16
        dict(name="attn_bwd_packed", op="attention", dir="backward", batch=1, sq=8005, sk=8005, heads=16, kv_heads=16,
             dim=128, causal=True, window=0, docs=21, cut=3, fused=True, dtype="fp16"),
        # a few tokens' activation: latency of store and restore
        dict(name="act8_few", op="act8", rows=16, cols=768, dtype="bf16"),
        # the input of a 14336-wide layer over 16 K tokens
        dict(name="act8_14336", op="act8", rows=16384, cols=14336, dtype="bf16"),
        # weight gradient of the 4096 -> 14336 layer over 16 K tokens
        dict(name="wgrad_14336", op="wgrad", rows=16384, cols=4096, out=14336, odtype="fp32", add=False),
        # one expert's layer with an odd share of the tokens, added to the gradient so far
        dict(name="wgrad_expert", op="wgrad", rows=1001, cols=2048, out=1408, odtype="fp32", add=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["layer_norm", "attention", "attention", "act8", "wgrad"])
    if op == "layer_norm":
        cols = _log(rng, 16, 16384)
        rows = min(_log(rng, 1, 65536), 32768 * 4096 // cols)
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        if dtype == "fp32":
            rows = max(1, rows // 2)
        return dict(op=op, dir=rng.choice(["forward", "backward"]), rows=rows, cols=cols, pad=rng.choice([0, 0, 8, 3]),
                    dtype=dtype, wdtype=rng.choice(["fp32", dtype]))
    if op == "attention":
        kv = rng.choice([1, 2, 4, 8, 12, 16])
        heads = kv * rng.choice([1, 1, 2, 4])
        dim = rng.choice([64, 128, 128, 80, 40])
        causal = rng.random() < 0.75
        window = _log(rng, 1, 4096) if causal and rng.random() < 0.25 else 0
        case = dict(op=op, dir=rng.choice(["forward", "backward", "backward"]), batch=1, sq=1, sk=1, heads=heads,
                    kv_heads=kv, dim=dim, causal=causal, window=window, docs=0, cut=0, fused=False,
                    dtype=rng.choice(["bf16", "bf16", "fp16"]))
        most = 32 * 8192 * 8192 // heads
        if rng.random() < 0.3:
            t = min(_log(rng, 16, 8192), math.isqrt(most))
            case.update(sq=t, sk=t, docs=rng.randint(2, 40), cut=rng.randrange(1000), fused=rng.random() < 0.5)
        else:
            sq = min(_log(rng, 1, 8192), math.isqrt(most))
            sk = sq if rng.random() < 0.6 else min(_log(rng, 1, 8192), most // sq)
            case.update(sq=sq, sk=sk, batch=max(1, min(_log(rng, 1, 16), most // (sq * sk))))
        return case
    if op == "act8":
        cols = _log(rng, 16, 16384)
        return dict(op=op, rows=min(_log(rng, 1, 65536), 16384 * 14336 // cols // 2), cols=cols,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    return dict(op=op, rows=_log(rng, 1, 16384), cols=_log(rng, 16, 4096), out=_log(rng, 16, 8192),
                odtype=rng.choice(["fp32", "fp32", "bf16"]), add=rng.random() < 0.3)


def _bounds(case):
    """Document boundaries of a packed case: uneven lengths, an empty one and one of a single token among them."""
    r = random.Random(case["cut"])
    t, n = case["sq"], case["docs"]
    at = sorted([0, t, t, min(1, t)] + [r.randint(1, t) for _ in range(n - 3)]) if n > 2 else [0, t // 2, t]
    return at


def _pairs(case):
    """Visible (query, key) pairs of one head over the whole batch."""
    spans = [(case["sq"], case["sk"])] * case["batch"]
    if case["docs"]:
        at = _bounds(case)
        spans = [(b - a, b - a) for a, b in zip(at, at[1:])]
    total = 0
    for sq, sk in spans:
        if not case["causal"]:
            total += sq * sk
            continue
        last = torch.arange(sq, dtype=torch.int64) + (sk - sq)
        first = (last - case["window"] + 1).clamp(min=0) if case["window"] else torch.zeros_like(last)
        total += int((last - first + 1).clamp(min=0).sum())
    return total


def work(case):
    if case["op"] == "layer_norm":
        r, c, s, w = case["rows"], case["cols"], SIZE[case["dtype"]], SIZE[case["wdtype"]]
        if case["dir"] == "forward":
            return {"bytes": 2 * r * c * s + 2 * c * w + 8 * r, "flops": 8 * r * c}
        return {"bytes": 3 * r * c * s + c * w + 8 * c + 8 * r, "flops": 14 * r * c}
    if case["op"] == "attention":
        s, d, b = SIZE[case["dtype"]], case["dim"], case["batch"]
        q, kv = b * case["sq"] * case["heads"] * d * s, b * case["sk"] * case["kv_heads"] * d * s
        lse, p = 4 * b * case["sq"] * case["heads"], _pairs(case) * case["heads"]
        if case["dir"] == "forward":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * d * p}
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 10 * d * p}
    if case["op"] == "act8":
        n, s = case["rows"] * case["cols"], SIZE[case["dtype"]]
        codes = n + case["rows"] * -(-case["cols"] // BLOCK)
        return {"bytes": 2 * n * s + 2 * codes, "flops": 4 * n}
    t, n, o = case["rows"], case["cols"], case["out"]
    s = SIZE[case["odtype"]]
    return {"bytes": 2 * t * o + t * n + t * -(-n // BLOCK) + n * o * s * (2 if case["add"] else 1),
            "flops": 2 * t * n * o}


# ------------------------------------------------------------------ inputs
def _activation(g, rows, cols):
    """Hidden activations: unit scale, a spread between channels, a few channels far above the rest."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    gain = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    far = torch.rand(cols, generator=g, device="cuda") < 0.004
    return x * torch.where(far, gain * 30.0, gain)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    st = dict(case=case)
    if case["op"] == "layer_norm":
        r, c, dt = case["rows"], case["cols"], DT[case["dtype"]]
        wide = (_activation(g, r, c + case["pad"]) + 0.3).to(dt)
        st.update(x=wide[:, :c], weight=(1 + 0.2 * randn(c)).to(DT[case["wdtype"]]),
                  bias=(0.1 * randn(c)).to(DT[case["wdtype"]]), eps=1e-5)
        if case["dir"] == "backward":
            x = st["x"].float()
            mean = x.mean(-1)
            st.update(mean=mean, rstd=torch.rsqrt((x - mean[:, None]).square().mean(-1) + st["eps"]),
                      dy=(randn(r, c + case["pad"]).to(dt))[:, :c])
    elif case["op"] == "attention":
        b, sq, sk, h, hk, d = (case[k] for k in ("batch", "sq", "sk", "heads", "kv_heads", "dim"))
        dt = DT[case["dtype"]]
        if case["fused"]:      # one projection's output, sliced
            q, k, v = randn(b, sq, h + 2 * hk, d).to(dt).split([h, hk, hk], 2)
        else:
            q, k, v = randn(b, sq, h, d).to(dt), randn(b, sk, hk, d).to(dt), randn(b, sk, hk, d).to(dt)
        st.update(q=q, k=k, v=v)
        if case["docs"]:
            st.update(cu=torch.tensor(_bounds(case), dtype=torch.int32, device="cuda"))
            st.update({n: st[n][0] for n in "qkv"})
        if case["dir"] == "backward":
            o, lse = _attention(st)
            st.update(o=o, lse=lse, do=randn(*o.shape).to(dt))
    elif case["op"] == "act8":
        st.update(x=_activation(g, case["rows"], case["cols"]).to(DT[case["dtype"]]))
    else:
        x = _activation(g, case["rows"], case["cols"]).to(torch.bfloat16)
        st.update(dy=(1e-2 * randn(case["rows"], case["out"])).to(torch.bfloat16))
        if case["add"]:
            st.update(so_far=(1e-1 * randn(case["out"], case["cols"])).to(DT[case["odtype"]]))
        codes, scales = _encode(x)
        # as the framework hands them out: rows of whole 128-column blocks, scales block by block over the tokens
        blocks, t16 = -(-case["cols"] // BLOCK), -(-case["rows"] // 16) * 16
        wide = torch.zeros(case["rows"], blocks * BLOCK, device="cuda", dtype=torch.float8_e4m3fn)
        wide[:, :case["cols"]] = codes
        tall = torch.zeros(blocks, t16, device="cuda", dtype=torch.uint8)
        tall[:, :case["rows"]] = scales.t()
        st.update(codes=wide[:, :case["cols"]], scales=tall[:, :case["rows"]])
    return st


# ------------------------------------------------------------- plain forms
def _mask(st):
    """True where a query sees a key, [queries, keys], or None."""
    case = st["case"]
    sq, sk = case["sq"], case["sk"]
    i = torch.arange(sq, device="cuda")[:, None] + (sk - sq)
    j = torch.arange(sk, device="cuda")[None, :]
    see = None
    if case["causal"]:
        see = j <= i
        if case["window"]:
            see = see & (j > i - case["window"])
    if case["docs"]:
        doc = torch.bucketize(torch.arange(sq, device="cuda", dtype=torch.int32), st["cu"][1:], right=True)
        same = doc[:, None] == doc[None, :]
        see = same if see is None else see & same
    return see


def _split(t, groups):
    """[.., tokens, heads, dim] in fp32 as [batch, groups, heads per group, tokens, dim]."""
    t = t.float() if t.dim() == 4 else t.float()[None]
    return t.unflatten(2, (groups, -1)).permute(0, 2, 3, 1, 4)


def _join(t, like):
    return t.permute(0, 3, 1, 2, 4).reshape(like.shape).to(like.dtype)


def _scores(st):
    case = st["case"]
    hk = case["kv_heads"]
    s = torch.matmul(_split(st["q"], hk), _split(st["k"], hk).transpose(-1, -2)) * (1.0 / math.sqrt(case["dim"]))
    see = _mask(st)
    return s if see is None else s.masked_fill(~see, float("-inf"))


def _attention(st):
    hk = st["case"]["kv_heads"]
    s = _scores(st)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, _split(st["v"], hk)) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total))[..., 0].flatten(1, 2)
    return _join(o, st["q"]), lse[0] if st["q"].dim() == 3 else lse


def _attention_backward(st):
    hk, scale = st["case"]["kv_heads"], 1.0 / math.sqrt(st["case"]["dim"])
    q, k, v, do, o = (_split(st[n], hk) for n in ("q", "k", "v", "do", "o"))
    lse = (st["lse"] if st["lse"].dim() == 3 else st["lse"][None]).unflatten(1, (hk, -1))[..., None]
    p = torch.exp(_scores(st) - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse))
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2, keepdim=True)
    ds = p * (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True)) * scale
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2, keepdim=True)
    return _join(dq, st["q"]), _join(dk, st["k"]), _join(dv, st["v"])


def _layer_norm(st):
    x = st["x"].float()
    mean = x.mean(-1)
    d = x - mean[:, None]
    rstd = torch.rsqrt(d.square().mean(-1) + st["eps"])
    return (d * rstd[:, None] * st["weight"].float() + st["bias"].float()).to(st["x"].dtype), mean, rstd


def _layer_norm_backward(st):
    dy, rstd = st["dy"].float(), st["rstd"][:, None]
    xhat = (st["x"].float() - st["mean"][:, None]) * rstd
    g = dy * st["weight"].float()
    dx = rstd * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    return dx.to(st["x"].dtype), (dy * xhat).sum(0), dy.sum(0)


def _power(scales):
    """2^(scale - 127) in fp32 from its bits (255: infinity)."""
    return (scales.to(torch.int32) << 23).view(torch.float32)


def _encode(x):
    """e4m3 codes [rows, cols] and scale exponents [rows, blocks]: the smallest power of two that brings a block's
    largest value to 448 or less, at least 2^-111; a block with a value that is not finite gets scale 255, codes 0."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    xb = torch.nn.functional.pad(x.float(), (0, blocks * BLOCK - cols)).view(rows, blocks, BLOCK)
    top = xb.abs().amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(m <= E4M3_MAX / 512, e - 9, e - 8).to(torch.int32) + 127
    e = torch.where(top == 0, torch.full_like(e, 16), e.clamp(min=16))
    fine = torch.isfinite(top)
    e = torch.where(fine, e, torch.full_like(e, 255))
    unit = _power(torch.where(fine, 254 - e, torch.zeros_like(e)))
    codes = torch.where(fine[..., None], xb * unit[..., None], torch.zeros_like(xb)).to(torch.float8_e4m3fn)
    return codes.view(rows, blocks * BLOCK)[:, :cols], e.to(torch.uint8)


def _decode(codes, scales):
    """The values that codes [rows, cols] and scale exponents [blocks, rows] stand for, fp32."""
    return codes.float() * _power(scales).t().repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _plain(st):
    case = st["case"]
    if case["op"] == "layer_norm":
        return _layer_norm(st) if case["dir"] == "forward" else _layer_norm_backward(st)
    if case["op"] == "attention":
        return _attention(st) if case["dir"] == "forward" else _attention_backward(st)
    if case["op"] == "act8":
        codes, scales = _encode(st["x"])
        return _decode(codes, scales.t()).to(st["x"].dtype), scales.t()
    dw = torch.matmul(st["dy"].float().t(), _decode(st["codes"], st["scales"]))
    if case["add"]:
        dw = st["so_far"].float() + dw
    return dw.to(DT[case["odtype"]])


def run(st):
    if not own:
        return _plain(st)
    import newton_schulz_orthogonalized_muon_gb300 as muon
    case = st["case"]
    if case["op"] == "layer_norm":
        if case["dir"] == "forward":
            return muon.layer_norm(st["x"], st["weight"], st["bias"], eps=st["eps"])
        return muon.layer_norm_backward(st["dy"], st["x"], st["mean"], st["rstd"], st["weight"])
    if case["op"] == "attention":
        kw = dict(causal=case["causal"], window=case["window"])
        if case["docs"]:
            kw.update(cu_seqlens_q=st["cu"], cu_seqlens_k=st["cu"])
        if case["dir"] == "forward":
            return muon.attention(st["q"], st["k"], st["v"], **kw)
        return muon.attention_backward(st["do"], st["q"], st["k"], st["v"], st["o"], st["lse"], **kw)
    if case["op"] == "act8":
        codes, scales = muon.act8_store(st["x"])
        return muon.act8_restore(codes, scales, dtype=st["x"].dtype), scales
    if case["add"]:
        return muon.act8_weight_grad(st["dy"], st["codes"], st["scales"], add=st["so_far"])
    return muon.act8_weight_grad(st["dy"], st["codes"], st["scales"], dtype=DT[case["odtype"]])


# ------------------------------------------------- the definitions, 64 bits
def _exact_attention(st, case):
    scale = 1.0 / math.sqrt(case["dim"])
    packed = case["docs"] > 0
    q, k, v = (st[n].double() if not packed else st[n].double()[None] for n in "qkv")
    do = st["do"].double().reshape(q.shape) if "do" in st else None
    o, dq = torch.zeros_like(q), torch.zeros_like(q)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    lse = torch.full((q.shape[0], q.shape[2], q.shape[1]), -math.inf, dtype=torch.float64, device=q.device)
    at = _bounds(case) if packed else None
    spans = list(zip(at, at[1:])) if packed else None
    group = case["heads"] // case["kv_heads"]
    for b in range(q.shape[0]):
        for q0, q1, k0, k1 in ([(a, e, a, e) for a, e in spans] if packed else [(0, case["sq"], 0, case["sk"])]):
            nq, nk = q1 - q0, k1 - k0
            if nq == 0 or nk == 0:
                continue
            off = nk - nq
            hidden = torch.zeros(nq, nk, dtype=torch.bool, device=q.device)
            if case["causal"]:
                full = torch.ones(nq, nk, dtype=torch.bool, device=q.device)
                hidden = full.triu(off + 1)
                if case["window"]:
                    hidden = hidden | full.tril(off - case["window"])
            for h in range(case["heads"]):
                kh, vh = k[b, k0:k1, h // group], v[b, k0:k1, h // group]
                s = (q[b, q0:q1, h] @ kh.T) * scale
                s[hidden] = -math.inf
                z = torch.logsumexp(s, dim=1)
                p = torch.exp(s - torch.where(z == -math.inf, 0.0, z)[:, None])
                oh = p @ vh
                o[b, q0:q1, h], lse[b, h, q0:q1] = oh, z
                if do is not None:
                    g = do[b, q0:q1, h]
                    dv[b, k0:k1, h // group] += p.T @ g
                    ds = p * (g @ vh.T - (g * oh).sum(1, keepdim=True)) * scale
                    dq[b, q0:q1, h] = ds @ kh
                    dk[b, k0:k1, h // group] += ds.T @ q[b, q0:q1, h]
    out = (o, lse) if do is None else (dq, dk, dv)
    return tuple(t[0] for t in out) if packed else out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "layer_norm":
        x, w = st["x"].double(), st["weight"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + st["eps"]) ** -0.5
        z = (x - mean.unsqueeze(1)) * rstd.unsqueeze(1)
        if case["dir"] == "forward":
            return z * w + st["bias"].double(), mean, rstd
        dy = st["dy"].double()
        a = dy * w
        dx = (a - a.sum(1, keepdim=True) / case["cols"] - z * ((a * z).sum(1, keepdim=True) / case["cols"])) * rstd.unsqueeze(1)
        return dx, torch.einsum("rc,rc->c", dy, z), torch.einsum("rc->c", dy)
    if case["op"] == "attention":
        if _pairs(case) * case["heads"] * case["dim"] > 2e11:
            return None
        return _exact_attention(st, case)
    if case["op"] == "act8":
        # per block: grid spacing of a value v under scale s is s * 2^(max(floor(log2|v/s|), -6) - 3)
        x = st["x"].double()
        out = torch.empty_like(x)
        for c in range(0, case["cols"], BLOCK):
            part = x[:, c:c + BLOCK]
            top = part.abs().amax(1, keepdim=True)
            e = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / E4M3_MAX))
            e = torch.clamp(torch.where(top * torch.exp2(-(e - 1)) <= E4M3_MAX, e - 1, e), min=-111.0)
            u = part * torch.exp2(-e)
            step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(u.abs(), min=1e-300))), min=-6.0) - 3.0)
            out[:, c:c + BLOCK] = torch.round(u / step) * step * torch.exp2(e)
        return out, None
    rows, blocks = case["rows"], -(-case["cols"] // BLOCK)
    xhat = torch.ldexp(st["codes"].double(), (st["scales"].long() - 127).t().unsqueeze(2).expand(rows, blocks, BLOCK).reshape(rows, -1)[:, :case["cols"]])
    dw = torch.mm(st["dy"].double().T, xhat)
    return dw + st["so_far"].double() if case["add"] else dw
