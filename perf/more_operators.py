"""Cases of a second set of training operators, for measurement.

What the linear layers of a mixture-of-experts model need around the Muon
step, and the optimizer's states in 8 bits:

  experts   products of a layer whose tokens are grouped by expert, ragged
            sizes: forward, the input's gradient, the weight's gradient;
  matmul8   the product of activations and weights that are both kept in 8
            bits (e4m3 codes; one power-of-two scale a token and 128 columns,
            and one a 128 x 128 block of the weight);
  weight8   a weight brought into that form, with its transpose;
  adamw8    an AdamW step over many tensors whose two states are kept in 8
            bits, blocks of 128 elements with a power-of-two scale each.

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
BLOCK = 128
E4M3_MAX = 448.0
ROOT_MAX = 248.0     # the largest value of a root's code: (1 + 15/16) 2^7
ADAM = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.1)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a handful of tokens, six experts each, through one layer of 64 experts: mostly weights to read
        dict(name="experts_few", op="experts", dir="forward", experts=64, rows=48, behind=0, cols=2048, out=1408, cut=1,
             spread=1.0, dtype="bf16", odtype="bf16", add=False),
        # a micro-batch of 8 K tokens, six experts each, through that layer
        dict(name="experts_fwd", op="experts", dir="forward", experts=64, rows=49152, behind=0, cols=2048, out=1408, cut=2,
             spread=0.4, dtype="bf16", odtype="bf16", add=False),
        # the gradient of that layer's input
        dict(name="experts_dx", op="experts", dir="input", experts=64, rows=49152, behind=0, cols=2048, out=1408, cut=3,
             spread=0.4, dtype="bf16", odtype="bf16", add=False),
        # the weights' gradients, as Muon takes them
        dict(name="experts_dw", op="experts", dir="weight", experts=64, rows=49152, behind=0, cols=2048, out=1408, cut=4,
             spread=0.4, dtype="bf16", odtype="bf16", add=False),
        # few experts of a narrow fp16 layer, an odd number of tokens and some of no expert, added to an fp32 gradient
        dict(name="experts_dw_odd", op="experts", dir="weight", experts=8, rows=1003, behind=21, cols=768, out=2304, cut=5,
             spread=1.2, dtype="fp16", odtype="fp32", add=True),
        # a few tokens through the 4096 -> 14336 layer in 8 bits: the weight has to be read
        dict(name="matmul8_few", op="matmul8", rows=16, cols=4096, out=14336, odtype="bf16"),
        # 16 K tokens through it
        dict(name="matmul8_14336", op="matmul8", rows=16384, cols=4096, out=14336, odtype="bf16"),
        # odd sizes, result in fp32
        dict(name="matmul8_odd", op="matmul8", rows=1001, cols=2042, out=1411, odtype="fp32"),
        # that layer's weight after a step, both ways round
        dict(name="weight8_14336", op="weight8", out=14336, cols=4096, dtype="bf16"),
        # a narrow one
        dict(name="weight8_768", op="weight8", out=2304, cols=768, dtype="fp32"),
        # norms and biases of a 768-wide model's last blocks: the call's latency
        dict(name="adamw8_vectors", op="adamw8", tensors=18, big=4, most=2304, small=768, cut=6, dtype="fp32", gdtype="fp32",
             step=10),
        # embedding and output head of a 4096-wide model with a vocabulary of 128 K, and its norms
        dict(name="adamw8_embed", op="adamw8", tensors=12, big=2, most=128256 * 4096, small=4096, cut=7, dtype="bf16",
             gdtype="bf16", step=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["experts", "experts", "experts", "matmul8", "matmul8", "weight8", "adamw8", "adamw8"])
    if op == "experts":
        way = rng.choice(["forward", "input", "weight"])
        experts = _log(rng, 1, 128)
        cols = 8 * _log(rng, 8, 512)
        out = 8 * _log(rng, 8, max(8, min(512, 64 * 1408 * 2048 // (experts * cols * 8))))
        most = 49152 * 2048 * 1408 // (cols * out)
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        odtype = rng.choice(["fp32", dtype]) if way == "weight" else dtype
        return dict(op=op, dir=way, experts=experts, rows=_log(rng, 1, max(1, min(49152, most))),
                    behind=rng.choice([0, 0, 5, 300]), cols=cols, out=out, cut=rng.randrange(1 << 20),
                    spread=rng.uniform(0.0, 1.0), dtype=dtype, odtype=odtype, add=way == "weight" and rng.random() < 0.3)
    if op == "matmul8":
        return dict(op=op, rows=_log(rng, 1, 16384), cols=_log(rng, 16, 4096), out=_log(rng, 16, 14336),
                    odtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op == "weight8":
        cols = _log(rng, 16, 8192)
        return dict(op=op, out=_log(rng, 16, min(16384, 14336 * 2048 // cols)), cols=cols,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    tensors = rng.randint(1, 20)
    big, most = rng.randint(1, min(4, tensors)), _log(rng, 100, 1 << 26)
    return dict(op=op, tensors=tensors, big=big, most=most, small=_log(rng, 1, min(most, 1 << 20)), cut=rng.randrange(1 << 20),
                dtype=rng.choice(["bf16", "bf16", "fp32"]), gdtype=rng.choice(["bf16", "fp32"]), step=_log(rng, 1, 100000))


def _sizes(case):
    """Tokens of each expert: uneven, the last of several has none."""
    r = random.Random(case["cut"])
    e, n = case["experts"], case["rows"]
    share = [math.exp(case["spread"] * r.gauss(0, 1)) for _ in range(e)]
    if e > 2:
        share[-1] = 0.0
    total, at, used = sum(share), 0.0, 0
    sizes = []
    for s in share:
        at += s
        end = int(round(n * at / total))
        sizes.append(end - used)
        used = end
    return sizes


def _numels(case):
    """Elements of each tensor: some of `most`, the others of up to `small`."""
    r = random.Random(case["cut"])
    out = [case["most"]] * case["big"] + [r.randint(1, case["small"]) for _ in range(case["tensors"] - case["big"])]
    r.shuffle(out)
    return out


def work(case):
    if case["op"] == "experts":
        s, e, t = SIZE[case["dtype"]], case["experts"], case["rows"]
        c, o, live = case["cols"], case["out"], sum(1 for n in _sizes(case) if n)
        every = t + case["behind"]
        flops = 2 * t * c * o
        if case["dir"] == "forward":
            return {"bytes": s * (t * c + live * c * o + every * o), "flops": flops}
        if case["dir"] == "input":
            return {"bytes": s * (t * o + live * c * o + every * c), "flops": flops}
        return {"bytes": s * t * (c + o) + e * c * o * SIZE[case["odtype"]] * (2 if case["add"] else 1), "flops": flops}
    if case["op"] == "matmul8":
        r, c, o = case["rows"], case["cols"], case["out"]
        kb = -(-c // BLOCK)
        return {"bytes": r * c + r * kb + o * c + kb * -(-o // BLOCK) + r * o * SIZE[case["odtype"]], "flops": 2 * r * c * o}
    if case["op"] == "weight8":
        c, o = case["cols"], case["out"]
        blocks = -(-c // BLOCK) * -(-o // BLOCK)
        # read once, two sets of codes written, read and their values written once each
        return {"bytes": c * o * (SIZE[case["dtype"]] * 3 + 4) + 3 * blocks, "flops": 6 * c * o}
    n = sum(_numels(case))
    blocks = sum(-(-k // BLOCK) for k in _numels(case))
    # the step reads and writes p, two codes and their scales and reads g; the states' values are then read and written
    return {"bytes": n * (2 * SIZE[case["dtype"]] + SIZE[case["gdtype"]] + 4) + 4 * blocks + n * (2 + 4) + 2 * blocks,
            "flops": 20 * n}


# ------------------------------------------------------------------ inputs
def _activation(randn, rand, rows, cols):
    """Hidden activations: unit scale, a spread between channels, a few channels far above the rest."""
    gain = torch.exp(0.5 * randn(cols))
    return randn(rows, cols) * torch.where(rand(cols) < 0.004, gain * 30.0, gain)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    st = dict(case=case)
    if case["op"] == "experts":
        e, t, c, o, dt = case["experts"], case["rows"] + case["behind"], case["cols"], case["out"], DT[case["dtype"]]
        sizes = _sizes(case)
        at = [0]
        for n in sizes:
            at.append(at[-1] + n)
        st.update(offsets=torch.tensor(at, dtype=torch.int32, device="cuda"), longest=max(sizes))
        if case["dir"] != "weight":
            st.update(w=(randn(e, o, c) / math.sqrt(c)).to(dt))
        if case["dir"] != "input":
            st.update(x=_activation(randn, rand, t, c).to(dt))
        if case["dir"] != "forward":
            st.update(dy=(1e-2 * randn(t, o)).to(dt))
        if case["add"]:
            st.update(so_far=(1e-1 * randn(e, o, c)).to(DT[case["odtype"]]))
    elif case["op"] == "matmul8":
        r, c, o = case["rows"], case["cols"], case["out"]
        kb, ob, r16 = -(-c // BLOCK), -(-o // BLOCK), -(-r // 16) * 16
        codes, scales = _encode(_activation(randn, rand, r, c))
        wcodes, wscales = _encode_weight(randn(o, c) / math.sqrt(c))
        # as the framework hands them out: rows of whole 128-column blocks, scales block by block over the tokens
        wide = torch.zeros(r, kb * BLOCK, device="cuda", dtype=torch.float8_e4m3fn)
        wide[:, :c] = codes
        tall = torch.zeros(kb, r16, device="cuda", dtype=torch.uint8)
        tall[:, :r] = scales.t()
        wwide = torch.zeros(o, kb * BLOCK, device="cuda", dtype=torch.float8_e4m3fn)
        wwide[:, :c] = wcodes
        st.update(codes=wide[:, :c], scales=tall[:, :r], wcodes=wwide[:, :c], wscales=wscales)
    elif case["op"] == "weight8":
        w = randn(case["out"], case["cols"]) / math.sqrt(case["cols"])
        st.update(w=(w * torch.exp(0.3 * randn(case["out"], 1))).to(DT[case["dtype"]]))
    else:
        # fp32 norm weights and embeddings of unit scale, bf16 weights of 0.02; gradients that differ in size from tensor
        # to tensor
        st.update(p=[], g=[], m=[], r=[], ms=[], rs=[])
        for n in _numels(case):
            size = 10.0 ** (-4 + 2 * float(torch.rand((), generator=torch.Generator().manual_seed(seed + n))))
            grad = size * randn(n)
            st["p"].append((randn(n) * (1.0 if case["dtype"] == "fp32" else 0.02)).to(DT[case["dtype"]]))
            st["g"].append(grad.to(DT[case["gdtype"]]))
            m, ms = _encode(0.3 * size * randn(n)[None])
            r, rs = _encode_root((size * (0.7 + 0.6 * rand(n)))[None], torch.full((1, n), 128, dtype=torch.int64, device="cuda"))
            st["m"].append(m[0])
            st["ms"].append(ms[0])
            st["r"].append(r[0])
            st["rs"].append(rs[0])
    return st


# ------------------------------------------------------------- plain forms
def _experts(st):
    """Each expert's tokens as one row of a padded batch, all products at once."""
    case, at = st["case"], st["offsets"].long()
    e, longest = case["experts"], st["longest"]
    place = at[:-1, None] + torch.arange(longest, device="cuda")            # [experts, longest]
    live = place < at[1:, None]

    def grouped(t):
        return torch.where(live[..., None], t.float()[place.clamp(max=t.shape[0] - 1)], torch.zeros((), device="cuda"))

    def flat(t, like):
        out = torch.zeros(like.shape[0], t.shape[-1], device="cuda")
        out[place[live]] = t[live]
        return out.to(like.dtype)

    if case["dir"] == "forward":
        return flat(torch.matmul(grouped(st["x"]), st["w"].float().transpose(1, 2)), st["x"])
    if case["dir"] == "input":
        return flat(torch.matmul(grouped(st["dy"]), st["w"].float()), st["dy"])
    if longest == 0:
        dw = torch.zeros(e, case["out"], case["cols"], device="cuda")
    else:
        dw = torch.matmul(grouped(st["dy"]).transpose(1, 2), grouped(st["x"]))
    return (st["so_far"].float() + dw if case["add"] else dw).to(DT[case["odtype"]])


def _power(scales):
    """2^(scale - 127) in fp32 from its bits (255: infinity)."""
    return (scales.to(torch.int32) << 23).view(torch.float32)


def _scale_of(top, largest, half):
    """Byte of the smallest power of two, at least 2^-111, that brings `top` to `largest` = half * 2^8 or less; 255 for
    what is not finite."""
    m, e = torch.frexp(top)                                                  # top = m 2^e, 0.5 <= m < 1
    e = torch.where(m <= half, e, e + 1).to(torch.int32) - int(math.log2(largest / half)) + 127
    e = torch.where(top == 0, torch.full_like(e, 16), e.clamp(min=16))
    return torch.where(torch.isfinite(top), e, torch.full_like(e, 255)).to(torch.uint8)


def _unit(scales):
    """What values are multiplied by before they are coded: 2^(127 - scale), 0 for 255."""
    s = scales.to(torch.int32)
    return torch.where(s == 255, torch.zeros((), device="cuda"), ((254 - s).clamp(min=0) << 23).view(torch.float32))


def _times(x, unit):
    """x unit, and 0 where unit is (x may be infinite or NaN there)."""
    return torch.where(unit == 0, torch.zeros((), device="cuda"), x * unit)


def _encode(x):
    """e4m3 codes [rows, cols] and scale bytes [rows, blocks of 128 columns]."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    xb = torch.nn.functional.pad(x.float(), (0, blocks * BLOCK - cols)).view(rows, blocks, BLOCK)
    s = _scale_of(xb.abs().amax(-1), E4M3_MAX, 0.875)
    return _times(xb, _unit(s)[..., None]).to(torch.float8_e4m3fn).view(rows, blocks * BLOCK)[:, :cols], s


def _spread(scales, rows, cols):
    """[column blocks, row blocks] values for every element of [rows, cols]."""
    return scales.t().repeat_interleave(BLOCK, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]


def _encode_weight(w):
    """e4m3 codes [out, cols] and scale bytes [column blocks, row blocks], one for 128 x 128."""
    o, c = w.shape
    kb, ob = -(-c // BLOCK), -(-o // BLOCK)
    w = w.float()
    wb = torch.nn.functional.pad(w, (0, kb * BLOCK - c, 0, ob * BLOCK - o)).view(ob, BLOCK, kb, BLOCK)
    s = _scale_of(wb.abs().amax(3).amax(1).t(), E4M3_MAX, 0.875)
    return _times(w, _spread(_unit(s), o, c)).to(torch.float8_e4m3fn), s


def _matmul8(st):
    case = st["case"]
    r, c, o = case["rows"], case["cols"], case["out"]
    x = st["codes"].float() * _power(st["scales"]).t().repeat_interleave(BLOCK, 1)[:, :c]
    w = st["wcodes"].float() * _spread(_power(st["wscales"]), o, c)
    return torch.matmul(x, w.t()).to(DT[case["odtype"]])


def _weight8(st):
    """The stored weight's values, from its codes and from those of its transpose."""
    o, c = st["w"].shape
    codes, s = _encode_weight(st["w"])
    value = (codes.float() * _spread(_power(s), o, c)).to(st["w"].dtype)
    return value, value.t(), s


def _noise(n, seed):
    """A byte for each element: the bytes, lowest first, of a 32-bit hash of (element / 4 + seed * 0x9E3779B1)."""
    low = 0xFFFFFFFF
    x = (torch.arange(-(-n // 4), device="cuda") + (seed * 0x9E3779B1 & low)) & low
    x = ((x ^ (x >> 16)) * 0x7FEB352D) & low
    x = ((x ^ (x >> 15)) * 0x846CA68B) & low
    x = x ^ (x >> 16)
    return ((x[:, None] >> torch.arange(0, 32, 8, device="cuda")) & 255).flatten()[:n]


def _encode_root(r, noise):
    """Codes and scale bytes of values that are not negative, in blocks of 128.  Code c > 0 stands for (1 + (c & 15) / 16)
    2^((c >> 4) - 8), 0 for 0; a value is rounded up where what it has past its code is at least 1 - (noise + 0.5) / 256 of
    the step.  What is not 0 gets code 1 at least."""
    rows, n = r.shape
    blocks = -(-n // BLOCK)
    rb = torch.nn.functional.pad(r, (0, blocks * BLOCK - n)).view(rows, blocks, BLOCK)
    s = _scale_of(rb.amax(-1), ROOT_MAX, 0.96875)
    y = _times(rb, _unit(s)[..., None])
    bits = y.view(torch.int32) + torch.nn.functional.pad((noise << 11) + 0x400, (0, blocks * BLOCK - n)).view(rows, blocks, BLOCK)
    code = torch.where(y > 0, ((bits >> 19) - 1904).clamp(1, 255), torch.zeros((), dtype=torch.int64, device="cuda"))
    return code.to(torch.uint8).view(rows, blocks * BLOCK)[:, :n], s


def _encode_average(x, noise):
    """e4m3 codes and scale bytes of a flat tensor in blocks of 128, magnitudes rounded by the same rule."""
    n = x.numel()
    xb = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
    s = _scale_of(xb.abs().amax(-1), E4M3_MAX, 0.875)
    y = _times(xb.abs(), _unit(s)[:, None])
    low = y < 2.0 ** -6                                                      # one step below: 2^-9
    bits = torch.where(low, y + 2.0 ** -6, y).view(torch.int32)
    bits = bits + torch.nn.functional.pad((noise << 12) + 0x800, (0, -n % BLOCK)).view(-1, BLOCK)
    code = torch.where(low, (bits >> 20) - 968, (bits >> 20) - 960).clamp(max=0x7E)
    code = torch.where(xb < 0, code + 128, code).to(torch.uint8)
    return code.view(-1)[:n].view(torch.float8_e4m3fn), s


def _each(scales, n):
    return _power(scales).repeat_interleave(BLOCK)[:n]


def _root(codes, scales):
    c = codes.to(torch.int32)
    value = ((c << 19) + (119 << 23)).view(torch.float32)
    return torch.where(c == 0, torch.zeros((), device="cuda"), value) * _each(scales, c.numel())


def _adamw8_one(p, g, m, ms, r, rs, step, noise):
    n, gf = p.numel(), g.float()
    avg = m.float() * _each(ms, n)
    avg = avg + (1.0 - ADAM["beta1"]) * (gf - avg)
    sq = _root(r, rs).square()
    root = torch.sqrt(sq + (1.0 - ADAM["beta2"]) * (gf * gf - sq))
    size = ADAM["lr"] * math.sqrt(1.0 - ADAM["beta2"] ** step) / (1.0 - ADAM["beta1"] ** step)
    p.copy_(p.float() * (1.0 - ADAM["lr"] * ADAM["wd"]) - size * avg / (ADAM["eps"] + root))
    new_m, new_ms = _encode_average(avg, noise)
    new_r, new_rs = _encode_root(root[None], noise[None])
    m.copy_(new_m)
    ms.copy_(new_ms)
    r.copy_(new_r[0])
    rs.copy_(new_rs[0])
    return p, (m.float() * _each(ms, n)).bfloat16(), _root(r, rs).bfloat16()


def _adamw8(st):
    step = st["case"]["step"]
    return [_adamw8_one(p, g, m, ms, r, rs, step, _noise(p.numel(), step))
            for p, g, m, ms, r, rs in zip(*(st[k] for k in ("p", "g", "m", "ms", "r", "rs")))]


def _plain(st):
    return {"experts": _experts, "matmul8": _matmul8, "weight8": _weight8, "adamw8": _adamw8}[st["case"]["op"]](st)


def run(st):
    if not own:
        return _plain(st)
    import newton_schulz_orthogonalized_muon_gb300 as muon
    case = st["case"]
    if case["op"] == "experts":
        if case["dir"] == "forward":
            return muon.expert_matmul(st["x"], st["w"], st["offsets"])
        if case["dir"] == "input":
            return muon.expert_matmul(st["dy"], st["w"], st["offsets"], transpose=True)
        return muon.expert_weight_grad(st["dy"], st["x"], st["offsets"], add=st.get("so_far"), dtype=DT[case["odtype"]])
    if case["op"] == "matmul8":
        return muon.act8_matmul(st["codes"], st["scales"], st["wcodes"], st["wscales"], dtype=DT[case["odtype"]])
    if case["op"] == "weight8":
        codes, scales, codes_t = muon.act8_store_weight(st["w"], transposed=True)
        dtype = st["w"].dtype
        return (muon.act8_restore_weight(codes, scales, dtype=dtype),
                muon.act8_restore_weight(codes_t, scales.t(), dtype=dtype), scales)
    states = [muon.Adamw8State(*s) for s in zip(st["m"], st["r"], st["ms"], st["rs"])]
    muon.adamw8_step(st["p"], st["g"], states, step=case["step"], **ADAM)
    return [(p, *values) for p, values in zip(st["p"], muon.adamw8_restore(states, dtype=torch.bfloat16))]


# ------------------------------------------------- the definitions, 64 bits
def _nearest_e4m3(u):
    """u rounded to the grid of e4m3: steps of 2^(max(floor(log2 |u|), -6) - 3)."""
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(u.abs(), min=1e-300))), min=-6.0) - 3.0)
    return torch.round(u / step) * step


def _exponent(top, largest):
    """The smallest whole e >= -111 with top 2^-e <= largest."""
    e = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / largest))
    e = torch.where(top * torch.exp2(-e) > largest, e + 1, e)
    return torch.clamp(torch.where(top * torch.exp2(-(e - 1)) <= largest, e - 1, e), min=-111.0)


def _blocks_of(t):
    """[blocks, 128] of a flat tensor, zeros behind it."""
    full = torch.zeros(-(-t.numel() // BLOCK) * BLOCK, dtype=t.dtype, device=t.device)
    full[:t.numel()] = t
    return full.view(-1, BLOCK)


def _exact_adamw8(st, case):
    out = []
    b1, b2 = ADAM["beta1"], ADAM["beta2"]
    for p, g, mc, ms, rc, rs in zip(st["p"], st["g"], st["m"], st["ms"], st["r"], st["rs"]):
        n = p.numel()
        m = (_blocks_of(mc.double()) * torch.exp2(ms.double() - 127).unsqueeze(1)).view(-1)[:n]
        c = rc.double()
        high = torch.floor(c / 16)
        r = torch.where(c == 0, 0.0, (1 + (c - 16 * high) / 16) * torch.exp2(high - 8))
        r = (_blocks_of(r) * torch.exp2(rs.double() - 127).unsqueeze(1)).view(-1)[:n]
        gd = g.double()
        m = b1 * m + (1 - b1) * gd
        v = b2 * r * r + (1 - b2) * gd * gd
        new = p.double() * (1 - ADAM["lr"] * ADAM["wd"])
        new -= ADAM["lr"] * (1 - b2 ** case["step"]) ** 0.5 / (1 - b1 ** case["step"]) * m / (v ** 0.5 + ADAM["eps"])
        mb, rb = _blocks_of(m), _blocks_of(v ** 0.5)
        # the hash, 32 bits at a time in halves of 16
        x = (torch.arange(mb.numel() // 4, device=p.device) + case["step"] * 2654435761) % 2 ** 32
        for shift, factor in ((16, 2146121005), (15, 2221713035)):
            x = torch.bitwise_xor(x, x // 2 ** shift)
            x = ((x % 65536) * factor + ((x // 65536) * (factor % 65536) % 65536) * 65536) % 2 ** 32
        x = torch.bitwise_xor(x, x // 65536)
        noise = torch.stack([x // 256 ** k % 256 for k in range(4)], 1).view(mb.shape).double()
        unit = torch.exp2(_exponent(mb.abs().amax(1, keepdim=True), E4M3_MAX))
        y = mb.abs() / unit
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(y, min=1e-300))), min=-6.0) - 3)
        kept = torch.clamp(torch.floor(y / step + (noise + 0.5) / 256) * step, max=E4M3_MAX)
        kept = (torch.where(mb < 0, -kept, kept) * unit).view(-1)[:n]
        unit = torch.exp2(_exponent(rb.amax(1, keepdim=True), ROOT_MAX))
        y = rb / unit
        step = torch.exp2(torch.floor(torch.log2(torch.clamp(y, min=1e-300))) - 4)
        coded = torch.floor(y / step + (noise + 0.5) / 256) * step
        coded = torch.where(y == 0, 0.0, torch.clamp(coded, min=1.0625 / 256, max=ROOT_MAX))
        out.append((new, kept, (coded * unit).view(-1)[:n]))
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "experts":
        e, t, at = case["experts"], case["rows"] + case["behind"], st["offsets"].tolist()
        if case["dir"] == "weight":
            dw = torch.zeros(e, case["out"], case["cols"], dtype=torch.float64, device="cuda")
            for i, (a, b) in enumerate(zip(at, at[1:])):
                dw[i] = st["dy"][a:b].double().T @ st["x"][a:b].double()
            return dw + st["so_far"].double() if case["add"] else dw
        given = st["x" if case["dir"] == "forward" else "dy"].double()
        y = torch.zeros(t, case["out" if case["dir"] == "forward" else "cols"], dtype=torch.float64, device="cuda")
        for i, (a, b) in enumerate(zip(at, at[1:])):
            y[a:b] = given[a:b] @ (st["w"][i].double().T if case["dir"] == "forward" else st["w"][i].double())
        return y
    if case["op"] == "matmul8":
        r, c, o = case["rows"], case["cols"], case["out"]
        total = torch.zeros(r, o, dtype=torch.float64, device="cuda")
        for k in range(-(-c // BLOCK)):
            a = st["codes"][:, k * BLOCK:(k + 1) * BLOCK].double() * torch.exp2(st["scales"][k].double() - 127)[:, None]
            b = st["wcodes"][:, k * BLOCK:(k + 1) * BLOCK].double()
            unit = torch.exp2(st["wscales"][k].double() - 127)
            total += a @ (b * unit[torch.arange(o, device="cuda") // BLOCK][:, None]).T
        return total
    if case["op"] == "weight8":
        w = st["w"].double()
        value = torch.empty_like(w)
        for i in range(0, w.shape[0], BLOCK):
            for j in range(0, w.shape[1], BLOCK):
                part = w[i:i + BLOCK, j:j + BLOCK]
                unit = torch.exp2(_exponent(part.abs().amax(), E4M3_MAX))
                value[i:i + BLOCK, j:j + BLOCK] = _nearest_e4m3(part / unit) * unit
        return value, value.T, None
    return _exact_adamw8(st, case)
