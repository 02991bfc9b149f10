"""The training operators on the GPU against their plain 64-bit forms.

Tolerances, element by element.  u is the unit roundoff of the storage type:
2^-8 for bf16 (8 significant bits), 2^-11 for fp16, 2^-24 for fp32.
  * One rounding to the output type: u |ref|.
  * Attention forms p (and ds) in fp32 and rounds it once to the operand type
    before the second product, so a sum of products is off by at most
    u sum |p||v|.  fp32 arithmetic before that (a dot product of up to 128
    products, an exponential of an argument below 2^8, the difference dP -
    delta) stays below 2^-15 of the terms' magnitudes.
  * Layer norm: fp32 sums of up to 16384 terms held in partial sums of at
    most a few dozen: 2^-19 of the terms' magnitudes; sums over rows 2^-18.
  * The weight gradient multiplies exact bf16 factors and sums in fp32, 16
    products at a time: (rows / 16 + 16) 2^-23 of the terms' magnitudes.
"""
import ctypes
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from _margins import record
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def muon():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import newton_schulz_orthogonalized_muon_gb300 as pkg
    torch.cuda.set_device(0)
    return pkg


def host(t):
    return t.detach().double().cpu().numpy()


def rand(seed, *shape, dtype=FP, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def close(name, got, ref, tol):
    """|got - ref| <= tol element by element; where ref is not finite, got is the same."""
    got, ref = host(got) if isinstance(got, torch.Tensor) else got, np.asarray(ref)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine], ref[~fine], equal_nan=True), name
    tol = np.broadcast_to(np.maximum(tol, 1e-30), ref.shape)
    ratio = float(np.max(np.abs(got[fine] - ref[fine]) / tol[fine], initial=0.0))
    record(name, ratio, 1.0)
    assert ratio <= 1.0, (name, ratio)


# ---------------------------------------------------------------- layer norm
NORM = [  # rows, cols, pad, dtype, wdtype
    (1, 1, 0, FP, FP), (3, 7, 0, BF, FP), (5, 256, 0, BF, BF), (9, 257, 0, HF, FP), (4, 768, 0, BF, FP),
    (33, 1023, 6, FP, FP), (2, 1024, 0, HF, HF), (7, 2048, 8, BF, FP), (3, 4096, 0, BF, BF), (611, 4096, 0, BF, FP),
    (2, 5000, 0, FP, FP), (3, 8192, 0, BF, FP), (3, 9001, 3, BF, FP), (5, 16384, 0, BF, FP), (2, 16384, 0, FP, FP),
    (1301, 33, 0, BF, FP), (700, 1000, 0, HF, FP), (0, 64, 0, BF, FP)]


@pytest.mark.parametrize("rows,cols,pad,dtype,wdtype", NORM)
def test_layer_norm(muon, rows, cols, pad, dtype, wdtype):
    x = (rand(1, rows, cols + pad) * 3 + 5).to(dtype)[:, :cols]
    dy = rand(2, rows, cols + pad, dtype=dtype)[:, :cols]
    w, b = (1 + rand(3, cols) * 0.3).to(wdtype), rand(4, cols, dtype=wdtype)
    y, mean, rstd = muon.layer_norm(x, w, b, eps=1e-5)
    dx, dw, db = muon.layer_norm_backward(dy, x, mean, rstd, w)
    assert y.dtype == dx.dtype == dtype and dw.dtype == db.dtype == FP
    xd, dyd, wd, bd = host(x), host(dy), host(w), host(b)
    yr, mr, rr = oo.layer_norm(xd, wd, bd, 1e-5) if rows else (np.zeros((0, cols)), np.zeros(0), np.zeros(0))
    tag = f"layer norm {rows}x{cols} {dtype}"
    e = 2.0 ** -19
    xmag = np.abs(xd).mean(1) if rows else np.zeros(0)
    close(tag + " mean", mean, mr, e * xmag)
    # the mean's error shifts every x - mean; relative to the spread it enters rstd squared
    off = e * xmag * rr
    close(tag + " rstd", rstd, rr, rr * (e + off * off + e * np.abs(xd).max(1, initial=0) * rr))
    xh = np.abs(xd - mr[:, None]) * rr[:, None]
    inner = off[:, None] + (e + (e * np.abs(xd).max(1, initial=0) * rr)[:, None]) * xh
    close(tag + " y", y, yr, U[dtype] * np.abs(yr) + inner * np.abs(wd) + e * (xh * np.abs(wd) + np.abs(bd)))
    # the backward pass takes the mean and rstd that it is given
    md, rd = host(mean), host(rstd)
    dxr, dwr, dbr = oo.layer_norm_backward(dyd, xd, md, rd, wd) if rows else (np.zeros((0, cols)), np.zeros(cols),
                                                                              np.zeros(cols))
    g = np.abs(dyd * wd)
    xh = (np.abs(xd) + np.abs(md)[:, None]) * rd[:, None]
    xt = np.abs(xd - md[:, None]) * rd[:, None]
    mag = rd[:, None] * (g + (g.mean(1, keepdims=True) if rows else 0)
                         + xh * ((g * xt).mean(1, keepdims=True) if rows else 0)
                         + xt * ((g * xh).mean(1, keepdims=True) if rows else 0))
    close(tag + " dx", dx, dxr, U[dtype] * np.abs(dxr) + e * mag)
    close(tag + " dw", dw, dwr, 2.0 ** -18 * (np.abs(dyd) * xh).sum(0))
    close(tag + " db", db, dbr, 2.0 ** -18 * np.abs(dyd).sum(0))


def test_layer_norm_without_weights_and_in_more_dimensions(muon):
    x = rand(5, 3, 4, 96, dtype=BF)
    y, mean, rstd = muon.layer_norm(x)
    assert y.shape == x.shape and mean.shape == rstd.shape == (3, 4)
    yr, _, _ = oo.layer_norm(host(x).reshape(12, 96), np.ones(96), np.zeros(96), 1e-5)
    close("layer norm plain", y.reshape(12, 96), yr, U[BF] * np.abs(yr) + 2.0 ** -17)
    dx, dw, db = muon.layer_norm_backward(x, x, mean, rstd)
    assert dx.shape == x.shape
    t = x.transpose(0, 1)                       # rows without one stride: copied
    assert torch.equal(muon.layer_norm(t)[0], y.transpose(0, 1))
    assert torch.equal(muon.layer_norm_backward(t, t, mean.t().contiguous(), rstd.t().contiguous())[0],
                       dx.transpose(0, 1))


def test_layer_norm_far_mean_does_not_cancel(muon):
    x = rand(6, 8, 1000) + 4096.0
    y, mean, rstd = muon.layer_norm(x)
    yr, _, rr = oo.layer_norm(host(x), 1.0, 0.0, 1e-5)
    # x - mean is exact to the mean's own rounding (half an ulp of 4096)
    close("far mean y", y, yr, 2.0 ** -12 + 2.0 ** -10 * np.abs(yr))
    close("far mean rstd", rstd, rr, 2.0 ** -18 * rr)


def test_layer_norm_gradient_against_differences(muon):
    x, w, b, g = rand(7, 4, 24), 1 + rand(8, 24) * 0.2, rand(9, 24), rand(10, 4, 24)
    _, mean, rstd = muon.layer_norm(x, w, b)
    dx, dw, db = muon.layer_norm_backward(g, x, mean, rstd, w)
    gd, h = host(g), 1e-6

    def loss(xx, ww, bb):
        return (oo.layer_norm(xx, ww, bb, 1e-5)[0] * gd).sum()
    args = [host(x), host(w), host(b)]
    for i, got in enumerate((dx, dw, db)):
        num = np.zeros(args[i].size)
        for j in range(args[i].size):
            up, dn = [a.copy() for a in args], [a.copy() for a in args]
            up[i].flat[j] += h
            dn[i].flat[j] -= h
            num[j] = (loss(*up) - loss(*dn)) / (2 * h)
        close(f"layer norm difference {i}", got, num.reshape(args[i].shape), np.full(args[i].shape, 2e-5))


def test_layer_norm_nan_stays_in_its_row(muon):
    x = rand(11, 5, 512, dtype=BF)
    want = muon.layer_norm(x)[0]
    x[2, 7] = float("nan")
    got = muon.layer_norm(x)[0]
    assert got[2].isnan().all() and torch.equal(got[[0, 1, 3, 4]], want[[0, 1, 3, 4]])


@pytest.mark.parametrize("cols", [512, 513])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_layer_norm_statistics_of_a_row_that_is_not_finite(muon, cols, value):
    x = rand(12, 3, cols, dtype=BF)
    x[1, 5] = value
    _, mean, rstd = muon.layer_norm(x)
    assert mean[1].isnan() and rstd[1].isnan()
    assert mean[[0, 2]].isfinite().all() and rstd[[0, 2]].isfinite().all()


# ----------------------------------------------------------------- attention
ATTN = [  # batch, sq, sk, heads, kv_heads, dim, causal, window, dtype
    (1, 1, 1, 1, 1, 8, True, 0, BF), (2, 61, 61, 3, 3, 64, True, 0, BF), (1, 128, 128, 2, 1, 128, True, 0, BF),
    (1, 129, 129, 4, 1, 128, True, 0, HF), (1, 127, 257, 2, 2, 64, False, 0, BF), (2, 300, 300, 4, 2, 128, True, 0, HF),
    (1, 1, 517, 4, 2, 128, True, 0, BF), (1, 517, 1, 2, 2, 64, False, 0, BF), (1, 200, 70, 2, 1, 64, True, 0, BF),
    (1, 70, 333, 2, 1, 40, True, 0, HF), (2, 260, 260, 2, 2, 72, True, 1, BF), (1, 400, 400, 2, 1, 128, True, 130, BF),
    (1, 513, 600, 1, 1, 96, True, 37, BF), (1, 300, 200, 1, 1, 64, True, 20, HF), (1, 640, 640, 2, 2, 64, True, 0, BF),
    (3, 65, 63, 2, 2, 24, False, 0, HF), (1, 256, 0, 2, 2, 64, False, 0, BF), (1, 1030, 1030, 1, 1, 128, False, 0, BF),
    (1, 5, 900, 8, 1, 120, True, 0, BF)]


def attn_tol(u, ref, mag, wide=None):
    return u * np.abs(ref) + (1.02 * u) * mag + 2.0 ** -15 * (mag if wide is None else wide)


def check_attention(tag, dtype, scale, causal, window, spans, q, k, v, do, o, lse, grads):
    """spans: (batch index or None, q0, q1, k0, k1) of each sequence."""
    qd, kd, vd, dod, od, ld = (host(t) for t in (q, k, v, do, o, lse))
    dq, dk, dv = (host(t) for t in grads)
    u = U[dtype]
    for n, (b, q0, q1, k0, k1) in enumerate(spans):
        at = (lambda t, i0, i1: t[i0:i1]) if b is None else (lambda t, i0, i1: t[b, i0:i1])
        ls = ld[:, q0:q1] if b is None else ld[b]
        qs, ks, vs, gs, os_ = at(qd, q0, q1), at(kd, k0, k1), at(vd, k0, k1), at(dod, q0, q1), at(od, q0, q1)
        ref, lr, mag = oo.attention(qs, ks, vs, causal, window, scale)
        close(f"{tag} o {n}", os_, ref, attn_tol(u, ref, mag))
        smag = np.abs(np.where(np.isfinite(lr), lr, 0)) + 1
        close(f"{tag} lse {n}", ls, lr, 2.0 ** -17 * smag)
        refs, mags, wides = oo.attention_backward(gs, qs, ks, vs, os_, causal, window, scale)
        for name, got, r, m, wd in zip(("dq", "dk", "dv"), (at(dq, q0, q1), at(dk, k0, k1), at(dv, k0, k1)), refs,
                                       mags, wides):
            close(f"{tag} {name} {n}", got, r, attn_tol(u, r, m, wd))


@pytest.mark.parametrize("batch,sq,sk,heads,kv,dim,causal,window,dtype", ATTN)
def test_attention(muon, batch, sq, sk, heads, kv, dim, causal, window, dtype):
    q, k, v = rand(20, batch, sq, heads, dim, dtype=dtype), rand(21, batch, sk, kv, dim, dtype=dtype), \
        rand(22, batch, sk, kv, dim, dtype=dtype)
    do = rand(23, batch, sq, heads, dim, dtype=dtype)
    kw = dict(causal=causal, window=window)
    o, lse = muon.attention(q, k, v, **kw)
    grads = muon.attention_backward(do, q, k, v, o, lse, **kw)
    assert muon.default_handle().check() == 0
    spans = [(b, 0, sq, 0, sk) for b in range(batch)]
    check_attention(f"attention {sq}x{sk} h{heads}/{kv} d{dim} {dtype}", dtype, dim ** -0.5, causal, window, spans, q,
                    k, v, do, o, lse, grads)
    # the same call again: the same bits
    assert torch.equal(o, muon.attention(q, k, v, **kw)[0])
    for a, b in zip(grads, muon.attention_backward(do, q, k, v, o, lse, **kw)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("batch,seq,heads,dim,window", [
    (8, 1024, 16, 128, 0), (8, 1024, 12, 64, 0), (70, 130, 16, 128, 0), (90, 65, 16, 64, 0), (9, 700, 16, 128, 150)])
def test_attention_of_many_items(muon, batch, seq, heads, dim, window):
    """More work items than CTAs: a head is computed as it is alone."""
    q, k, v, do = (rand(24 + i, batch, seq, heads, dim, dtype=BF) for i in range(4))
    kw = dict(causal=True, window=window)
    o, lse = muon.attention(q, k, v, **kw)
    grads = muon.attention_backward(do, q, k, v, o, lse, **kw)
    assert muon.default_handle().check() == 0
    for b, h in ((0, 0), (batch // 2, heads - 1), (batch - 1, 3)):
        at = (slice(b, b + 1), slice(None), slice(h, h + 1))
        one, one_lse = muon.attention(q[at], k[at], v[at], **kw)
        assert torch.equal(one, o[at]) and torch.equal(one_lse, lse[b:b + 1, h:h + 1])
        for a, g in zip(muon.attention_backward(do[at], q[at], k[at], v[at], one, one_lse, **kw), grads):
            assert torch.equal(a, g[at])
    b, h = batch - 1, slice(1, 2)
    check_attention(f"attention {batch}x{seq} h{heads} d{dim}", BF, dim ** -0.5, True, window, [(0, 0, seq, 0, seq)],
                    *(t[b:, :, h] for t in (q, k, v, do, o)), lse[b:, h], [g[b:, :, h] for g in grads])


@pytest.mark.parametrize("lengths", [
    [1, 107, 429, 532, 881, 175, 906, 40, 575, 54, 246, 96, 128, 14, 256, 1735, 58, 0, 501],
    [30 * (i % 7) + i for i in range(75)], [3] * 31, [200] * 32])
def test_packed_documents_of_many_items(muon, lengths):
    cuts = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    q, k, v, do = (rand(28 + i, cuts[-1], 16, 128, dtype=HF) for i in range(4))
    cu = torch.tensor(cuts, dtype=torch.int32).cuda()
    kw = dict(causal=True, cu_seqlens_q=cu, cu_seqlens_k=cu)
    o, lse = muon.attention(q, k, v, **kw)
    grads = muon.attention_backward(do, q, k, v, o, lse, **kw)
    assert muon.default_handle().check() == 0
    for a, b in zip(cuts, cuts[1:]):
        if a == b:
            continue
        at = (slice(a, b), slice(5, 7))
        one, one_lse = muon.attention(*(t[at][None] for t in (q, k, v)), causal=True)
        assert torch.equal(one[0], o[at]) and torch.equal(one_lse[0], lse[5:7, a:b])
        for x, g in zip(muon.attention_backward(*(t[at][None] for t in (do, q, k, v)), one, one_lse, causal=True), grads):
            assert torch.equal(x[0], g[at])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cuts_q,cuts_k", [
    ([0, 0, 1, 130, 130, 386, 391, 647], None), ([0, 300], None), ([0, 5, 135, 140], [0, 200, 210, 210]),
    ([0, 64, 64, 128], [0, 0, 30, 300])])
def test_packed_attention(muon, causal, cuts_q, cuts_k):
    cuts_k = cuts_q if cuts_k is None else cuts_k
    h, kv, d, dtype = 4, 2, 64, BF
    fused = rand(30, max(cuts_q[-1], cuts_k[-1]), h + 2 * kv, d, dtype=dtype)
    q, k, v = fused[:cuts_q[-1], :h], fused[:cuts_k[-1], h:h + kv], fused[:cuts_k[-1], h + kv:]
    do = rand(31, cuts_q[-1], h, d, dtype=dtype)
    kw = dict(causal=causal, cu_seqlens_q=torch.tensor(cuts_q, dtype=torch.int32).cuda(),
              cu_seqlens_k=torch.tensor(cuts_k, dtype=torch.int32).cuda())
    o, lse = muon.attention(q, k, v, **kw)
    grads = muon.attention_backward(do, q, k, v, o, lse, **kw)
    spans = [(None, *s) for s in zip(cuts_q, cuts_q[1:], cuts_k, cuts_k[1:])]
    check_attention(f"packed {cuts_q} {causal}", dtype, d ** -0.5, causal, 0, spans, q, k, v, do, o, lse, grads)


def test_packed_tokens_of_no_sequence_and_bad_offsets(muon):
    q = rand(32, 400, 2, 64, dtype=BF)
    for cuts in ([10, 200, 390], [0, 200, 100, 5000], [-7, 150, 150]):
        cu = torch.tensor(cuts, dtype=torch.int32).cuda()
        kw = dict(causal=True, cu_seqlens_q=cu, cu_seqlens_k=cu)
        o, lse = muon.attention(q, q, q, **kw)
        grads = muon.attention_backward(q, q, q, q, o, lse, **kw)
        cut = lambda c: min(max(c, 0), 400)  # noqa: E731
        spans = [(cut(a), max(cut(b), cut(a))) for a, b in zip(cuts, cuts[1:])]
        inside = torch.zeros(400, dtype=torch.bool)
        for a, b in spans:
            inside[a:b] = True
        if cuts[0] == 10:
            assert (o[~inside] == 0).all() and (lse[:, ~inside.cuda()] == -math.inf).all()
            assert all((g[~inside] == 0).all() for g in grads)
        assert all(torch.isfinite(g).all() for g in grads) and torch.isfinite(o).all()
    assert muon.default_handle().check() == 0


def test_attention_keys_past_the_end_have_no_part(muon):
    """NaN and infinity next to a sequence (rows past its end, other documents, other heads)."""
    for bad in (float("nan"), float("inf"), -float("inf")):
        big = [rand(40 + i, 2, 300, 4, 64, dtype=BF) for i in range(4)]
        q, k, v, do = (t[:, 20:181, 1:3] for t in big)
        want = [t.clone() for t in (q, k, v, do)]
        o0, l0 = muon.attention(*want[:3], causal=True)
        g0 = muon.attention_backward(want[3], *want[:3], o0, l0, causal=True)
        for t in big:
            keep = t[:, 20:181, 1:3].clone()
            t.fill_(bad)
            t[:, 20:181, 1:3] = keep
        o1, l1 = muon.attention(q, k, v, causal=True)
        g1 = muon.attention_backward(do, q, k, v, o1, l1, causal=True)
        assert torch.equal(o0, o1) and torch.equal(l0, l1) and all(torch.equal(a, b) for a, b in zip(g0, g1))
        # a document of such values beside a fine one
        cu = torch.tensor([0, 100, 161, 300], dtype=torch.int32).cuda()
        x = rand(44, 300, 2, 64, dtype=BF)
        kw = dict(causal=False, cu_seqlens_q=cu, cu_seqlens_k=cu)
        o0, l0 = muon.attention(x, x, x, **kw)
        g0 = muon.attention_backward(x, x, x, x, o0, l0, **kw)
        y = x.clone()
        y[100:161] = bad
        o1, l1 = muon.attention(y, y, y, **kw)
        g1 = muon.attention_backward(y, y, y, y, o1, l1, **kw)
        for a, b in ((o0, o1), *zip(g0, g1)):
            assert torch.equal(a[:100], b[:100]) and torch.equal(a[161:], b[161:])


@pytest.mark.parametrize("gain", [1e-4, 8.0, 40.0])
def test_attention_range_of_scores(muon, gain):
    """Scores near zero (a flat softmax) and far beyond exp's range."""
    q, k, v, do = (rand(50 + i, 1, 333, 2, 64, dtype=BF) for i in range(4))
    q = (q.float() * gain).to(BF)
    o, lse = muon.attention(q, k, v)
    ref, lr, mag = oo.attention(host(q)[0], host(k)[0], host(v)[0], False, 0, 0.125)
    # an fp32 score of magnitude s is off by up to 2^-22 s, and p by as much, relatively
    smax = np.abs(lr).max() + 1
    extra = 2.0 ** -21 * smax
    close(f"scores x{gain} o", o[0], ref, attn_tol(U[BF], ref, mag) + extra * mag)
    close(f"scores x{gain} lse", lse[0], lr, 2.0 ** -17 + 2.0 ** -21 * np.abs(lr))
    grads = muon.attention_backward(do, q, k, v, o, lse)
    refs, mags, wides = oo.attention_backward(*(host(t)[0] for t in (do, q, k, v, o)), False, 0, 0.125)
    for name, g, r, m, w in zip(("dq", "dk", "dv"), grads, refs, mags, wides):
        close(f"scores x{gain} {name}", g[0], r, attn_tol(U[BF], r, m, w) + extra * w)


def test_attention_gradient_against_differences(muon):
    """Directional differences of the 64-bit forward form."""
    q, k, v, do = (rand(60 + i, 1, 40, 2, 32, dtype=HF) for i in range(4))
    o, lse = muon.attention(q, k, v, causal=True, scale=0.2)
    grads = muon.attention_backward(do, q, k, v, o, lse, causal=True, scale=0.2)
    args, g, h = [host(t)[0] for t in (q, k, v)], host(do)[0], 1e-5
    rng = np.random.default_rng(1)
    for i in range(3):
        for _ in range(4):
            d = rng.standard_normal(args[i].shape)
            up, dn = [a.copy() for a in args], [a.copy() for a in args]
            up[i] += h * d
            dn[i] -= h * d
            num = ((oo.attention(*up, True, 0, 0.2)[0] - oo.attention(*dn, True, 0, 0.2)[0]) * g).sum() / (2 * h)
            got = (host(grads[i])[0] * d).sum()
            # o is rounded before delta, each gradient once at the end: u of the sum's magnitude, with room for
            # the roundings inside
            tol = 4 * U[HF] * (np.abs(host(grads[i])[0]) * np.abs(d)).sum() + 1e-6
            record(f"attention difference {i}", abs(got - num) / tol, 1.0)
            assert abs(got - num) <= tol


def test_attention_strided_and_expanded_operands(muon):
    qkv = rand(70, 2, 190, 3, 4, 64, dtype=BF)
    q, k, v = qkv.unbind(2)
    want = [t.contiguous() for t in (q, k, v)]
    assert torch.equal(muon.attention(q, k, v, causal=True)[0], muon.attention(*want, causal=True)[0])
    bhsd = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in want]     # heads outside tokens
    o, lse = muon.attention(*bhsd, causal=True)
    assert torch.equal(o, muon.attention(*want, causal=True)[0])
    one = torch.ones(1, 1, 1, 1, dtype=BF, device="cuda").expand(2, 190, 4, 64)   # the gradient of a sum
    a = muon.attention_backward(one, *want, o, lse, causal=True)
    b = muon.attention_backward(one.contiguous(), q, k, v, o, lse, causal=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


# --------------------------------------------------- activations in 8 bits
@pytest.mark.parametrize("rows,cols,pad,dtype", [
    (1, 1, 0, BF), (5, 127, 0, BF), (17, 128, 0, HF), (33, 129, 0, FP), (16, 768, 0, BF), (40, 1000, 24, BF),
    (21, 1001, 2, HF), (50, 513, 0, FP), (100, 256, 0, FP)])
def test_act8_codes_are_exact(muon, rows, cols, pad, dtype):
    x = (rand(80, rows, cols + pad) * torch.exp(2 * rand(81, cols + pad))).to(dtype)
    if rows > 12:
        x[2] = 0
        x[3] *= 0.0
        x[4] = x[4] * 1e-5 if dtype == HF else x[4] * 1e-37      # below the smallest scale in part
        x[5] = 448.0
        x[6] = 449.0
        x[7, :] = torch.tensor([2.0 ** -9, 3 * 2.0 ** -10, 17.0, 19.0, 448.0, -464.0, 27.0, 25.0]).to(dtype).cuda()[
            torch.arange(cols + pad) % 8]                         # midpoints between codes
        x[8, 0] = float("nan")
        x[9, cols - 1] = float("inf")
        if dtype != HF:
            x[10] *= 1e37
    x = x[:, :cols]
    codes, scales = muon.act8_store(x)
    cr, sr = oo.act8_encode(host(x))
    assert codes.dtype == torch.float8_e4m3fn and codes.shape == x.shape
    assert np.array_equal(scales.cpu().numpy(), sr)
    assert np.array_equal(codes.view(torch.uint8).cpu().numpy() & np.where(cr & 0x7F, 0xFF, 0x7F), cr & np.where(
        cr & 0x7F, 0xFF, 0x7F))                                   # the sign of a zero aside
    want = oo.act8_decode(cr, sr)
    for out in (FP, BF, HF):
        got = muon.act8_restore(codes, scales, dtype=out)
        with np.errstate(over="ignore", invalid="ignore"):
            ref = host(torch.tensor(want).to(FP).to(out))
        assert np.array_equal(host(got), ref, equal_nan=True), out


@pytest.mark.parametrize("rows,cols", [(3, 5), (17, 128), (6, 1001)])
def test_act8_writes_its_codes_and_scales_alone(muon, rows, cols):
    x = rand(83, rows, cols, dtype=BF)
    want = muon.act8_store(x)
    ldc, lds, blocks = -(-cols // 128) * 128 + 128, -(-rows // 16) * 16 + 16, -(-cols // 128)
    codes = torch.full((rows + 1, ldc), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((blocks + 1, lds), 77, dtype=torch.uint8, device="cuda")
    h = muon.default_handle()
    st = h._lib.muon_act8_store(h.ptr, x.data_ptr(), cols, codes.data_ptr(), ldc, scales.data_ptr(), lds, rows, cols,
                                muon._binding.MUON_BF16, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(codes[:rows, :cols], want[0].view(torch.uint8)) and torch.equal(scales[:blocks, :rows], want[1])
    codes[:rows, :cols] = scales[:blocks, :rows] = 77
    assert (codes == 77).all() and (scales == 77).all()


def test_act8_error_is_a_sixteenth(muon):
    x = rand(82, 64, 512, dtype=BF)
    codes, scales = muon.act8_store(x)
    back = host(muon.act8_restore(codes, scales))
    top = np.abs(host(x)).reshape(64, 4, 128).max(2).repeat(128, 1)
    # half an e4m3 step: 2^-4 of the value, or of 2^-6 of the scaled grid's smallest normal number
    assert (np.abs(back - host(x)) <= np.maximum(2.0 ** -4 * np.abs(host(x)), top * 2.0 ** -17)).all()


WGRAD = [  # rows, cols, out, odtype, add
    (1, 16, 16, FP, False), (64, 128, 128, FP, False), (65, 130, 139, FP, True), (200, 256, 256, BF, False),
    (333, 300, 511, BF, True), (1001, 512, 264, FP, True), (5000, 384, 200, FP, False), (2049, 1, 1, FP, False),
    (0, 40, 24, FP, False), (0, 40, 24, FP, True), (130, 1409, 40, FP, False)]


@pytest.mark.parametrize("rows,cols,out,odtype,add", WGRAD)
def test_act8_weight_grad(muon, rows, cols, out, odtype, add):
    x, dy = rand(83, rows, cols, dtype=BF) + 0.2, rand(84, rows, out, dtype=BF)
    codes, scales = muon.act8_store(x)
    base = rand(85, out, cols, dtype=odtype) if add else None
    got = muon.act8_weight_grad(dy, codes, scales, add=base, dtype=odtype)
    ref, mag = oo.act8_weight_grad(host(dy), host(muon.act8_restore(codes, scales, dtype=FP)))
    ref = ref + (host(base) if add else 0)
    mag = mag + (np.abs(host(base)) if add else 0)
    tol = U[odtype] * np.abs(ref) + (rows / 16 + 16) * 2.0 ** -23 * mag
    close(f"weight grad {rows}x{cols}x{out} {odtype}", got, ref, tol)
    assert torch.equal(got, muon.act8_weight_grad(dy, codes, scales, add=base, dtype=odtype))
    if add:                                      # in place
        assert muon.act8_weight_grad(dy, codes, scales, add=base, out=base) is base
        assert torch.equal(base, got)
    # other layouts of the same values
    wide = torch.zeros(rows, out + 3, dtype=BF, device="cuda")
    wide[:, :out] = dy
    dst = torch.full((out, cols + 5), 7.0, dtype=odtype, device="cuda")
    if not add:
        muon.act8_weight_grad(wide[:, :out], codes.clone(), scales.contiguous(), out=dst[:, :cols])
        assert torch.equal(dst[:, :cols], got) and (dst[:, cols:] == 7.0).all()


def test_act8_weight_grad_carries_nan(muon):
    x, dy = rand(86, 40, 256, dtype=BF), rand(87, 40, 24, dtype=BF)
    x[7, 130] = float("inf")
    dw = muon.act8_weight_grad(dy, *muon.act8_store(x))
    assert torch.isfinite(dw[:, :128]).all() and dw[:, 128:].isnan().all()


# ------------------------------------------------- streams, refusals, errors
def test_offsets_past_32_bits(muon):
    """Rows and tokens 2^30 elements apart."""
    step, n = 1 << 30, 3
    store = torch.empty((n - 1) * step + 1024, dtype=BF, device="cuda")

    def apart(t, at=0):                               # t's rows (first dimension), far from each other
        size = t.shape[1:].numel()
        view = store.as_strided((n, size), (step, 1), at)
        view.copy_(t.reshape(n, size))
        return view.view(n, *t.shape[1:])

    x, dy = rand(84, n, 256, dtype=BF), rand(85, n, 256, dtype=BF)
    y, mean, rstd = muon.layer_norm(x)
    far_x, far_dy = apart(x), apart(dy, 256)
    assert far_x.stride(0) == step
    assert torch.equal(muon.layer_norm(far_x)[0], y)
    for a, b in zip(muon.layer_norm_backward(far_dy, far_x, mean, rstd), muon.layer_norm_backward(dy, x, mean, rstd)):
        assert torch.equal(a, b)
    for a, b in zip(muon.act8_store(far_x), muon.act8_store(x)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    codes, scales = muon.act8_store(x)
    assert torch.equal(muon.act8_weight_grad(far_dy, codes, scales), muon.act8_weight_grad(dy, codes, scales))
    q, k, v, do = (rand(86 + i, n, 2, 64, dtype=BF) for i in range(4))
    o, lse = muon.attention(q[None], k[None], v[None], causal=True)
    want = muon.attention_backward(do[None], q[None], k[None], v[None], o, lse, causal=True)
    far = [apart(t, 128 * i)[None] for i, t in enumerate((q, k, v, do, o[0]))]
    assert torch.equal(muon.attention(*far[:3], causal=True)[0], o)
    for a, b in zip(muon.attention_backward(far[3], *far[:3], far[4], lse, causal=True), want):
        assert torch.equal(a, b)
    assert muon.default_handle().check() == 0


def test_operators_on_a_side_stream_and_in_a_graph(muon):
    x, dy = rand(90, 64, 512, dtype=BF), rand(91, 64, 64, dtype=BF)
    q = rand(92, 1, 200, 2, 64, dtype=BF)

    def work(stream=None):
        y, mean, rstd = muon.layer_norm(x, stream=stream)
        dx, dw, db = muon.layer_norm_backward(x, x, mean, rstd, stream=stream)
        c, s = muon.act8_store(x, stream=stream)
        w = muon.act8_weight_grad(dy, c, s, stream=stream)
        o, lse = muon.attention(q, q, q, causal=True, stream=stream)
        return [y, dx, dw, db, muon.act8_restore(c, s, stream=stream), w, o, lse,
                *muon.attention_backward(q, q, q, q, o, lse, causal=True, stream=stream)]

    want = work()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = work(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for t in held:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, held))


def test_operators_count_their_launches(muon):
    h = muon.default_handle()
    n0 = h.launch_count()
    muon.layer_norm(rand(93, 4, 64, dtype=BF))
    assert h.launch_count() > n0


def test_refusals(muon):
    x, v = rand(94, 4, 64, dtype=BF), rand(95, 64)
    q, k = rand(96, 1, 8, 4, 64, dtype=BF), rand(97, 1, 8, 2, 64, dtype=BF)
    o, lse = muon.attention(q, k, k)
    cu = torch.tensor([0, 8], dtype=torch.int32).cuda()
    codes, scales = muon.act8_store(x)
    mean = torch.zeros(4, device="cuda")
    calls = [
        lambda: muon.layer_norm(x.double()), lambda: muon.layer_norm(x, v[:32]), lambda: muon.layer_norm(x, v.half()),
        lambda: muon.layer_norm(rand(98, 2, 16385)), lambda: muon.layer_norm(x, eps=float("nan")),
        lambda: muon.layer_norm(x, v, v.to(BF)), lambda: muon.layer_norm(torch.zeros(3, 0, device="cuda")),
        lambda: muon.layer_norm_backward(x.float(), x, mean, mean), lambda: muon.layer_norm_backward(x, x, mean[:3], mean),
        lambda: muon.attention(q.float(), k.float(), k.float()), lambda: muon.attention(q, k, k.half()),
        lambda: muon.attention(q, k[:, :, :, :32], k[:, :, :, :32]), lambda: muon.attention(q, k, k, window=4),
        lambda: muon.attention(q, k, k, causal=True, window=-1), lambda: muon.attention(q[:, :, :3], k, k),
        lambda: muon.attention(q[0], k[0], k[0]), lambda: muon.attention(q, k, k, cu_seqlens_q=cu),
        lambda: muon.attention(q[0], k[0], k[0], cu_seqlens_q=cu, cu_seqlens_k=cu.long()),
        lambda: muon.attention(rand(99, 1, 4, 2, 12, dtype=BF), *[rand(99, 1, 4, 2, 12, dtype=BF)] * 2),
        lambda: muon.attention(*[rand(99, 1, 4, 2, 136, dtype=BF)] * 3),
        lambda: muon.attention(*[rand(99, 1, 4, 2, 20, dtype=BF)[..., 2:18]] * 3),
        lambda: muon.attention(q, k, k, scale=float("inf")), lambda: muon.attention_backward(o, q, k, k, o, lse.double()),
        lambda: muon.attention_backward(o[:, :4], q, k, k, o, lse), lambda: muon.act8_store(x[0]),
        lambda: muon.act8_store(x.int()), lambda: muon.act8_restore(codes, scales[:, :2]),
        lambda: muon.act8_restore(codes, scales, dtype=torch.int32),
        lambda: muon.act8_weight_grad(x.half(), codes, scales), lambda: muon.act8_weight_grad(x[:2], codes, scales),
        lambda: muon.act8_weight_grad(x, codes, scales, dtype=HF),
        lambda: muon.act8_weight_grad(x, codes, scales, add=torch.zeros(64, 63, device="cuda")),
        lambda: muon.act8_weight_grad(x, codes, scales, out=torch.zeros(64, 64, device="cuda").t()),
    ]
    n0 = muon.default_handle().launch_count()
    for i, call in enumerate(calls):
        with pytest.raises((ValueError, muon.MuonError)):
            call()
            raise AssertionError(f"call {i} was not refused")
    assert muon.default_handle().launch_count() == n0


# ------------------------------------------------------------ bounded waits
def run_with_short_waits(muon, call):
    """Calls under a wait limit of a nanosecond.  A wait that is still open after its first polls then gives up: the
    call ends, the error word tells, and the next call is whole again.  (Data mostly arrives within the polls.)"""
    h = muon.default_handle()
    want = call()
    assert h.check() == 0
    seen = set()
    try:
        h.set_timeout_ns(1)
        for _ in range(8):
            got = call()
            seen.add(h.check())
            if seen == {0}:
                assert all(torch.equal(a, b) for a, b in zip(want, got))
    finally:
        h.set_timeout_ns(4_000_000_000)
    assert seen <= {0, 6}
    assert all(torch.equal(a, b) for a, b in zip(want, call())) and h.check() == 0
    return seen


@pytest.mark.parametrize("rows,cols,dtype", [(8000, 4096, BF), (40000, 256, BF), (3000, 8192, FP)])
def test_layer_norm_waits_end(muon, rows, cols, dtype):
    x, dy = rand(110, rows, cols, dtype=dtype), rand(111, rows, cols, dtype=dtype)
    y, mean, rstd = muon.layer_norm(x)
    run_with_short_waits(muon, lambda: (*muon.layer_norm(x), *muon.layer_norm_backward(dy, x, mean, rstd)))


@pytest.mark.parametrize("rows,cols,out", [(5000, 2048, 2048), (1000, 3000, 20000), (20000, 256, 250)])
def test_act8_weight_grad_waits_end(muon, rows, cols, out):
    dy, kept = rand(112, rows, out, dtype=BF), muon.act8_store(rand(113, rows, cols, dtype=BF))
    run_with_short_waits(muon, lambda: (muon.act8_weight_grad(dy, *kept),))


# ------------------------------------------- attention over very many keys
def attention_reference(q, k, v, do, causal=False, window=0):
    """One sequence whose heads share one key head, in fp64 on the GPU: o, lse, (dq, dk, dv), and the magnitudes of
    the products that are summed into o and into each gradient (|do||v| + |do||o| in the place of their difference)."""
    q, k, v, do = q.double(), k.double()[:, 0], v.double()[:, 0], do.double()
    o, dq, mo, mq = (torch.zeros_like(q) for _ in range(4))
    dk, dv, mk, mv = (torch.zeros_like(k) for _ in range(4))
    lse = torch.zeros(q.shape[1], q.shape[0], dtype=torch.float64, device="cuda")
    scale, step = q.shape[2] ** -0.5, max(1, (1 << 25) // len(k))
    for h in range(q.shape[1]):
        for i in range(0, len(q), step):
            at = (slice(i, i + step), h)
            s = (q[at] @ k.T) * scale
            if causal:
                place = torch.arange(i, i + len(s), device="cuda")[:, None] + (len(k) - len(q))
                j = torch.arange(len(k), device="cuda")
                s[(j > place) | (j <= place - window if window else j > place)] = -torch.inf
            z = torch.logsumexp(s, 1)
            p = torch.exp(s - z[:, None])
            o[at], mo[at], lse[h, i:i + step] = p @ v, p @ v.abs(), z
            g = do[at]
            ds = p * (g @ v.T - (g * o[at]).sum(1, keepdim=True)) * scale
            wide = p * (g.abs() @ v.abs().T + (g * o[at]).abs().sum(1, keepdim=True)) * scale
            dq[at], mq[at] = ds @ k, wide @ k.abs()
            dv += p.T @ g
            mv += p.T @ g.abs()
            dk += ds.T @ q[at]
            mk += wide.T @ q[at].abs()
    return o, lse, (dq, dk[:, None], dv[:, None]), mo, (mq, mk[:, None], mv[:, None])


def near_on_gpu(name, got, ref, tol):
    ratio = ((got.double() - ref).abs() / tol.clamp(min=1e-30)).max().item()
    record(name, ratio, 1.0)
    assert ratio <= 1.0, (name, ratio)


# The tolerance of attn_tol.  fp16 results are themselves rounded in steps of 2^-24 at least.
def gpu_tol(u, ref, mag, wide):
    return u * ref.abs() + 1.02 * u * mag + 2.0 ** -15 * wide + 2.0 ** -25


def test_fp16_probabilities_that_are_small_but_many(muon):
    n = 1 << 18
    # forward: one key far above 2^18 others, which have 2^-26 of its weight each and 2^-8 together
    q = torch.zeros(1, 40, 1, 64, dtype=HF, device="cuda")
    k, v = torch.zeros(1, n + 5, 1, 64, dtype=HF, device="cuda"), torch.ones(1, n + 5, 1, 64, dtype=HF, device="cuda")
    q[..., 0] = 12.0
    k[0, 3, 0, 0], v[0, 3] = 12.015625, 0.0                       # score 18.02 = 26 log(2)
    o, lse = muon.attention(q, k, v)
    ro, rl, _, mag, _ = attention_reference(q[0], k[0], v[0], q[0])
    near_on_gpu("many small probabilities o", o[0], ro, gpu_tol(U[HF], ro, mag, mag))
    near_on_gpu("many small probabilities lse", lse[0], rl, 2.0 ** -17 * (rl.abs() + 1))
    assert muon.default_handle().check() == 0


def test_fp16_gradient_of_a_flat_softmax(muon):
    """2^18 keys with probabilities of 2^-18."""
    n = 1 << 18
    q, do = rand(120, 1, 64, 1, 64, dtype=HF, scale=0.5), rand(121, 1, 64, 1, 64, dtype=HF, scale=64.0)
    k, v = rand(122, 1, n, 1, 64, dtype=HF), rand(123, 1, n, 1, 64, dtype=HF)
    o, lse = muon.attention(q, k, v)
    grads = muon.attention_backward(do, q, k, v, o, lse)
    _, _, (_, _, rv), _, (_, _, mv) = attention_reference(q[0], k[0], v[0], do[0])
    near_on_gpu("small probabilities dv", grads[2][0], rv, gpu_tol(U[HF], rv, mv, mv))
    assert muon.default_handle().check() == 0


# Walks over so many rows that the tensor core's truncation shows in values of one sign: the tolerance knows no length.
@pytest.mark.parametrize("dim,dtype", [(64, HF), (128, HF), (128, BF)])
@pytest.mark.parametrize("sq,sk,heads,causal,window", [
    (65536, 128, 8, False, 0), (128, 1 << 19, 1, False, 0), (200, 70001, 3, True, 0), (20011, 20011, 2, True, 0),
    (20011, 20011, 2, True, 9001)])
def test_attention_over_many_rows_of_one_sign(muon, sq, sk, heads, causal, window, dim, dtype):
    q, k = rand(130, 1, sq, heads, dim).abs().to(dtype), rand(131, 1, sk, 1, dim).abs().to(dtype)
    v, do = (rand(132, 1, sk, 1, dim).abs() + 0.5).to(dtype), (rand(133, 1, sq, heads, dim).abs() + 0.5).to(dtype)
    kw = dict(causal=causal, window=window)
    o, lse = muon.attention(q, k, v, **kw)
    grads = muon.attention_backward(do, q, k, v, o, lse, **kw)
    assert muon.default_handle().check() == 0
    ro, rl, refs, mo, mags = attention_reference(q[0], k[0], v[0], do[0], **kw)
    tag = f"one sign {sq}x{sk} h{heads} d{dim} w{window} {dtype}"
    near_on_gpu(tag + " o", o[0], ro, gpu_tol(U[dtype], ro, mo, mo))
    near_on_gpu(tag + " lse", lse[0], rl, 2.0 ** -17 * (rl.abs() + 1))
    for n, g, r, m in zip(("dq", "dk", "dv"), grads, refs, mags):
        near_on_gpu(f"{tag} {n}", g[0], r, gpu_tol(U[dtype], r, m, m))
    assert torch.equal(o, muon.attention(q, k, v, **kw)[0])
    for a, b in zip(grads, muon.attention_backward(do, q, k, v, o, lse, **kw)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dim,dtype", [(64, BF), (128, HF)])
def test_long_documents_beside_short_ones(muon, dim, dtype):
    lengths = [100, 9000, 1, 12001, 300]
    cuts = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    q, do = rand(134, cuts[-1], 4, dim, dtype=dtype), rand(135, cuts[-1], 4, dim, dtype=dtype)
    k, v = rand(136, cuts[-1], 2, dim, dtype=dtype), rand(137, cuts[-1], 2, dim, dtype=dtype)
    cu = torch.tensor(cuts, dtype=torch.int32).cuda()
    kw = dict(causal=True, cu_seqlens_q=cu, cu_seqlens_k=cu)
    o, lse = muon.attention(q, k, v, **kw)
    grads = muon.attention_backward(do, q, k, v, o, lse, **kw)
    assert muon.default_handle().check() == 0
    for a, b in zip(cuts, cuts[1:]):
        one, one_lse = muon.attention(*(t[None, a:b] for t in (q, k, v)), causal=True)
        assert torch.equal(one[0], o[a:b]) and torch.equal(one_lse[0], lse[:, a:b])
        for x, g in zip(muon.attention_backward(*(t[None, a:b] for t in (do, q, k, v)), one, one_lse, causal=True), grads):
            assert torch.equal(x[0], g[a:b])


def test_attention_without_scratch(muon):
    """The call without a workspace: the same bits up to 8192 keys, one accumulator beyond; a workspace that is too
    small is refused."""
    from newton_schulz_orthogonalized_muon_gb300 import _binding
    h, stream = muon.default_handle(), torch.cuda.current_stream().cuda_stream
    for sk in (8192, 8200):
        q, k, v = (rand(138 + i, 1, n, 1, 64, dtype=HF) for i, n in enumerate((130, sk, sk)))
        o, lse = torch.empty_like(q), torch.empty(1, 1, 130, device="cuda")
        a = _binding.MuonAttentionC(q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), o=o.data_ptr(), lse=lse.data_ptr(),
                                    batch=1, sq=130, sk=sk, heads=1, kv_heads=1, dim=64, dtype=_binding.MUON_F16,
                                    scale=0.125)
        for n in ("q", "k", "v", "o"):
            getattr(a, n + "_stride")[:] = [1 << 20, 64, 64]
        need = ctypes.c_uint64()
        assert h._lib.muon_attention_forward_workspace(h.ptr, bytes(a), ctypes.byref(need)) == 0
        assert (need.value > 0) == (sk > 8192)
        assert h._lib.muon_attention_forward(h.ptr, bytes(a), stream) == 0
        want, want_lse = muon.attention(q, k, v)
        if sk == 8192:
            assert torch.equal(o, want) and torch.equal(lse, want_lse)
        else:
            assert (o - want).abs().max().item() < 2.0 ** -8 and torch.equal(lse, want_lse)
            ws = torch.empty(need.value, dtype=torch.uint8, device="cuda")
            assert h._lib.muon_attention_forward_ex(h.ptr, bytes(a), ws.data_ptr(), need.value - 1, stream) == 1
            assert h._lib.muon_attention_forward_ex(h.ptr, bytes(a), ws.data_ptr(), need.value, stream) == 0
            assert torch.equal(o, want)
    assert h.check() == 0


# ------------------------------------------------------------------ threads
def test_first_cuda_call_of_a_thread(muon):
    """Calls that build tensor maps, from a thread that has used no CUDA function before."""
    import threading
    q = rand(150, 1, 200, 2, 64, dtype=BF)
    o, lse = muon.attention(q, q, q, causal=True)
    kept, dy = muon.act8_store(rand(151, 200, 256, dtype=BF)), rand(152, 200, 72, dtype=BF)
    w, g = rand(153, 256, 512, dtype=BF), rand(154, 256, 512, dtype=BF)
    m = torch.zeros(256, 512, device="cuda")
    calls = [lambda: muon.attention(q, q, q, causal=True),
             lambda: muon.attention_backward(q, q, q, q, o, lse, causal=True),
             lambda: (muon.act8_weight_grad(dy, *kept),),
             lambda: muon.muon_step([w], [g], [m], lr=0.02, wd=0.1)]
    want = [call() for call in calls[:3]]
    calls[3]()
    for call, ref in zip(calls, want + [None]):
        got = []

        def work():
            try:
                got.append(call())
            except Exception as e:          # the thread's own: raised below
                got.append(e)
        torch.cuda.synchronize()
        t = threading.Thread(target=work)
        t.start()
        t.join()
        if isinstance(got[0], Exception):
            raise got[0]
        if ref is not None:
            assert all(torch.equal(a, b) for a, b in zip(got[0], ref))


# ------------------------------------------------ many steps of a CTA (pair)
def test_act8_weight_grad_repeats_its_bits(muon):
    """Both CTAs of a pair write an operand that one of them reads: many steps, the same bits every time."""
    dy, kept = rand(140, 9000, 2500, dtype=BF), muon.act8_store(rand(141, 9000, 1500, dtype=BF))
    want = muon.act8_weight_grad(dy, *kept)
    for _ in range(30):
        assert torch.equal(muon.act8_weight_grad(dy, *kept), want)
    ref = torch.mm(dy.double().t(), muon.act8_restore(*kept, dtype=FP).double())
    mag = torch.mm(dy.double().abs().t(), muon.act8_restore(*kept, dtype=FP).double().abs())
    near_on_gpu("weight grad 9000x1500x2500", want, ref, U[FP] * ref.abs() + (9000 / 16 + 16) * 2.0 ** -23 * mag)
    assert muon.default_handle().check() == 0


# ------------------------------------------------ storage of codes and scales
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (17, 130), (33, 1001)])
def test_act8_storage_holds_whole_groups(muon, rows, cols):
    """What the kernels load lies inside the tensors' storage; codes and scales on storage that ends with their last
    element are taken too."""
    x, dy = rand(160, rows, cols, dtype=BF), rand(161, rows, 24, dtype=BF)
    codes, scales = muon.act8_store(x)
    for t, group in ((codes, 8), (scales, 16)):
        end = (t.shape[0] - 1) * t.stride(0) + -(-t.shape[1] // group) * group
        assert t.storage_offset() + end <= t.untyped_storage().nbytes()
    want = muon.act8_restore(codes, scales), muon.act8_weight_grad(dy, codes, scales)

    def tight(t):
        ld = t.stride(0)
        flat = torch.empty((t.shape[0] - 1) * ld + t.shape[1], dtype=torch.uint8, device="cuda")
        out = flat.as_strided(t.shape, (ld, 1))
        out.copy_(t.view(torch.uint8))
        return out.view(t.dtype)
    tc, ts = tight(codes), tight(scales)
    assert tc.untyped_storage().nbytes() == (rows - 1) * codes.stride(0) + cols
    assert torch.equal(muon.act8_restore(tc, ts), want[0])
    assert torch.equal(muon.act8_weight_grad(dy, tc, ts), want[1])


def test_other_threads_run_while_the_launch_queue_is_full(muon):
    """Calls that wait for room in the launch queue, behind a kernel of about a second, leave Python to other threads."""
    import threading
    import time
    x = rand(155, 4, 64, dtype=BF)
    kept = muon.act8_store(x)
    muon.layer_norm(x), muon.act8_restore(*kept)
    torch.cuda.synchronize()
    stamps, done = [], threading.Event()

    def work():
        torch.cuda._sleep(1_500_000_000)             # device cycles
        t0 = time.monotonic()
        for _ in range(1500):
            muon.layer_norm(x)
            muon.act8_restore(*kept)
        stamps.append(time.monotonic() - t0)
        done.set()
    t = threading.Thread(target=work)
    t.start()
    last, gap = time.monotonic(), 0.0
    while not done.is_set():
        time.sleep(0.001)
        now = time.monotonic()
        gap, last = max(gap, now - last), now
    t.join()
    torch.cuda.synchronize()
    assert stamps[0] > 0.3                           # the calls did wait
    assert gap < stamps[0] / 3, (gap, stamps[0])


def test_threads_share_a_handle(muon):
    """Threads in the library at once: every launch is counted, every error is told, every result is right."""
    import threading
    h, n = muon.default_handle(), 2000
    x = rand(156, 8, 64, dtype=BF)
    want = muon.layer_norm(x)[0]
    ps = [[torch.ones(64, device="cuda") for _ in range(4)] for _ in range(2)]
    wrong = []

    def norm():
        for _ in range(n):
            if not torch.equal(muon.layer_norm(x)[0], want):
                wrong.append("layer norm")

    def adam(p, times=n):
        for i in range(times):
            muon.adamw_step([p[0]], [p[1]], [p[2]], [p[3]], step=i + 1, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.0)

    def refused():
        for _ in range(n):
            try:
                muon.attention(*[x.view(1, 8, 1, 64)] * 3, scale=-1.0)
                wrong.append("not refused")
            except muon.MuonError as e:
                if "scale" not in str(e):
                    wrong.append(str(e))
    counts = [h.launch_count()]
    for call in (lambda: muon.layer_norm(x), lambda: adam(ps[0], 1)):
        call()
        counts.append(h.launch_count())
    threads = [threading.Thread(target=f, args=a) for f, a in ((norm, ()), (adam, (ps[0],)), (adam, (ps[1],)), (refused, ()))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]
    assert h.launch_count() - counts[2] == n * (counts[1] - counts[0]) + 2 * n * (counts[2] - counts[1])
    assert h.check() == 0


EDGES = """
import ctypes, sys
import torch
import newton_schulz_orthogonalized_muon_gb300 as muon
g = torch.Generator().manual_seed(1)
r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
x, dy, q = r(2000, 256), r(2000, 250), r(1, 200, 2, 64)
y, mean, rstd = muon.layer_norm(x)
kept = muon.act8_store(x)
o, lse = muon.attention(q, q, q, causal=True)
calls = [lambda: muon.layer_norm_backward(x, x, mean, rstd), lambda: (muon.act8_weight_grad(dy, *kept),),
         lambda: muon.attention_backward(q, q, q, q, o, lse, causal=True)]
rt = ctypes.CDLL("libcudart.so.13")
out = []
for call in calls:
    out += [t.cpu() for t in call()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    raw, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t()
    assert rt.cudaGraphGetEdges(raw, None, None, None, ctypes.byref(n)) == 0
    a, b, data = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * n.value)(), (ctypes.c_ubyte * (8 * n.value))()
    assert rt.cudaGraphGetEdges(raw, a, b, data, ctypes.byref(n)) == 0
    print(n.value, sum(data[8 * i + 2] for i in range(n.value)))       # the edge's type: 1 programmatic
assert muon.default_handle().check() == 0
torch.save(out, sys.argv[1])
"""


def test_dependent_launches_can_be_switched_off(muon, tmp_path):
    """MUON_PDL=0: every launch of the operators waits for the one before it, and the bits are the same."""
    got = {}
    for level in ("0", "1"):
        r = subprocess.run([sys.executable, "-c", EDGES, str(tmp_path / level)], cwd=ROOT, capture_output=True, text=True,
                           env={**os.environ, "MUON_PDL": level})
        assert r.returncode == 0, r.stdout + r.stderr
        got[level] = [tuple(map(int, line.split())) for line in r.stdout.split("\n") if line]
    assert [n for n, _ in got["0"]] == [n for n, _ in got["1"]] and all(n > 0 for n, _ in got["0"])
    assert all(p == 0 for _, p in got["0"]), got
    assert all(p > 0 for _, p in got["1"]), got
    for a, b in zip(torch.load(tmp_path / "0"), torch.load(tmp_path / "1")):
        assert torch.equal(a, b)


# --------------------------- many rows, steps and items of a CTA (or CTA pair)
# Row kernels with several rows a group, batch kernels whose ring goes round, uneven last batches.
@pytest.mark.parametrize("rows,cols,pad,dtype", [
    (40001, 33, 0, BF), (4099, 1023, 6, FP), (9001, 1023, 0, HF), (60007, 256, 0, BF), (60007, 256, 0, FP), (30011, 768, 8, HF),
    (8003, 4096, 0, BF), (4001, 4096, 0, FP), (1501, 8192, 0, FP), (3001, 8192, 0, BF), (901, 9001, 0, BF),
    (1201, 16384, 0, BF), (701, 16384, 0, FP)])
def test_layer_norm_over_many_rows(muon, rows, cols, pad, dtype):
    """The formulas and tolerances of test_layer_norm, the reference in fp64 on the GPU."""
    x = (rand(170, rows, cols + pad) * 3 + 5).to(dtype)[:, :cols]
    dy = rand(171, rows, cols + pad, dtype=dtype)[:, :cols]
    w, b = 1 + rand(172, cols) * 0.3, rand(173, cols)
    y, mean, rstd = muon.layer_norm(x, w, b, eps=1e-5)
    dx, dw, db = muon.layer_norm_backward(dy, x, mean, rstd, w)
    assert muon.default_handle().check() == 0
    tag, e = f"layer norm {rows}x{cols} {dtype}", 2.0 ** -19
    xd, dyd, wd, bd = x.double(), dy.double(), w.double(), b.double()
    mr = xd.mean(1)
    rr = (xd - mr[:, None]).square().mean(1).add(1e-5).rsqrt()
    top, size = e * xd.abs().amax(1) * rr, e * xd.abs().mean(1)
    off = size * rr
    near_on_gpu(tag + " mean", mean, mr, size)
    near_on_gpu(tag + " rstd", rstd, rr, rr * (e + off * off + top))
    z = (xd - mr[:, None]) * rr[:, None]
    yr = z * wd + bd
    inner = off[:, None] + (e + top[:, None]) * z.abs()
    near_on_gpu(tag + " y", y, yr, U[dtype] * yr.abs() + inner * wd.abs() + e * (z.abs() * wd.abs() + bd.abs()))
    md, rd = mean.double()[:, None], rstd.double()[:, None]
    z, g = (xd - md) * rd, dyd * wd
    ref = rd * (g - g.mean(1, keepdim=True) - z * (g * z).mean(1, keepdim=True))
    xh, xt, g = (xd.abs() + md.abs()) * rd, z.abs(), g.abs()
    mag = rd * (g + g.mean(1, keepdim=True) + xh * (g * xt).mean(1, keepdim=True) + xt * (g * xh).mean(1, keepdim=True))
    near_on_gpu(tag + " dx", dx, ref, U[dtype] * ref.abs() + e * mag)
    near_on_gpu(tag + " dw", dw, (dyd * z).sum(0), 2.0 ** -18 * (dyd.abs() * xh).sum(0))
    near_on_gpu(tag + " db", db, dyd.sum(0), 2.0 ** -18 * dyd.abs().sum(0))
    for a, c in zip((dx, dw, db), muon.layer_norm_backward(dy, x, mean, rstd, w)):
        assert torch.equal(a, c)


# Both accumulators and their phases (more than 2048 tokens, several thousand of them), rings carried from item to item
# (more tiles than pairs), output bands past the first eight tiles, splits of more than 2048 tokens.
@pytest.mark.parametrize("rows,cols,out,odtype,add", [
    (4239, 1500, 4100, FP, False), (4239, 1500, 4100, FP, True), (6273, 1500, 4100, BF, True), (20001, 1024, 2600, FP, False),
    (70, 3000, 9000, FP, True), (8200, 300, 20000, BF, False), (200001, 200, 136, FP, True), (400003, 300, 250, BF, False)])
def test_act8_weight_grad_over_many_tokens_and_tiles(muon, rows, cols, out, odtype, add):
    x, dy = rand(174, rows, cols, dtype=BF) + 0.2, rand(175, rows, out, dtype=BF)
    kept = muon.act8_store(x)
    base = rand(176, out, cols, dtype=odtype) if add else None
    got = muon.act8_weight_grad(dy, *kept, add=base, dtype=odtype)
    assert muon.default_handle().check() == 0
    xd, dyd = muon.act8_restore(*kept, dtype=FP).double(), dy.double()
    ref, mag = dyd.t() @ xd, dyd.abs().t() @ xd.abs()
    if add:
        ref, mag = ref + base.double(), mag + base.double().abs()
    # 16 products an addition, 128 additions an accumulator; then one rounded addition each 2048 tokens, of a split
    # (its steps of 64 tokens over the splits), and one a split
    terms = min(rows, 2048) / 16 + rows / 2048 + 16
    tol = U[odtype] * ref.abs() + terms * 2.0 ** -23 * mag
    near_on_gpu(f"weight grad {rows}x{cols}x{out} {odtype}", got, ref, tol)
    assert torch.equal(got, muon.act8_weight_grad(dy, *kept, add=base, dtype=odtype))
    if add:
        muon.act8_weight_grad(dy, *kept, add=base, out=base)
        assert torch.equal(base, got)


# ----------------------------------------------- offsets that are not in order
def clamped(cuts, axis):
    """The documented rule: cut to the axis, and raised to the largest before."""
    out = []
    for c in cuts:
        out.append(max(min(max(c, 0), axis), out[-1] if out else 0))
    return out


@pytest.mark.parametrize("cuts_q,cuts_k", [
    ([10, 200, 390], None), ([0, 200, 100, 5000], None), ([-7, 150, 150], None), ([390, 10, 400], None),
    ([5, 60, 50, 300], [-3, 130, 260, 100]), ([7], None),
    ([3 + 9 * i - (40 if i % 13 == 5 else 0) + (9999 if i == 60 else 0) for i in range(64)], None),
    ([6 * i - (100 if i == 40 else 0) for i in range(50)], [2 ** 31 - 1 if i > 45 else 8 * i - 20 for i in range(50)])])
def test_packed_offsets_follow_the_rule(muon, cuts_q, cuts_k):
    n, h, dim = 400, 2, 64
    cuts_k = cuts_q if cuts_k is None else cuts_k
    q, k, v, do = (rand(180 + i, n, h, dim, dtype=BF) for i in range(4))
    kw = dict(causal=True, cu_seqlens_q=torch.tensor(cuts_q, dtype=torch.int32).cuda(),
              cu_seqlens_k=torch.tensor(cuts_k, dtype=torch.int32).cuda())
    o, lse = muon.attention(q, k, v, **kw)
    grads = muon.attention_backward(do, q, k, v, o, lse, **kw)
    assert muon.default_handle().check() == 0
    cq, ck = clamped(cuts_q, n), clamped(cuts_k, n)
    spans = [(None, *s) for s in zip(cq, cq[1:], ck, ck[1:])]
    check_attention(f"offsets {cuts_q[:4]} {cuts_k[:4]}", BF, dim ** -0.5, True, 0, spans, q, k, v, do, o, lse, grads)
    for cuts, tensors in ((cq, (o, grads[0], lse.t())), (ck, grads[1:])):
        outside = torch.ones(n, dtype=torch.bool, device="cuda")
        outside[cuts[0]:cuts[-1]] = False
        for t in tensors:
            want = -math.inf if t.dtype == FP else 0.0
            assert (t[outside] == want).all()


@pytest.mark.parametrize("dim,heads,kv,seq", [(64, 12, 12, 1024), (128, 16, 4, 2048), (128, 1, 1, 9000)])
def test_attention_waits_end(muon, dim, heads, kv, seq):
    q, k, v, do = (rand(184 + i, 2, seq, n, dim, dtype=HF) for i, n in enumerate((heads, kv, kv, heads)))
    o, lse = muon.attention(q, k, v, causal=True)
    run_with_short_waits(muon, lambda: (*muon.attention(q, k, v, causal=True),
                                        *muon.attention_backward(do, q, k, v, o, lse, causal=True)))


def test_long_attention_in_a_graph_and_on_two_streams(muon):
    """Walks in parts: scratch and counter are the call's own."""
    q, do = rand(190, 1, 9001, 2, 64, dtype=HF), rand(191, 1, 9001, 2, 64, dtype=HF)
    k, v = rand(192, 1, 9001, 1, 64, dtype=HF), rand(193, 1, 9001, 1, 64, dtype=HF)

    def work():
        o, lse = muon.attention(q, k, v, causal=True)
        return [o, lse, *muon.attention_backward(do, q, k, v, o, lse, causal=True)]
    want = work()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(work())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for _ in range(2):
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held))
    assert muon.default_handle().check() == 0
