"""Weights in 8 bits and products of 8-bit operands, against plain 64-bit forms.

Tolerances of the product, element by element: one rounding to the output type,
half a step (2^-8, 2^-11, 2^-24 of the value; 2^-25 where fp16 is not normal),
and what fp32 sums lose that are truncated with every 32 products:
(cols / 32 + 16) 2^-23 of the sum of the products' magnitudes.  Codes and the
values that they stand for are exact.
"""
import numpy as np
import pytest
import torch

from _margins import record
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def muon():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import newton_schulz_orthogonalized_muon_gb300 as pkg
    torch.cuda.set_device(0)
    yield pkg
    torch.cuda.synchronize()
    assert pkg.default_handle().check() == 0


def host(t):
    return t.detach().double().cpu().numpy()


def rand(seed, *shape, dtype=BF, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def bits(t):
    return t.view(torch.uint8).cpu().numpy()


WEIGHTS = [(1, 1), (3, 7), (128, 128), (127, 129), (130, 1), (1, 300), (200, 136), (257, 520), (16, 2050), (640, 384)]


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("out,cols", WEIGHTS)
def test_store_weight(muon, out, cols, dtype):
    w = (rand(1, out, cols, dtype=FP) * torch.exp(2 * rand(2, out, 1, dtype=FP))).to(dtype)
    codes, scales, codes_t = muon.act8_store_weight(w, transposed=True)
    want, want_s = oo.act8_encode_weight(host(w))
    assert codes.dtype == codes_t.dtype == torch.float8_e4m3fn and scales.dtype == torch.uint8
    got = bits(codes.contiguous())
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(oo.e4m3_table()[got], oo.e4m3_table()[want])
    assert np.array_equal(bits(codes_t.contiguous()), got.T)
    alone = muon.act8_store_weight(w)
    assert len(alone) == 2 and np.array_equal(bits(alone[0].contiguous()), got) and torch.equal(alone[1], scales)
    value = oo.act8_decode_weight(want, want_s)
    exact = torch.tensor(value).to(dtype).cuda()
    assert torch.equal(muon.act8_restore_weight(codes, scales, dtype=dtype), exact)
    assert torch.equal(muon.act8_restore_weight(codes_t, scales.t(), dtype=dtype), exact.t())


def test_store_weight_of_odd_values(muon):
    w = rand(3, 300, 300, dtype=FP)
    w[5, 7], w[200, 10], w[:128, 256:] = float("nan"), float("-inf"), 0.0
    w[256:, :128] = 1e-42
    w[256:, 128:256] = 3e38
    w[130, 130] = 448.0 * 2.0 ** 9
    codes, scales = muon.act8_store_weight(w)
    want, want_s = oo.act8_encode_weight(host(w))
    assert np.array_equal(scales.cpu().numpy(), want_s) and scales[0, 0] == 255 and scales[0, 1] == 255 and scales[2, 0] == 16
    back = muon.act8_restore_weight(codes, scales, dtype=FP)
    assert torch.isnan(back[:128, :128]).all() and torch.isnan(back[128:256, :128]).all()
    assert np.array_equal(host(back), oo.act8_decode_weight(want, want_s), equal_nan=True)


def test_nothing_is_written_past_the_last_column(muon):
    import ctypes
    h = muon.default_handle()
    w = rand(4, 130, 140)
    codes = torch.full((130, 256), 7, dtype=torch.uint8, device="cuda")
    codes_t = torch.full((140, 256), 7, dtype=torch.uint8, device="cuda")
    scales = torch.full((2, 5), 7, dtype=torch.uint8, device="cuda")
    vp = ctypes.c_void_p
    assert h._lib.muon_act8_store_weight(h.ptr, vp(w.data_ptr()), 140, vp(codes.data_ptr()), 256, vp(codes_t.data_ptr()), 256,
                                         vp(scales.data_ptr()), 5, 130, 140, 1,
                                         vp(torch.cuda.current_stream().cuda_stream)) == 0
    torch.cuda.synchronize()
    assert (codes[:, 140:] == 7).all() and (codes_t[:, 130:] == 7).all() and (scales[:, 2:] == 7).all()
    assert torch.equal(codes[:, :140].t(), codes_t[:, :130])


def product(muon, x, w, dtype, tag):
    codes, scales = muon.act8_store(x)
    wc, ws = muon.act8_store_weight(w)
    got = muon.act8_matmul(codes, scales, wc, ws, dtype=dtype)
    xv, wv = host(muon.act8_restore(codes, scales, dtype=FP)), host(muon.act8_restore_weight(wc, ws, dtype=FP))
    with np.errstate(invalid="ignore"):
        ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    assert got.dtype == dtype and got.shape == ref.shape
    fine = np.isfinite(ref)
    g = host(got)
    assert np.isnan(g[~fine]).all(), tag
    tol = np.maximum(U[dtype] * np.abs(ref), 2.0 ** -25 if dtype == HF else 0.0) + (x.shape[1] / 32 + 16) * 2.0 ** -23 * mag
    ratio = float(np.max(np.abs(g - ref)[fine] / np.maximum(tol[fine], 1e-30), initial=0.0))
    record(tag, ratio, 1.0)
    assert ratio <= 1.0, (tag, ratio)
    return got


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("rows,cols,out", [(1, 1, 1), (5, 16, 8), (16, 128, 128), (33, 127, 129), (224, 256, 256), (225, 512, 264),
                                           (100, 640, 130), (7, 1000, 3), (450, 2042, 391), (1001, 520, 1411), (64, 4096, 512)])
def test_matmul8(muon, rows, cols, out, dtype):
    # rows and blocks of very different sizes, so that a scale in the wrong place shows
    x = rand(5, rows, cols, dtype=FP) * torch.exp2(torch.randint(-6, 7, (rows, -(-cols // 128)), device="cuda",
                                                                 generator=torch.Generator("cuda").manual_seed(6)).float()
                                                   ).repeat_interleave(128, 1)[:, :cols]
    unit = torch.exp2(torch.randint(-5, 4, (-(-out // 128), -(-cols // 128)), device="cuda",
                                    generator=torch.Generator("cuda").manual_seed(7)).float())
    w = rand(8, out, cols, dtype=FP) * unit.repeat_interleave(128, 0)[:out].repeat_interleave(128, 1)[:, :cols] / cols
    product(muon, x, w, dtype, f"matmul8 {rows}x{cols}x{out} {dtype}")


def test_matmul8_of_values_that_are_not_finite(muon):
    x, w = rand(9, 70, 400, dtype=FP), rand(10, 300, 400, dtype=FP)
    x[3, 130], x[66, 399], w[140, 5] = float("nan"), float("inf"), float("nan")
    got = product(muon, x, w, FP, "matmul8 not finite")
    assert torch.isnan(got[3]).all() and torch.isnan(got[66]).all() and torch.isnan(got[:, 128:256]).all()
    rest = torch.ones(70, dtype=torch.bool)
    rest[[3, 66]] = False
    assert torch.isfinite(got[rest][:, :128]).all() and torch.isfinite(got[rest][:, 256:]).all()


def test_transposed_codes_give_the_inputs_gradient(muon):
    w, dy = rand(11, 330, 200), rand(12, 90, 330)
    codes, scales, codes_t = muon.act8_store_weight(w, transposed=True)
    g, gs = muon.act8_store(dy)
    dx = muon.act8_matmul(g, gs, codes_t, scales.t(), dtype=FP)
    gv, wv = host(muon.act8_restore(g, gs, dtype=FP)), host(muon.act8_restore_weight(codes, scales, dtype=FP))
    assert np.all(np.abs(host(dx) - gv @ wv) <= (330 / 32 + 16) * 2.0 ** -23 * (np.abs(gv) @ np.abs(wv)) + 2.0 ** -24 * np.abs(gv @ wv))


def test_layouts_streams_graphs(muon):
    x, w = rand(13, 300, 500), rand(14, 260, 500)
    codes, scales = muon.act8_store(x)
    wc, ws, wt = muon.act8_store_weight(w, transposed=True)
    want = muon.act8_matmul(codes, scales, wc, ws)
    assert torch.equal(muon.act8_matmul(codes.contiguous(), scales.contiguous(), wc.contiguous(), ws.t().contiguous().t()), want)
    assert torch.equal(muon.act8_matmul(codes.view(torch.uint8), scales, wc.view(torch.uint8), ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = muon.act8_matmul(codes, scales, wc, ws, stream=side)
    here = muon.act8_matmul(codes, scales, wc, ws)
    side.synchronize()
    assert torch.equal(other, want) and torch.equal(here, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c, s = muon.act8_store_weight(w)
        kept = muon.act8_matmul(codes, scales, c, s)
    w.mul_(3.0)
    graph.replay()
    assert torch.equal(kept, muon.act8_matmul(codes, scales, *muon.act8_store_weight(w)))
    assert not torch.equal(kept, want)


def test_refusals(muon):
    x, w = rand(15, 20, 256), rand(16, 40, 256)
    codes, scales = muon.act8_store(x)
    wc, ws = muon.act8_store_weight(w)
    for call in (lambda: muon.act8_store_weight(w[0]), lambda: muon.act8_store_weight(w.int()), lambda: muon.act8_store_weight(w.cpu()),
                 lambda: muon.act8_matmul(codes, scales, wc, ws.t()), lambda: muon.act8_matmul(codes, scales[:1], wc, ws),
                 lambda: muon.act8_matmul(codes, scales, wc[:, :128], ws[:1]), lambda: muon.act8_matmul(codes, scales, wc.float(), ws),
                 lambda: muon.act8_matmul(codes, scales, wc, ws, dtype=torch.int8), lambda: muon.act8_matmul(codes, scales, wc, ws.int()),
                 lambda: muon.act8_restore_weight(wc, ws[:1]), lambda: muon.act8_matmul(codes.cpu(), scales, wc, ws)):
        with pytest.raises(ValueError):
            call()
    assert muon.act8_matmul(codes[:0], scales[:, :0], wc, ws).shape == (0, 40)
    assert muon.act8_matmul(codes, scales, wc[:0], ws[:, :0]).shape == (20, 0)
    assert (muon.act8_matmul(codes[:, :0], scales[:0], wc[:, :0], ws[:0]) == 0).all()
    c, s, t = muon.act8_store_weight(w[:, :0], transposed=True)
    assert c.shape == (40, 0) and s.shape == (0, 1) and t.shape == (0, 40)
