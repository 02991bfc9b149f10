"""Products by expert on the GPU against their plain 64-bit forms.

Tolerances, element by element: one rounding to the output type, u |ref| (u as
in test_gpu_ops.py: 2^-8, 2^-11, 2^-24; 2^-25 where fp16 is not normal), and what the tensor cores' fp32 sums
lose, truncated with every 16 products that are added:
(n / 16 + 16) 2^-23 of the sum of the n products' magnitudes.
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


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def offsets_of(lens):
    return ints(np.concatenate([[0], np.cumsum(lens)]))


def close(name, got, ref, tol):
    got = host(got)
    assert got.shape == ref.shape and np.isfinite(got).all(), name
    ratio = float(np.max(np.abs(got - ref) / np.maximum(tol, 1e-30), initial=0.0))
    record(name, ratio, 1.0)
    assert ratio <= 1.0, (name, ratio)


def rounded(dtype, ref):
    """One rounding: half a step.  Steps of fp16 are 2^-24 and no smaller below 2^-14, where u |ref| < 2^-25."""
    return np.maximum(U[dtype] * np.abs(ref), 2.0 ** -25 if dtype == HF else 0.0)


def sums(n):
    return (n / 16 + 16) * 2.0 ** -23


# tokens of each expert, cols, out, tokens of no expert behind them
CASES = [
    ([1], 8, 8, 0), ([5], 64, 64, 0), ([3, 0, 2], 72, 136, 4), ([33, 31, 1, 64, 0], 264, 40, 1),
    ([257], 128, 256, 0), ([0, 300, 0, 511, 7], 200, 520, 9), ([1000, 1, 90], 512, 768, 0),
    ([0, 0, 0], 64, 64, 5), ([17] * 40, 136, 264, 0), ([700, 130, 260], 1032, 1416, 3), ([2500, 40], 384, 328, 0),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens,cols,out,behind", CASES)
def test_expert_matmul(muon, lens, cols, out, behind, dtype):
    tokens = sum(lens) + behind
    x, dy = rand(1, tokens, cols, dtype=dtype), rand(2, tokens, out, dtype=dtype)
    w = rand(3, len(lens), out, cols, dtype=dtype)
    at = offsets_of(lens)
    for given, transpose in ((x, False), (dy, True)):
        got = muon.expert_matmul(given, w, at, transpose=transpose)
        ref, mag = oo.expert_matmul(host(given), host(w), at.cpu().numpy(), transpose)
        assert got.dtype == dtype
        close(f"experts {lens[:3]} {cols}x{out} {dtype} {transpose}", got, ref,
              rounded(dtype, ref) + sums(given.shape[1]) * mag)


@pytest.mark.parametrize("dtype,odtype,add", [(BF, FP, False), (BF, BF, False), (HF, FP, True), (HF, HF, False), (BF, BF, True)])
@pytest.mark.parametrize("lens,cols,out,behind", CASES)
def test_expert_weight_grad(muon, lens, cols, out, behind, dtype, odtype, add):
    tokens = sum(lens) + behind
    x, dy = rand(4, tokens, cols, dtype=dtype), rand(5, tokens, out, dtype=dtype)
    so_far = rand(6, len(lens), out, cols, dtype=odtype) if add else None
    at = offsets_of(lens)
    got = muon.expert_weight_grad(dy, x, at, add=so_far, dtype=odtype)
    ref, mag = oo.expert_weight_grad(host(dy), host(x), at.cpu().numpy())
    if add:
        ref, mag = ref + host(so_far), mag + np.abs(host(so_far))
    assert got.dtype == odtype
    close(f"experts dw {lens[:3]} {cols}x{out} {dtype} {odtype}", got, ref, rounded(odtype, ref) + sums(max(lens)) * mag)


@pytest.mark.parametrize("first", [0, 1, 14, 15, 16, 17, 47, 63, 64, 65, 127])
def test_tokens_of_others_have_no_part(muon, first):
    """Infinite and NaN rows of a neighbour, and of no expert, next to an expert's last token."""
    lens, cols, out = [first, 100], 192, 128
    x, dy = rand(7, sum(lens) + 70, cols), rand(8, sum(lens) + 70, out)
    at = offsets_of(lens)
    w = rand(9, 2, out, cols)
    clean = [muon.expert_matmul(x, w, at), muon.expert_matmul(dy, w, at, transpose=True),
             muon.expert_weight_grad(dy, x, at)]
    for bad in (float("nan"), float("inf")):
        x2, dy2 = x.clone(), dy.clone()
        x2[first:], dy2[first:] = bad, bad
        got = [muon.expert_matmul(x2, w, at), muon.expert_matmul(dy2, w, at, transpose=True),
               muon.expert_weight_grad(dy2, x2, at)]
        assert torch.equal(got[0][:first], clean[0][:first]) and torch.equal(got[1][:first], clean[1][:first])
        assert torch.equal(got[2][0], clean[2][0])
        for g in got[:2]:
            assert not torch.isfinite(g[first:first + 100]).any() and (g[first + 100:] == 0).all()


def test_offsets_that_break_the_rule(muon):
    tokens, cols, out = 200, 64, 72
    x, dy, w = rand(10, tokens, cols), rand(11, tokens, out), rand(12, 4, out, cols)
    for at in ([5, 100, 40, 90, 150], [-7, 20, 20, 300, 400], [50, 10, 10, 10, 10], [2 ** 31 - 1] * 5, [-1] * 5, [30, 60, 90, 120, 10]):
        ref, mag = oo.expert_matmul(host(x), host(w), at)
        close(f"experts offsets {at}", muon.expert_matmul(x, w, ints(at)), ref, rounded(BF, ref) + sums(cols) * mag)
        ref, mag = oo.expert_weight_grad(host(dy), host(x), at)
        close(f"experts dw offsets {at}", muon.expert_weight_grad(dy, x, ints(at)), ref, sums(tokens) * mag + rounded(FP, ref))


def test_many_experts_and_long_sums(muon):
    lens = [(7 * i) % 5 for i in range(1024)]
    x, w, at = rand(13, sum(lens), 16), rand(14, 1024, 24, 16), offsets_of(lens)
    ref, mag = oo.expert_matmul(host(x), host(w), at.cpu().numpy())
    close("1024 experts", muon.expert_matmul(x, w, at), ref, rounded(BF, ref) + sums(16) * mag)
    # one sign: 2048 tokens are truncated at a time, then added with rounding
    x, dy = rand(15, 70001, 40).abs(), rand(16, 70001, 24).abs()
    ref, mag = oo.expert_weight_grad(host(dy), host(x), [0, 1, 70000])
    close("70 K tokens", muon.expert_weight_grad(dy, x, ints([0, 1, 70000])), ref, (sums(2048) + 40 * 2.0 ** -24) * mag)


@pytest.mark.parametrize("dtype,odtype,add", [(BF, FP, True), (HF, HF, False)])
@pytest.mark.parametrize("lens,cols,out", [([6001], 136, 72), ([900, 0, 3001], 256, 200), ([0, 2999], 520, 24), ([11000, 1], 64, 8)])
def test_weight_grad_of_few_tiles(muon, lens, cols, out, dtype, odtype, add):
    """Tokens of an expert in splits: ends inside steps, splits without tokens, and an expert that has none."""
    x, dy = rand(30, sum(lens) + 3, cols, dtype=dtype), rand(31, sum(lens) + 3, out, dtype=dtype, scale=0.1)
    x[sum(lens):], dy[sum(lens):] = float("inf"), float("nan")
    so_far = rand(32, len(lens), out, cols, dtype=odtype) if add else None
    at = offsets_of(lens)
    got = muon.expert_weight_grad(dy, x, at, add=so_far, dtype=odtype)
    ref, mag = oo.expert_weight_grad(host(dy), host(x), at.cpu().numpy())
    if add:
        ref, mag = ref + host(so_far), mag + np.abs(host(so_far))
    close(f"experts dw splits {lens} {cols}x{out} {odtype}", got, ref, rounded(odtype, ref) + (sums(2048) + 16 * 2.0 ** -24) * mag)
    assert torch.equal(got, muon.expert_weight_grad(dy, x, at, add=so_far, dtype=odtype))
    wide = torch.zeros(len(lens), out, cols + 5, dtype=odtype, device="cuda")[:, :, 2:2 + cols]
    muon.expert_weight_grad(dy, x, at, add=so_far, out=wide)
    assert torch.equal(got, wide)


def test_strides_and_places(muon):
    lens, cols, out = [40, 25], 64, 48
    wide, wdy = rand(17, 70, 3 * cols), rand(18, 70, out + 16)
    x, dy, at = wide[2:67, cols:2 * cols], wdy[2:67, 8:8 + out], offsets_of(lens)
    w = rand(19, 2, 2 * out, cols)[:, ::2]
    plain = [muon.expert_matmul(x.contiguous(), w.contiguous(), at),
             muon.expert_matmul(dy.contiguous(), w.contiguous(), at, transpose=True),
             muon.expert_weight_grad(dy.contiguous(), x.contiguous(), at)]
    odd_x, odd_dy = torch.zeros(65, cols + 3, dtype=BF, device="cuda")[:, 1:1 + cols], dy.t().contiguous().t()
    odd_x.copy_(x)
    for xx, gg in ((x, dy), (odd_x, odd_dy)):
        got = [muon.expert_matmul(xx, w, at), muon.expert_matmul(gg, w, at, transpose=True), muon.expert_weight_grad(gg, xx, at)]
        assert all(torch.equal(a, b) for a, b in zip(got, plain))
    # into a part of a larger tensor, in place, and rows that no vector store fits
    for pad in (0, 8, 3):
        big = torch.full((2, out + 1, cols + pad), 7.0, device="cuda")
        view = big[:, :out, :cols]
        view.copy_(rand(20, 2, out, cols, dtype=FP))
        want = view.clone() + plain[2]
        got = muon.expert_weight_grad(dy, x, at, add=view, out=view)
        assert got.data_ptr() == view.data_ptr() and torch.equal(view, want)
        assert (big[:, out] == 7).all() and (big[:, :, cols:] == 7).all()


def test_streams_graphs_and_repeats(muon):
    lens, cols, out = [300, 0, 219, 90], 512, 264
    x, dy, w, at = rand(21, 620, cols), rand(22, 620, out), rand(23, 4, out, cols), offsets_of(lens)

    def all_three():
        return [muon.expert_matmul(x, w, at), muon.expert_matmul(dy, w, at, transpose=True), muon.expert_weight_grad(dy, x, at)]

    want = all_three()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = muon.expert_matmul(x, w, at, stream=side)
    other = muon.expert_weight_grad(dy, x, at, stream=side)
    again = all_three()
    side.synchronize()
    assert torch.equal(got, want[0]) and torch.equal(other, want[2])
    assert all(torch.equal(a, b) for a, b in zip(again, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = all_three()
    at.copy_(offsets_of([10, 400, 100, 99]))
    x.mul_(0.5)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(kept, all_three()))


def test_refusals(muon):
    x, w, at = rand(24, 16, 64), rand(25, 2, 32, 64), ints([0, 8, 16])
    dy = rand(26, 16, 32)
    for call in (lambda: muon.expert_matmul(x.float(), w.float(), at), lambda: muon.expert_matmul(x, w.half(), at),
                 lambda: muon.expert_matmul(x, w, at[:2]), lambda: muon.expert_matmul(x, w, at.long()),
                 lambda: muon.expert_matmul(x, w[0], at), lambda: muon.expert_matmul(x, w, at, transpose=True),
                 lambda: muon.expert_matmul(x, w.cpu(), at), lambda: muon.expert_matmul(x, w, at.cpu()),
                 lambda: muon.expert_weight_grad(dy, x[:8], at), lambda: muon.expert_weight_grad(dy, x, at[:1]),
                 lambda: muon.expert_weight_grad(dy, x, at, dtype=HF),
                 lambda: muon.expert_weight_grad(dy, x, at, add=torch.zeros(2, 32, 64, device="cuda"), dtype=BF),
                 lambda: muon.expert_weight_grad(dy, x, at, out=torch.zeros(2, 64, 32, device="cuda")),
                 lambda: muon.expert_weight_grad(dy, x, at, out=torch.zeros(1, 32, 64, device="cuda").expand(2, 32, 64))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: muon.expert_matmul(rand(1, 4, 12), rand(2, 2, 8, 12), at),
                 lambda: muon.expert_matmul(rand(1, 4, 8), rand(2, 2, 12, 8), at),
                 lambda: muon.expert_matmul(x, rand(3, 1025, 32, 64), torch.zeros(1026, dtype=torch.int32, device="cuda"))):
        with pytest.raises(muon.MuonError, match="INVALID_ARG"):
            call()
    assert muon.expert_matmul(x[:0], w, at).shape == (0, 32)
    assert (muon.expert_weight_grad(dy[:0], x[:0], at) == 0).all()
