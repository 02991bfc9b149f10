"""Products by expert over long sums of one sign, which truncation makes too
small: by up to 2^-23 of themselves with each 16 products."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
U = {BF: 2.0 ** -8, HF: 2.0 ** -11}


@pytest.fixture(scope="module")
def muon():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import newton_schulz_orthogonalized_muon_gb300 as pkg
    torch.cuda.set_device(0)
    yield pkg
    torch.cuda.synchronize()
    assert pkg.default_handle().check() == 0


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("long", [1416, 16384, 65536])
def test_long_sums_of_one_sign(muon, long, transpose, dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    at = torch.tensor([0, 70, 70, 133], dtype=torch.int32, device="cuda")
    x = torch.randn(133, long, generator=g, device="cuda").abs().to(dtype)
    w = (torch.randn(3, 136, long, generator=g, device="cuda").abs() / long ** 0.5).to(dtype)
    y = muon.expert_matmul(x, w.transpose(1, 2).contiguous() if transpose else w, at, transpose=transpose).double()
    ref = torch.cat([x[:70].double() @ w[0].double().t(), x[70:].double() @ w[2].double().t()])
    lost = (long / 16 + 16) * 2.0 ** -23
    assert ((y - ref).abs() <= (U[dtype] + lost) * ref).all()
    # roundings go both ways, so their mean over 18088 results is below U / 100: what is lost shows in it
    assert -lost - U[dtype] / 100 <= (y / ref - 1).mean() <= U[dtype] / 100


def test_sums_that_would_lose_a_rounding_are_refused(muon):
    """2^16 products of one sign lose up to 2^-11, a rounding of fp16."""
    at = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    wide = 2 ** 16 + 8
    x, w = torch.zeros(4, wide, dtype=BF, device="cuda"), torch.zeros(1, 8, wide, dtype=BF, device="cuda")
    tall, short = w.transpose(1, 2).contiguous(), torch.zeros(4, 8, dtype=BF, device="cuda")
    for call in (lambda: muon.expert_matmul(x, w, at), lambda: muon.expert_matmul(x, tall, at, transpose=True)):
        with pytest.raises(muon.MuonError, match="INVALID_ARG"):
            call()
    # as many results are none the less
    assert muon.expert_matmul(short, tall, at).shape == (4, wide)
    assert muon.expert_matmul(short, w, at, transpose=True).shape == (4, wide)
    assert muon.expert_weight_grad(short, x, at).shape == (1, 8, wide)
