"""AdamW with states in 8 bits where gradients are finite and their squares are
not."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def muon():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import newton_schulz_orthogonalized_muon_gb300 as pkg
    torch.cuda.set_device(0)
    yield pkg
    torch.cuda.synchronize()
    assert pkg.default_handle().check() == 0


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,big", [(512, 130), (512 + 77, 512 + 76), (8192, 5000)])
def test_large_gradients(muon, n, big, dtype):
    """A finite gradient is at most 2^63: its block's states stay finite, the next step's parameters too, and its
    neighbours move as they would beside a gradient of 2^63."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    p0, g0 = (torch.randn(n, generator=gen, device="cuda").to(dtype) for _ in range(2))
    hyper = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.1)
    kept = []
    for value in (2.0 ** 63, 1e20, -3e38):
        p, g = p0.clone(), g0.clone()
        g[big] = value
        state = muon.adamw8_state(p)
        for step in (1, 2):
            muon.adamw8_step([p], [g], [state], step=step, **hyper)
            assert torch.isfinite(p).all()
        (avg, root), = muon.adamw8_restore([state])
        assert torch.isfinite(avg).all() and torch.isfinite(root).all()
        assert abs(avg[big].abs().item() / (0.19 * 2.0 ** 63) - 1) <= 2 * 2.0 ** -3
        assert abs(root[big].item() / (0.0975 ** 0.5 * 2.0 ** 63) - 1) <= 2 * 2.0 ** -4
        kept.append((p[torch.arange(n, device="cuda") != big], *(t.view(torch.uint8)[torch.arange(t.numel(), device="cuda") != big]
                                                                for t in state[:2]), *state[2:]))
    for other in kept[1:]:
        assert all(torch.equal(a, b) for a, b in zip(kept[0], other))
