"""AdamW with states in 8 bits over many steps, against averages in 64 bits.

What rounding that is right on average leaves, s a code's step as a part of the
value, 1/32 to 1/16 (roots) or 1/16 to 1/8 (m):
  zero gradients  a root moves by (1 - beta2) / 2 of itself each step, which adds
                  (1 - beta2) / 2 s to its relative variance: s after 2 / (1 - beta2)
                  steps, so the mean of 32768 roots is within 7 (1/16 / 32768)^(1/2)
                  = 0.01 and their squares' mean at most 1/16 too large, and as much;
  constant ones   a state goes to and fro between the codes around its value: squares
                  off by at most 2 (1/32)^2, and what fp32 loses, 2^-23 of a root each
                  step against (1 - beta2) / 2: 0.3%; together below 2%;
  normal ones     moves of 0.97 (1 - beta2) / 2 on average give a root a relative
                  variance of 0.242 s, its square's mean (where E[g^2 / r] = E[r]) an
                  excess of twice that, 1.5% to 3.0%; -1% to 4.5% with what is above.
"""
import numpy as np
import pytest
import torch

from oracle import ops_oracle as oo

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


def state_of(muon, n, exponent):
    """m and root 2^exponent each, by the format's rule: codes 1.0 2^8 and 1.0 2^7."""
    kw = dict(dtype=torch.uint8, device="cuda")
    return muon.Adamw8State(torch.full((n,), 0x78, **kw).view(torch.float8_e4m3fn), torch.full((n,), 0xF0, **kw),
                            torch.full((n // 128,), 119 + exponent, **kw), torch.full((n // 128,), 120 + exponent, **kw))


def settle(muon, gradient, start, steps, beta1, beta2, n=32768):
    """(m, r) that the states end with, and the 64-bit averages of the same gradients."""
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    state = state_of(muon, n, start)
    m = torch.full((n,), 2.0 ** start, device="cuda", dtype=torch.float64)
    v = m * m
    if gradient != "normal":
        g.fill_(gradient)
    for step in range(1, steps + 1):
        if gradient == "normal":
            g.normal_(generator=gen)
        muon.adamw8_step([p], [g], [state], step=step, lr=1e-6, beta1=beta1, beta2=beta2, eps=1e-8, wd=0.0)
        d = g.double()
        m.lerp_(d, 1 - beta1)
        v.lerp_(d.square_(), 1 - beta2)
    (avg, root), = muon.adamw8_restore([state])
    return avg.double(), root.double(), m, v


@pytest.mark.parametrize("beta2", [0.98, 0.999, 0.9999])
def test_zero_gradients(muon, beta2):
    _, r, _, v = settle(muon, 0.0, 0, round(2 / (1 - beta2)), 0.9, beta2)
    assert abs(r.mean() / v.sqrt().mean() - 1) < 0.01
    assert -0.02 < r.square().mean() / v.mean() - 1 < 0.0645 + 0.02


@pytest.mark.parametrize("gradient,start", [(0.5, 0), (0.55, 0), (0.9, -1), (1.1, 0)])
@pytest.mark.parametrize("beta2", [0.95, 0.999, 0.9999])
def test_constant_gradients(muon, beta2, gradient, start):
    _, r, _, v = settle(muon, gradient, start, round(5 / (1 - beta2)), 0.9, beta2)
    assert abs(r.square().mean() / v.mean() - 1) < 0.02


@pytest.mark.parametrize("beta2", [0.95, 0.999, 0.9999])
def test_normal_gradients(muon, beta2):
    _, r, _, v = settle(muon, "normal", 0, round(5 / (1 - beta2)), 0.9, beta2)
    assert -0.01 < r.square().mean() / v.mean() - 1 < 0.045


@pytest.mark.parametrize("beta1", [0.9, 0.99, 0.999])
def test_slow_averages_of_gradients(muon, beta1):
    """Linear in m: right on average up to the dead zone of a byte at beta1 = 0.9, 1/512 of a step of 1/8 over 0.1."""
    for gradient, start in ((0.55, 0), (0.9, -1)):
        m, _, ref, _ = settle(muon, gradient, start, round(8 / (1 - beta1)), beta1, 0.95)
        assert abs(m.mean() / ref.mean() - 1) < 0.005


@pytest.mark.parametrize("beta1,beta2", [(0.9, 0.999), (0.99, 0.95), (0.97, 0.97), (31 / 32, 31 / 32)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_codes_of_one_step(muon, beta1, beta2, dtype):
    """The codes that the rule gives for the 64-bit values, where those are not within 2^-12 of a step of the next."""
    n, seed = 40000, 12345
    gen = torch.Generator(device="cuda").manual_seed(2)
    p, g = (torch.randn(n, generator=gen, device="cuda").to(dtype) for _ in range(2))
    state = muon.adamw8_state(p)
    hyper = dict(lr=1e-2, beta1=beta1, beta2=beta2, eps=1e-8, wd=0.1)
    for step in (1, 2):
        before = [t.view(torch.uint8).cpu().numpy() for t in state]
        p0 = p.double().cpu().numpy()
        muon.adamw8_step([p], [g], [state], step=step, seed=seed, **hyper)
        _, m, r = oo.adamw8_step(p0, g.double().cpu().numpy(), *oo.adamw8_decode(*before), step, **hyper)
        noise = oo.adamw8_noise(n, seed, max(beta1, beta2))
        avg, root, avg_scale, root_scale = (t.view(torch.uint8).cpu().numpy() for t in state)
        for got, scale, x, table, largest, least in ((avg & 0x7F, avg_scale, m, oo.e4m3_table()[:0x7F], 448.0, 0),
                                                     (root, root_scale, r, oo.root_table(), 248.0, 1)):
            want, want_s, near = oo.adamw8_codes(np.abs(x), noise, table, largest, least, scale)
            assert np.array_equal(scale, want_s)
            sure = near > 2.0 ** -12
            assert sure.mean() > 0.99 and np.array_equal(got[sure], want[sure])
