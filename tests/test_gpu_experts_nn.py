"""The autograd wrappers of the experts' and the 8-bit products, AdamW's 8-bit
states in the optimizer, and the example that trains with all of them.

Gradients are compared with torch's autograd in fp64 on the same values (norm
against norm): 16-bit results are rounded by at most 2^-8 of themselves.  Where
products run in 8 bits the reference multiplies the stored values, which the
operators give exactly."""
import os
import sys

import pytest
import torch

from _margins import record

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


@pytest.fixture(scope="module")
def muon():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    import newton_schulz_orthogonalized_muon_gb300 as pkg
    yield pkg
    torch.cuda.synchronize()
    assert pkg.default_handle().check() == 0


@pytest.fixture(scope="module")
def nn(muon):
    from newton_schulz_orthogonalized_muon_gb300 import nn as mod
    return mod


def near(name, got, ref, tol):
    err = ((got.double() - ref.double()).norm() / ref.double().norm()).item()
    record(name, err, tol)
    assert err < tol, (name, err)


def leaf(t, dtype=None):
    return t.detach().to(dtype or t.dtype).clone().requires_grad_(True)


def grouped(x, w, at):
    parts = [x[a:b] @ w[e].t() for e, (a, b) in enumerate(zip(at, at[1:]))]
    return torch.cat(parts + [torch.zeros(x.shape[0] - at[-1], w.shape[1], dtype=x.dtype, device=x.device)])


@pytest.mark.parametrize("dtype", [BF, torch.float16])
def test_expert_linear_gradients(nn, dtype):
    torch.manual_seed(1)
    at = [0, 30, 30, 97, 180]
    x, g = torch.randn(190, 64, device="cuda").to(dtype), torch.randn(190, 48, device="cuda").to(dtype)
    layer = nn.ExpertLinear(4, 64, 48, device="cuda", dtype=dtype)
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    mine = leaf(x)
    y = layer(mine, offsets)
    y.backward(g)
    ref, w = leaf(x, torch.float64), leaf(layer.weight, torch.float64)
    want = grouped(ref, w.view(4, 48, 64), at)
    want.backward(g.double())
    assert layer.weight.grad.dtype == dtype and layer.weight.grad.shape == (192, 64)
    tol = 2.0 ** -8 if dtype == BF else 2.0 ** -11
    near(f"nn experts {dtype} y", y, want, tol)
    near(f"nn experts {dtype} x", mine.grad, ref.grad, tol)
    near(f"nn experts {dtype} weight", layer.weight.grad, w.grad, tol)


def test_expert_linear_against_differences(nn):
    """The gradient of a sum of squares against a difference: a half step of 2^-8 of fp16 values, whose sum is exact to
    2^-10 of the terms."""
    torch.manual_seed(2)
    at = torch.tensor([0, 5, 20], dtype=torch.int32, device="cuda")
    x, w = torch.randn(20, 16, device="cuda").half(), torch.randn(2, 8, 16, device="cuda").half()
    xl, wl = leaf(x), leaf(w)
    c = torch.randn(20, 8, device="cuda").half()
    nn.expert_linear(xl, wl, at).backward(c)

    def value(xx, ww):
        return (grouped(xx.double(), ww.double(), [0, 5, 20]) * c.double()).sum()

    for t, grad, f in ((x, xl.grad, lambda v: value(v, w)), (w, wl.grad, lambda v: value(x, v))):
        for _ in range(5):
            d = torch.randn_like(t.double())
            slope = (f(t.double() + 0.5 * d) - f(t.double() - 0.5 * d)).item()          # linear in each: exact
            assert abs((grad.double() * d).sum().item() - slope) <= 2.0 ** -11 * (grad.double() * d).abs().sum().item() + 1e-3


def test_gradients_that_nobody_wants_and_watched_offsets(nn):
    at = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    x, w = torch.randn(8, 16, device="cuda").to(BF), torch.randn(2, 8, 16, device="cuda").to(BF)
    xl = leaf(x)
    nn.expert_linear(xl, w, at).sum().backward()
    wl = leaf(w)
    nn.expert_linear(x, wl, at).sum().backward()
    assert xl.grad is not None and wl.grad is not None
    y = nn.expert_linear(leaf(x), wl, at)
    at.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("wants", [(True, True), (True, False), (False, True)])
def test_linear8_with_8_bit_products(muon, nn, wants):
    torch.manual_seed(3)
    x, g = torch.randn(3, 50, 200, device="cuda").to(BF), torch.randn(3, 50, 136, device="cuda").to(BF)
    w = (torch.randn(136, 200, device="cuda") / 14).to(BF)
    xl, wl = x.clone().requires_grad_(wants[0]), w.clone().requires_grad_(wants[1])
    y = nn.linear8(xl, wl, products8=True)
    y.backward(g)

    def kept(t):
        return muon.act8_restore(*muon.act8_store(t.reshape(-1, t.shape[-1])), dtype=torch.float32).double()

    wk = muon.act8_restore_weight(*muon.act8_store_weight(w), dtype=torch.float32).double()
    near("nn linear8 products y", y.reshape(150, 136), kept(x) @ wk.t(), 2.0 ** -8)
    if wants[0]:
        near("nn linear8 products x", xl.grad.reshape(150, 200), kept(g) @ wk, 2.0 ** -8)
    if wants[1]:
        near("nn linear8 products weight", wl.grad, g.reshape(150, 136).double().t() @ kept(x), 2.0 ** -8)
    with torch.no_grad():
        assert torch.equal(nn.linear8(x, w, products8=True), y)


def test_expanded_gradients(nn):
    at = torch.tensor([0, 7, 20], dtype=torch.int32, device="cuda")
    x, w = torch.randn(20, 64, device="cuda").to(BF), torch.randn(2, 32, 64, device="cuda").to(BF)
    for f in (lambda a, b: nn.expert_linear(a, b, at), lambda a, b: nn.linear8(a, b[0], products8=True)):
        one, two = [leaf(x), leaf(w)], [leaf(x), leaf(w)]
        f(*one).sum().backward()                     # stride 0
        y = f(*two)
        y.backward(torch.ones_like(y))
        assert torch.equal(one[0].grad, two[0].grad) and torch.equal(one[1].grad, two[1].grad)


def test_a_captured_step(muon, nn):
    """Forward, backward and the optimizer's 8-bit step in one graph, against the same calls outside."""
    torch.manual_seed(4)
    at = torch.tensor([0, 40, 96], dtype=torch.int32, device="cuda")
    x = torch.randn(96, 64, device="cuda").to(BF)
    layer, norm = nn.ExpertLinear(2, 64, 64, device="cuda"), nn.LayerNorm(64, device="cuda", dtype=BF)
    states = [muon.adamw8_state(p) for p in norm.parameters()]
    hyper = dict(step=3, lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.1)
    params = [layer.weight, *norm.parameters()]

    def step():
        grads = torch.autograd.grad(layer(norm(x), at).float().square().mean(), params)
        with torch.no_grad():
            muon.adamw8_step(list(norm.parameters()), list(grads[1:]), states, **hyper)
        return grads

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    before = [t.detach().clone() for t in [*norm.parameters(), *[s for st in states for s in st]]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = step()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.detach().clone() for t in [*norm.parameters(), *[s for st in states for s in st]]]
    with torch.no_grad():
        for t, b in zip([*norm.parameters(), *[s for st in states for s in st]], before):
            t.copy_(b)
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    assert all(torch.equal(a.view(torch.uint8), b.detach().view(torch.uint8))
               for a, b in zip(got, [*norm.parameters(), *[s for st in states for s in st]]))


def make(muon, seed, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    named = [("a.weight", (96, 64)), ("a.bias", (96,)), ("embed.weight", (130, 64)), ("norm.weight", (64,))]
    params = [(n, torch.nn.Parameter(torch.randn(s, generator=g, device="cuda").to(BF))) for n, s in named]
    return params, muon.Muon(params, lr=0.02, adamw_lr=1e-2, **kw)


def gradients(params, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    for _, p in params:
        p.grad = torch.randn(p.shape, generator=g, device="cuda").to(BF)


def test_optimizer_with_8_bit_states(muon):
    params, opt = make(muon, 5, adamw_states=8)
    plain, other = make(muon, 5)
    states = [muon.adamw8_state(p) for n, p in plain if n != "a.weight"]
    for step in range(1, 4):
        gradients(params, step)
        gradients(plain, step)
        opt.step()
        with torch.no_grad():
            muon.adamw8_step([p for n, p in plain if n != "a.weight"], [p.grad for n, p in plain if n != "a.weight"], states,
                             step=step, lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.1)
    for (n, p), (_, q) in zip(params, plain):
        if n != "a.weight":
            assert torch.equal(p, q), n
    # saved, loaded into another one, and going on alike
    saved = opt.state_dict()
    copies = [(n, torch.nn.Parameter(p.detach().clone())) for n, p in params]
    again = muon.Muon(copies, lr=0.5, adamw_states=8)
    again.load_state_dict(saved)
    for o, ps in ((opt, params), (again, copies)):
        gradients(ps, 9)
        o.step()
    assert all(torch.equal(p, q) for (_, p), (_, q) in zip(params, copies))
    with pytest.raises(ValueError, match="not kept in 32 bits"):
        other.load_state_dict(saved)
    with pytest.raises(ValueError, match="not kept in 8 bits"):
        again.load_state_dict(other.state_dict())
    with pytest.raises(ValueError, match="adamw_states"):
        make(muon, 5, adamw_states=16)


def test_experts_are_orthogonalised_apart_with_their_own_scale(muon, nn):
    """A weight of experts one below the other against one parameter an expert."""
    torch.manual_seed(6)
    w = torch.randn(3 * 64, 48, device="cuda").to(BF)
    g = torch.randn(3 * 64, 48, device="cuda").to(BF)
    whole = torch.nn.Parameter(w.clone())
    apart = [torch.nn.Parameter(w[64 * e:64 * e + 64].clone()) for e in range(3)]
    one = muon.Muon([("up.weight", whole)], lr=0.1, split_heads={"up.weight": 3}, scale_dims={"up.weight": 64})
    three = muon.Muon([(f"up{e}.weight", p) for e, p in enumerate(apart)], lr=0.1)
    whole.grad = g.clone()
    for e, p in enumerate(apart):
        p.grad = g[64 * e:64 * e + 64].clone()
    one.step()
    three.step()
    assert torch.equal(whole.detach(), torch.cat([p.detach() for p in apart]))


@pytest.mark.parametrize("kw", [dict(experts=4), dict(experts=4, bits=8), dict(bits=8)])
def test_the_example_trains(kw):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_block
    finally:
        sys.path.pop(0)
    losses = train_block.train(steps=3, dim=128, heads=2, seq=64, batch=4, layers=2, log=None, **kw)
    assert len(losses) == 3 and all(torch.isfinite(torch.tensor(losses)))
