"""The autograd wrappers of the training operators, and the example that
trains with them.

Gradients are compared with torch's autograd in fp64 on the same (bf16)
values.  A bf16 result is rounded at every operator, each rounding at most
2^-8 of its value; through the few operators of these tests the relative
error of a whole gradient stays below 2^-5 (norm against norm)."""
import os
import sys

import pytest
import torch

from _margins import record

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


@pytest.fixture(scope="module")
def nn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    from newton_schulz_orthogonalized_muon_gb300 import nn as mod
    return mod


def near(name, got, ref, tol=2.0 ** -5):
    err = ((got.double() - ref.double()).norm() / ref.double().norm()).item()
    record(name, err, tol)
    assert err < tol, (name, err)


def leaf(t, dtype=None):
    return t.detach().to(dtype or t.dtype).clone().requires_grad_(True)


@pytest.mark.parametrize("dtype,wdtype", [(BF, torch.float32), (torch.float16, torch.float16),
                                          (torch.float32, torch.float32)])
def test_layer_norm_gradients(nn, dtype, wdtype):
    torch.manual_seed(1)
    x, w, b = (torch.randn(3, 50, 96, device="cuda") + 1).to(dtype), torch.rand(96, device="cuda").to(wdtype), \
        torch.randn(96, device="cuda").to(wdtype)
    g = torch.randn(3, 50, 96, device="cuda").to(dtype)
    mine = [leaf(t) for t in (x, w, b)]
    nn.layer_norm(*mine).backward(g)
    ref = [leaf(t, torch.float64) for t in (x, w, b)]
    torch.nn.functional.layer_norm(ref[0], (96,), ref[1], ref[2]).backward(g.double())
    for n, a, r in zip(("x", "weight", "bias"), mine, ref):
        assert a.grad.dtype == a.dtype
        near(f"nn layer norm {dtype} {n}", a.grad, r.grad, 2.0 ** -18 if dtype == torch.float32 else 2.0 ** -8)


def test_attention_gradients_and_expanded_heads(nn):
    torch.manual_seed(2)
    q, k, v = (torch.randn(2, 150, h, 64, device="cuda").to(BF) for h in (4, 2, 2))
    mine = [leaf(t) for t in (q, k, v)]
    nn.attention(*mine, causal=True).sum().backward()          # the gradient of a sum has stride 0
    ref = [leaf(t, torch.float64) for t in (q, k, v)]
    qq = ref[0].transpose(1, 2)
    kk, vv = (t.transpose(1, 2).repeat_interleave(2, 1) for t in ref[1:])
    s = (qq @ kk.transpose(-1, -2)) / 8.0
    s = s.masked_fill(torch.ones(150, 150, device="cuda").triu(1).bool(), -torch.inf)
    (torch.softmax(s, -1) @ vv).sum().backward()
    for n, a, r in zip("qkv", mine, ref):
        near(f"nn attention d{n}", a.grad, r.grad)


def test_linear8_gradients(nn):
    torch.manual_seed(3)
    import newton_schulz_orthogonalized_muon_gb300 as muon
    x, w = torch.randn(5, 40, 200, device="cuda").to(BF), torch.randn(72, 200, device="cuda").to(BF)
    g = torch.randn(5, 40, 72, device="cuda").to(BF)
    a, b = leaf(x), leaf(w)
    y = nn.linear8(a, b)
    assert torch.equal(y, x @ w.t())
    y.backward(g)
    kept = muon.act8_restore(*muon.act8_store(x.flatten(0, 1)), dtype=torch.float32).double()
    near("linear8 dx", a.grad, g.double() @ w.double(), 2.0 ** -8)
    near("linear8 dw of the kept input", b.grad, g.flatten(0, 1).double().t() @ kept, 2.0 ** -8)
    # against the unrounded input: the codes' own error, at most 2^-4 of a value and about 2^-5.4 in the mean
    near("linear8 dw", b.grad, g.flatten(0, 1).double().t() @ x.flatten(0, 1).double(), 2.0 ** -4)
    with pytest.raises(ValueError):
        nn.linear8(x.float(), w.float())


def test_example_trains(nn):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_block
    finally:
        sys.path.pop(0)
    losses = train_block.train(steps=60, log=None)
    assert all(v == v for v in losses)
    # a uniform guess over 64 tokens is 4.16; copying is learned within the run
    assert losses[0] > 3.5 and min(losses[-5:]) < 1.0, losses[::10]


def test_second_derivatives_are_refused(nn):
    x, w = leaf(torch.randn(4, 64, device="cuda")), leaf(torch.rand(64, device="cuda"))
    q = leaf(torch.randn(1, 8, 1, 64, device="cuda").to(BF))
    a, b = leaf(torch.randn(8, 64, device="cuda").to(BF)), leaf(torch.randn(32, 64, device="cuda").to(BF))
    for out, arg in ((nn.layer_norm(x, w), x), (nn.attention(q, q, q, causal=True), q), (nn.linear8(a, b), b)):
        grad, = torch.autograd.grad(out.float().square().sum(), arg, create_graph=True)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(grad.float().sum(), arg)


def test_attention_offsets_are_kept_like_the_other_inputs(nn):
    """Offsets that are refilled before the backward pass raise; offsets that a saved-tensor hook moves are the ones
    that the backward pass takes."""
    torch.manual_seed(4)
    base = [torch.randn(300, 2, 64, device="cuda").to(BF) for _ in range(3)]
    g = torch.randn(300, 2, 64, device="cuda").to(BF)
    cu = torch.tensor([0, 100, 161, 300], dtype=torch.int32, device="cuda")
    want = [leaf(t) for t in base]
    nn.attention(*want, causal=True, cu_seqlens_q=cu, cu_seqlens_k=cu).backward(g)
    late = [leaf(t) for t in base]
    buf = cu.clone()
    o = nn.attention(*late, causal=True, cu_seqlens_q=buf, cu_seqlens_k=buf)
    buf.copy_(torch.tensor([0, 50, 60, 300], dtype=torch.int32))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.backward(g)
    kept = [leaf(t) for t in base]
    buf = cu.clone()
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(), lambda t: t):
        o = nn.attention(*kept, causal=True, cu_seqlens_q=buf, cu_seqlens_k=buf)
    buf.zero_()
    o.backward(g)
    for a, b in zip(want, kept):
        assert torch.equal(a.grad, b.grad)


def test_attention_gradient_that_starts_anywhere(nn):
    """The gradient of one part of a concatenation is a view into the whole's, at an odd offset."""
    torch.manual_seed(5)
    base = [torch.randn(1, 50, 2, 64, device="cuda").to(BF) for _ in range(3)]
    g = torch.randn(3 + 50 * 2 * 64, device="cuda").to(BF)
    mine, want = [leaf(t) for t in base], [leaf(t) for t in base]
    odd = leaf(torch.zeros(3, device="cuda", dtype=BF))
    torch.cat([odd, nn.attention(*mine, causal=True).flatten()]).backward(g)
    nn.attention(*want, causal=True).backward(g[3:].clone().view(1, 50, 2, 64))
    for a, b in zip(mine, want):
        assert torch.equal(a.grad, b.grad)


def test_a_written_out_is_seen_by_autograd(nn):
    import newton_schulz_orthogonalized_muon_gb300 as muon
    x, dy = torch.randn(40, 64, device="cuda").to(BF), torch.randn(40, 32, device="cuda").to(BF)
    kept, out = muon.act8_store(x), torch.ones(32, 64, device="cuda")
    w = leaf(torch.ones(32, 64, device="cuda"))
    loss = (w * out).sum()                           # keeps out for w's gradient
    version = out._version
    muon.act8_weight_grad(dy, *kept, out=out)
    assert out._version > version
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_linear8_does_no_work_for_gradients_that_nobody_wants(nn, monkeypatch):
    torch.manual_seed(6)
    x, w = torch.randn(30, 200, device="cuda").to(BF), torch.randn(72, 200, device="cuda").to(BF)
    g = torch.randn(30, 72, device="cuda").to(BF)
    both = leaf(x), leaf(w)
    nn.linear8(*both).backward(g)
    stored = []
    store = nn.ops.act8_store
    monkeypatch.setattr(nn.ops, "act8_store", lambda t: stored.append(t.shape) or store(t))
    with torch.no_grad():
        assert torch.equal(nn.linear8(*both), x @ w.t())
    frozen = leaf(x)                                 # a frozen weight: nothing is stored
    nn.linear8(frozen, w).backward(g)
    assert torch.equal(frozen.grad, both[0].grad) and stored == []
    first = leaf(w)                                  # a first layer: no product with the weight
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as prof:
        nn.linear8(x, first).backward(g)
    assert sum(e.name == "aten::mm" for e in prof.events()) == 1
    assert torch.equal(first.grad, both[1].grad) and stored == [torch.Size([30, 200])]
