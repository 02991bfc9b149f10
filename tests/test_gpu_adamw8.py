"""AdamW with states in 8 bits on the GPU against its plain 64-bit form.

Tolerances.  The parameter: half a step of its type, and 2^-19 of the update's
magnitude (fp32 arithmetic of a dozen operations, two of them to 2^-22).  The
states' codes: the ones that the rule gives for the 64-bit values wherever the
part past a code plus the element's number is further than 2^-12 of a step from
1; fp32 values are off by at most 2^-20 of themselves, 2^-16 of a step of 1/16.
The scale's power of two is either of two where a block's largest is within
2^-20 of a power's limit: gradients in bf16 times 1 - beta1 = 0.1 do meet 448 2^e
(g = 4480 2^e has 8 bits), which 0.1 in fp32 puts 2^-22 above it.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.1)


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
    return t.detach().double().cpu().numpy().reshape(-1)


def flat(state):
    return [t.view(torch.uint8).cpu().numpy().reshape(-1) for t in state]


def rand(seed, *shape, dtype=FP, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


POS = oo.e4m3_table()[:0x7F]


def check(before, state, p0, p, g, step, seed, hyper=HYPER):
    m, r = oo.adamw8_decode(*before)
    new, m, r = oo.adamw8_step(host(p0), host(g), m, r, step, **hyper)
    u = 2.0 ** -8 if p.dtype == BF else 2.0 ** -24
    assert np.all(np.abs(host(p) - new) <= u * np.abs(new) + 2.0 ** -19 * np.abs(new - host(p0)) + 2.0 ** -22 * np.abs(new))
    noise = oo.adamw8_noise(len(m), seed)
    avg, root, avg_scale, root_scale = flat(state)
    for got, got_s, x, table, largest, least in ((avg, avg_scale, m, POS, 448.0, 0), (root, root_scale, r, oo.root_table(), 248.0, 1)):
        want, want_s, near = oo.adamw8_codes(np.abs(x), noise, table, largest, least, got_s)
        assert np.array_equal(got_s, want_s)
        value = got & 0x7F if table is POS else got
        sure = near > 2.0 ** -12
        assert sure.mean() > 0.99 or len(x) < 1000
        assert np.array_equal(value[sure], want[sure])
        assert np.all(np.abs(value.astype(int) - want.astype(int)) <= 1)
        if table is POS:
            assert np.all((got >> 7 == 1)[value > 0] == (x < 0)[value > 0])


@pytest.mark.parametrize("ptype,gtype", [(BF, BF), (BF, FP), (FP, BF), (FP, FP)])
def test_steps(muon, ptype, gtype):
    sizes = [(1,), (7,), (127,), (128,), (129,), (4096,), (64, 65), (3, 5000), (4095,), (12289,)]
    params = [rand(i, *s).to(ptype) for i, s in enumerate(sizes)]
    states = [muon.adamw8_state(p) for p in params]
    for step in range(1, 5):
        # gradients of very different sizes, some of them zero
        grads = [(rand(100 * step + i, *s) * torch.exp(3 * rand(200 * step + i, *s)) * 10.0 ** (-i) *
                  (rand(300 * step + i, *s) > -1)).to(gtype) for i, s in enumerate(sizes)]
        before = [flat(s) for s in states]
        old = [p.clone() for p in params]
        seed = 77 * step if step > 2 else None
        muon.adamw8_step(params, grads, states, step=step, seed=seed, **HYPER)
        for b, s, p0, p, g in zip(before, states, old, params, grads):
            check(b, s, p0, p, g, step, seed or step)
        for s, (avg, root) in zip(states, muon.adamw8_restore(states)):
            m, r = oo.adamw8_decode(*flat(s))
            assert avg.shape == s.avg.shape and np.array_equal(host(avg), m) and np.array_equal(host(root), r)
        for (a, r), (a16, r16) in zip(muon.adamw8_restore(states), muon.adamw8_restore(states, dtype=BF)):
            assert torch.equal(a, a16.float()) and torch.equal(r, r16.float())


def test_misaligned_tensors(muon):
    base = [rand(1, 9000), rand(2, 9000), torch.zeros(9000, dtype=torch.uint8, device="cuda"),
            torch.zeros(9000, dtype=torch.uint8, device="cuda")]
    p, g, m, r = (t[3:3 + 8700] for t in base)
    blocks = -(-8700 // 128)
    state = muon.Adamw8State(m, r, torch.zeros(blocks, dtype=torch.uint8, device="cuda"),
                             torch.zeros(blocks, dtype=torch.uint8, device="cuda"))
    q = p.clone()
    other = muon.adamw8_state(q)
    muon.adamw8_step([p], [g], [state], step=1, **HYPER)
    muon.adamw8_step([q], [g.clone()], [other], step=1, **HYPER)
    assert torch.equal(p, q) and all(np.array_equal(a, b) for a, b in zip(flat(state), flat(other)))
    assert (base[2][:3] == 0).all() and (base[2][8703:] == 0).all() and torch.equal(base[0][:3], rand(1, 9000)[:3])


def test_many_tensors_are_one_call(muon):
    sizes = [(13 * i) % 700 + 1 for i in range(250)]
    params = [rand(i, n).to(BF if i % 3 else FP) for i, n in enumerate(sizes)]
    grads = [rand(1000 + i, n, dtype=FP if i % 2 else BF) for i, n in enumerate(sizes)]
    apart, states, alone = [p.clone() for p in params], [muon.adamw8_state(p) for p in params], [muon.adamw8_state(p) for p in params]
    for step in (1, 2):
        muon.adamw8_step(params, grads, states, step=step, **HYPER)
        for p, g, s in zip(apart, grads, alone):
            muon.adamw8_step([p], [g], [s], step=step, **HYPER)
    assert all(torch.equal(a, b) for a, b in zip(params, apart))
    assert all(np.array_equal(a, b) for s, t in zip(states, alone) for a, b in zip(flat(s), flat(t)))


def test_an_average_that_moves_little_still_moves(muon):
    """Squares that fall from 1 to 1/4: each step is far below half a step of the codes."""
    n = 1 << 16
    p, g = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    state = muon.adamw8_state(p)
    hyper = dict(HYPER, beta2=0.999, beta1=0.99)
    v = m = 0.0
    for step in range(1, 1501):
        if step == 300:
            g.fill_(0.5)
        muon.adamw8_step([p], [g], [state], step=step, **hyper)
        gv = 1.0 if step < 300 else 0.5
        v, m = v + (1 - 0.999) * (gv * gv - v), m + (1 - 0.99) * (gv - m)
    (avg, root), = muon.adamw8_restore([state])
    # a rounding's error is below a step (1/8, 1/16) and forgotten with 1 - beta: its mean over 65536 elements below 1%;
    # squares of roots rounded right on average are too large by less than the steps' squares, 1/256 / 12 a step of the
    # last 1 / (1 - beta2) (in r: (1 - beta2) of them a step), at most 17% of v
    assert abs(avg.mean().item() / m - 1) < 0.01
    assert -0.01 < root.square().mean().item() / v - 1 < 0.17


def test_values_that_are_not_finite(muon):
    p, g = rand(1, 600), rand(2, 600)
    g[130], g[300] = float("nan"), float("inf")
    state = muon.adamw8_state(p)
    muon.adamw8_step([p], [g], [state], step=1, **HYPER)
    assert torch.isnan(p[130]) and torch.isfinite(p[:128]).all() and torch.isfinite(p[384:]).all()
    assert torch.isfinite(p[131:256]).all()
    (avg, root), = muon.adamw8_restore([state])
    for t in (avg, root):
        assert torch.isnan(t[128:384]).all() and torch.isfinite(t[:128]).all() and torch.isfinite(t[384:]).all()


def test_small_and_large_values(muon):
    p = torch.zeros(512, device="cuda")
    g = torch.cat([torch.full((128,), v, device="cuda") for v in (0.0, 1e-15, 1e15, 1.0)])
    g[300:384], g[384:400] = 1e-10, 0.0
    state = muon.adamw8_state(p)
    before, p0 = flat(state), p.clone()
    muon.adamw8_step([p], [g], [state], step=1, **HYPER)
    check(before, state, p0, p, g, 1, 1)
    root = flat(state)[1]
    assert (root[:128] == 0).all() and (root[300:384] == 1).all() and (root[384:400] == 0).all()


def test_streams_graphs_and_the_list(muon):
    def fresh():
        ps = [rand(1, 5000, dtype=BF), rand(2, 300, dtype=BF)]
        return ps, [rand(3, 5000, dtype=BF), rand(4, 300, dtype=BF)], [muon.adamw8_state(p) for p in ps]
    a, b = fresh(), fresh()
    muon.adamw8_step(*a, step=1, **HYPER)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    muon.adamw8_step(*b, step=1, stream=side, **HYPER)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a[0], b[0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        muon.adamw8_step(*a, step=2, **HYPER)
    graph.replay()
    muon.adamw8_step(*b, step=2, **HYPER)
    assert all(torch.equal(x, y) for x, y in zip(a[0], b[0]))
    assert all(np.array_equal(x, y) for s, t in zip(a[2], b[2]) for x, y in zip(flat(s), flat(t)))
    muon.adamw8_step([], [], [], step=1, **HYPER)
    assert muon.adamw8_restore([]) == []
    empty = torch.zeros(0, device="cuda")
    muon.adamw8_step([empty], [empty], [muon.adamw8_state(empty)], step=1, **HYPER)


def test_refusals(muon):
    p, g = rand(1, 256), rand(2, 256)
    s = muon.adamw8_state(p)

    def call(p=p, g=g, s=s, **kw):
        muon.adamw8_step([p], [g], [s], **dict(HYPER, step=1) | kw)

    for kw in (dict(p=p.half()), dict(g=g.half()), dict(g=g[:128]), dict(g=rand(3, 512)[::2]), dict(s=s[:3]), dict(s=p),
               dict(s=s._replace(root=s.root[:200])), dict(s=s._replace(avg_scale=s.avg_scale[:1])), dict(g=g.cpu()),
               dict(s=s._replace(avg=s.avg.float()))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ValueError):
        muon.adamw8_step([p], [g, g], [s], step=1, **HYPER)
    for kw in (dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(lr=float("nan"))):
        with pytest.raises(muon.MuonError, match="INVALID_ARG"):
            call(**kw)
    # one tensor twice, and two that overlap
    for pair in (([p, p], [s, muon.adamw8_state(p)]), ([p, rand(5, 256)], [s, s]), ([p[:200], p[100:]], None)):
        params, states = pair
        states = states or [muon.adamw8_state(q) for q in params]
        with pytest.raises(muon.MuonError, match="INVALID_ARG"):
            muon.adamw8_step(params, [rand(6, q.numel()) for q in params], states, step=1, **HYPER)
    with pytest.raises(ValueError):
        muon.adamw8_restore([s], dtype=torch.float16)
    assert ctypes.sizeof(__import__("newton_schulz_orthogonalized_muon_gb300._binding", fromlist=["x"]).MuonAdamw8C) == 64
