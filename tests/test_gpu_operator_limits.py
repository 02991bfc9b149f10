"""The experts', 8-bit and AdamW8 operators at their limits: wait limits that run
out, elements past the 32-bit offsets, calls of two threads and of two captured
graphs at once, and the sizes that are refused."""
import threading

import pytest
import torch

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


def rand(seed, *shape, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def offsets_of(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def products(muon):
    """Calls of each kind: several tiles a pair, ragged experts, split sums, sums of several parts."""
    at, one = offsets_of([900, 0, 77, 1501, 3]), offsets_of([6001])
    x, w, dy = rand(1, 2481, 1096), rand(2, 5, 776, 1096), rand(3, 2481, 776)
    lx, ldy = rand(4, 6001, 136), rand(5, 6001, 72)
    c, s = muon.act8_store(rand(6, 1500, 2100))
    wc, ws = muon.act8_store_weight(rand(7, 3001, 2100))
    return {"forward": lambda: muon.expert_matmul(x, w, at), "input": lambda: muon.expert_matmul(dy, w, at, transpose=True),
            "weight": lambda: muon.expert_weight_grad(dy, x, at), "split": lambda: muon.expert_weight_grad(ldy, lx, one),
            "8 bits": lambda: muon.act8_matmul(c, s, wc, ws)}


@pytest.mark.parametrize("kind", ["forward", "input", "weight", "split", "8 bits"])
def test_waits_are_bounded(muon, kind):
    """A wait limit of a nanosecond: a wait that is open after its first polls gives up, the call ends, the error word
    tells, and the next call is whole again."""
    call, h = products(muon)[kind], muon.default_handle()
    want = call()
    assert h.check() == 0
    seen = set()
    try:
        h.set_timeout_ns(1)
        for _ in range(8):
            got = call()
            seen.add(h.check())
            if seen == {0}:
                assert torch.equal(want, got)
    finally:
        h.set_timeout_ns(4_000_000_000)
    assert seen <= {0, 6}
    assert torch.equal(want, call()) and h.check() == 0


def test_two_threads(muon):
    calls = products(muon)
    want = {k: f() for k, f in calls.items()}
    torch.cuda.synchronize()
    wrong = []

    def work(order):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(5):
                for k in order:
                    if not torch.equal(calls[k](), want[k]):
                        wrong.append(k)
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(o,)) for o in (list(calls), list(calls)[::-1])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_two_graphs_at_once(muon):
    """Each has scratch of its own."""
    calls = products(muon)
    want = {k: f() for k, f in calls.items()}
    graphs, kept = [], []
    for order in (list(calls), list(calls)[::-1]):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kept.append({k: calls[k]() for k in order})
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for got in kept for k in want)


# ------------------------------------------------- offsets past 32 bits
def test_far_experts(muon):
    """Inputs, results and weights of more than 2^31 elements, against the last experts alone."""
    tokens, cols, out = 2 ** 20 + 2 ** 15 + 40, 2048, 2056
    x = rand(1, 4096, cols).repeat(tokens // 4096 + 1, 1)[:tokens]
    w = rand(2, 2, out, cols)
    at = torch.tensor([0, tokens - 777, tokens - 5], dtype=torch.int32, device="cuda")
    tail = torch.tensor([0, 772], dtype=torch.int32, device="cuda")
    y = muon.expert_matmul(x, w, at)
    assert y.numel() > 2 ** 31 and x.numel() > 2 ** 31
    assert torch.equal(y[-777:-5], muon.expert_matmul(x[-777:-5], w[1:], tail)) and (y[-5:] == 0).all()
    back = muon.expert_matmul(y, w, at, transpose=True)
    assert torch.equal(back[-777:-5], muon.expert_matmul(y[-777:-5], w[1:], tail, transpose=True))
    dw = muon.expert_weight_grad(y, x, at)
    assert torch.equal(dw[1], muon.expert_weight_grad(y[-777:-5], x[-777:-5], tail)[0])
    del y, back, dw
    experts = 520
    many = offsets_of([0] * (experts - 1) + [100])
    assert experts * out * cols > 2 ** 31
    dw = muon.expert_weight_grad(rand(3, 100, out), x[:100], many, dtype=BF)
    alone = muon.expert_weight_grad(rand(3, 100, out), x[:100], offsets_of([100]), dtype=BF)
    assert torch.equal(dw[-1], alone[0]) and (dw[-2] == 0).all()
    assert torch.equal(muon.expert_matmul(x[:100], dw, many), muon.expert_matmul(x[:100], alone, offsets_of([100])))


def test_far_codes(muon):
    """A weight and a result of more than 2^31 elements, against their last rows and columns alone."""
    out, cols = 2 ** 18 + 128, 8200
    w = rand(1, 2048, cols).repeat(out // 2048 + 1, 1)[:out]
    assert w.numel() > 2 ** 31
    codes, scales, codes_t = muon.act8_store_weight(w, transposed=True)
    c, s, ct = muon.act8_store_weight(w[-128:], transposed=True)
    assert torch.equal(codes[-128:].view(torch.uint8), c.view(torch.uint8)) and torch.equal(scales[:, -1:], s)
    assert torch.equal(codes_t[:, -128:].contiguous().view(torch.uint8), ct.contiguous().view(torch.uint8))
    assert torch.equal(muon.act8_restore_weight(codes, scales)[-128:], muon.act8_restore_weight(c, s))
    xc, xs = muon.act8_store(rand(2, 260, cols))
    assert torch.equal(muon.act8_matmul(xc, xs, codes, scales)[:, -128:], muon.act8_matmul(xc, xs, c, s))
    # the result: the weight's codes as rows of activations, whose scales are a row's
    rows = 2 ** 18 + 130
    big, bs = muon.act8_store(rand(3, 1024, 256).repeat(rows // 1024 + 1, 1)[:rows])
    v, vs = muon.act8_store_weight(rand(4, 8200, 256))
    y = muon.act8_matmul(big, bs, v, vs)
    assert y.numel() > 2 ** 31
    assert torch.equal(y[-130:], muon.act8_matmul(big[-130:], bs[:, -130:], v, vs))


def test_far_elements_of_adamw8(muon):
    """Parameters do not hang on the elements' numbers, whose hash the states' rounding takes."""
    n, tail = 2 ** 31 + 128 * 33, 128 * 40 + 9
    p = torch.ones(n + 9, device="cuda", dtype=BF)
    g = torch.zeros(n + 9, device="cuda", dtype=BF)
    g[-tail:] = rand(1, tail)
    state = muon.adamw8_state(p)
    q, h = p[-tail:].clone(), g[-tail:].clone()
    muon.adamw8_step([p], [g], [state], step=1, **HYPER)
    small = muon.adamw8_state(q)
    muon.adamw8_step([q], [h], [small], step=1, **HYPER)
    assert torch.equal(p[-tail:], q) and torch.equal(p[:1000], p[1000:2000])
    assert torch.equal(state.avg_scale[-41:], small.avg_scale) and torch.equal(state.root_scale[-41:], small.root_scale)
    far = state.root[-tail:].int() - small.root.int()
    assert (far.abs() <= 1).all() and (far != 0).any()
    (m, r), = muon.adamw8_restore([state], dtype=BF)
    (sm, sr), = muon.adamw8_restore([small], dtype=BF)
    # codes of roots are 2^-4 apart at most, of averages 2^-3 or 2^-9 of the scale's unit: neighbours in both
    assert ((r[-tail:] - sr).abs() <= 2.0 ** -4 * sr).all() and (m[:1000] == 0).all()
    assert ((m[-tail:] - sm).abs() <= 2.0 ** -3 * sm.abs() + 2.0 ** -9 / 128).all()


def test_refused_sizes(muon):
    cols = 2 ** 20 + 128
    c, s = muon.act8_store(torch.zeros(1, cols, device="cuda", dtype=BF))
    w, ws = muon.act8_store_weight(torch.zeros(1, cols, device="cuda", dtype=BF))
    with pytest.raises(muon.MuonError, match="INVALID_ARG"):
        muon.act8_matmul(c, s, w, ws)
    got = muon.act8_matmul(c[:, :2 ** 20], s[:2 ** 13], w[:, :2 ** 20], ws[:2 ** 13])
    assert (got == 0).all()
    p = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError, match="Adamw8State"):
        muon.adamw8_step([p], [p.clone()], [iter(muon.adamw8_state(p))], step=1, **HYPER)
