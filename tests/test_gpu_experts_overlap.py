"""The experts' weight gradient into memory that it shares with an operand: as
one tensor or in each other's gaps, or refused."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
E, OUT, COLS, TOKENS = 3, 24, 40, 50


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


def operands():
    return rand(1, TOKENS, OUT), rand(2, TOKENS, COLS), torch.tensor([0, 20, 20, TOKENS], dtype=torch.int32, device="cuda")


BUFFERS = {
    "columns": ((E, OUT, 2 * COLS), lambda t: (t[:, :, :COLS], t[:, :, COLS:])),
    "columns the other way round": ((E, OUT, 2 * COLS), lambda t: (t[:, :, COLS:], t[:, :, :COLS])),
    "rows by turns": ((E, 2 * OUT, COLS), lambda t: (t[:, ::2], t[:, 1::2])),
    "halves of an expert": ((E, 2 * OUT, COLS), lambda t: (t[:, OUT:], t[:, :OUT])),
    "experts by turns": ((2 * E, OUT, COLS), lambda t: (t[::2], t[1::2])),
    "one after the other": ((2 * E, OUT, COLS), lambda t: (t[:E], t[E:])),
    "an expert's gap": ((E, OUT + 30, COLS + 8), lambda t: (t[:, :OUT, :COLS], t[:, OUT:OUT + 24, 8:])),
}


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("name", list(BUFFERS))
def test_in_each_others_gaps(muon, name, dtype):
    dy, x, at = operands()
    shape, views = BUFFERS[name]
    buffer = rand(3, *shape, dtype=dtype)
    add, out = views(buffer)
    kept = add.clone()
    want = muon.expert_weight_grad(dy, x, at, add=kept)
    muon.expert_weight_grad(dy, x, at, add=add, out=out)
    assert torch.equal(out, want) and torch.equal(add, kept)
    muon.expert_weight_grad(dy, x, at, add=add, out=add)
    assert torch.equal(add, want)


OVERLAPS = {
    "the next expert": ((E + 1, OUT, COLS), lambda t: (t[:E], t[1:])),
    "the next row": ((E, OUT + 1, COLS), lambda t: (t[:, :OUT], t[:, 1:])),
    "the next columns": ((E, OUT, COLS + 8), lambda t: (t[:, :, :COLS], t[:, :, 8:])),
    "a column less than its width": ((E, OUT, 2 * COLS - 1), lambda t: (t[:, :, :COLS], t[:, :, COLS - 1:])),
    "one start, other rows": ((E * OUT * 2 * COLS,), lambda t: (t[:E * OUT * COLS].view(E, OUT, COLS), t.view(E, OUT, 2 * COLS)[:, :, :COLS])),
    "one start, other experts": ((2 * E, OUT, COLS), lambda t: (t[:E], t[::2])),
    "half an expert on": ((E, OUT + 12, COLS), lambda t: (t[:, :OUT], t[:, 12:])),
}


@pytest.mark.parametrize("name", list(OVERLAPS))
def test_overlaps_are_refused(muon, name):
    dy, x, at = operands()
    shape, views = OVERLAPS[name]
    buffer = rand(4, *shape, dtype=FP)
    before = buffer.clone()
    for add, out in (views(buffer), views(buffer)[::-1]):
        with pytest.raises(muon.MuonError, match="INVALID_ARG.*overlap"):
            muon.expert_weight_grad(dy, x, at, add=add, out=out)
    assert torch.equal(buffer, before)


def test_results_over_inputs_are_refused(muon):
    dy, x, at = rand(5, 200, 16), rand(6, 200, 40), torch.tensor([0, 90, 200], dtype=torch.int32, device="cuda")
    for out in (x[:32].view(2, 16, 40), dy.view(-1)[1280:2560].view(2, 16, 40)):
        with pytest.raises(muon.MuonError, match="INVALID_ARG.*overlap"):
            muon.expert_weight_grad(dy, x, at, out=out)
    assert torch.equal(x, rand(6, 200, 40)) and torch.equal(dy, rand(5, 200, 16))
    # behind the tokens that it reads
    both = rand(7, 300, 40)
    want = muon.expert_weight_grad(dy, both[:200], at, dtype=BF)
    assert torch.equal(muon.expert_weight_grad(dy, both[:200], at, out=both[200:232].view(2, 16, 40)), want)
