"""Host-side checks of the training operators (no GPU needed): the 64-bit
forms against independent statements of the same formulas, the ABI struct's
layout, and refusals that need no device."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import ops_oracle as oo

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from newton_schulz_orthogonalized_muon_gb300 import _build
    if not os.path.exists(_build.LIB_PATH):
        _build.build()
    import newton_schulz_orthogonalized_muon_gb300 as pkg
    return pkg.load_library()


def test_layer_norm_oracle_against_autograd():
    rng = np.random.default_rng(0)
    x, w, b, dy = (rng.standard_normal(s) for s in ((7, 33), (33,), (33,), (7, 33)))
    t = [torch.tensor(a, requires_grad=True) for a in (x, w, b)]
    y = torch.nn.functional.layer_norm(t[0], (33,), t[1], t[2], 1e-5)
    y.backward(torch.tensor(dy))
    yo, mean, rstd = oo.layer_norm(x, w, b, 1e-5)
    assert np.allclose(yo, y.detach().numpy(), atol=1e-12)
    for got, want in zip(oo.layer_norm_backward(dy, x, mean, rstd, w), t):
        assert np.allclose(got, want.grad.numpy(), atol=1e-12)


@pytest.mark.parametrize("nq,nk,causal,window", [(5, 9, False, 0), (9, 5, True, 0), (6, 6, True, 2), (1, 7, True, 3)])
def test_attention_oracle_against_autograd(nq, nk, causal, window):
    rng = np.random.default_rng(nq * 100 + nk)
    q, k, v, do = (rng.standard_normal(s) for s in ((nq, 4, 8), (nk, 2, 8), (nk, 2, 8), (nq, 4, 8)))
    t = [torch.tensor(a, requires_grad=True) for a in (q, k, v)]
    see = torch.tensor(oo.visible(nq, nk, causal, window))
    kk, vv = t[1].repeat_interleave(2, 1), t[2].repeat_interleave(2, 1)
    s = torch.einsum("ihd,jhd->hij", t[0], kk) * 0.3
    live = see.any(1)
    p = torch.zeros(4, nq, nk, dtype=torch.float64)
    p[:, live] = torch.softmax(s.masked_fill(~see, -torch.inf)[:, live], -1)
    o = torch.einsum("hij,jhd->ihd", p, vv)
    o.backward(torch.tensor(do))
    oo_o, lse, _ = oo.attention(q, k, v, causal, window, 0.3)
    assert np.allclose(oo_o, o.detach().numpy(), atol=1e-12)
    assert np.array_equal(np.isfinite(lse), np.tile(live.numpy(), (4, 1)))
    grads, _, _ = oo.attention_backward(do, q, k, v, oo_o, causal, window, 0.3)
    for got, want in zip(grads, t):
        assert np.allclose(got, want.grad.numpy(), atol=1e-12)


def test_act8_oracle_against_torch_casts():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((40, 300)) * np.exp(3 * rng.standard_normal(300))).astype(np.float32)
    x[3, 128:256] = 0
    x[4] *= 1e-38
    codes, scales = oo.act8_encode(x.astype(np.float64))
    unit = np.repeat(2.0 ** (scales.astype(np.float64) - 127), 128, 0)[:300].T
    cast = torch.tensor(x.astype(np.float64) / unit).float().to(torch.float8_e4m3fn)
    assert np.array_equal(cast.view(torch.uint8).numpy(), codes)
    top = np.abs(x[:, :128].astype(np.float64)).max(1) / 2.0 ** (scales[0].astype(np.float64) - 127)
    assert (top <= 448).all() and ((top > 224) | (scales[0] == 16)).all()
    assert np.array_equal(oo.act8_decode(codes, scales), cast.double().numpy() * unit)


def test_attention_struct_layout_matches_the_c_compiler(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    from newton_schulz_orthogonalized_muon_gb300._binding import MuonAttentionC as A
    names = [n for n, _ in A._fields_]
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"muon.h\"\nint main(void) {\n"
                   "printf(\"%zu\\n\", sizeof(muon_attention_t));\n"
                   + "".join(f"printf(\"%zu\\n\", offsetof(muon_attention_t, {n}));\n" for n in names) + "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(A)] + [getattr(A, n).offset for n in names]


def test_operators_reject_a_null_handle(lib):
    from newton_schulz_orthogonalized_muon_gb300._binding import MuonAttentionC
    a, out = bytes(MuonAttentionC()), ctypes.c_uint64()
    assert lib.muon_layer_norm_forward(None, None, 1, None, None, None, 1, None, None, 1, 1, 0, 0, 1e-5, None) == 1
    assert lib.muon_layer_norm_backward(None, None, 1, None, 1, None, None, None, None, 1, None, None, 1, 1, 0, 0, None,
                                        0, None) == 1
    assert lib.muon_attention_forward(None, a, None) == 1
    assert lib.muon_attention_backward(None, a, None, 0, None) == 1
    assert lib.muon_act8_store(None, None, 1, None, 128, None, 16, 1, 1, 0, None) == 1
    assert lib.muon_act8_restore(None, None, 128, None, 16, None, 1, 1, 1, 0, None) == 1
    assert lib.muon_act8_weight_grad(None, None, 1, None, 128, None, 16, None, 1, None, 1, 1, 1, 1, 0, None, 0,
                                     None) == 1
    assert lib.muon_layer_norm_workspace(None, 1, 1, ctypes.byref(out)) == 1
    assert lib.muon_attention_workspace(None, a, ctypes.byref(out)) == 1
    assert lib.muon_act8_weight_grad_workspace(None, None, 1, 1, 1, 1, ctypes.byref(out)) == 1


def test_operators_refuse_host_tensors():
    import newton_schulz_orthogonalized_muon_gb300 as muon
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    q = torch.zeros(1, 4, 2, 8, dtype=torch.bfloat16)
    for call in (lambda: muon.layer_norm(x), lambda: muon.act8_store(x), lambda: muon.attention(q, q, q),
                 lambda: muon.layer_norm_backward(x, x, x[:, 0].float(), x[:, 0].float())):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_extension_module_loads_and_checks_its_arguments(lib):
    from newton_schulz_orthogonalized_muon_gb300 import _torch_ops as native
    x = torch.zeros(4, 8)
    for call in (lambda: native.layer_norm(0, 0), lambda: native.layer_norm(0, 0, x, None, None, 1e-5),
                 lambda: native.act8_store(0, 0, "x"), lambda: native.attention(0, 0, x, x, x, True, 0, None, None, None)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        native.act8_store("handle", 0, x)


@pytest.fixture
def fake_build(tmp_path, monkeypatch):
    """build() into a folder of its own, with commands that only touch their outputs."""
    from newton_schulz_orthogonalized_muon_gb300 import _build
    ran, broken = [], set()
    monkeypatch.setattr(_build, "BUILD_DIR", str(tmp_path / "build"))
    monkeypatch.setattr(_build, "LIB_PATH", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build, "MODULE_PATH", str(tmp_path / "module.so"))
    monkeypatch.setattr(_build, "nvcc_path", lambda: "nvcc")

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        if any(b in " ".join(cmd) for b in broken):
            return subprocess.CompletedProcess(cmd, 1, "", "broken")
        with open(out, "w") as f:
            f.write(" ".join(cmd))
        ran.append(os.path.basename(out))
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(_build.subprocess, "run", run)
    return _build, ran, broken, tmp_path


def test_module_is_linked_again_for_another_torch(fake_build, monkeypatch):
    build, ran, _, tmp = fake_build
    for version in ("1.0", "2.0", "1.0", "1.0"):
        monkeypatch.setattr(torch, "__version__", version)
        ran.clear()
        build.build()
        assert f"torch_ops-{version}.o" in (tmp / "module.so").read_text()
    assert ran == []                                 # nothing changed: nothing built


def test_library_is_built_where_the_module_is_not(fake_build):
    build, ran, broken, tmp = fake_build
    broken.add("torch_ops.cpp")
    with pytest.raises(RuntimeError, match="torch_ops.cpp"):
        build.build()
    assert (tmp / "lib.so").exists() and not (tmp / "module.so").exists()
    broken.clear()
    build.build()
    assert (tmp / "module.so").exists()


# ------------------------------- experts, products and states in 8 bits
def test_expert_oracle_against_autograd():
    rng = np.random.default_rng(5)
    x, w, g = (rng.standard_normal(s) for s in ((20, 6), (4, 5, 6), (20, 5)))
    at = [0, 7, 7, 18, 19]
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    y = torch.cat([tx[a:b] @ tw[e].t() for e, (a, b) in enumerate(zip(at, at[1:]))] + [torch.zeros(1, 5, dtype=torch.float64)])
    y.backward(torch.tensor(g))
    assert np.allclose(oo.expert_matmul(x, w, at)[0], y.detach().numpy(), atol=1e-12)
    assert np.allclose(oo.expert_matmul(g, w, at, True)[0], tx.grad.numpy(), atol=1e-12)
    assert np.allclose(oo.expert_weight_grad(g, x, at)[0], tw.grad.numpy(), atol=1e-12)


def test_expert_ranges_of_offsets_that_break_the_rule():
    assert oo.expert_ranges([5, 100, 40, 90, 150], 120) == [(5, 100), (100, 100), (100, 100), (100, 120)]
    assert oo.expert_ranges([-3, 2, 1], 10) == [(0, 2), (2, 2)]


def test_weight_oracle_against_torch_casts():
    rng = np.random.default_rng(6)
    w = (rng.standard_normal((200, 300)) * np.exp(2 * rng.standard_normal((200, 1)))).astype(np.float32)
    codes, scales = oo.act8_encode_weight(w.astype(np.float64))
    unit = np.repeat(np.repeat(2.0 ** (scales.T.astype(np.float64) - 127), 128, 0)[:200], 128, 1)[:, :300]
    cast = torch.tensor(w / unit).float().to(torch.float8_e4m3fn)
    assert np.array_equal(cast.view(torch.uint8).numpy(), codes)
    assert np.array_equal(oo.act8_decode_weight(codes, scales), cast.double().numpy() * unit)
    top = np.abs(w[:128, :128]).max() / unit[0, 0]
    assert 224 < top <= 448
    # the transpose's codes are the codes transposed
    other, other_s = oo.act8_encode_weight(w.T.astype(np.float64))
    assert np.array_equal(other, codes.T) and np.array_equal(other_s, scales.T)


def test_adamw8_oracle():
    # the tables are those of the formats
    assert oo.root_table()[1] == (1 + 1 / 16) / 256 and oo.root_table()[255] == 248.0 and oo.root_table()[0] == 0
    assert (np.diff(oo.root_table()) > 0).all()
    # the noise: the bytes of the hash, uniform enough
    z = oo.adamw8_noise(1 << 16, 7)
    assert abs(z.mean() - 0.5) < 0.005 and len(np.unique(z)) == 256
    assert not np.array_equal(z, oo.adamw8_noise(1 << 16, 8))
    # rounding is right on average: the mean of many roundings of one value
    x = np.full(1 << 16, 0.3)
    x[::128] = 1.0                                  # the block's largest
    for table, largest, least in ((oo.e4m3_table()[:0x7F], 448.0, 0), (oo.root_table(), 248.0, 1)):
        codes, scales, _ = oo.adamw8_codes(x, z, table, largest, least)
        value = table[codes] * 2.0 ** (np.repeat(scales.astype(float), 128) - 127)
        assert abs(value[x == 0.3].mean() - 0.3) < 0.3 * 2.0 ** -4 / 64
    # the step itself is the 64-bit form's of AdamW
    import oracle
    rng = np.random.default_rng(8)
    p, g, m, v = rng.standard_normal(50), rng.standard_normal(50), rng.standard_normal(50), rng.random(50)
    kw = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.1)
    new, m1, r1 = oo.adamw8_step(p, g, m, np.sqrt(v), 3, **kw)
    want, m2, v2 = oracle.adamw_step(p, g, m, v, 3, **kw)
    assert np.allclose(new, want, atol=1e-13) and np.allclose(m1, m2, atol=1e-13) and np.allclose(r1 * r1, v2, atol=1e-13)


def test_new_operators_reject_a_null_handle(lib):
    out = ctypes.c_uint64()
    assert lib.muon_expert_matmul(None, None, 8, None, 8, 64, None, None, 8, 1, 8, 8, 1, 0, 1, None) == 1
    assert lib.muon_expert_weight_grad(None, None, 8, None, 8, None, None, 8, 64, None, 8, 64, 1, 8, 8, 1, 1, 0, None, 0, None) == 1
    assert lib.muon_expert_weight_grad_workspace(None, 1, 8, 8, 1, ctypes.byref(out)) == 1
    assert lib.muon_act8_store_weight(None, None, 1, None, 128, None, 128, None, 1, 1, 1, 0, None) == 1
    assert lib.muon_act8_restore_weight(None, None, 128, None, 1, 1, None, 1, 1, 1, 0, None) == 1
    assert lib.muon_act8_matmul(None, None, 128, None, 16, None, 128, None, 1, 1, None, 1, 1, 1, 1, 0, None) == 1
    assert lib.muon_adamw8_step(None, None, 0, 1, 0, 1e-3, 0.9, 0.95, 1e-8, 0.1, None) == 1
    assert lib.muon_adamw8_restore(None, None, None, None, 0, 0, None) == 1


def test_new_operators_refuse_host_tensors():
    import newton_schulz_orthogonalized_muon_gb300 as muon
    x, w, at = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(1, 8, 8, dtype=torch.bfloat16), torch.tensor([0, 4]).int()
    state = muon.adamw8_state(x)
    assert state.avg.shape == x.shape and state.avg_scale.shape == (1,)
    for call in (lambda: muon.expert_matmul(x, w, at), lambda: muon.expert_weight_grad(x, x, at), lambda: muon.act8_store_weight(x),
                 lambda: muon.act8_matmul(x, x, x, x), lambda: muon.act8_restore_weight(x, x),
                 lambda: muon.adamw8_step([x], [x], [state], step=1, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.1),
                 lambda: muon.adamw8_restore([state])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="length"):
        muon.adamw8_step([], [x], [], step=1, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.1)


def test_adamw8_struct_layout_matches_the_c_compiler(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    from newton_schulz_orthogonalized_muon_gb300._binding import MuonAdamw8C as A
    names = [n for n, _ in A._fields_]
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"muon.h\"\nint main(void) {\n"
                   "printf(\"%zu\\n\", sizeof(muon_adamw8_t));\n"
                   + "".join(f"printf(\"%zu\\n\", offsetof(muon_adamw8_t, {n}));\n" for n in names) + "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(A)] + [getattr(A, n).offset for n in names]
