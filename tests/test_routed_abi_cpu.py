"""Host-only tests of the routed half: the oracle's own pins, validation, workspace sizes,
and the host code under sanitizers.  No GPU: every call fails validation first or is a pure
host function."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from conftest import ROOT
from oracle import routed

binding = pytest.importorskip("moe_shared_expert_amd.binding")

BF16, FP32 = binding.SMLP_BF16, binding.SMLP_FP32
NULL, SHAPE, ALIGN, ALIAS, WORKSPACE, DTYPE, ARG = 1, 2, 3, 4, 5, 6, 8
A, B, C, D, E_, F, G, W = (0x10000000 * i for i in range(1, 9))  # far apart, never read


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIB_PATH):
        pytest.fail("libsmlp.so is not built (python -m moe_shared_expert_amd.build)")
    return binding.lib()


# ------------------------------------------------------------------ oracle pins

def test_oracle_rounding_is_the_format():
    """Every e4m3 value is kept, midpoints go to the even neighbour, the rest to the nearer."""
    code = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    v = np.unique(code[np.isfinite(code)])
    assert v.max() == 448 and np.array_equal(routed.e4m3_round(v), v)
    mid = (v[1:] + v[:-1]) / 2
    up = torch.tensor(mid, dtype=torch.float32).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(routed.e4m3_round(mid), up)
    g = np.random.default_rng(0).standard_normal(4000) * np.exp2(np.random.default_rng(1).integers(-10, 8, 4000))
    near = v[np.abs(v[None, :] - g[:, None]).argmin(axis=1)]
    assert np.array_equal(routed.e4m3_round(g), near)


def test_oracle_route_small_case_by_hand():
    logits = np.log(np.array([[1.0, 3.0, 1 / 3, 3.0, 1.0, 1.0]]))  # sigmoid: .5 .75 .25 .75 .5 .5
    ids, w = routed.route(logits, 3, renormalize=False)
    assert ids.tolist() == [[1, 3, 0]] and np.allclose(w, [[0.75, 0.75, 0.5]])
    # groups (.5 .75) (.25 .75) (.5 .5): by sum of two 1.25, 1.0, 1.0 -> groups 0 and 1
    ids, w = routed.route(logits, 3, groups=3, top_groups=2, group_top=2, scale=2.0)
    assert ids.tolist() == [[1, 3, 0]] and np.allclose(w, [[0.75, 0.75, 0.5]])
    bias = np.array([0, 0, 0.6, 0, 0, 0.3])
    ids, w = routed.route(logits, 2, bias=bias, renormalize=False)
    assert ids.tolist() == [[2, 5]] and np.allclose(w, [[0.25, 0.5]])
    ids, w = routed.route(logits, 2, score="softmax", renormalize=False)
    e = np.exp(logits[0])
    assert ids.tolist() == [[1, 3]] and np.allclose(w, e[[1, 3]] / e.sum())


def test_oracle_experts_is_the_dense_mlp_without_rounding():
    """h on a grid of the 8-bit form: the sum over experts is the plain formula."""
    rng = np.random.default_rng(2)
    x, wgu, wd = rng.standard_normal((3, 8)), rng.standard_normal((2, 8, 8)), rng.standard_normal((2, 8, 4))
    ids, w = np.array([[0, 1], [1, -1], [5, 0]]), rng.random((3, 2))
    out = routed.experts(x, ids, w, wgu, wd)[0]
    for t in range(3):
        ref = np.zeros(8)
        for j, e in enumerate(ids[t]):
            if e in (0, 1):
                g, u = wgu[e, :4] @ x[t], wgu[e, 4:] @ x[t]
                q, s = routed.quantize((g / (1 + np.exp(-g)) * u)[None].astype(np.float32))
                ref += w[t, j] * (wd[e] @ (q[0] * np.float64(s[0, 0])))
        assert np.allclose(out[t], ref)


# ------------------------------------------------------------------ refusals

def _route(L, T=4, E=64, ld=64, dtype=FP32, bias=None, ids=B, w=C, logits=A, **kw):
    o = dict(score=0, groups=1, top_groups=1, group_top=1, topk=4, renormalize=1, scale=1.0)
    o.update(kw)
    r = binding._Route(*o.values())
    return L.shared_mlp_route(logits, dtype, T, E, ld, bias, ctypes.byref(r), ids, w, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 0), (dict(T=0, logits=None), 0), (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(w=None), NULL),
    (dict(dtype=9), DTYPE), (dict(T=-1), SHAPE), (dict(ld=63), SHAPE), (dict(T=2 ** 31), SHAPE),
    (dict(E=0), ARG), (dict(E=1025, ld=2000), ARG), (dict(groups=0), ARG), (dict(groups=5), ARG),
    (dict(groups=65, E=65, ld=65), ARG), (dict(groups=4, top_groups=5), ARG), (dict(groups=4, top_groups=0), ARG),
    (dict(group_top=3, groups=4), ARG), (dict(groups=64, top_groups=9, group_top=2), ARG), (dict(topk=0), ARG),
    (dict(topk=65, E=128, ld=128), ARG), (dict(topk=17, groups=4), ARG), (dict(score=2), ARG),
    (dict(score=1, groups=4, group_top=2, top_groups=2), ARG),
    (dict(logits=A + 2), ALIGN), (dict(ids=B + 1), ALIGN), (dict(bias=D + 2), ALIGN),
    (dict(ids=A), ALIAS), (dict(w=A + 4 * 100), ALIAS), (dict(w=B), ALIAS), (dict(bias=B, ids=B), ALIAS),
])
def test_route_refusals(L, kw, status):
    assert _route(L, **kw) == status
    assert bool(L.shared_mlp_last_error()) == (status != 0)


def test_route_null_options(L):
    assert L.shared_mlp_route(A, FP32, 4, 64, 64, None, None, B, C, None) == NULL


@pytest.mark.parametrize("kw,status", [
    (dict(parts=0), 0), (dict(dtype=2), DTYPE), (dict(block=64), ARG), (dict(parts=-1), SHAPE), (dict(rows=0), SHAPE),
    (dict(cols=8, ld=8), SHAPE), (dict(cols=40, ld=40), SHAPE), (dict(ld=120), SHAPE), (dict(ld=132), SHAPE),
    (dict(rows=2 ** 30, parts=2 ** 30), SHAPE), (dict(x=None), NULL), (dict(q=None), NULL), (dict(s=None), NULL),
    (dict(x=A + 8), ALIGN), (dict(q=B + 8), ALIGN), (dict(s=C + 2), ALIGN), (dict(q=A + 64), ALIAS), (dict(s=A), ALIAS),
    (dict(s=B), ALIAS),
])
def test_quant_refusals(L, kw, status):
    o = dict(x=A, dtype=BF16, parts=2, rows=100, cols=128, ld=128, block=1, q=B, s=C)
    o.update(kw)
    assert L.shared_mlp_quant_fp8(*o.values(), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), 0), (dict(M=-1), SHAPE), (dict(K=8), SHAPE), (dict(K=24), SHAPE), (dict(N=0), SHAPE), (dict(ldy=99), SHAPE),
    (dict(M=2 ** 24), SHAPE), (dict(N=2 ** 24, ldy=2 ** 24), SHAPE), (dict(ldy=2 ** 28), SHAPE), (dict(f32=2), DTYPE),
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(ws=None), NULL), (dict(y=None), NULL), (dict(buf=None), NULL),
    (dict(x=A + 8), ALIGN), (dict(w=C + 8), ALIGN), (dict(y=E_ + 1), ALIGN), (dict(f32=1, y=E_ + 2), ALIGN),
    (dict(buf=W + 16), ALIGN), (dict(xs=B + 1), ALIGN), (dict(n=100), WORKSPACE), (dict(y=A), ALIAS), (dict(y=C), ALIAS),
    (dict(y=D), ALIAS), (dict(buf=A), ALIAS), (dict(buf=C), ALIAS), (dict(y=W), ALIAS), (dict(xs=E_), ALIAS),
])
def test_linear_refusals(L, kw, status):
    o = dict(x=A, xs=None, w=C, ws=D, y=E_, M=40, K=256, N=100, ldy=100, f32=0, buf=W, n=1 << 20)
    o.update(kw)
    assert L.shared_mlp_linear_fp8(*o.values(), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 0), (dict(T=-1), SHAPE), (dict(H=0), SHAPE), (dict(H=264), SHAPE), (dict(I=0), SHAPE), (dict(I=100), SHAPE),
    (dict(E=0), ARG), (dict(E=1025), ARG), (dict(k=0), ARG), (dict(k=65), ARG), (dict(first=-1), ARG),
    (dict(first=2 ** 31), ARG), (dict(T=2 ** 23), SHAPE), (dict(H=2 ** 20, I=2 ** 10), SHAPE),
    (dict(x=None), NULL), (dict(ids=None), NULL), (dict(w=None), NULL), (dict(gu=None), NULL), (dict(sgu=None), NULL),
    (dict(dn=None), NULL), (dict(sdn=None), NULL), (dict(out=None), NULL), (dict(buf=None), NULL),
    (dict(x=A + 8), ALIGN), (dict(ids=B + 2), ALIGN), (dict(gu=D + 8), ALIGN), (dict(out=0x90000008), ALIGN),
    (dict(buf=W + 128), ALIGN), (dict(n=1000), WORKSPACE), (dict(out=A), ALIAS), (dict(out=D + 16), ALIAS),
    (dict(buf=D), ALIAS), (dict(out=W), ALIAS), (dict(out=B), ALIAS),
])
def test_experts_refusals(L, kw, status):
    o = dict(x=A, ids=B, w=C, gu=D, sgu=E_, dn=F, sdn=G, out=0x90000000, T=16, H=256, I=128, E=4, k=2, first=0, f32=0,
             buf=W, n=1 << 24)
    o.update(kw)
    assert L.shared_mlp_experts_fp8(*o.values(), None) == status


def test_workspace_sizes(L):
    assert binding.shared_mlp_linear_fp8_workspace_bytes(0, 256, 64, False) == 0
    # x of up to 16 rows is brought to its 8-bit form inside the product
    assert binding.shared_mlp_linear_fp8_workspace_bytes(1, 7168, 2112, False) == 0
    assert binding.shared_mlp_linear_fp8_workspace_bytes(16, 1024, 132, False) == 0
    for M in (17, 100, 5000):
        assert binding.shared_mlp_linear_fp8_workspace_bytes(M, 7168, 2112, False) >= M * (7168 + 4 * 56)
    small = binding.shared_mlp_experts_fp8_workspace_bytes(1, 7168, 768, 128, 8)
    big = binding.shared_mlp_experts_fp8_workspace_bytes(8192, 7168, 768, 128, 8)
    assert 0 < small < big < 2 ** 32
    with pytest.raises(binding.SmlpError):
        binding.shared_mlp_experts_fp8_workspace_bytes(1, 7168, 768, 0, 8)
    with pytest.raises(binding.SmlpError):
        binding.shared_mlp_linear_fp8_workspace_bytes(1, 7, 64, False)
    assert L.shared_mlp_linear_fp8_workspace_bytes(1, 256, 64, 0, None) == NULL
    assert L.shared_mlp_experts_fp8_workspace_bytes(1, 256, 128, 4, 2, 0, None) == NULL


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.zeros(64, 256, dtype=binding.FP8)
    s = torch.zeros(1, 2)
    with pytest.raises(ValueError):
        binding.linear_fp8(x, w, s)                       # not on the GPU
    with pytest.raises(ValueError):
        binding.linear_fp8(x.float(), w, s)
    with pytest.raises(ValueError):
        binding.linear_fp8(x, w.float(), s)
    with pytest.raises(ValueError):
        binding.linear_fp8(x, w, s[:, :1])
    with pytest.raises(ValueError):
        binding.route(torch.zeros(4, 64), 4)
    with pytest.raises(ValueError):
        binding.quantize_fp8(x)
    with pytest.raises(ValueError):
        binding.experts_fp8(x, torch.zeros(4, 2), torch.zeros(4, 2), w, s, w[None], s)


def test_host_code_under_asan_and_ubsan(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"):
        pytest.skip("needs g++ and the ROCm headers")
    exe = str(tmp_path / "routed_sanitize")
    csrc = os.path.join(ROOT, "moe_shared_expert_amd", "csrc")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
           "-I", os.path.join(ROOT, "include"), "-I", csrc, os.path.join(csrc, "moe.cpp"),
           os.path.join(ROOT, "tests", "sanitize", "routed_driver.cpp"), "-o", exe, "-L/opt/rocm/lib", "-lamdhip64",
           "-Wl,-rpath,/opt/rocm/lib", "-pthread"]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=env)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "all checks passed" in out and "runtime error" not in out, out[-4000:]
