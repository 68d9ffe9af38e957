"""Host-only tests of the routed half's plans and binding: what the launchers are handed, and
what the Python entry points do around a call.  No GPU."""
import os
import shutil
import subprocess

import pytest
import torch

from conftest import ROOT

binding = pytest.importorskip("moe_shared_expert_amd.binding")


def test_plans_stay_inside_the_workspace(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"):
        pytest.skip("needs g++ and the ROCm headers")
    exe = str(tmp_path / "routed_plans")
    csrc = os.path.join(ROOT, "moe_shared_expert_amd", "csrc")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
           "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", csrc,
           os.path.join(csrc, "moe.cpp"), os.path.join(ROOT, "tests", "sanitize", "routed_plan_driver.cpp"), "-o", exe,
           "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-pthread"]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0 and "all checks passed" in r.stdout, (r.stdout + r.stderr)[-4000:]


def test_quantize_allocates_for_the_callers_stream(monkeypatch):
    """Memory from the current stream's pool may still be in use there when the work on the
    caller's stream starts, and is free for others as soon as the caller drops it."""
    steps = []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            steps.append(("on", self.stream))

        def __exit__(self, *_):
            steps.append("off")

    empty = torch.empty
    monkeypatch.setattr(binding, "_on", On)
    monkeypatch.setattr(binding, "shared_mlp_quant_fp8", lambda *a: steps.append("call"))
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (steps.append("empty"), empty(*a, **k))[1])
    x = torch.zeros(3, 256, dtype=torch.bfloat16)
    binding.quantize_fp8(x, stream=77)
    assert steps == [("on", 77), "empty", "empty", "call", "off"]
    steps.clear()
    q, s = binding.quantize_fp8(x, 128)
    assert steps == ["empty", "empty", "call"] and q.shape == (3, 256) and s.shape == (1, 2)


def test_library_is_linked_without_the_python_module(tmp_path, monkeypatch):
    """The C ABI needs hipcc alone: the module's compiler or headers may be missing."""
    from moe_shared_expert_amd import build as b
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libsmlp.so"))
    monkeypatch.setattr(b, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(b, "SOURCES", ["layout.cpp"])

    def no_compiler():
        raise RuntimeError("no compiler for the module")

    monkeypatch.setattr(b, "_compile_calls", no_compiler)
    with pytest.raises(RuntimeError, match="no compiler for the module"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.CALLS)
    # without torch there is nobody to use the module, and nothing to build it against
    os.remove(b.LIB)
    monkeypatch.setattr(b, "_has_torch", lambda: False, raising=False)
    assert b.build() == b.LIB and os.path.exists(b.LIB) and not os.path.exists(b.CALLS)


@pytest.mark.parametrize("name", ["groups", "top_groups", "group_top", "topk"])
def test_route_options_past_32_bits_are_refused(name):
    o = dict(score="sigmoid", groups=1, top_groups=1, group_top=1, topk=4, renormalize=True, scale=1.0)
    for v in (2 ** 32 + 1, -2 ** 32 + 1, 2 ** 31):
        with pytest.raises(ValueError):
            binding._route_options(*{**o, name: v}.values())


def test_quant_block_rows_past_32_bits_are_refused():
    class Rows:  # stands for a GPU tensor: the check comes before anything is read
        is_cuda, dtype, shape = True, torch.bfloat16, torch.Size((256, 128))

        def dim(self):
            return 2

        def stride(self, i):
            return (128, 1)[i]

    for v in (2 ** 32 + 1, 2 ** 32 + 128, -2 ** 32 + 1):
        with pytest.raises(ValueError, match="block_rows"):
            binding.shared_mlp_quant_fp8(Rows(), None, None, v)
