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
        def __init__(self, stream, device):
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


class FakeTensor:
    """Stands for a tensor of GPU 1 (nothing reads it)."""
    is_cuda, device = True, torch.device("cuda:1")

    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, torch.Size(shape)

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        st = [1]
        for n in reversed(self.shape[1:]):
            st.insert(0, st[0] * n)
        return st if i is None else st[i]

    def get_device(self):
        return 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 1


@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_with_the_tensors_gpu_current(monkeypatch, current):
    """A default stream's handle names no GPU: a launch on it goes to the current one."""
    now, seen = [current], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *_):
            now[0] = self.before

    class Library:
        def __getattr__(self, name):
            return lambda *a: (seen.append((name, now[0])), 0)[1]

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    monkeypatch.setattr(binding, "lib", Library)
    f = FakeTensor
    bf, f32, i32, f8 = torch.bfloat16, torch.float32, torch.int32, binding.FP8
    buf = f(torch.uint8, 1 << 20)
    binding.shared_mlp_route(f(f32, 4, 64), f(i32, 4, 2), f(f32, 4, 2))
    binding.shared_mlp_quant_fp8(f(bf, 4, 128), f(f8, 4, 128), f(f32, 4, 1))
    binding.shared_mlp_linear_fp8(f(bf, 4, 128), f(f8, 64, 128), f(f32, 1, 1), f(bf, 4, 64), workspace=buf)
    binding.shared_mlp_experts_fp8(f(bf, 4, 128), f(i32, 4, 2), f(f32, 4, 2), f(f8, 2, 256, 128), f(f32, 2, 2, 1),
                                   f(f8, 2, 128, 128), f(f32, 2, 1, 1), f(bf, 4, 128), workspace=buf)
    assert [g for _, g in seen] == [1] * 4 and len({n for n, _ in seen}) == 4 and now == [current]


def test_a_stream_of_another_gpu_is_refused(monkeypatch):
    class Stream:
        cuda_stream, device = 0x77, torch.device("cuda:0")

    x = FakeTensor(torch.bfloat16, 4, 128)
    ids, weights = FakeTensor(torch.int32, 4, 2), FakeTensor(torch.float32, 4, 2)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    for call in (lambda: binding.shared_mlp_route(x, ids, weights, stream=Stream()),
                 lambda: binding.route(x, 2, stream=Stream()), lambda: binding.quantize_fp8(x, stream=Stream()),
                 lambda: binding.linear_fp8(x, x, x, stream=Stream()),
                 lambda: binding.experts_fp8(x, x, x, x, x, x, x, stream=Stream())):
        with pytest.raises(ValueError, match="stream"):
            call()
