"""The routed half on the GPU at the edges of its ranges: few experts and many choices, rows
whose offsets pass 31 bits, caller's streams, graphs that run side by side.

Tolerances are those of tests/test_routed_gpu.py (n fp32 additions: n 2^-24 of the sum of the
absolute products; half a unit of what is stored; two flips of h per pair) where nothing else
is said."""
import numpy as np
import pytest
import torch

from oracle import routed
from test_routed_gpu import DEV, U, check_experts, f64, gen, make_experts, randn

pytestmark = pytest.mark.gpu
binding = pytest.importorskip("moe_shared_expert_amd.binding")


# ------------------------------------------------------------------ one token

@pytest.mark.parametrize("partial", [False, True])
@pytest.mark.parametrize("size", [(256, 512, 1, 13), (256, 512, 2, 26), (16, 128, 1, 64), (128, 2048, 1, 4),
                                  (512, 256, 1, 32), (144, 336, 2, 21)])
def test_one_token_of_many_choices_among_few_experts(size, partial):
    H, I, E, k = size
    d = make_experts(500 + k, 1, H, I, E, 1)
    d["ids"] = (torch.arange(k, device=DEV, dtype=torch.int32) % (E + 1))[None]  # repeats, and an expert of another rank
    d["weights"] = torch.rand(1, k, generator=gen(k)).to(DEV)
    need = binding.shared_mlp_experts_fp8_workspace_bytes(1, H, I, E, k, partial)
    buf = torch.full((need + (1 << 16),), 0xA5, dtype=torch.uint8, device=DEV)
    out = torch.full((1, H), float("nan"), device=DEV, dtype=torch.float32 if partial else torch.bfloat16)
    binding.shared_mlp_experts_fp8(d["x"], d["ids"], d["weights"], d["qgu"], d["sgu"], d["qd"], d["sd"], out,
                                   workspace=buf[:need])
    assert bool((buf[need:] == 0xA5).all())
    check_experts(d, out)
