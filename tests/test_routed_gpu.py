"""Routing, the 8-bit block-scaled product and the routed experts on the GPU, against the
fp64 oracle.

Tolerances.  A product of n terms summed in fp32 in any order is within n 2^-24 of the sum
S of the absolute products (n: 128 terms inside a block, then the blocks); storing bf16
adds half a unit in the last of 8 bits, at most 2^-8 of the value.  In the experts, h is a sum of that kind through SiLU,
so a value of h that lies near the middle between two e4m3 values may round to either side:
two such flips per pair are allowed on top.  Routing weights: a few fp32 roundings.
"""
import numpy as np
import pytest
import torch

from oracle import routed

pytestmark = pytest.mark.gpu
binding = pytest.importorskip("moe_shared_expert_amd.binding")
DEV = torch.device("cuda:0")
U = 2.0 ** -24


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g)


# ------------------------------------------------------------------ routing

ROUTES = [
    # T, E, topk, options
    (1, 1, 1, dict(score="sigmoid")),
    (1, 256, 8, dict(score="sigmoid", bias=True, groups=8, top_groups=4, group_top=2, scale=2.5)),
    (5, 64, 64, dict(score="softmax")),
    (7, 65, 3, dict(score="softmax", renormalize=False)),
    (130, 72, 6, dict(score="softmax", groups=6, top_groups=2)),
    (33, 96, 5, dict(score="softmax", bias=True, groups=4, top_groups=3, group_top=2)),
    (64, 192, 7, dict(score="sigmoid", bias=True, renormalize=False, scale=0.5)),
    (9, 512, 16, dict(score="sigmoid", groups=64, top_groups=9, group_top=2)),
    (3, 1024, 2, dict(score="sigmoid", bias=True, groups=2, top_groups=1)),
    (1027, 160, 6, dict(score="sigmoid", bias=True, groups=8, top_groups=3, group_top=2)),
    # many tokens
    (2049, 256, 8, dict(score="sigmoid", bias=True, groups=8, top_groups=4, group_top=2, scale=2.5)),
    (2051, 96, 5, dict(score="softmax", groups=32, top_groups=7)),
    (2100, 33, 32, dict(score="softmax")),
    (2048, 20, 3, dict(score="sigmoid", groups=2, top_groups=1, group_top=2)),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", range(len(ROUTES)))
def test_route(case, dtype):
    T, E, k, opt = ROUTES[case]
    opt = dict(opt)
    g = gen(100 + case)
    logits = randn(g, T, E).to(dtype)
    bias = 0.1 * randn(g, E) if opt.pop("bias", False) else None
    ids, w = binding.route(logits.to(DEV), k, bias=None if bias is None else bias.to(DEV), **opt)
    ids, w = ids.cpu().numpy(), f64(w)
    ref_ids, ref_w = routed.route(f64(logits), k, bias=None if bias is None else f64(bias), **opt)
    s, c = routed.route_choice(f64(logits), opt["score"], None if bias is None else f64(bias))
    same = (ids == ref_ids).all(axis=1)
    assert same.mean() > 0.99
    # Another choice is right only where the choice values are within fp32 roundings.
    for t in np.nonzero(~same)[0]:
        assert len(set(ids[t])) == k
        assert np.abs(c[t, ids[t]] - c[t, ref_ids[t]]).max() <= 8 * U * max(1.0, np.abs(c[t]).max())
    # exp, sum, divide, the weights' sum and divide: under 64 + topk roundings
    assert np.abs(w - ref_w)[same].max() <= (64 + k) * U * np.abs(ref_w).max()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_ties_take_the_lower_index(score):
    logits = torch.zeros(6, 100)
    logits[1, 50:] = 1.0
    logits[2, ::2] = -0.0
    logits[3, 99] = 2.0
    logits[4] = torch.arange(100) // 10 * 0.5
    logits[5] = -float("inf")
    opt = dict(score=score, groups=5, top_groups=3)
    ids, _ = binding.route(logits.to(DEV), 8, **opt)
    ref, _ = routed.route(f64(logits), 8, **opt)
    assert np.array_equal(ids.cpu().numpy(), ref)


def test_route_masked_rows_and_nan():
    inf = float("inf")
    logits = torch.zeros(5, 40)
    logits[0] = -inf                      # nothing left
    logits[1] = -inf
    logits[1, 7] = 1.0                    # one expert left
    logits[2, 3] = float("nan")           # never chosen while others are there
    logits[3] = torch.finfo(torch.float32).min
    logits[4] = float("nan")
    for score in ("sigmoid", "softmax"):
        ids, w = binding.route(logits.to(DEV), 4, score=score)
        ids, w = ids.cpu().numpy(), f64(w)
        assert ((ids >= 0) & (ids < 40)).all() and all(len(set(r)) == 4 for r in ids)
        assert (ids[0] == [0, 1, 2, 3]).all() and (w[0] == 0).all()
        assert ids[1][0] == 7 and w[1][0] == 1 and (w[1][1:] == 0).all()
        assert 3 not in ids[2]
        assert (ids[3] == [0, 1, 2, 3]).all()
        assert np.isnan(w[4]).all()
    # sigmoid(lowest) is 0 for every expert; softmax of equal logits is uniform
    assert (f64(binding.route(logits.to(DEV), 4, score="sigmoid")[1])[3] == 0).all()
    assert np.allclose(f64(binding.route(logits.to(DEV), 4, score="softmax")[1])[3], 0.25)


def test_route_strided_logits_and_empty():
    g = gen(5)
    wide = randn(g, 20, 300).to(DEV)
    view = wide[:, 37:165]
    a = binding.route(view, 6, score="softmax")
    b = binding.route(view.contiguous(), 6, score="softmax")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ids, w = binding.route(wide[:0], 6)
    assert ids.shape == (0, 6) and w.shape == (0, 6)


# ------------------------------------------------------------------ the 8-bit form

@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(1, 16), (3, 128), (130, 144), (257, 400), (5, 7168)])
def test_quantize(shape, dtype, block_rows):
    g = gen(shape[0] + shape[1])
    x = (randn(g, *shape) * torch.exp(3 * randn(g, shape[0], 1))).to(dtype)
    x[0, :16] = 0
    q, s = binding.quantize_fp8(x.to(DEV), block_rows)
    rq, rs = routed.quantize(x.float().numpy(), block_rows)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(f64(q), rq)


def test_quantize_parts_strides_and_special_values():
    g = gen(9)
    x = randn(g, 3, 100, 272)
    q, s = binding.quantize_fp8(x.to(DEV), 128)
    for p in range(3):
        rq, rs = routed.quantize(x[p].numpy(), 128)
        assert np.array_equal(f64(q)[p], rq) and np.array_equal(s[p].cpu().numpy(), rs)
    wide = randn(g, 10, 512).to(DEV).bfloat16()
    q, s = binding.quantize_fp8(wide[:, 64:208])
    q2, s2 = binding.quantize_fp8(wide[:, 64:208].contiguous())
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
    y = torch.zeros(4, 128)
    y[1, 5] = float("nan")
    y[1, 6] = 2.0
    y[2, 9] = float("inf")
    y[3] = 1e-38
    q, s = binding.quantize_fp8(y.to(DEV))
    q = f64(q)
    assert (q[0] == 0).all() and np.isfinite(s.cpu().numpy()[[0, 1, 3]]).all()
    assert np.isnan(q[1, 5]) and q[1, 6] == 448 and np.isinf(s.cpu().numpy()[2, 0])
    assert (q[3] == 0).all()


# ------------------------------------------------------------------ the product

LINEARS = [(1, 16, 1), (1, 128, 132), (3, 144, 17), (16, 7168, 132), (17, 1024, 130), (32, 400, 257), (33, 384, 96),
           (64, 2000, 300), (129, 256, 127), (1, 8208, 40), (200, 768, 1031), (257, 1040, 512), (300, 128, 4096), (1100, 272, 260)]


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("out_fp32", [False, True])
@pytest.mark.parametrize("size", LINEARS)
def test_linear(size, out_fp32, fmt):
    M, K, N = size
    g = gen(M + K + N)
    x = randn(g, M, K).bfloat16()
    wq, ws = binding.quantize_fp8((randn(g, N, K) / K ** 0.5).to(DEV), 128)
    rq, rs = routed.quantize(x.float().numpy())
    if fmt == "fp8":
        xq, xs = binding.quantize_fp8(x.to(DEV))
    else:
        xq, xs = x.to(DEV), None
    y = torch.full((M, N + 5), float("nan"), device=DEV, dtype=torch.float32 if out_fp32 else torch.bfloat16)
    need = binding.shared_mlp_linear_fp8_workspace_bytes(M, K, N, fmt == "fp8")
    ws_buf = torch.full((max(need, 256),), 255, dtype=torch.uint8, device=DEV)
    binding.shared_mlp_linear_fp8(xq, wq, ws, y[:, :N], xs, ws_buf)
    assert torch.isnan(y[:, N:]).all()
    ref, size_ = routed.linear(routed.dequantize(rq, rs), routed.dequantize(f64(wq), ws.cpu().numpy(), 128))
    tol = (128 + routed.blocks(K) + 4) * U * size_ + (0 if out_fp32 else 2.0 ** -8 * np.abs(ref))
    err = np.abs(f64(y[:, :N]) - ref)
    assert bool((err <= tol).all()), float((err / tol).max())


def test_linear_on_many_streams():
    """The K split keeps counters for a limited number of streams; further streams do without."""
    g = gen(21)
    x = randn(g, 16, 4096).bfloat16().to(DEV)
    xl = randn(g, 64, 4096).bfloat16().to(DEV)
    wq, ws = binding.quantize_fp8(randn(g, 132, 4096).to(DEV), 128)
    one, many = binding.linear_fp8(x, wq, ws, out_fp32=True), binding.linear_fp8(xl, wq, ws, out_fp32=True)
    torch.cuda.synchronize()
    for s in [torch.cuda.Stream() for _ in range(24)]:
        a, b = binding.linear_fp8(x, wq, ws, out_fp32=True, stream=s), binding.linear_fp8(xl, wq, ws, out_fp32=True, stream=s)
        s.synchronize()
        assert (a - one).abs().max() <= 1e-5 * one.abs().max() and (b - many).abs().max() <= 1e-5 * many.abs().max()


def test_allocating_forms_equal_the_others_on_any_stream():
    d = make_experts(14, 20, 256, 128, 8, 2)
    logits = randn(gen(2), 20, 8).to(DEV)
    want = run_experts(d)
    ids, w = torch.empty_like(d["ids"]), torch.empty_like(d["weights"])
    binding.shared_mlp_route(logits, ids, w, score="softmax")
    args = (d["x"], d["ids"], d["weights"], d["qgu"], d["sgu"], d["qd"], d["sd"])
    torch.cuda.synchronize()
    for stream in (None, torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        got = [binding.route(logits, 2, score="softmax", stream=stream), binding.experts_fp8(*args, stream=stream)]
        out = torch.empty_like(want)
        binding.shared_mlp_experts_fp8(*args, out, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got[0][0], ids) and torch.equal(got[0][1], w)
        assert torch.equal(got[1], want) and torch.equal(out, want)
    with pytest.raises(ValueError):
        binding.experts_fp8(*args[:1], args[1].long(), *args[2:])
    with pytest.raises(binding.SmlpError):
        binding.route(logits, 9)
    with pytest.raises(binding.SmlpError):
        binding.linear_fp8(d["x"][:, :24].contiguous(), torch.zeros(8, 24, device=DEV).to(binding.FP8),
                           torch.ones(1, 1, device=DEV))


def test_linear_nan_stays_in_its_row():
    g = gen(3)
    x = randn(g, 40, 256).bfloat16()
    x[7, 3] = float("nan")
    x[9, 200] = float("inf")
    wq, ws = binding.quantize_fp8(randn(g, 64, 256).to(DEV), 128)
    for m in (16, 40):
        y = binding.linear_fp8(x[:m].to(DEV), wq, ws, out_fp32=True).cpu()
        bad = [r for r in (7, 9) if r < m]
        assert torch.isnan(y[bad]).all()
        assert torch.isfinite(y[[r for r in range(m) if r not in bad]]).all()


# ------------------------------------------------------------------ the experts

def make_experts(seed, T, H, I, E, k, every=None, dtype=torch.bfloat16):
    g = gen(seed)
    x = randn(g, T, H).to(dtype)
    wgu = randn(g, 2 * E, I, H) / H ** 0.5
    wd = randn(g, E, H, I) / I ** 0.5
    qgu, sgu = binding.quantize_fp8(wgu.to(DEV), 128)
    qd, sd = binding.quantize_fp8(wd.to(DEV), 128)
    every = E if every is None else every
    ids = torch.stack([torch.randperm(every, generator=g)[:k] for _ in range(T)]).int() if T else torch.zeros(0, k).int()
    weights = torch.rand(T, k, generator=g)
    return dict(x=x.to(DEV), ids=ids.to(DEV), weights=weights.to(DEV), qgu=qgu.view(E, 2 * I, H),
                sgu=sgu.view(E, 2 * routed.blocks(I), routed.blocks(H)), qd=qd, sd=sd)


def run_experts(d, first=0, partial=False, workspace=None):
    out = torch.full(d["x"].shape, float("nan"), device=DEV, dtype=torch.float32 if partial else torch.bfloat16)
    T, H = d["x"].shape
    E, _, I = d["qd"].shape
    need = binding.shared_mlp_experts_fp8_workspace_bytes(T, H, I, E, d["ids"].shape[1], partial)
    ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device=DEV) if workspace is None else workspace
    binding.shared_mlp_experts_fp8(d["x"], d["ids"], d["weights"], d["qgu"], d["sgu"], d["qd"], d["sd"], out, first, ws)
    return out


def check_experts(d, out, first=0):
    E, H, I = d["qd"].shape
    partial = out.dtype == torch.float32
    q, s = routed.quantize(d["x"].float().cpu().numpy())
    nb = routed.blocks(I)
    sgu = d["sgu"].cpu().numpy()
    qgu = f64(d["qgu"])
    wgu = np.stack([np.concatenate([routed.dequantize(qgu[e, :I], sgu[e, :nb], 128),
                                    routed.dequantize(qgu[e, I:], sgu[e, nb:], 128)]) for e in range(E)])
    wd = np.stack([routed.dequantize(f64(d["qd"][e]), d["sd"][e].cpu().numpy(), 128) for e in range(E)])
    ref, size, flip, parts = routed.experts(routed.dequantize(q, s), d["ids"].cpu().numpy(), f64(d["weights"]), wgu, wd, first)
    # out is stored in bf16, and each pair's y may be before the sum
    k = d["ids"].shape[1]
    stored = 0.0 if partial else 2.0 ** -8 * (np.abs(ref) + 1.01 * parts)
    tol = (128 + nb + k + 8) * U * size + 2 * flip + stored + 1e-30
    err = np.abs(f64(out) - ref)
    assert bool((err <= tol).all()), float((err / tol).max())
    if np.abs(ref).max() > 0:
        rel = np.linalg.norm(err) / np.linalg.norm(ref)
        assert rel <= (5e-3 if not partial else 3e-3), rel


EXPERTS = [  # T, H, I, E, k, experts the ids range over
    (1, 16, 16, 1, 1, 1), (1, 256, 128, 8, 4, 8), (2, 272, 144, 5, 2, 5), (7, 512, 336, 3, 3, 9),
    (40, 400, 256, 16, 4, 16), (33, 128, 400, 2, 1, 2), (70, 256, 128, 4, 2, 4), (130, 384, 272, 3, 2, 6),
    (300, 144, 128, 2, 2, 2), (520, 256, 160, 2, 1, 2), (64, 128, 128, 64, 8, 64), (24, 640, 128, 300, 6, 300),
    (1700, 64, 48, 5, 3, 7), (6, 144, 2320, 3, 2, 3), (5, 128, 1296, 4, 1, 4), (1, 8208, 128, 2, 2, 2),
    (1, 144, 2320, 9, 8, 12),
]


@pytest.mark.parametrize("partial", [False, True])
@pytest.mark.parametrize("case", range(len(EXPERTS)))
def test_experts(case, partial):
    T, H, I, E, k, every = EXPERTS[case]
    d = make_experts(200 + case, T, H, I, E, k, every)
    check_experts(d, run_experts(d, partial=partial))


def test_experts_empty_and_rows_without_experts():
    d = make_experts(1, 0, 128, 128, 4, 2)
    assert run_experts(d).shape == (0, 128)
    for T in (6, 200):
        d = make_experts(2, T, 256, 128, 4, 2)
        d["ids"][0] = -1
        d["ids"][1] = torch.tensor([4, 2 ** 31 - 1])
        d["ids"][2] = torch.tensor([-2 ** 31, 3])
        d["weights"][0] = float("nan")  # never used
        out = run_experts(d)
        assert (out[:2] == 0).all()
        d["weights"][0] = 0
        check_experts(d, out)
        d["ids"][:] = -1
        assert (run_experts(d) == 0).all()


@pytest.mark.parametrize("T", [5, 40, 600])
def test_experts_uneven_and_repeated(T):
    d = make_experts(31, T, 256, 256, 6, 3)
    d["ids"][:, 0] = 4           # one expert takes a row of every token
    d["ids"][:, 1] = 4           # and some twice
    d["ids"][T // 2:, 1] = 5
    check_experts(d, run_experts(d))


@pytest.mark.parametrize("T", [4, 100])
def test_experts_parallel_ranks_add_up(T):
    d = make_experts(77, T, 256, 128, 8, 4)
    whole = run_experts(d, partial=True)
    parts = []
    for r in range(4):
        p = dict(d)
        for n in ("qgu", "sgu", "qd", "sd"):
            p[n] = d[n][2 * r:2 * r + 2].contiguous()
        out = run_experts(p, first=2 * r, partial=True)
        check_experts(p, out, 2 * r)
        parts.append(out)
    diff = (sum(parts) - whole).abs().max()
    # same products; a different order of fp32 additions, and flips of h where a rank's
    # smaller share takes another kernel
    assert diff <= 0.05 * whole.abs().max()
    assert ((sum(parts) - whole).norm() / whole.norm()) < 3e-3


def test_experts_repeat_bit_for_bit_and_other_stream():
    d = make_experts(8, 50, 384, 256, 8, 2)
    a = run_experts(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = run_experts(d)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, b)
    for _ in range(3):
        assert torch.equal(a, run_experts(d))


@pytest.mark.parametrize("T", [2, 64, 400])
def test_whole_block_in_a_graph(T):
    """Routing, experts and the 8-bit projection captured once and replayed on new inputs."""
    H, I, E, k = 256, 128, 8, 2
    d = make_experts(12, T, H, I, E, k)
    logits = torch.zeros(T, E, device=DEV)
    wq, ws = binding.quantize_fp8(torch.randn(96, H, generator=gen(4)).to(DEV), 128)
    out = torch.empty(T, H, device=DEV, dtype=torch.bfloat16)
    y = torch.empty(T, 96, device=DEV, dtype=torch.bfloat16)
    buf = torch.empty(max(256, binding.shared_mlp_experts_fp8_workspace_bytes(T, H, I, E, k)), dtype=torch.uint8,
                      device=DEV)
    lbuf = torch.empty(max(256, binding.shared_mlp_linear_fp8_workspace_bytes(T, H, 96, False)), dtype=torch.uint8,
                       device=DEV)

    def step():
        binding.shared_mlp_route(logits, d["ids"], d["weights"])
        binding.shared_mlp_experts_fp8(d["x"], d["ids"], d["weights"], d["qgu"], d["sgu"], d["qd"], d["sd"], out,
                                       workspace=buf)
        binding.shared_mlp_linear_fp8(out, wq, ws, y, workspace=lbuf)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        g = gen(seed)
        logits.copy_(torch.randn(T, E, generator=g))
        d["x"].copy_(torch.randn(T, H, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (d["ids"], d["weights"], out, y)]
        buf.fill_(255)
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (d["ids"], d["weights"], out, y)):
            assert torch.equal(a, b)
    check_experts(d, out)


@pytest.mark.parametrize("tokens", [1, 40])
def test_example_block(tokens, capsys):
    """The example's block: roundings of bf16 between its calls, and 8-bit flips behind them
    (each bf16 rounding before a quantisation moves values across an e4m3 midpoint now and
    then; a few percent of a value's spacing, in the 2-norm well under 2e-2)."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    off = module.main(["--tokens", str(tokens), "--hidden", "512", "--inter", "256", "--experts", "8", "--topk", "2",
                       "--latent", "132", "--steps", "2"])
    assert off < 2e-2


# ------------------------------------------------------------------ several tiles per workgroup

@pytest.mark.parametrize("out_fp32", [False, True])
@pytest.mark.parametrize("size", [(8192, 2300, 1280), (3000, 3001, 1040), (1900, 1890, 2048)])
def test_linear_of_many_tiles(size, out_fp32):
    """More tiles than workgroups (of 256, 128 and 64 rows).  fp32 sums as above; with bf16
    results the 8-bit instruction may be 1.8e-5 of a block's absolute products off."""
    M, K, N = size[0], size[2], size[1]
    g = torch.Generator(device=DEV).manual_seed(M)
    x, xs = binding.quantize_fp8(torch.randn(M, K, generator=g, device=DEV))
    w, ws = binding.quantize_fp8(torch.randn(N, K, generator=g, device=DEV), 128)
    x64 = x.double() * xs.double().repeat_interleave(128, 1)[:, :K]
    w64 = w.double() * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    ref, size_ = x64 @ w64.t(), x64.abs() @ w64.abs().t()
    y = binding.linear_fp8(x, w, ws, xs, out_fp32).double()
    n = 132 + routed.blocks(K)
    tol = n * U * size_ if out_fp32 else (1.8e-5 + n * U) * size_ + 2.0 ** -8 * ref.abs()
    assert bool(((y - ref).abs() <= tol).all())


def test_experts_of_many_tiles():
    """More row tiles than workgroups in both products: the same rows as in small calls, up to
    flips of h (a tile out of place would be off by the whole of its rows)."""
    T, H, I, E, k = 4096, 2048, 1152, 4, 2
    d = make_experts(6, T, H, I, E, k)
    for partial in (False, True):
        whole = run_experts(d, partial=partial).double()
        for t0 in range(0, T, 256):
            part = dict(d)
            for n in ("x", "ids", "weights"):
                part[n] = d[n][t0:t0 + 256].contiguous()
            small = run_experts(part, partial=partial).double()
            off = (whole[t0:t0 + 256] - small).norm(dim=1) / small.norm(dim=1)
            assert off.max() < 2e-2, (partial, t0, off.max())
