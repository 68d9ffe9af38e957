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


# ------------------------------------------------------------------ offsets past 31 bits

def product_within(y, x, xs, w, ws, K, out_fp32=False):
    """y [M, n] against the product in fp64 (K <= 512: exact products, fp32 sums)."""
    x64 = x.double() * xs.double().repeat_interleave(128, 1)[:, :K]
    w64 = w.double() * ws[:, :, None, None].double().expand(-1, -1, 128, 128).permute(0, 2, 1, 3).reshape(
        ws.shape[0] * 128, -1)[:w.shape[0], :K]
    ref, size = x64 @ w64.t().contiguous(), x64.abs() @ w64.abs().t().contiguous()
    tol = (128 + routed.blocks(K) + 4) * U * size + (0 if out_fp32 else 2.0 ** -8 * ref.abs())
    return bool(((y.double() - ref).abs() <= tol).all())


def test_linear_result_past_2_31_bytes():
    """A tile of 200 rows whose 256-row frame ends behind byte 2^31 of y: the frame's missing
    rows are dropped, not stored there (row 178 from column 5741824 on)."""
    M, K, N = 200, 128, 6_000_000
    g = torch.Generator(device=DEV).manual_seed(1)
    x, xs = binding.quantize_fp8(torch.randn(M, K, generator=g, device=DEV).bfloat16())
    w, ws = binding.quantize_fp8(torch.randn(N, K, generator=g, device=DEV, dtype=torch.bfloat16), 128)
    y = binding.linear_fp8(x, w, ws, xs)
    at = (1 << 30) - 178 * N
    for c0 in (0, at - at % 128, 128 * 20000, N // 128 * 128 - 4096):
        c1 = min(N, c0 + 16384)
        assert product_within(y[:, c0:c1], x, xs, w[c0:c1], ws[c0 // 128:-(-c1 // 128)], K), c0


def test_linear_rows_far_apart():
    M, K, N, ldy = 60, 128, 64, 35_000_000
    g = torch.Generator(device=DEV).manual_seed(2)
    x, xs = binding.quantize_fp8(torch.randn(M, K, generator=g, device=DEV).bfloat16())
    w, ws = binding.quantize_fp8(torch.randn(N, K, generator=g, device=DEV), 128)
    y = torch.full((M, ldy), 3.0, dtype=torch.bfloat16, device=DEV)
    binding.shared_mlp_linear_fp8(x, w, ws, y[:, :N], xs)
    assert product_within(y[:, :N], x, xs, w, ws, K)
    assert bool((y[:, N:] == 3.0).all())


def check_columns(d, out, wgu64, cols, hcols):
    """Columns `cols` of out, one expert and one choice per token; h's columns `hcols` (whole
    groups) are the only ones with a weight in w_down."""
    q, s = routed.quantize(d["x"].float().cpu().numpy())
    x64 = routed.dequantize(q, s)
    I = hcols.numel()
    wd = f64(d["qd"][0][:, hcols][cols]) * f64(d["sd"][0][cols // 128][:, hcols // 128])
    gu = x64 @ wgu64.T
    hq, hs = routed.quantize((gu[:, :I] / (1.0 + np.exp(-gu[:, :I])) * gu[:, I:]).astype(np.float32))
    h = routed.dequantize(hq, hs)
    w = f64(d["weights"])
    ref, size = w * (h @ wd.T), w * (np.abs(h) @ np.abs(wd).T)
    step = np.maximum(np.abs(h) / 8.0, np.repeat(hs.astype(np.float64), 128, 1)[:, :I] * 2.0 ** -9)
    flip = np.stack([w[t] * (np.abs(wd) * step[t]).max(axis=1) for t in range(h.shape[0])])
    tol = (128 + routed.blocks(I) + 9) * U * size + 2 * flip + 2.0 ** -8 * 2.01 * np.abs(ref) + 1e-30
    err = np.abs(f64(out[:, cols]) - ref)
    assert bool((err <= tol).all()), float((err / tol).max())


def test_experts_wide_rows():
    """62 rows of y of one expert end behind byte 2^31.  x is zero past its first block, so the
    sums over 18 million elements stay exact."""
    T, H, I = 62, 18_000_016, 16
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    x[:, :128] = torch.randn(T, 128, generator=g, device=DEV)
    qgu, sgu = binding.quantize_fp8(torch.randn(2, I, H, generator=g, device=DEV, dtype=torch.bfloat16), 128)
    qd, sd = binding.quantize_fp8(torch.randn(1, H, I, generator=g, device=DEV, dtype=torch.bfloat16), 128)
    d = dict(x=x, ids=torch.zeros(T, 1, dtype=torch.int32, device=DEV),
             weights=torch.rand(T, 1, generator=g, device=DEV), qgu=qgu.view(1, 2 * I, H),
             sgu=sgu.view(1, 2, -1), qd=qd, sd=sd)
    out = binding.experts_fp8(x, d["ids"], d["weights"], d["qgu"], d["sgu"], qd, sd)
    wgu = torch.cat([qgu[p, :, :128].double() * sgu[p, 0, 0].double() for p in (0, 1)]).cpu().numpy()
    at = (1 << 30) - 59 * H
    cols = torch.cat([torch.arange(c, c + 512) for c in (0, at, H - 512)]).to(DEV)
    x128 = dict(d, x=x[:, :128])
    check_columns(x128, out, wgu, cols, torch.arange(I, device=DEV))


def test_experts_wide_intermediate():
    """112 rows of h on a frame of 256 rows of 18 million: offsets of the missing rows pass 32
    bits.  w_down is zero except for the columns that wrapped offsets would reach, so the sums
    stay exact."""
    T, H, I = 112, 16, 18_000_000
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    qgu, sgu = binding.quantize_fp8(torch.randn(2, I, H, generator=g, device=DEV, dtype=torch.bfloat16), 128)
    hcols = torch.cat([torch.arange(c, c + 128) for c in (0, 7_040_000, 14_080_000, I - 128)]).to(DEV)
    wd = torch.zeros(1, H, I, dtype=torch.bfloat16, device=DEV)
    wd[0][:, hcols] = torch.randn(H, hcols.numel(), generator=g, device=DEV).bfloat16()
    qd, sd = binding.quantize_fp8(wd, 128)
    d = dict(x=x, ids=torch.zeros(T, 1, dtype=torch.int32, device=DEV), weights=torch.rand(T, 1, generator=g, device=DEV),
             qgu=qgu.view(1, 2 * I, H), sgu=sgu.view(1, -1, 1), qd=qd, sd=sd)
    assert all(int(c) % 128 == 0 for c in hcols[::128])  # whole groups of h: its 8-bit form is theirs alone
    out = binding.experts_fp8(x, d["ids"], d["weights"], d["qgu"], d["sgu"], qd, sd)
    wgu = torch.cat([qgu[p][hcols].double() * sgu[p, hcols // 128].double() for p in (0, 1)]).cpu().numpy()
    check_columns(d, out, wgu, torch.arange(H, device=DEV), hcols)


# ------------------------------------------------------------------ a caller's stream

@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_on_any_stream(block_rows):
    x = randn(gen(6), 300, 1040).to(DEV)
    q, s = binding.quantize_fp8(x, block_rows)
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        q2, s2 = binding.quantize_fp8(x, block_rows, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
        # The memory belongs to that stream: the current one does not get it when it is freed.
        at, n = q2.data_ptr(), q2.numel()
        del q2, s2
        assert torch.empty(n, dtype=torch.uint8, device=DEV).data_ptr() != at


# ------------------------------------------------------------------ graphs side by side

@pytest.mark.parametrize("size", [(16, 4096, 132), (64, 4096, 1000)])  # both kernels that split K
def test_graphs_captured_on_one_stream_run_side_by_side(size):
    M, K, N = size
    cap, lanes = torch.cuda.Stream(), [torch.cuda.Stream(), torch.cuda.Stream()]
    need = max(256, binding.shared_mlp_linear_fp8_workspace_bytes(M, K, N, False))
    jobs = []
    for j in range(3):
        g = gen(40 + j)
        x = randn(g, M, K).bfloat16().to(DEV)
        w, ws = binding.quantize_fp8(randn(g, N, K).to(DEV), 128)
        jobs.append(dict(x=x, w=w, ws=ws, y=torch.empty(30, M, N, device=DEV),
                         buf=torch.empty(need, dtype=torch.uint8, device=DEV)))

    def products(job):
        for y in job["y"]:
            binding.shared_mlp_linear_fp8(job["x"], job["w"], job["ws"], y, workspace=job["buf"])

    for job in jobs:
        products(job)
    torch.cuda.synchronize()
    for job in jobs[:2]:
        job["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(job["graph"], stream=cap):
            products(job)
    for job in jobs[:2]:
        job["y"].fill_(float("nan"))
        job["graph"].replay()
        torch.cuda.synchronize()
    with torch.cuda.stream(cap):
        products(jobs[2])
    torch.cuda.synchronize()
    for job in jobs:
        job["alone"] = job["y"][0].clone()
        xq, xs = binding.quantize_fp8(job["x"])
        x64 = xq.double() * xs.double().repeat_interleave(128, 1)
        w64 = job["w"].double() * job["ws"].double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
        tol = (128 + K // 128 + 4) * U * (x64.abs() @ w64.abs().t())
        assert bool(((job["alone"].double() - x64 @ w64.t()).abs() <= tol).all())
    for _ in range(5):
        for job in jobs:
            job["y"].fill_(float("nan"))
        torch.cuda.synchronize()
        for job, lane in zip(jobs, lanes):
            with torch.cuda.stream(lane):
                job["graph"].replay()
        with torch.cuda.stream(cap):
            products(jobs[2])
        torch.cuda.synchronize()
        for job in jobs:
            assert all(torch.equal(y, job["alone"]) for y in job["y"])


# ------------------------------------------------------------------ SiLU(g) u where g u overflows

@pytest.mark.parametrize("T", [1, 3, 100, 300])
def test_experts_with_gate_times_up_past_the_range(T):
    """Half of h is SiLU(-200) 2e36 = 0, the other SiLU(-30) 1e38 = -2.8e26 (less the 8-bit
    rounding of the weights)."""
    H, I = 256, 256
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    x[:, 0] = 1
    wgu, wd = torch.zeros(2, I, H), torch.zeros(1, H, I)
    half = torch.arange(I) >= I // 2
    wgu[0, :, 0], wgu[1, :, 0] = torch.where(half, -30.0, -200.0), torch.where(half, 1e38, 2e36)
    wd[0, 0, :I // 2] = 1
    wd[0, 1, I // 2:] = 2.0 ** -6
    qgu, sgu = binding.quantize_fp8(wgu.to(DEV), 128)
    qd, sd = binding.quantize_fp8(wd.to(DEV), 128)
    gate, up = [float(f64(qgu[p, I - 1, :1].cpu())[0] * sgu[p, 1, 0].item()) for p in (0, 1)]
    ref = I // 2 * f64(qd[0, 1, -1:].cpu())[0] * sd[0, 0, 1].item() * (gate / (1 + np.exp(-gate)) * up)
    for partial in (False, True):
        out = binding.experts_fp8(x.to(DEV), torch.zeros(T, 1, dtype=torch.int32, device=DEV),
                                  torch.ones(T, 1, device=DEV), qgu.view(1, 2 * I, H), sgu.view(1, 4, 2), qd, sd,
                                  partial_fp32=partial).cpu().double()
        assert bool((out[:, 0].abs() < 1e-30).all()) and bool((out[:, 2:] == 0).all())
        # every h of the half is its group's largest: 448 times the scale, within fp32 roundings
        assert bool(((out[:, 1] - ref).abs() <= 2.0 ** -7 * abs(ref)).all()), (out[:, 1], ref)


@pytest.mark.parametrize("T", [3, 1100])
def test_experts_result_past_the_range_stays_in_its_column(T):
    """One output column overflows to infinity; its neighbours (64 columns share an exponent
    where y is held in fp16: 1100 rows of 4224) keep their values."""
    H, I = 4224, 256
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    x[:, 0] = 1
    wgu, wd = torch.zeros(1, 2 * I, H), torch.zeros(1, H, I)
    wgu[0, :, 0] = 1          # h = SiLU(1) = 0.731 everywhere
    wd[0, 5, :128], wd[0, 6, 128:], wd[0, 70, 128:] = 448.0, 1.0, -1.0
    sgu, sd = torch.ones(1, 4, H // 128), torch.tensor([1e36, 1.0]).repeat(H // 128, 1)[None].contiguous()
    out = binding.experts_fp8(x.to(DEV), torch.zeros(T, 1, dtype=torch.int32, device=DEV), torch.ones(T, 1, device=DEV),
                              wgu.to(DEV).to(binding.FP8), sgu.to(DEV), wd.to(DEV).to(binding.FP8), sd.to(DEV))
    out = out.cpu().double()
    ref = 128 / (1 + np.exp(-1.0))
    assert bool((out[:, 5] == float("inf")).all())
    for col, sign in ((6, 1), (70, -1)):
        assert bool(((out[:, col] - sign * ref).abs() <= 2.0 ** -7 * ref).all()), out[:, col]
    out[:, [5, 6, 70]] = 0
    assert bool((out == 0).all())


# ------------------------------------------------------------------ arguments

def test_route_options_past_32_bits_are_refused():
    logits = randn(gen(1), 4, 64).to(DEV)
    for kw in (dict(groups=2 ** 32 + 1), dict(top_groups=2 ** 32 + 1), dict(group_top=2 ** 32 + 1), dict(groups=-2 ** 32 + 1)):
        with pytest.raises(ValueError):
            binding.route(logits, 4, **kw)
    # any truth value is one
    a, b = binding.route(logits, 4, renormalize=2 ** 32), binding.route(logits, 4, renormalize=np.bool_(True))
    c = binding.route(logits, 4)
    assert torch.equal(a[1], c[1]) and torch.equal(b[1], c[1])
    d, e = binding.route(logits, 4, renormalize=None), binding.route(logits, 4, renormalize=False)
    assert torch.equal(d[1], e[1]) and not torch.equal(d[1], c[1])

    class NoTruth:
        def __bool__(self):
            raise KeyError("no truth value")

    with pytest.raises(KeyError):
        binding.route(logits, 4, renormalize=NoTruth())
    x = torch.zeros(2, 128, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(KeyError):
        binding.linear_fp8(x, x.to(binding.FP8), torch.ones(1, 1, device=DEV), out_fp32=NoTruth())


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_parts_of_one_row(block_rows):
    """Parts of one row: their distance is the rows' distance, whatever the unused row stride is."""
    base = randn(gen(11), 6, 4, 272).to(DEV)
    for x in (base[:, 2:3], base[:, 1].unsqueeze(1), base[2].unsqueeze(0).transpose(0, 1), base[:1, :1]):
        assert x.shape[1] == 1 and x.stride(-1) == 1
        q, s = binding.quantize_fp8(x, block_rows)
        q2, s2 = binding.quantize_fp8(x.contiguous(), block_rows)
        assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
    q, s = binding.quantize_fp8(base[:, :0], block_rows)
    assert q.shape == (6, 0, 272) and s.shape == (6, 0, 3)


# ------------------------------------------------------------------ y held in fp16

def quantized64(x):
    """What the 8-bit form of x stands for (fp64; the scale and the scaled value are fp32 numbers)."""
    rows, cols = x.shape
    pad = torch.nn.functional.pad(x.float(), (0, -cols % 128)).view(rows, -1, 128)
    a = pad.abs().amax(2, keepdim=True).clamp_min(1e-30)
    q = (pad * (448.0 * (1.0 / a))).to(binding.FP8)
    s = a / 448.0
    return (q.double() * s.double()).view(rows, -1)[:, :cols], s.double().expand(-1, -1, 128).reshape(rows, -1)[:, :cols]


def experts64(d, first=0):
    """Output, sum of absolute products, largest change by one flip of h per pair, and sum of the
    pairs' magnitudes, in fp64 on the GPU."""
    E, H, I = d["qd"].shape
    nb = routed.blocks(I)

    def blocks(q, s):
        return q.double() * s.double().repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]

    x = quantized64(d["x"])[0]
    out, size, flip, parts = (torch.zeros(x.shape, dtype=torch.float64, device=DEV) for _ in range(4))
    for e in range(E):
        t, j = (d["ids"] == e + first).nonzero(as_tuple=True)
        if not t.numel():
            continue
        g = x[t] @ blocks(d["qgu"][e, :I], d["sgu"][e, :nb]).t().contiguous()
        u = x[t] @ blocks(d["qgu"][e, I:], d["sgu"][e, nb:]).t().contiguous()
        h, s = quantized64(g / (1 + torch.exp(-g)) * u)
        w = blocks(d["qd"][e], d["sd"][e])
        p = d["weights"][t, j, None].double()
        y = p * (h @ w.t().contiguous())
        out.index_add_(0, t, y)
        parts.index_add_(0, t, y.abs())
        size.index_add_(0, t, p * (h.abs() @ w.abs().t().contiguous()))
        step = torch.maximum(h.abs() / 8, s * 2.0 ** -9)
        flip.index_add_(0, t, p * torch.cat([(w.abs() * r).amax(1)[None] for r in step]))
    return out, size, flip, parts


@pytest.mark.parametrize("partial", [False, True])
@pytest.mark.parametrize("size", [(600, 2000, 336, 24, 40, 4, 8),   # tiles of 64 rows, an H that is no multiple of 64,
                                  (301, 7168, 384, 24, 24, 4, 0),   # other ranks' experts
                                  (2048, 1040, 208, 8, 9, 2, 1)])   # tiles of 256 rows
def test_experts_of_many_pairs(size, partial):
    """Sizes whose y passes through fp16 where out is bf16, every second row of w_down 64 times
    smaller than its neighbours.

    Errors, relative and rms: rounding to bf16 1.66e-3 (half a unit, spread over the mantissas);
    g and u through the 8-bit instruction are about 1.4e-5 off, h 2e-5, which moves a share of
    2e-5 / spacing of its values by one spacing (0.09 of the value): sqrt(0.8 * 2e-5 * 0.09) =
    1.2e-3; y in fp16 2e-4.  Together 2.1e-3 (y in bf16 instead of fp16: 2.6e-3).  In fp32: h
    some 5e-7 off (sums and exponential), so 1.9e-4.  Per output: fp32 sums as elsewhere, the
    8-bit instruction's 1.8e-5 for the products and twice for h's scale, three flips per pair
    (0.1 are expected)."""
    T, H, I, E, every, k, first = size
    d = make_experts(700 + T, T, H, I, E, k, every)
    wd = randn(gen(T), E, H, I) / I ** 0.5
    wd[:, 1::2] /= 64
    d["qd"], d["sd"] = binding.quantize_fp8(wd.to(DEV), 128)
    rows = T * k / min(T * k, E)
    assert rows > 12 and T * k * H > 4 << 20
    out = binding.experts_fp8(d["x"], d["ids"], d["weights"], d["qgu"], d["sgu"], d["qd"], d["sd"], first_expert=first,
                              partial_fp32=partial).double()
    ref, size_, flip, parts = experts64(d, first)
    nb = routed.blocks(I)
    tol = (128 + nb + k + 8) * U * size_ + (2 if partial else 3) * flip + 1e-30
    if not partial:
        tol += 3 * 1.8e-5 * size_ + 2.0 ** -8 * ref.abs() + 1.01 * 2.0 ** -11 * parts
    err = (out - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    for half in (0, 1):
        rel = float(err[:, half::2].norm() / ref[:, half::2].norm())
        assert rel <= (5e-4 if partial else 2.4e-3), (half, rel)
