"""What the routed half of a mixture-of-experts layer is measured on: routing to experts,
the 8-bit block-scaled matrix product, and the routed experts' SwiGLU.

`run` computes an operator in its plain form (elementary torch operations in fp32) or,
where `own` is true, through the library's binding.  Sizes are those of the library's own
layers (hidden 7168, latent width 2112 and its TP16 rank's 132, the TP8 and TP16 slices
768 and 384 of the intermediate dimension) and generic ones.

8-bit values are e4m3 (largest finite value 448).  Activations carry one fp32 scale per
row and 128 columns, weights one per 128 x 128 block; with a = max(max|x|, 1e-30) of a
group, the scale is a / 448 and the stored value x * (448 / a) rounded to nearest even,
with scale, reciprocal and product held in fp32.
"""
import math

import torch

own = False

BLOCK = 128
FP8 = torch.float8_e4m3fn
TINY = 1e-30
TOP = 448.0


def listed():
    return [
        # One decoded token through a grouped sigmoid router with a balance bias: latency.
        dict(name="route_token", op="route", tokens=1, experts=256, dtype="fp32", score="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, topk=8, renorm=True, scale=2.5),
        # A decode batch, softmax scores from bf16 logits (exact ties), no groups, odd sizes.
        dict(name="route_batch", op="route", tokens=100, experts=72, dtype="bf16", score="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, topk=6, renorm=False, scale=1.0),
        # A prompt's tokens through the grouped router.
        dict(name="route_prompt", op="route", tokens=8192, experts=256, dtype="fp32", score="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, topk=8, renorm=True, scale=2.5),
        # The merged latent projection for one token: streaming 15 MB of weights.
        dict(name="linear_token", op="linear", m=1, n=2112, k=7168, x="bf16", y="bf16"),
        # One TP16 rank's 132 rows of it for a decode batch: the smallest product.
        dict(name="linear_rank", op="linear", m=16, n=132, k=7168, x="bf16", y="bf16"),
        # A TP8 slice's down projection on activations quantised beforehand, fp32 partial.
        dict(name="linear_partial", op="linear", m=128, n=7168, k=768, x="fp8", y="fp32"),
        # Ragged everywhere: rows, columns and a last block of K that is not full.
        dict(name="linear_ragged", op="linear", m=333, n=1000, k=2000, x="bf16", y="bf16"),
        # A prompt through a full-width projection: the compute-bound end.
        dict(name="linear_prompt", op="linear", m=8192, n=7168, k=6144, x="bf16", y="bf16"),
        # One decoded token: eight experts' weights are read for eight rows.
        dict(name="experts_token", op="experts", tokens=1, hidden=7168, inter=768, experts=128, topk=8, outside=0),
        # A decode batch: most experts active with one or two rows each.
        dict(name="experts_decode", op="experts", tokens=32, hidden=7168, inter=768, experts=128, topk=8, outside=0),
        # An expert-parallel rank that holds 24 of 40 experts; rows without any local expert,
        # an intermediate width that is no multiple of 128.
        dict(name="experts_ragged", op="experts", tokens=301, hidden=2000, inter=336, experts=24, topk=4, outside=16),
        # A prompt: hundreds of rows per expert, uneven.
        dict(name="experts_prompt", op="experts", tokens=8192, hidden=7168, inter=768, experts=64, topk=8, outside=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "linear", "linear", "experts", "experts"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = _log_int(rng, 4, 448 // groups)
        score = rng.choice(["sigmoid", "softmax"])
        top_groups = rng.randint(1, groups)
        topk = rng.randint(1, min(8, top_groups * per))
        return dict(op=op, tokens=_log_int(rng, 1, 8192), experts=groups * per, dtype=rng.choice(["fp32", "bf16"]),
                    score=score, bias=score == "sigmoid", groups=groups, top_groups=top_groups,
                    group_top=rng.randint(1, 2) if score == "sigmoid" else 1, topk=topk,
                    renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]))
    if op == "linear":
        while True:
            m, n, k = _log_int(rng, 1, 8192), _log_int(rng, 16, 12288), 16 * _log_int(rng, 4, 448)
            if m * n * k <= 8192 * 7168 * 6144:
                return dict(op=op, m=m, n=n, k=k, x=rng.choice(["bf16", "bf16", "fp8"]),
                            y=rng.choice(["bf16", "bf16", "fp32"]))
    while True:
        tokens, hidden, inter = _log_int(rng, 1, 8192), 16 * _log_int(rng, 16, 448), 16 * _log_int(rng, 4, 64)
        experts, topk = _log_int(rng, 8, 128), rng.randint(1, 8)
        if tokens * topk * hidden * inter <= 8192 * 8 * 7168 * 768 and experts * hidden * inter <= 128 * 7168 * 768:
            return dict(op=op, tokens=tokens, hidden=hidden, inter=inter, experts=experts, topk=topk,
                        outside=rng.choice([0, 0, experts // 2]))


def _blocks(n):
    return -(-n // BLOCK)


def _fp8_weight(gen, parts, rows, cols, fan_in):
    """parts x rows x cols e4m3 values, N(0, 1 / fan_in) once scaled, and their block scales."""
    q = torch.empty(parts, rows, cols, dtype=FP8, device="cuda")
    for p in range(0, parts, max(1, (1 << 28) // (rows * cols))):
        part = q[p:p + max(1, (1 << 28) // (rows * cols))]
        w = torch.randn(part.shape, generator=gen, device="cuda", dtype=torch.float32)
        part.copy_(w.mul_(100.0).clamp_(-TOP, TOP))
    s = torch.rand(parts, _blocks(rows), _blocks(cols), generator=gen, device="cuda") * 0.4 + 0.8
    return q, s / (100.0 * math.sqrt(fan_in))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = dict(case)
    if case["op"] == "route":
        # Logits of about unit size around what each expert attracts; a small balance bias.
        logits = randn(case["tokens"], case["experts"]) + 0.5 * randn(case["experts"])
        s["logits"] = logits.bfloat16() if case["dtype"] == "bf16" else logits
        s["bias_v"] = 0.05 * randn(case["experts"]) if case["bias"] else None
    elif case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        x = randn(m, k).bfloat16()
        s["x_v"], s["xs"] = (_quant(x) if case["x"] == "fp8" else (x, None))
        w, ws = _fp8_weight(gen, 1, n, k, k)
        s["w"], s["ws"] = w[0], ws[0]
    else:
        t, h, i, e, k = case["tokens"], case["hidden"], case["inter"], case["experts"], case["topk"]
        s["x_v"] = randn(t, h).bfloat16()
        # The router's answer: the best of scores around each expert's popularity.
        every = e + case["outside"]
        score = randn(t, every) + 0.3 * randn(every)
        top, ids = torch.topk(score, min(k, every), dim=1)
        s["ids"] = ids.int()  # ids at or past the number of local experts belong to another rank
        s["weights"] = torch.softmax(top, dim=1)
        # gate rows, then up rows, of every expert; each half has row blocks of its own
        wgu, sgu = _fp8_weight(gen, 2 * e, i, h, h)
        s["wgu"], s["sgu"] = wgu.view(e, 2 * i, h), sgu.view(e, 2 * _blocks(i), _blocks(h))
        s["wd"], s["sd"] = _fp8_weight(gen, e, h, i, i)
    return s


# ---------------------------------------------------------------- the plain forms

def _quant(x):
    """e4m3 values and scales of the last dimension's groups of 128, and nothing else."""
    x = x.float()
    rows, cols = x.shape
    pad = torch.nn.functional.pad(x, (0, _blocks(cols) * BLOCK - cols)).view(rows, -1, BLOCK)
    amax = pad.abs().amax(dim=2).clamp_min(TINY)
    q = (pad * (TOP / amax)[:, :, None]).to(FP8)
    return q.view(rows, -1)[:, :cols].contiguous(), amax / TOP


def _dequant_rows(q, s):
    return q.float() * s.repeat_interleave(BLOCK, dim=1)[:, :q.shape[1]]


def _dequant_blocks(q, s):
    """q [..., rows, cols], s [..., row blocks, column blocks] -> fp32."""
    rows, cols = q.shape[-2:]
    s = s.repeat_interleave(BLOCK, dim=-2)[..., :rows, :]
    return q.float() * s.repeat_interleave(BLOCK, dim=-1)[..., :cols]


def _best(c, k):
    """Indices of the k largest of the last dimension, largest first, ties to the lower index."""
    return torch.sort(c, dim=-1, descending=True, stable=True)[1][..., :k]


def _route_plain(s):
    logits = s["logits"].float()
    t, e = logits.shape
    if s["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logits))
        choice = score if s["bias_v"] is None else score + s["bias_v"]
    else:
        p = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        score = p / p.sum(dim=1, keepdim=True)
        choice = logits
    if s["groups"] > 1:
        by = choice.view(t, s["groups"], -1)
        two = torch.sort(by, dim=2, descending=True)[0][:, :, :s["group_top"]]
        stay = _best(two.sum(dim=2), s["top_groups"])
        keep = torch.zeros(t, s["groups"], dtype=torch.bool, device=logits.device).scatter_(1, stay, True)
        choice = torch.where(keep[:, :, None], by, -math.inf).reshape(t, e)
    ids = _best(choice, s["topk"])
    w = score.gather(1, ids)
    if s["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return ids.int(), w * s["scale"]


def _linear_plain(s):
    x, xs = (s["x_v"], s["xs"]) if s["xs"] is not None else _quant(s["x_v"])
    y = _dequant_rows(x, xs) @ _dequant_blocks(s["w"], s["ws"]).t()
    return y if s["y"] == "fp32" else y.bfloat16()


def _experts_plain(s):
    """Pairs (token, choice) sorted by expert and cut into tiles of one expert each; the
    number of tiles is the most that any routing needs, so nothing waits for the counts."""
    x, ids, weights = s["x_v"], s["ids"].long(), s["weights"]
    t, h = x.shape
    k, e, inter = ids.shape[1], s["wgu"].shape[0], s["wd"].shape[2]
    pairs, dev = t * k, x.device
    b = 256 if pairs > 128 * e else 64 if pairs > 16 * e else 8
    tiles = pairs // b + min(e, pairs)
    flat = torch.where((ids >= 0) & (ids < e), ids, e).view(-1)
    order = torch.sort(flat, stable=True)[1]
    count = torch.zeros(e + 1, dtype=torch.long, device=dev).scatter_add_(0, flat, torch.ones_like(flat))[:e]
    start = count.cumsum(0) - count
    need = (count + b - 1) // b
    last = need.cumsum(0)
    at = torch.arange(tiles, device=dev)
    of = torch.searchsorted(last, at, right=True).clamp_max(e - 1)
    row = (at - (last - need)[of])[:, None] * b + torch.arange(b, device=dev)
    real = (row < count[of][:, None]) & (at < last[-1])[:, None]
    pair = order[(start[of][:, None] + row).clamp(0, pairs - 1)]
    xq = _dequant_rows(*_quant(x))
    xt = xq[torch.div(pair, k, rounding_mode="floor")]

    def expert(w, sc, rows):
        return _dequant_blocks(w.view(torch.uint8)[of].view(FP8).view(tiles, -1, rows, w.shape[2]),
                               sc[of].view(tiles, w.shape[1] // rows, -1, sc.shape[2])).view(tiles, w.shape[1], -1)

    gu = torch.bmm(xt, expert(s["wgu"], s["sgu"], inter).transpose(1, 2))
    gate, up = gu[:, :, :inter], gu[:, :, inter:]
    act = gate / (1.0 + torch.exp(-gate)) * up
    hq = _dequant_rows(*_quant(act.reshape(tiles * b, inter))).view(tiles, b, inter)
    y = torch.bmm(hq, expert(s["wd"], s["sd"], h).transpose(1, 2))
    out = torch.zeros(pairs + 1, h, device=dev)
    out.index_copy_(0, torch.where(real, pair, pairs).view(-1), y.view(-1, h))
    out = out[:pairs].view(t, k, h)
    local = ((ids >= 0) & (ids < e))[:, :, None]
    return torch.where(local, out * weights[:, :, None], 0.0).sum(dim=1).bfloat16()


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    if not own:
        if s["op"] == "route":
            ids, w = _route_plain(s)
            return {"ids": ids, "weights": w}
        return {"out": _linear_plain(s) if s["op"] == "linear" else _experts_plain(s)}
    from moe_shared_expert_amd import binding
    if s["op"] == "route":
        ids, w = binding.route(s["logits"], s["topk"], score=s["score"], bias=s["bias_v"], groups=s["groups"],
                               top_groups=s["top_groups"], group_top=s["group_top"], renormalize=s["renorm"],
                               scale=s["scale"])
        return {"ids": ids, "weights": w}
    if s["op"] == "linear":
        return {"out": binding.linear_fp8(s["x_v"], s["w"], s["ws"], x_scales=s["xs"], out_fp32=s["y"] == "fp32")}
    return {"out": binding.experts_fp8(s["x_v"], s["ids"], s["weights"], s["wgu"], s["sgu"], s["wd"], s["sd"])}


def work(case):
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        return {"bytes": t * e * (2 if case["dtype"] == "bf16" else 4) + (4 * e if case["bias"] else 0) + 8 * t * k,
                "flops": 4 * t * e}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        x = 2 * m * k if case["x"] == "bf16" else m * k + 4 * m * _blocks(k)
        return {"bytes": x + n * k + 4 * _blocks(n) * _blocks(k) + (4 if case["y"] == "fp32" else 2) * m * n,
                "flops": 2 * m * n * k}
    t, h, i, e, k = case["tokens"], case["hidden"], case["inter"], case["experts"], case["topk"]
    every = e + case["outside"]
    k = min(k, every)
    active = e * (1.0 - (1.0 - k / every) ** t)  # experts that some token chose, for even routing
    scales = 4 * (2 * _blocks(i) * _blocks(h) + _blocks(h) * _blocks(i))
    return {"bytes": int(active * (3 * h * i + scales)) + 4 * t * h + 8 * t * k,
            "flops": int(6 * t * k * e / every * h * i)}


# ---------------------------------------------------------------- the definition in 64 bits

def _e4m3(v):
    """v rounded to the nearest e4m3 value, ties to even (|v| is at most 448 but for rounding)."""
    _, ex = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (ex - 1).clamp_min(-6) - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def _quant64(x):
    """What the 8-bit form of x stands for; scale, reciprocal and scaled value are held in 32 bits
    (bf16 inputs often lie exactly between two e4m3 values once scaled)."""
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], BLOCK):
        g = x[:, c:c + BLOCK]
        a = g.abs().amax(dim=1, keepdim=True).clamp_min(TINY).float()
        out[:, c:c + BLOCK] = _e4m3((g * (TOP / a).double()).float().double()) * (a / TOP).double()
    return out


def _blocks64(q, s):
    out = q.double()
    for r in range(s.shape[0]):
        for c in range(s.shape[1]):
            out[r * BLOCK:(r + 1) * BLOCK, c * BLOCK:(c + 1) * BLOCK] *= s[r, c].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        # Which experts are chosen is decided on scores held in 32 bits; the weights are theirs in 64.
        ids = _route_plain(s)[0].long()
        v = s["logits"].double()
        score = torch.sigmoid(v) if case["score"] == "sigmoid" else torch.softmax(v, dim=1)
        w = torch.take_along_dim(score, ids, dim=1)
        if case["renorm"]:
            w = w / w.sum(dim=1, keepdim=True)
        return {"ids": None, "weights": w * case["scale"]}
    if case["op"] == "linear":
        x = s["x_v"].double()
        if s["xs"] is None:
            x = _quant64(x)
        else:
            for c in range(s["xs"].shape[1]):
                x[:, c * BLOCK:(c + 1) * BLOCK] *= s["xs"][:, c:c + 1].double()
        return {"out": torch.matmul(x, _blocks64(s["w"], s["ws"]).T)}
    x = _quant64(s["x_v"].double())
    e, i, h = s["wgu"].shape[0], case["inter"], case["hidden"]
    nb = _blocks(i)
    out = torch.zeros_like(x)
    for j in range(e):
        rows, col = (s["ids"] == j).nonzero(as_tuple=True)
        if not rows.numel():
            continue
        xe = x[rows]
        g = xe @ _blocks64(s["wgu"][j, :i], s["sgu"][j, :nb]).T
        u = xe @ _blocks64(s["wgu"][j, i:], s["sgu"][j, nb:]).T
        act = _quant64(g * torch.sigmoid(g) * u)
        out.index_add_(0, rows, (act @ _blocks64(s["wd"][j], s["sd"][j]).T) * s["weights"][rows, col, None].double())
    return {"out": out}
