"""What is measured of the expert-sorting and MXFP4 operators.

Three operators, used one after the other by a MoE layer whose experts run in
4 bits on both sides:

  * sorting tokens by expert and back ("permute", "permute_backward",
    "unpermute", "unpermute_backward"): rows copied into the aligned expert
    order, the weighted sum back to tokens, and the gradient of each;
  * MXFP4 quantisation ("quantize"): blocks of 32 values share one power-of-two
    scale (E8M0), each value is held in 4 bits (E2M1), and the values that the
    4 bits stand for are returned;
  * the experts' product ("experts"): BF16 token rows are quantised to MXFP4
    in expert order and multiplied by MXFP4 weights, FP32 accumulation, with
    an optional SiLU(gate) * up.

With `own` false, run() computes them with elementary torch operations in 32
bits; with `own` true, it makes the library's calls.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
SORTING = ("permute", "permute_backward", "unpermute", "unpermute_backward")
BLOCK = 32                                              # values that share a scale
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)       # E2M1 magnitudes by code


def _sorting(name, op, tokens, hidden, experts, local, topk, dtype, block):
    return dict(name=name, op=op, tokens=tokens, hidden=hidden, experts=experts, local=local, topk=topk,
                dtype=dtype, block=block)


def _experts(name, tokens, K, N, experts, local, topk, block, silu, zipf=0.0):
    return dict(name=name, op="experts", tokens=tokens, K=K, N=N, experts=experts, local=local, topk=topk,
                block=block, silu=silu, zipf=zipf)


def listed():
    return [
        # one step of decoding on one of 8 expert-parallel ranks: latency of a few dozen rows
        _sorting("permute decode", "permute", 64, 7168, 384, 48, 8, "bf16", 16),
        # the same rank's share of an 8192-token prompt chunk: bandwidth
        _sorting("permute prefill", "permute", 8192, 7168, 384, 48, 8, "bf16", 128),
        # a training step on all experts of one GPU, a row length that no vector divides
        _sorting("permute gradient odd rows", "permute_backward", 1021, 2051, 8, 8, 2, "fp16", 16),
        # decoding with every expert on the GPU, outputs kept in FP32
        _sorting("unpermute decode fp32", "unpermute", 128, 7168, 384, 384, 8, "fp32", 8),
        # the weighted sum's gradient for a training batch of one expert-parallel rank
        _sorting("unpermute gradient", "unpermute_backward", 8192, 7168, 384, 48, 8, "bf16", 16),
        # one decoded token's activations
        dict(name="quantize one token", op="quantize", rows=1, K=7168, dtype="bf16"),
        # a prompt chunk's activations
        dict(name="quantize prefill", op="quantize", rows=8192, K=7168, dtype="bf16"),
        # one token, its 8 experts' gate/up product on one of 8 tensor-parallel ranks: latency
        _experts("experts one token", 1, 7168, 512, 384, 384, 8, 8, True),
        # a decoding batch on one expert-parallel rank: every local expert's weights are streamed once
        _experts("experts decode gate/up", 64, 7168, 4096, 384, 48, 8, 16, True),
        # the down product of a tensor-parallel rank, short K, skewed expert popularity
        _experts("experts decode down skewed", 128, 256, 7168, 384, 384, 8, 8, False, 1.1),
        # a prompt chunk on one expert-parallel rank: about 170 rows for each expert
        _experts("experts prefill gate/up", 8192, 7168, 4096, 384, 48, 8, 128, True),
        # few experts and thousands of rows for each: bound by the tensor cores
        _experts("experts many rows", 8192, 7168, 4096, 8, 8, 2, 128, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(SORTING + ("quantize", "quantize", "experts", "experts", "experts", "experts"))
    experts, local, topk = rng.choice(((384, 48, 8), (384, 384, 8), (8, 8, 2), (64, 16, 6), (16, 16, 1)))
    block = rng.choice((8, 16, 32, 64, 128))
    if op in SORTING:
        tokens, hidden = _log(rng, 1, 8192), _log(rng, 64, 7168)
        if rng.random() < 0.7:
            hidden = max(8, hidden // 8 * 8)
        while tokens * min(topk, topk * local / experts) * hidden > 60e6:
            tokens = tokens * 3 // 4
        return dict(op=op, tokens=max(1, tokens), hidden=hidden, experts=experts, local=local, topk=topk,
                    dtype=rng.choice(("bf16", "bf16", "fp16", "fp32")), block=block)
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 8192), K=32 * _log(rng, 1, 224),
                    dtype=rng.choice(("bf16", "bf16", "fp16", "fp32")))
    tokens, K, N = _log(rng, 1, 8192), 32 * _log(rng, 4, 224), 32 * _log(rng, 4, 224)
    while local * K * N > 48 * 4096 * 7168:
        N = max(32, N // 2 // 32 * 32)
    rows = tokens * topk * local / experts
    if rows * K * N > 16384 * 4096 * 7168:
        tokens = max(1, int(tokens * 16384 * 4096 * 7168 / (rows * K * N)))
    silu = rng.random() < 0.5
    return dict(op="experts", tokens=tokens, K=K, N=max(64, N // 64 * 64) if silu else N, experts=experts,
                local=local, topk=topk, block=block, silu=silu, zipf=rng.choice((0.0, 1.1)))


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _routing(case, g):
    """topk_ids [M, k] (distinct) and their normalised weights."""
    M, E, k = case["tokens"], case["experts"], case["topk"]
    logits = _normal(g, M, E)
    if case.get("zipf"):
        rank = torch.randperm(E, generator=g, device="cuda").float() + 1
        u = torch.rand((M, E), generator=g, device="cuda").clamp(1e-7, 1 - 1e-6)
        logits = -case["zipf"] * rank.log() - (-u.log()).log()
    score, ids = logits.topk(k, dim=1)
    score = torch.sigmoid(score)
    return ids.int().contiguous(), (score / score.sum(1, keepdim=True)).contiguous()


def _capacity(case):
    n, bm = case["tokens"] * case["topk"], case["block"]
    return -(-(n + min(n, case["local"]) * (bm - 1)) // bm) * bm


def _align(case, ids):
    """The aligned expert order: each local expert's assignments in ascending
    order, padded to a multiple of the block; the first `local` experts are local."""
    n, E, bm, cap = ids.numel(), case["local"], case["block"], _capacity(case)
    e = ids.reshape(-1).long()
    counts = torch.bincount(e, minlength=case["experts"])[:E]
    ends = (((counts + bm - 1) // bm) * bm).cumsum(0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    starts = counts.cumsum(0) - counts
    order = torch.argsort(e, stable=True)
    se = e[order]
    is_local = se < E
    sl = se.clamp(max=E - 1)
    row = torch.where(is_local, torch.arange(n, device="cuda") - starts[sl] + offsets[sl], -1)
    positions = torch.empty(n, dtype=torch.long, device="cuda")
    positions[order] = row
    table = torch.full((cap + 1,), n, dtype=torch.long, device="cuda")
    table[torch.where(is_local, row, cap)] = order
    return dict(positions=positions.int(), sorted=table[:cap].int().contiguous(), counts=counts.int(),
                offsets=offsets.int(), ntpp=ends[-1:].int().contiguous())


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = dict(case=case)
    if own:
        from w4a16_int4_weight_sigmoid_gb300 import chord
        s["chord"] = chord
    if op == "quantize":
        # activations: most of unit size, some channels ten times larger
        ch = 1 + 9 * (torch.rand(case["K"], generator=g, device="cuda") < 0.02)
        s["x"] = (_normal(g, case["rows"], case["K"]) * ch).to(TYPES[case["dtype"]])
        if own:
            s["codes"] = torch.empty((case["rows"], case["K"] // 2), dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty((case["rows"], case["K"] // BLOCK), dtype=torch.uint8, device="cuda")
            s["values"] = torch.empty_like(s["x"])
        return s
    ids, s["weights"] = _routing(case, g)
    s.update(_align(case, ids))
    M, cap, k = case["tokens"], _capacity(case), case["topk"]
    if op in SORTING:
        H, dtype = case["hidden"], TYPES[case["dtype"]]
        if op in ("permute", "unpermute_backward"):
            s["x"] = _normal(g, M, H).to(dtype)             # token rows (or their gradient)
        if op != "permute":
            s["y"] = _normal(g, cap, H).to(dtype)           # expert rows (or their gradient)
        if own:
            # rows past the padded total are never written
            s["rows"] = torch.zeros((cap, H), dtype=dtype, device="cuda")
            s["tokens"] = torch.empty((M, H), dtype=dtype, device="cuda")
            s["dweights"] = torch.empty((M, k), device="cuda")
        return s
    E, N, K = case["local"], case["N"], case["K"]
    s["x"] = _normal(g, M, K).to(torch.bfloat16)
    s["w_codes"] = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, generator=g, device="cuda")
    s["w_scales"] = torch.randint(117, 122, (E, N, K // BLOCK), dtype=torch.uint8, generator=g, device="cuda")
    if own:
        c = s["chord"]
        s["packed"] = torch.empty(c.chord_mxfp4_prepack_bytes(E, N, K), dtype=torch.uint8, device="cuda")
        c.chord_mxfp4_prepack(s["w_codes"], s["w_scales"], case["silu"], s["packed"])
        s["rows"] = torch.empty(c.chord_mxfp4_rows_bytes(cap, K), dtype=torch.uint8, device="cuda")
        s["ws"] = torch.zeros(c.chord_mxfp4_moe_gemm_workspace_bytes(), dtype=torch.uint8, device="cuda")
        # padding rows are never written
        s["C"] = torch.zeros((cap, N // 2 if case["silu"] else N), dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------- plain forms
def _quantized(x):
    """The values that MXFP4 holds for x [rows, K] (FP32): x / scale rounded to
    the nearest E2M1 value, ties to the even code, at most 6."""
    b = x.reshape(x.shape[0], -1, BLOCK)
    top = b.abs().amax(-1, keepdim=True)
    exponent = torch.frexp(top).exponent - 3            # floor(log2(top)) - 2
    exponent = torch.where(top > 0, exponent, -127).clamp(min=-127)
    a = torch.ldexp(b.abs(), -exponent)
    q = (0.5 * (a > 0.25) + 0.5 * (a >= 0.75) + 0.5 * (a > 1.25) + 0.5 * (a >= 1.75)
         + 1.0 * (a > 2.5) + 1.0 * (a >= 3.5) + 2.0 * (a > 5.0))
    return (torch.ldexp(q, exponent) * b.sign()).reshape(x.shape)


def _weights(codes, scales):
    """FP32 weights [..., N, K] of packed codes (low nibble = even k) and scales."""
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    pair = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1)
    w = pair.reshape(*scales.shape, BLOCK)
    return torch.ldexp(w, scales.int().unsqueeze(-1) - 127).reshape(*codes.shape[:-1], -1)


def _plain_experts(s):
    case = s["case"]
    E, k, cap, n = case["local"], case["topk"], _capacity(case), s["positions"].numel()
    x = _quantized(s["x"].float())
    touched = torch.nonzero(s["counts"]).reshape(-1)
    C = torch.zeros((cap, case["N"] // 2 if case["silu"] else case["N"]), dtype=torch.bfloat16, device="cuda")
    if touched.numel() == 0:
        return C
    w = _weights(s["w_codes"][touched], s["w_scales"][touched])
    most = int(s["counts"].max())
    slot = torch.arange(most, device="cuda")
    row = s["offsets"][touched].long()[:, None] + slot                      # [experts, most]
    used = slot < s["counts"][touched][:, None]
    f = s["sorted"].long()[row.clamp(max=cap - 1)].clamp(max=n - 1)
    y = torch.bmm(x[f // k], w.transpose(1, 2))
    if case["silu"]:
        gate, up = y.chunk(2, -1)
        y = gate / (1 + torch.exp(-gate)) * up
    C[row[used]] = y[used].to(torch.bfloat16)
    return C


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "quantize":
        return _quantized(s["x"].float()).to(s["x"].dtype)
    if op == "experts":
        return _plain_experts(s)
    k, n = case["topk"], s["positions"].numel()
    dtype = TYPES[case["dtype"]]
    f = s["sorted"].long()
    filled = (f < n)[:, None]
    f = f.clamp(max=n - 1)
    if op == "permute":
        return torch.where(filled, s["x"].float()[f // k], 0.0).to(dtype)
    at = s["positions"].long().reshape(-1, k)
    here = at >= 0
    y = s["y"].float()[at.clamp(min=0)] * here[..., None]                   # [M, k, H]
    if op == "permute_backward":
        return y.sum(1).to(dtype)
    if op == "unpermute":
        return (y * s["weights"][..., None]).sum(1).to(dtype)
    x = s["x"].float()
    dy = torch.where(filled, x[f // k] * s["weights"].reshape(-1)[f][:, None], 0.0).to(dtype)
    return dy, (y * x[:, None]).sum(-1)


# ------------------------------------------------------------- the library
def _library(s):
    case, op, c = s["case"], s["case"]["op"], s["chord"]
    if op == "quantize":
        c.chord_mxfp4_quantize(s["x"], s["codes"], s["scales"])
        c.chord_mxfp4_dequantize(s["codes"], s["scales"], s["values"])
        return s["values"]
    if op == "experts":
        c.chord_mxfp4_quantize_rows(s["x"], s["positions"], case["topk"], s["ntpp"], _capacity(case), s["rows"])
        c.chord_mxfp4_moe_gemm(s["rows"], s["packed"], case["local"], case["N"], case["K"], s["counts"],
                               s["offsets"], _capacity(case),
                               c.CHORD_EPI_SILU_MUL if case["silu"] else c.CHORD_EPI_STORE, s["C"], s["ws"])
        return s["C"]
    if op == "permute":
        c.chord_moe_permute(s["x"], s["positions"], s["sorted"], s["ntpp"], case["topk"], s["rows"])
        return s["rows"]
    if op == "permute_backward":
        c.chord_moe_permute_backward(s["y"], s["positions"], case["topk"], s["tokens"])
        return s["tokens"]
    if op == "unpermute":
        c.chord_moe_unpermute(s["y"], s["weights"], s["positions"], s["tokens"])
        return s["tokens"]
    c.chord_moe_unpermute_backward(s["x"], s["y"], s["weights"], s["positions"], s["sorted"], s["ntpp"],
                                   s["rows"], s["dweights"])
    return s["rows"], s["dweights"]


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------- work
def _expected(case):
    """Expected local assignments, tokens with one, and experts touched."""
    M, k, E, L = case["tokens"], case["topk"], case["experts"], case["local"]
    rows = M * k * L / E
    tokens = M * (1 - (1 - L / E) ** k)
    if case.get("zipf"):
        p = [(r + 1) ** -case["zipf"] for r in range(E)]
        total = sum(p)
        touched = sum(1 - (1 - v / total) ** (M * k) for v in p) * L / E
    else:
        touched = L * (1 - (1 - k / E) ** M)
    return rows, tokens, max(touched, min(1.0, rows))


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["K"]
        # read, codes and scales written and read back, values written
        return {"bytes": n * (2 * SIZE[case["dtype"]] + 2 * (0.5 + 1 / BLOCK)), "flops": 4 * n}
    rows, tokens, touched = _expected(case)
    index = 4 * case["tokens"] * case["topk"]
    if op == "experts":
        N, K = case["N"], case["K"]
        out = N // 2 if case["silu"] else N
        return {"bytes": touched * N * K * (0.5 + 1 / BLOCK) + tokens * K * 2 + 2 * rows * K * (0.5 + 1 / BLOCK)
                + rows * out * 2 + index, "flops": 2 * rows * N * K}
    row = case["hidden"] * SIZE[case["dtype"]]
    moved = {"permute": (tokens + rows) * row + index, "permute_backward": (rows + case["tokens"]) * row + index,
             "unpermute": (rows + case["tokens"]) * row + 2 * index,
             "unpermute_backward": (tokens + 2 * rows) * row + 3 * index}[op]
    return {"bytes": moved, "flops": rows * case["hidden"] * {"unpermute": 2, "unpermute_backward": 3}.get(op, 1)}


# ------------------------------------------------------------------- exact
def _exact_quantized(x):
    """E2M1 rounding in 64 bits by the nearest of the eight magnitudes."""
    v = x.double().reshape(-1, BLOCK)
    top = v.abs().max(1, keepdim=True).values
    scale = torch.where(top > 0, 2.0 ** (torch.floor(torch.log2(top.clamp(min=2.0 ** -149))) - 2), 1.0)
    scale = torch.where(top >= scale * 8, scale * 2, torch.where((top > 0) & (top < scale * 4), scale / 2, scale))
    scale = scale.clamp(min=2.0 ** -127)
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    middle = (levels[1:] + levels[:-1]) / 2
    a = v.abs() / scale
    code = torch.bucketize(a, middle)                   # a tie goes to the lower code here
    tie = (code < 7) & (a == middle[code.clamp(max=6)])
    code = code + (tie & (code % 2 == 1))
    return (torch.sign(v) * levels[code] * scale).reshape(x.shape)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "quantize":
        return _exact_quantized(s["x"])
    cap, k = _capacity(case), case["topk"]
    counts, offsets, table = s["counts"].tolist(), s["offsets"].tolist(), s["sorted"].long()
    if op == "experts":
        x = _exact_quantized(s["x"])
        out = torch.zeros((cap, case["N"] // 2 if case["silu"] else case["N"]), dtype=torch.float64, device="cuda")
        signed = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float64, device="cuda")
        for e, rows in enumerate(counts):
            if not rows:
                continue
            at = slice(offsets[e], offsets[e] + rows)
            c = s["w_codes"][e].long()
            w = torch.empty((case["N"], case["K"]), dtype=torch.float64, device="cuda")
            w[:, 0::2], w[:, 1::2] = signed[c % 16], signed[c // 16]
            w *= (2.0 ** (s["w_scales"][e].double() - 127)).repeat_interleave(BLOCK, 1)
            y = x[table[at] // k] @ w.T
            if case["silu"]:
                half = case["N"] // 2
                y = y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]
            out[at] = y
        return out
    M, H = case["tokens"], case["hidden"]
    filled = torch.nonzero(table < M * k).reshape(-1)   # rows that hold an assignment
    f = table[filled]
    if op == "permute":
        out = torch.zeros((cap, H), dtype=torch.float64, device="cuda")
        out[filled] = s["x"].double()[f // k]
        return out
    y, w = s["y"].double(), s["weights"].double().reshape(-1)
    if op == "unpermute_backward":
        g = s["x"].double()[f // k]
        dy = torch.zeros((cap, H), dtype=torch.float64, device="cuda")
        dy[filled] = g * w[f][:, None]
        dw = torch.zeros(M * k, dtype=torch.float64, device="cuda")
        dw[f] = (g * y[filled]).sum(1)
        return dy, dw.reshape(M, k)
    rows = y[filled] * (w[f][:, None] if op == "unpermute" else 1.0)
    return torch.zeros((M, H), dtype=torch.float64, device="cuda").index_add_(0, f // k, rows)
