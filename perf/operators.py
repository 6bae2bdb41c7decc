"""Measured cases of the 8-bit floating-point layer and of the model's judged answers.

Three operators, as a quantized model's forward pass and its evaluation meet them:

  quantize   x -> e4m3 codes and one fp32 scale per block of 128 columns (per row, for
             activations) or per 128 x 128 tile (for weights).  The scale is the smallest
             power of two 2^e >= 2^-126 with max|x| <= 448 2^e (1 for a block of zeros), so
             x / 2^e is exact and each code is rounded once, to nearest even.
  matmul     Y = X W^T (+ bias) from such codes: block products scaled by the row's and the
             tile's scale, summed in fp32, rounded once to Y's type.
  logprobs   for every row of logits: the log probability of the given token, the entropy,
             and the top_k tokens (equal logits: lowest token first) with theirs.

``own`` selects the library's calls; otherwise plain torch operations in fp32.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
E4M3 = torch.float8_e4m3fn
BLK = 128


def listed():
    return [
        # one token's activations on their way into a layer: a launch's latency
        dict(name="quantize_token", op="quantize", m=1, k=4096, rows=1, x="bf16"),
        # a prompt's activations into a wide layer
        dict(name="quantize_prompt", op="quantize", m=8192, k=12288, rows=1, x="f16"),
        # weights of odd sizes read once from fp32, in tiles
        dict(name="quantize_weight_odd", op="quantize", m=11001, k=4099, rows=128, x="f32"),
        # one token through an up projection (weights streamed)
        dict(name="matmul_token", op="matmul", m=1, n=11008, k=4096, out="f16", bias=False),
        # a decode batch of odd size through a layer of odd sizes, with its bias
        dict(name="matmul_batch_odd", op="matmul", m=27, n=5003, k=4165, out="bf16", bias=True),
        # a short prompt through an attention projection
        dict(name="matmul_short", op="matmul", m=384, n=4096, k=4096, out="bf16", bias=True),
        # a long prompt through a wide layer
        dict(name="matmul_prompt", op="matmul", m=4096, n=12288, k=4096, out="f16", bias=False),
        # a calibration batch through the vocabulary projection: fp32 logits, odd vocabulary
        dict(name="matmul_vocabulary", op="matmul", m=1000, n=50001, k=1536, out="f32", bias=False),
        # one decoded token with its 20 alternatives
        dict(name="logprobs_token", op="logprobs", n=1, v=128000, top=20, x="bf16"),
        # a decode batch, odd vocabulary in fp32
        dict(name="logprobs_batch_odd", op="logprobs", n=61, v=50001, top=5, x="f32"),
        # an evaluation's text with its best alternative
        dict(name="logprobs_text", op="logprobs", n=4096, v=65536, top=1, x="bf16"),
        # a small model's text, log probabilities and entropy alone
        dict(name="logprobs_plain", op="logprobs", n=8192, v=32000, top=0, x="f16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "logprobs"])
    if op == "quantize":
        k = _log_int(rng, 64, 16384)
        m = _log_int(rng, 1, min(16384, 8192 * 12288 // k))
        return dict(op=op, m=m, k=k, rows=rng.choice([1, 1, 128]), x=rng.choice(sorted(TYPES)))
    if op == "matmul":
        k = _log_int(rng, 128, 12288)
        n = _log_int(rng, 256, 16384)
        m = _log_int(rng, 1, min(4096, 4096 * 12288 * 4096 // (n * k)))
        if rng.random() < 0.5:            # most layers' widths are multiples of 64
            k, n = -(-k // 64) * 64, -(-n // 64) * 64
        return dict(op=op, m=m, n=n, k=k, out=rng.choice(sorted(TYPES)), bias=rng.random() < 0.5)
    v = _log_int(rng, 1000, 160000)
    n = _log_int(rng, 1, min(8192, 4096 * 65536 // v))
    return dict(op=op, n=n, v=v, top=rng.choice([0, 1, 5, 20]), x=rng.choice(sorted(TYPES)))


# ------------------------------------------------------------------ inputs
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000 + salt)
    return g


def _activations(m, k, seed, dtype=torch.float32):
    """Rows with a few loud channels, as the inputs of a model's layers have."""
    g = _gen(seed, 1)
    loud = torch.rand(k, device="cuda", generator=g) < 0.01
    return (torch.randn(m, k, device="cuda", generator=g) * torch.where(loud, 20.0, 1.0)).to(dtype)


def _held(x, rows):
    """(codes, scales) in the layout a program keeps: rows of codes 128 bytes apart."""
    codes, scales = _quantize_plain(x, rows)
    m, k = x.shape
    buf = torch.zeros(m, -(-k // BLK) * BLK, dtype=E4M3, device="cuda")
    buf[:, :k] = codes
    return buf[:, :k], scales


def prepare(case, seed):
    op = case["op"]
    if op == "quantize":
        if case["rows"] == 1:
            x = _activations(case["m"], case["k"], seed, TYPES[case["x"]])
        else:
            x = (torch.randn(case["m"], case["k"], device="cuda", generator=_gen(seed, 2)) * 0.015).to(TYPES[case["x"]])
        return dict(op=op, x=x, rows=case["rows"])
    if op == "matmul":
        xc, xs = _held(_activations(case["m"], case["k"], seed), 1)
        w = torch.randn(case["n"], case["k"], device="cuda", generator=_gen(seed, 3)) * 0.015
        wc, ws = _held(w, 128)
        out = TYPES[case["out"]]
        bias = torch.randn(case["n"], device="cuda", generator=_gen(seed, 4)).to(out) if case["bias"] else None
        return dict(op=op, xc=xc, xs=xs, wc=wc, ws=ws, bias=bias, out=out)
    g = _gen(seed, 5)
    # sharp and flat rows: logits of a trained model have a few tokens far above the rest
    temper = torch.rand(case["n"], 1, device="cuda", generator=g) * 3.0 + 1.0
    logits = (torch.randn(case["n"], case["v"], device="cuda", generator=g) * temper).to(TYPES[case["x"]])
    tokens = torch.randint(0, case["v"], (case["n"],), device="cuda", generator=g)
    return dict(op=op, logits=logits, tokens=tokens, top=case["top"])


# ------------------------------------------------------------------ plain forms
def _spread(scales, rows, m, k):
    """One scale per element of an [m x k] matrix from its block scales."""
    if rows == 1:
        return scales.t().repeat_interleave(BLK, 1)[:, :k]
    return scales.repeat_interleave(BLK, 0)[:m].repeat_interleave(BLK, 1)[:, :k]


def _quantize_plain(x, rows):
    x = x.float()
    m, k = x.shape
    kb, mb = -(-k // BLK), -(-m // rows)
    a = torch.nn.functional.pad(x.abs(), (0, kb * BLK - k, 0, mb * rows - m))
    a = a.reshape(mb, rows, kb, BLK).amax((1, 3))
    f, e = torch.frexp(a)                                  # a = f 2^e, f in [1/2, 1)
    e = torch.where(f > 0.875, e - 8, e - 9).clamp(min=-126)
    s = torch.where(a > 0, ((e + 127) << 23).view(torch.float32), 1.0)
    scales = (s.t() if rows == 1 else s).contiguous()
    return (x / _spread(scales, rows, m, k)).to(E4M3), scales


def _matmul_plain(s):
    m, k = s["xc"].shape
    n = s["wc"].shape[0]
    x = s["xc"].float() * _spread(s["xs"], 1, m, k)
    w = s["wc"].float() * _spread(s["ws"], 128, n, k)
    y = x @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["out"])


def _logprobs_plain(s):
    x = s["logits"].float()
    n, v = x.shape
    top = x.amax(1, keepdim=True)
    below = top - x
    p = torch.exp(-below)
    total = p.sum(1, keepdim=True)
    log_total = torch.log(total)
    given = -below.gather(1, s["tokens"][:, None]) - log_total
    entropy = log_total + (p * below).sum(1, keepdim=True) / total
    # one whole number per token that orders by logit, then by lower index
    bits = (x + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() * (1 << 32) + (v - 1 - torch.arange(v, device=x.device))
    ids = v - 1 - (torch.topk(key, s["top"], 1).values & 0xFFFFFFFF)
    return given[:, 0], entropy[:, 0], ids.to(torch.int32), -below.gather(1, ids) - log_total


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["op"]
    if own:
        import post_weight_quantization_02_amd as G
        if op == "quantize":
            return G.gptq_fp8_quantize(state["x"], state["rows"])
        if op == "matmul":
            return G.gptq_fp8_matmul(state["xc"], state["xs"], state["wc"], state["ws"], state["bias"],
                                     out_dtype=state["out"])
        return G.gptq_token_logprobs(state["logits"], state["tokens"], state["top"])
    if op == "quantize":
        return _quantize_plain(state["x"], state["rows"])
    if op == "matmul":
        return _matmul_plain(state)
    return _logprobs_plain(state)


def work(case):
    if case["op"] == "quantize":
        m, k, r = case["m"], case["k"], case["rows"]
        blocks = -(-m // r) * -(-k // BLK)
        return dict(bytes=m * k * (SIZE[case["x"]] + 1) + 4 * blocks, flops=2 * m * k)
    if case["op"] == "matmul":
        m, n, k, z = case["m"], case["n"], case["k"], SIZE[case["out"]]
        kb = -(-k // BLK)
        held = (m + n) * k + 4 * kb * (m + -(-n // BLK))
        return dict(bytes=held + z * (m * n + (n if case["bias"] else 0)), flops=2 * m * n * k)
    n, v = case["n"], case["v"]
    return dict(bytes=n * v * SIZE[case["x"]] + n * (16 + 8 * case["top"]), flops=5 * n * v)


# ------------------------------------------------------------------ the definitions in 64 bits
def _two64(e):
    """2^e from its bits: exact."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _values64(codes):
    """The numbers that e4m3 bit patterns stand for."""
    b = codes.view(torch.uint8).long()
    e, f = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e > 0, (8 + f) * _two64(e - 10), f * 2.0 ** -9)
    return torch.where(b > 127, -mag, mag)


def _blocks64(codes, scales, rows):
    v = _values64(codes)
    at = torch.arange(v.shape[1], device=v.device) // BLK
    if rows == 1:
        return v * scales.double()[at].t()
    return v * scales.double()[torch.arange(v.shape[0], device=v.device) // BLK][:, at]


def _quantize64(x, rows):
    m, k = x.shape
    mb, kb = -(-m // rows), -(-k // BLK)
    x = x.double()
    scales = torch.ones(mb, kb, dtype=torch.float64, device=x.device)
    out = torch.empty_like(x)
    for j in range(kb):
        part = x[:, j * BLK:(j + 1) * BLK]
        peak = part.abs().amax(1)
        if rows > 1:
            peak = torch.stack([p.max() for p in peak.split(rows)])
        s = _two64(torch.ceil(torch.log2((peak / 448.0).clamp(min=2.0 ** -126))))
        s = torch.where(peak > 448.0 * s, 2 * s, torch.where(peak <= 224.0 * s, s / 2, s))   # what log2 rounds
        s = torch.where(peak > 0, s.clamp(min=2.0 ** -126), 1.0)
        scales[:, j] = s
        u = part / s.repeat_interleave(rows)[:m, None]
        # the spacing of e4m3 values at |u|: the exponent from the bits, none below 2^-9
        step = _two64(((u.abs().clamp(min=2.0 ** -6).view(torch.int64) >> 52) - 1023) - 3)
        out[:, j * BLK:(j + 1) * BLK] = torch.round(u / step) * step
    return out, (scales.t() if rows == 1 else scales).contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "quantize":
        return _quantize64(s["x"], s["rows"])
    if s["op"] == "matmul":
        y = torch.matmul(_blocks64(s["xc"], s["xs"], 1), _blocks64(s["wc"], s["ws"], 128).t().contiguous())
        return y if s["bias"] is None else y + s["bias"].double()
    given, entropy, best = [], [], []
    for x, t in zip(s["logits"].split(512), s["tokens"].split(512)):
        lp = torch.log_softmax(x.double(), 1)
        given.append(lp.gather(1, t[:, None])[:, 0])
        entropy.append(-(lp.exp() * lp).sum(1))
        best.append(torch.topk(lp, s["top"], 1).values)
    return torch.cat(given), torch.cat(entropy), None, torch.cat(best)
