"""GPU parity of the distillation loss and its gradient against the fp64 oracle.

With u = 2^-24: an element's exponent y = (z - m) c is off by at most 4 u |y| (difference,
c itself, product), its power of two by 2 u; a sum of v terms by (v / 256 + 160) u at most
(256 or more threads, each adding its elements one after the other, then 64-wide trees).  So
log S is off by at most
    D = u (v / 256 + 170 + 6 spread),   spread = the mean of |z - m| / T under the terms' weights,
and the loss, whose terms are joined in 64 bits, by 2 D (for S and the rest's S) and its own
rounding.  The gradient of token v is off by |w| / T times
    p_v (Q + q_r / p_r) (D + u (6 |z_v - M| / T + 8)) + 2 u (p_v Q + q_v),
and half a step of its type.
"""
import math

import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import post_weight_quantization_02_amd as G  # noqa: E402

U32 = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = {"f32": 2.0 ** -120, "f16": 2.0 ** -24, "bf16": 2.0 ** -120}


def f64(t):
    return t.detach().double().cpu().numpy()


def make(n, v, top, seed, dtype, noise=0.3, T=1.0):
    """(logits, ids, log probabilities of another model's top tokens at temperature T)."""
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(n, v, generator=g, dtype=torch.float64) * (torch.rand(n, 1, generator=g, dtype=torch.float64) * 3 + 0.5)
    z = (t + noise * torch.randn(n, v, generator=g)).to(TYPES[dtype])
    best = torch.topk(t, top, 1)
    lp = best.values / T - torch.logsumexp(t / T, 1, keepdim=True)
    return z, best.indices.to(torch.int32), lp.float()


def check(z, ids, lp, T, tail, weights, loss, grad, rows=None):
    """Rows of the device's results against the oracle's."""
    name = {t: k for k, t in TYPES.items()}[z.dtype]
    v = z.shape[1]
    for i in (range(z.shape[0]) if rows is None else rows):
        w = 1.0 if weights is None else float(weights[i])
        x = f64(z[i])
        ref, g, spread = O.distill.row(x, ids[i].tolist(), lp[i].tolist(), T, tail, w)
        D = U32 * (v / 256 + 170 + 6 * max(spread))
        got = float(loss[i])
        if math.isfinite(ref):
            assert abs(got - ref) <= 2 * D + 2 * U32 * abs(ref), (i, got, ref, D)
        else:
            assert got == ref or (math.isnan(got) and math.isnan(ref)), (i, got, ref)
        if grad is None:
            continue
        out = f64(grad[i])
        if np.isnan(g).any() or not np.isfinite(x).any():
            np.testing.assert_array_equal(np.isnan(out), np.isnan(g))
            keep = ~np.isnan(g)
            assert np.all(np.abs(out[keep] - g[keep]) <= 1e-2)
            continue
        if w == 0.0 or all(int(t) < 0 for t in ids[i]):
            assert (out == 0.0).all()
            continue
        fine = np.isfinite(x)
        d = np.where(fine, x - np.max(x), -1e4) / T
        p = np.where(fine, np.exp(d), 0.0)
        p = p / p.sum()
        q, rest = O.distill.teacher(ids[i].tolist(), lp[i].tolist(), v, T, tail)
        mass = q.sum() + rest
        others = p[q == 0].sum()
        own = p * mass + np.where(q == 0, p * (rest / others if others > 0 else 0.0), 0.0)
        bound = abs(w) / T * (own * (D + U32 * (6 * np.abs(d) + 8)) + 2 * U32 * (p * mass + q))
        step = torch.finfo(z.dtype).eps / 2
        bound = bound * (1 + step) + np.abs(g) * step + TINY[name]
        assert np.all(np.abs(out - g) <= bound), (i, float(np.max(np.abs(out - g) / bound)))


def both(z, ids, lp, T=1.0, tail=False, weights=None, **kw):
    loss, grad = G.gptq_distill_loss(z.cuda(), ids.cuda(), lp.cuda(), T, tail, None if weights is None else weights.cuda(),
                                     want_grad=True, **kw)
    alone, none = G.gptq_distill_loss(z.cuda(), ids.cuda(), lp.cuda(), T, tail)
    torch.cuda.synchronize()
    assert none is None and grad.shape == z.shape and grad.dtype == z.dtype and loss.dtype == torch.float32
    return loss, grad, alone


CASES = [(1, 2, 1), (3, 5, 4), (2, 7, 7), (5, 8, 3), (4, 9, 2), (300, 17, 5), (2, 100, 64), (3, 1000, 20), (7, 4097, 8), (1, 50001, 20),
         (2, 128000, 64), (600, 1003, 6), (513, 5000, 3), (520, 9001, 17), (130, 20011, 9), (300, 33001, 8), (530, 70001, 5),
         (515, 131072, 4), (514, 140005, 3), (2, 1 << 20, 10)]


@pytest.mark.parametrize("T,tail", [(1.0, True), (1.0, False), (2.0, False), (0.7, True)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,v,top", CASES, ids=[f"{n}x{v}_{t}" for n, v, t in CASES])
def test_parity(n, v, top, dtype, T, tail):
    if tail:
        top = min(top, v - 1)
    if n * v > 10 ** 7:                                  # the oracle looks at some of the rows
        z, ids, lp = make(4, v, top, v + n, dtype, T=T)
        z, ids, lp = (t.repeat(-(-n // 4), 1)[:n].contiguous() for t in (z, ids, lp))
        rows = [0, 1, 2 if n > 2 else 1, n - 1]
    else:
        z, ids, lp = make(n, v, top, v + n, dtype, T=T)
        rows = sorted({0, 1 % n, n // 2, n - 1} | set(range(0, n, max(1, n // 12))))
    weights = torch.rand(n, generator=torch.Generator().manual_seed(n)) * 2 - 0.5
    loss, grad, alone = both(z, ids, lp, T, tail, weights)
    check(z, ids, lp, T, tail, weights, loss, grad, rows)
    check(z, ids, lp, T, tail, None, alone, None, rows)
    if n > 4 and n * v > 10 ** 7:                        # equal rows: equal bits
        assert torch.equal(loss[4:8], loss[:4]) and torch.equal(loss[-n % 4:][:4].sort().values, loss[:4].sort().values) or n % 4


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,v", [(3, 300), (2, 30000), (600, 3001)])
def test_rows_and_entries_that_are_not_there(n, v, dtype):
    z, ids, lp = make(n, v, 6, 1, dtype)
    ids[0] = -1
    lp[0] = float("nan")                                 # of no entry: not looked at
    ids[1, 2], lp[1, 2] = -7, 5.0
    weights = torch.ones(n)
    weights[1] = 0.0
    if n > 2:
        z[0] = float("nan")
        ids[2, 5] = v
        weights[2] = 0.5
    for tail in (False, True):
        loss, grad, alone = both(z, ids, lp, 1.0, tail, weights)
        check(z, ids, lp, 1.0, tail, weights, loss, grad, range(min(n, 5)))
        assert loss[0] == 0 and (grad[0] == 0).all() and (grad[1] == 0).all() and torch.isfinite(loss[1])
        if n > 2:
            assert torch.isnan(loss[2]) and torch.isnan(grad[2]).all()
            assert torch.isnan(alone[2])


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("v", [11, 1000, 40003])
def test_masked_logits(v, tail):
    """-inf, the types' lowest values, everything masked but one, everything, NaN, infinities."""
    for dtype in ("f32", "f16", "bf16"):
        z, ids, lp = make(14, v, 3, 2, dtype)
        low = torch.finfo(TYPES[dtype]).min
        z[0, v // 2:] = -math.inf
        z[1, v // 2:] = low
        z[2] = -math.inf
        z[3] = low
        z[4, 0] = math.nan
        z[5, v - 1] = math.inf
        z[6] = -math.inf
        z[6, 3] = 1.0
        z[7] = z[7] * 0 + low
        z[7, 4] = 0.0
        z[8, ids[8].long()] = -math.inf                  # what the teacher wants is not there
        keep = torch.zeros(v, dtype=torch.bool)
        keep[ids[9].long()] = True
        z[9, ~keep] = -math.inf                          # nothing of the rest is there
        lp[10, 1] = -math.inf
        lp[11, 0] = math.nan
        lp[12, 0] = math.inf
        z[13] = z[13] * 100 if dtype == "f16" else z[13] * 1e6
        loss, grad, alone = both(z, ids, lp, 1.0, tail)
        check(z, ids, lp, 1.0, tail, None, loss, grad)
        check(z, ids, lp, 1.0, tail, None, alone, None)


def test_probabilities_far_apart():
    """A rest or listed tokens of probability e^-300: their logarithms are no underflow."""
    for v in (50, 5000):
        z, ids, lp = make(4, v, 4, 3, "f32")
        for i in range(4):
            z[i, ids[i].long()] += 300.0 if i < 2 else -300.0
        for tail in (False, True):
            loss, grad, _ = both(z, ids, lp, 1.0, tail)
            check(z, ids, lp, 1.0, tail, None, loss, grad)
            # the terms q_j log q_j are at least -1 / e each, and each -log p_j here at least 290
            mass = lp[2:].exp().sum(1) if tail else torch.ones(2)
            assert torch.isfinite(loss).all() and (loss[2:].cpu() > 290 * mass - 2).all()


@pytest.mark.parametrize("T", [1e-4, 1e4])
def test_extreme_temperatures(T):
    z, ids, lp = make(5, 3000, 5, 4, "f32", T=T)
    for tail in (False, True):
        loss, grad, _ = both(z, ids, lp, T, tail)
        for i in range(5):
            ref, g, spread = O.distill.row(f64(z[i]), ids[i].tolist(), lp[i].tolist(), T, tail)
            assert abs(float(loss[i]) - ref) <= 2 * U32 * (3000 / 256 + 170 + 6 * max(spread)) + 2 * U32 * abs(ref)
            assert torch.isfinite(grad[i]).all()


@pytest.mark.parametrize("v", [10, 20000])
def test_tokens_listed_twice(v):
    z, ids, lp = make(6, v, 5, 5, "f32")
    ids[:, 3] = ids[:, 0]
    ids[1] = ids[1, 0]
    ids[2, 1:4] = ids[2, 4]
    for tail in (False, True):
        loss, grad, _ = both(z, ids, lp, 1.0, tail)
        check(z, ids, lp, 1.0, tail, None, loss, grad)


def test_neighbours_in_one_vector():
    """Every listed token next to the others, at both ends and behind the last whole vector."""
    for v in (16, 30, 1003, 70003):
        for dtype in ("f32", "bf16"):
            z, _, _ = make(5, v, 1, 6, dtype)
            ids = torch.stack([torch.arange(9), torch.arange(9).flip(0), v - 1 - torch.arange(9), (v - 9 + torch.arange(9)) // 2,
                               torch.arange(9) * ((v - 1) // 8)]).to(torch.int32)
            lp = torch.log_softmax(torch.randn(5, 9, generator=torch.Generator().manual_seed(v)), 1) - 0.2
            for tail in (False, True):
                loss, grad, alone = both(z, ids, lp, 1.0, tail)
                check(z, ids, lp, 1.0, tail, None, loss, grad)


@pytest.mark.parametrize("n,v", [(3, 70), (4, 9003), (600, 2001), (520, 40001)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_strides_and_given_outputs(n, v, dtype):
    """Rows at odd addresses inside wider tensors: the same bits, and nothing else written."""
    z, ids, lp = (t.cuda() for t in make(min(n, 4), v, 5, 7, dtype))
    z, ids, lp = (t.repeat(-(-n // t.shape[0]), 1)[:n].contiguous() for t in (z, ids, lp))
    w = torch.rand(n, device="cuda")
    ref, gref = G.gptq_distill_loss(z, ids, lp, 1.0, True, w, want_grad=True)
    wide = torch.full((n, v + 8), math.nan, dtype=TYPES[dtype], device="cuda")
    wide[:, 3:3 + v] = z
    out = torch.full((n, v + 6), 7.0, dtype=TYPES[dtype], device="cuda")
    loss = torch.full((n + 2,), 7.0, device="cuda")
    a, b = G.gptq_distill_loss(wide[:, 3:3 + v], ids, lp, 1.0, True, w, loss=loss[1:1 + n], grad=out[:, 1:1 + v])
    torch.cuda.synchronize()
    assert torch.equal(a, ref) and torch.equal(b, gref)
    assert loss[0] == 7.0 and loss[-1] == 7.0 and (out[:, 0] == 7.0).all() and (out[:, 1 + v:] == 7.0).all()


def test_gradient_against_differences():
    z, ids, lp = make(3, 40, 6, 8, "f32")
    for T, tail in ((1.0, True), (1.7, False)):
        w = torch.tensor([1.0, -2.0, 0.5])
        _, grad, _ = both(z, ids, lp, T, tail, w)
        h = 2.0 ** -6                                    # exact in every logit's steps
        for j in range(40):
            up, down = z.clone(), z.clone()
            up[:, j] += h
            down[:, j] -= h
            a, b = (G.gptq_distill_loss(t.cuda(), ids.cuda(), lp.cuda(), T, tail)[0].double().cpu() for t in (up, down))
            # losses of order 1 are off by 2 D < 4e-5, the difference's own error is h^2 / 6
            assert torch.allclose((a - b) / (2 * h) * w.double(), grad[:, j].double().cpu(), rtol=1e-3, atol=2 * (4e-5 / h + h * h))


def test_it_is_the_divergence_of_the_top_tokens_of_another_model():
    """From the other model's own top tokens; at most the divergence over all tokens, and 0 of a
    model from itself within the roundings."""
    g = torch.Generator(device="cuda").manual_seed(9)
    t = torch.randn(50, 3001, device="cuda", generator=g) * 2
    z = t + 0.5 * torch.randn(50, 3001, device="cuda", generator=g)
    none = torch.full((50,), -1, dtype=torch.int64, device="cuda")
    _, _, ids, lp = G.gptq_token_logprobs(t, none, 40)
    loss, _ = G.gptq_distill_loss(z, ids, lp, tail=True)
    p, q = torch.log_softmax(z.double(), 1), torch.log_softmax(t.double(), 1)
    assert (loss > 0).all() and (loss.double() <= (q.exp() * (q - p)).sum(1) + 1e-5).all()
    same, grad = G.gptq_distill_loss(t, ids, lp, tail=True, want_grad=True)
    assert same.abs().max() < 2e-5 and grad.abs().max() < 2e-5


def test_more_than_2_to_31_elements():
    n, v = 40000, 65536
    z = torch.zeros(n, v, dtype=torch.bfloat16, device="cuda")
    a, ids, lp = make(3, v, 5, 10, "bf16")
    z[-3:] = a.cuda()
    full = torch.full((n, 5), -1, dtype=torch.int32, device="cuda")
    full[-3:] = ids.cuda()
    t = torch.zeros(n, 5, device="cuda")
    t[-3:] = lp.cuda()
    loss, grad = G.gptq_distill_loss(z, full, t, 1.0, True, want_grad=True)
    check(a, ids, lp, 1.0, True, None, loss[-3:].cpu(), grad[-3:].cpu())
    assert (loss[:-3] == 0).all() and (grad[:-3].view(torch.int16) == 0).all()


def test_refusals():
    z, ids, lp = (t.cuda() for t in make(4, 50, 3, 11, "f32"))
    w = torch.ones(4, device="cuda")
    for kw, error in ((dict(ids=ids.long()), TypeError), (dict(ids=ids[:3]), ValueError), (dict(logprobs=lp.double()), TypeError),
                      (dict(logprobs=lp[:, :2]), ValueError), (dict(ids=ids[:, 0]), ValueError), (dict(weights=w.half()), TypeError),
                      (dict(weights=w[:3]), ValueError), (dict(temperature=0.0), G.GPTQError), (dict(temperature=math.nan), G.GPTQError),
                      (dict(logits=z.double()), TypeError), (dict(logits=z.t()), ValueError), (dict(ids=ids.cpu()), ValueError),
                      (dict(grad=z.half()), TypeError), (dict(grad=z[:, :40]), ValueError), (dict(loss=w[:3]), ValueError),
                      (dict(ids=torch.zeros(4, 6, dtype=torch.int32, device="cuda")[:, ::2]), ValueError),
                      (dict(ids=ids[:, :0].contiguous(), logprobs=lp[:, :0].contiguous()), G.GPTQError),
                      (dict(logits=z.clone().requires_grad_(True)), ValueError)):
        with pytest.raises(error):
            G.gptq_distill_loss(**dict(dict(logits=z, ids=ids, logprobs=lp), **kw))
    for kw in (dict(grad=z), dict(loss=lp.view(-1)[:4]), dict(loss=w, weights=w), dict(ws=z)):
        with pytest.raises(ValueError, match="overlaps"):
            G.gptq_distill_loss(z, ids, lp, **kw)
    assert G.gptq_distill_loss(z[:0], ids[:0], lp[:0])[0].shape == (0,)


def test_two_streams_and_given_workspaces():
    cases = [tuple(t.cuda() for t in make(n, 20000, 6, n, "bf16")) for n in (2, 3)]
    ref = [G.gptq_distill_loss(*c, want_grad=True) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [G.gptq_distill_loss(*cases[i % 2], want_grad=True, stream=streams[i % 2]) for i in range(20)]
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(got):
        assert torch.equal(a, ref[i % 2][0]) and torch.equal(b, ref[i % 2][1])
    need = G.gptq_distill_loss_workspace_size(2, 20000)
    assert need > 0
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    a, b = G.gptq_distill_loss(*cases[0], want_grad=True, ws=ws[:need])
    torch.cuda.synchronize()
    assert torch.equal(a, ref[0][0]) and torch.equal(b, ref[0][1]) and (ws[need:] == 0x5A).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [256, 257])
@pytest.mark.parametrize("vectors", [300, 2047, 2048, 2049, 4096, 4097, 8192, 8193, 9216, 9217, 13311, 13312, 13313, 16384, 16385])
def test_gradients_where_the_work_groups_change(n, vectors, dtype):
    """Row lengths and numbers around which other work-groups take a row: three rows against the
    oracle, and every copy of them bit by bit."""
    v = vectors * (4 if dtype == "f32" else 8) + 3
    z, ids, lp = (t.cuda() for t in make(3, v, 17, vectors, dtype))
    of = torch.arange(n, device="cuda") % 3
    ids[1, 0] = v - 1                                    # behind the vectors
    ids[2, 1] = v - 5                                    # in the last one
    loss, grad = G.gptq_distill_loss(z[of], ids[of], lp[of], 1.0, True, want_grad=True)
    torch.cuda.synchronize()
    check(z, ids, lp, 1.0, True, None, loss[:3], grad[:3])
    assert torch.equal(loss, loss[of]) and torch.equal(grad, grad[of])


@pytest.mark.parametrize("at", [0, 8, 77, 1001])
def test_workspace_at_any_address(at):
    case = tuple(t.cuda() for t in make(3, 20000, 6, 9, "f32"))
    need = G.gptq_distill_loss_workspace_size(3, 20000)
    assert need > 0
    ws = torch.full((at + need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    got = G.gptq_distill_loss(*case, 1.0, True, want_grad=True, ws=ws[at:at + need])
    ref = G.gptq_distill_loss(*case, 1.0, True, want_grad=True)
    torch.cuda.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert (ws[at + need:] == 0x5A).all() and (ws[:at] == 0x5A).all()


@pytest.mark.parametrize("n,v", [(2, 30000), (5, 600), (600, 9000)])
def test_graph_replays_match_eager(n, v):
    z, ids, lp = (t.cuda() for t in make(n, v, 6, 12, "bf16"))
    G.gptq_distill_loss(z, ids, lp, 1.0, True, want_grad=True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss, grad = G.gptq_distill_loss(z, ids, lp, 1.0, True, want_grad=True)
    for r in range(3):
        z.copy_(torch.randn(n, v, device="cuda"))
        ids.copy_(torch.randint(0, v, (n, 6), device="cuda"))
        a, b = G.gptq_distill_loss(z, ids, lp, 1.0, True, want_grad=True)
        loss.fill_(0)
        grad.fill_(0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, a) and torch.equal(grad, b), r
    del g
