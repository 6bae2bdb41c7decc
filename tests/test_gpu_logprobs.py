"""GPU parity of token log probabilities, entropy and top tokens against the fp64
oracle.

Ids exact.  Sums: with d = x - M, each term e^d carries |d| u (the subtraction), two
roundings of the exponent's product (2 |d| u) and the exponential's last place (2 u);
a lane adds at most v / 64 of them one after another, then a tree (64 u allowed).  So
S is off by eS = u (v / 64 + 64 + 3 E|d|) relative, E|d| = -T / S; then log p by
eS + 2 u (|d| + log S + 1), the entropy by (eS + 8 u) (1 + E|d| + log S).
"""
import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import post_weight_quantization_02_amd as G  # noqa: E402

U32 = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def check(logits, tokens, top_k, got, where=None):
    x = logits.detach().double().cpu().numpy()
    lp, ent, ids, tops = O.fp8.token_logprobs(x, tokens.cpu().numpy(), top_k)
    g_lp, g_ent, g_ids, g_tops = (t.cpu().numpy() for t in got)
    np.testing.assert_array_equal(g_ids, ids)
    v = x.shape[1]
    M = np.max(x, 1)
    with np.errstate(all="ignore"):
        d = x - M[:, None]
        p = np.where(np.isfinite(d), np.exp(d), 0.0)
        S = p.sum(1)
        Ed = np.where(p > 0, -p * d, 0.0).sum(1) / S
        eS = U32 * (v / 64 + 64 + 3 * Ed)
        logS = np.log(S)

    def near(got, ref, tol):
        same = (got == ref) | (np.isnan(got) & np.isnan(ref))
        with np.errstate(all="ignore"):
            ok = same | (np.abs(got - ref) <= tol)
        assert np.all(ok), (where, np.argwhere(~ok)[:4], got[~ok][:4], ref[~ok][:4])

    with np.errstate(all="ignore"):
        near(g_lp, lp, eS + 2 * U32 * (np.abs(lp) + 2 * logS + 1))
        near(g_ent, ent, (eS + 8 * U32) * (1 + Ed + logS))
        near(g_tops, tops, (eS + 2 * U32 * (2 * logS + 1))[:, None] + 2 * U32 * np.abs(tops))


def make(n, v, seed, dtype, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, v, generator=g) * (torch.rand(n, 1, generator=g) * 4 + 0.5)
    if kind == "shifted":
        x = x + 500.0
    elif kind == "equal":
        x = torch.full((n, v), 1.5)
    elif kind == "coarse":                  # many equal logits, zeros of both signs
        x = torch.round(x)
    elif kind == "ascending":
        x = torch.arange(v).float().expand(n, v) * 1e-2
    elif kind == "masked":
        x[torch.rand(n, v, generator=g) < 0.9] = -float("inf")
    elif kind == "sharp":
        x[torch.arange(n), torch.randint(0, v, (n,), generator=g)] = 60.0
    elif kind == "ends":                    # the best ones at the row's two ends
        x[:, 0], x[:, -1], x[:, v // 2] = 30.0, 30.0, 29.0
    elif kind == "all_lowest":
        x = torch.full((n, v), torch.finfo(TYPES[dtype]).min)
        x[0, v // 3] = 1.0
    elif kind == "all_largest":
        x = torch.full((n, v), torch.finfo(TYPES[dtype]).max)
        x[:, ::2] = 5.0
    elif kind == "lowest":                  # masked with the type's lowest value
        x[torch.rand(n, v, generator=g) < 0.5] = torch.finfo(TYPES[dtype]).min
    tok = torch.randint(0, v, (n,), generator=g)
    return x.to(TYPES[dtype]), tok


CASES = [(1, 1, 1, "normal"), (3, 2, 2, "normal"), (2, 7, 0, "normal"), (5, 63, 20, "normal"), (4, 64, 64, "coarse"),
         (2, 100, 64, "masked"), (3, 513, 5, "sharp"), (2, 2049, 20, "ends"), (1, 4097, 1, "coarse"), (3, 5000, 20, "equal"),
         (2, 9001, 33, "ascending"), (1, 20011, 20, "masked"), (2, 30000, 64, "shifted"), (1100, 300, 5, "normal"),
         (1030, 2500, 20, "coarse"), (7, 12345, 0, "lowest"), (2, 6000, 7, "lowest"), (4, 5001, 3, "all_lowest"), (3, 3000, 2, "all_largest"),
         (9, 260, 1, "masked"), (1500, 77, 77 - 20, "coarse"), (3, 70000, 64, "ascending"), (4, 8200, 64, "equal"), (1, 131072, 20, "normal"), (2, 140001, 64, "coarse"), (1, 270000, 32, "masked"),
         (3, 40001, 20, "ends"), (2, 33000, 7, "lowest"), (3, 50001, 9, "all_lowest"), (2, 30001, 5, "all_largest"),
         (2, 40000, 20, "equal"), (4, 60001, 3, "sharp"), (130, 16003, 20, "coarse"), (257, 30000, 5, "masked"),
         (2, 90000, 20, "ascending"), (1, 25000, 64, "normal")]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,v,top,kind", CASES, ids=[f"{c[0]}x{c[1]}_k{c[2]}_{c[3]}" for c in CASES])
def test_parity(n, v, top, kind, dtype):
    x, tok = make(n, v, n * 31 + v, dtype, kind)
    if n > 2:
        tok[1] = -1
        tok[2] = v + 3
    got = G.gptq_token_logprobs(x.cuda(), tok.cuda(), top)
    torch.cuda.synchronize()
    check(x, tok, top, got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("v", [40, 3001, 40003])
def test_rows_without_a_softmax(v, dtype):
    x, tok = make(8, v, 3, dtype)
    inf = float("inf")
    x[0] = -inf                              # nothing left by the mask
    x[1, v // 2] = inf
    x[2, v - 1] = float("nan")
    x[3] = inf
    x[4] = -inf
    x[4, v - 2] = 3.0                        # one token left
    x[5] = -inf
    tok[4] = v - 2
    tok[5] = -1                              # a masked row without a token
    got = G.gptq_token_logprobs(x.cuda(), tok.cuda(), 20)
    torch.cuda.synchronize()
    check(x, tok, 20, got)
    # one token left: S is its own 2^y, |y| <= half a step of M log2 e < 2^-20, off by 2 u;
    # log2 S then by 3 u, T / S by u |y|: log p and the entropy are within 4 u of 0
    assert abs(got[0][4]) <= 4 * U32 and abs(got[1][4]) <= 4 * U32 and got[0][5] == 0.0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("off,v", [(0, 2051), (1, 2051), (3, 2051), (1, 30011), (5, 30011)])
def test_rows_at_any_address(off, v, dtype):
    """Rows of a wider tensor, starting at every alignment; what lies beside them is
    larger than any logit and must not be seen."""
    x, tok = make(9, v, off, dtype)
    wide = torch.full((9, v + 7), 1000.0, dtype=x.dtype)
    wide[:, off:off + v] = x
    got = G.gptq_token_logprobs(wide.cuda()[:, off:off + v], tok.cuda(), 6)
    torch.cuda.synchronize()
    check(x, tok, 6, got)


def test_given_outputs_and_empty_batch():
    x, tok = make(6, 777, 1, "f16")
    out = (torch.full((6,), 9.0, device="cuda"), torch.full((6,), 9.0, device="cuda"),
           torch.full((6, 4), 9, dtype=torch.int32, device="cuda"), torch.full((6, 4), 9.0, device="cuda"))
    got = G.gptq_token_logprobs(x.cuda(), tok.cuda(), 4, *out)
    torch.cuda.synchronize()
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(got, out))
    check(x, tok, 4, got)
    e = G.gptq_token_logprobs(x.cuda()[:0], tok.cuda()[:0], 4)
    assert [t.shape[0] for t in e] == [0, 0, 0, 0]


def test_more_than_2_to_31_logits_and_overlaps():
    n, v = 33000, 65600
    x = torch.zeros(n, v, dtype=torch.bfloat16, device="cuda")
    tail, tok = make(4, v, 11, "bf16")
    x[-4:] = tail.cuda()
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    t[-4:] = tok.cuda()
    got = G.gptq_token_logprobs(x, t, 3)
    torch.cuda.synchronize()
    check(tail, tok, 3, tuple(a[-4:] for a in got))
    out = torch.zeros(8, device="cuda")
    with pytest.raises(ValueError, match="overlaps"):
        G.gptq_token_logprobs(x[:4], t[:4], 0, logprobs=out[:4], entropy=out[3:7])


@pytest.mark.parametrize("n,v", [(1, 6000), (1, 40000), (1200, 6000)])
def test_graph_replays_match_eager(n, v):
    x = torch.randn(n, v, device="cuda").to(torch.bfloat16)
    tok = torch.randint(0, v, (n,), device="cuda")
    G.gptq_token_logprobs(x, tok, 8)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = G.gptq_token_logprobs(x, tok, 8)
    for r in range(3):
        x.copy_(torch.randn(n, v, device="cuda"))
        tok.random_(0, v)
        ref = G.gptq_token_logprobs(x, tok, 8)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref)), r
    del g
