"""Log probabilities of rows whose logits, or whose masks' values, are far from zero.

The exponent y = (x - M) log2 e carries the roundings of the difference, of the product
and of log2 e itself, 2.3 u |d| with d = x - M, or, where x log2 e and M log2 e are
subtracted in one rounding, u (1.5 |d| + 1/16); the exponential adds 2 u.  A lane adds at
most v / 64 terms one after another, a tree the lanes and parts (64 u allowed): S is off by
eS = u (v / 64 + 64 + 3 E|d|), E|d| = -T / S.  log p = ln 2 (y - log2 S) has three more
roundings and that of ln 2: eS + 4 u (|log p| + 2 log S + 1).  The entropy is off by
(eS + 8 u) (1 + E|d| + log S).
"""
import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import post_weight_quantization_02_amd as G  # noqa: E402

U32 = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FAR = {"f16": [-6e4, -3e4, 1000.0, 6e4],
       "f32": [-1e6, -1e9, -1e10, -1e12, -1e20, -1e30, 2.0 ** 20, -2.0 ** 20, 2.0 ** 24, 2.0 ** 29, 2.0 ** 30, -2.0 ** 31,
               2.0 ** 31, 1e30, 2.0 ** 126, -2.0 ** 126]}
FAR["bf16"] = FAR["f32"]


def steps_above(c, dtype, j):
    """Values j steps of the type away from c towards zero."""
    bits, whole = (torch.int32, torch.float32) if dtype == "f32" else (torch.int16, TYPES[dtype])
    at = torch.tensor(c, dtype=torch.float32).to(whole).view(bits)
    return (at - j.to(bits)).view(whole)


def rows(v, dtype):
    g = torch.Generator().manual_seed(v)
    out = []
    for c in FAR[dtype]:
        out.append(steps_above(c, dtype, torch.zeros(v)))                               # one value throughout
        out.append(steps_above(c, dtype, torch.randint(0, 6, (v,), generator=g)))       # a few steps apart
        if c < 0:                                                                       # a mask's value
            x = torch.randn(v, generator=g)
            x[:min(5000, v - 9)] = c
            out.append(x.to(TYPES[dtype]))
            x = torch.randn(v, generator=g)
            x[9:] = c
            out.append(x.to(TYPES[dtype]))
            x = torch.randn(v, generator=g)
            x[torch.rand(v, generator=g) < 0.5] = c
            out.append(x.to(TYPES[dtype]))
        else:                                                                           # one token far above the rest
            x = torch.randn(v, generator=g)
            x[v // 3] = c
            out.append(x.to(TYPES[dtype]))
    return torch.stack(out), torch.randint(0, v, (len(out),), generator=g)


@pytest.mark.parametrize("top", [0, 5])
@pytest.mark.parametrize("v", [700, 3001, 40003])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rows_far_from_zero(dtype, v, top):
    x, tok = rows(v, dtype)
    tok[::2] = x[::2].float().argmax(1)
    got = [t.cpu().numpy() for t in G.gptq_token_logprobs(x.cuda(), tok.cuda(), top)]
    ref = O.fp8.token_logprobs(x.double().numpy(), tok.numpy(), top)
    np.testing.assert_array_equal(got[2], ref[2])
    d = x.double().numpy() - x.double().numpy().max(1)[:, None]
    p = np.exp(d)
    S = p.sum(1)
    Ed, logS = -(p * d).sum(1) / S, np.log(S)
    eS = U32 * (v / 64 + 64 + 3 * Ed)
    for name, a, b, tol in (("log p", got[0], ref[0], eS + 4 * U32 * (np.abs(ref[0]) + 2 * logS + 1)),
                            ("entropy", got[1], ref[1], (eS + 8 * U32) * (1 + Ed + logS)),
                            ("top", got[3], ref[3], eS[:, None] + 4 * U32 * (np.abs(ref[3]) + 2 * logS[:, None] + 1))):
        bad = ~(np.abs(a - b) <= tol)
        assert not bad.any(), (name, np.argwhere(bad)[:5].tolist(), a[bad][:5], b[bad][:5])
