"""The fp64 oracle of the e4m3 codes, their product and token log probabilities
against closed forms and torch's own e4m3 cast."""
import math

import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")


def test_e4m3_table_and_rounding_match_the_format():
    v = O.fp8.e4m3_value(np.arange(256))
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    np.testing.assert_array_equal(np.isnan(v), np.isnan(ref))
    np.testing.assert_array_equal(v[~np.isnan(v)], ref[~np.isnan(ref)])
    assert np.nanmax(v) == 448.0 and v[1] == 2.0 ** -9
    x = np.concatenate([np.random.default_rng(0).standard_normal(4000) * s for s in (0.01, 1.0, 100.0)])
    x = np.clip(x, -448, 448).astype(np.float32)
    mids = (v[:126] + v[1:127]) / 2                      # ties
    for u in (x, mids.astype(np.float32), -mids.astype(np.float32)):
        got = O.fp8.e4m3_code(u)
        exp = torch.from_numpy(u).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        np.testing.assert_array_equal(got, exp)


@pytest.mark.parametrize("a,s", [(448.0, 1.0), (448.0001, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8),
                                 (1.76, 2.0 ** -7), (0.0, 1.0), (1e-45, 2.0 ** -126), (3e38, 2.0 ** 120)])
def test_block_scale_closed_forms(a, s):
    assert O.fp8.block_scale(np.array([0.0, -a])) == s
    assert O.fp8.block_scale(np.array([np.inf, -a, np.nan])) == s


def test_quantize_layouts_and_error():
    x = np.random.default_rng(1).standard_normal((130, 200)).astype(np.float32)
    for rows, shape in ((1, (2, 130)), (128, (2, 2))):
        c, s = O.fp8.quantize(x, rows)
        assert s.shape == shape
        d = O.fp8.dequantize(c, s, rows)
        # half a step of e4m3 relative to the value, or half a subnormal step of the block
        bound = np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10 * s.max())
        assert np.all(np.abs(d - x) <= bound)


def test_matmul_of_exact_codes():
    x = np.random.default_rng(2).integers(-8, 9, (3, 300)).astype(np.float64)
    w = np.random.default_rng(3).integers(-8, 9, (5, 300)).astype(np.float64)
    xc, xs = O.fp8.quantize(x, 1)
    wc, ws = O.fp8.quantize(w, 128)
    y, _ = O.fp8.matmul(xc, xs, wc, ws, np.arange(5.0))
    np.testing.assert_array_equal(y, x @ w.T + np.arange(5.0))


def test_token_logprobs_closed_forms():
    lp, ent, ids, tops = O.fp8.token_logprobs(np.zeros((1, 8)), [3], 3)
    assert math.isclose(lp[0], -math.log(8)) and math.isclose(ent[0], math.log(8))
    assert ids.tolist() == [[0, 1, 2]] and np.allclose(tops, -math.log(8))
    x = np.array([[0.0, -np.inf, math.log(3.0), -np.inf], [-np.inf] * 4, [1.0, np.inf, 0.0, 2.0], [0.0, np.nan, 1.0, 2.0]])
    lp, ent, ids, tops = O.fp8.token_logprobs(x, [2, 0, -1, 9], 4)
    assert math.isclose(lp[0], math.log(0.75)) and np.isnan(lp[1]) and lp[2] == 0.0 and np.isnan(lp[3])
    assert math.isclose(ent[0], -(0.75 * math.log(0.75) + 0.25 * math.log(0.25))) and np.isnan(ent[1:]).all()
    assert ids.tolist() == [[2, 0, 1, 3], [0, 1, 2, 3], [1, 3, 0, 2], [1, 3, 2, 0]]
    assert tops[0, 2] == -np.inf
    ref = torch.log_softmax(torch.randn(6, 50, dtype=torch.float64, generator=torch.Generator().manual_seed(0)), 1)
    lp, ent, _, _ = O.fp8.token_logprobs(ref.numpy() + 100.0, [0] * 6, 0)
    np.testing.assert_allclose(lp, ref[:, 0].numpy(), rtol=0, atol=1e-12)
    np.testing.assert_allclose(ent, -(ref.exp() * ref).sum(1).numpy(), rtol=0, atol=1e-12)
