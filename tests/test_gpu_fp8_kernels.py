"""Every kernel that the fp8 product's rule picks, with operands and outputs inside wider
tensors and with NaN codes; workspaces of the caller's own.

Bounds as in test_gpu_fp8: the elementwise bound of the sums and half a step of the type.
"""
import ctypes
import os

import pytest

torch = pytest.importorskip("torch")

import post_weight_quantization_02_amd as G  # noqa: E402

FEW, T64x32, T64x64, T96x64, T128x64, T128x128_TWO, T128x128, T256x256 = range(8)
SPLIT = 100
# what the rule picks for 16-bit and for fp32 outputs, m, n, k
CASES = [(FEW, FEW, 9, 301, 1000), (FEW, FEW, 27, 301, 1030), (FEW, FEW, 50, 301, 1024),
         (T64x32, T64x32, 70, 203, 1000), (T64x32 + SPLIT, T64x32 + SPLIT, 100, 161, 5000),
         (T64x64, T64x64, 200, 2101, 1000), (T96x64, T96x64, 260, 4001, 1000), (T128x64, T128x64, 500, 4001, 520),
         (T128x128_TWO, T128x128_TWO, 1001, 2101, 1000), (T128x128, T128x128, 513, 16501, 384),
         (T128x128, T128x128, 1030, 20999, 1000), (T256x256, T128x128, 4001, 4007, 1000), (T256x256, T128x128, 4001, 4007, 897),
         (T256x256, T128x128, 4090, 4090, 1024), (T256x256, T128x128, 4397, 7097, 900)]
IDS = [f"{c[0]}_{c[2]}x{c[3]}x{c[4]}" for c in CASES]


class _Plan(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("splits", ctypes.c_int), ("ws_bytes", ctypes.c_size_t)]


@pytest.mark.skipif(not os.path.exists(G.lib_path()), reason="libgptq.so not built (run __graft_entry__.build())")
def test_the_cases_reach_every_kernel():
    rule = G.library()["_ZN4gptq8fp8_planElllb"]             # gptq::fp8_plan(m, n, k, wide)
    rule.restype, rule.argtypes = _Plan, [ctypes.c_int64] * 3 + [ctypes.c_bool]
    for narrow, wide, m, n, k in CASES:
        for want, is_wide in ((narrow, False), (wide, True)):
            p = rule(m, n, k, is_wide)
            assert p.kind + (SPLIT if p.splits > 1 else 0) == want, (m, n, k, is_wide, p.kind, p.splits)
    assert {c[0] for c in CASES} == set(range(8)) | {T64x32 + SPLIT} and {c[1] for c in CASES} == set(range(7)) | {T64x32 + SPLIT}


def inside(t, before, after, fill):
    """t as columns of a wider tensor, and that tensor."""
    wide = torch.full((t.shape[0], before + t.shape[1] + after), fill, dtype=t.dtype, device=t.device)
    view = wide[:, before:before + t.shape[1]]
    view.copy_(t)
    return view, wide


@pytest.mark.gpu
@pytest.mark.parametrize("wide_out", [False, True], ids=["16bit", "f32"])
@pytest.mark.parametrize("at", range(len(CASES)), ids=IDS)
def test_strides_and_nan_codes(at, wide_out):
    from test_gpu_fp8 import TYPES, check, operands
    _, _, m, n, k = CASES[at]
    out = "f32" if wide_out else ("f16", "bf16")[at % 2]
    xc, sx, wc, sw = operands(m, n, k, at)
    if out == "f16":
        sx = sx * 1e-3
    pad = -k % 16 + 16                                       # rows a multiple of 16 bytes apart
    (xc, _), (wc, _) = inside(xc, 16, pad, 0x7F), inside(wc, 32, pad, 0x7F)
    (sx, _), (sw, _) = inside(sx, 1, 2, float("nan")), inside(sw, 2, 1, float("nan"))
    bias = torch.randn(n + 1, device="cuda").to(TYPES[out])[1:]
    y, wide = inside(torch.zeros(m, n, dtype=TYPES[out], device="cuda"), 5, 2, 7.0)
    assert G.gptq_fp8_matmul(xc, sx, wc, sw, bias, Y=y) is y
    torch.cuda.synchronize()
    check(y, out, xc, sx, wc, sw, bias)
    assert (wide[:, :5] == 7.0).all() and (wide[:, 5 + n:] == 7.0).all()
    ref = y.clone()
    i, j = m // 2, n - 50
    xc[i, k - 1] = 0x7F
    wc[j, 7] = 0xFF
    G.gptq_fp8_matmul(xc, sx, wc, sw, bias, Y=y)
    torch.cuda.synchronize()
    assert torch.isnan(y[i]).all() and torch.isnan(y[:, j]).all()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[i], keep[:, j] = False, False
    assert torch.equal(y[keep], ref[keep])
    assert (wide[:, :5] == 7.0).all() and (wide[:, 5 + n:] == 7.0).all()


@pytest.mark.gpu
def test_workspaces_of_the_callers_own():
    """The same bits as with the call's own; what lies behind the workspace is left alone,
    one byte too few is refused."""
    from test_gpu_fp8 import operands
    xc, sx, wc, sw = operands(100, 161, 5000, 3)
    x = torch.randn(3, 50000, device="cuda")
    t = torch.tensor([1, -1, 49999], device="cuda")
    for need, call in ((G.gptq_fp8_matmul_workspace_size(100, 161, 5000), lambda ws: [G.gptq_fp8_matmul(xc, sx, wc, sw, ws=ws)]),
                       (G.gptq_token_logprobs_workspace_size(3, 50000, 7), lambda ws: G.gptq_token_logprobs(x, t, 7, ws=ws))):
        assert need > 0
        ref = call(None)
        ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        for at in (0, 0, 1000, 77):                          # twice the same, and at an odd address
            got = call(ws[at:at + need])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, ref)) and (ws[at + need:] == 0x5A).all()
            assert at == 0 or (ws[:at] == 0x5A).all()
            ws.fill_(0x5A)
        with pytest.raises(G.GPTQError):
            call(ws[:need - 1])


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_a_row_alone_and_among_many(out):
    """What the product promises of a row whose call has other rows: fp32 outputs within
    2 (k + 4) u sum |x w|, 16-bit ones within that, 7 * 2^-13 sum |x w| and the two roundings."""
    import numpy as np
    import oracle as O
    from test_gpu_fp8 import TINY, TYPES, U32, bits, f64, operands
    m, n, k = 300, 260, 1030
    xc, sx, wc, sw = operands(m, n, k, 8)
    sx = sx * 1e-3
    many = G.gptq_fp8_matmul(xc, sx, wc, sw, out_dtype=TYPES[out])
    few = torch.cat([G.gptq_fp8_matmul(xc[i:i + 10], sx[:, i:i + 10], wc, sw, out_dtype=TYPES[out]) for i in range(0, m, 10)])
    torch.cuda.synchronize()
    y, mag = O.fp8.matmul(bits(xc), sx.cpu().numpy(), bits(wc), sw.cpu().numpy())
    off = (2 * (k + 4) * U32 + (0.0 if out == "f32" else 7 * 2.0 ** -13)) * mag
    off = off + 2 * ((np.abs(y) + off) * torch.finfo(TYPES[out]).eps / 2 + TINY[out])
    assert np.all(np.abs(f64(many) - f64(few)) <= off)
