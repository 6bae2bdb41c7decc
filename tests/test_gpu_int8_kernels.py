"""Every kernel that the rules of the int8 products pick, with operands and outputs inside
wider tensors, NaN scales, biases, and rows at odd addresses: bitwise the definition, or for
experts the plain product of their rows."""
import ctypes
import os

import pytest

torch = pytest.importorskip("torch")

import post_weight_quantization_02_amd as G  # noqa: E402

(FEW16, FEW16_OWN, FEW16_OWN_DEEP, FEW32, FEW64, T64x32, T64x64, T96x64, T128x64, T128x128_TWO, T128x128,
 T256x256) = range(12)
SPLIT = 100
CASES = [(FEW16, 9, 301, 1000), (FEW16_OWN_DEEP, 13, 8201, 1000), (FEW16_OWN_DEEP, 1, 9001, 130), (FEW32, 27, 301, 1030),
         (FEW64, 50, 301, 1024), (T64x32, 70, 203, 1000), (T64x32 + SPLIT, 100, 161, 5000), (T64x64, 200, 2101, 1000),
         (T96x64, 260, 4001, 1000), (T128x64, 500, 4001, 520), (T128x128_TWO, 1001, 2101, 1000), (T128x128, 513, 16501, 384),
         (T256x256, 4001, 4007, 1000), (T256x256, 4001, 4007, 897), (T256x256, 4090, 4090, 1024), (T256x256, 4397, 7097, 900)]
GROUPED = [(FEW16, 40, 4, 1300, 2100), (FEW16_OWN, 9, 5, 301, 1000), (FEW16_OWN, 6, 20, 300, 128), (FEW16_OWN_DEEP, 5, 7, 301, 2060),
           (FEW32, 40, 10, 1300, 2100), (T128x64, 4, 30, 1001, 1000), (T128x64, 3, 90, 500, 2100), (T128x128_TWO, 20, 35, 1001, 520),
           (T128x128, 30, 40, 1300, 385), (T128x128, 12, 200, 2100, 260), (T256x256, 4, 520, 4001, 640), (T256x256, 3, 900, 4100, 1000)]


class _Plan(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("splits", ctypes.c_int), ("ws_bytes", ctypes.c_size_t)]


@pytest.mark.skipif(not os.path.exists(G.lib_path()), reason="libgptq.so not built (run __graft_entry__.build())")
def test_the_cases_reach_every_kernel():
    rule = G.library()["_ZN4gptq9int8_planElll"]                       # gptq::int8_plan(m, n, k)
    rule.restype, rule.argtypes = _Plan, [ctypes.c_int64] * 3
    for want, m, n, k in CASES:
        p = rule(m, n, k)
        assert p.kind + (SPLIT if p.splits > 1 else 0) == want, (m, n, k, p.kind, p.splits)
    assert {c[0] for c in CASES} == (set(range(12)) | {T64x32 + SPLIT}) - {FEW16_OWN}
    rule = G.library()["_ZN4gptq17int8_grouped_planEllll"]             # gptq::int8_grouped_plan(m, n, k, experts)
    rule.restype, rule.argtypes = _Plan, [ctypes.c_int64] * 4
    for want, experts, each, n, k in GROUPED:
        assert rule(experts * each, n, k, experts).kind == want, (experts, each, n, k, rule(experts * each, n, k, experts).kind)
    assert {c[0] for c in GROUPED} == set(range(12)) - {FEW64, T64x32, T64x64, T96x64}
    seen = set()
    for m in range(1, 3000, 7):                                        # the rule by experts picks nothing else
        for experts in (1, 3, 17, 300, 4096):
            for n, k in ((1, 1), (300, 3000), (5000, 500), (70000, 9000)):
                seen.add(rule(m, n, k, experts).kind)
    assert seen == {c[0] for c in GROUPED}


def inside(t, before, after, fill):
    """t as columns of a wider tensor, and that tensor."""
    wide = torch.full((*t.shape[:-1], before + t.shape[-1] + after), fill, dtype=t.dtype, device=t.device)
    view = wide[..., before:before + t.shape[-1]]
    view.copy_(t)
    return view, wide


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("at", range(len(CASES)), ids=[f"{c[0]}_{c[1]}x{c[2]}x{c[3]}" for c in CASES])
def test_strides_and_nan_scales(at, out):
    from test_gpu_int8 import TYPES, defined, operands
    _, m, n, k = CASES[at]
    xc, sx, wc, sw = operands(m, n, k, at)
    if out == "f16":
        sx = sx * 1e-3
    i, j = m // 2, n - 5
    sx[i], sw[j] = float("nan"), float("inf")
    pad = -k % 16 + 16                                       # rows a multiple of 16 bytes apart
    (xc, _), (wc, _) = inside(xc, 16, pad, 99), inside(wc, 32, pad, 99)
    ref = defined(xc, sx, wc, sw)
    y, wide = inside(torch.zeros(m, n, dtype=TYPES[out], device="cuda"), 5, 2, 7.0)
    assert G.gptq_int8_matmul(xc, sx, wc, sw, Y=y) is y
    torch.cuda.synchronize()
    assert torch.equal(torch.nan_to_num(y, 1.0, 2.0, 3.0), torch.nan_to_num(ref.to(TYPES[out]), 1.0, 2.0, 3.0))
    assert torch.isnan(y[i]).all() and (wide[:, :5] == 7.0).all() and (wide[:, 5 + n:] == 7.0).all()
    bias = torch.randn(n + 1, device="cuda").to(TYPES[out])[1:]
    z = G.gptq_int8_matmul(xc, sx, wc, sw, bias, out_dtype=TYPES[out])
    few = G.gptq_int8_matmul(xc[-3:], sx[-3:], wc, sw, bias, out_dtype=TYPES[out])       # another kernel
    torch.cuda.synchronize()
    assert torch.equal(torch.nan_to_num(z[-3:], 1.0, 2.0, 3.0), torch.nan_to_num(few, 1.0, 2.0, 3.0)) and torch.isnan(z[i]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("at", range(len(GROUPED)), ids=[f"{c[0]}_{c[1]}x{c[2]}x{c[3]}x{c[4]}" for c in GROUPED])
def test_by_expert(at):
    """Parts of unlike sizes around the mean, one of them all of the rest; a bad row."""
    from test_gpu_int8 import TYPES
    from test_gpu_int8_grouped import by_parts, inputs, offsets, stack
    _, experts, each, n, k = GROUPED[at]
    out = ("bf16", "f32", "f16")[at % 3]
    g = torch.Generator().manual_seed(at)
    m = experts * each
    counts = torch.bincount(torch.randint(0, experts, (m,), generator=g) // 2 * 2 % experts, minlength=experts).tolist()
    xc, sx = inputs(m // 2 + 1, k, at)
    wc, sw = stack(experts, n, k, at + 1, pitch=-(-k // 16) * 16 + 16, gap=3)
    sx = sx * (1e-3 if out == "f16" else 1.0)
    rows = torch.randint(0, m // 2 + 1, (m,), generator=g).to(torch.int32).cuda()
    bias = torch.randn(experts, n, device="cuda").to(TYPES[out]) if at % 2 else None
    for sizes in (counts, [0] * (experts - 1) + [m], [m - experts + 1] + [1] * (experts - 1)):
        off = offsets(sizes)
        y = G.gptq_int8_matmul_grouped(xc, sx, wc, sw, off, rows, bias, out_dtype=TYPES[out])
        ref = by_parts(xc, sx, wc, sw, off, rows, bias, TYPES[out], torch.zeros(m, n, dtype=TYPES[out], device="cuda"))
        torch.cuda.synchronize()
        assert torch.equal(y, ref), sizes[:10]
    bad = rows.clone()
    bad[m // 2] = -1
    z = G.gptq_int8_matmul_grouped(xc, sx, wc, sw, off, bad, bias, out_dtype=TYPES[out])
    torch.cuda.synchronize()
    assert torch.isnan(z[m // 2]).all()
    z[m // 2] = y[m // 2]
    assert torch.equal(z, y)


@pytest.mark.gpu
def test_workspaces_of_the_callers_own():
    """The same bits as with the call's own; what lies behind the workspace is left alone, one
    byte too few is refused, and so is one that shares an operand's memory."""
    from test_gpu_int8 import operands
    xc, sx, wc, sw = operands(100, 161, 5000, 3)
    need = G.gptq_int8_matmul_workspace_size(100, 161, 5000)
    assert need > 0
    ref = G.gptq_int8_matmul(xc, sx, wc, sw)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    for at in (0, 0, 1000, 77):                              # twice the same, and at an odd address
        got = G.gptq_int8_matmul(xc, sx, wc, sw, ws=ws[at:at + need])
        torch.cuda.synchronize()
        assert torch.equal(got, ref) and (ws[at + need:] == 0x5A).all() and (at == 0 or (ws[:at] == 0x5A).all())
        ws.fill_(0x5A)
    with pytest.raises(G.GPTQError):
        G.gptq_int8_matmul(xc, sx, wc, sw, ws=ws[:need - 1])
    for taken in (xc, wc):
        whole = torch.empty(0, dtype=torch.uint8, device="cuda").set_(taken.untyped_storage())
        with pytest.raises(ValueError, match="overlaps"):
            G.gptq_int8_matmul(xc, sx, wc, sw, ws=whole)
