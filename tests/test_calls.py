"""The short way of the int8 and distillation calls: the same bits as the binding's own path,
and left to that path wherever a call is not an ordinary one."""
import os

import pytest

import post_weight_quantization_02_amd as G

torch = pytest.importorskip("torch")

CALLS = os.path.join(os.path.dirname(G.__file__), "_lib", "_calls.so")
pytestmark = pytest.mark.skipif(not os.path.exists(CALLS), reason="_calls.so not built (run __graft_entry__.build())")


def test_what_is_no_ordinary_call_is_left_alone():
    """On the host: tensors of other places, things that are no tensors, too few arguments."""
    c = G._calls()
    x, s = torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for args in ((torch.zeros(4, 8),), (None,), (3,), ("x",), (), (x, x), (torch.zeros(4),), (torch.zeros(0, 4),)):
        assert c.int8_quantize(*args) is None
    for args in ((x, s, x, s, None, None), (x, s, x, s, None, 7), (x, s, x, s, "b", torch.float16), (x, s), (None,) * 6, (1, 2, 3, 4, 5, 6),
                 (x.to("meta"), s.to("meta"), x.to("meta"), s.to("meta"), None, None)):
        assert c.int8_matmul(*args) is None
    for args in ((x, s, x[None], s[None], ids[0], None, None, None), (x, s, x, s, ids[0], None, None, None), (None,) * 8, ()):
        assert c.int8_matmul_grouped(*args) is None
    for args in ((torch.zeros(4, 8), ids, torch.zeros(4, 2), 1.0, False, None, True), (x, ids, s, 1, 0, None, 1), (None,) * 7, (1,)):
        assert c.distill_loss(*args) is None


def cases():
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(30, 200, device="cuda", generator=g)
    xc, sx = G.gptq_int8_quantize(x)
    w = torch.randn(4, 70, 200, device="cuda", generator=g)
    wc, sw = G.gptq_int8_quantize(w.view(-1, 200))
    wc, sw = wc.view(4, 70, 200), sw.view(4, 70)
    off = torch.tensor([0, 5, 5, 20, 30], dtype=torch.int32, device="cuda")
    rows = torch.randperm(30, device="cuda", generator=g).int()
    bias = torch.randn(4, 70, device="cuda", generator=g).half()
    z = torch.randn(9, 700, device="cuda", generator=g).bfloat16()
    ids = torch.randint(0, 700, (9, 5), device="cuda", generator=g, dtype=torch.int32)
    lp = torch.log_softmax(torch.randn(9, 5, device="cuda", generator=g), 1) - 0.1
    weights = torch.rand(9, device="cuda", generator=g)
    xl, sl = G.gptq_int8_quantize(torch.randn(100, 5000, device="cuda", generator=g))      # a product in parts
    return [("int8_quantize", G.gptq_int8_quantize, (x,)), ("int8_quantize", G.gptq_int8_quantize, (x[:, 3:].half(),)),
            ("int8_quantize", G.gptq_int8_quantize, (x[:, 3:190],)),
            ("int8_matmul", G.gptq_int8_matmul, (xc, sx, wc[1], sw[1], None, None)),
            ("int8_matmul", G.gptq_int8_matmul, (xc, sx, wc[1], sw[1], bias[1], torch.float16)),
            ("int8_matmul", G.gptq_int8_matmul, (xl, sl, xl, sl, None, torch.bfloat16)),
            ("int8_matmul_grouped", G.gptq_int8_matmul_grouped, (xc, sx, wc, sw, off, None, None, None)),
            ("int8_matmul_grouped", G.gptq_int8_matmul_grouped, (xc, sx, wc, sw, off, rows, bias, torch.float16)),
            ("distill_loss", G.gptq_distill_loss, (z, ids, lp, 1.0, False, None, False)),
            ("distill_loss", G.gptq_distill_loss, (z.float(), ids, lp, 2.0, True, weights, True))]


def own_path(name, fn, args):
    """The same call with a stream given, which the binding's own path takes."""
    stream = torch.cuda.current_stream()
    if name == "int8_matmul":
        return fn(*args[:5], out_dtype=args[5], stream=stream)
    if name == "int8_matmul_grouped":
        return fn(*args[:7], out_dtype=args[7], stream=stream)
    return fn(*args, stream=stream)


def same(a, b):
    a, b = (t if isinstance(t, tuple) else (t,) for t in (a, b))
    return len(a) == len(b) and all((u is None and v is None) or (u.dtype == v.dtype and u.shape == v.shape and u.stride() == v.stride()
                                    and torch.equal(u, v)) for u, v in zip(a, b))


@pytest.mark.gpu
def test_the_same_bits_as_the_bindings_own_path():
    for name, fn, args in cases():
        short = getattr(G._calls(), name)(*args)
        assert short is not None, name
        whole = own_path(name, fn, args)
        torch.cuda.synchronize()
        assert same(short, whole), name


@pytest.mark.gpu
def test_on_the_current_stream():
    """The stream that is current where the call is made, behind work that is still running there."""
    todo = cases()
    ref = [own_path(*c) for c in todo]
    torch.cuda.synchronize()
    side, busy = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda")
    with torch.cuda.stream(side):
        got = []
        for name, fn, args in todo:
            for _ in range(3):
                busy = busy @ busy * 1e-3
            late = tuple(a.clone() + (torch.nan_to_num(busy[0, 0]) * 0).to(a.dtype) if isinstance(a, torch.Tensor) and a.is_contiguous()
                         else a for a in args)
            got.append(getattr(G._calls(), name)(*late))
    side.synchronize()
    assert all(same(a, b) for a, b in zip(ref, got))


@pytest.mark.gpu
def test_gradients_tangents_traces_and_odd_tensors_go_the_other_way():
    import torch.autograd.forward_ad as fwd
    c = G._calls()
    for name, fn, args in cases():
        call = getattr(c, name)
        for at, a in enumerate(args):
            if not isinstance(a, torch.Tensor):
                continue
            short = a.cpu() if name == "int8_matmul_grouped" and at == 5 else a.flatten()[:-1]      # fewer rows are fine
            for other in (a.cpu(), a.double(), a[None], short, a.repeat_interleave(2, -1)[..., ::2]):
                assert call(*args[:at], other, *args[at + 1:]) is None, (name, at, other.shape, other.dtype)
            if a.is_floating_point():
                wanted = a.detach().clone().requires_grad_(True)
                assert call(*args[:at], wanted, *args[at + 1:]) is None
                with torch.no_grad():
                    assert call(*args[:at], wanted, *args[at + 1:]) is not None
        with fwd.dual_level():
            assert call(*args) is None
        with torch.inference_mode():
            assert call(*args) is not None
        fine = args[0] if args[0].is_floating_point() else args[1]
        with pytest.raises(Exception, match="cannot be traced"):
            torch.jit.trace(lambda v: [t for t in (fn(v, *args[1:]) if args[0] is fine else fn(args[0], v, *args[2:])) if t is not None][0]
                            if name != "int8_matmul" and name != "int8_matmul_grouped" else
                            (fn(args[0], v, *args[2:5]) if name == "int8_matmul" else fn(args[0], v, *args[2:7])), (fine,))
