"""Refusals of the int8 and distillation calls, on the host before any launch, in the C ABI
and in the binding (no GPU needed)."""
import math
import os
import subprocess
import sys

import pytest

import post_weight_quantization_02_amd as G
from post_weight_quantization_02_amd import _build

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(not os.path.exists(G.lib_path()),
                                reason="libgptq.so not built (run __graft_entry__.build())")

FAKE = 0x1000  # never dereferenced: validation fails first
OK, NULL, SIZE, LD, DTYPE, WS, LARGE, TEMPERATURE = 0, 1, 2, 3, 4, 8, 11, 9


def test_quantize_refusals():
    base = dict(X=FAKE, dt=0, m=4, k=300, ld=300, codes=FAKE, ldc=300, s=FAKE)

    def call(**kw):
        a = dict(base, **kw)
        return G.library().gptq_int8_quantize(a["X"], a["dt"], a["m"], a["k"], a["ld"], a["codes"], a["ldc"], a["s"], None)

    assert call(m=-1) == SIZE and call(k=0) == SIZE
    assert call(m=(1 << 30) + 1) == LARGE and call(k=1 << 21, ld=1 << 21, ldc=1 << 21) == LARGE
    assert call(dt=3) == DTYPE and call(dt=-1) == DTYPE
    assert call(X=None) == NULL and call(codes=None) == NULL and call(s=None) == NULL
    assert call(ld=299) == LD and call(ldc=299) == LD
    assert call(m=0, X=None, codes=None, s=None) == OK


def test_matmul_refusals():
    base = dict(x=FAKE, ldx=300, sx=FAKE, w=FAKE, ldw=300, sw=FAKE, m=4, n=10, k=300, b=None, y=FAKE, dt=0, ldy=10,
                ws=FAKE, wsb=1 << 40)

    def call(**kw):
        a = dict(base, **kw)
        return G.library().gptq_int8_matmul(a["x"], a["ldx"], a["sx"], a["w"], a["ldw"], a["sw"], a["m"], a["n"], a["k"],
                                            a["b"], a["y"], a["dt"], a["ldy"], a["ws"], a["wsb"], None)

    assert call(m=-1) == SIZE and call(n=0) == SIZE and call(k=0) == SIZE
    assert call(n=1 << 21, ldy=1 << 21) == LARGE
    assert call(k=1 << 17, ldx=1 << 17, ldw=1 << 17) == LARGE          # a sum may pass 2^31
    assert call(dt=5) == DTYPE
    for p in ("x", "sx", "w", "sw", "y"):
        assert call(**{p: None}) == NULL
    assert call(ldx=299) == LD and call(ldw=299) == LD and call(ldy=9) == LD
    assert call(m=0, x=None, y=None) == OK
    assert G.gptq_int8_matmul_workspace_size(0, 4, 4) == 0
    for m, n, k in ((1, 4096, 4096), (64, 4096, 4096), (512, 4096, 4096), (300, 128, 16384)):
        need = G.gptq_int8_matmul_workspace_size(m, n, k)
        if need:
            big = dict(m=m, n=n, k=k, ldx=k, ldw=k, ldy=n)
            assert call(ws=None, **big) == WS and call(wsb=need - 1, **big) == WS


def test_grouped_refusals():
    base = dict(x=FAKE, ldx=300, sx=FAKE, rx=4, r=FAKE, m=9, off=FAKE, e=3, w=FAKE, ldw=300, st=3000, sw=FAKE, n=10, k=300,
                b=None, y=FAKE, dt=0, ldy=10)

    def call(**kw):
        a = dict(base, **kw)
        return G.library().gptq_int8_matmul_grouped(a["x"], a["ldx"], a["sx"], a["rx"], a["r"], a["m"], a["off"], a["e"],
                                                    a["w"], a["ldw"], a["st"], a["sw"], a["n"], a["k"], a["b"], a["y"],
                                                    a["dt"], a["ldy"], None)

    assert call(m=-1) == SIZE and call(rx=-1) == SIZE and call(e=0) == SIZE and call(n=0) == SIZE and call(k=0) == SIZE
    assert call(rx=0) == SIZE and call(r=None) == SIZE                 # fewer rows than positions
    assert call(m=1 << 21) == LARGE and call(rx=1 << 21) == LARGE and call(e=4097) == LARGE
    assert call(k=1 << 17, ldx=1 << 17, ldw=1 << 17) == LARGE
    assert call(dt=3) == DTYPE
    for p in ("x", "sx", "off", "w", "sw", "y"):
        assert call(**{p: None}) == NULL
    assert call(ldx=299) == LD and call(ldw=299) == LD and call(ldy=9) == LD and call(st=2999) == LD
    assert call(m=0, x=None, rx=0) == OK


def test_distill_refusals():
    base = dict(x=FAKE, dt=0, n=2, v=100, ld=100, ids=FAKE, lp=FAKE, top=3, T=1.0, tail=0, w=None, loss=FAKE, g=None, ldg=100,
                ws=FAKE, wsb=1 << 40)

    def call(**kw):
        a = dict(base, **kw)
        return G.library().gptq_distill_loss(a["x"], a["dt"], a["n"], a["v"], a["ld"], a["ids"], a["lp"], a["top"], a["T"],
                                             a["tail"], a["w"], a["loss"], a["g"], a["ldg"], a["ws"], a["wsb"], None)

    assert call(n=-1) == SIZE and call(v=0) == SIZE and call(top=0) == SIZE and call(top=65) == SIZE
    assert call(v=2, ld=2) == SIZE and call(v=3, ld=3, tail=1) == SIZE     # with the rest: some token is in it
    assert call(v=1 << 21, ld=1 << 21) == LARGE and call(n=1 << 21) == LARGE
    assert call(dt=7) == DTYPE
    for T in (0.0, -1.0, 1e-5, 2e4, math.inf, math.nan):
        assert call(T=T) == TEMPERATURE
    for p in ("x", "ids", "lp", "loss"):
        assert call(**{p: None}) == NULL
    assert call(ld=99) == LD and call(g=FAKE, ldg=99) == LD
    assert call(n=0, x=None, ids=None) == OK
    need = G.gptq_distill_loss_workspace_size(1, 128000)
    assert need > 0
    big = dict(n=1, v=128000, ld=128000)
    assert call(ws=None, **big) == WS
    assert G.gptq_distill_loss_workspace_size(0, 5) == 0
    assert "temperature" in G.gptq_status_string(TEMPERATURE)


def test_binding_refuses_what_is_no_device_matrix():
    x, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    c, s = torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4)
    for f in (lambda: G.gptq_int8_quantize(x), lambda: G.gptq_int8_matmul(c, s, c, s),
              lambda: G.gptq_int8_matmul_grouped(c, s, c[None], s[None], torch.zeros(2, dtype=torch.int32)),
              lambda: G.gptq_distill_loss(x, ids, torch.zeros(4, 2)), lambda: G.gptq_distill_loss(torch.zeros(4), ids, x)):
        with pytest.raises(ValueError):
            f()


def test_refusals_are_clean_under_asan_and_ubsan():
    if os.environ.get("GPTQ_LIBRARY"):
        pytest.skip("already the sanitized build")
    env = dict(os.environ)
    env.update(GPTQ_LIBRARY=_build.build_sanitized(), LD_PRELOAD=_build.sanitizer_runtime(),
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-k", "refusals and not asan",
                          os.path.abspath(__file__)], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = res.stdout + res.stderr
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert res.returncode == 0 and "4 passed" in out, out[-4000:]


def test_top_logprobs_wants_a_token_at_least():
    from post_weight_quantization_02_amd import pipeline as P
    for kw in (dict(top_k=0), dict(top_k=-3), dict(rows_per_call=0)):
        with pytest.raises(ValueError, match="at least 1"):
            P.top_logprobs([], torch.nn.Linear(4, 6), [torch.zeros(1, 2, 4)], **kw)
