"""qmm_profile_next around every call of the block-scaled path, one launch, two, and
several parts (needs an MI355X)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_quantized_amd as qmm  # noqa: E402
import test_gpu_fp8 as base  # noqa: E402
from test_gpu_fp8 import DEV, _gpu, say  # noqa: E402,F401

NAMES = ["qmm_norm_residual", "qmm_route_topk", "qmm_fp8_grouped_gemm_swiglu", "qmm_fp8_quant", "qmm_fp8_grouped_gemm",
         "qmm_moe_gather", "qmm_fp8_gemm"]


def bracketed(call):
    """Milliseconds between the events of one call; its outputs are done at the second."""
    hip = ctypes.CDLL("libamdhip64.so")
    ev = [ctypes.c_void_p(), ctypes.c_void_p()]
    for e in ev:
        assert hip.hipEventCreate(ctypes.byref(e)) == 0
    try:
        qmm.qmm_profile_next(ev[0].value, ev[1].value)
        call()
        assert hip.hipEventSynchronize(ev[1]) == 0
        ms = ctypes.c_float(-1.0)
        assert hip.hipEventElapsedTime(ctypes.byref(ms), ev[0], ev[1]) == 0
        return ms.value
    finally:
        torch.cuda.synchronize()
        for e in ev:
            hip.hipEventDestroy(e)


# 3 tokens: few-row kernels and one router launch; 200: tiles and two router launches
@pytest.mark.parametrize("t", [3, 200])
@pytest.mark.parametrize("name", NAMES)
def test_events_bracket_each_call(name, t, monkeypatch):
    say("profile", name, t)
    v, run, fill, reset = base.layer(t, 12, 4, 256, 144, 7300 + t)
    fill(7)
    run()
    want = {n: x.clone() for n, x in v.items()}
    real, seen = getattr(qmm, name), []

    def timed(*args, **kw):
        seen.append(bracketed(lambda: real(*args, **kw)))

    monkeypatch.setattr(qmm, name, timed)
    run()
    torch.cuda.synchronize()
    assert len(seen) == 1 and 0.0 < seen[0] < 100.0
    assert all(torch.equal(x.view(torch.uint8), want[n].view(torch.uint8)) for n, x in v.items())


def test_events_bracket_all_parts_of_a_gather():
    """2^24 tokens are two launches: the events are the first's start and the last's end."""
    def gather(t):
        slot = torch.zeros(t, 1, dtype=torch.int32, device=DEV)
        w, o = torch.ones(t, 1, device=DEV), torch.ones(1, 8, dtype=torch.bfloat16, device=DEV)
        out = torch.zeros(t, 8, dtype=torch.bfloat16, device=DEV)
        call = lambda: qmm.qmm_moe_gather(o, 1, 8, t, 1, slot, w, None, out)  # noqa: E731
        call()
        ms = min(bracketed(call) for _ in range(3))
        assert bool((out == 1.0).all())
        return ms
    half, whole = gather(1 << 23), gather(1 << 24)
    say("gather of 2^23, 2^24 tokens, ms", half, whole)
    assert whole > 1.5 * half
