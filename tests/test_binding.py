"""What the Python binding takes for a pointer (CPU only: the calls have no rows, so
nothing is read or launched whatever they take)."""
import os

import numpy as np
import pytest

import bit_weight_quantized_amd as qmm

needs_lib = pytest.mark.skipif(not os.path.exists(qmm.lib_path()),
                               reason="libqmm.so not built (run __graft_entry__.build())")
P = 1 << 20


@needs_lib
@pytest.mark.parametrize("wrong", [b"\0" * 4096, "text", bytearray(16), np.zeros(16, np.uint8), [1], 1.5],
                         ids=lambda v: type(v).__name__)
def test_only_tensors_addresses_and_none_are_pointers(wrong):
    def calls(p):
        qmm.qmm_fp8_quant(p, 0, 128, 128, P, P, stream=0)
        qmm.qmm_fp8_gemm(P, P, 0, 32, 128, P, p, P, 32, stream=0)
        qmm.qmm_moe_gather(P, 8, 64, 0, 2, P, p, P, P, stream=0)

    calls(P)
    calls(None)
    for call in (lambda: qmm.qmm_fp8_quant(wrong, 0, 128, 128, P, P, stream=0),
                 lambda: qmm.qmm_fp8_gemm(P, P, 0, 32, 128, P, wrong, P, 32, stream=0),
                 lambda: qmm.qmm_moe_gather(P, 8, 64, 0, 2, P, wrong, P, P, stream=0),
                 lambda: qmm.qmm_norm_residual(0, 64, None, 64, None, None, 0, 1, wrong, qmm.QMM_BF16, 64, 1.0, P, 64, P,
                                               0.0, 1e-6, P, 64, None, None, stream=0)):
        with pytest.raises(AttributeError):
            call()


def test_addresses_and_none_raise_nothing_inside(monkeypatch):
    """An address is looked at by its type, not by a failed attribute: 0.09 us, not 0.39."""
    import enum

    class Address(enum.IntEnum):
        A = P

    import sys
    events = []
    sys.settrace(lambda frame, event, arg: (events.append(event), lambda f, e, a: events.append(e))[1])
    try:
        got = [qmm._ptr(v) for v in (None, 0, P)]
    finally:
        sys.settrace(None)
    assert got == [None, 0, P] and "exception" not in events
    assert qmm._ptr(Address.A) == P


def test_current_stream_without_the_private_lookup(monkeypatch):
    """A torch without its private function for the raw handle: the public one serves."""
    torch = pytest.importorskip("torch")

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(qmm, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream() if device == 3 else None)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert qmm._stream(None) == 77
    assert qmm._stream(0) == 0 and qmm._stream(Stream()) == 77
