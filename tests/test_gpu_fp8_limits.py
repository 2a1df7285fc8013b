"""The gather and the norms at the most rows they take, which are more than one
launch holds (needs an MI355X)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_quantized_amd as qmm  # noqa: E402
from test_gpu_fp8 import DEV, _gpu, say  # noqa: E402,F401

T = 1 << 24
AT = [0, T // 2 - 500, T - 1000]                              # a launch of 256 threads a row ends at T / 2


def test_gather_of_the_most_tokens():
    say("gather", T)
    g = torch.Generator(device=DEV).manual_seed(1)
    o = torch.randn(1000, 8, device=DEV, generator=g).bfloat16()
    slot = torch.randint(-1, 1000, (T, 1), device=DEV, generator=g, dtype=torch.int32)
    w = torch.rand(T, 1, device=DEV, generator=g)
    out = torch.full((T, 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    qmm.qmm_moe_gather(o, 1000, 8, T, 1, slot, w, None, out)
    # one term: an fp32 product, rounded once
    want = torch.where(slot >= 0, w * o.float()[slot[:, 0].clamp(min=0)], torch.zeros((), device=DEV)).bfloat16()
    assert torch.equal(out, want)


def test_norm_of_the_most_rows():
    d = 520                                                   # 256 threads a row
    say("norm", T, d)
    g = torch.Generator(device=DEV).manual_seed(2)
    r = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    r.normal_(generator=g)
    w = torch.randn(d, device=DEV, generator=g).bfloat16()
    h = torch.full((T, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    qmm.qmm_norm_residual(T, d, None, d, None, None, 0, 1, r, qmm.QMM_BF16, d, 1.0, None, d, w, 0.0, 1e-6, h, d, None, None)
    for at in AT:
        v = r[at:at + 1000].double()
        want = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * w.double()
        # d / 8 + 24 roundings of the sum and a few more, then bf16
        tol = want.abs() * (2.0 ** -8 + (d // 8 + 32) * 2.0 ** -23) + 1e-40
        assert bool(((h[at:at + 1000].double() - want).abs() <= tol).all()), at
    for at in range(0, T, 1 << 21):
        assert bool(torch.isfinite(h[at:at + (1 << 21)]).all()), at
