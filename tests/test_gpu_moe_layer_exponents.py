"""The expert layer at the ends of its weights' exponents (needs an MI355X)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:overflow encountered in exp")]   # silu of -2^40

import bit_weight_quantized_amd as qmm  # noqa: E402
from oracle import mxfp4  # noqa: E402
from test_gpu_moe_layer import DEV, F32, M, Layer, bf16_bits, say  # noqa: E402
from test_gpu_moe_layer_half import Half  # noqa: E402
from test_gpu_mxfp4 import _check_guards, _gpu, as_f64, dev  # noqa: E402,F401


def drawn(rng, n, d, lo, hi, codes):
    """A matrix of given codes (of either sign) and exponents."""
    q = mxfp4.pack_codes(rng.choice(codes, (n, d)) | rng.integers(0, 2, (n, d)) << 3)
    e = rng.integers(lo, hi + 1, (n, d // 32)).astype(np.uint8)
    packed = torch.empty(qmm.qmm_packed_bytes(M, n, d), dtype=torch.uint8, device=DEV)
    qmm.qmm_pack(M, n, d, dev(q), dev(e), None, packed)
    return mxfp4.dequant(q, e), packed


def layer(kind, up, down, x, seed, codes=range(8)):
    """Exponents of the two stacks, ends included, and activations' magnitude."""
    l = kind((5, 4, 2, 288, 160, "softmax", False, 1, 1, False, True, F32, 0, False), seed)
    l.scale = 1.0
    rng = np.random.default_rng(seed)
    for e in range(l.ne):
        for n, d, (lo, hi), into, blob in ((320, 288, up, l.gu, l.gate_up), (288, 160, down, l.dn, l.down)):
            into[e], packed = drawn(rng, n, d, lo, hi, codes)
            blob[e].copy_(packed)
    l.x = bf16_bits(rng.normal(0, 1, (5, 288)) * x)
    return l


# gate and up exponents, down's, activations: sums and h stay normal fp32 numbers
@pytest.mark.parametrize("up,down,x", [((0, 0), (120, 127), 2.0 ** 120), ((0, 2), (120, 127), 2.0 ** 120),
                                       ((100, 102), (0, 1), 2.0 ** 60), ((2, 2), (120, 127), 2.0 ** 120), ((252, 252), (27, 30), 2.0 ** -90),
                                       ((247, 252), (20, 27), 2.0 ** -90), ((126, 128), (2, 3), 2.0 ** 50),
                                       ((100, 102), (252, 252), 2.0 ** 3), ((100, 102), (247, 252), 2.0 ** 3)])
@pytest.mark.parametrize("kind", [Layer, Half])
def test_exponents_to_252_are_exact(kind, up, down, x):
    say("exponents", kind.__name__, up, down, x)
    l = layer(kind, up, down, x, 4000 + up[0] + down[0])
    o = l.run()
    assert np.all(np.isfinite(as_f64(o["out"]))) and np.all(as_f64(o["out"]).any(1))
    l.check(o)


# the codes whose values bf16 holds; the least that it does not
@pytest.mark.parametrize("e,most,over", [(253, 5, 6), (254, 3, 4)])
def test_the_largest_exponents(e, most, over):
    """Exact while no value is 2^128 or more; one that is makes its outputs infinite or NaN."""
    for up, down, x in (((e, e), (27, 30), 2.0 ** -90), ((100, 102), (e, e), 2.0 ** 3)):
        l = layer(Layer, up, down, x, 4100 + e, range(most + 1))
        o = l.run()
        assert np.all(np.isfinite(as_f64(o["out"])))
        l.check(o)
    l = layer(Layer, (100, 102), (e, e), 2.0 ** 3, 4200 + e, [over])
    assert not np.any(np.isfinite(as_f64(l.run()["out"])))
