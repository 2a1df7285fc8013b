"""examples/fp8_moe_block.py: the block-scaled operators as they are used together."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("fp8_moe_block", os.path.join(ROOT, "examples", "fp8_moe_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


# The block's own roundings against fp32: the activation's codes (a relative 2^-4 at most,
# uniform: 2^-4/sqrt(12) rms of the larger half, about 0.025 of the expert's output), the
# bf16 outputs (2^-9 each).  The residual dilutes them: |rms(out)| is about |r|.
@pytest.mark.parametrize("t, d, i, e, k, groups, keep", [(1, 256, 128, 8, 2, 1, 1), (5, 272, 176, 16, 4, 4, 2),
                                                         (130, 512, 384, 32, 6, 8, 4), (300, 1024, 256, 12, 3, 1, 1)])
def test_block_against_fp32(t, d, i, e, k, groups, keep):
    m = example()
    far = m.main(["--tokens", str(t), "--dim", str(d), "--inter", str(i), "--experts", str(e), "--top-k", str(k),
                  "--groups", str(groups), "--keep-groups", str(keep), "--repeat", "2"])
    assert far < 0.03


def test_block_in_a_graph():
    m = example()
    block = m.Fp8MoeBlock(64, 512, 256, 16, 4, 4, 2, scale=2.5)
    r = torch.randn(64, 512, device="cuda").bfloat16()
    eager = [x.clone() for x in block(r)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(r)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = block(r)
    for seed in range(4):
        r.copy_(torch.randn(64, 512, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).bfloat16())
        g.replay()
        torch.cuda.synchronize()
        replayed = [x.clone() for x in got]
        eager = [x.clone() for x in block(r)]
        torch.cuda.synchronize()
        for a, b in zip(replayed, eager):
            assert torch.equal(a, b)
