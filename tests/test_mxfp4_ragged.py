"""Which kernel a ragged SwiGLU call gets (CPU only)."""
from mxfp4_ragged_shapes import RAGGED
from test_mxfp4_host import ask  # noqa: F401


def test_every_kernel_has_a_ragged_shape(ask):  # noqa: F811
    lines = [f"grouped {n} {d} {len(lengths)} {sum(lengths)} {max(lengths)} 1" for _, (n, d, lengths) in RAGGED]
    assert ask(lines) == [kernel for kernel, _ in RAGGED]
