"""The choice of kernels of the microscaled 4-bit path (CPU only: g++ compiles
tests/mxfp4_host_driver.cpp against the ROCm headers)."""
import os
import shutil
import subprocess

import pytest

import mxfp4_shapes as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    gxx, inc = shutil.which("g++"), "/opt/rocm/include"
    if not gxx or not os.path.isdir(inc):
        pytest.skip("g++ or the ROCm headers are not available")
    exe = tmp_path_factory.mktemp("mxfp4_host") / "driver"
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", f"-I{inc}",
                        f"-I{os.path.join(ROOT, 'bit_weight_quantized_amd', 'csrc')}",
                        os.path.join(ROOT, "tests", "mxfp4_host_driver.cpp"), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]

    def run(lines):
        r = subprocess.run([str(exe)], input="\n".join(lines) + "\n", capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr[-2000:]
        out = r.stdout.splitlines()
        assert len(out) == len(lines)
        return out
    return run


def test_every_dense_kernel_has_a_shape(ask):
    assert ask([f"dense {t} {n} {d}" for t, n, d in S.DENSE_ROWS.values()]) == [f"rows {r} {x} {w}" for r, x, w in S.DENSE_ROWS]
    assert set(ask([f"dense {t} {n} {d}" for t, n, d in S.DENSE_64])) == {"tile 64"}
    assert set(ask([f"dense {t} {n} {d}" for t, n, d in S.DENSE_256])) == {"tile 256"}
    lines = [f"dense {t} {n} {d}" for t in (1, 8, 9, 16, 17, 32, 33, 48, 49, 60, 64, 65, 100, 200, 600)
             for n in (1, 300, 1030, 2000, 2570, 4100, 5130, 8200, 10200, 13824, 40000) for d in (32, 288, 1056, 4096, 8192)]
    reached = {x for x in ask(lines) if x.startswith("rows")}
    assert reached == {f"rows {r} {x} {w}" for r, x, w in S.DENSE_ROWS}, "the variants that the source compiles"


def test_every_grouped_kernel_has_a_shape(ask):
    def line(n, d, lengths, glu):
        return f"grouped {n} {d} {len(lengths)} {sum(lengths)} {max(lengths)} {int(glu)}"
    got = ask([line(*s, g) for (_, _, g), s in S.GROUPED_ROWS.items()])
    assert got == [f"rows {x} {w}" for x, w, _ in S.GROUPED_ROWS]
    for glu in (False, True):
        assert set(ask([line(*s, glu) for s in S.GROUPED_64])) == {"tile 64"}
        assert set(ask([line(*s, glu) for s in S.GROUPED_256])) == {"tile 256"}


def test_few_rows_of_one_round(ask):
    """Weight rows a workgroup so that its workgroups are one round of 256 CUs where they can be."""
    want = {(1, 4096, 4096): "rows 1 1 4", (1, 5120, 13824): "rows 2 1 4", (1, 13824, 5120): "rows 4 1 4",
            (47, 5120, 13824): "rows 2 6 4", (64, 4096, 7168): "rows 2 4 4"}
    assert ask([f"dense {t} {n} {d}" for t, n, d in want]) == list(want.values())
