"""Host checks of the block-scaled e4m3 path's address functions and of its choice of
kernels (CPU only: g++ compiles tests/fp8_host_driver.cpp against the ROCm headers)."""
import os
import shutil
import subprocess

import pytest

import fp8_shapes as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    gxx, inc = shutil.which("g++"), "/opt/rocm/include"
    if not gxx or not os.path.isdir(inc):
        pytest.skip("g++ or the ROCm headers are not available")
    exe = tmp_path_factory.mktemp("fp8_host") / "driver"
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", f"-I{inc}",
                        f"-I{os.path.join(ROOT, 'bit_weight_quantized_amd', 'csrc')}",
                        os.path.join(ROOT, "tests", "fp8_host_driver.cpp"), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]

    def run(*args, text=""):
        r = subprocess.run([str(exe), *map(str, args)], input=text, capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
        return r.stdout
    return run


def test_no_wave_reads_past_the_weight_scales(driver):
    driver("scale_rows")


def test_few_row_copies_stay_inside_their_buffers(driver):
    driver("rows_copies")


def ask(driver, lines):
    out = driver("kernels", text="\n".join(lines) + "\n").splitlines()
    assert len(out) == len(lines)
    return out


def test_every_product_kernel_has_a_shape(driver):
    """The shapes that the GPU tests run for each kernel still choose it, and the
    few-row variants are all those that the source compiles."""
    got = ask(driver, [f"dense {t} {n} {d}" for t, n, d in S.DENSE_ROWS.values()])
    assert got == [f"rows {w} {r} {x}" for w, r, x in S.DENSE_ROWS]
    assert set(ask(driver, [f"dense {t} {n} {d}" for t, n, d in S.DENSE_64])) == {"tile 64"}
    assert set(ask(driver, [f"dense {t} {n} {d}" for t, n, d in S.DENSE_256])) == {"tile 256"}

    def grouped(n, d, lengths):
        return f"grouped {n} {d} {len(lengths)} {sum(lengths)} {max(lengths)}"
    assert ask(driver, [grouped(*s) for s in S.GROUPED_ROWS.values()]) == [f"rows {w} {r} {x}" for w, r, x in S.GROUPED_ROWS]
    assert set(ask(driver, [grouped(*s) for s in S.GROUPED_64])) == {"tile 64"}
    assert set(ask(driver, [grouped(*s) for s in S.GROUPED_256])) == {"tile 256"}
    # every variant that any number of rows and columns can reach
    lines = [f"dense {t} {n} {d}" for t in (1, 8, 9, 16, 17, 32, 33, 64, 65, 100, 200, 600)
             for n in (1, 300, 2570, 5130, 10200, 40000) for d in (16, 272, 1040, 2064, 8192)]
    reached = {x for x in ask(driver, lines) if x.startswith("rows")}
    assert reached == {f"rows {w} {r} {x}" for w, r, x in S.DENSE_ROWS}


def test_every_norm_kernel_has_a_shape(driver):
    got = ask(driver, [f"norm {t} {d}" for t, d in S.NORMS.values()])
    assert got == [f"norm {w} {g}" for w, g in S.NORMS]
    reached = set(ask(driver, [f"norm {t} {d}" for t in (1, 256, 257, 9000) for d in range(8, 65537, 8 * 61)]))
    assert reached == set(got)


def test_few_row_kernel_fills_the_compute_units_once(driver):
    """Fewer weight rows a workgroup are taken to fill 256 CUs, never where that makes
    a second round of them."""
    want = {(64, 4096, 7168): "rows 4 1 8", (64, 4097, 7168): "rows 4 2 8", (64, 5119, 7168): "rows 4 2 8",
            (33, 8192, 4096): "rows 4 2 8", (33, 8193, 4096): "rows 4 4 8", (1, 4224, 13824): "rows 4 2 1",
            (32, 4608, 4096): "rows 4 2 4"}
    assert ask(driver, [f"dense {t} {n} {d}" for t, n, d in want]) == list(want.values())
    sizes = [(t, n) for t in (1, 9, 17, 33, 64) for n in range(16, 12000, 48)]
    for (t, n), got in zip(sizes, ask(driver, [f"dense {t} {n} 1024" for t, n in sizes])):
        waves, r, x8 = map(int, got.split()[1:])
        if r < (4 if t > 16 else 2):
            assert -(-n // (16 * r)) * -(-t // (8 * x8)) <= 256, (t, n, got)


def test_eight_waves_are_one_round(driver):
    """Eight waves take 32 rows a pass: 33 .. 64 rows are two passes, which count."""
    want = {(64, 2048, 7168): "rows 8 1 4", (64, 2049, 7168): "rows 4 1 8", (33, 2304, 2048): "rows 4 1 8",
            (64, 2560, 4096): "rows 4 1 8", (32, 2560, 4096): "rows 8 1 4", (1, 4096, 7168): "rows 8 1 1"}
    assert ask(driver, [f"dense {t} {n} {d}" for t, n, d in want]) == list(want.values())
    sizes = [(t, n) for t in (1, 16, 32, 33, 64, 81, 300, 943) for n in range(16, 4200, 48)]
    for (t, n), got in zip(sizes, ask(driver, [f"dense {t} {n} 7168" for t, n in sizes])):
        if got.startswith("rows 8"):
            assert -(-n // 16) * -(-t // (8 * int(got.split()[3]))) <= 256, (t, n, got)
