"""Host checks of the block-scaled e4m3 path's address functions (CPU only:
g++ compiles tests/fp8_host_driver.cpp against the ROCm headers)."""
import os
import shutil
import subprocess

import pytest

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

    def run(*args):
        r = subprocess.run([str(exe), *map(str, args)], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
        return r.stdout
    return run


def test_no_wave_reads_past_the_weight_scales(driver):
    driver("scale_rows")


def test_few_row_copies_stay_inside_their_buffers(driver):
    driver("rows_copies")
