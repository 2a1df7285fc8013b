"""The generated-code checks of tests/test_build.py on every source of the
block-scaled e4m3 path: both files that copy to LDS by inline asm own m0, and no
kernel has packed fp32 instructions or vector registers in memory."""
import re

import pytest

import test_build


@pytest.mark.slow
@pytest.mark.parametrize("src", ["qmm_fp8_rows.hip", "qmm_fp8_tile.hip"])
def test_lds_copy_asm_owns_m0(tmp_path, src):
    test_build.test_lds_copy_asm_owns_m0(tmp_path, src)


@pytest.mark.slow
@pytest.mark.parametrize("src", ["qmm_fp8_quant.hip", "qmm_fp8_rows.hip", "qmm_fp8_tile.hip", "qmm_norm.hip", "qmm_topk.hip"])
def test_no_packed_fp32_and_no_scratch(tmp_path, src):
    text = test_build.device_asm(tmp_path, src).read_text()
    assert not re.search(r"v_pk_(fma|mul|add)_f32", text)
    for key in (".vgpr_spill_count", ".private_segment_fixed_size"):
        got = re.findall(re.escape(key) + r":\s*(\d+)", text)
        assert got and set(got) == {"0"}, key
