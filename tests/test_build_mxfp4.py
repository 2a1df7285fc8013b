"""The generated-code checks on the sources of the microscaled 4-bit path (CPU only)."""
import re

import pytest

import test_build
import test_build_copy_waits

SOURCES = ["qmm_mx4_quant.hip", "qmm_mx4_rows.hip", "qmm_mx4_tile.hip", "qmm_moe_layer.hip"]
COPIES = ["qmm_mx4_rows.hip", "qmm_mx4_tile.hip", "qmm_moe_layer.hip"]


@pytest.mark.slow
@pytest.mark.parametrize("src", SOURCES)
def test_no_packed_fp32_and_no_scratch(tmp_path, src):
    text = test_build.device_asm(tmp_path, src).read_text()
    assert not re.search(r"v_pk_(fma|mul|add)_f32", text)
    for key in (".vgpr_spill_count", ".private_segment_fixed_size"):
        got = re.findall(re.escape(key) + r":\s*(\d+)", text)
        assert got and set(got) == {"0"}, key


@pytest.mark.slow
@pytest.mark.parametrize("src", COPIES)
def test_copies_own_m0_and_have_their_wait_states(tmp_path, src):
    test_build.test_lds_copy_asm_owns_m0(tmp_path, src)
    test_build_copy_waits.test_copies_have_their_wait_states(tmp_path, src)


@pytest.mark.slow
@pytest.mark.parametrize("src", COPIES[:2])
def test_products_use_the_scaled_fp4_instruction(tmp_path, src):
    text = test_build.device_asm(tmp_path, src).read_text()
    ops = re.findall(r"v_mfma_\S+.*", text)
    assert ops and all("v_mfma_scale_f32_16x16x128_f8f6f4" in o and "cbsz:4 blgp:4" in o for o in ops)
