"""The generated-code checks of tests/test_build.py on the block-scaled e4m3
tile kernel, which uses the same global -> LDS copies."""
import pytest

import test_build


@pytest.mark.slow
def test_lds_copy_asm_owns_m0(tmp_path):
    test_build.test_lds_copy_asm_owns_m0(tmp_path, "qmm_fp8_tile.hip")


@pytest.mark.slow
def test_no_packed_fp32_and_no_spills(tmp_path):
    text = test_build.device_asm(tmp_path, "qmm_fp8_tile.hip").read_text()
    assert "v_mfma_f32_16x16x128_f8f6f4" in text and "v_mfma_scale" not in text
    assert "v_pk_fma_f32" not in text and "v_pk_mul_f32" not in text and "v_pk_add_f32" not in text
    assert all(line.split(":")[1].strip() == "0" for line in text.splitlines() if ".vgpr_spill_count" in line)
