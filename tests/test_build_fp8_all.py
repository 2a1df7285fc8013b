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


def dpp_reads_of_asm(path):
    """(wait states between an inline-asm VALU result and a DPP read of it, line), in order."""
    inside, clock, written, out = False, 0, {}, []
    for line in path.read_text().splitlines():
        code = line.split(";")[0].strip()
        if "ASMSTART" in line or "ASMEND" in line:
            inside = "ASMSTART" in line
            continue
        if not code or code.startswith(".") or code.endswith(":"):
            if code.endswith(":") and not code.startswith(".L"):
                written = {}   # a new function
            continue
        ops = [o for o in re.split(r"[\s,]+", code) if o]
        clock += int(ops[1]) + 1 if ops[0] == "s_nop" else 1
        if re.search(r"_dpp\b|quad_perm|row_", code) and len(ops) > 2:
            out += [(clock - written[r] - 1, line.strip()) for r in test_build._vgprs(ops[2]) if r in written]
        if len(ops) > 1 and ops[0].startswith("v_"):
            for r in test_build._vgprs(ops[1]):
                if inside:
                    written[r] = clock
                else:
                    written.pop(r, None)
    return out


@pytest.mark.slow
def test_inline_asm_results_reach_dpp_after_two_wait_states(tmp_path):
    """A DPP read needs two wait states after the VALU write of its source, which the
    compiler inserts for its own instructions only: the router's 64-bit maxima are
    inline asm, and their results go to other lanes by DPP."""
    reads = dpp_reads_of_asm(test_build.device_asm(tmp_path, "qmm_topk.hip"))
    assert len(reads) >= 64, "no DPP reads of asm results found: the check would be vacuous"
    assert not [r for r in reads if r[0] < 2]


def test_the_dpp_check_sees_a_short_distance(tmp_path):
    text = "f:\n;;#ASMSTART\n\tv_max_f64 v[2:3], v[4:5], v[6:7]\n;;#ASMEND\n{}\tv_mov_b32_dpp v9, v3 quad_perm:[1,0,3,2]\n"
    for between, want in (("", 0), ("\ts_nop 0\n", 1), ("\ts_nop 1\n", 2), ("\tv_add_u32 v1, v1, v1\n\ts_nop 0\n", 2)):
        path = tmp_path / "a.s"
        path.write_text(text.format(between))
        assert [d for d, _ in dpp_reads_of_asm(path)] == [want]
