"""Wait states of the copies to LDS, which are inline asm, in the generated gfx950 code
(CPU only).  The compiler inserts them for its own instructions: one between a write
of m0 and a copy to LDS, five between a vector instruction that writes a scalar
register and a vector-memory instruction that reads it."""
import re

import pytest

import test_build

SOURCES = ["qmm_gemm.hip", "qmm_mrow.hip", "qmm_fp8_rows.hip", "qmm_fp8_tile.hip"]


def scalars(op):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", op)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.fullmatch(r"s(\d+)", op)
    return {int(m.group(1))} if m else set()


def functions(text):
    """Instructions (operands, in asm, text) and labels of every function, in order."""
    out, name, inside = {}, None, False
    for line in text.splitlines():
        code = line.split(";")[0].strip()
        if "ASMSTART" in line or "ASMEND" in line:
            inside = "ASMSTART" in line
            continue
        if not code or (code.startswith(".") and not code.endswith(":")):
            continue
        if code.endswith(":"):
            if code.startswith(".L"):
                out.setdefault(name, []).append(code[:-1])
            else:
                name = code[:-1]
            continue
        out.setdefault(name, []).append(([o for o in re.split(r"[\s,]+", code) if o], inside, code))
    return out


def straight(items):
    """(copies seen, violations) of instructions one after the other."""
    clock, m0, written, copies, bad = 0, None, {}, 0, []
    for item in items:
        if isinstance(item, str):
            continue
        ops, inside, code = item
        clock += int(ops[1]) + 1 if ops[0] == "s_nop" else 1
        if inside and ops[0].startswith("buffer_load") and ops[-1] == "lds":
            copies += 1
            if m0 is not None and clock - m0 - 1 < 1:
                bad.append(("m0", clock - m0 - 1, code))
            for op in ops[2:]:
                bad += [("scalar", clock - written[r] - 1, code) for r in scalars(op)
                        if r in written and clock - written[r] - 1 < 5]
        if len(ops) > 1 and ops[1] == "m0":
            m0 = clock
        if len(ops) > 1 and ops[0].startswith(("v_readlane", "v_readfirstlane", "v_cmp")):
            for r in scalars(ops[1]):
                written[r] = clock
        elif len(ops) > 1 and ops[0].startswith("s_"):
            for r in scalars(ops[1]):
                written.pop(r, None)
    return copies, bad


def check(text):
    """The same over every function, and over what each branch back joins."""
    copies, bad = 0, []
    for items in functions(text).values():
        n, b = straight(items)
        copies, bad = copies + n, bad + b
        labels = {x: i for i, x in enumerate(items) if isinstance(x, str)}
        for i, item in enumerate(items):
            if not isinstance(item, str) and item[0][0].startswith(("s_cbranch", "s_branch")) and item[0][1] in labels:
                at = labels[item[0][1]]
                bad += straight(items[max(0, i - 12):i + 1] + items[at:at + 12])[1]
    return copies, bad


@pytest.mark.slow
@pytest.mark.parametrize("src", SOURCES)
def test_copies_have_their_wait_states(tmp_path, src):
    copies, bad = check(test_build.device_asm(tmp_path, src).read_text())
    assert copies > 0, "no copies to LDS found: the check would be vacuous"
    assert not bad, (len(bad), bad[:5])


COPY = ";;#ASMSTART\n\t{}buffer_load_dwordx4 v0, s[4:7], 0 offen lds\n;;#ASMEND\n"


@pytest.mark.parametrize("text,kinds", [
    ("f:\n\ts_mov_b32 m0, s2\n" + COPY.format(""), ["m0"]),
    ("f:\n\ts_mov_b32 m0, s2\n" + COPY.format("s_nop 0\n\t"), []),
    ("f:\n\tv_readlane_b32 s6, v9, 1\n\ts_nop 3\n" + COPY.format(""), ["scalar"]),
    ("f:\n\tv_readlane_b32 s6, v9, 1\n\ts_nop 3\n" + COPY.format("s_nop 0\n\t"), []),
    ("f:\n\tv_readfirstlane_b32 s6, v9\n\ts_mov_b32 s6, 0\n" + COPY.format(""), []),
    ("f:\n.LBB0:\n" + COPY.format("") + "\ts_mov_b32 m0, s2\n\ts_cbranch_scc1 .LBB0\n", []),
    ("f:\n.LBB0:\n" + COPY.format("") + "\tv_readlane_b32 s6, v9, 1\n\ts_cbranch_scc1 .LBB0\n", ["scalar"]),
])
def test_the_check_sees_short_distances(text, kinds):
    assert [k for k, _, _ in check(text)[1]] == kinds
