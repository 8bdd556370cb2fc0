"""Wait states around the operand loads that are written as inline assembly (no GPU needed).

gfx9 hardware needs five wait states between a vector instruction that writes a scalar register and
a buffer load that reads it.  The compiler counts them for its own instructions, not for those of
an assembly statement.  The assembly that hipcc makes of this library's kernels is searched for
buffer loads into LDS that come too soon.
"""
import os
import re
import subprocess

import pytest

from conftest import ROOT

import adamw_optimizer_step_muon_amd.build as _build

CSRC = os.path.join(ROOT, "adamw_optimizer_step_muon_amd", "csrc")
WAITS = 5


def _registers(operand):
    m = re.match(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return range(int(m[1]), int(m[2]) + 1)
    m = re.match(r"s(\d+)$", operand)
    return [int(m[1])] if m else ["m0"] if operand == "m0" else []


def _too_soon(lines):
    """(loads seen, [(function, writer, wait states, load)]) of a listing."""
    found, loads, function, written, at = [], 0, None, {}, 0
    for line in lines:
        m = re.match(r"^(\w+):", line)
        if m:
            function, written, at = m[1], {}, 0
        text = line.split(";")[0].strip()
        if not text or text[0] == "." or text.endswith(":"):
            continue
        op = text.split()[0]
        operands = [x.strip().split()[0] for x in text[len(op):].split(",") if x.strip()]
        at += 1
        if op == "s_nop":
            at += int(operands[0], 0)
        elif op.startswith("buffer_load") and text.endswith("lds"):
            loads += 1
            for r in [r for x in operands for r in _registers(x)] + ["m0"]:
                if r in written and at - written[r][0] - 1 < WAITS:
                    found.append((function, written[r][1], at - written[r][0] - 1, text))
        elif op.startswith("v_") and operands:
            for r in _registers(operands[0]):
                written[r] = (at, text)
        elif op.startswith("s_") and operands:
            for r in _registers(operands[0]):
                written.pop(r, None)
    return loads, found


def test_a_short_wait_is_found():
    text = ["kernel:", "  v_readfirstlane_b32 s4, v1", "  s_mov_b32 s7, 0", "  s_nop 0",
            "  buffer_load_dwordx4 v2, s[4:7], 0 offen lds"]
    assert _too_soon(text)[1] and not _too_soon(text[:3] + ["  s_nop 4"] + text[4:])[1]


@pytest.mark.parametrize("source", ["head_loss.hip", "ns_gemm.hip"])
def test_loads_wait(source, tmp_path):
    if not os.path.exists(_build.HIPCC):
        pytest.skip("no hipcc")
    out = tmp_path / "listing.s"
    subprocess.run([_build.HIPCC, *_build.CFLAGS, "--cuda-device-only", "-S", os.path.join(CSRC, source), "-o", str(out)],
                   check=True, capture_output=True)
    loads, found = _too_soon(out.read_text().splitlines())
    assert loads > 50 and not found, found[:3]
