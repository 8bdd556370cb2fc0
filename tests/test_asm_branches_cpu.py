"""Wait states around the operand loads written as inline assembly, along every path (no GPU needed).

gfx9 hardware needs five wait states between a vector instruction that writes a scalar register and
a buffer load that reads it; the compiler counts none for an assembly statement.  Each listing of
hipcc is taken as a graph of basic blocks: the wait states since a register was last written by
a vector instruction are carried along fall-through and branch edges, loops included, with the least of
all paths at a label, until nothing changes.
"""
import os
import re
import subprocess

import pytest

from conftest import ROOT

import adamw_optimizer_step_muon_amd.build as _build

CSRC = os.path.join(ROOT, "adamw_optimizer_step_muon_amd", "csrc")
WAITS = 5
# scalar instructions whose first operand is read, or is no register
READS_FIRST = re.compile(r"s_(cmp|cmpk|bitcmp|cbranch|branch|waitcnt|nop|barrier|endpgm|setprio|sleep|setreg|set_gpr_idx|"
                         r"setpc|sendmsg|store|buffer_store|dcache|icache|trap|sethalt|code_end)")


def _registers(operand):
    m = re.match(r"s\[(\d+):(\d+)\]$", operand)
    if m:
        return list(range(int(m[1]), int(m[2]) + 1))
    m = re.match(r"s(\d+)$", operand)
    if m:
        return [int(m[1])]
    return {"vcc": ["vcc_lo", "vcc_hi"], "m0": ["m0"], "vcc_lo": ["vcc_lo"], "vcc_hi": ["vcc_hi"]}.get(operand, [])


def _functions(lines):
    """(name, [(label or None, instruction, operands, text)]) of each function: labels stand alone."""
    out, name, body = [], None, []
    for line in lines:
        text = line.split(";")[0].strip()
        m = re.match(r"^([\w.$]+):", text)
        if m:
            if m[1].startswith(".L"):
                body.append((m[1], None, [], text))
            else:
                if body:
                    out.append((name, body))
                name, body = m[1], []
            text = text[m.end():].strip()
        if not text or text[0] == ".":
            continue
        op = text.split()[0]
        body.append((None, op, [x.strip().split()[0] for x in text[len(op):].split(",") if x.strip()], text))
    if body:
        out.append((name, body))
    return out


def _blocks(body):
    """Basic blocks, and each one's successors."""
    blocks, label_of = [[]], {}
    for label, op, operands, text in body:
        if label is not None:
            if blocks[-1]:
                blocks.append([])
            label_of[label] = len(blocks) - 1
            continue
        blocks[-1].append((op, operands, text))
        if op.startswith(("s_branch", "s_cbranch", "s_endpgm", "s_setpc")):
            blocks.append([])
    after = []
    for i, b in enumerate(blocks):
        last = b[-1] if b else ("", [], "")
        to = []
        if last[0].startswith(("s_branch", "s_cbranch")):
            to.append(label_of[last[1][0]])
        if not last[0].startswith(("s_branch", "s_endpgm", "s_setpc")) and i + 1 < len(blocks):
            to.append(i + 1)
        after.append(to)
    return blocks, after


def _run(block, state, found=None):
    """The state {register: (wait states since its write, the writer)} behind a block; loads that
    come too soon are appended to `found`."""
    state, loads = dict(state), 0
    for op, operands, text in block:
        if op.startswith("buffer_load") and text.endswith("lds"):
            loads += 1
            if found is not None:
                for r in [r for x in operands for r in _registers(x)] + ["m0"]:
                    if r in state:
                        found.append((state[r][1], state[r][0], text))
        waits = 1 + (int(operands[0], 0) if op == "s_nop" else 0)
        state = {r: (w + waits, by) for r, (w, by) in state.items() if w + waits < WAITS}
        if op.startswith("v_"):
            # (the second operand is a carry, or a condition that is written as well)
            for r in [r for x in operands[:2 if "_co_" in op or op.startswith("v_div_scale") else 1] for r in _registers(x)]:
                state[r] = (0, text)
        elif op.startswith("s_") and operands and not READS_FIRST.match(op):
            for r in _registers(operands[0]):
                state.pop(r, None)
    return state, loads


def _too_soon(lines):
    """(loads seen, [(function, writer, wait states, load)]) of a listing, over all paths."""
    loads, found = 0, []
    for name, body in _functions(lines):
        blocks, after = _blocks(body)
        before = [None] * len(blocks)
        before[0] = {}
        work = [0]
        while work:
            i = work.pop()
            state, _ = _run(blocks[i], before[i])
            for j in after[i]:
                joined = dict(before[j]) if before[j] is not None else {}
                for r, (w, by) in state.items():
                    if r not in joined or w < joined[r][0]:
                        joined[r] = (w, by)
                if before[j] is None or joined != before[j]:
                    before[j] = joined
                    work.append(j)
        for i, b in enumerate(blocks):
            here = []
            loads += _run(b, before[i] or {}, here)[1]
            found += [(name, *x) for x in here]
    return loads, found


LOAD = "  buffer_load_dwordx4 v2, s[4:7], 0 offen lds"
WRITE = "  v_readfirstlane_b32 s4, v1"


@pytest.mark.parametrize("lines,bad", [
    ([WRITE, "  s_nop 3", LOAD], True),
    ([WRITE, "  s_nop 4", LOAD], False),
    # behind the back edge of a loop
    ([".LBB0_1:", "  s_nop 0", LOAD, "  s_nop 7", WRITE, "  s_cbranch_scc1 .LBB0_1", "  s_endpgm"], True),
    ([".LBB0_1:", "  s_nop 4", LOAD, "  s_nop 7", WRITE, "  s_cbranch_scc1 .LBB0_1", "  s_endpgm"], False),
    # a scalar write on one path does not clear the other's
    ([WRITE, "  s_cbranch_scc1 .LBB0_2", "  s_mov_b32 s4, 0", ".LBB0_2:", LOAD], True),
    ([WRITE, "  s_mov_b32 s4, 0", ".LBB0_2:", LOAD], False),
    # a branch over the block in between; nothing passes behind the program's end or a jump
    ([WRITE, "  s_branch .LBB0_3", ".LBB0_2:", "  s_nop 7", ".LBB0_3:", LOAD], True),
    ([".LBB0_1:", "  s_branch .LBB0_3", WRITE, "  s_endpgm", ".LBB0_3:", LOAD], False),
    # comparisons read their first operand; carries are written
    ([WRITE, "  s_cmp_eq_u32 s4, 0", LOAD], True),
    (["  v_add_co_u32_e64 v1, s[6:7], v2, v3", LOAD], True),
    (["  v_add_u32_e32 v1, s4, v3", LOAD], False),
    (["  v_readfirstlane_b32 s9, v1", "  v_readfirstlane_b32 m0, v1", LOAD], True),
])
def test_paths(lines, bad):
    loads, found = _too_soon(["kernel:", *lines])
    assert loads == 1 and bool(found) == bad, found


@pytest.mark.parametrize("source", ["head_loss.hip", "ns_gemm.hip"])
def test_loads_wait_on_every_path(source, tmp_path):
    if not os.path.exists(_build.HIPCC):
        pytest.skip("no hipcc")
    out = tmp_path / "listing.s"
    subprocess.run([_build.HIPCC, *_build.CFLAGS, "--cuda-device-only", "-S", os.path.join(CSRC, source), "-o", str(out)],
                   check=True, capture_output=True)
    loads, found = _too_soon(out.read_text().splitlines())
    assert loads > 50 and not found, found[:3]
