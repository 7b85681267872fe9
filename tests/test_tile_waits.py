"""The tiled products' matrix instructions are written as assembly, so the
compiler adds no waits around them.  This reads the library's own machine code
(as built here) and checks that nothing but another matrix instruction touches a
sum within the states that the longest of them takes, and that operands that a
vector instruction writes have two states before their use."""
import os
import re
import struct
import subprocess

import pytest

import gated_activation_amd as ga

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
STATES = 19      # result of a matrix instruction of 16 passes to its first reader (all here take 8 or fewer)
OPERAND = 2      # a vector instruction's result to a matrix instruction


def code_objects():
    data = open(ga.library_path, "rb").read()
    magic = b"__CLANG_OFFLOAD_BUNDLE__"
    at = data.find(magic)
    while at >= 0:
        n, = struct.unpack_from("<Q", data, at + 24)
        p = at + 32
        for _ in range(n):
            offset, size, length = struct.unpack_from("<QQQ", data, p)
            name = data[p + 24:p + 24 + length]
            p += 24 + length
            if b"gfx950" in name and size:
                yield data[at + offset:at + offset + size]
        at = data.find(magic, at + 1)


def registers(text):
    """Vector registers named in an operand list, by operand."""
    out = []
    for op in re.split(r",\s*(?![^\[]*\])", text):
        m = re.match(r"\s*(?:-|\|)?v\[(\d+):(\d+)\]", op) or re.match(r"\s*(?:-|\|)?v(\d+)\b", op)
        out.append(set() if m is None else set(range(int(m.group(1)), int(m.group(m.lastindex)) + 1)))
    return out


def parse(lines):
    """[(text, opcode, registers by operand, states, following instructions)] of objdump's lines of a kernel."""
    at, rows = {}, []
    for line in lines:
        code, _, tail = line.partition("//")
        parts = code.split(None, 1)
        if not parts:
            continue
        m = re.match(r"\s*([0-9A-Fa-f]+):", tail)
        target = re.search(r"<[^>+]*(?:\+0x([0-9a-f]+))?>", tail)
        if m:
            at[int(m.group(1), 16)] = len(rows)
        rows.append((code.strip(), parts[0], registers(parts[1]) if len(parts) > 1 else [],
                     int(m.group(1), 16) if m else None, int(target.group(1) or "0", 16) if target else None))
    start = rows[0][3] if rows else None
    out = []
    for i, (code, op, regs, _, target) in enumerate(rows):
        following = [] if op in ("s_branch", "s_endpgm", "s_setpc_b64") else [i + 1] if i + 1 < len(rows) else []
        if op.startswith(("s_branch", "s_cbranch")):
            following.append(at[start + target])
        out.append((code, op, regs, int(code.split()[1], 0) + 1 if op == "s_nop" else 1, following))
    return out


def reach(rows, i, most, touches):
    """An instruction that `touches` fewer than `most` states after the one at i, along any path."""
    todo, seen = [(j, 1) for j in rows[i][4]], {}
    while todo:
        j, states = todo.pop()
        if states >= most or seen.get(j, most) <= states:
            continue
        seen[j] = states
        if touches(rows[j]):
            return rows[j][0]
        todo += [(k, states + rows[j][3]) for k in rows[j][4]]
    return None


def hazards(lines):
    rows, found = parse(lines), []
    for i, (code, op, regs, _, _) in enumerate(rows):
        if op.startswith("v_mfma"):
            hit = reach(rows, i, STATES, lambda r: not r[1].startswith("v_mfma") and any(regs[0] & x for x in r[2]))
        elif op.startswith("v_") and regs and regs[0]:
            hit = reach(rows, i, OPERAND + 1, lambda r: r[1].startswith("v_mfma") and any(regs[0] & x for x in r[2][1:]))
        else:
            continue
        if hit:
            found.append(f"{code} -> {hit}")
    return found


def test_the_check_sees_a_read_that_comes_too_soon():
    mfma = "v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]"
    assert hazards([mfma, "s_nop 15", "v_add_f32_e32 v20, v1, v21"]) and not hazards([mfma, "s_nop 15", "s_nop 15", "v_add_f32_e32 v20, v1, v21"])
    assert hazards(["v_mov_b32_e32 v9, v30", mfma]) and not hazards(["v_mov_b32_e32 v9, v30", "s_nop 1", mfma])
    assert hazards([mfma, "v_mov_b32_e32 v2, 0"]) and not hazards([mfma, "v_mov_b32_e32 v20, 0"])


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="needs llvm-objdump")
def test_matrix_instructions_have_their_waits(tmp_path):
    kernels = products = 0
    for i, code in enumerate(code_objects()):
        if b"tile_kernel" not in code:
            continue
        path = tmp_path / f"{i}.co"
        path.write_bytes(code)
        text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", str(path)], capture_output=True, text=True, check=True).stdout
        for body in re.split(r"^[0-9a-f]+ <", text, flags=re.M)[1:]:
            name, _, rest = body.partition(">:\n")
            lines = [ln.strip() for ln in rest.splitlines()]
            if "tile_kernel" not in name:
                continue
            kernels += 1
            products += sum(ln.startswith("v_mfma") for ln in lines)
            bad = hazards(lines)
            assert not bad, f"{name}: {len(bad)}, first {bad[0]}"
    assert kernels > 20 and products > 1000
