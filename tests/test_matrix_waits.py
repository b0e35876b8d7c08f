"""In the built library no vector operation and no load writes a register of a matrix instruction's
result before the instruction has: where a kernel reads one register of a result, the others are free for
the compiler, but not until its wait states have passed (an operation that reads the result waits for
it anyway). On the CPU, from the library's own listing."""
import os
import re
import shutil
import subprocess

import pytest

import bit_quantized_moe_dequant_amd as mq

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
REGS = re.compile(r"([va])(?:\[(\d+):(\d+)\]|(\d+)\b)")


def registers(operand):
    m = REGS.match(operand.strip())
    if not m:
        return frozenset()
    a, b = (int(m[2]), int(m[3])) if m[2] else (int(m[4]), int(m[4]))
    return frozenset(f"{m[1]}{i}" for i in range(a, b + 1))


def states(op):
    """Wait states behind a matrix instruction: four passes and more."""
    return 12 if "16x16x128" in op or "32x32" in op else 8


def early_writes(lines):
    """(matrix instruction, writer, states between) of a listing's instructions in order."""
    found = []
    for i, line in enumerate(lines):
        if not line.startswith("v_mfma"):
            continue
        op, args = line.split(None, 1)
        result, need, passed = registers(args.split(",")[0]), states(op), 0
        for other in lines[i + 1:i + 1 + need]:
            name, _, rest = other.partition(" ")
            if passed >= need or name in ("s_endpgm", "s_branch", "s_setpc_b64"):
                break
            if name.startswith(("v_", "ds_read", "global_load", "buffer_load", "scratch_load")) and not name.startswith("v_cmp"):
                first, *others = rest.split(",")
                if any(registers(o) & result for o in others):
                    break  # reads the result
                if registers(first) & result:
                    if not name.startswith("v_mfma"):
                        found.append((line, other, passed))
                    break
            m = re.match(r"s_nop (\d+)", other)
            passed += int(m[1]) + 1 if m else 1
    return found


def test_the_search_finds_an_early_write():
    mfma = "v_mfma_f32_16x16x32_bf16 v[4:7], v[0:3], v[8:11], 0"
    bad = [mfma, "s_nop 2", "v_add_u32_e32 v5, v20, v21", "v_mov_b32_e32 v30, v4"]
    assert [f[2] for f in early_writes(bad)] == [3]
    assert early_writes([mfma, "s_nop 7", *bad[2:]]) == []
    assert early_writes([mfma, "v_add_f32_e32 v5, v5, v6"]) == []  # reads it: waits for it
    assert early_writes([mfma, "v_add_f32_e32 v30, v31, v32", "global_load_dwordx4 v[6:9], v[40:41], off"]) != []
    assert early_writes([mfma, "s_endpgm", "v_mov_b32_e32 v5, 0"]) == []


@pytest.mark.skipif(not os.path.exists(mq.library_path()) or not os.path.exists(OBJDUMP), reason="no library, or no llvm-objdump")
def test_no_result_is_overwritten_before_it_is_there(tmp_path):
    lib = shutil.copy(mq.library_path(), tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True, cwd=tmp_path)
    parts = sorted(p for p in os.listdir(tmp_path) if "gfx950" in p)
    assert parts
    seen, found = 0, []
    for part in parts:
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", part], check=True, capture_output=True, text=True, cwd=tmp_path).stdout
        for body in re.split(r"^[0-9a-f]+ <.*>:$", text, flags=re.M):
            if "v_mfma" in body:
                lines = [line.split("//")[0].strip() for line in body.splitlines()]
                lines = [line for line in lines if line]
                seen += sum(line.startswith("v_mfma") for line in lines)
                found += early_writes(lines)
    assert seen > 1000
    assert found == []
