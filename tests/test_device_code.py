"""The library's own gfx950 code, read back: what its hand-written instructions
owe the hardware and the compiler does not see to."""
import glob
import os
import re
import shutil
import subprocess

import pytest

from second_order_optimizer_amd import build as B

OBJDUMP = os.path.join(os.path.dirname(os.path.realpath(B.HIPCC)), "..", "llvm", "bin", "llvm-objdump")
OBJDUMP = OBJDUMP if os.path.exists(OBJDUMP) else "/opt/rocm/llvm/bin/llvm-objdump"
MEMORY = re.compile(r"(global|buffer|flat|scratch)_")
SCALARS = re.compile(r"\bs(?:\[(\d+):(\d+)\]|(\d+)\b)|\bvcc\b")
WAIT_STATES = 5      # from a vector instruction's write of a scalar register to a memory instruction's read of it


def kernels(text):
    """(name, [instruction, ...]) of a disassembly."""
    name, body = None, []
    for line in text.splitlines():
        head = re.match(r"[0-9a-f]+ <(.+)>:$", line)
        if head:
            if body:
                yield name, body
            name, body = head.group(1), []
        elif line.startswith("\t") and name:
            body.append(line.split("//")[0].strip())
    if body:
        yield name, body


def scalars(operands):
    found = set()
    for low, high, one in SCALARS.findall(operands):
        found |= {"vcc"} if not (low or one) else set(range(int(low or one), int(high or one) + 1))
    return found


def written(instruction):
    """Scalar registers that a vector instruction writes: its first operand, and
    the carry or flag behind it where an instruction has one."""
    op, _, operands = instruction.partition(" ")
    if not op.startswith("v_"):
        return set()
    parts = re.split(r",\s*(?![^\[]*\])", operands)
    return scalars(parts[0]) | (scalars(parts[1]) if "_co_" in op or "div_scale" in op else set())


def too_near(body):
    """Memory instructions within five wait states of a vector instruction that
    writes a scalar register of theirs."""
    bad = []
    for i, ins in enumerate(body):
        if not MEMORY.match(ins):
            continue
        used, states = scalars(ins.partition(" ")[2]), 0
        for back in range(i - 1, -1, -1):
            if states >= WAIT_STATES or not used:
                break
            if written(body[back]) & used:
                bad.append(f"{states} states: {body[back]} | {ins}")
                break
            wait = re.match(r"s_nop (0x[0-9a-f]+|\d+)", body[back])
            states += int(wait.group(1), 0) + 1 if wait else 1
    return bad


def test_the_scan_itself():
    near = ["v_readfirstlane_b32 s1, v5", "s_mov_b32 m0, s7", "s_nop 0", "global_load_lds_dwordx4 v2, s[0:1]"]
    assert len(too_near(near)) == 1
    assert not too_near(near[:2] + ["s_nop 3"] + near[3:])
    assert len(too_near(near[:2] + ["s_nop 2"] + near[3:])) == 1
    assert not too_near(near[:3] + ["global_load_lds_dwordx4 v2, s[2:3]"])
    assert not too_near(near[:2] + ["s_mov_b64 s[8:9], s[0:1]", "global_load_lds_dwordx4 v2, s[8:9]"])      # a copy
    assert not too_near(["s_mov_b32 s1, s5"] + near[1:])
    assert len(too_near(["v_cmp_lt_i32_e64 s[0:1], v1, v2", "buffer_load_dword v1, v2, s[0:3], 0 offen"])) == 1
    assert not too_near(["v_add_f32 v0, s1, v2", "global_load_dword v1, v2, s[0:1]"])      # a read
    assert len(too_near(["v_add_co_u32_e64 v0, s[0:1], v1, v2", "global_load_dword v1, v2, s[0:1]"])) == 1


def disassembled(tmp_path):
    """(name, [instruction, ...]) of every kernel of the built library."""
    if not os.path.exists(B.LIB):
        B.build()
    lib = shutil.copy(B.LIB, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=tmp_path, check=True, capture_output=True)
    for part in glob.glob(str(tmp_path / "*gfx950")):
        yield from kernels(subprocess.run([OBJDUMP, "-d", part], check=True, capture_output=True, text=True).stdout)


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_memory_instructions_wait_for_scalar_bases(tmp_path):
    """A memory instruction that reads a scalar register which a vector
    instruction wrote needs five wait states between; the hardware does not wait,
    and the compiler does not look into inline assembly."""
    loads, bad = 0, {}
    for name, body in disassembled(tmp_path):
        loads += sum("load_lds" in ins for ins in body)
        near = too_near(body)
        if near:
            bad[name] = near
    assert loads > 100, "the loads into LDS are there"
    assert not bad, "\n".join(f"{k}: {len(v)}, e.g. {v[0]}" for k, v in bad.items())


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_loads_into_lds_have_m0_to_themselves(tmp_path):
    """Each sets m0 two instructions before it, and nothing else in its kernel
    uses m0."""
    loads = 0
    for name, body in disassembled(tmp_path):
        at = [i for i, ins in enumerate(body) if "load_lds" in ins]
        if at:
            loads += len(at)
            assert all(body[i - 2].startswith("s_mov_b32 m0, ") for i in at), name
            assert sum("m0" in ins for ins in body) == len(at), name
    assert loads > 100


def vectors(operands):
    """Vector registers (file, number) in operands."""
    found = set()
    for file, low, high, one in re.findall(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)", operands):
        found |= {(file, k) for k in range(int(low or one), int(high or one) + 1)}
    return found


def split(operands):
    return re.split(r",\s*(?![^\[]*\])", operands)


def products_unready(body):
    """What goes against hand-written matrix instructions whose hazards the
    compiler does not see: an operand that a vector instruction wrote less than
    two wait states before; an accumulator that anything else uses between the
    first product and the last; results used before 48 wait states behind it."""
    at = [i for i, ins in enumerate(body) if ins.startswith("v_mfma")]
    sums, bad = set(), []
    for i in at:
        parts = split(body[i].partition(" ")[2])
        sums |= vectors(parts[0])
        states, used = 0, set().union(*(vectors(p) for p in parts[1:]))
        for back in range(i - 1, -1, -1):
            if states >= 2:
                break
            op, _, operands = body[back].partition(" ")
            if op.startswith("v_") and not op.startswith("v_mfma") and vectors(split(operands)[0]) & used:
                bad.append(f"{states} states: {body[back]} | {body[i]}")
            wait = re.match(r"s_nop (0x[0-9a-f]+|\d+)", body[back])
            states += int(wait.group(1), 0) + 1 if wait else 1
    for ins in body[at[0]:at[-1]]:
        if not ins.startswith("v_mfma") and vectors(ins.partition(" ")[2]) & sums:
            bad.append(f"between the products: {ins}")
    states = 0
    for ins in body[at[-1] + 1:]:
        if states >= 48:
            break
        if vectors(ins.partition(" ")[2]) & sums:
            bad.append(f"{states} states behind the last product: {ins}")
        wait = re.match(r"s_nop (0x[0-9a-f]+|\d+)", ins)
        states += int(wait.group(1), 0) + 1 if wait else 1
    return bad


def test_the_scan_of_products_itself():
    product = "v_mfma_scale_f32_16x16x128_f8f6f4 a[0:3], v[8:15], v[16:23], a[0:3], v1, v2 op_sel_hi:[0,0,0]"
    wait = ["s_nop 15"] * 3
    assert not products_unready(["v_accvgpr_write_b32 a0, 0", "s_nop 1", product] + wait + ["ds_write_b128 v5, a[0:3]"])
    assert len(products_unready(["v_accvgpr_write_b32 a0, 0", "s_nop 0", product] + wait)) == 1
    assert len(products_unready(["v_mov_b32_e32 v2, v3", product] + wait)) == 1
    assert not products_unready(["v_mov_b32_e32 v3, v2", product] + wait)
    assert len(products_unready([product, "v_accvgpr_read_b32 v4, a3", product] + wait)) == 1
    assert len(products_unready([product] + wait[:2] + ["ds_write_b128 v5, a[0:3]"])) == 1


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_hand_written_products_wait(tmp_path):
    seen = 0
    for name, body in disassembled(tmp_path):
        if "k_mul8_big" in name:
            seen += 1
            bad = products_unready(body)
            assert not bad, f"{name}: {len(bad)}, e.g. {bad[0]}"
    assert seen == 4
