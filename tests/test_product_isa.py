"""Checks on the compiled gfx950 code of the layer operators' kernels (CPU only: hipcc -S).

The tiled product shares the GEMM's main loop, whose MFMAs are assembly statements that the compiler neither schedules nor
guards: the same properties are checked as for the plain GEMM, in its four forms and both tile edges.
"""

import os
import re
import subprocess

import pytest

from tests import test_kernel_isa as isa

pytestmark = isa.pytestmark

FORMS = {0: "NT", 1: "NN", 2: "TN", 3: "NT e4m3"}
CASES = [(edge, form, mode) for edge in (256, 128) for form in FORMS for mode in (2, 0)]  # dynamic, non-persistent


def compile_to_asm(tmp, source):
    out = tmp / (source + ".s")
    cmd = [isa.HIPCC if os.path.exists(isa.HIPCC) else "hipcc", "--offload-arch=gfx950", "-O3", "-std=c++17",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", os.path.join(isa.REPO, "include"), "-I", isa.CSRC,
           "--cuda-device-only", "-S", "-o", str(out), os.path.join(isa.CSRC, source)]
    subprocess.run(cmd, check=True, capture_output=True)
    return out.read_text()


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    return compile_to_asm(tmp_path_factory.mktemp("isa"), "product_kernel.hip")


def kernel_text(asm_text, edge, form, mode):
    i = asm_text.index(f"\n_ZN3ptg18ptg_product_kernelILi{edge}ELi{form}ELi{mode}EEE")
    i = asm_text.index(":", i)
    return asm_text[i:asm_text.index(".Lfunc_end", i)]


def loops(text):
    blocks = [isa.instructions(b) for b in re.split(r"\n\.LBB\d+_\d+:", text)]
    return [b for b in blocks if sum(x.startswith("v_mfma") for x in b) > 0]


@pytest.mark.parametrize("edge,form,mode", CASES)
def test_main_loop_is_one_block_without_copies(asm, edge, form, mode):
    step = (64 if edge == 256 else 16) * (2 if form == 3 else 1)  # MFMAs a k-step
    bodies = loops(kernel_text(asm, edge, form, mode))
    counts = [sum(x.startswith("v_mfma") for x in b) for b in bodies]
    # four-step and two-step trips (e4m3: the two-step ones are the K tail's), dynamic: before and after the claim goes out
    assert sorted(set(counts)) == [2 * step, 4 * step] and counts.count(4 * step) == (2 if mode == 2 else 1), counts
    for body, n in zip(bodies, counts):
        assert not [x for x in body if x.startswith(("v_accvgpr", "scratch_"))]
        assert sum(x.startswith("s_barrier") for x in body) == n // step
        if edge == 256 and n == 4 * step and form != 3:
            # nothing between the MFMAs but reads, loads and scalars (an address or two may be left)
            assert sum(x.startswith("v_") and not x.startswith("v_mfma") for x in body) <= 4


@pytest.mark.parametrize("edge,form,mode", CASES)
def test_mfma_hazard_distances(asm, edge, form, mode):
    """An MFMA result reaches any other reader only after at least the wait states the longest MFMA needs, and a
    vector write reaches an MFMA that reads it only after the two wait states that takes."""
    f = isa.instructions(kernel_text(asm, edge, form, mode))
    first = next(n for n, x in enumerate(f) if x.startswith("v_mfma"))
    last_mfma, last_valu, pos, result, operand = {}, {}, 0, None, None
    for x in f[first - 64:]:
        pos += isa.slots(x)
        op, ops = x.split()[0], isa.operands(x)
        if op.startswith("v_mfma"):
            for r in ops[1:3]:
                for reg in isa.regs(r):
                    if reg in last_valu:
                        operand = min(operand or 10 ** 9, pos - last_valu[reg])
            for reg in isa.regs(ops[0]):
                last_mfma[reg] = pos
                last_valu.pop(reg, None)
            continue
        if op.startswith("s_") or not ops:
            continue
        store = op.startswith(("global_store", "buffer_store", "flat_store", "ds_write"))
        for r in (ops if store else ops[1:]):
            for reg in isa.regs(r):
                if reg in last_mfma:
                    result = min(result or 10 ** 9, pos - last_mfma[reg])
        if not store:
            for reg in isa.regs(ops[0]):
                last_mfma.pop(reg, None)
                last_valu.pop(reg, None)
                if op.startswith("v_") and not op.startswith(("v_cmp", "v_readfirstlane", "v_readlane")):
                    last_valu[reg] = pos
    assert result is None or result >= isa.MIN_MFMA_RESULT_DISTANCE, result
    assert operand is None or operand >= 3, operand


def test_no_product_kernel_uses_scratch(asm):
    sizes = re.findall(r"\.amdhsa_kernel (\S+).*?\.amdhsa_private_segment_fixed_size (\d+)", asm, re.S)
    assert len(sizes) == len(CASES) + 4
    assert not [k for k, s in sizes if int(s) != 0]


@pytest.mark.parametrize("source", ["rows_kernel.hip", "act_kernel.hip", "norm_kernel.hip"])
def test_no_other_kernel_uses_scratch(tmp_path, source):
    sizes = re.findall(r"\.amdhsa_kernel (\S+).*?\.amdhsa_private_segment_fixed_size (\d+)", compile_to_asm(tmp_path, source), re.S)
    assert sizes and not [k for k, s in sizes if int(s) != 0]


def test_small_tiles_leave_room_for_their_neighbours(asm):
    """TN's 128 x 128 tiles run two workgroups a CU: at most 256 registers (vector and accumulator) a lane."""
    m = re.search(r"\.amdhsa_kernel _ZN3ptg18ptg_product_kernelILi128ELi2ELi2E\S+.*?\.amdhsa_next_free_vgpr (\d+)", asm, re.S)
    assert int(m.group(1)) <= 256
