"""Checks on the compiled gfx950 code of the int8, scaled and loss kernels (CPU only: hipcc -S): the shared main loop's
properties, as for the other products, and no scratch anywhere."""

import re

import pytest

from tests import test_kernel_isa as isa
from tests.test_product_isa import compile_to_asm, loops

pytestmark = isa.pytestmark

# source, kernels as (name and template arguments before the LDS stages and the mode)
KERNELS = {
    "product_i8_kernel.hip": [("ptg_product_i8_kernel", "Li{edge}E")],
    "product_scaled_kernel.hip": [("ptg_product_scaled_kernel", "Li{edge}ELi5E"), ("ptg_product_scaled_kernel", "Li{edge}ELi6E")],
    "loss_kernel.hip": [("ptg_loss_kernel", "Li{edge}ELi7E"), ("ptg_loss_kernel", "Li{edge}ELi8E")],
}
CASES = [(source, name, args, edge, stages, mode) for source, kernels in KERNELS.items() for name, args in kernels
         for edge, stages, mode in ((256, 4, 2), (256, 4, 0), (128, 4, 2), (128, 4, 0), (128, 8, 0)) if stages == 4 or "Li6E" not in args]


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("isa")
    return {source: compile_to_asm(tmp, source) for source in [*KERNELS, "quantise_kernel.hip", "rows_shared_kernel.hip"]}


def kernel_text(text, name, args, edge, stages, mode):
    i = text.index(f"\n_ZN3ptg{len(name)}{name}I{args.format(edge=edge)}Li{stages}ELi{mode}EEE")
    i = text.index(":", i)
    return text[i:text.index(".Lfunc_end", i)]


@pytest.mark.parametrize("source,name,args,edge,stages,mode", CASES)
def test_main_loop_is_one_block_without_copies(asm, source, name, args, edge, stages, mode):
    step = 64 if edge == 256 else 16  # MFMAs a k-step
    text = kernel_text(asm[source], name, args, edge, stages, mode)
    bodies = loops(text)
    counts = [sum(x.startswith("v_mfma") for x in b) for b in bodies]
    assert sorted(set(counts)) == [2 * step, 4 * step] and counts.count(4 * step) == (2 if mode == 2 else 1), counts
    kinds = {x.split()[0] for b in bodies for x in b if x.startswith("v_mfma")}
    assert kinds == {"v_mfma_i32_16x16x64_i8" if "i8" in name else "v_mfma_f32_16x16x32_bf16"}
    for body, n in zip(bodies, counts):
        assert not [x for x in body if x.startswith(("v_accvgpr", "scratch_"))]
        assert sum(x.startswith("s_barrier") for x in body) == n // step
        if edge == 256 and n == 4 * step:
            # nothing between the MFMAs but reads, loads and scalars (an address or two, or a few scalars that were kept in
            # a vector register, may be left: one to 32 MFMAs)
            assert sum(x.startswith("v_") and not x.startswith("v_mfma") for x in body) <= 8


@pytest.mark.parametrize("source,name,args,edge,stages,mode", CASES)
def test_mfma_hazard_distances(asm, source, name, args, edge, stages, mode):
    """An MFMA result reaches any other reader only after the wait states the longest MFMA needs."""
    f = isa.instructions(kernel_text(asm[source], name, args, edge, stages, mode))
    first = next(n for n, x in enumerate(f) if x.startswith("v_mfma"))
    last_mfma, pos, result = {}, 0, None
    for x in f[first - 64:]:
        pos += isa.slots(x)
        op, ops = x.split()[0], isa.operands(x)
        if op.startswith("v_mfma"):
            for reg in isa.regs(ops[0]):
                last_mfma[reg] = pos
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
    assert result is None or result >= isa.MIN_MFMA_RESULT_DISTANCE, result


@pytest.mark.parametrize("source", [*KERNELS, "quantise_kernel.hip", "rows_shared_kernel.hip"])
def test_no_kernel_uses_scratch(asm, source):
    sizes = re.findall(r"\.amdhsa_kernel (\S+).*?\.amdhsa_private_segment_fixed_size (\d+)", asm[source], re.S)
    assert sizes and not [k for k, s in sizes if int(s) != 0]


def test_small_tiles_leave_room_for_their_neighbours(asm):
    """128 x 128 tiles in four stages run two workgroups a CU: at most 256 registers (vector and accumulator) a lane, and half
    the LDS."""
    for source, kernels in KERNELS.items():
        for name, args in kernels:
            start = f"_ZN3ptg{len(name)}{name}I{args.format(edge=128)}Li4E"
            found = re.findall(r"\.amdhsa_kernel " + start + r"\S+(.*?)\.end_amdhsa_kernel", asm[source], re.S)
            assert len(found) == 2, start
            for text in found:
                assert int(re.search(r"\.amdhsa_next_free_vgpr (\d+)", text).group(1)) <= 256
                assert int(re.search(r"\.amdhsa_group_segment_fixed_size (\d+)", text).group(1)) <= 80 * 1024


def test_large_tiles_fit_the_lds_of_a_cu(asm):
    for source in KERNELS:
        sizes = re.findall(r"\.amdhsa_kernel (\S+).*?\.amdhsa_group_segment_fixed_size (\d+)", asm[source], re.S)
        assert sizes and all(int(s) <= 160 * 1024 for _, s in sizes), sizes
