"""The waits that the inline matrix and load instructions of the products on fp16
mirrors need (inline_waits.py), in the library as it was built; and the checks
themselves, on listings with a mistake in each."""
import os

import pytest

import inline_waits as W
from block_quantized_decode_q4_amd import build

needs_objdump = pytest.mark.skipif(not os.path.exists(W.OBJDUMP), reason="no llvm-objdump")


@needs_objdump
def test_built_kernels(tmp_path):
    from block_quantized_decode_q4_amd import q4k
    q4k.load_library()                         # built, if it was not
    checked = loads = products = 0
    for code_object in W.code_objects(build.LIB, b"f16_act_kernel", str(tmp_path)):
        for name, code in W.functions(W.disassemble(code_object)).items():
            here = sum("_load_lds_" in i.name for i in code)
            if here:
                assert W.faults(code) == [], name
                checked += 1
                loads += here
                products += sum(i.matrix for i in code)
    # six shapes, with and without a gate, dense and grouped
    assert checked == 24 and loads > 24 * 8 and products > 24 * 8


def _faults(*lines):
    """Of a function of these instructions, four bytes each."""
    text = "0000000000001000 <f>:\n" + "".join(
        "\t%s // %012X: 00000000%s\n" % (line.split(" -> ")[0], 0x1000 + 4 * i,
                                         " <f+0x%x>" % (4 * int(line.split(" -> ")[1]))
                                         if " -> " in line else "")
        for i, line in enumerate(lines))
    return W.faults(W.functions(text)["f"])


MFMA = "v_mfma_f32_16x16x32_f16 a[0:3], v[2:5], v[6:9], a[0:3]"
DMA = ("s_mov_b32 m0, s1", "s_nop 0", "global_load_lds_dwordx4 v1, s[4:5]")


def test_sound_listings():
    assert _faults("v_mov_b32_e32 v2, v1", "s_nop 1", MFMA, MFMA, "s_nop 15", "s_nop 1",
                   "v_accvgpr_read_b32 v1, a2", "s_endpgm") == []
    # 3 wait states, and M0's two instructions
    assert _faults("v_readfirstlane_b32 s4, v1", "s_nop 2", *DMA, "s_endpgm") == []
    # a loop: its last instructions lie before its first
    assert _faults("s_nop 0", MFMA, "v_mov_b32_e32 v9, v1", "s_nop 0", "s_cbranch_scc1 1 -> 1",
                   "s_nop 15", "s_nop 1", "v_accvgpr_read_b32 v1, a2", "s_endpgm") == []


@pytest.mark.parametrize("lines", [
    ("v_mov_b32_e32 v9, v1", "s_nop 0", MFMA, "s_endpgm"),
    ("v_accvgpr_write_b32 a3, v1", MFMA, "s_endpgm"),
    (MFMA, "s_nop 15", "v_accvgpr_read_b32 v1, a2", "s_endpgm"),
    (MFMA, "s_nop 15", "s_nop 0", "ds_write_b128 v1, a[0:3]", "s_endpgm"),
    (MFMA, "v_mfma_f32_16x16x32_f16 a[2:5], v[2:5], v[6:9], a[2:5]", "s_endpgm"),
    (MFMA, "v_mfma_f32_16x16x32_f16 a[8:11], a[0:3], v[6:9], a[8:11]", "s_endpgm"),
    # round a loop: the write stands behind the product
    (MFMA, "v_mov_b32_e32 v9, v1", "s_cbranch_scc1 1 -> 0", "s_endpgm"),
    ("v_readfirstlane_b32 s5, v1", "s_nop 0", *DMA, "s_endpgm"),
    ("s_mov_b32 m0, s1", "global_load_lds_dwordx4 v1, s[4:5]", "s_endpgm"),
    ("s_mov_b32 m0, s1", "s_nop 0", "s_add_u32 s4, s4, s6", "global_load_lds_dwordx4 v1, s[4:5]",
     "s_endpgm"),
    (*DMA, "s_mov_b32 s3, m0", "s_endpgm"),
    ("s_mov_b32 m0, s1", "s_nop 0", "s_branch 1 -> 4", "s_nop 0",
     "global_load_lds_dwordx4 v1, s[4:5]", "s_endpgm"),
], ids=lambda lines: str(len(lines)))
def test_listings_with_a_mistake(lines):
    assert len(_faults(*lines)) >= 1
