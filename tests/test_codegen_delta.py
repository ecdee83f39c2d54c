"""The scan for hazards around MFMAs written in inline asm
(test_regression_amd/codegen_check.py) on known sequences; tests/test_codegen.py
runs it over the built kernels."""
from test_regression_amd import codegen_check

GOOD = """
v_mov_b32_e32 v0, 0
;;#ASMSTART
s_nop 1
;;#ASMEND
;;#ASMSTART
v_mfma_f32_16x16x32_f16 v[0:3], v[8:11], v[12:15], v[0:3]
;;#ASMEND
;;#ASMSTART
v_mfma_f32_16x16x32_f16 v[0:3], v[16:19], v[12:15], v[0:3]
;;#ASMEND
;;#ASMSTART
s_nop 11
;;#ASMEND
v_mul_f32_e32 v5, v0, v6
"""


def test_clean_sequence():
    assert codegen_check.scan_asm_mfma(GOOD) == []


def test_accumulator_or_operand_written_too_late():
    assert len(codegen_check.scan_asm_mfma(GOOD.replace("s_nop 1\n", "s_nop 0\n"))) == 1
    late = GOOD.replace("v_mov_b32_e32 v0, 0", "v_add_f32_e32 v9, v20, v21").replace("s_nop 1\n", "s_nop 0\n")
    assert len(codegen_check.scan_asm_mfma(late)) == 1


def test_result_read_or_rewritten_too_early():
    early = GOOD.replace("s_nop 11", "s_nop 3")
    assert len(codegen_check.scan_asm_mfma(early)) == 1
    assert len(codegen_check.scan_asm_mfma(early.replace("v_mul_f32_e32 v5, v0, v6", "ds_read_b128 v[0:3], v9"))) == 1
    assert len(codegen_check.scan_asm_mfma(early.replace(
        "v_mul_f32_e32 v5, v0, v6", "v_mfma_f32_16x16x32_f16 v[4:7], v[0:3], v[8:11], v[4:7]"))) == 1
