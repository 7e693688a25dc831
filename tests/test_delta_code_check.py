"""The build of libsdm_delta refuses machine code that reads a matrix-core result too early (CPU only: a small kernel is
compiled, none is run)."""

import os

import pytest

from deterministic_fp32_gemm_amd import _build, _code_check

# The product's result is read where a long and a short path meet.
KERNEL = """
#include <hip/hip_runtime.h>
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
extern "C" __global__ void meet(const bf16x8* a, const bf16x8* b, f32x4* o, float* p, int n, float q) {
    const bf16x8 x = a[threadIdx.x], y = b[threadIdx.x];
    f32x4 r = {0, 0, 0, 0};
    float t = q;
    r = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, r, 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    if (n > 3) {
#pragma unroll
        for (int i = 0; i < 12; ++i) asm volatile("v_add_f32 %0, %0, %0" : "+v"(t));
    } else {
        asm volatile("v_sub_f32 %0, %0, %0" : "+v"(t));
        SHORT
    }
    __builtin_amdgcn_sched_barrier(0);
    o[threadIdx.x] = r * q;
    p[threadIdx.x] = t;
}
"""


def built(tmp_path, short):
    src = tmp_path / "meet.hip"
    src.write_text(KERNEL.replace("SHORT", short))
    return str(tmp_path / "libmeet.so"), (str(src),)


def test_an_early_read_is_refused(tmp_path):
    out, sources = built(tmp_path, "")
    (tmp_path / "libmeet.so").write_text("what was there")
    with pytest.raises(_code_check.CodeError, match="meet reads a matrix-core result too early"):
        _build.build_delta(out, sources=sources)
    assert (tmp_path / "libmeet.so").read_text() == "what was there"
    assert not os.path.exists(out + ".tmp")


def test_the_wait_in_place_is_accepted(tmp_path):
    out, sources = built(tmp_path, 'asm volatile("s_nop 7");')
    assert _build.build_delta(out, sources=sources) == out
    assert _code_check.verify(out, _build.llvm()) == 1


def test_scratch_memory_is_refused(tmp_path):
    src = tmp_path / "spill.hip"
    src.write_text("""
#include <hip/hip_runtime.h>
extern "C" __global__ void spill(const float* a, float* o, int n) {
    float v[64];
    for (int i = 0; i < 64; ++i) v[i] = a[i * 64 + threadIdx.x];
    o[threadIdx.x] = v[n & 63] + v[a[0] > 0.f ? n & 31 : 5];
}
""")
    with pytest.raises(_code_check.CodeError, match="scratch"):
        _build.build_delta(str(tmp_path / "lib.so"), sources=(str(src),))


def step(op, *operands):
    return [op, list(operands), None]


@pytest.mark.parametrize("between,early", [
    ([], True), ([step("s_nop", "6")], True), ([step("s_nop", "7")], False),
    ([step("v_mov_b32_e32", "v2", "v8")], True),                                    # an overwrite
    ([step("v_mfma_f32_16x16x32_bf16", "v[20:23]", "v[8:11]", "v[12:15]", "v[1:4]")] + [step("s_nop", "7")], True),
    ([step("v_mfma_f32_16x16x32_bf16", "v[0:3]", "v[8:11]", "v[12:15]", "v[0:3]")] + [step("s_nop", "7")], False),
    ([step("global_store_dwordx4", "v30", "v[0:3]", "s[8:9]")] + [step("s_nop", "7")], True),
])
def test_reads(between, early):
    code = [step("v_mfma_f32_16x16x32_bf16", "v[0:3]", "v[4:7]", "v[8:11]", "v[0:3]"), *between,
            step("v_mul_f32_e32", "v9", "v3", "v9"), step("s_endpgm")]
    assert bool(_code_check.early_reads(code)) == early


@pytest.mark.parametrize("operand,names", [
    ("v3", {"v3"}), ("-v3", {"v3"}), ("|v3|", {"v3"}), ("-|a12|", {"a12"}), ("v[2:4]", {"v2", "v3", "v4"}), ("s3", set()),
    ("v[2:3] offset:16", {"v2", "v3"}), ("v3 quad_perm:[1", {"v3"}), ("v3 row_half_mirror row_mask:0xf", {"v3"}),
    ("neg(v3)", {"v3"}), ("vcc", set()), ("off", set()), ("0x3f", set()), ("vmcnt(0)", set())])
def test_registers_of_an_operand(operand, names):
    assert _code_check.registers(operand) == names


@pytest.mark.parametrize("read", [step("ds_write_b128", "v30", "v[0:3] offset:16"),
                                  step("v_mov_b32_dpp", "v9", "v2 quad_perm:[1", "0", "3", "2] row_mask:0xf bank_mask:0xf")])
def test_reads_with_modifiers(read):
    product = step("v_mfma_f32_16x16x32_bf16", "v[0:3]", "v[4:7]", "v[8:11]", "v[0:3]")
    assert _code_check.early_reads([product, read, step("s_endpgm")])
    assert not _code_check.early_reads([product, step("s_nop", "7"), read, step("s_endpgm")])


def test_an_unknown_product_is_refused():
    with pytest.raises(_code_check.CodeError, match="not known"):
        _code_check.early_reads([step("v_mfma_f32_32x32x16_bf16", "v[0:15]", "v[16:19]", "v[20:23]", "v[0:15]")])
