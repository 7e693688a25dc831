"""The build refuses machine code in which m0 is used beside the loads into LDS that assembly writes it for (CPU only: a small
kernel is compiled, none is run)."""

import pytest

from deterministic_fp32_gemm_amd import _build, _code_check


def step(op, *operands, to=None):
    return [op, list(operands), to]


SET, NOP = step("s_mov_b32", "m0", "s24"), step("s_nop", "0")
LOAD = step("buffer_load_dwordx4", "v3", "s[4:7]", "0 offen lds")


@pytest.mark.parametrize("code,found", [
    ([SET, NOP, LOAD, SET, NOP, LOAD], 0),
    ([step("buffer_load_dwordx4", "v[0:3]", "v3", "s[4:7]", "0 offen"), step("v_mov_b32_e32", "v0", "s0")], 0),
    ([NOP, LOAD], 1), ([SET, LOAD], 2), ([SET, NOP, NOP, LOAD], 2),
    ([SET, NOP, LOAD, step("s_mov_b32", "s3", "m0")], 1), ([SET, NOP, LOAD, step("v_mov_b32_e32", "v0", "m0")], 1),
    ([SET, NOP, LOAD, step("s_add_u32", "m0", "m0", "s2")], 1), ([SET, NOP, LOAD, step("v_movrels_b32_e32", "v0", "v1")], 1),
    ([step("s_sendmsg", "sendmsg(MSG_INTERRUPT)")], 1),
    ([SET, NOP, LOAD, step("s_branch", "65533", to=2)], 2),     # a way to the load past its m0
    ([SET, NOP, LOAD, step("s_branch", "65533", to=0)], 0),
])
def test_uses_of_m0(code, found):
    assert len(_code_check.m0_uses(code)) == found


KERNEL = """
#include <hip/hip_runtime.h>
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
extern "C" __global__ void place(u32x4 r, unsigned off, unsigned* out) {
    __shared__ unsigned lds[256];
    lds[threadIdx.x] = off;
    __syncthreads();
    unsigned seen = 0;
    asm volatile("s_mov_b32 m0, %0\\n\\ts_nop 0\\n\\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(64u), "v"(off), "s"(r) : "memory");
    OTHER
    __syncthreads();
    out[threadIdx.x] = lds[threadIdx.x ^ 1] + seen;
}
"""


@pytest.mark.parametrize("other,fine", [("", True), ('asm volatile("s_mov_b32 %0, m0" : "=s"(seen));', False)])
def test_built(tmp_path, other, fine):
    src = tmp_path / "place.hip"
    src.write_text(KERNEL.replace("OTHER", other))
    out = str(tmp_path / "libplace.so")
    if fine:
        assert _build.build_block(out, sources=(str(src),)) == out
        return
    with pytest.raises(_code_check.CodeError, match="place uses m0"):
        _build.build_block(out, sources=(str(src),))


def test_the_library():
    loads = 0
    for _, text in _code_check.code_objects(_build.BLOCK_LIB_PATH, _build.llvm()):
        for name, code in _code_check.kernels(text).items():
            assert not _code_check.m0_uses(code), name
            loads += sum(op.startswith("buffer_load") and any("lds" in x for x in b) for op, b, _ in code)
    assert loads > 100
