"""libsdm_block's host entry points without a GPU: glr_api.cpp and ffn_api.cpp built by the host compiler beside stand-ins for
the device checks and the launches, which note what they were called with."""

import ctypes
import functools
import os
import shutil
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "deterministic_fp32_gemm_amd", "csrc")

STAND_INS = r"""
#include <hip/hip_runtime.h>
#include "delta_host.h"
#include "glr.h"
#include "ffn.h"
namespace sdm_delta {
int record_hip_error(hipError_t) { return SDM_GX_ERR_HIP; }
int last_hip_error() { return 0; }
const char* status_text(int) { return ""; }
int current_gfx950(int* dev) { *dev = 0; return SDM_GX_OK; }
static uintptr_t g_host_from = 0;                       // addresses from here on are not the device's
int pointer_on(const void* p, int) { return reinterpret_cast<uintptr_t>(p) >= g_host_from ? SDM_GX_ERR_DEVICE : SDM_GX_OK; }

struct Note { int64_t kind, a, b, c, d; };
static Note g_notes[64];
static int g_n = 0;
static hipError_t note(int64_t kind, int64_t a = 0, int64_t b = 0, int64_t c = 0, int64_t d = 0) {
    if (g_n < 64) g_notes[g_n++] = Note{kind, a, b, c, d};
    return hipSuccess;
}
// kinds: 0 recurrence forward (rows of the queue), 1 gradient (parts), 2 step, 3 pair (type, tile, workgroup rows), 4 both
// products (type, tile, parts of dx, parts of the weights'), 5 few rows, 6 laid out, 7 dg and du (parts), 8 joined
hipError_t launch_glr_forward(const sdm_glr_args_t&, const GlrPlan& p, void*, hipStream_t) { return note(0, p.rows, p.cblocks); }
hipError_t launch_glr_backward(const sdm_glr_args_t&, const GlrPlan& p, void*, hipStream_t) { return note(1, p.segs, p.cblocks); }
hipError_t launch_glr_step(const sdm_glr_step_args_t&, hipStream_t) { return note(2); }
hipError_t launch_ffn_pair(const FfnProduct& p, int tile, hipStream_t) { return note(3, p.type, tile); }
hipError_t launch_ffn_products(const FfnProduct (&p)[2], int tile, hipStream_t) { return note(4, p[0].type, tile, p[0].parts, p[1].parts); }
hipError_t launch_ffn_few(const sdm_ffn_args_t& a, hipStream_t) { return note(5, a.dtype); }
hipError_t launch_ffn_lay(const FfnLay (&l)[3], hipStream_t) { return note(6, l[0].R, l[1].R, l[2].R); }
hipError_t launch_ffn_grad(const FfnGrad& g, const FfnLay (&)[3], hipStream_t) { return note(7, g.parts); }
hipError_t launch_ffn_join(const FfnJoin (&j)[2], hipStream_t) { return note(8, j[0].parts, j[1].parts); }
}  // namespace sdm_delta
extern "C" {
void stub_reset(uint64_t host_from) { sdm_delta::g_n = 0; sdm_delta::g_host_from = host_from; }
int stub_notes(int64_t* out) {
    for (int i = 0; i < sdm_delta::g_n; ++i) __builtin_memcpy(out + 5 * i, &sdm_delta::g_notes[i], 40);
    return sdm_delta::g_n;
}
}
"""

KINDS = ("glr_forward", "glr_backward", "glr_step", "pair", "products", "few", "lay", "grad", "join")
HOST = 1 << 46          # addresses from here on are the host's


@functools.lru_cache(None)
def library():
    work = tempfile.mkdtemp(prefix="block_stub_")
    src, out = os.path.join(work, "stand_ins.cpp"), os.path.join(work, "stub.so")
    try:
        with open(src, "w") as f:
            f.write(STAND_INS)
        rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"), "-I", CSRC,
                        src, os.path.join(CSRC, "glr_api.cpp"), os.path.join(CSRC, "ffn_api.cpp"), "-o", out], check=True)
        lib = ctypes.CDLL(out)
    finally:
        shutil.rmtree(work)
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    lib.stub_reset.argtypes = [ctypes.c_uint64]
    for n in ("sdm_glr_forward", "sdm_glr_backward", "sdm_ffn_forward", "sdm_ffn_backward"):
        getattr(lib, n).argtypes = [vp, vp, i64, vp]
    lib.sdm_glr_step.argtypes = [vp, vp]
    for n in ("sdm_glr_workspace", "sdm_ffn_workspace"):
        getattr(lib, n).argtypes, getattr(lib, n).restype = [vp, ctypes.c_int32], i64
    lib.sdm_glr_marks.argtypes, lib.sdm_glr_marks.restype = [vp], i64
    return lib


def call(name, *args):
    """The entry point's status and the launches it made: (kind, four numbers) each."""
    lib = library()
    lib.stub_reset(HOST)
    status = getattr(lib, name)(*args)
    notes = (ctypes.c_int64 * 320)()
    n = lib.stub_notes(notes)
    return status, [(KINDS[notes[5 * i]], *notes[5 * i + 1:5 * i + 5]) for i in range(n)]
