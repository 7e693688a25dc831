"""The code objects of libsdm_delta (built here, read with the ROCm LLVM tools; CPU only).

No kernel uses scratch memory. A register that is spilled where only some lanes are active comes back without the
others' values, and a matrix-core operand needs all 64.

No instruction reads a matrix-core result before it is there. The compiler adds the wait states within straight code
but has been seen to miss them where a branch lies between the product and its first read (the results were then those
of the product before, now and then), so every path from every product is followed until the wait is over."""

import os
import re
import subprocess

import pytest

from deterministic_fp32_gemm_amd._build import DELTA_LIB_PATH
from tests.test_code_objects import LLVM, MAGIC

# wait states before a vector instruction may read the result (4 passes: 8; the float32 product of 8 passes: 10)
WAITS = {"v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_16x16x4_f32": 10}


def code_objects(tmp_path):
    tools = [os.path.join(LLVM, t) for t in ("llvm-objcopy", "clang-offload-bundler", "llvm-readelf", "llvm-objdump")]
    if not (os.path.exists(DELTA_LIB_PATH) and all(map(os.path.exists, tools))):
        pytest.skip("library not built or ROCm LLVM tools missing")
    objcopy, bundler, readelf, objdump = tools
    fat = tmp_path / "fatbin.bin"
    subprocess.run([objcopy, f"--dump-section=.hip_fatbin={fat}", DELTA_LIB_PATH], check=True)
    data = fat.read_bytes()
    starts = [m.start() for m in re.finditer(re.escape(MAGIC), data)]
    found = []
    for k, a in enumerate(starts):
        part, co = tmp_path / f"b{k}.bin", tmp_path / f"b{k}.co"
        part.write_bytes(data[a:starts[k + 1] if k + 1 < len(starts) else len(data)])
        subprocess.run([bundler, "--type=o", f"--input={part}", "--targets=hipv4-amdgcn-amd-amdhsa--gfx950",
                        f"--output={co}", "--unbundle"], check=True)
        found.append((subprocess.run([readelf, "--notes", str(co)], check=True, capture_output=True, text=True).stdout,
                      subprocess.run([objdump, "-d", "--no-show-raw-insn", str(co)], check=True, capture_output=True,
                                     text=True).stdout))
    return found


def registers(operand):
    m = re.fullmatch(r"-?\|?([av])(\d+)\|?", operand)
    if m:
        return {m[1] + m[2]}
    m = re.fullmatch(r"-?([av])\[(\d+):(\d+)\]", operand)
    return {m[1] + str(i) for i in range(int(m[2]), int(m[3]) + 1)} if m else set()


def parse(text):
    """Kernels as lists of (operation, operands, branch target's index or None)."""
    kernels, addresses, code, name = {}, {}, [], None
    for line in text.splitlines():
        m = re.match(r"^[0-9a-f]+ <(.+)>:", line)
        if m:
            name = m[1]
            kernels[name] = code = []
            addresses[name] = {}
            continue
        m = re.match(r"^\s+(\S.*?)\s*//\s*([0-9A-Fa-f]+):?(.*)$", line)
        if m and name:
            op, *rest = m[1].split(None, 1)
            to = re.search(r"<(.+?)\+0x([0-9a-f]+)>", m[3] + " " + m[1])
            addresses[name][int(m[2], 16)] = len(code)
            code.append([op, [x.strip() for x in rest[0].split(",")] if rest else [], int(to[2], 16) if to else None])
    for name, code in kernels.items():
        base = min(addresses[name], default=0)
        for ins in code:
            if ins[2] is not None:
                ins[2] = addresses[name][base + ins[2]]
    return kernels


def early_reads(code):
    bad = []
    for i, (op, operands, _) in enumerate(code):
        if not op.startswith("v_mfma"):
            continue
        need, result = WAITS[op], registers(operands[0])
        todo, seen = [(i + 1, 0)], {}
        while todo:
            at, waited = todo.pop()
            while at < len(code) and waited < need and seen.get(at, need) > waited:
                seen[at] = waited
                o, b, to = code[at]
                if o == "s_endpgm":
                    break
                memory = o.startswith(("ds_", "global_", "buffer_", "scratch_", "flat_"))
                reads = b[1:3] if o.startswith("v_mfma") else b if memory and "load" not in o and "read" not in o else b[1:]
                if any(registers(x) & result for x in reads):
                    bad.append((i, op, operands[0], at, o, b, waited))
                    break
                if o.startswith("v_") and b and registers(b[0]) & result:
                    if not o.startswith("v_mfma"):
                        bad.append((i, op, operands[0], at, o, b, waited))
                    break
                waited += int(b[0], 0) + 1 if o == "s_nop" else 1
                if o == "s_branch":
                    at = to
                    continue
                if o.startswith("s_cbranch"):
                    todo.append((to, waited))
                at += 1
    return bad


def test_no_scratch_and_no_early_reads(tmp_path):
    kernels = products = 0
    for notes, text in code_objects(tmp_path):
        for size in re.findall(r"\.private_segment_fixed_size:\s*(\d+)", notes):
            assert size == "0"
        for count in re.findall(r"\.vgpr_spill_count:\s*(\d+)", notes):
            assert count == "0"
        for name, code in parse(text).items():
            kernels += 1
            products += sum(op.startswith("v_mfma") for op, _, _ in code)
            assert not early_reads(code), (name, early_reads(code)[:3])
            assert not any(op.startswith("v_pk_") and "f32" in op for op, _, _ in code), name
    assert kernels > 40 and products > 1000


def test_early_reads_are_seen():
    mfma = ["v_mfma_f32_16x16x32_bf16", ["a[0:3]", "v[0:3]", "v[4:7]", "a[0:3]"], None]
    read, nop, end = ["v_accvgpr_read_b32", ["v9", "a2"], None], ["s_nop", ["6"], None], ["s_endpgm", [], None]
    other = ["v_mov_b32_e32", ["v9", "v8"], None]
    assert early_reads([mfma, read, end])
    assert early_reads([mfma, nop, read, end])
    assert not early_reads([mfma, nop, other, read, end])
    assert early_reads([mfma, ["s_cbranch_vccnz", ["x"], 4], nop, other, read, end])        # past the wait
    assert not early_reads([mfma, mfma, nop, other, read, end])
