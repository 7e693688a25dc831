"""Checks of a built library's code objects that no source can promise, made by every build of libsdm_delta and libsdm_block.

A matrix-core result may be read only some wait states after its product; the hardware does not wait by itself and the
compiler puts the wait there. This one counts it along one path where two lead from the product to the read: of

    r = product; if (uniform) { many instructions } else { few }; read r

the short side is left too early (6 of 8 wait states, with 12 instructions on the long side). The result read is then the
register's value of before. So every path from every product is followed in the machine code here.

No kernel may use scratch memory: a register spilled where only some lanes are active comes back without the others'
values, and a matrix-core operand needs all 64. And none may hold packed float32 instructions."""

from __future__ import annotations

import os
import re
import subprocess
import tempfile

TARGET = "hipv4-amdgcn-amd-amdhsa--gfx950"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
# wait states before a vector instruction may read the result (4 passes: 8; the float32 product of 8 passes: 10)
WAITS = {"v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_16x16x4_f32": 10}
# libsdm_block's beside them (8 passes: 12; 16 passes: 20, of float32 18)
BLOCK_WAITS = {**WAITS, "v_mfma_f32_16x16x32_f16": 8, "v_mfma_f32_16x16x32_fp8_fp8": 8, "v_mfma_f32_32x32x16_bf16": 12,
               "v_mfma_f32_32x32x16_f16": 12, "v_mfma_f32_32x32x64_f8f6f4": 20}
_STORES = ("ds_", "global_", "buffer_", "scratch_", "flat_")


class CodeError(RuntimeError):
    """A built code object that must not run."""


def code_objects(path: str, llvm: str):
    """(notes, disassembly) of each gfx950 code object of a shared library."""
    run = lambda tool, *args: subprocess.run([os.path.join(llvm, tool), *args], check=True, capture_output=True,  # noqa: E731
                                             text=True).stdout
    with tempfile.TemporaryDirectory() as tmp:
        fat, part, co = (os.path.join(tmp, n) for n in ("fat", "part", "co"))
        run("llvm-objcopy", f"--dump-section=.hip_fatbin={fat}", path)
        with open(fat, "rb") as f:
            data = f.read()
        starts = [m.start() for m in re.finditer(re.escape(MAGIC), data)]
        if not starts:
            raise CodeError(f"{path}: no code objects")
        for a, b in zip(starts, starts[1:] + [len(data)]):
            with open(part, "wb") as f:
                f.write(data[a:b])
            run("clang-offload-bundler", "--type=o", f"--input={part}", f"--targets={TARGET}", f"--output={co}",
                "--unbundle")
            yield run("llvm-readelf", "--notes", co), run("llvm-objdump", "-d", "--no-show-raw-insn", co)


def registers(operand: str) -> set:
    """The vector registers that an operand names, with or without a sign, an absolute value or modifiers after it."""
    m = re.match(r"(?:-|neg\()?(?:\||abs\()?([av])(?:(\d+)\b|\[(\d+):(\d+)\])", operand)
    if not m:
        return set()
    lo, hi = (m[2], m[2]) if m[2] else (m[3], m[4])
    return {m[1] + str(i) for i in range(int(lo), int(hi) + 1)}


def kernels(text: str) -> dict:
    """A disassembly's functions as lists of (operation, operands, index that a branch goes to)."""
    found, addresses, name = {}, {}, None
    for line in text.splitlines():
        m = re.match(r"^[0-9a-f]+ <(.+)>:", line)
        if m:
            name = m[1]
            found[name], addresses[name] = [], {}
            continue
        m = re.match(r"^\s+(\S.*?)\s*//\s*([0-9A-Fa-f]+):?(.*)$", line)
        if m and name:
            op, *rest = m[1].split(None, 1)
            to = re.search(r"<.+?\+0x([0-9a-f]+)>", m[3] + " " + m[1])
            addresses[name][int(m[2], 16)] = len(found[name])
            found[name].append([op, [x.strip() for x in rest[0].split(",")] if rest else [], int(to[1], 16) if to else None])
    for name, code in found.items():
        base = min(addresses[name], default=0)
        for ins in code:
            if ins[0].startswith(("s_branch", "s_cbranch")):
                if ins[2] is None or base + ins[2] not in addresses[name]:
                    raise CodeError(f"{name}: a branch to an unknown place")
                ins[2] = addresses[name][base + ins[2]]
            elif ins[0] in ("s_setpc_b64", "s_swappc_b64"):
                raise CodeError(f"{name}: calls cannot be followed")
    return found


def early_reads(code, waits=WAITS) -> list:
    """Reads (or overwrites) of a product's result before its wait is over, on any path."""
    bad = []
    for i, (op, operands, _) in enumerate(code):
        if not op.startswith(("v_mfma", "v_smfmac")):
            continue
        if op not in waits:
            raise CodeError(f"{op}: its wait states are not known here")
        need, result = waits[op], registers(operands[0])
        todo, seen = [(i + 1, 0)], {}
        while todo:
            at, waited = todo.pop()
            while at < len(code) and waited < need and seen.get(at, need) > waited:
                seen[at] = waited
                o, b, to = code[at]
                if o == "s_endpgm":
                    break
                product = o.startswith("v_mfma")
                store = o.startswith(_STORES) and "load" not in o and "read" not in o
                # a product may take this one's whole result as the sum it adds to: that goes from one to the next
                reads = b[1:3] + ([b[3]] if registers(b[3]) != result else []) if product else b if store else b[1:]
                over = bool(b) and bool(registers(b[0]) & result)
                if any(registers(x) & result for x in reads) or (over and o.startswith("v_") and not product):
                    bad.append((i, op, operands[0], at, o, b, waited))
                    break
                if over and o.startswith("v_"):
                    break
                waited += int(b[0], 0) + 1 if o == "s_nop" else 1
                if o == "s_branch":
                    at = to
                    continue
                if o.startswith("s_cbranch"):
                    todo.append((to, waited))
                at += 1
    return bad


# what reads m0 without naming it, beside loads into LDS
_M0_READERS = ("v_movrel", "s_movrel", "s_sendmsg", "s_set_gpr_idx", "v_interp", "ds_gws", "ds_ordered", "ds_append", "ds_consume")


def m0_uses(code) -> list:
    """Uses of m0 other than writing it for a load into LDS that follows at once. Such loads are written in assembly, which cannot
    say that it overwrites m0 (a register that the compiler keeps for itself): nothing else of a kernel may rely on it."""
    written, targets = set(), {to for _, _, to in code if to is not None}
    bad = []
    for i, (op, operands, _) in enumerate(code):
        if any(re.search(r"\blds\b", x) for x in operands) and op.startswith(("buffer_load", "global_load")):
            before = [(o, b[:1]) for o, b, _ in code[max(i - 2, 0):i]]
            if before == [("s_mov_b32", ["m0"]), ("s_nop", ["0"])] and not targets & {i - 1, i}:
                written.add(i - 2)
            else:
                bad.append((i, op, operands))
    for i, (op, operands, _) in enumerate(code):
        if (any(re.search(r"\bm0\b", x) for x in operands) or op.startswith(_M0_READERS)) and i not in written:
            bad.append((i, op, operands))
    return bad


def verify(path: str, llvm: str, waits=WAITS) -> int:
    """The number of matrix products of a library's kernels; raises CodeError for code that must not run."""
    products = 0
    for notes, text in code_objects(path, llvm):
        for field in ("private_segment_fixed_size", "vgpr_spill_count"):
            if any(int(n) for n in re.findall(rf"\.{field}:\s*(\d+)", notes)):
                raise CodeError(f"{path}: a kernel uses scratch memory ({field})")
        for name, code in kernels(text).items():
            bad = early_reads(code, waits)
            if bad:
                raise CodeError(f"{path}: {name} reads a matrix-core result too early: {bad[0]}")
            bad = m0_uses(code)
            if bad:
                raise CodeError(f"{path}: {name} uses m0, or does not set it for a load into LDS: {bad[0]}")
            if any(op.startswith("v_pk_") and "f32" in op for op, _, _ in code):
                raise CodeError(f"{path}: {name} holds packed float32 instructions")
            products += sum(op.startswith("v_mfma") for op, _, _ in code)
    return products
