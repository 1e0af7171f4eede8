"""Wait states in the compiled gfx950 code (CPU: only the library's own machine code is
read, nothing runs).

Two distances between instructions are the program's to keep on this architecture:

 * five wait states from a vector instruction that writes a scalar register to a memory
   instruction that reads it (its address);
 * one from a scalar instruction that writes M0 to a copy from global memory into LDS.

The compiler keeps them for the instructions that it knows; copies written as inline
assembly are its blind spot, so every kernel of the library is checked here as built.
"""
import os
import re
import shutil
import struct
import subprocess

import pytest

import gated_deltanet_layer_amd as gdn

OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
SGPR = re.compile(r"\bs(?:(\d+)|\[(\d+):(\d+)\])(?![\w:])")


def code_objects(path):
    """The GPU code objects that a library carries."""
    data, at = open(path, "rb").read(), 0
    while (at := data.find(MAGIC, at)) >= 0:
        n, = struct.unpack_from("<Q", data, at + 24)
        p = at + 32
        for _ in range(n):
            off, size, length = struct.unpack_from("<QQQ", data, p)
            if b"gfx" in data[p + 24:p + 24 + length] and size:
                yield data[at + off:at + off + size]
            p += 24 + length
        at += len(MAGIC)


def functions(text):
    """(name, [(address, mnemonic, operands, branch target or None)]) of a listing."""
    name, code = None, []
    for line in text.splitlines():
        head = re.match(r"^[0-9a-f]+ <(\S+)>:$", line)
        if head:
            if code:
                yield name, code
            name, code = head[1], []
            continue
        m = re.match(r"^\s+(\S+)\s*(.*?)\s*// ([0-9A-F]+):.*?(?:<.*?(?:\+0x([0-9a-f]+))?>)?$", line)
        if name and m:
            op = m[1]
            to = None
            if "branch" in op:   # the offset in instruction words from the next instruction
                d = int(m[2].split()[0])
                to = int(m[3], 16) + 4 + 4 * (d - 65536 if d >= 32768 else d)
            code.append((int(m[3], 16), op, m[2], to))
    if code:
        yield name, code


def scalars(operands):
    """Scalar registers named in operands; vcc and m0 by name."""
    out = set()
    for a, lo, hi in SGPR.findall(operands):
        out.update(range(int(a), int(a) + 1) if a else range(int(lo), int(hi) + 1))
    out.update(x for x in ("vcc", "m0") if re.search(rf"\b{x}(_lo|_hi)?\b", operands))
    return out


def vector_writes(op, operands):
    """Scalar registers that a vector instruction writes."""
    if not op.startswith("v_"):
        return set()
    args = re.split(r",\s*(?![^\[]*\])", operands)
    out = scalars(args[0])
    if "_co_" in op or "div_scale" in op:   # the carry is the second operand
        out |= scalars(args[1])
    return out


def is_memory(op):
    return op.startswith(("global_", "flat_", "buffer_", "scratch_", "tbuffer_"))


def hazards(code):
    """(address, instruction, writer, wait states that are there) of every violation."""
    at = {a: i for i, (a, _, _, _) in enumerate(code)}
    into = {}
    for i, (_, _, _, to) in enumerate(code):
        if to is not None:
            into.setdefault(at.get(to), []).append(i)

    def before(i):
        if i > 0 and code[i - 1][1] not in ("s_branch", "s_endpgm", "s_setpc_b64"):
            yield i - 1
        yield from into.get(i, ())

    def find(i, writes, regs, need):
        """A writer of regs fewer than `need` wait states before instruction i."""
        todo, best = [(j, 0) for j in before(i)], {}
        while todo:
            j, states = todo.pop()
            if states >= need or best.get(j, need) <= states:
                continue
            best[j] = states
            _, op, args, _ = code[j]
            if writes(op, args) & regs:
                return j, states
            step = int(args, 0) + 1 if op == "s_nop" else 1
            todo += [(k, states + step) for k in before(j)]
        return None

    def m0_writes(op, args):
        return {"m0"} if op.startswith("s_") and re.match(r"m0\b", args) else set()

    for i, (a, op, args, _) in enumerate(code):
        if not is_memory(op):
            continue
        if regs := scalars(args):
            if hit := find(i, vector_writes, regs, 5):
                yield a, f"{op} {args}", " ".join(code[hit[0]][1:3]), hit[1]
        if "_load_lds_" in op or re.search(r"\blds\b", args):
            if hit := find(i, m0_writes, {"m0"}, 1):
                yield a, f"{op} {args}", " ".join(code[hit[0]][1:3]), hit[1]


def listing(obj, tmp):
    path = os.path.join(tmp, "object")
    with open(path, "wb") as f:
        f.write(obj)
    return subprocess.run([OBJDUMP, "-d", path], capture_output=True, text=True, check=True).stdout


SHORT = """
0000000000001000 <k>:
\tv_readlane_b32 s4, v1, 3                                   // 000000001000: D2890004 00010701
\tv_readlane_b32 s5, v2, 3                                   // 000000001008: D2890005 00010702
\ts_mov_b32 m0, s9                                           // 000000001010: BEFC0009
{nop}\tglobal_load_lds_dwordx4 v3, s[4:5]                         // 000000001018: DDF48000 00040003
\ts_endpgm                                                   // 000000001020: BF810000
"""
NOP = "\ts_nop {n}                                                    // 000000001014: BF80000{n}\n"


@pytest.mark.parametrize("nop,found", [("", {1, 0}), (NOP.format(n=0), {2}), (NOP.format(n=2), {4}), (NOP.format(n=3), set())])
def test_the_search_itself(nop, found):
    (_, code), = functions(SHORT.format(nop=nop))
    assert {h[3] for h in hazards(code)} == found


def test_the_search_follows_branches():
    text = """
0000000000001000 <k>:
\tglobal_load_dword v1, v2, s[4:5]                           // 000000001000: DC508000 01040002
\ts_nop 1                                                    // 000000001008: BF800001
\tv_readfirstlane_b32 s5, v1                                 // 00000000100C: 7E0A0501
\ts_cbranch_scc0 65531                                       // 000000001010: BF84FFFB <k>
\ts_endpgm                                                   // 000000001014: BF810000
"""
    (_, code), = functions(text)
    assert [h[3] for h in hazards(code)] == [1]


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_every_kernel_keeps_its_wait_states(tmp_path):
    if not os.path.exists(gdn.LIB_PATH):
        from gated_deltanet_layer_amd import build
        build.build()
    copies, bad = 0, []
    for obj in code_objects(gdn.LIB_PATH):
        for name, code in functions(listing(obj, str(tmp_path))):
            copies += sum("_load_lds_" in op for _, op, _, _ in code)
            bad += [f"{name}+{a - code[0][0]:#x}: {ins}: {states} wait states behind {w}" for a, ins, w, states in hazards(code)]
    assert copies > 100   # the listing was understood
    assert not bad, f"{len(bad)} places:\n" + "\n".join(bad[:20])
