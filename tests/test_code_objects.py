"""The gfx950 code of the built library, disassembled (CPU)."""
import os
import re
import shutil
import struct
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects():
    """The gfx950 ELF images of libmok.so, one per source file."""
    from mixture_experts_layer_stable_amd import build
    if not os.path.exists(build.LIB):
        build.build()
    blob, out, at = open(build.LIB, "rb").read(), [], 0
    while (at := blob.find(MAGIC, at)) >= 0:
        pos = at + len(MAGIC)
        n, = struct.unpack_from("<Q", blob, pos)
        pos += 8
        for _ in range(n if n < 16 else 0):   # the magic also stands in the library's own strings
            offset, size, length = struct.unpack_from("<QQQ", blob, pos)
            name = blob[pos + 24: pos + 24 + length]
            pos += 24 + length
            if b"gfx950" in name and size:
                out.append(blob[at + offset: at + offset + size])
        at += len(MAGIC)
    return out


def unwaited(text):
    """Loads into LDS that take M0 from the scalar instruction right in front of them."""
    bad, loads, kernel, before = [], 0, None, ""
    for line in text.splitlines():
        if (m := re.match(r"[0-9a-f]+ <(.*)>:", line)):
            kernel, before = m[1], ""
        elif line.startswith("\t"):
            ins = line.split("//")[0].strip()
            if re.match(r"(global|buffer|scratch)_load_lds_|buffer_load_.*\blds\b", ins):
                loads += 1
                if re.match(r"s_\w+ m0,", before):
                    bad.append((kernel, before, ins))
            before = ins
    return bad, loads


def sgprs(operand):
    m = re.match(r"s\[(\d+):(\d+)\]$|s(\d+)$", operand)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1)) if m[1] else {int(m[3])}
    return {"vcc"} if operand == "vcc" else set()


def early_addresses(text):
    """Memory instructions less than five wait states behind a vector instruction's write of an SGPR of theirs."""
    bad, count, kernel, past = [], 0, None, []
    for line in text.splitlines():
        if (m := re.match(r"[0-9a-f]+ <(.*)>:", line)):
            kernel, past = m[1], []
        elif line.startswith("\t"):
            op, _, rest = line.split("//")[0].strip().partition(" ")
            operands = [o.split(" ")[0] for o in rest.split(", ")]
            if re.match(r"(global|buffer|scratch|flat)_", op):
                count += 1
                need, states = set().union(*map(sgprs, operands)), 0
                for o, written, wait in reversed(past):
                    if states >= 5 or not need:
                        break
                    if o.startswith("v_") and need & written:
                        bad.append((kernel, o, states, op, rest))
                        break
                    need, states = need - written, states + wait
            written = sgprs(operands[0]) if op.startswith(("s_", "v_")) else set()
            if re.match(r"s_(cmp|nop|wait|branch|cbranch|barrier|bitcmp)", op):
                written = set()
            if re.match(r"v_(div_scale|\w+_co_)", op):
                written |= sgprs(operands[1])
            past = past[-7:] + [(op, written, 1 + int(operands[0]) if op == "s_nop" else 1)]
    return bad, count


def scan_all(scan, tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")

    def one(job):
        i, image = job
        p = tmp_path / ("%d.elf" % i)
        p.write_bytes(image)
        return scan(subprocess.run([OBJDUMP, "-d", str(p)], check=True, capture_output=True, text=True).stdout)

    with ThreadPoolExecutor(8) as ex:
        got = list(ex.map(one, enumerate(code_objects())))
    return [b for g in got for b in g[0]], sum(g[1] for g in got)


def test_the_scan_finds_an_adjacent_pair():
    """On a listing of its own."""
    pair = "0 <k>:\n\ts_mov_b32 m0, s2 // 0: 00\n%s\tglobal_load_lds_dwordx4 v1, s[4:5] // 8: 00\n"
    assert len(unwaited(pair % "")[0]) == 1
    assert unwaited(pair % "\ts_nop 0 // 4: 00\n") == ([], 1)


def test_loads_into_lds_wait_for_m0(tmp_path):
    """A scalar write of M0 needs one wait state before a load into LDS reads it. The compiler keeps it for its
    own loads and cannot see into inline asm, where the DMA of the matrix products is written."""
    bad, loads = scan_all(unwaited, tmp_path)
    assert loads > 1000
    assert not bad, (len(bad), bad[:3])


def test_the_scan_finds_an_early_address():
    """On a listing of its own: the write is four states ahead, moved by a scalar instruction, five ahead."""
    code = "0 <k>:\n\tv_readlane_b32 s5, v9, 3 // 0: 00\n\ts_nop %d // 4: 00\n%s\tglobal_load_lds_dwordx4 v1, %s // 8: 00\n"
    assert len(early_addresses(code % (3, "", "s[4:5]"))[0]) == 1
    assert early_addresses(code % (0, "\ts_mov_b64 s[6:7], s[4:5] // 4: 00\n", "s[6:7]")) == ([], 1)
    assert early_addresses(code % (4, "", "s[4:5]")) == ([], 1)


def test_loads_do_not_read_an_address_too_early(tmp_path):
    """A memory instruction that reads an SGPR needs five wait states behind a vector instruction's write of it. The
    compiler keeps them for its own instructions and does not see the loads of inline asm."""
    bad, loads = scan_all(early_addresses, tmp_path)
    assert loads > 10000
    assert not bad, (len(bad), bad[:3])
