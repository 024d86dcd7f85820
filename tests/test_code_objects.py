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


def test_the_scan_finds_an_adjacent_pair():
    """On a listing of its own."""
    pair = "0 <k>:\n\ts_mov_b32 m0, s2 // 0: 00\n%s\tglobal_load_lds_dwordx4 v1, s[4:5] // 8: 00\n"
    assert len(unwaited(pair % "")[0]) == 1
    assert unwaited(pair % "\ts_nop 0 // 4: 00\n") == ([], 1)


def test_loads_into_lds_wait_for_m0(tmp_path):
    """A scalar write of M0 needs one wait state before a load into LDS reads it. The compiler keeps it for its
    own loads and cannot see into inline asm, where the DMA of the matrix products is written."""
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")

    def scan(job):
        i, image = job
        p = tmp_path / ("%d.elf" % i)
        p.write_bytes(image)
        return unwaited(subprocess.run([OBJDUMP, "-d", str(p)], check=True, capture_output=True, text=True).stdout)

    with ThreadPoolExecutor(8) as ex:
        got = list(ex.map(scan, enumerate(code_objects())))
    bad = [b for g in got for b in g[0]]
    assert sum(g[1] for g in got) > 1000
    assert not bad, (len(bad), bad[:3])
