"""The built library's loads straight to LDS keep the distance from what writes their
scalar operands: gfx950 needs five wait states between a VALU write of a scalar register
and a vector memory access that reads it.  The compiler keeps it for the instructions it
makes, but does not look into inline assembly."""
import os
import re
import shutil
import struct
import subprocess

import pytest

from mxfp8_grouped_gemm_group_amd import build_lib

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
NEEDED = 5


def code_objects(path):
    """The gfx950 code objects in the library, one to a source file."""
    with open(path, "rb") as f:
        data = f.read()
    at = data.find(MAGIC)
    while at >= 0:
        (entries,), p = struct.unpack_from("<Q", data, at + 24), at + 32
        for _ in range(entries):
            offset, size, name = struct.unpack_from("<QQQ", data, p)
            if size and data[p + 24:p + 24 + name].endswith(b"gfx950"):
                yield data[at + offset:at + offset + size]
            p += 24 + name
        at = data.find(MAGIC, at + len(MAGIC))


def scalars(text):
    """The scalar registers an operand text names."""
    out = {int(n) for n in re.findall(r"\bs(\d+)\b", text)}
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        out.update(range(int(a), int(b) + 1))
    return out


def too_close(lines):
    """(loads straight to LDS, those that read a scalar register written by a vector
    instruction fewer than NEEDED states before)."""
    loads, close, kernel, before = 0, [], "", []
    for line in lines:
        if line.endswith(">:"):
            kernel = line
        code = line.split("//")[0].strip()
        if not line.startswith("\t") or not code:
            continue
        op, _, rest = code.partition(" ")
        if op.startswith("buffer_load") and " lds" in rest:
            loads += 1
            reads, states = scalars(rest), 0
            for earlier, args in reversed(before):
                if states >= NEEDED:
                    break
                if earlier.startswith("v_") and scalars(args.split(",")[0]) & reads:
                    close.append((kernel, earlier + " " + args, code, states))
                states += int(args, 0) + 1 if earlier == "s_nop" else 1
        before = before[-8:] + [(op, rest)]
    return loads, close


def test_the_reader_sees_a_short_distance():
    text = ["<k>:", "\tv_readfirstlane_b32 s10, v4 // 0", "\ts_mov_b32 m0, s4", "\ts_nop {}",
            "\tbuffer_load_dwordx4 v1, s[8:11], s3 offen lds // 0"]
    assert len(too_close([t.format(0) for t in text])[1]) == 1
    assert len(too_close([t.format(2) for t in text])[1]) == 1
    assert too_close([t.format(3) for t in text]) == (1, [])
    assert too_close([t.format(0).replace("s10", "s12") for t in text]) == (1, [])


@pytest.mark.skipif(not shutil.which(OBJDUMP), reason="no llvm-objdump")
def test_loads_to_lds_wait_for_their_scalar_operands(tmp_path):
    if not os.path.exists(build_lib.LIB):
        build_lib.build()
    loads = 0
    for i, code in enumerate(code_objects(build_lib.LIB)):
        path = tmp_path / f"{i}.o"
        path.write_bytes(code)
        run = subprocess.run([OBJDUMP, "-d", str(path)], capture_output=True, text=True, check=True)
        n, close = too_close(run.stdout.split("\n"))
        assert not close, f"{len(close)} of {n} loads, first {close[:3]}"
        loads += n
    assert loads > 500
