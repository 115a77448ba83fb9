"""The built code of kernels whose last workgroup reads what the others stored:
what the instructions wait for, which no run on a GPU shows for certain."""
import os
import re
import struct
import subprocess

import pytest

from software_pipelined_tiled_pgemm_amd import _lib, build

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(data):
    """The gfx950 code objects of a library's offload bundles."""
    at = data.find(MAGIC)
    while at >= 0:
        (count,) = struct.unpack_from("<Q", data, at + 24)
        entry = at + 32
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, entry)
            if b"gfx950" in data[entry + 24:entry + 24 + length] and size:
                yield data[at + offset:at + offset + size]
            entry += 24 + length
        at = data.find(MAGIC, at + 24)


def kernels(tmp_path, name):
    """(symbol, instructions) of the kernels whose symbols hold `name`."""
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    with open(_lib.LIB_PATH, "rb") as f:
        data = f.read()
    for i, code in enumerate(c for c in code_objects(data) if name.encode() in c):
        path = tmp_path / ("%d.co" % i)
        path.write_bytes(code)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", str(path)],
                              capture_output=True, text=True, check=True).stdout
        parts = re.split(r"^[0-9a-f ]*<(\S+)>:$", text, flags=re.M)
        for symbol, body in zip(parts[1::2], parts[2::2]):
            if name in symbol:
                lines = [ln.split("//")[0].strip() for ln in body.splitlines()]
                yield symbol, [ln for ln in lines if ln]


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no disassembler")
def test_stores_are_done_before_the_workgroup_is_counted(tmp_path):
    """One lane counts its workgroup after a barrier.  The barrier waits for no store to
    memory, and the lane's release for those of its own wave: so each wave has to
    wait for its own before the barrier."""
    found = 0
    for symbol, code in kernels(tmp_path, "piece_gather_kernel"):
        releases = [i for i, ins in enumerate(code) if ins.startswith("buffer_wbl2")]
        assert releases, symbol
        for at in releases:
            barrier = max(i for i in range(at) if code[i].startswith("s_barrier"))
            waits = []
            for ins in reversed(code[:barrier]):
                if ins.startswith(("global_", "flat_", "buffer_", "s_barrier", "s_cbranch", "s_branch")):
                    break
                waits.append(ins)
            assert any(w.startswith("s_waitcnt") and "vmcnt(0)" in w for w in waits), (symbol, at)
            found += 1
    assert found >= 3  # fp32, fp16, bf16
