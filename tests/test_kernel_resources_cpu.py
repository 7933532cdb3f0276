"""The kernels of the 4-bit products, the gated projection and the clipping hold
their sums in registers: none of the built library's has memory of its own per lane
(a tile whose sums the compiler moves there is over ten times slower, and right)."""
import re
import struct

import pytest

from matmul_pack_b1_amd import binding as hb

msgpack = pytest.importorskip("msgpack")

BUNDLE = b"__CLANG_OFFLOAD_BUNDLE__"
NOTE, METADATA = 7, 32   # SHT_NOTE, NT_AMDGPU_METADATA
NAMES = re.compile(r"k_(q4|gated|clip|gemv_gated)")


def code_objects(path):
    """The gfx950 ELF images of a library."""
    with open(path, "rb") as f:
        blob = f.read()
    at = blob.find(BUNDLE)
    while at >= 0:
        count, = struct.unpack_from("<Q", blob, at + 24)
        p = at + 32
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", blob, p)
            name = blob[p + 24:p + 24 + length]
            p += 24 + length
            if b"gfx950" in name and size:
                yield blob[at + offset:at + offset + size]
        at = blob.find(BUNDLE, at + 24)


def kernels(elf):
    """What the image's metadata says of each kernel."""
    assert elf[:4] == b"\x7fELF"
    sections, = struct.unpack_from("<Q", elf, 0x28)
    each, count = struct.unpack_from("<HH", elf, 0x3A)
    for i in range(count):
        _, kind, _, _, at, size = struct.unpack_from("<IIQQQQ", elf, sections + i * each)
        end = at + size if kind == NOTE else at
        while at < end:
            name, length, note = struct.unpack_from("<III", elf, at)
            at += 12 + -(-name // 4) * 4
            if note == METADATA:
                yield from msgpack.unpackb(elf[at:at + length])["amdhsa.kernels"]
            at += -(-length // 4) * 4


def test_no_kernel_keeps_registers_in_memory():
    seen, bad = 0, []
    for elf in code_objects(hb.LIB_PATH):
        for k in kernels(elf):
            if NAMES.search(k[".name"]):
                seen += 1
                if k[".private_segment_fixed_size"] or k[".vgpr_spill_count"]:
                    bad.append((k[".name"], k[".private_segment_fixed_size"], k[".vgpr_spill_count"]))
    assert seen > 100
    assert not bad, bad
