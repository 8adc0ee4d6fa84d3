"""The two-stage tiles of 128 x 128 (csrc/block_shape.h's middle ones) are chosen as two
workgroups of four waves a compute unit: 256 of a SIMD's 512 registers and half of its 160
KB of shared memory each.  Read from the kernels' metadata in the built library."""

import os
import re
import struct

import pytest

msgpack = pytest.importorskip("msgpack")


def section(elf, name):
    """(offset, size) of a section of a 64-bit ELF image."""
    shoff, = struct.unpack_from("<Q", elf, 40)
    size, num, names = struct.unpack_from("<HHH", elf, 58)
    heads = [struct.unpack_from("<IIQQQQ", elf, shoff + i * size) for i in range(num)]
    strings = heads[names][4]
    for h in heads:
        start = strings + h[0]
        if elf[start:elf.index(b"\0", start)] == name:
            return h[4], h[5]
    return None


def code_objects(lib):
    """The gfx950 images of the bundles in a library's .hip_fatbin."""
    off, size = section(lib, b".hip_fatbin")
    magic = b"__CLANG_OFFLOAD_BUNDLE__"
    at = lib.find(magic, off, off + size)
    while at >= 0:
        entries, = struct.unpack_from("<Q", lib, at + len(magic))
        pos = at + len(magic) + 8
        for _ in range(entries):
            start, length, chars = struct.unpack_from("<QQQ", lib, pos)
            target = lib[pos + 24:pos + 24 + chars]
            pos += 24 + chars
            if b"gfx950" in target and length:
                yield lib[at + start:at + start + length]
        at = lib.find(magic, pos, off + size)


def kernels(image):
    off, size = section(image, b".note")
    name, desc, _ = struct.unpack_from("<III", image, off)
    start = off + 12 + (name + 3) // 4 * 4
    return msgpack.unpackb(image[start:start + desc])["amdhsa.kernels"]


def test_middle_tiles_hold_two_workgroups():
    import token_routing_amd as mg
    if not os.path.exists(mg.LIB_PATH):
        from token_routing_amd import build
        build.build()
    with open(mg.LIB_PATH, "rb") as f:
        lib = f.read()
    found = set()
    for image in code_objects(lib):
        for k in kernels(image):
            m = re.search(r"(block_fwd|gated_bwd)_kernelINS_7RingCfgILi128ELi128ELi2ELi2ELb[01]"
                          r"ELi64ELi2E", k[".name"])
            if m:
                found.add(m.group(1))
                assert k[".vgpr_count"] <= 256, k[".name"]
                assert k[".group_segment_fixed_size"] <= 80 << 10, k[".name"]
    assert found == {"block_fwd", "gated_bwd"}
