"""Where LDS that is sized at the launch begins: behind the kernel's own, which its metadata in the built library gives. The layer for a few
tokens and the choice of experts go through it sixteen bytes at a time."""
import struct

import pytest

import mx_block_scaled_amax_amd as qf8

msgpack = pytest.importorskip("msgpack")


def code_objects(lib):
    """The gfx950 code objects of a library built by hipcc: bundles of (offset, size, name) entries."""
    magic, at = b"__CLANG_OFFLOAD_BUNDLE__", lib.find(b"__CLANG_OFFLOAD_BUNDLE__")
    while at >= 0:
        entry = at + len(magic) + 8
        for _ in range(struct.unpack_from("<Q", lib, at + len(magic))[0]):
            offset, size, length = struct.unpack_from("<QQQ", lib, entry)
            if b"gfx950" in lib[entry + 24:entry + 24 + length]:
                yield lib[at + offset:at + offset + size]
            entry += 24 + length
        at = lib.find(magic, at + 1)


def kernels(elf):
    """The kernels' metadata: the AMDGPU note (type 32) of a 64-bit ELF file."""
    table, = struct.unpack_from("<Q", elf, 32)
    size, count = struct.unpack_from("<HH", elf, 54)
    for i in range(count):
        kind, = struct.unpack_from("<I", elf, table + i * size)
        offset, = struct.unpack_from("<Q", elf, table + i * size + 8)
        length, = struct.unpack_from("<Q", elf, table + i * size + 32)
        at = offset if kind == 4 else offset + length        # PT_NOTE
        while at < offset + length:
            name, desc, note = struct.unpack_from("<III", elf, at)
            start = at + 12 + (name + 3) // 4 * 4
            if note == 32:
                return msgpack.unpackb(elf[start:start + desc])["amdhsa.kernels"]
            at = start + (desc + 3) // 4 * 4
    return []


@pytest.mark.parametrize("name,least", [("layer_down_kernel", 4), ("route", 1)])
def test_launch_sized_lds_is_aligned(name, least):
    qf8._load()
    with open(qf8._LIB_PATH, "rb") as f:
        sizes = {k[".name"]: k[".group_segment_fixed_size"] for elf in code_objects(f.read()) for k in kernels(elf) if name in k[".name"]}
    assert len(sizes) >= least
    assert not {k: v for k, v in sizes.items() if v % 16}
