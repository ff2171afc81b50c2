"""No serving kernel keeps registers in scratch memory.  The attention kernels and the tiled product are laid out to the last
register, with barriers for LDS alone and loads that are counted by hand; what a spill does between those is neither timed nor
tested, so a compiler that spills is found here, in the library as it was built, and not in a result."""
import re
import struct

import pytest

from block_wise_int8_amd import build

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def _code_objects(blob):
    """The gfx950 ELF images in a library's offload bundles (one bundle for each source)."""
    at = blob.find(MAGIC)
    while at >= 0:
        count, = struct.unpack_from("<Q", blob, at + len(MAGIC))
        entry = at + len(MAGIC) + 8
        for _ in range(count):
            offset, size, name = struct.unpack_from("<QQQ", blob, entry)
            triple = blob[entry + 24:entry + 24 + name]
            entry += 24 + name
            if triple.startswith(b"hip") and size:
                assert build.ARCH.encode() in triple
                yield blob[at + offset:at + offset + size]
        at = blob.find(MAGIC, entry)


def _kernels(elf):
    """{name: scratch bytes of a lane}, from the kernel descriptors: 64 bytes behind each symbol NAME.kd, the scratch size in
    the second word."""
    sections_at, = struct.unpack_from("<Q", elf, 0x28)
    size, count = struct.unpack_from("<HH", elf, 0x3A)
    # type, address, offset, size and link of each section
    sections = [struct.unpack_from("<4xI8xQQQI", elf, sections_at + i * size) for i in range(count)]
    found = {}
    for kind, _, offset, length, link in sections:
        if kind != 11:                                                  # dynamic symbols
            continue
        names = sections[link][2]
        for at in range(offset, offset + length, 24):
            name, section, value = struct.unpack_from("<I2xHQ", elf, at)
            text = elf[names + name:elf.index(b"\0", names + name)].decode()
            if text.endswith(".kd"):
                _, address, start, _, _ = sections[section]
                found[text[:-3]] = struct.unpack_from("<I", elf, value - address + start + 4)[0]
    return found


def scratch_of(path):
    """{kernel: scratch bytes of a lane} of a library's or an object's kernels."""
    with open(path, "rb") as f:
        blob = f.read()
    return {name: size for elf in _code_objects(blob) for name, size in _kernels(elf).items()}


def test_no_serving_kernel_spills():
    kernels = scratch_of(build.LIBRARY)
    for part, least in (("kv8_shared_kernel", 18), ("kv8_attend", 6), ("mx4_tiled", 6), ("mx4_few_rows", 6), ("norm_rotate", 18)):
        assert sum(part in name for name in kernels) >= least, part
    spilled = {name: size for name, size in kernels.items() if re.search(r"kv8|mx4|rotate", name) and size}
    assert not spilled
