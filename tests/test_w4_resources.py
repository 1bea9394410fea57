"""What the compiler made of the 4-bit kernels, from the metadata of the built library (no GPU)."""
import os
import re
import struct

import pytest

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def _metadata(elf):
    """The AMDGPU metadata note of a code object."""
    import msgpack
    shoff, = struct.unpack_from("<Q", elf, 0x28)
    size, count = struct.unpack_from("<HH", elf, 0x3A)
    for i in range(count):
        at = shoff + i * size
        if struct.unpack_from("<I", elf, at + 4)[0] != 7:  # SHT_NOTE
            continue
        off, length = struct.unpack_from("<QQ", elf, at + 24)
        end = off + length
        while off < end:
            name, desc, kind = struct.unpack_from("<III", elf, off)
            off += 12
            start = off + (name + 3) // 4 * 4
            if kind == 32 and elf[off:off + 6] == b"AMDGPU":
                return msgpack.unpackb(elf[start:start + desc], strict_map_key=False)
            off = start + (desc + 3) // 4 * 4
    raise AssertionError("no metadata")


@pytest.fixture(scope="module")
def kernels():
    """{mangled name: metadata} of every gfx950 kernel of the library."""
    pytest.importorskip("msgpack")
    from skinny_gemm_qlin_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from skinny_gemm_qlin_amd import _build
        _build.build()
    with open(_lib.LIB_PATH, "rb") as f:
        data = f.read()
    out = {}
    for m in re.finditer(re.escape(MAGIC), data):
        at, (n,) = m.start() + len(MAGIC) + 8, struct.unpack_from("<Q", data, m.start() + len(MAGIC))
        for _ in range(n):
            off, size, name = struct.unpack_from("<QQQ", data, at)
            target = data[at + 24:at + 24 + name]
            at += 24 + name
            if b"gfx950" in target and size:
                blob = data[m.start() + off:m.start() + off + size]
                out.update({k[".name"]: k for k in _metadata(blob)["amdhsa.kernels"]})
    return out


def test_decode_kernels_keep_nothing_in_private_memory(kernels):
    """Private memory's loads queue behind the weights' and are waited for with them."""
    few = [k for n, k in kernels.items() if "w4_few_kernel" in n]
    assert len(few) == 116 and not any(k[".private_segment_fixed_size"] for k in few)


def test_mid_kernels_keep_nothing_in_private_memory(kernels):
    mid = [k for n, k in kernels.items() if "w4_mid_kernel" in n]
    assert len(mid) == 54 and not any(k[".private_segment_fixed_size"] for k in mid)
