"""Registers that the built kernels spill, from the metadata of the code objects in libgeg.so
(built here from source). A second variant of a kernel in the same unit can cost the first ones
registers without a word from the compiler; these are the counts that the plain dgrad kernels had
before they got a variant for adapter dropout."""
import os
import re
import struct
import subprocess

import pytest

import grouped_expert_gemm_amd as geg

READELF = "/opt/rocm/llvm/bin/llvm-readelf"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def _kernels(path, tmp):
    """{kernel name: (spilled vector registers, bytes of scratch per lane)} of a library."""
    data = open(path, "rb").read()
    out = {}
    for start in (m.start() for m in re.finditer(re.escape(MAGIC), data)):
        at = start + len(MAGIC)
        (entries,) = struct.unpack_from("<Q", data, at)
        at += 8
        for _ in range(entries):
            offset, size, length = struct.unpack_from("<QQQ", data, at)
            name = data[at + 24:at + 24 + length]
            at += 24 + length
            if b"gfx950" not in name or size == 0:
                continue
            obj = tmp / "object"
            obj.write_bytes(data[start + offset:start + offset + size])
            notes = subprocess.run([READELF, "--notes", str(obj)], capture_output=True, text=True, check=True).stdout
            for k in re.split(r"\n  - \.a", notes)[1:]:
                fields = dict(re.findall(r"^\s+\.(\w+):\s+(\S+)$", k, re.M))
                out[fields["name"]] = (int(fields["vgpr_spill_count"]), int(fields["private_segment_fixed_size"]))
    return out


@pytest.mark.skipif(not os.path.exists(READELF), reason="no llvm-readelf")
def test_plain_dgrad_kernels_keep_their_registers(tmp_path):
    geg.lib()
    kernels = _kernels(geg.LIB_PATH, tmp_path)
    # tile_kernel<format, dgrad, tail, masked>: format 0 NF4, 1 MXFP4
    for fmt, tail, spills, scratch in ((1, 0, 0, 0), (1, 1, 4, 20), (0, 0, 76, 308), (0, 1, 83, 336)):
        found = [v for n, v in kernels.items() if re.search(rf"11tile_kernelILNS_3FmtE{fmt}ELb1ELb{tail}ELb0EE", n)]
        assert len(found) == 1
        assert found[0][0] <= spills and found[0][1] <= scratch, (fmt, tail, found[0])
