"""Dynamic shared memory declared as bytes holds vectors and tiles: it says its alignment, or the
kernel rounds its address up (CPU only: the sources are read)."""
import glob
import os
import re

from mixture_experts_forward_moe_gb300 import build


def test_dynamic_shared_memory_of_bytes_is_aligned():
    seen = 0
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cu"))):
        with open(path, encoding="utf-8") as f:
            text = f.read()
        for m in re.finditer(r"extern\s+__shared__\s+([^;]*\buint8_t\s+(\w+)\[\]);", text):
            seen += 1
            said = re.search(r"__align__\((\d+)\)", m.group(1))
            rounded = f"{m.group(2)} + ((1024u - (raw & 1023u)) & 1023u)" in text[m.end():]
            assert rounded or (said and int(said.group(1)) >= 16), (os.path.basename(path), m[0])
    assert seen >= 6
