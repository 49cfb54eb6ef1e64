"""Bounded waits of the 8-bit attention kernels, read from their sources.

A wait that a whole warp takes may run out for some of its lanes and not for others, and the code
behind it holds instructions that all lanes execute together. So its lanes vote before they part:
``warp_wait``, or ``mbar_wait`` whose result a vote follows. (Such a wait cannot be made to run out on
a GPU without a kernel that is broken on purpose.)"""
import glob
import os
import re

import exact_scaled_dot_flash_gb300 as pkg

CSRC = os.path.join(os.path.dirname(pkg.__file__), "csrc")


def test_a_warp_leaves_a_wait_together():
    waits = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "attn_kv8*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\bmbar_wait\(", text):
            line = text[text.rfind("\n", 0, m.start()) + 1:m.start()]
            name = re.match(r"\s*const bool (\w+) = $", line)
            behind = text[text.index(";", m.start()) + 1:].lstrip()
            assert name and behind.startswith(f"if (__any_sync(0xffffffffu, !{name.group(1)}))"), \
                f"{os.path.basename(path)}: a wait without a vote: {line.strip()} mbar_wait(...)"
            waits += 1
        waits += len(re.findall(r"\bwarp_wait\(", text))
    assert waits >= 8  # the sources were read
