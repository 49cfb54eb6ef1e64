"""Launches that come up before the one in front of them has ended (launch.cuh), read from the sources.

A grid has ended when its threads have, whether or not the launch before it has. What comes next on the
stream may overwrite what that one still uses, so a kernel waits for it on every way out, also where it has nothing to
do. (The fault is a race: a kernel without the wait is not run to see it.)"""
import glob
import os
import re

import exact_scaled_dot_flash_gb300 as pkg

CSRC = os.path.join(os.path.dirname(pkg.__file__), "csrc")


def kernels(text):
    """(name, body) of each kernel of a source without comments."""
    for m in re.finditer(r"__global__ void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\))?\s*(\w+)\(", text):
        begin = i = text.index("{", m.end()) + 1
        depth = 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(1), text[begin:i - 1]


def test_a_kernel_waits_on_every_way_out():
    seen = set()
    for path in sorted(glob.glob(os.path.join(CSRC, "*prefix*.cuh")) + [os.path.join(CSRC, "attn_pages.cu")]):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for name, body in kernels(text):
            first = re.search(r"(?m)^  wait_before\(\);", body)
            if not first:  # tc_kernel and suffix_kernel wait where their stage has to, without a way out before that
                continue
            seen.add(name)
            for m in re.finditer(r"\breturn;", body[:first.start()]):
                before = body[:m.start()].rstrip()
                assert before.endswith("wait_before();"), f"{os.path.basename(path)}: {name} ends without a wait"
    assert seen == {"prefix_kernel", "join_kernel", "rows_kernel", "copy_kernel", "reserve_kernel", "compact_kernel"}
