"""Which kernel takes a call of attn_paged_kv8_fwd, told by its workspace: the kernel for few rows cuts
sequences of more than 512 keys and needs one; the kernel for many rows needs one for runs of keys only."""
import ctypes

import pytest

from exact_scaled_dot_flash_gb300 import attn as A
from tests.test_boundary import lib  # noqa: F401


def workspace(num_seqs, heads, max_queries, keys, Hkv=4, page=64, D=128):
    n = ctypes.c_size_t(7)
    s = A.PagedShape(num_seqs, num_seqs * max_queries, Hkv * heads, Hkv, D, page, num_seqs * keys // page, keys // page,
                     max_queries)
    assert A.load_library().attn_paged_kv8_workspace_bytes(s, n) == 0
    return n.value


@pytest.mark.parametrize("seqs", [20, 24, 30, 36, 37])
def test_50_rows_of_sequences_that_are_not_cut(lib, seqs):  # noqa: F811
    # 80 to 148 CTAs of 256 rows: over at most 3.5k keys those of the kernel for many rows, whole; over
    # 7.9k keys the other kernel, where they are few
    assert workspace(seqs, 10, 5, 3520) == 0
    assert workspace(seqs, 10, 5, 2048) == 0
    assert (workspace(seqs, 10, 5, 7936) > 0) == (seqs <= 30)


def test_few_rows_share_out_the_keys(lib):  # noqa: F811
    assert workspace(30, 1, 1, 3520) > 0 and workspace(30, 8, 5, 3520) > 0
    assert workspace(30, 8, 1, 512) == 0
