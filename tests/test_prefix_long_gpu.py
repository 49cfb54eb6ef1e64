"""Shared prefixes of many key blocks on the GPU (attn_paged_prefix_fwd): CTAs that go through several
blocks, units and groups, row blocks of every height, few slots for the parts of a row, and the page
sizes of the tcgen05 kernel. Against 64 bits on the GPU (each sequence by its own row; the tolerances are
pages_ref.near's), in the normal and in the bounds-checked build."""
import math

import numpy as np
import pytest

from tests.gpu_util import to_f64
from tests.pages_ref import Shared, near
from tests.test_guard_bands_gpu import checked_path  # noqa: F401
from tests.test_prefix_gpu import ones

pytestmark = pytest.mark.gpu


def reference(b, d, positions=None, causal=True, scale=None):
    """pages_ref.attention's results for a batch whose table names pages of the cache wherever a sequence
    holds tokens, by products in 64 bits on the GPU."""
    import torch
    q, kc, vc = d[:3]
    scale = b.D ** -0.5 if scale is None else scale
    n, Hq, D = q.shape
    heads = Hq // b.H
    out, mass = (torch.zeros((n, Hq, D), dtype=torch.float64, device="cuda") for _ in range(2))
    lse, noise = (torch.zeros((n, Hq), dtype=torch.float64, device="cuda") for _ in range(2))
    for s, L in enumerate(b.lens.tolist()):
        lo, hi = int(b.offs[s]), int(b.offs[s + 1])
        if lo == hi:
            continue
        j = torch.arange(L, device="cuda")
        page = d[3][s, j // b.P].long()
        k, v = (x[page, j % b.P].double() for x in (kc, vc))  # [L, H, D]
        pos = (torch.from_numpy(positions[lo:hi]).cuda().long() if positions is not None
               else torch.arange(L - (hi - lo), L, device="cuda"))
        seen = (j <= pos[:, None]) if causal else torch.ones((hi - lo, L), dtype=torch.bool, device="cuda")
        none = ~seen.any(1)
        for h in range(b.H):
            at = slice(h * heads, (h + 1) * heads)
            x = q[lo:hi, at].double()
            s_ = torch.einsum("ihd,jd->ihj", x, k[:, h]) * scale
            size = torch.einsum("ihd,jd->ihj", x.abs(), k[:, h].abs()) * scale
            noise[lo:hi, at] = size.masked_fill(~seen[:, None], 0.0).amax(2)
            s_ = s_.masked_fill(~seen[:, None], -math.inf)
            l = torch.logsumexp(s_, 2)
            lse[lo:hi, at] = l
            p = torch.exp(s_ - l[..., None])
            out[lo:hi, at] = torch.einsum("ihj,jd->ihd", p, v[:, h])
            mass[lo:hi, at] = torch.einsum("ihj,jd->ihd", p, v[:, h].abs())
        out[lo:hi][none] = math.nan
    return tuple(x.cpu().numpy() for x in (out, lse, mass, noise))


def check_both(b, checked, positions=None, causal=True, scale=None):
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    d = b.device()
    ref = reference(b, d, positions, causal, scale)
    pos = torch.from_numpy(positions).cuda() if positions is not None else None
    kw = dict(positions=pos, causal=causal, scale=scale, return_lse=True, max_queries=b.max_q, max_group_queries=b.max_gq)
    got = []
    for path in (None, checked):
        if path is None:
            got.append(attn.paged_prefix_fwd(*d, **kw))
            assert attn.device_status(0, clear=True) == 0
        else:
            with attn.use_library(path):
                got.append(attn.paged_prefix_fwd(*d, **kw))
                torch.cuda.synchronize()
                assert attn.device_status(0, clear=True) == 0
        near(to_f64(got[-1][0]), to_f64(got[-1][1]), ref, b.dtype, b.D)
    for x, y in zip(*got):  # the checks change no arithmetic
        assert torch.equal(x, y)


# Many rows: 8 kv heads of 4 heads; blocks of 256 rows and 128 keys, shared out over 152 CTAs
MANY = {
    # 800 rows (three row blocks and one of 32), 160 (one block of more than 128), 40 and 256 (whole)
    "unequal": [(9001, ones(25, 8, 60, new=8)), (4100, ones(5, 8, 40, new=8)), (None, ones(2, 30, 300)),
                (19999, ones(10, 1, 30)), (300, ones(64, 1, 200))],
    "one_group": [(20001, ones(12, 1, 40, new=3))],
    # their own keys on the tcgen05 kernel as well
    "prompts": [(9001, [(80, 70), (33, 33), (129, 128)]), (5000, [(10, 10)]), (12345, [(200, 190)]), (None, [(700, 650)])],
    # rows that leave room for two parts and for three
    "two_parts": [(4000, ones(16, 100, 140, new=100))],
    "three_parts": [(2000, ones(5, 100, 140, new=100)), (5003, ones(7, 100, 300, new=100))],
}
# Few rows: 8 kv heads of one head; blocks of 32 keys, shared out over some 900 CTAs
FEW = {
    "unequal": [(20000, ones(10)), (9001, ones(32)), (517, ones(3)), (33333, [(5, 1)]), (None, ones(2, 3000, 9000))],
    "eight": [(30000, ones(8)), (12345, ones(3)), (64, ones(2)), (7001, ones(7, 1, 2000))],
    "sixteen": [(15001, ones(16)), (22222, ones(11, 1, 300))],
    "drafts": [(25000, ones(6, 4, 60, new=4)), (11111, ones(2, 4, 3000, new=3))],
}


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("name", MANY)
def test_many_rows(name, dtype, D, checked_path):  # noqa: F811
    b = Shared(71, MANY[name], dtype=dtype, D=D, P=64, H=8, Hq=32)
    check_both(b, checked_path)


@pytest.mark.parametrize("name", ["unequal", "prompts"])
def test_many_rows_at_positions(name, checked_path):  # noqa: F811
    # a row may see any part of the prefix, none of it, or everything
    b = Shared(73, MANY[name], dtype="bf16", D=128, P=64, H=8, Hq=32)
    pos = np.random.RandomState(2).randint(-2, 22000, len(b.q)).astype(np.int32)
    check_both(b, checked_path, pos)
    check_both(b, checked_path, causal=False, scale=0.2)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("name", FEW)
def test_few_rows(name, dtype, D, checked_path):  # noqa: F811
    b = Shared(79, FEW[name], dtype=dtype, D=D, P=16, H=8, Hq=8)
    check_both(b, checked_path)
    check_both(b, checked_path, np.random.RandomState(3).randint(0, 34000, len(b.q)).astype(np.int32))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("P", [8, 16, 32, 128, 256, 384])
@pytest.mark.parametrize("name", ["unequal", "prompts"])
def test_page_sizes(name, P, dtype, D, checked_path):  # noqa: F811
    groups = {"unequal": [(1500, ones(25, 8, 60, new=8)), (None, ones(2, 30, 300)), (733, ones(10, 8, 900, new=6))],
              "prompts": [(901, [(80, 70), (300, 300)]), (500, [(10, 10)])]}[name]
    b = Shared(83, groups, dtype=dtype, D=D, P=P, H=2, Hq=8)
    check_both(b, checked_path)


@pytest.mark.parametrize("dtype,D,new", [("bf16", 128, 20), ("f16", 64, 1), ("f32", 128, 2)])
def test_a_cache_past_32_bits(dtype, D, new, checked_path):  # noqa: F811
    # the batch's pages are the last of a cache of more than 2^32 elements
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    b = Shared(127, [(700, ones(5, new, 300, new=new))], dtype=dtype, D=D, P=64, H=8, Hq=32, hidden=0.0)
    d = list(b.device())
    kw = dict(max_queries=b.max_q, max_group_queries=b.max_gq, return_lse=True)
    ref = reference(b, d)
    n = len(b.kc)
    pages = (1 << 32) // (b.P * b.H * D) + n
    for i in (1, 2):
        big = torch.zeros((pages, b.P, b.H, D), dtype=d[i].dtype, device="cuda")
        big[pages - n:] = d[i]
        d[i] = big
    d[3] = torch.where(d[3] >= 0, d[3] + (pages - n), d[3])
    for path in (None, checked_path):
        if path is None:
            out, lse = attn.paged_prefix_fwd(*d, **kw)
        else:
            with attn.use_library(path):
                out, lse = attn.paged_prefix_fwd(*d, **kw)
                torch.cuda.synchronize()
                assert attn.device_status(0, clear=True) == 0
        near(to_f64(out), to_f64(lse), ref, b.dtype, b.D)


def test_calls_on_several_streams_at_once():
    # calls with few and with many rows, each stream its own workspaces: the same bits as one after another
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    batches = [Shared(131, g, dtype="bf16", D=128, P=64, H=8, Hq=32)
               for g in (MANY["one_group"], MANY["prompts"], [(3000, ones(60, 1, 900))], [(500, ones(3)), (None, ones(2, 9, 80))])]
    d = [b.device() for b in batches]
    kw = [dict(max_queries=b.max_q, max_group_queries=b.max_gq, return_lse=True) for b in batches]
    want = [attn.paged_prefix_fwd(*x, **k) for x, k in zip(d, kw)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    got = []
    for i in range(24):
        s = streams[i % 4]
        which = (i * 3 + i // 4) % 4
        with torch.cuda.stream(s):
            got.append((which, attn.paged_prefix_fwd(*d[which], **kw[which])))
    torch.cuda.synchronize()
    for which, x in got:
        assert torch.equal(x[0], want[which][0]) and torch.equal(x[1], want[which][1])
    assert attn.device_status(0, clear=True) == 0
