"""Refusals and host-side rules of the pages of a cache, of attention of sequences that share a prefix
and of rotary positions with axes, without a GPU (made-up addresses as in test_kv8_rope_boundary.py)."""
import ctypes
import math

import numpy as np
import pytest

from exact_scaled_dot_flash_gb300 import attn as A
from tests import pages_ref as R
from tests.test_boundary import codes, lib, no_gpu_only  # noqa: F401

FAR = 1 << 44
I3 = ctypes.c_int64 * 3


def bufs(*b):
    """(address, bytes of a page) pairs as the calls take them."""
    n = len(b)
    return (ctypes.c_void_p * n)(*[x for x, _ in b]), (ctypes.c_int64 * n)(*[y for _, y in b]), n


def pool(num_seqs=4, max_pages=3, page_size=16, num_pages=9):
    return A.Pages(num_seqs, max_pages, page_size, num_pages)


TWO = ((10 * FAR, 4096), (11 * FAR, 100))


def copy(pages=9, b=TWO, src=FAR, dst=2 * FAR, n=5):
    return A.load_library().attn_pages_copy(pages, *bufs(*b), src, dst, n, None)


def fork(p=None, table=FAR, lens=2 * FAR, refs=3 * FAR, parents=4 * FAR, kids=5 * FAR, n=2):
    return A.load_library().attn_pages_fork(p or pool(), table, lens, refs, parents, kids, n, None)


def free(p=None, table=FAR, lens=2 * FAR, refs=3 * FAR, seqs=4 * FAR, n=2):
    return A.load_library().attn_pages_free(p or pool(), table, lens, refs, seqs, n, None)


def reserve(p=None, table=FAR, lens=2 * FAR, refs=3 * FAR, new=4 * FAR, b=TWO, result=5 * FAR, ws=6 * FAR, wsb=1 << 40):
    return A.load_library().attn_pages_reserve(p or pool(), table, lens, refs, new, *bufs(*b), result, ws, wsb, None)


def compact(p=None, table=FAR, refs=3 * FAR, b=TWO, to=4 * FAR, used=5 * FAR, ws=6 * FAR, wsb=1 << 40):
    return A.load_library().attn_pages_compact(p or pool(), table, refs, *bufs(*b), to, used, ws, wsb, None)


def err(name):
    return codes["ATTN_ERR_" + name]


BAD_POOLS = [dict(num_seqs=-1), dict(max_pages=-1), dict(page_size=0), dict(num_pages=-1),
             dict(max_pages=1 << 28), dict(num_seqs=1 << 30), dict(num_seqs=1, max_pages=(1 << 24) + 1, page_size=1)]


@no_gpu_only
@pytest.mark.parametrize("kw", BAD_POOLS)
def test_bad_pools(lib, kw):  # noqa: F811
    p = pool(**kw)
    n = ctypes.c_size_t()
    assert lib.attn_pages_workspace_bytes(p, n) == err("SHAPE")
    assert [f(p) for f in (fork, free, reserve, compact)] == [err("SHAPE")] * 4


@no_gpu_only
@pytest.mark.parametrize("kw,e", [
    (dict(n=-1), "SHAPE"), (dict(pages=-1), "SHAPE"), (dict(src=None), "NULL"), (dict(dst=None), "NULL"),
    (dict(src=FAR + 2), "ALIGN"), (dict(b=((10 * FAR, 0),)), "SHAPE"), (dict(b=((10 * FAR, -16),)), "SHAPE"),
    (dict(b=((None, 16),)), "NULL"), (dict(b=((10 * FAR, 1 << 41),)), "SHAPE"),
    (dict(pages=(1 << 31) - 1, b=((10 * FAR, 1 << 40),)), "SHAPE"),
    (dict(b=((10 * FAR, 16), (10 * FAR + 143, 16))), "OVERLAP"), (dict(b=((11 * FAR, 16), (11 * FAR - 143, 16))), "OVERLAP"),
    (dict(b=((FAR - 140, 16),)), "OVERLAP"), (dict(b=tuple(((20 + i) * FAR, 16) for i in range(1025))), "SHAPE")])
def test_copy_refusals(lib, kw, e):  # noqa: F811
    assert copy(**kw) == err(e)


@no_gpu_only
@pytest.mark.parametrize("kw,e", [
    (dict(n=-1), "SHAPE"), (dict(table=None), "NULL"), (dict(lens=None), "NULL"), (dict(refs=None), "NULL"),
    (dict(kids=None), "NULL"), (dict(parents=None), "NULL"), (dict(kids=5 * FAR + 1), "ALIGN"),
    (dict(refs=FAR + 44), "OVERLAP"), (dict(parents=2 * FAR + 12), "OVERLAP"), (dict(kids=3 * FAR + 32), "OVERLAP")])
def test_fork_refusals(lib, kw, e):  # noqa: F811
    assert fork(**kw) == err(e)
    if "parents" not in kw:
        kw = {"seqs" if k == "kids" else k: v for k, v in kw.items()}
        assert free(**kw) == err(e)


@no_gpu_only
@pytest.mark.parametrize("kw,e", [
    (dict(table=None), "NULL"), (dict(refs=None), "NULL"), (dict(ws=None), "WORKSPACE"), (dict(wsb=100), "WORKSPACE"),
    (dict(ws=6 * FAR + 4), "ALIGN"), (dict(refs=3 * FAR + 2), "ALIGN"), (dict(ws=FAR), "OVERLAP"),
    (dict(refs=FAR + 16), "OVERLAP"), (dict(b=((6 * FAR, 16),)), "OVERLAP"), (dict(b=((3 * FAR - 16, 16),)), "OVERLAP")])
def test_plan_refusals(lib, kw, e):  # noqa: F811
    assert reserve(**kw) == err(e)
    assert compact(**kw) == err(e)


@no_gpu_only
def test_plan_refusals_of_one_call(lib):  # noqa: F811
    for f, kw, e in ((reserve, dict(lens=None), "NULL"), (reserve, dict(new=None), "NULL"), (reserve, dict(result=None), "NULL"),
                     (reserve, dict(result=4 * FAR + 8), "OVERLAP"), (reserve, dict(new=5 * FAR + 4), "OVERLAP"),
                     (compact, dict(to=None), "NULL"), (compact, dict(used=None), "NULL"),
                     (compact, dict(used=4 * FAR + 32), "OVERLAP"), (compact, dict(to=3 * FAR), "OVERLAP")):
        assert f(**kw) == err(e), kw
    n = ctypes.c_size_t()
    assert lib.attn_pages_workspace_bytes(None, n) == err("NULL")
    assert lib.attn_pages_workspace_bytes(pool(), None) == err("NULL")
    assert lib.attn_pages_workspace_bytes(pool(num_seqs=5, num_pages=9), n) == 0
    assert n.value == 4 * (3 * 12 + 3 * 8 + 8)
    assert reserve(wsb=n.value - 1, p=pool(num_seqs=5)) == err("WORKSPACE")


@no_gpu_only
def test_empty_page_calls_do_nothing(lib):  # noqa: F811
    assert copy(n=0) == 0 and copy(pages=0) == 0 and copy(b=()) == 0
    assert fork(n=0) == 0 and fork(pool(num_seqs=0)) == 0
    assert free(n=0) == 0 and free(pool(num_seqs=0)) == 0


def shape(**kw):
    a = dict(num_seqs=2, num_queries=3, Hq=4, Hkv=2, D=64, page_size=16, num_pages=4, max_pages=2, max_queries=3)
    a.update(kw)
    return A.PagedShape(*a.values())


def prefix(s=None, ng=1, mgq=3, **kw):
    a = dict(q=FAR, kc=2 * FAR, vc=3 * FAR, bt=4 * FAR, sl=5 * FAR, qo=6 * FAR, pos=None, go=7 * FAR, pl=8 * FAR, causal=1,
             scale=0.1, dtype=A.ATTN_F16, ws=9 * FAR, wsb=1 << 40, out=10 * FAR, lse=None)
    a.update(kw)
    return A.load_library().attn_paged_prefix_fwd(s or shape(), ng, mgq, a["q"], a["kc"], a["vc"], a["bt"], a["sl"], a["qo"],
                                                  a["pos"], a["go"], a["pl"], a["causal"], a["scale"], a["dtype"], a["ws"],
                                                  a["wsb"], a["out"], a["lse"], None)


BAD_SHAPES = [(dict(s=dict(Hq=3)), "SHAPE"), (dict(s=dict(num_queries=-1)), "SHAPE"), (dict(s=dict(D=80)), "HEAD_DIM"),
              (dict(s=dict(page_size=0)), "SHAPE"), (dict(ng=-1), "SHAPE"), (dict(mgq=-1), "SHAPE"),
              (dict(s=dict(num_pages=(1 << 31) - 1, page_size=1 << 20, max_pages=1, Hq=1 << 15, Hkv=1 << 15, D=128)), "SHAPE"),
              (dict(s=dict(max_pages=1 << 28)), "SHAPE"), (dict(ng=1 << 30), "SHAPE"), (dict(ng=(1 << 30) + 1, s=dict(Hkv=1)), "SHAPE"), (dict(mgq=(1 << 31) - 1), "SHAPE")]


@no_gpu_only
@pytest.mark.parametrize("kw,e", BAD_SHAPES + [
    (dict(dtype=3), "DTYPE"), (dict(causal=2), "MASK"), (dict(scale=0.0), "SCALE"), (dict(scale=math.inf), "SCALE"),
    (dict(q=None), "NULL"), (dict(kc=None), "NULL"), (dict(bt=None), "NULL"), (dict(sl=None), "NULL"),
    (dict(go=None), "NULL"), (dict(pl=None), "NULL"), (dict(out=None), "NULL"), (dict(ws=None), "WORKSPACE"),
    (dict(wsb=16), "WORKSPACE"), (dict(q=FAR + 2), "ALIGN"), (dict(ws=9 * FAR + 8), "ALIGN"), (dict(go=7 * FAR + 2), "ALIGN"),
    (dict(pos=11 * FAR + 1), "ALIGN"), (dict(lse=11 * FAR + 2), "ALIGN"), (dict(out=FAR), "OVERLAP"),
    (dict(out=8 * FAR), "OVERLAP"), (dict(lse=10 * FAR + 4), "OVERLAP"), (dict(ws=7 * FAR), "OVERLAP")])
def test_prefix_refusals(lib, kw, e):  # noqa: F811
    kw = dict(kw)
    s = shape(**kw.pop("s", {}))
    assert prefix(s, **kw) == err(e)
    if (kw, e) in [({k: v for k, v in x.items() if k != "s"}, y) for x, y in BAD_SHAPES]:
        assert lib.attn_paged_prefix_workspace_bytes(s, kw.get("ng", 1), kw.get("mgq", 3), ctypes.c_size_t()) == err(e)


@no_gpu_only
def test_prefix_workspace_and_empty_calls(lib):  # noqa: F811
    n = ctypes.c_size_t()
    assert lib.attn_paged_prefix_workspace_bytes(None, 1, 1, n) == err("NULL")
    assert lib.attn_paged_prefix_workspace_bytes(shape(), 1, 1, None) == err("NULL")
    assert lib.attn_paged_prefix_workspace_bytes(shape(), 1, 3, n) == 0 and n.value > 0
    assert prefix(wsb=n.value - 1) == err("WORKSPACE")
    assert prefix(shape(num_queries=0)) == 0 and prefix(shape(num_seqs=0)) == 0 and prefix(shape(max_queries=0)) == 0


def rope(A_=2, stride=5, axis=7 * FAR, S=5, Hq=4, D=64, rot=64, q=FAR, pos=3 * FAR, freq=4 * FAR, qo=5 * FAR):
    s = A.RopeShape(1, S, Hq, 0, D, rot, I3(0, Hq * D, D), I3(), I3(0, Hq * D, D), I3(), 0)
    return A.load_library().attn_rope_axes(s, q, None, pos, stride, A_, axis, freq, 0, 0, 1.0, A.ATTN_BF16, qo, None, None)


@no_gpu_only
@pytest.mark.parametrize("kw,e", [
    (dict(A_=0), "SHAPE"), (dict(A_=257), "SHAPE"), (dict(stride=-1), "SHAPE"), (dict(stride=1 << 60), "SHAPE"),
    (dict(axis=None), "NULL"), (dict(axis=7 * FAR + 2), "ALIGN"), (dict(pos=None), "NULL"), (dict(rot=63), "SHAPE"),
    (dict(qo=7 * FAR + 64), "OVERLAP"), (dict(stride=FAR // 4, qo=4 * FAR), "OVERLAP"), (dict(qo=FAR + 16), "OVERLAP")])
def test_axes_refusals(lib, kw, e):  # noqa: F811
    assert rope(**kw) == err(e)


def _batch():
    import torch
    i = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    c = torch.zeros((4, 16, 2, 64))
    return dict(q=torch.zeros((3, 4, 64)), k_cache=c, v_cache=c.clone(), block_table=i(2, 2), seq_lens=i(2), q_offsets=i(3),
                group_offsets=i(2), prefix_lens=i(1))


@pytest.mark.parametrize("change", [dict(), dict(q=(3, 4, 32)), dict(q="float16"), dict(v_cache=(4, 16, 2, 32)),
                                    dict(k_cache=(4, 16, 128)), dict(block_table="int64"), dict(block_table=(3, 2)),
                                    dict(seq_lens=(2, 1)), dict(q_offsets=(2,)), dict(group_offsets=(0,)),
                                    dict(group_offsets=(3,)), dict(prefix_lens="int64")])
def test_binding_refuses_malformed_batches(change):
    import torch
    t = _batch()
    for name, c in change.items():
        t[name] = t[name].to(getattr(torch, c)) if isinstance(c, str) else torch.zeros(c, dtype=t[name].dtype)
    with pytest.raises(A.AttnError):  # without a change: host tensors
        A.paged_prefix_fwd(**t, max_queries=1, max_group_queries=1)


def test_binding_refuses_malformed_pools():
    import torch
    i = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    table, lens, refs, c = i(4, 3), i(4), i(9), [torch.zeros((9, 16, 2))]
    calls = [lambda: A.pages_free(table, lens, refs, i(1)),  # no CUDA device
             lambda: A.pages_free(table, lens[:3], refs, i(1)), lambda: A.pages_free(table, lens, refs, i(1, 1)),
             lambda: A.pages_free(table.long(), lens, refs, i(1)), lambda: A.pages_free(table, lens, refs, i(1).long()),
             lambda: A.pages_fork(table, lens, refs, i(2), i(3), page_size=16),
             lambda: A.pages_fork(table.T, lens, refs, i(2), i(2), page_size=16),
             lambda: A.pages_reserve(table, lens, refs, i(3), c, page_size=16),
             lambda: A.pages_reserve(table, lens, refs, i(4), [c[0][:8]], page_size=16),
             lambda: A.pages_reserve(table, lens, refs, i(4), [c[0][:, ::2]], page_size=16),
             lambda: A.pages_reserve(table, lens, refs, i(4), c, page_size=16, result=i(3)),
             lambda: A.pages_compact(table, refs, c, page_map=i(8)), lambda: A.pages_compact(table, refs, c, used=i(2)),
             lambda: A.pages_copy(c, i(2), i(3)), lambda: A.pages_copy(c, i(2).long(), i(2)),
             lambda: A.rope_axes([]), lambda: A.rope_axes([3, -1]),
             lambda: A.rope(torch.zeros((3, 2, 8)), None, i(3), torch.zeros(4, dtype=torch.float64), axes=i(4)),
             lambda: A.rope(torch.zeros((3, 2, 8)), None, i(2, 4), torch.zeros(4, dtype=torch.float64), axes=i(4)),
             lambda: A.rope(torch.zeros((3, 2, 8)), None, i(2, 3), torch.zeros(4, dtype=torch.float64), axes=i(3))]
    for f in calls:
        with pytest.raises(A.AttnError):
            f()


def test_axes_of_pairs():
    assert A.rope_axes([2, 1, 3]).tolist() == [0, 0, 1, 2, 2, 2]
    assert A.rope_axes([2, 1, 3], cycle=True).tolist() == [0, 1, 2, 0, 2, 2]
    assert A.rope_axes([0, 2], cycle=True).tolist() == [1, 1]


def test_sequential_pool():
    # the restatement that the GPU tests compare with
    x = np.arange(12)[:, None] * 10 + np.arange(4)
    p = R.Pool(4, 3, 4, 12, [x])
    assert p.reserve([6, 0, 0, 0]) == (2, 0) and p.table[0].tolist() == [0, 1, -1]
    p.lens[0] = 6
    p.fork([0, 0], [1, 2])
    assert p.refs[:3].tolist() == [3, 3, 0]
    assert p.reserve([1, 1, 1, 0]) == (2, 0)  # two copy, the last keeps
    assert p.table[:3, 1].tolist() == [2, 3, 1] and x[2].tolist() == [10, 11, 12, 13]
    p.free([0])
    assert p.refs[:4].tolist() == [2, 1, 0, 1]
    to, used = p.compact()
    assert used == 3 and to[:4].tolist() == [0, 1, -1, 2] and p.table[1, 1] == 2
    p.check()


def test_sequential_attention_agrees_with_the_oracle():
    import oracle
    b = R.Shared(3, [(37, [(9, 2), (1, 1)]), (None, [(20, 3)])], dtype="f32", D=16, P=8, H=2, Hq=4, hidden=0.0)
    out, lse, _, _ = b.ref()
    want = oracle.paged_attention(b.q.numpy(), b.kc.numpy(), b.vc.numpy(), b.table, b.lens, b.offs, causal=True, scale=0.25,
                                  dtype="f32")
    assert np.allclose(out, want, rtol=0, atol=1e-12) and np.isfinite(lse).all()
