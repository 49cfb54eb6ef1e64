"""Refusals and host-side rules of the 8-bit paged cache and of rotary positions, without a GPU.

Made-up addresses are passed only where no GPU is visible (see test_boundary.py): validation
must reject each call before any of them could reach a kernel."""
import ctypes
import math

import numpy as np
import pytest

from exact_scaled_dot_flash_gb300 import attn as A
from tests import kv8_ref as R
from tests.test_boundary import codes, lib, no_gpu_only  # noqa: F401

FAR = 1 << 44  # addresses 16 terabytes apart: no two buffers meet
I2, I3 = ctypes.c_int64 * 2, ctypes.c_int64 * 3


def cache(pages=4, P=16, H=2, D=64, G=8, fmt=A.KV8_INT8):
    return A.Kv8Cache(pages, P, H, D, G, fmt)


def write(c=None, ns=1, mp=2, nt=3, **kw):
    a = dict(k=FAR, v=2 * FAR, ks=(128, 64), vs=(128, 64), bt=3 * FAR, sl=4 * FAR, to=5 * FAR, dtype=A.ATTN_BF16,
             kc=6 * FAR, vc=7 * FAR, kq=8 * FAR, vq=9 * FAR)
    a.update(kw)
    return A.load_library().attn_kv8_write(c or cache(), ns, mp, nt, a["k"], a["v"], I2(*a["ks"]) if a["ks"] else None,
                                           I2(*a["vs"]), a["bt"], a["sl"], a["to"], a["dtype"], a["kc"], a["vc"],
                                           a["kq"], a["vq"], None)


def read(c=None, ns=1, mp=2, nr=3, **kw):
    a = dict(kc=FAR, vc=2 * FAR, kq=3 * FAR, vq=4 * FAR, bt=5 * FAR, sl=6 * FAR, ro=7 * FAR, st=None,
             dtype=A.ATTN_BF16, ko=8 * FAR, vo=9 * FAR)
    a.update(kw)
    return A.load_library().attn_kv8_read(c or cache(), ns, mp, nr, a["kc"], a["vc"], a["kq"], a["vq"], a["bt"],
                                          a["sl"], a["ro"], a["st"], a["dtype"], a["ko"], a["vo"], None)


def shape(**kw):
    a = dict(num_seqs=1, num_queries=3, Hq=4, Hkv=2, D=64, page_size=16, num_pages=4, max_pages=2, max_queries=3)
    a.update(kw)
    return A.PagedShape(*a.values())


def fwd(s=None, group=8, fmt=A.KV8_E4M3, **kw):
    a = dict(q=FAR, kc=2 * FAR, vc=3 * FAR, kq=4 * FAR, vq=5 * FAR, bt=6 * FAR, sl=7 * FAR, qo=8 * FAR, pos=None,
             causal=1, scale=0.1, dtype=A.ATTN_F16, ws=9 * FAR, wsb=1 << 40, out=10 * FAR, lse=None)
    a.update(kw)
    return A.load_library().attn_paged_kv8_fwd(s or shape(), group, fmt, a["q"], a["kc"], a["vc"], a["kq"], a["vq"],
                                               a["bt"], a["sl"], a["qo"], a["pos"], a["causal"], a["scale"],
                                               a["dtype"], a["ws"], a["wsb"], a["out"], a["lse"], None)


def rope(B=1, S=5, Hq=4, Hk=2, D=64, rot=64, q=FAR, k=2 * FAR, pos=3 * FAR, freq=4 * FAR, layout=0, inverse=0,
         mscale=1.0, dtype=A.ATTN_BF16, qo=5 * FAR, ko=6 * FAR, qs=None, ks=None, qos=None, kos=None, pb=0):
    s = A.RopeShape(B, S, Hq, Hk, D, rot, I3(*(qs or (0, Hq * D, D))), I3(*(ks or (0, max(Hk, 0) * D, D))),
                    I3(*(qos or (0, Hq * D, D))), I3(*(kos or (0, max(Hk, 0) * D, D))), pb)
    return A.load_library().attn_rope(s, q, k, pos, freq, layout, inverse, mscale, dtype, qo, ko, None)


BAD_CACHE = [(dict(P=0), "SHAPE"), (dict(H=0), "SHAPE"), (dict(pages=-1), "SHAPE"), (dict(G=0), "SHAPE"),
             (dict(G=5), "SHAPE"), (dict(G=32), "SHAPE"), (dict(D=48), "HEAD_DIM"), (dict(D=256), "HEAD_DIM"),
             (dict(fmt=2), "DTYPE"), (dict(fmt=-1), "DTYPE"), (dict(H=40000), "SHAPE")]


@no_gpu_only
@pytest.mark.parametrize("kw,err", BAD_CACHE)
def test_bad_caches(lib, kw, err):  # noqa: F811
    assert write(cache(**kw)) == codes["ATTN_ERR_" + err]
    assert read(cache(**kw)) == codes["ATTN_ERR_" + err]


@no_gpu_only
@pytest.mark.parametrize("kw,err", [
    (dict(ns=-1), "SHAPE"), (dict(mp=-1), "SHAPE"), (dict(nt=-1), "SHAPE"), (dict(mp=1 << 30), "SHAPE"),
    (dict(dtype=3), "DTYPE"), (dict(ks=None), "NULL"), (dict(ks=(-1, 64)), "SHAPE"), (dict(vs=(128, -64)), "SHAPE"),
    (dict(ks=(1 << 40, 64)), "SHAPE"), (dict(k=None), "NULL"), (dict(vc=None), "NULL"), (dict(kq=None), "NULL"),
    (dict(bt=None), "NULL"), (dict(to=None), "NULL"), (dict(k=FAR + 1), "ALIGN"), (dict(kc=6 * FAR + 8), "ALIGN"),
    (dict(vq=9 * FAR + 2), "ALIGN"), (dict(kc=7 * FAR), "OVERLAP"), (dict(vc=2 * FAR + 16), "OVERLAP"),
    (dict(kq=6 * FAR + 4096), "OVERLAP"), (dict(kq=4 * FAR), "OVERLAP")])
def test_write_refusals(lib, kw, err):  # noqa: F811
    assert write(**kw) == codes["ATTN_ERR_" + err]


@no_gpu_only
@pytest.mark.parametrize("kw,err", [
    (dict(nr=-1), "SHAPE"), (dict(dtype=7), "DTYPE"), (dict(ko=None), "NULL"), (dict(ro=None), "NULL"),
    (dict(kc=None), "NULL"), (dict(vo=9 * FAR + 2), "ALIGN"), (dict(st=10 * FAR + 1), "ALIGN"),
    (dict(ko=9 * FAR), "OVERLAP"), (dict(vo=2 * FAR), "OVERLAP"), (dict(ko=6 * FAR), "OVERLAP")])
def test_read_refusals(lib, kw, err):  # noqa: F811
    assert read(**kw) == codes["ATTN_ERR_" + err]


@no_gpu_only
@pytest.mark.parametrize("kw,err", [
    (dict(s=dict(Hq=3)), "SHAPE"), (dict(s=dict(num_queries=-1)), "SHAPE"), (dict(s=dict(D=80)), "HEAD_DIM"),
    (dict(s=dict(page_size=0)), "SHAPE"), (dict(group=0), "SHAPE"), (dict(group=6), "SHAPE"), (dict(fmt=2), "DTYPE"),
    (dict(dtype=3), "DTYPE"), (dict(causal=2), "MASK"), (dict(scale=0.0), "SCALE"), (dict(scale=math.nan), "SCALE"),
    (dict(q=None), "NULL"), (dict(kq=None), "NULL"), (dict(bt=None), "NULL"), (dict(out=None), "NULL"),
    (dict(q=FAR + 2), "ALIGN"), (dict(lse=11 * FAR + 2), "ALIGN"), (dict(out=FAR), "OVERLAP"),
    (dict(out=5 * FAR), "OVERLAP"), (dict(lse=10 * FAR + 4), "OVERLAP")])
def test_attention_refusals(lib, kw, err):  # noqa: F811
    kw = dict(kw)
    s = shape(**kw.pop("s", {}))
    assert fwd(s, **kw) == codes["ATTN_ERR_" + err]


@no_gpu_only
def test_attention_workspace_refusals(lib):  # noqa: F811
    n = ctypes.c_size_t(7)
    assert lib.attn_paged_kv8_workspace_bytes(None, n) == codes["ATTN_ERR_NULL"]
    assert lib.attn_paged_kv8_workspace_bytes(shape(), None) == codes["ATTN_ERR_NULL"]
    assert lib.attn_paged_kv8_workspace_bytes(shape(Hq=5), n) == codes["ATTN_ERR_SHAPE"]
    assert lib.attn_paged_kv8_workspace_bytes(shape(D=20), n) == codes["ATTN_ERR_HEAD_DIM"]
    s = shape(D=128, num_queries=1, max_queries=1)
    assert lib.attn_paged_kv8_workspace_bytes(s, n) == 0
    if n.value:
        assert fwd(s, ws=None) == codes["ATTN_ERR_WORKSPACE"]
        assert fwd(s, wsb=n.value - 1) == codes["ATTN_ERR_WORKSPACE"]
        assert fwd(s, ws=9 * FAR + 8) == codes["ATTN_ERR_ALIGN"]
        assert fwd(s, ws=2 * FAR) == codes["ATTN_ERR_OVERLAP"]


@no_gpu_only
@pytest.mark.parametrize("kw,err", [
    (dict(B=-1), "SHAPE"), (dict(Hq=0), "SHAPE"), (dict(Hk=-1), "SHAPE"), (dict(D=514), "SHAPE"), (dict(rot=0), "SHAPE"),
    (dict(rot=63), "SHAPE"), (dict(rot=66), "SHAPE"), (dict(layout=2), "SHAPE"), (dict(inverse=2), "SHAPE"),
    (dict(pb=3), "SHAPE"), (dict(qs=(0, -256, 64)), "SHAPE"), (dict(dtype=5), "DTYPE"), (dict(mscale=math.inf), "SCALE"),
    (dict(q=None), "NULL"), (dict(k=None), "NULL"), (dict(pos=None), "NULL"), (dict(ko=None), "NULL"),
    (dict(q=FAR + 1), "ALIGN"), (dict(freq=4 * FAR + 4), "ALIGN"),
    (dict(qo=FAR + 16), "OVERLAP"),                         # shifted onto its input
    (dict(qo=FAR, qos=(0, 512, 64)), "OVERLAP"),            # in place, but with other strides
    (dict(qo=2 * FAR), "OVERLAP"), (dict(ko=5 * FAR), "OVERLAP"), (dict(qo=3 * FAR), "OVERLAP"),
    (dict(qos=(0, 0, 64)), "OVERLAP"), (dict(qos=(0, 192, 64)), "OVERLAP"),  # rows on one another
    (dict(B=2, qos=(64, 256, 64)), "OVERLAP")])
def test_rope_refusals(lib, kw, err):  # noqa: F811
    assert rope(**kw) == codes["ATTN_ERR_" + err]


@no_gpu_only
def test_fused_slices_are_told_apart(lib):  # noqa: F811
    # q, k of one projection [tokens, (4 + 2 + 2) * 64]: k may not be written over q's columns
    t = 8 * 64
    kw = dict(q=FAR, k=FAR + 4 * 64 * 2, qs=(0, t, 64), ks=(0, t, 64), qos=(0, t, 64), kos=(0, t, 64))
    assert rope(qo=FAR, ko=FAR + 3 * 64 * 2, **kw) == codes["ATTN_ERR_OVERLAP"]
    assert rope(qo=FAR + 6 * 64 * 2, ko=FAR + 4 * 64 * 2, **kw) == codes["ATTN_ERR_OVERLAP"]


@no_gpu_only
def test_empty_calls_do_nothing(lib):  # noqa: F811
    assert write(nt=0) == 0 and write(ns=0) == 0 and write(mp=0) == 0 and write(cache(pages=0)) == 0
    assert read(nr=0) == 0 and read(ns=0) == 0
    assert fwd(shape(num_queries=0)) == 0 and fwd(shape(num_seqs=0)) == 0
    assert rope(S=0) == 0 and rope(B=0) == 0


def _tensors():
    import torch
    kc = torch.zeros((4, 16, 2, 64), dtype=torch.int8)
    ks = torch.zeros((4, 2, 2), dtype=torch.float32)
    i = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    return dict(k_cache=kc, v_cache=kc.clone(), k_scale=ks, v_scale=ks.clone(), block_table=i(1, 2), seq_lens=i(1))


@pytest.mark.parametrize("change", [
    dict(k_cache="uint8"), dict(v_cache="float8_e4m3fn"), dict(k_scale="float64"), dict(block_table="int64"),
    dict(k_scale=(4, 2, 3)), dict(k_scale=(4, 1, 2)), dict(v_scale=(4, 2, 1)), dict(k_cache=(4, 16, 64)),
    dict(v_cache=(3, 16, 2, 64)), dict(block_table=(2, 2)), dict(seq_lens=(1, 1)), dict(offsets=(3,))])
def test_binding_refuses_malformed_caches(change):
    import torch
    t = _tensors()
    offsets = torch.zeros(2, dtype=torch.int32)
    for name, c in change.items():
        if name == "offsets":
            offsets = torch.zeros(c, dtype=torch.int32)
        elif isinstance(c, str):
            t[name] = t[name].to(getattr(torch, c))
        else:
            t[name] = torch.zeros(c, dtype=t[name].dtype)
    x = torch.zeros((3, 2, 64))
    with pytest.raises(A.AttnError):
        A.kv8_write(x, x, **t, tok_offsets=offsets)
    with pytest.raises(A.AttnError):
        A.kv8_read(**t, row_offsets=offsets, num_rows=3)
    with pytest.raises(A.AttnError):
        A.paged_kv8_fwd(torch.zeros((3, 4, 64)), **t, q_offsets=offsets, max_queries=3)


def test_binding_refuses_host_tensors_and_bad_rows():
    import torch
    t, off, x = _tensors(), torch.zeros(2, dtype=torch.int32), torch.zeros((3, 2, 64))
    pos, f = torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    calls = [lambda: A.kv8_write(x, x, **t, tok_offsets=off),  # no CUDA device
             lambda: A.kv8_write(x, x.half(), **t, tok_offsets=off),
             lambda: A.kv8_write(x[:, :1], x[:, :1], **t, tok_offsets=off),
             lambda: A.kv8_write(x.transpose(1, 2), x.transpose(1, 2), **t, tok_offsets=off),
             lambda: A.kv8_read(**t, row_offsets=off, num_rows=3),
             lambda: A.kv8_read(**t, row_offsets=off, k_out=x, v_out=x[:2]),
             lambda: A.kv8_read(**t, row_offsets=off, num_rows=3, dtype=torch.float64),
             lambda: A.paged_kv8_fwd(x[:, :, :32].contiguous(), **t, q_offsets=off, max_queries=1),
             lambda: A.paged_kv8_fwd(x.transpose(0, 1), **t, q_offsets=off, max_queries=1),
             lambda: A.paged_kv8_fwd(x, **t, q_offsets=off, max_queries=1),
             lambda: A.rope(x, x, pos, f),
             lambda: A.rope(x, x, pos, f, layout="pairs"),
             lambda: A.rope(x, x[:2], pos, f),
             lambda: A.rope(x, x.half(), pos, f),
             lambda: A.rope(x, None, pos[:2], f),
             lambda: A.rope(x, None, pos.long(), f),
             lambda: A.rope(x, None, pos, f.float()),
             lambda: A.rope(x[:, :, ::2], None, pos, f[:16]),
             lambda: A.rope(x, None, pos, f, q_out=x[:2])]
    for c in calls:
        with pytest.raises(A.AttnError):
            c()


def test_frequencies():
    w, m = A.rope_frequencies(64, base=500000.0)
    i = np.arange(0, 64, 2)
    assert m == 1.0 and np.allclose(w.numpy(), 500000.0 ** (-i / 64), rtol=1e-14)
    lin, _ = A.rope_frequencies(64, scaling="linear", factor=4.0)
    base, _ = A.rope_frequencies(64)
    assert np.allclose(lin.numpy() * 4, base.numpy(), rtol=1e-14)
    ntk, m = A.rope_frequencies(64, scaling="ntk", factor=4.0)  # the fastest kept, the slowest divided by 4
    assert m == 1.0 and ntk[0] == 1.0 and np.isclose(float(ntk[-1] * 4), float(base[-1]), rtol=1e-13)
    part, m = A.rope_frequencies(64, scaling="by_parts", factor=8.0, original_positions=4096)
    turns = 4096 * base.numpy() / (2 * math.pi)
    assert np.isclose(m, 0.1 * math.log(8.0) + 1)
    assert np.allclose(part.numpy()[turns >= 32], base.numpy()[turns >= 32], rtol=1e-14)
    assert np.allclose(part.numpy()[turns <= 1] * 8, base.numpy()[turns <= 1], rtol=1e-14)
    assert (np.diff(part.numpy()) < 0).all()
    for kw in (dict(rot=3), dict(rot=0), dict(rot=4, factor=0.5), dict(rot=4, base=0.0), dict(rot=4, scaling="x"),
               dict(rot=4, scaling="by_parts", slow_turns=40.0)):
        with pytest.raises(A.AttnError):
            A.rope_frequencies(**kw)


def test_reference_codes():
    # the 64-bit restatement itself: the e4m3 table and rounding against torch's conversions
    import torch
    b = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(b).view(torch.float8_e4m3fn).float().numpy()
    keep = (b & 0x7f) != 0x7f
    assert np.array_equal(R.values(b, "e4m3")[keep], t[keep].astype(np.float64))
    x = np.random.RandomState(0).uniform(-448, 448, 20000).astype(np.float32) * 2.0 ** -np.arange(20000) ** 0.2
    x = np.concatenate([x.astype(np.float32), np.linspace(-2, 2, 4097, dtype=np.float32) * 2.0 ** -7])
    y = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.encode(x.astype(np.float64), "e4m3"), y)
    assert R.new_scale(448.0, "e4m3") == 1.0 and R.new_scale(449.0, "e4m3") == 2.0


@no_gpu_only
def test_extents_past_64_bits(lib):  # noqa: F811
    top = (1 << 31) - 1
    big = cache(pages=top, P=1 << 20, H=32767, D=128, G=1)
    wide = cache(P=1, G=1)
    for call in (write, read):
        assert call(big) == codes["ATTN_ERR_SHAPE"]
        assert call(wide, ns=(1 << 30) - 1, mp=top) == codes["ATTN_ERR_SHAPE"]
    for kw in (dict(num_pages=top, page_size=1 << 20, Hkv=1 << 15, Hq=1 << 15, D=128),
               dict(num_queries=top, Hkv=1 << 20, Hq=1 << 30, max_queries=1),
               dict(num_seqs=(1 << 30) - 1, page_size=1, Hkv=2, max_pages=top)):
        assert fwd(shape(**kw)) == codes["ATTN_ERR_SHAPE"], kw
        assert lib.attn_paged_kv8_workspace_bytes(shape(**kw), ctypes.c_size_t()) == codes["ATTN_ERR_SHAPE"], kw
