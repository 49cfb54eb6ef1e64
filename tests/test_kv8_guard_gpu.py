"""Guard bands around what the 8-bit cache and the rotary calls write, in the normal and in the
bounds-checked build (the scheme of test_guard_bands_gpu.py): bytes on both sides of every output,
cache, scale and workspace keep their pattern, fully written outputs hold no pattern, the status
word stays clear and the two builds agree bit for bit."""
import numpy as np
import pytest

from tests.test_guard_bands_gpu import Guarded, _clean_status, checked_path, guarded_ws, run_both  # noqa: F401
from tests.test_kv8_gpu import Problem, gpu, tdt

pytestmark = pytest.mark.gpu

SHAPES = [
    dict(lens=[700, 1, 333], new=[1, 1, 1], dtype="bf16", fmt="e4m3", D=128, P=64, G=16, H=2, Hq=8),
    dict(lens=[700, 40, 333], new=[5, 2, 4], dtype="f16", fmt="int8", D=64, P=8, G=2, H=3, Hq=21),
    dict(lens=[300, 45, 290], new=[150, 45, 70], dtype="bf16", fmt="int8", D=128, P=32, G=32, H=2, Hq=8),
    dict(lens=[2050, 45], new=[70, 45], dtype="f16", fmt="e4m3", D=64, P=24, G=4, H=1, Hq=5),
    dict(lens=[100, 45, 61], new=[9, 45, 1], dtype="f32", fmt="e4m3", D=32, P=5, G=1, H=2, Hq=4),
]


def ids(kw):
    return "-".join(str(v) for v in kw.values())


def problem(kw):
    kw = dict(kw)
    return Problem(31, kw.pop("lens"), kw.pop("new"), **kw)


def guarded_copy(x, sentinel):
    g = Guarded(tuple(x.shape), x.dtype, sentinel)
    g.t.copy_(x)
    return g


@pytest.mark.parametrize("kw", SHAPES, ids=ids)
def test_write_and_read_guard_bands(kw, checked_path):  # noqa: F811
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    p = problem(kw)
    kc, vc, ks, vs, table, lens = p.cache()
    rows = int(p.lens.sum())
    offs = gpu(np.concatenate([[0], np.cumsum(p.lens)]).astype(np.int32))
    caches = []

    def call(sentinel):
        bufs = [guarded_copy(t.view(torch.uint8) if i < 2 else t, sentinel) for i, t in enumerate((kc, vc, ks, vs))]
        args = [bufs[0].t.view(tdt(p.fmt)), bufs[1].t.view(tdt(p.fmt)), bufs[2].t, bufs[3].t, table, lens]
        attn.kv8_write(p.k.cuda(), p.v.cuda(), *args, gpu(p.offs))
        outs = [Guarded((rows, p.H, p.D), tdt(p.dtype), sentinel) for _ in range(2)]
        attn.kv8_read(*args, offs, k_out=outs[0].t, v_out=outs[1].t)
        caches.append([b.words().copy() for b in bufs])
        names = ("k_cache", "v_cache", "k_scale", "v_scale")
        return {**{n: (b, False) for n, b in zip(names, bufs)}, "k_out": (outs[0], True), "v_out": (outs[1], True)}
    run_both(checked_path, call)
    assert all(np.array_equal(a, b) for a, b in zip(*caches))


@pytest.mark.parametrize("kw", SHAPES, ids=ids)
@pytest.mark.parametrize("causal", [True, False])
def test_attention_guard_bands(kw, causal, checked_path):  # noqa: F811
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    p = problem(kw)
    cache, q, offs, mq = p.cache(), p.q.cuda(), gpu(p.offs), int(p.new.max())
    shape = attn.PagedShape(len(p.lens), p.tokens, p.Hq, p.H, p.D, p.P, p.pages, p.table.shape[1], mq)

    def call(sentinel):
        out = Guarded(tuple(q.shape), q.dtype, sentinel)
        lse = Guarded((p.tokens, p.Hq), torch.float32, sentinel)
        ws = guarded_ws(attn.paged_kv8_workspace_bytes(shape), sentinel)
        attn.paged_kv8_fwd(q, *cache, offs, causal=causal, max_queries=mq, out=out.t, return_lse=True, lse_out=lse.t,
                           workspace=ws.t)
        return {"out": (out, True), "lse": (lse, True), "workspace": (ws, False)}
    run_both(checked_path, call)


@pytest.mark.parametrize("dtype,D,rot", [("bf16", 128, 64), ("f16", 18, 6), ("f32", 512, 512)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T", [3, 2501])
def test_rope_guard_bands(dtype, D, rot, layout, T, checked_path):  # noqa: F811
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    r = np.random.RandomState(T)
    q, k = (torch.from_numpy(r.randn(T, h, D)).to(tdt(dtype)).cuda() for h in (5, 2))
    pos = gpu(r.randint(0, 10000, T).astype(np.int32))
    f = attn.rope_frequencies(rot)[0].cuda()

    def call(sentinel):
        outs = [Guarded(tuple(x.shape), x.dtype, sentinel) for x in (q, k)]
        attn.rope(q, k, pos, f, layout=layout, q_out=outs[0].t, k_out=outs[1].t)
        return {"q_out": (outs[0], True), "k_out": (outs[1], True)}
    run_both(checked_path, call)
