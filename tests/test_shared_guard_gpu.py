"""Guard bands around what the page calls, the shared-prefix attention and the rotary calls with axes
write, in the normal and in the bounds-checked build (the scheme of test_guard_bands_gpu.py)."""
import numpy as np
import pytest

from tests.pages_ref import Shared
from tests.test_guard_bands_gpu import Guarded, _clean_status, checked_path, guarded_ws, run_both  # noqa: F401
from tests.test_prefix_gpu import BATCHES, FORMS

pytestmark = pytest.mark.gpu


def put(x, sentinel):
    g = Guarded(tuple(x.shape), x.dtype, sentinel)
    g.t.copy_(x)
    return g


def ids(f):
    return "-".join(str(v) for v in f.values())


@pytest.mark.parametrize("form", FORMS, ids=ids)
@pytest.mark.parametrize("name", ["in_page", "ragged", "outside", "empty_groups", "no_queries", "mixed", "prompts"])
def test_prefix_guard_bands(name, form, checked_path):  # noqa: F811
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    b = Shared(43, BATCHES[name], **form)
    d = b.device()
    shape = attn.PagedShape(len(b.lens), len(b.q), b.Hq, b.H, b.D, b.P, len(b.kc), b.table.shape[1], b.max_q)
    need = attn.paged_prefix_workspace_bytes(shape, len(b.pre), b.max_gq)

    def call(sentinel):
        out = Guarded(tuple(b.q.shape), b.q.dtype, sentinel)
        lse = Guarded((len(b.q), b.Hq), torch.float32, sentinel)
        ws = guarded_ws(need, sentinel)
        attn.paged_prefix_fwd(*d, max_queries=b.max_q, max_group_queries=b.max_gq, out=out.t, return_lse=True,
                              lse_out=lse.t, workspace=ws.t)
        return {"out": (out, True), "lse": (lse, True), "workspace": (ws, False)}
    run_both(checked_path, call)


@pytest.mark.parametrize("S,M,P,N", [(6, 7, 4, 40), (700, 3, 8, 2600)])
def test_pages_guard_bands(S, M, P, N, checked_path):  # noqa: F811
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    r = np.random.RandomState(S)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    kids = r.permutation(S)[:S // 3]
    parents = r.choice(np.setdiff1d(np.arange(S), kids), len(kids))
    first, more = r.randint(1, 2 * P, S), r.randint(0, P, S)
    caches = [torch.from_numpy(r.randint(0, 255, (N, *s)).astype(np.uint8)).cuda() for s in ((P, 16), (7,), (4096 * 5,))]

    def call(sentinel):
        bufs = {"table": put(i32(np.full((S, M), -1)), sentinel), "lens": put(i32(np.zeros(S)), sentinel),
                "refs": put(i32(np.zeros(N)), sentinel)}
        bufs |= {f"cache{i}": put(c, sentinel) for i, c in enumerate(caches)}
        bufs |= {n: Guarded((k,), torch.int32, sentinel) for n, k in (("result", 2), ("page_map", N), ("used", 1))}
        ws = guarded_ws(attn.pages_workspace_bytes(attn.Pages(S, M, P, N)), sentinel)
        t, lens, refs, x = bufs["table"].t, bufs["lens"].t, bufs["refs"].t, [bufs[f"cache{i}"].t for i in range(3)]
        kw = dict(page_size=P, result=bufs["result"].t, workspace=ws.t)
        attn.pages_reserve(t, lens, refs, i32(first), x, **kw)
        lens += i32(first)
        attn.pages_fork(t, lens, refs, i32(parents), i32(kids), page_size=P)
        attn.pages_reserve(t, lens, refs, i32(more), x, **kw)
        attn.pages_free(t, lens, refs, i32(parents[:3]))
        attn.pages_compact(t, refs, x, page_map=bufs["page_map"].t, used=bufs["used"].t, workspace=ws.t)
        attn.pages_copy(x, i32([0, 1, -1]), i32([N - 1, N - 2, 0]))
        return {**{n: (g, n in ("result", "page_map", "used")) for n, g in bufs.items()}, "workspace": (ws, False)}
    run_both(checked_path, call)


@pytest.mark.parametrize("dtype,D,rot", [("bfloat16", 128, 64), ("float16", 18, 6), ("float32", 64, 64)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_axes_guard_bands(dtype, D, rot, layout, checked_path):  # noqa: F811
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    r = np.random.RandomState(D)
    q, k = (torch.from_numpy(r.randn(301, h, D)).to(getattr(torch, dtype)).cuda() for h in (5, 2))
    pos = torch.from_numpy(r.randint(0, 10000, (3, 301)).astype(np.int32)).cuda()
    axes = torch.from_numpy(r.randint(-1, 4, rot // 2).astype(np.int32)).cuda()
    f = attn.rope_frequencies(rot)[0].cuda()

    def call(sentinel):
        outs = [Guarded(tuple(x.shape), x.dtype, sentinel) for x in (q, k)]
        attn.rope(q, k, pos, f, layout=layout, axes=axes, q_out=outs[0].t, k_out=outs[1].t)
        return {"q_out": (outs[0], True), "k_out": (outs[1], True)}
    run_both(checked_path, call)
