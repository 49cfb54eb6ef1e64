"""Query rows of no sequence in attention of sequences that share a prefix (attn_paged_prefix_fwd): the padded
rows of a captured step."""
import numpy as np
import pytest

from tests.gpu_util import to_f64
from tests.pages_ref import Shared, near
from tests.test_prefix_gpu import ones

pytestmark = pytest.mark.gpu
FORMS = [dict(dtype="bf16", D=128, P=64, H=8, Hq=32), dict(dtype="f16", D=64, P=24, H=2, Hq=6),
         dict(dtype="f32", D=128, P=16, H=2, Hq=4)]


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(str(v) for v in f.values()))
@pytest.mark.parametrize("bounds", [(1, 4), (1, 100), (100, 400)])
@pytest.mark.parametrize("prefix", [3000, None])
@pytest.mark.parametrize("at", ["front", "back"])
def test_a_call_without_a_row_of_a_sequence(at, prefix, bounds, form):
    # all offsets equal, in a graph whose next kernel owns the workspace: nothing of the call is left to run then
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    b = Shared(109, [(prefix, ones(40, 1, 4000))], **form)
    n = len(b.q)
    b.offs[:] = 0 if at == "back" else n
    d = b.device()
    out, lse = torch.full_like(d[0], 768.0), torch.full(d[0].shape[:2], 768.0, device="cuda")
    shape = attn.PagedShape(len(b.lens), n, b.Hq, b.H, b.D, b.P, len(b.kc), b.table.shape[1], bounds[0])
    ws = torch.empty(attn.paged_prefix_workspace_bytes(shape, len(b.pre), bounds[1]), dtype=torch.uint8, device="cuda")
    kw = dict(max_queries=bounds[0], max_group_queries=bounds[1], return_lse=True, out=out, lse_out=lse, workspace=ws)
    attn.paged_prefix_fwd(*d, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn.paged_prefix_fwd(*d, **kw)
        ws.fill_(0x5A)
    for _ in range(50):
        ws.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert bool((ws == 0x5A).all())
    for _ in range(50):  # and without one
        attn.paged_prefix_fwd(*d, **kw)
        ws.fill_(0x5A)
        torch.cuda.synchronize()
        assert bool((ws == 0x5A).all())
    assert bool((out == 768).all()) and bool((lse == 768).all())
    assert attn.device_status(0, clear=True) == 0


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(str(v) for v in f.values()))
def test_one_row_among_many_of_no_sequence(form):
    # the last of 4000 rows, and the first
    import torch
    b = Shared(113, [(2000, ones(1)), (500, ones(1))], **form)
    ref = b.ref()
    rows = 4000
    q = b.q
    b.q = torch.randn((rows, b.Hq, b.D), generator=torch.Generator().manual_seed(3)).to(q.dtype)
    for first in (rows - 2, 0, 1234):
        b.q[first:first + 2] = q
        d = list(b.device())
        d[5] += first
        out, lse = torch.full_like(d[0], 768.0), torch.full(d[0].shape[:2], 768.0, device="cuda")
        from exact_scaled_dot_flash_gb300 import attn
        attn.paged_prefix_fwd(*d, max_queries=1, max_group_queries=1, return_lse=True, out=out, lse_out=lse)
        o, z = to_f64(out), to_f64(lse)
        mine = np.arange(first, first + 2)
        near(o[mine], z[mine], ref, b.dtype, b.D)
        rest = np.setdiff1d(np.arange(rows), mine)
        assert (o[rest] == 768).all() and (z[rest] == 768).all()
