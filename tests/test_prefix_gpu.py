"""Attention of sequences that share a prefix on the GPU (attn_paged_prefix_fwd) against 64 bits
(pages_ref.attention, each sequence by its own row; its tolerances are derived in pages_ref.near).
Everything in the caches that no sequence holds is NaN."""
import numpy as np
import pytest

from tests.gpu_util import to_f64
from tests.pages_ref import Shared, near

pytestmark = pytest.mark.gpu


def run(b, positions=None, causal=True, scale=None, **kw):
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    pos = torch.from_numpy(positions).cuda() if positions is not None else None
    kw = dict(dict(max_queries=b.max_q, max_group_queries=b.max_gq), **kw)
    return attn.paged_prefix_fwd(*b.device(), positions=pos, causal=causal, scale=scale, return_lse=True, **kw)


def check(b, positions=None, causal=True, scale=None, **kw):
    out, lse = run(b, positions, causal, scale, **kw)
    near(to_f64(out), to_f64(lse), b.ref(positions, causal, scale), b.dtype, b.D)
    from exact_scaled_dot_flash_gb300 import attn
    assert attn.device_status(0, clear=True) == 0
    return out, lse


def ones(n, lo=1, hi=40, new=1, seed=0):
    r = np.random.RandomState(seed)
    return [(max(new, int(x)), new) for x in r.randint(lo, hi + 1, n)]


BATCHES = {
    "one": [(37, [(1, 1)])],
    "page": [(32, ones(3))],
    "in_page": [(301, ones(4))],
    "short": [(3, ones(5, 1, 6))],
    "long_suffix": [(130, ones(2, 500, 900))],
    "wide": [(700, ones(40, 1, 90, seed=2))],
    "ragged": [(500, ones(3)), (40, ones(1, 200, 300)), (1030, ones(11, 1, 150, seed=3)), (129, ones(2))],
    "outside": [(200, ones(3)), (None, ones(2, 30, 300)), (77, ones(2)), (None, ones(3, 1, 200))],
    "empty_groups": [(200, []), (333, ones(3)), (5, []), (9, []), (64, ones(2)), (100, [])],
    "no_queries": [(150, [(5, 1), (300, 0), (8, 1), (1, 0)]), (99, [(3, 0), (4, 0)])],
    "no_prefix": [(0, ones(4, 1, 200))],
    "drafts": [(450, ones(6, 5, 60, new=5, seed=4)), (90, ones(2, 3, 30, new=3))],
    "mixed": [(260, [(1, 1), (90, 80), (300, 7), (33, 33), (2, 2)])],
    "prompts": [(400, [(150, 150), (61, 61), (129, 128)]), (None, [(200, 190)])],
}
FORMS = [dict(dtype="bf16", D=128, P=64, H=2, Hq=8), dict(dtype="f16", D=64, P=16, H=1, Hq=7),
         dict(dtype="f16", D=128, P=128, H=1, Hq=1), dict(dtype="bf16", D=64, P=24, H=3, Hq=9),
         dict(dtype="bf16", D=128, P=1, H=1, Hq=8), dict(dtype="f32", D=128, P=16, H=2, Hq=4),
         dict(dtype="f32", D=16, P=5, H=1, Hq=3), dict(dtype="f16", D=32, P=8, H=2, Hq=2)]


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(str(v) for v in f.values()))
@pytest.mark.parametrize("name", BATCHES)
@pytest.mark.parametrize("wide", [True, False])
def test_batches(name, form, wide):
    b = Shared(len(name), BATCHES[name], wide=wide, **form)
    check(b)
    check(b, causal=False, scale=0.3)


@pytest.mark.parametrize("form", FORMS[:3] + FORMS[5:6], ids=lambda f: "-".join(str(v) for v in f.values()))
def test_positions(form):
    # anywhere: before the prefix's end, before the first key, past the last
    b = Shared(5, [(300, ones(4, 5, 40, new=5)), (20, ones(2, 3, 30, new=2))], **form)
    r = np.random.RandomState(1)
    n = len(b.q)
    pos = r.randint(-3, 400, n).astype(np.int32)
    pos[:4] = [-1, 0, 299, 300]
    pos[-1], pos[-2] = (1 << 31) - 1, -(1 << 31)
    check(b, pos)


@pytest.mark.parametrize("form", FORMS[:2] + FORMS[5:6], ids=lambda f: "-".join(str(v) for v in f.values()))
def test_members_shorter_than_the_prefix(form):
    # prefix 200 of members with 1, 90, 200 and 260 tokens: lengths are cut afterwards, and the row of the
    # shortest, which comes first, names no page past its own
    b = Shared(7, [(200, [(1, 1), (1, 1), (1, 1), (60, 1)])], **form)
    b.lens[:3] = [1, 90, 200]
    for i, L in enumerate(b.lens):
        b.table[i, -(-int(L) // b.P):] = -1
    check(b)
    b.lens[3] = 150  # none reaches it
    b.table[3, -(-150 // b.P):] = -1
    check(b)


def test_rows_without_keys_and_of_no_sequence():
    import torch
    for form in FORMS[:2] + FORMS[5:6]:
        b = Shared(9, [(100, ones(3)), (50, ones(2))], **form)
        b.lens[1] = 0
        b.table[1] = -1
        b.offs = b.offs + 1  # a row before the first sequence and two behind the last
        b.q = torch.cat([b.q[:1], b.q, b.q[:2]])
        out = torch.full(b.q.shape, 768.0, dtype=b.q.dtype, device="cuda")
        lse = torch.full(b.q.shape[:2], 768.0, device="cuda")
        run(b, out=out, lse_out=lse)
        o, z = to_f64(out), to_f64(lse)
        for i in (0, -1, -2):
            assert (o[i] == 768).all() and (z[i] == 768).all()
        ref = b.ref()
        near(o[1:-2], z[1:-2], [x[1:-2] for x in ref], b.dtype, b.D)


def test_pages_outside_the_cache_read_as_zeros():
    for form in FORMS[:4] + FORMS[5:6]:
        b = Shared(11, [(300, ones(5, 1, 200, seed=1))], **form)
        b.table[:, 1] = 10 ** 6
        b.table[2, -2] = -5
        check(b)


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(str(v) for v in f.values()))
@pytest.mark.parametrize("strange", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("name", ["drafts", "mixed", "prompts"])
@pytest.mark.parametrize("wide", [True, False])
def test_what_a_row_does_not_see_does_not_reach_it(name, form, strange, wide):
    # keys and values that are no numbers at tokens that only the last rows of a sequence see: those rows are no
    # numbers, all others as without them
    b = Shared(37, BATCHES[name], wide=wide, **form)
    ref = list(b.ref())
    hit = np.zeros(len(b.q), bool)
    for s in range(len(b.lens)):
        if b.new[s] > 2:
            j = int(b.lens[s]) - 2  # the last two queries see it
            page = b.table[s, j // b.P]
            b.vc[page, j % b.P] = strange
            if s % 2:
                b.kc[page, j % b.P] = strange
            hit[b.offs[s + 1] - 2:b.offs[s + 1]] = True
    assert hit.any()
    out, lse = run(b)
    o, z = to_f64(out), to_f64(lse)
    assert not np.isfinite(o[hit]).any()
    near(o[~hit], z[~hit], [x[~hit] for x in ref], b.dtype, b.D)


@pytest.mark.parametrize("form", FORMS[:4] + FORMS[5:6], ids=lambda f: "-".join(str(v) for v in f.values()))
def test_positions_that_leave_keys_to_no_row(form):
    # every query stands at key 10 of its own: what lies behind it is no number
    b = Shared(41, [(150, [(90, 70), (60, 1), (40, 33)])], **form)
    pos = np.full(len(b.q), 160, np.int32)
    ref = b.ref(pos)
    for s in range(3):
        for j in range(161, int(b.lens[s])):
            b.vc[b.table[s, j // b.P], j % b.P] = float("nan")
            b.kc[b.table[s, j // b.P], j % b.P] = float("inf")
    out, lse = run(b, pos)
    near(to_f64(out), to_f64(lse), ref, b.dtype, b.D)


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("dtype,D,H,Hq,n", [("f16", 64, 1, 7, 2), ("f16", 128, 2, 2, 4), ("bf16", 128, 2, 16, 1),
                                            ("bf16", 64, 1, 4, 4)])
def test_few_rows_keep_their_weights(dtype, D, H, Hq, n, wide):
    # at most 16 rows of a kv head, in the group and in each sequence
    b = Shared(61, [(300, ones(n, 1, 500)), (77, ones(1, 20, 40))], dtype=dtype, D=D, P=16, H=H, Hq=Hq, wide=wide)
    for causal in (True, False):
        out, lse = run(b, causal=causal)
        near(to_f64(out), to_f64(lse), b.ref(None, causal, None), dtype, D, pairs=True)


def test_the_groups_do_not_change_the_result():
    # the same batch as one group, as two, as none: equal up to the order of the sums
    import torch
    form = FORMS[0]
    b = Shared(13, [(256, ones(6, 1, 80))], **form)
    whole = check(b)
    b.goff, b.pre = np.array([0, 2, 6], np.int32), np.array([256, 100], np.int32)
    halves = check(b)
    b.goff, b.pre = np.array([0], np.int32), np.array([], np.int32)
    none = check(b)
    for x in (halves, none):
        assert torch.allclose(whole[1], x[1], rtol=0, atol=2e-5)


def test_repeated_calls_give_identical_bits():
    import torch
    for name in ("wide", "ragged", "mixed", "prompts"):
        for form in FORMS[:2]:
            b = Shared(3, BATCHES[name], **form)
            a = run(b)
            for _ in range(3):
                c = run(b)
                assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


def test_offsets_clamped():
    # group offsets outside [0, num_seqs] are cut off
    b = Shared(17, [(200, ones(4))], **FORMS[0])
    b.goff = np.array([-3, 99], np.int32)
    b.max_gq = 4
    check(b)


def test_large_scores_and_a_dominant_key():
    # scores of several hundred; one key that outweighs all others, in the prefix or in the suffix
    for form in FORMS[:2] + FORMS[5:6]:
        for where in (100, 319):
            b = Shared(19, [(300, ones(3, 20, 30))], **form)
            for s in range(3):
                b.kc[b.table[s, where // b.P], where % b.P] = 0
            b.kc[b.table[0, where // b.P], where % b.P] = b.q[0, 0] * 4
            if where < 300 // b.P * b.P:
                pass  # one page for all
            else:
                for s in range(1, 3):
                    b.kc[b.table[s, where // b.P], where % b.P] = b.q[0, 0] * 4
            check(b, scale=1.0)


def test_graph_streams_and_workspace():
    # two captured calls that share a workspace, on a side stream, replayed with other inputs in place
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    b = Shared(23, BATCHES["ragged"], **FORMS[0])
    d = b.device()
    kw = dict(max_queries=b.max_q, max_group_queries=b.max_gq, return_lse=True)
    P = attn.PagedShape(len(b.lens), len(b.q), b.Hq, b.H, b.D, b.P, len(b.kc), b.table.shape[1], b.max_q)
    ws = torch.empty(attn.paged_prefix_workspace_bytes(P, len(b.pre), b.max_gq), dtype=torch.uint8, device="cuda")
    want = attn.paged_prefix_fwd(*d, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = attn.paged_prefix_fwd(*d, stream=side, workspace=ws, **kw)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    g = torch.cuda.CUDAGraph()
    q2 = d[0].flip(0).contiguous()
    with torch.cuda.graph(g):
        one = attn.paged_prefix_fwd(*d, workspace=ws, **kw)
        two = attn.paged_prefix_fwd(q2, *d[1:], workspace=ws, **kw)
    ws.fill_(255)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(one[0], want[0]) and torch.equal(one[1], want[1])
    assert torch.equal(two[0], attn.paged_prefix_fwd(q2, *d[1:], **kw)[0])


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("name", ["short", "wide", "mixed", "prompts"])
def test_captured_between_other_work(name, wide):
    # in one graph: the inputs come from a memset, a copy and another stream's kernels, the results go to
    # another stream and the inputs are overwritten right behind the call
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    b = Shared(47, BATCHES[name], wide=wide, **FORMS[0])
    d = b.device()
    kw = dict(max_queries=b.max_q, max_group_queries=b.max_gq, return_lse=True)
    want = attn.paged_prefix_fwd(*d, **kw)
    src = [x.clone() for x in d[:3]]
    live = [torch.empty_like(x) for x in d[:3]]
    got = [torch.empty_like(x) for x in want]
    big = torch.empty(1 << 26, device="cuda")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        for form in range(2):
            side.wait_stream(main)
            with torch.cuda.stream(side):
                big.fill_(form)  # so that the copies come late
                live[0].copy_(src[0])
            live[1].zero_()
            live[1].copy_(src[1])
            live[2].copy_(src[2])
            if form:  # the other stream's kernel is the last before the call, or a memset of this one is
                live[1].zero_()
                live[1].add_(src[1])
            else:
                big[:5].zero_()
            main.wait_stream(side)
            out, lse = attn.paged_prefix_fwd(*live, *d[3:], **kw)
            side.wait_stream(main)
            with torch.cuda.stream(side):
                got[0].copy_(out)
                got[1].copy_(lse)
            for x in live:
                x.fill_(float("nan"))
            main.wait_stream(side)
    for _ in range(4):
        for x in got:
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    # without a graph, in a chain: each call reads what the one before it wrote
    def chain(wait):
        x = d[0]
        for _ in range(6):
            x = attn.paged_prefix_fwd(x, *d[1:], **kw)[0]
            if wait:
                torch.cuda.synchronize()
        return x
    assert torch.equal(chain(False), chain(True))


def test_bounds_are_computed_when_not_given():
    import torch
    b = Shared(29, BATCHES["mixed"], **FORMS[0])
    a = run(b)
    c = run(b, max_queries=None, max_group_queries=None)
    assert torch.equal(a[0], c[0])


@pytest.mark.parametrize("form", FORMS[:2] + FORMS[5:6], ids=lambda f: "-".join(str(v) for v in f.values()))
def test_bounds_far_too_large(form):
    for name in ("one", "mixed", "drafts"):
        b = Shared(53, BATCHES[name], **form)
        check(b, max_queries=200000, max_group_queries=500000)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_through_the_paged_backward(dtype):
    # attn_paged_bwd takes the output and lse of the shared call: a shared page gets every reader's
    # gradient. Against the one with attn_paged_fwd's own results, and differences of the loss.
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    b = Shared(31, [(48, [(9, 3), (20, 1), (5, 5)])], dtype=dtype, D=64, P=16, H=1, Hq=2, hidden=0.0)
    q, kc, vc, table, lens, offs, goff, pre = b.device()
    do = torch.randn(q.shape, generator=torch.Generator().manual_seed(1)).to(q.dtype).cuda()
    out, lse = run(b)
    got = attn.paged_bwd(q, kc, vc, table, lens, offs, do, out=out, lse=lse, max_queries=b.max_q)
    o2, l2 = attn.paged_fwd(q, kc, vc, table, lens, offs, max_queries=b.max_q, return_lse=True)
    want = attn.paged_bwd(q, kc, vc, table, lens, offs, do, out=o2, lse=l2, max_queries=b.max_q)
    for x, y in zip(got, want):
        # D_i = dout . out sums D outputs of which each side rounds its own (half a step each), and
        # lse differ by 2^-20 or so: 2 u of the largest term for 16-bit types, 2^-16 for fp32
        tol = (2.0 ** -6 if dtype == "bf16" else 2.0 ** -16) * float(y.float().abs().max())
        assert float((x.float() - y.float()).abs().max()) <= tol
    if dtype == "f32":
        page, h = int(b.table[0, 1]), 1e-2
        loss = lambda: float((run(b)[0].double() * do.double()).sum())  # noqa: E731
        for x, grad in ((b.kc, got[1]), (b.vc, got[2])):
            at = (page, 3, 0, 5)
            v = float(x[at])
            x[at] = v + h
            up = loss()
            x[at] = v - h
            down = loss()
            x[at] = v
            # the loss is a sum of 2 * 9 * 64 fp32 outputs of size 1, each off by 2^-22 at most in a
            # difference of 2 h; the third derivative's h^2 / 6 of a few
            assert abs((up - down) / (2 * h) - float(grad[at])) <= 2 * 9 * 64 * 2.0 ** -22 / (2 * h) + 1e-3
