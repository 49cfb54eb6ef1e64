"""The pages of a cache on the GPU (attn_pages_*) against a sequential restatement in integers:
every table entry, length, count and byte has to be equal."""
import numpy as np
import pytest

from tests.pages_ref import Pool

pytestmark = pytest.mark.gpu


class Both:
    """A pool on the GPU and its restatement, changed together and compared after every step."""

    def __init__(self, num_seqs, max_pages, page_size, num_pages, shapes=(), seed=0):
        import torch
        self.t = torch
        r = np.random.RandomState(seed)
        np_dt = {"u8": np.uint8, "i16": np.int16, "f32": np.float32}
        arrays = [r.randint(0, 200, (num_pages, *s)).astype(np_dt[d]) for d, s in shapes]
        self.ref = Pool(num_seqs, max_pages, page_size, num_pages, [a.copy() for a in arrays])
        self.P = page_size
        self.table, self.lens, self.refs = (torch.from_numpy(a.copy()).cuda()
                                            for a in (self.ref.table, self.ref.lens, self.ref.refs))
        self.caches = [torch.from_numpy(a).cuda() for a in arrays]

    def ints(self, a):
        return self.t.tensor(list(a), dtype=self.t.int32, device="cuda")

    def compare(self):
        for name in ("table", "lens", "refs"):
            assert np.array_equal(getattr(self, name).cpu().numpy(), getattr(self.ref, name)), name
        for x, y in zip(self.caches, self.ref.caches):
            assert np.array_equal(x.cpu().numpy(), y)
        self.ref.check()

    def fork(self, parents, children):
        from exact_scaled_dot_flash_gb300 import attn
        attn.pages_fork(self.table, self.lens, self.refs, self.ints(parents), self.ints(children), page_size=self.P)
        self.ref.fork(parents, children)
        self.compare()

    def free(self, seqs):
        from exact_scaled_dot_flash_gb300 import attn
        attn.pages_free(self.table, self.lens, self.refs, self.ints(seqs))
        self.ref.free(seqs)
        self.compare()

    def reserve(self, new, write=True):
        from exact_scaled_dot_flash_gb300 import attn
        got = attn.pages_reserve(self.table, self.lens, self.refs, self.ints(new), self.caches, page_size=self.P)
        want = self.ref.reserve(new)
        assert tuple(got.tolist()) == want
        self.compare()
        if write and not want[1]:  # the tokens arrive
            add = np.minimum(np.maximum(new, 0), self.ref.table.shape[1] * self.P - self.ref.lens)
            self.ref.lens += add.astype(np.int32)
            self.lens += self.ints(add)
        return want

    def compact(self):
        from exact_scaled_dot_flash_gb300 import attn
        page_map, used = attn.pages_compact(self.table, self.refs, self.caches)
        to, U = self.ref.compact()
        assert int(used) == U and np.array_equal(page_map.cpu().numpy(), to)
        self.compare()


SHAPES = [("i16", (4, 3, 8)), ("u8", (4, 3, 5)), ("f32", (3, 2))]  # 16-byte pages, odd bytes, scales


@pytest.mark.parametrize("S,M,P,N,seed", [(5, 6, 4, 23, 0), (1, 1, 1, 1, 1), (40, 9, 3, 150, 2), (300, 4, 16, 1100, 3),
                                          (17, 300, 2, 5000, 4), (1500, 3, 8, 9000, 5)])
def test_a_long_run(S, M, P, N, seed):
    b = Both(S, M, P, N, SHAPES, seed)
    r = np.random.RandomState(seed)
    lacked = 0
    for step in range(30 if S < 300 else 10):
        b.reserve(np.where(r.rand(S) < 0.7, r.randint(-1, 2 * P + 2, S), 0))
        live = np.flatnonzero(b.ref.lens > 0)
        if len(live) and S > 1:
            order = r.permutation(S)
            children = order[:r.randint(1, max(2, S // 4))]
            parents = np.setdiff1d(live, children)
            if len(parents):
                b.fork(r.choice(parents, len(children)).tolist(), children.tolist())
        if step % 3 == 2:
            b.free(r.permutation(S)[:max(1, S // 3)].tolist())
        if step % 4 == 3:
            b.compact()
        lacked += b.reserve(r.randint(0, 2, S))[1] > 0
    b.compact()
    b.free(range(S))
    assert b.ref.refs.sum() == 0


def test_the_last_writer_keeps_a_page():
    # a part-filled page of 4 rows: when all write, three copy and the last keeps it; when three do, all three copy
    for writers, taken in (([1, 1, 1, 1], 3), ([1, 0, 1, 1], 3), ([0, 0, 0, 1], 1)):
        b = Both(4, 3, 4, 12, SHAPES)
        b.reserve([6, 0, 0, 0])
        b.fork([0, 0, 0], [1, 2, 3])
        assert b.reserve(writers) == (taken, 0)


def test_all_or_nothing():
    b = Both(3, 4, 4, 5, SHAPES)
    b.reserve([9, 4, 0])  # 3 + 1 pages
    assert b.reserve([0, 0, 12]) == (0, 2)
    assert b.reserve([0, 0, 4]) == (1, 0)
    assert b.reserve([4, 1, 1]) == (0, 3)
    b.free([1])
    assert b.reserve([4, 0, 0]) == (1, 0)


def test_reserved_pages_of_a_parent_stay_its_own():
    b = Both(3, 6, 4, 20, SHAPES)
    b.reserve([5, 0, 0])
    b.reserve([9, 0, 0], write=False)  # room that nothing has been written to yet
    b.fork([0], [1])
    assert (b.ref.table[1] >= 0).sum() == 2
    assert b.reserve([9, 9, 0])[1] == 0


def test_rows_and_pages_outside_are_passed_over():
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    b = Both(4, 3, 2, 9, SHAPES)
    b.reserve([3, 0, 2, 0])
    b.fork([0, -1, 9, 2, 1 << 30], [1, 3, 3, 2, -(1 << 31)])
    b.free([-7, 4, 1 << 30])
    b.free([0, 0, 0])  # counts once
    src, dst = b.ints([0, 5, -1, 3, 9]), b.ints([6, 5, 2, 1 << 30, 1])
    attn.pages_copy(b.caches, src, dst)
    for x in b.ref.caches:
        x[6] = x[0]
    b.compare()
    # entries that name no page of the pool count as none
    b.table[3, 0] = 77
    b.ref.table[3, 0] = 77
    b.reserve([1, 1, 1, 1])
    b.compact()
    torch.cuda.synchronize()


def test_the_same_child_or_row_twice_keeps_the_counts():
    from exact_scaled_dot_flash_gb300 import attn
    b = Both(8, 70, 2, 700)
    b.reserve([140, 100, 60, 0, 0, 0, 0, 0])
    attn.pages_fork(b.table, b.lens, b.refs, b.ints([0, 1, 2, 3, 4]), b.ints([3, 3, 3, 4, 0]), page_size=2)
    t = b.table.cpu().numpy()
    assert np.array_equal(np.bincount(t[t >= 0], minlength=700), b.refs.cpu().numpy())


def test_empty_pools_and_calls():
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    b = Both(3, 2, 4, 6, SHAPES)
    b.fork([], [])
    b.free([])
    b.compact()
    assert b.reserve([0, 0, -3]) == (0, 0)
    attn.pages_copy(b.caches, b.ints([]), b.ints([]))
    attn.pages_copy([], b.ints([1]), b.ints([2]))
    none = Both(3, 2, 4, 0)
    assert none.reserve([1, 0, 1]) == (0, 2)
    none.compact()
    rows = Both(0, 2, 4, 5, SHAPES)
    assert rows.reserve([]) == (0, 0)
    rows.compact()
    blocks = Both(2, 0, 4, 5, SHAPES)
    blocks.fork([0], [1])
    blocks.free([0])
    assert blocks.reserve([3, 3]) == (0, 0)
    blocks.compact()
    torch.cuda.synchronize()


def test_room_ends_at_the_table():
    b = Both(2, 3, 4, 20, SHAPES)
    assert b.reserve([100, 11]) == (6, 0)
    assert b.reserve([5, 5]) == (0, 0)
    b.lens.fill_(1 << 30)
    b.ref.lens[:] = 1 << 30
    assert b.reserve([(1 << 31) - 1, 1], write=False) == (0, 0)
    b.lens.fill_(-5)
    b.ref.lens[:] = -5
    assert b.reserve([(1 << 31) - 1, 1], write=False) == (0, 0)


def test_many_buffers_and_views():
    # 70 buffers take two launches; slices of one allocation, addresses that vectors do not fit
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    r = np.random.RandomState(3)
    whole = torch.from_numpy(r.randint(0, 255, (70, 13, 7, 6)).astype(np.uint8)).cuda()
    odd = torch.from_numpy(r.randint(0, 255, 13 * 32 + 1).astype(np.uint8)).cuda()[1:].view(13, 32)
    big = torch.from_numpy(r.randn(13, 5000, 3).astype(np.float32)).cuda()
    caches = [*whole, odd, big]
    want = [c.clone() for c in caches]
    src, dst = [3, 7, 3, 0], [1, 12, 2, 11]
    for w in want:
        w[dst] = w[src]
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    attn.pages_copy(caches, i(src), i(dst))
    for c, w in zip(caches, want):
        assert torch.equal(c, w)


def test_in_a_graph_and_on_another_stream():
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    b = Both(6, 5, 4, 40, SHAPES)
    b.reserve([9, 6, 0, 0, 0, 0])
    new, parents, kids = b.ints([0, 0, 1, 1, 1, 0]), b.ints([0, 0, 1]), b.ints([2, 3, 4])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(attn.pages_workspace_bytes(attn.Pages(6, 5, 4, 40)), dtype=torch.uint8, device="cuda")
    result, page_map, used = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (2, 40, 1))

    def step(**kw):
        attn.pages_free(b.table, b.lens, b.refs, kids, **kw)
        attn.pages_fork(b.table, b.lens, b.refs, parents, kids, page_size=4, **kw)
        attn.pages_reserve(b.table, b.lens, b.refs, new, b.caches, page_size=4, result=result, workspace=ws, **kw)
        attn.pages_compact(b.table, b.refs, b.caches, page_map=page_map, used=used, workspace=ws, **kw)

    def ref_step():
        b.ref.free([2, 3, 4])
        b.ref.fork([0, 0, 1], [2, 3, 4])
        b.ref.reserve([0, 0, 1, 1, 1, 0])
        b.ref.compact()
    step(stream=side)
    side.synchronize()
    ref_step()
    b.compare()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
        ref_step()
        torch.cuda.synchronize()
        b.compare()


def test_large_pages_past_32_bits():
    # 2^31 bytes lie before the last pages of the buffer
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    x = torch.zeros((5, (1 << 29) + 16), dtype=torch.uint8, device="cuda")
    x[4, -3:] = torch.tensor([5, 6, 7], dtype=torch.uint8, device="cuda")
    x[0, :2] = 9
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    attn.pages_copy([x], i([4, 0]), i([1, 3]))
    assert torch.equal(x[1], x[4]) and torch.equal(x[3], x[0]) and int(x[2].max()) == 0
