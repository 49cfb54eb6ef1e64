"""The calls of a batch that shares a prompt, together as a program makes them: rotary positions with axes, a
prompt into pages, forks of it, room for each answer's tokens (copy on write), decode steps whose
attention reads the prompt once, answers that leave, and a compaction, against a plain cache for each
answer in 64 bits."""
import numpy as np
import pytest

from tests.gpu_util import to_f64
from tests.pages_ref import attention, near

pytestmark = pytest.mark.gpu


def i32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Program:
    """One prompt and its answers. Rows 0 .. answers-1 of the table are the answers, the last one the prompt."""

    def __init__(self, dtype, prompt, answers, P, H=2, Hq=8, D=128, pages=80, seed=0, width=500):
        import torch
        from exact_scaled_dot_flash_gb300 import attn
        self.attn, self.torch = attn, torch
        self.dt = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[dtype]
        self.dtype, self.P, self.H, self.Hq, self.D, self.n = dtype, P, H, Hq, D, answers
        rows = answers + 1
        self.table, self.lens, self.refs = i32(np.full((rows, width), -1)), i32(np.zeros(rows)), i32(np.zeros(pages))
        self.cache = [torch.full((pages, P, H, D), float("nan"), dtype=self.dt, device="cuda") for _ in range(2)]
        self.gen = torch.Generator().manual_seed(seed)
        self.freq, self.axes = attn.rope_frequencies(D)[0].cuda(), attn.rope_axes([D // 8, D // 8, D // 4]).cuda()
        self.shadow = [[] for _ in range(rows)]  # each row's (k, v) as the program computed them
        self.prompt = prompt
        self.step([rows - 1], prompt)

    def new(self, n, heads):
        return self.torch.randn((n, heads, self.D), generator=self.gen).to(self.dt).cuda()

    def step(self, rows, n):
        """n new tokens for each of the rows, in ascending order: their output, or None for the prompt."""
        torch, attn = self.torch, self.attn
        total = n * len(rows)
        new = np.zeros(len(self.shadow))
        new[rows] = n
        result = attn.pages_reserve(self.table, self.lens, self.refs, i32(new), self.cache, page_size=self.P)
        assert int(result[1]) == 0
        at = np.array([sum(len(k) for k, _ in self.shadow[r]) for r in rows])
        p = (at[:, None] + np.arange(n)).ravel()
        pos = i32(np.stack([p // 100, p % 100, p]))  # a grid, and the order
        qkv = self.new(total, self.Hq + 2 * self.H)
        q, k = attn.rope(qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.H], pos, self.freq, axes=self.axes)
        v = qkv[:, self.Hq + self.H:]
        table = self.table.cpu().numpy()
        row = np.repeat(rows, n)
        page = torch.from_numpy(table[row, p // self.P].astype(np.int64)).cuda()
        for x, y in zip(self.cache, (k, v)):  # the program's own write
            x[page, torch.from_numpy(p % self.P).cuda()] = y
        self.lens += i32(new)
        for i, r in enumerate(rows):
            self.shadow[r] = self.shadow[r] + [tuple(x[i * n:(i + 1) * n].float().cpu().numpy() for x in (k, v))]
        return q

    def attend(self, q, rows, n, **kw):
        """Attention of the rows' newest n tokens; the other rows of the table have no queries."""
        off = np.concatenate([[0], np.cumsum([n if s in rows else 0 for s in range(self.n)])])
        return self.attn.paged_prefix_fwd(q, *self.cache, self.table[:self.n], self.lens[:self.n], i32(off),
                                          i32([0, self.n]), i32([self.prompt]), max_queries=n,
                                          max_group_queries=n * len(rows), return_lse=True, **kw)

    def check(self, q, rows, n, out, lse):
        refs = []
        for i, r in enumerate(rows):
            k, v = (np.concatenate([x[j] for x in self.shadow[r]]) for j in (0, 1))
            L = len(k)
            refs.append(attention(q[i * n:(i + 1) * n].float().cpu().numpy(), k[None], v[None], np.zeros((1, 1), np.int64),
                                  np.array([L]), np.array([0, n]), None, True, self.D ** -0.5))
        near(to_f64(out), to_f64(lse), [np.concatenate(x) for x in zip(*refs)], self.dtype, self.D)

    def counts(self):
        t = self.table.cpu().numpy()
        assert np.array_equal(np.bincount(t[t >= 0], minlength=len(self.refs)), self.refs.cpu().numpy())


@pytest.mark.parametrize("dtype,prompt,answers,P", [("bf16", 301, 5, 16), ("f16", 256, 12, 64), ("f32", 77, 3, 8),
                                                    ("bf16", 130, 2, 24)])
def test_answers_to_one_prompt(dtype, prompt, answers, P):
    m = Program(dtype, prompt, answers, P)
    attn = m.attn
    attn.pages_fork(m.table, m.lens, m.refs, i32([answers] * answers), i32(np.arange(answers)), page_size=P)
    for r in range(answers):
        m.shadow[r] = list(m.shadow[answers])
    m.counts()
    rows = list(range(answers))
    for n in (1, 1, 5, 1):
        q = m.step(rows, n)
        m.check(q, rows, n, *m.attend(q, rows, n))
        m.counts()
    # answer 0 leaves, and goes on as a copy of answer 1
    attn.pages_free(m.table, m.lens, m.refs, i32([0]))
    attn.pages_fork(m.table, m.lens, m.refs, i32([1]), i32([0]), page_size=P)
    m.shadow[0] = list(m.shadow[1])
    q = m.step(rows, 1)
    before = m.attend(q, rows, 1)
    m.check(q, rows, 1, *before)
    # an answer ends; the pool is compacted; the others' results keep their bits
    if answers > 2:
        rows = rows[:-1]
        attn.pages_free(m.table, m.lens, m.refs, i32([answers - 1]))
    _, used = attn.pages_compact(m.table, m.refs, m.cache)
    m.counts()
    assert int(used) == int((m.refs > 0).sum()) and bool((m.refs[:int(used)] > 0).all())
    m.n = len(rows)
    after = m.attend(q[:len(rows)], rows, 1)
    m.check(q[:len(rows)], rows, 1, *after)
    q = m.step(rows, 2)
    m.check(q, rows, 2, *m.attend(q, rows, 2))
    assert attn.device_status(0, clear=True) == 0


def test_calls_on_two_streams_at_once():
    import torch
    m = Program("bf16", 400, 6, 16, width=200)
    attn = m.attn
    attn.pages_fork(m.table, m.lens, m.refs, i32([6] * 6), i32(np.arange(6)), page_size=16)
    for r in range(6):
        m.shadow[r] = list(m.shadow[6])
    rows = list(range(6))
    q = m.step(rows, 1)
    want = m.attend(q, rows, 1)
    other = (q.float() * 0.5).to(q.dtype)
    want2 = m.attend(other, rows, 1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(20):
        for st, x in zip(streams, (q, other)):
            got.append(m.attend(x, rows, 1, stream=st))
    torch.cuda.synchronize()
    for i, (o, z) in enumerate(got):
        w = (want, want2)[i % 2]
        assert torch.equal(o, w[0]) and torch.equal(z, w[1])


def test_a_decode_loop_in_one_graph():
    # reserve, attention and the pool's other calls captured together and replayed, lengths moving on the device
    import torch
    m = Program("f16", 200, 4, 16, width=30)
    attn = m.attn
    attn.pages_fork(m.table, m.lens, m.refs, i32([4] * 4), i32(np.arange(4)), page_size=16)
    for r in range(4):
        m.shadow[r] = list(m.shadow[4])
    rows = list(range(4))
    q = m.step(rows, 1)
    new = i32([1, 1, 1, 1, 0])
    ones = i32(np.arange(5))
    result = torch.zeros(2, dtype=torch.int32, device="cuda")
    P = attn.PagedShape(4, 4, m.Hq, m.H, m.D, 16, 80, 30, 1)
    ws = torch.empty(attn.paged_prefix_workspace_bytes(P, 1, 4), dtype=torch.uint8, device="cuda")
    pws = torch.empty(attn.pages_workspace_bytes(attn.Pages(5, 30, 16, 80)), dtype=torch.uint8, device="cuda")
    goff, pre = i32([0, 4]), i32([200])
    kv = [torch.zeros((4, m.H, m.D), dtype=m.dt, device="cuda") for _ in range(2)]
    table, lens = m.table[:4], m.lens[:4]

    def body():
        attn.pages_reserve(m.table, m.lens, m.refs, new, m.cache, page_size=16, result=result, workspace=pws)
        page = table.gather(1, (lens // 16).long()[:, None])[:, 0].long()
        for x, y in zip(m.cache, kv):
            x[page, (lens % 16).long()] = y
        m.lens.add_(new)
        return attn.paged_prefix_fwd(q, *m.cache, table, lens, ones, goff, pre, max_queries=1, max_group_queries=4,
                                     return_lse=True, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        for x, h in zip(kv, (1, 2)):
            x.copy_(m.new(4, m.H))
        for r in rows:
            m.shadow[r] = m.shadow[r] + [tuple(x[r:r + 1].float().cpu().numpy() for x in kv)]
        body()  # once eagerly
        side.synchronize()
    with torch.cuda.graph(g):
        out, lse = body()
    for _ in range(20):  # past the end of a page
        for x in kv:
            x.copy_(m.new(4, m.H))
        for r in rows:
            m.shadow[r] = m.shadow[r] + [tuple(x[r:r + 1].float().cpu().numpy() for x in kv)]
        g.replay()
        torch.cuda.synchronize()
        assert result.tolist()[1] == 0
        m.check(q, rows, 1, out, lse)
    m.counts()
