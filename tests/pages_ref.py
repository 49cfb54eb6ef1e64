"""Plain sequential restatement of the pages of a cache (attn_pages_*) in Python integers, and of
attention over a paged cache (attn_paged_prefix_fwd) in 64 bits, for the tests."""
import math

import numpy as np


class Pool:
    """block_table, seq_lens and refs as numpy int32 arrays; caches: arrays [num_pages, ...]."""

    def __init__(self, num_seqs, max_pages, page_size, num_pages, caches=()):
        self.P, self.n = page_size, num_pages
        self.table = np.full((num_seqs, max_pages), -1, np.int32)
        self.lens = np.zeros(num_seqs, np.int32)
        self.refs = np.zeros(num_pages, np.int32)
        self.caches = list(caches)

    def row_ok(self, s):
        return 0 <= s < len(self.lens)

    def page_ok(self, e):
        return 0 <= e < self.n

    def tokens(self, s):
        return min(max(int(self.lens[s]), 0), self.table.shape[1] * self.P)

    def put(self, s, b, page):
        old = int(self.table[s, b])
        if self.page_ok(page):
            self.refs[page] += 1
        self.table[s, b] = page
        if self.page_ok(old):
            self.refs[old] -= 1

    def fork(self, parents, children):
        for p, c in zip(parents, children):
            if not (self.row_ok(p) and self.row_ok(c)) or p == c:
                continue
            L = self.tokens(p)
            for b in range(self.table.shape[1]):
                e = int(self.table[p, b])
                self.put(c, b, e if b * self.P < L and self.page_ok(e) else -1)
            self.lens[c] = L

    def free(self, seqs):
        for s in seqs:
            if self.row_ok(s):
                for b in range(self.table.shape[1]):
                    self.put(s, b, -1)
                self.lens[s] = 0

    def reserve(self, new):
        """(taken, lacking)"""
        before = self.table.copy(), self.refs.copy()
        free = [p for p in range(self.n) if self.refs[p] == 0]
        at, copies = 0, []
        for s in range(len(self.lens)):
            L = self.tokens(s)
            end = min(L + max(int(new[s]), 0), self.table.shape[1] * self.P)
            if end <= L:
                continue
            for b in range(L // self.P, (end - 1) // self.P + 1):
                e = int(self.table[s, b])
                if self.page_ok(e) and self.refs[e] == 1:
                    continue
                page = free[at] if at < len(free) else None
                at += 1
                if page is None:  # still counts, with its old page given back, as the rule goes on
                    if self.page_ok(e):
                        self.refs[e] -= 1
                    continue
                if self.page_ok(e) and b * self.P < L:
                    copies.append((e, page))
                self.put(s, b, page)
        if at > len(free):
            self.table[:], self.refs[:] = before
            return 0, at - len(free)
        for e, page in copies:
            for x in self.caches:
                x[page] = x[e]
        return at, 0

    def compact(self):
        used = [p for p in range(self.n) if self.refs[p] > 0]
        U = len(used)
        to = np.full(self.n, -1, np.int32)
        holes = [p for p in range(U) if self.refs[p] == 0]
        movers = [p for p in used if p >= U]
        for p in used:
            to[p] = p
        for dst, src in zip(holes, movers):
            to[src] = dst
            for x in self.caches:
                x[dst] = x[src]
            self.refs[dst], self.refs[src] = self.refs[src], 0
        for s in range(self.table.shape[0]):
            for b in range(self.table.shape[1]):
                e = int(self.table[s, b])
                if self.page_ok(e) and to[e] >= 0:
                    self.table[s, b] = to[e]
        return to, U

    def check(self):
        count = np.bincount(self.table[(self.table >= 0) & (self.table < self.n)], minlength=self.n)
        assert np.array_equal(count, self.refs)


def attention(q, kc, vc, table, lens, offs, positions, causal, scale):
    """out [n, Hq, D], lse [n, Hq], mass = sum_j p_j |v_j| and noise = the largest sum of |q||k| scale
    of a row, all float64; rows of no sequence are left NaN with lse NaN."""
    n, Hq, D = q.shape
    P, H = kc.shape[1:3]
    out = np.full((n, Hq, D), np.nan)
    mass, lse, noise = np.zeros((n, Hq, D)), np.full((n, Hq), np.nan), np.zeros((n, Hq))
    for s in range(len(lens)):
        lo, hi = offs[s], offs[s + 1]
        L = min(max(int(lens[s]), 0), table.shape[1] * P)
        j = np.arange(L)
        page = table[s, j // P]
        ok = (page >= 0) & (page < kc.shape[0])
        page = np.where(ok, page, 0)
        k, v = (np.where(ok[:, None, None], x[page, j % P].astype(np.float64), 0.0) for x in (kc, vc))
        for i in range(lo, hi):
            pos = positions[i] if positions is not None else L - (hi - i)
            vis = min(L, int(pos) + 1) if causal else L
            for h in range(Hq):
                if vis <= 0:
                    lse[i, h] = -np.inf
                    continue
                a, b = k[:vis, h * H // Hq], q[i, h].astype(np.float64)
                x = a @ b * scale
                m = x.max()
                e = np.exp(x - m)
                lse[i, h] = m + math.log(e.sum())
                p = e / e.sum()
                out[i, h] = p @ v[:vis, h * H // Hq]
                mass[i, h] = p @ np.abs(v[:vis, h * H // Hq])
                noise[i, h] = (np.abs(a) @ np.abs(b)).max() * scale
    return out, lse, mass, noise


def near(out, lse, ref, dtype, D, pairs=False):
    """Checks a result against attention()'s. Tolerances:
    a score is a sum of D products in fp32, off by at most (D + 4) 2^-24 noise, its exponential by
    2^-21 more (the product with log2 e, the difference to the maximum, exp2), so a weight by a
    factor 1 + 2 w, w = (D + 4) 2^-24 noise + 2^-21, the normalisation included; 16-bit kernels
    round a weight to the type (u), or with ``pairs`` what that leaves of it once more (u u, and half of F16's
    smallest step, 2^-25, where a warp's largest weight is 2^8: 2^-33 of each of at most 2^12 values of 8 or
    less); sums of fp32 terms, a few thousand one after another in a
    tile's and the tiles' order, lose 2^-18 of the mass at most; the result is rounded once (u of
    it, and half of F16's smallest step). A lse is off by w + 2^-22 of itself."""
    o_ref, l_ref, mass, noise = ref
    u = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    w = (D + 4) * 2.0 ** -24 * noise + 2.0 ** -21
    seen = np.isfinite(l_ref)
    none = l_ref == -np.inf
    assert np.isnan(out[none]).all() and (lse[none] == -np.inf).all(), "rows without keys"
    tol = u * np.abs(o_ref) + (2 * w[..., None] + 2.0 ** -18 + (0.0 if dtype == "f32" else u * u if pairs else u)) * mass
    tol = tol + (2.0 ** -25 if dtype == "f16" else 0.0) + (2.0 ** -33 * 2 ** 12 * 8 if pairs and dtype == "f16" else 0.0)
    err = np.abs(out - o_ref)
    assert (err[seen] <= tol[seen]).all(), f"out off by {np.nanmax(err[seen] / tol[seen]):.2f} of what is allowed"
    el = np.abs(lse[seen] - l_ref[seen])
    tl = w[seen] + 2.0 ** -22 * (1 + np.abs(l_ref[seen]))
    assert (el <= tl).all(), f"lse off by {np.max(el / tl):.2f} of what is allowed"


class Shared:
    """A batch of groups. groups: [(prefix, [(own tokens, new tokens), ...]), ...]; a prefix of None is
    sequences of no group. Everything that no sequence holds is NaN. ``wide``: a table so wide that the
    call cannot know from its shape that there is nothing to be gained by sharing."""

    def __init__(self, seed, groups, *, dtype, D, P, H, Hq, hidden=float("nan"), wide=True):
        import torch
        self.dtype, self.D, self.P, self.H, self.Hq = dtype, D, P, H, Hq
        r = np.random.RandomState(seed)
        goff, pre, members, lens, new = [0], [], [], [], []
        for prefix, seqs in groups:
            members.append((prefix, len(lens), len(lens) + len(seqs)))
            for own, n in seqs:
                lens.append((prefix or 0) + own)
                new.append(n)
            if prefix is not None:
                pre.append(prefix)
        # groups without sequences of no group between them need none; a gap takes a group of prefix 0
        self.goff, self.pre = [], []
        for prefix, a, b in members:
            self.goff.append(a)
            self.pre.append(prefix or 0)
        if members and members[-1][0] is None:  # a last run of sequences of no group
            self.pre.pop()
        else:
            self.goff.append(len(lens))
        if not self.goff:
            self.goff = [0]
        self.goff, self.pre = np.array(self.goff, np.int32), np.array(self.pre, np.int32)
        self.lens, self.new = np.array(lens, np.int32), np.array(new, np.int32)
        self.offs = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        blocks = max(1, int(-(-self.lens.max() // P))) + 1
        if wide:
            blocks = max(blocks, (8 << 20) // (4 * H * D * P * len(lens)) + 1, 65536 // P)
        self.table = np.full((len(lens), blocks), -1, np.int32)
        pages = int((-(-self.lens // P)).sum()) + 3
        perm = r.permutation(pages)
        at, copies = 0, []
        for prefix, a, b in members:
            full = (prefix or 0) // P
            common = perm[at:at + full]
            at += full
            for i in range(a, b):
                held = min(full, -(-int(self.lens[i]) // P))
                own = -(-int(self.lens[i]) // P) - held
                self.table[i, :held] = common[:held]
                self.table[i, held:held + own] = perm[at:at + own]
                at += own
                if prefix and prefix % P and i > a and own > 0:
                    copies.append((self.table[a, full], self.table[i, full], prefix % P))
        tdt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
        kc, vc = (np.full((pages, P, H, D), hidden, np.float32) for _ in range(2))
        for s, L in enumerate(self.lens):
            for b in range(-(-int(L) // P)):
                e, rows = self.table[s, b], min(P, int(L) - b * P)
                for x in (kc, vc):
                    fresh = np.isnan(x[e, :rows, 0, 0]) if np.isnan(hidden) else np.ones(rows, bool)
                    x[e, :rows][fresh] = r.randn(int(fresh.sum()), H, D)
        for src, dst, n in copies:
            for x in (kc, vc):
                x[dst, :n] = x[src, :n]
        self.q = torch.from_numpy(r.randn(int(self.new.sum()), Hq, D).astype(np.float32)).to(tdt)
        self.kc, self.vc = (torch.from_numpy(x).to(tdt) for x in (kc, vc))
        self.max_q = int(self.new.max()) if len(new) else 0
        at = self.offs[np.clip(self.goff, 0, len(lens))]
        self.max_gq = max([int(x) for x in np.diff(at)] + [0])

    def device(self):
        """q, kc, vc, table, lens, offs, goff, pre on the GPU."""
        import torch
        i = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
        return (self.q.cuda(), self.kc.cuda(), self.vc.cuda(), i(self.table), i(self.lens), i(self.offs), i(self.goff),
                i(self.pre))

    def ref(self, positions=None, causal=True, scale=None):
        f = lambda t: t.float().numpy()  # noqa: E731
        return attention(f(self.q), f(self.kc), f(self.vc), self.table, self.lens, self.offs, positions, causal,
                         self.D ** -0.5 if scale is None else scale)
