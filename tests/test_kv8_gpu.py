"""The 8-bit paged cache on the GPU (attn_kv8_write, attn_kv8_read, attn_paged_kv8_fwd) against
its restatement in 64 bits (kv8_ref.py).

Codes and scales are defined exactly, so they are compared for equality. Values read back are
code * scale rounded once: half a step of the output type (the fp32 product adds 2^-24).

Attention, element by element, with u half a step of the type of q (bf16 2^-8, f16 2^-11, f32
2^-24), A = sum_j p_j |v_j| and b = max_j scale sum_d |q_d| |k_jd|:
  u |o|              the output's rounding,
  u A                the rounding of p_j v_scale_j (F16 and BF16 only; to F16 for both),
  2^-24 (16 b + 128) A   fp32: a score's dot product is off by a few 2^-24 b and moves p_j by as
                     much; exp2 by 2^-22, the sums by some 2^-24 for each of their steps,
  2^-24 n max|v|     F16 and BF16: the products are F16 with the row's largest p_j v_scale_j (or a
                     bound of it) brought to (1/2, 1], so one below 2^-14 of that is subnormal and
                     off by up to 2^-25 of at most twice the largest scale, times a code; n of them
                     add up. It shows where the keys that count hold zeros in an element,
  2^-24              F16 outputs below its normal range,
  2^-126 n max|v|    the range of fp32: exp2 gives 0 for a p_j that is below 2^-126 of the largest
                     (a key whose p_j is nearly 1 and whose element is 0 leaves such sums alone).
The log-sum-exp: 2^-24 (16 b + 128 + 4 |lse|)."""
import numpy as np
import pytest

from tests import kv8_ref as R
from tests.gpu_util import to_f64

pytestmark = pytest.mark.gpu
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _clean_status():
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    torch.cuda.synchronize()
    attn.device_status(torch.cuda.current_device(), clear=True)
    yield
    torch.cuda.synchronize()
    assert attn.device_status(torch.cuda.current_device(), clear=True) == 0, "a kernel wait timed out"


def tdt(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
            "int8": torch.int8, "e4m3": torch.float8_e4m3fn}[name]


def gpu(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Problem:
    """Sequences with lengths ``lens`` of which the last ``new`` tokens are new, over scattered
    pages of a cache that earlier writes left full of codes."""

    def __init__(self, seed, lens, new, dtype="bf16", fmt="int8", D=64, P=16, G=8, H=2, Hq=None, spare=2, loud=1.0):
        import torch
        r = np.random.RandomState(seed)
        self.lens, self.new = np.asarray(lens, np.int32), np.asarray(new, np.int32)
        self.dtype, self.fmt, self.D, self.P, self.G, self.H, self.Hq = dtype, fmt, D, P, G, H, Hq or H
        need = -(-self.lens // P)
        self.pages = int(need.sum()) + spare
        perm = r.permutation(self.pages)
        self.table = np.full((len(lens), max(1, int(need.max()))), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = perm[at:at + n]
            at += n
        self.offs = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.tokens = int(self.offs[-1])
        cast = lambda a: torch.from_numpy(a).to(tdt(dtype))  # noqa: E731
        big = np.exp(r.randn(self.tokens, H, 1) * 0.7) * loud
        self.k = cast(r.randn(self.tokens, H, D) * big)
        self.v = cast(r.randn(self.tokens, H, D) * big)
        self.q = cast(r.randn(self.tokens, self.Hq, D) * 1.5)
        self.kc, self.vc = (self.codes(r) for _ in range(2))
        self.ks, self.vs = (self.scales(r) for _ in range(2))

    def codes(self, r):
        c = r.randint(0, 256, (self.pages, self.P, self.H, self.D)).astype(np.uint8)
        if self.fmt == "int8":
            return np.where(c == 128, 129, c).astype(np.uint8)
        return np.where((c & 0x7f) == 0x7f, 0, c).astype(np.uint8)

    def scales(self, r):
        shape = (self.pages, self.H, self.P // self.G)
        if self.fmt == "int8":
            return (np.exp(r.randn(*shape) * 0.5) * 0.02).astype(np.float32)
        return (2.0 ** r.randint(-9, -6, shape)).astype(np.float32)

    def cache(self):
        return [gpu(self.kc).view(tdt(self.fmt)), gpu(self.vc).view(tdt(self.fmt)), gpu(self.ks), gpu(self.vs),
                gpu(self.table), gpu(self.lens)]

    def written(self):
        """The cache after the write, in 64 bits: codes and scales of k and v."""
        out = []
        for x, c, s in ((self.k, self.kc, self.ks), (self.v, self.vc, self.vs)):
            c, s = c.copy(), s.copy()
            R.write_one(x.double().numpy(), c, s, self.table, self.lens, self.offs, self.fmt, self.G)
            out += [c, s]
        return out


def same_cache(p, cache, want, what=""):
    import torch
    kc, ks, vc, vs = want
    for name, got, ref in (("k_scale", cache[2], ks), ("v_scale", cache[3], vs)):
        assert np.array_equal(got.cpu().numpy(), ref, equal_nan=True), what + name
    for name, got, ref in (("k_cache", cache[0], kc), ("v_cache", cache[1], vc)):
        g = got.view(torch.uint8).cpu().numpy()
        bad = R.values(g, p.fmt) != R.values(ref, p.fmt)  # e4m3: -0 is 0
        assert not bad.any(), f"{what}{name}: {bad.sum()} codes differ, first at {np.argwhere(bad)[0]}"


def write(p, cache, k=None, v=None, **kw):
    from exact_scaled_dot_flash_gb300 import attn
    attn.kv8_write(p.k.cuda() if k is None else k, p.v.cuda() if v is None else v, *cache, gpu(p.offs), **kw)


WRITES = [
    dict(lens=[5], new=[5], G=8),
    dict(lens=[1], new=[1], G=1, P=1, D=16, H=1),
    dict(lens=[40, 3, 17, 64], new=[1, 1, 1, 1], G=8, fmt="e4m3"),
    dict(lens=[40, 3, 17, 64], new=[1, 2, 1, 3], G=16, loud=20.0),
    dict(lens=[40, 3, 17, 64], new=[1, 2, 1, 3], G=16, loud=20.0, fmt="e4m3", dtype="f16"),
    dict(lens=[70, 1, 33, 130], new=[70, 0, 30, 5], G=4, dtype="f32", H=3, D=32),
    dict(lens=[70, 1, 33, 130], new=[70, 0, 30, 5], G=4, dtype="f32", H=3, D=32, fmt="e4m3"),
    dict(lens=[300, 257], new=[299, 100], G=128, P=128, D=128, H=2),           # a CTA for a unit
    dict(lens=[300, 257], new=[299, 100], G=128, P=128, D=128, H=1, fmt="e4m3", dtype="f16"),
    dict(lens=[500], new=[400], G=256, P=256, D=128, H=1, dtype="f32"),        # more than the registers keep
    dict(lens=[100, 90], new=[61, 50], G=24, P=48, D=64, H=5),                 # sizes that are no powers of two
    dict(lens=[100, 90], new=[61, 50], G=3, P=9, D=16, H=7, fmt="e4m3"),
    dict(lens=list(range(1, 71)), new=[1 + i % 3 if i else 1 for i in range(70)], G=2, P=4, D=16, H=1),
    dict(lens=[9, 30], new=[20, 4], G=8),                                      # more new tokens than the length
]


@pytest.mark.parametrize("kw", WRITES, ids=lambda kw: "-".join(str(v) for k, v in kw.items() if k not in ("lens", "new")))
def test_write(kw):
    kw = dict(kw)
    p = Problem(3, kw.pop("lens"), kw.pop("new"), **kw)
    cache, want = p.cache(), p.written()
    write(p, cache)
    same_cache(p, cache, want)
    write(p, cache)  # again: nothing changes
    same_cache(p, cache, want, "second call: ")


@pytest.mark.parametrize("dtype,fmt", [("bf16", "int8"), ("f16", "e4m3"), ("f32", "int8")])
def test_write_strided_and_unaligned(dtype, fmt):
    import torch
    p = Problem(4, [37, 80], [20, 33], dtype=dtype, fmt=fmt, H=3)
    want = p.written()
    for shift in (0, 1):  # slices of a fused projection; then one element off every boundary
        buf = torch.zeros((p.tokens, 4 + 2 * 3, 64 + shift), dtype=tdt(dtype)).cuda()
        buf[:, 4:7, shift:], buf[:, 7:, shift:] = p.k.cuda(), p.v.cuda()
        cache = p.cache()
        write(p, cache, buf[:, 4:7, shift:], buf[:, 7:, shift:])
        same_cache(p, cache, want, f"shift {shift}: ")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_write_ties_and_extremes(fmt):
    # values on and next to the borders between codes, zeros, tiny and huge magnitudes
    import torch
    p = Problem(5, [64], [64], dtype="f32", fmt=fmt, G=4, P=16, H=1)
    r = np.random.RandomState(0)
    x = np.zeros((64, 1, 64), np.float32)
    for g in range(16):
        amax = np.float32([0, 1e-38, 1e-30, 2.0 ** -93, 3e38, 127, 448, 1.7, 12.3, 0.031, 1e10, 127.5, 447, 449, 1, 5e-39][g])
        s = R.new_scale(float(amax), fmt)
        top = 127 if fmt == "int8" else 448
        half = np.clip((r.randint(-2 * top, 2 * top, (4, 1, 64)) / 2.0) * float(s), -float(amax), float(amax))
        half = half.astype(np.float32)
        y = np.nextafter(half, np.float32(np.inf) * r.choice([-1, 1], half.shape).astype(np.float32))
        y = np.where(r.rand(*half.shape) < 0.5, half, y)
        x[4 * g:4 * g + 4] = np.clip(y, -amax, amax)
        x[4 * g, 0, 0] = amax
    p.k, p.v = torch.from_numpy(x), torch.from_numpy(-x)
    cache = p.cache()
    write(p, cache)
    same_cache(p, cache, p.written())


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_write_not_finite(fmt):
    # a NaN or an infinity makes its group (of its head) NaN, until the group starts over
    import torch
    p = Problem(6, [24, 20], [24, 3], fmt=fmt, G=4, H=2)
    p.k[5, 1, 7], p.v[9, 0, 0], p.k[25, 0, 3] = float("nan"), float("inf"), float("-inf")
    cache = p.cache()
    write(p, cache)
    same_cache(p, cache, p.written())
    assert np.isnan(cache[2].cpu().numpy()).sum() == 2 and np.isnan(cache[3].cpu().numpy()).sum() == 1
    p2 = Problem(6, [24, 20], [24, 3], fmt=fmt, G=4, H=2)  # the same tokens, finite
    write(p2, cache)
    ks = cache[2].cpu().numpy()
    assert np.isnan(ks).sum() == 1  # sequence 1's tokens 17..19 join a group that was NaN and started at 16
    assert np.isfinite(ks[p.table[0, :2]]).all() and torch.isfinite(cache[3]).all()


def test_write_leaves_the_rest_alone():
    import torch
    p = Problem(7, [30, 12, 16], [4, 2, 3], G=8, fmt="e4m3")
    p.table[1, 0] = p.pages + 5   # a page outside the cache
    p.table[2, 0] = -1
    cache, want = p.cache(), p.written()
    write(p, cache)
    same_cache(p, cache, want)
    got = cache[0].view(torch.uint8).cpu().numpy()
    touched = np.zeros(got.shape[:2], bool)
    touched[p.table[0, 1], 8:14] = True  # tokens 24..29 (24, 25 may be brought to a larger scale)
    assert np.array_equal(got[~touched], p.kc[~touched])


@pytest.mark.parametrize("fmt,G", [("int8", 16), ("e4m3", 4), ("int8", 1)])
def test_decode_appends_token_by_token(fmt, G):
    # every step's codes and scales, over three pages, with scales that grow
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    p = Problem(8, [48, 48], [48, 48], fmt=fmt, G=G)
    cache = p.cache()
    kc, ks = p.kc.copy(), p.ks.copy()
    for step in range(1, 48, 3):
        lens = np.array([step, step + 1], np.int32)
        k = p.k[[step - 1, 48 + step]] * (1.0 + step)
        offs = np.array([0, 1, 2], np.int32)
        R.write_one(k.double().numpy(), kc, ks, p.table, lens, offs, fmt, G)
        attn.kv8_write(k.cuda(), k.cuda(), *cache[:5], gpu(lens), gpu(offs))
        assert np.array_equal(cache[2].cpu().numpy(), ks)
        assert np.array_equal(R.values(cache[0].view(torch.uint8).cpu().numpy(), fmt), R.values(kc, fmt))


@pytest.mark.parametrize("dtype,fmt,D,G,P", [("bf16", "int8", 64, 8, 16), ("f16", "e4m3", 128, 1, 16),
                                             ("f32", "int8", 16, 4, 4), ("f32", "e4m3", 32, 48, 48)])
def test_read(dtype, fmt, D, G, P):
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    p = Problem(9, [61, 5, 0, 100], [1, 1, 0, 1], dtype=dtype, fmt=fmt, D=D, G=G, P=P, H=3)
    p.table[3, 0] = -1
    p.vs[p.table[0, 0], 1, 0] = np.nan
    cache = p.cache()
    starts = np.array([50, -2, 3, 0], np.int32)
    offs = np.array([2, 22, 31, 33, 133], np.int32)  # rows 0, 1 and 133.. of no sequence
    for st in (None, starts):
        outs = [torch.full((140, 3, D), 7.0, dtype=tdt(dtype), device="cuda") for _ in range(2)]
        attn.kv8_read(*cache, gpu(offs), starts=None if st is None else gpu(st), k_out=outs[0], v_out=outs[1])
        for got, c, s in ((outs[0], p.kc, p.ks), (outs[1], p.vc, p.vs)):
            ref = R.read_rows(c, s, p.table, p.lens, offs, 140, fmt, starts=st, fill=7.0)
            g = to_f64(got)
            assert np.array_equal(np.isnan(g), np.isnan(ref))
            ok = ~np.isnan(ref)
            tol = (U[dtype] + 2.0 ** -24) * np.abs(ref[ok]) + (2.0 ** -25 if dtype == "f16" else 0.0)
            assert (np.abs(g[ok] - ref[ok]) <= tol).all()
    k, v = attn.kv8_read(*cache, gpu(np.concatenate([[0], np.cumsum(p.lens)]).astype(np.int32)))
    assert k.dtype == torch.bfloat16 and tuple(k.shape) == (166, 3, D)


def attend(p, cache, positions=None, causal=True, scale=None, **kw):
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    out = torch.full(p.q.shape, 777.0, dtype=p.q.dtype, device="cuda")
    return attn.paged_kv8_fwd(p.q.cuda(), *cache, gpu(p.offs), positions=None if positions is None else gpu(positions),
                              causal=causal, scale=scale, return_lse=True, out=out, **kw)


def check_attention(p, got, kc, ks, vc, vs, positions=None, causal=True, scale=None):
    out, lse = to_f64(got[0]), got[1].cpu().numpy().astype(np.float64)
    scale = 1 / np.sqrt(p.D) if scale is None else scale
    k, v = R.read_all(kc, ks, p.fmt), R.read_all(vc, vs, p.fmt)
    ref, rl, mag, big = R.attention(p.q.double().numpy(), k, v, p.table, p.lens, p.offs, positions, causal, scale)
    none = np.isneginf(rl)
    assert np.array_equal(np.isnan(out), np.isnan(ref))
    assert np.array_equal(np.isneginf(lse), none)
    ok = np.isfinite(ref)
    u, c32 = U[p.dtype], 2.0 ** -24 * (16 * big[..., None] + 128)
    tol = u * np.abs(ref) + c32 * mag + 2.0 ** -126 * int(p.lens.max()) * float(np.nanmax(np.abs(v)))
    if p.dtype != "f32":
        tol = tol + u * mag + 2.0 ** -24 * int(p.lens.max()) * float(np.nanmax(np.abs(v)))
    if p.dtype == "f16":
        tol = tol + 2.0 ** -24
    err = np.abs(out - ref)
    bad = err[ok] > tol[ok]
    assert not bad.any(), f"{bad.sum()} of {ok.sum()} off, worst {np.max(err[ok] / tol[ok]):.2f} of the tolerance"
    fin = np.isfinite(rl)
    e = np.abs(lse[fin] - rl[fin])
    assert (e <= 2.0 ** -24 * (16 * big[fin] + 128 + 4 * np.abs(rl[fin]))).all(), e.max()


ATTENDS = [
    dict(lens=[1], new=[1], Hq=4, dtype="bf16"),
    dict(lens=[17, 200, 33], new=[1, 1, 1], Hq=8, dtype="bf16", fmt="e4m3", D=128),
    dict(lens=[17, 200, 33], new=[1, 1, 1], Hq=8, dtype="f16", G=1, D=128),
    dict(lens=[300, 1, 129], new=[2, 1, 4], Hq=14, dtype="f16", fmt="e4m3", P=32, G=32),           # 7 heads each
    dict(lens=[300, 5, 129], new=[4, 4, 4], Hq=16, dtype="bf16", P=64, G=16, D=128),               # drafts
    dict(lens=[700], new=[1], H=1, Hq=24, dtype="f16", P=128, G=64, D=128),                        # one kv head
    dict(lens=[700, 650], new=[3, 2], H=1, Hq=40, dtype="bf16", P=16, G=2, D=64, fmt="e4m3"),      # many rows
    dict(lens=[260, 90, 400], new=[150, 90, 33], Hq=8, dtype="bf16", P=64, G=16, D=128),           # prefill
    dict(lens=[260, 90, 400], new=[150, 90, 33], Hq=8, dtype="f16", P=32, G=1, D=64, fmt="e4m3"),
    dict(lens=[260, 90], new=[70, 90], Hq=6, dtype="f16", P=256, G=256, D=128),                    # 3 heads each
    dict(lens=[60, 70], new=[40, 5], Hq=4, dtype="bf16", P=24, G=8, D=64),                         # pages of 24
    dict(lens=[60, 70], new=[1, 1], Hq=4, dtype="bf16", P=5, G=5, D=128),
    dict(lens=[60, 0, 70], new=[20, 3, 1], Hq=4, dtype="f32", D=32, fmt="e4m3"),
    dict(lens=[60, 0, 70], new=[1, 1, 1], Hq=4, dtype="f32", D=128),
    dict(lens=[60, 0, 70], new=[20, 3, 1], Hq=4, dtype="bf16", D=16, fmt="e4m3"),
    dict(lens=[130, 0, 70], new=[2, 3, 0], Hq=4, dtype="f16", D=64),                               # no keys; no queries
    dict(lens=[130, 0, 70], new=[64, 30, 0], Hq=4, dtype="bf16", D=64),
    dict(lens=[4, 300], new=[9, 1], Hq=4, dtype="bf16", D=128),                                    # queries before token 0
    dict(lens=[2500, 9000, 40, 0, 6001], new=[1, 1, 1, 1, 1], Hq=8, dtype="bf16", P=64, G=8, D=128, fmt="e4m3"),
    dict(lens=[9000, 4100], new=[3, 3], Hq=6, dtype="f16", P=16, G=16, D=64),
    dict(lens=[2100, 130, 1500], new=[70, 0, 90], Hq=8, dtype="bf16", P=64, G=16, D=128),          # runs of key tiles
    dict(lens=[3000], new=[130], H=1, Hq=3, dtype="f16", P=40, G=4, D=64, fmt="e4m3"),
    dict(lens=[1300, 0, 2000], new=[40, 20, 2], H=1, Hq=2, dtype="bf16", P=16, G=1, D=128, fmt="e4m3"),
]


@pytest.mark.parametrize("kw", ATTENDS, ids=lambda kw: "-".join(str(v) for k, v in kw.items()))
@pytest.mark.parametrize("mask", ["causal", "full", "positions"])
def test_attention(kw, mask):
    kw = dict(kw)
    p = Problem(11, kw.pop("lens"), kw.pop("new"), **kw)
    pos = None
    if mask == "positions":  # any order, some before the first key, some past the last
        r = np.random.RandomState(2)
        pos = np.concatenate([r.randint(-3, L + 5, n) for L, n in zip(p.lens, p.new)]).astype(np.int32)
    cache = p.cache()
    got = attend(p, cache, pos, mask != "full")
    check_attention(p, got, p.kc, p.ks, p.vc, p.vs, pos, mask != "full")
    again = attend(p, cache, pos, mask != "full")
    assert all(a.cpu().float().numpy().tobytes() == b.cpu().float().numpy().tobytes()
               for a, b in zip(got, again)), "two calls differ"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_peaks_and_uneven_scales(dtype, new):
    # one key takes nearly everything; value scales a thousand times apart; zero groups; a flat row
    p = Problem(12, [400, 333], [new, new], dtype=dtype, Hq=8, D=128, G=8, H=2)
    r = np.random.RandomState(1)
    p.q = (p.q.float() * 6).to(p.q.dtype)
    p.q[0] = 0
    p.vs *= 10.0 ** r.uniform(-2, 1, p.vs.shape).astype(np.float32)
    p.vs[p.table[0, 3]] = 2.0 ** -100
    p.vc[p.table[0, 3]] = 0
    p.ks[p.table[0, 1], :, 0] *= 40
    check_attention(p, attend(p, p.cache(), scale=0.3), p.kc, p.ks, p.vc, p.vs, scale=0.3)


@pytest.mark.parametrize("dtype,fmt,D", [("bf16", "int8", 128), ("f16", "e4m3", 64), ("f32", "int8", 64)])
@pytest.mark.parametrize("new", [1, 5, 90])
def test_attention_ignores_what_it_does_not_see(dtype, fmt, D, new):
    # behind the last token: any byte, and NaN scales of the groups there; pages of no sequence: NaN
    kw = dict(dtype=dtype, fmt=fmt, D=D, Hq=8, P=32, G=4)
    p = Problem(13, [99, 150], [new, new], **kw)
    clean = [p.kc.copy(), p.ks.copy(), p.vc.copy(), p.vs.copy()]
    for c in (p.kc, p.vc):
        for s, L in enumerate(p.lens):
            c[p.table[s, L // 32], L % 32:] = 0xff
    for c in (p.ks, p.vs):
        for s, L in enumerate(p.lens):
            c[p.table[s, L // 32], :, -(-(L % 32) // 4):] = np.nan
    free = np.setdiff1d(np.arange(p.pages), p.table[p.table >= 0])
    p.ks[free], p.vs[free] = np.nan, np.nan
    check_attention(p, attend(p, p.cache()), *clean)
    # a visible NaN group: the rows that see it are NaN, the others are not
    q = Problem(13, [99, 150], [new, new], **kw)
    q.vs[q.table[0, 0], 0, 0] = np.nan
    out = to_f64(attend(q, q.cache())[0])
    assert np.isnan(out[:new, :4]).all() and np.isfinite(out[:new, 4:]).all() and np.isfinite(out[new:]).all()
    # a NaN group that only later positions see, through the causal mask
    m = Problem(13, [99, 150], [new, new], **kw)
    m.ks[m.table[1, 4], 1, 5] = np.nan  # tokens 148, 149 of sequence 1
    out = to_f64(attend(m, m.cache())[0])
    seen = [i for i in range(new) if 150 - new + i >= 148]
    assert np.isnan(out[new:, 4:][seen]).all()
    rest = np.setdiff1d(np.arange(new), seen)
    assert np.isfinite(out[new:][rest]).all() and np.isfinite(out[new:, :4]).all() and np.isfinite(out[:new]).all()


@pytest.mark.parametrize("new", [1, 70])
def test_attention_pages_outside_the_cache_are_zeros(new):
    p = Problem(14, [100, 130], [new, new], dtype="bf16", Hq=8, D=128, P=32, G=16)
    p.table[0, 1], p.table[1, 0] = -1, p.pages
    check_attention(p, attend(p, p.cache()), p.kc, p.ks, p.vc, p.vs)


@pytest.mark.parametrize("new", [1, 70])
def test_rows_of_no_sequence_and_a_wide_table(new):
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    p = Problem(15, [100, 130], [new, new], dtype="f16", Hq=8, D=64)
    want = attend(p, p.cache())
    wide = np.full((2, 40), 12345, np.int32)  # entries past a sequence's end are never followed
    wide[:, :p.table.shape[1]] = p.table
    cache = p.cache()
    cache[4] = gpu(wide)
    pad = torch.zeros((8, 8, 64), dtype=p.q.dtype)
    q = torch.cat([pad[:3], p.q, pad[3:]]).cuda()
    out = torch.full_like(q, 777.0)
    lse = torch.full((q.shape[0], 8), 777.0, device="cuda")
    attn.paged_kv8_fwd(q, *cache, gpu(p.offs + 3), return_lse=True, out=out, lse_out=lse, max_queries=new)
    for got, ref in ((out, want[0]), (lse, want[1])):
        assert (got[:3] == 777).all() and (got[-5:] == 777).all()
        assert torch.equal(got[3:-5], ref)


def test_long_cache_past_32_bits():
    # codes more than 2^32 bytes into the cache
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    pages, P, H, D, G = (1 << 32) // (64 * 8 * 128) + 20, 64, 8, 128, 16
    kc, vc = (torch.zeros((pages, P, H, D), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, H, P // G), 0.01, device="cuda") for _ in range(2))
    r = np.random.RandomState(3)
    table = np.array([[pages - 1, 5, pages - 3], [pages - 7, pages - 2, 1]], np.int32)
    kw = dict(D=D, P=P, G=G, H=H, Hq=16)
    p = Problem(16, [150, 170], [150, 170], **kw)
    p.table, p.pages = table, pages
    cache = [kc, vc, ks, vs, gpu(table), gpu(p.lens)]
    write(p, cache)
    rows = [attn.kv8_read(*cache, gpu(p.offs), dtype=torch.float32)]
    small = Problem(16, [150, 170], [150, 170], **kw)
    sc = small.cache()
    write(small, sc)
    rows.append(attn.kv8_read(*sc, gpu(p.offs), dtype=torch.float32))
    assert all(torch.equal(a, b) for a, b in zip(*rows))
    for n in (1, 40):
        offs = gpu(np.array([0, n, 2 * n], np.int32))
        q = torch.from_numpy(r.randn(2 * n, 16, D)).to(torch.bfloat16).cuda()
        assert torch.equal(attn.paged_kv8_fwd(q, *cache, offs, max_queries=n),
                           attn.paged_kv8_fwd(q, *sc, offs, max_queries=n))


@pytest.mark.parametrize("fmt,dtype,layout", [("int8", "bf16", "half"), ("e4m3", "f16", "interleaved")])
def test_serving_steps_together(fmt, dtype, layout):
    # prompts, then steps of turned, written and attended tokens; each stage against 64 bits
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    H, Hq, D, P, G, S = 2, 8, 128, 32, 16, 3
    r = np.random.RandomState(4)
    base = Problem(17, [120, 97, 64], [1, 1, 1], dtype=dtype, fmt=fmt, D=D, P=P, G=G, H=H, Hq=Hq)
    cache = base.cache()
    kc, ks, vc, vs = base.kc.copy(), base.ks.copy(), base.vc.copy(), base.vs.copy()
    freq, m = attn.rope_frequencies(D, scaling="by_parts", factor=4.0)
    lens = np.zeros(S, np.int32)
    for new in ([50, 33, 1], [1, 1, 1], [4, 2, 3], [1, 1, 1]):
        lens = lens + np.array(new, np.int32)
        offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(offs[-1])
        pos = np.concatenate([np.arange(L - n, L) for L, n in zip(lens, new)]).astype(np.int32)
        qkv = torch.from_numpy(r.randn(T, Hq + 2 * H, D)).to(tdt(dtype)).cuda()
        q, k = attn.rope(qkv[:, :Hq], qkv[:, Hq:Hq + H], gpu(pos), freq.cuda(), layout=layout, mscale=m)
        for x, y in ((qkv[:, :Hq], q), (qkv[:, Hq:Hq + H], k)):
            ref = R.rope(to_f64(x), pos, freq.numpy(), layout, m)
            assert np.abs(to_f64(y) - ref).max() <= (U[dtype] + 2.0 ** -20) * np.abs(ref).max()
        cache[5] = gpu(lens)
        attn.kv8_write(k, qkv[:, Hq + H:], *cache, gpu(offs))
        R.write_one(to_f64(k), kc, ks, base.table, lens, offs, fmt, G)
        R.write_one(to_f64(qkv[:, Hq + H:]), vc, vs, base.table, lens, offs, fmt, G)
        base.lens, base.offs, base.q = lens, offs, q.cpu()
        same_cache(base, cache, (kc, ks, vc, vs))
        got = attn.paged_kv8_fwd(q, *cache, gpu(offs), return_lse=True)
        check_attention(base, got, kc, ks, vc, vs)


@pytest.mark.parametrize("new", [1, 60])
def test_graph_and_streams(new):
    # captured and replayed on new inputs; two side streams at once
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    kw = dict(dtype="bf16", D=128, Hq=8, P=64, G=16)
    p, x = (Problem(seed, [300, 200], [new, new], **kw) for seed in (18, 19))
    cache, offs = p.cache(), gpu(p.offs)
    q, k, v = p.q.cuda(), p.k.cuda(), p.v.cuda()

    def step(cache, q, k, v, stream=None):
        attn.kv8_write(k, v, *cache, offs, stream=stream)
        out = attn.paged_kv8_fwd(q, *cache, offs, max_queries=new, return_lse=True, stream=stream)
        rows = attn.kv8_read(*cache, offs, 2 * new, dtype=torch.float32, stream=stream)
        return (*out, *rows)

    want = []
    for a in (p, x):
        c = p.cache()
        want.append([t.clone() for t in step(c, a.q.cuda(), a.k.cuda(), a.v.cuda())])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step(cache, q, k, v)
    for a, w in zip((p, x, p), (want[0], want[1], want[0])):
        for dst, src in zip(cache, p.cache()):
            dst.copy_(src)
        for dst, src in ((q, a.q), (k, a.k), (v, a.v)):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, t) for o, t in zip(outs, w))
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    caches = [p.cache(), p.cache()]
    args = [[t.cuda() for t in (a.q, a.k, a.v)] for a in (p, x)]
    torch.cuda.synchronize()
    got = [step(caches[i], *args[i], stream=sides[i]) for i in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, t) for i in range(2) for o, t in zip(got[i], want[i]))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new", [1, 33])
def test_attention_over_small_and_large_codes(dtype, new):
    import torch
    # e4m3 codes below the format's normal range in one sequence, the largest in the other; queries
    # whose rows differ by many powers of two
    p = Problem(20, [200, 150], [new, new], dtype=dtype, fmt="e4m3", D=128, Hq=8, P=32, G=4)
    r = np.random.RandomState(5)
    for c in (p.kc, p.vc):
        for s, codes in ((0, [0, 1, 2, 3, 7, 0x81, 0x87, 8]), (1, [0x7e, 0xfe, 0x78, 0xf0, 0x80])):
            for b in p.table[s][p.table[s] >= 0]:
                c[b] = r.choice(codes, c[b].shape)
    p.ks[p.table[0, :7]] *= 2.0 ** 9
    p.q = (p.q.double() * torch.from_numpy(0.2 * 2.0 ** r.randint(-12, 3, (p.tokens, 8, 1)))).to(p.q.dtype)
    check_attention(p, attend(p, p.cache()), p.kc, p.ks, p.vc, p.vs)


@pytest.mark.parametrize("heads,new", [(3, 3), (5, 2), (7, 5), (8, 7), (16, 4), (1, 20), (1, 60)])
@pytest.mark.parametrize("H", [1, 3, 20])
def test_attention_row_counts(heads, new, H):
    # 9 .. 64 rows of a kv head, one and two groups of rows; heads that divide nothing; uneven lengths
    p = Problem(21, [300, 64, 1000], [new, 1, new - 1], dtype="f16", fmt="int8", D=64, P=16, G=4, H=H, Hq=H * heads)
    check_attention(p, attend(p, p.cache()), p.kc, p.ks, p.vc, p.vs)


@pytest.mark.parametrize("new", [2, 90])
@pytest.mark.parametrize("dtype,G", [("bf16", 1), ("f16", 16), ("f32", 4)])
def test_positions_at_the_ends_of_int32(new, dtype, G):
    # the lowest positions see no key of any tile, the highest see all
    p = Problem(25, [400], [new], Hq=4, P=32, D=64, G=G, dtype=dtype)
    pos = np.full(new, 350, np.int32)
    pos[0], pos[1], pos[new // 2], pos[-1] = -2 ** 31 + 5, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1
    got = attend(p, p.cache(), pos)
    check_attention(p, got, p.kc, p.ks, p.vc, p.vs, pos)


def test_calls_that_share_a_workspace_in_turn():
    # captured calls of one workspace, replayed back to back: sequences that are cut, one key block
    # each (nothing to cut), few rows over runs of key tiles, and rows of no sequence
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    kw = dict(Hq=8, P=64, G=16, D=128)
    ps = [Problem(26, [3000, 700], [1, 1], **kw), Problem(27, [60, 90, 2], [1, 1, 1], **kw),
          Problem(28, [2500], [80], **kw), Problem(29, [2500, 40], [3, 1], **kw)]
    for p in ps:  # a table with room for more than 512 keys each
        p.table = np.pad(p.table, ((0, 0), (0, max(0, 10 - p.table.shape[1]))), constant_values=-1)
    sets = [(p, p.cache(), p.q.cuda(), gpu(p.offs), torch.empty(p.q.shape, dtype=p.q.dtype, device="cuda"),
             int(p.new.max())) for p in ps]
    p, cache, q, offs, _, new = sets[0]
    sets.append((p, cache, q, torch.zeros_like(offs), torch.empty_like(q), new))
    work = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    want = [attn.paged_kv8_fwd(q, *cache, offs, max_queries=new) for _, cache, q, offs, _, new in sets[:4]]
    for (p, cache, q, offs, _, new), w in zip(sets, want):
        out, lse = attn.paged_kv8_fwd(q, *cache, offs, max_queries=new, return_lse=True)
        check_attention(p, (out, lse), p.kc, p.ks, p.vc, p.vs)
        assert torch.equal(out, w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in (0, 1, 2, 4, 3, 0, 4, 1):
            _, cache, q, offs, out, new = sets[i]
            attn.paged_kv8_fwd(q, *cache, offs, max_queries=new, out=out, workspace=work)
    for _ in range(20):
        for s in sets[:4]:
            s[4].zero_()
        g.replay()
        assert all(torch.equal(s[4], w) for s, w in zip(sets, want))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("seqs,new,Hq,H", [(1, 4, 20, 4), (2, 2, 60, 4), (20, 5, 21, 3), (30, 9, 24, 3), (45, 2, 52, 2), (9, 3, 20, 1)])
def test_attention_by_every_way_of_cutting(seqs, new, Hq, H, wide):
    # few and many rows over few, half and enough sequences to fill the GPU, whole and cut into runs
    r = np.random.RandomState(30)
    lens = r.randint(new, 1300, seqs)
    lens[0] = 1300
    p = Problem(30, lens, np.full(seqs, new), Hq=Hq, H=H, P=64, G=16, D=64, dtype="f16", fmt="e4m3")
    if wide:  # room for 8192 keys
        p.table = np.pad(p.table, ((0, 0), (0, 128 - p.table.shape[1])), constant_values=-1)
    cache = p.cache()
    got = attend(p, cache)
    check_attention(p, got, p.kc, p.ks, p.vc, p.vs)
    again = attend(p, cache)
    assert all(a.cpu().float().numpy().tobytes() == b.cpu().float().numpy().tobytes() for a, b in zip(got, again))
