"""The 8-bit paged cache on the GPU where bytes, scales and scores are not those that this library's
writer makes of ordinary values: e4m3 codes 0x7f and 0xff, keys that are not there, value scales far
apart, scales of another program. Against the restatement in 64 bits (kv8_ref.py).

``close`` counts only what a row sees. With u half a step of the type of q, A = sum_j p_j |v_j|,
b = max_j scale sum_d |q_d| |k_jd|, w = max_j p_j v_scale_j and c the largest code among the n keys
that the row sees:
  u |o|                    the output's rounding,
  2^-11 A                  p_j v_scale_j as F16 (F16 and BF16 only),
  2^-24 n w c              one below 2^-14 of w is subnormal in F16: off by up to 2^-24 of w,
  2^-24 (16 b + 128) A     fp32: scores, exp2 and sums,
  2^-126 n max|v|          the range of fp32: exp2 gives 0 below 2^-126,
  2^-24                    F16 outputs below its normal range."""
import numpy as np
import pytest

from tests import kv8_ref as R
from tests.gpu_util import to_f64
from tests.test_kv8_gpu import U, Problem, _clean_status, attend, gpu, same_cache, tdt, write  # noqa: F401

pytestmark = pytest.mark.gpu


def close(p, got, positions=None, causal=True, scale=None, rows=None):
    out, lse = to_f64(got[0]), got[1].cpu().numpy().astype(np.float64)
    scale = 1 / np.sqrt(p.D) if scale is None else scale
    k, v = R.read_all(p.kc, p.ks, p.fmt), R.read_all(p.vc, p.vs, p.fmt)
    code = np.abs(R.values(p.vc, p.fmt))
    u = U[p.dtype]
    q = p.q.double().numpy()
    for s, L in enumerate(p.lens):
        j = np.arange(L)
        page, row = p.table[s, j // p.P], j % p.P
        ok = (page >= 0) & (page < p.pages)
        at = np.where(ok, page, 0)
        kk, vv = (np.where(ok[:, None, None], x[at, row], 0.0) for x in (k, v))
        cc = np.where(ok[:, None], code[at, row].max(-1), 0.0)                      # [L, H]
        vs = np.where(ok[:, None], p.vs[at, :, row // p.G].astype(np.float64), 0.0)  # [L, H]
        for i in range(int(p.offs[s]), int(p.offs[s + 1])):
            if rows is not None and not rows[i]:
                continue
            pos = int(positions[i]) if positions is not None else L - int(p.offs[s + 1]) + i
            n = min(L, pos + 1) if causal else L
            for h in range(p.Hq):
                hk = h // (p.Hq // p.H)
                t = kk[:n, hk] @ q[i, h] * scale
                e = np.exp(t - t.max())
                pr = e / e.sum()
                o, A = pr @ vv[:n, hk], pr @ np.abs(vv[:n, hk])
                b = (np.abs(kk[:n, hk]) @ np.abs(q[i, h])).max() * scale
                tol = u * np.abs(o) + 2.0 ** -24 * (16 * b + 128) * A + 2.0 ** -126 * n * np.abs(vv[:n, hk]).max()
                if p.dtype != "f32":
                    tol = tol + 2.0 ** -11 * A + 2.0 ** -24 * n * (pr * vs[:n, hk]).max() * cc[:n, hk].max()
                if p.dtype == "f16":
                    tol = tol + 2.0 ** -24
                err = np.abs(out[i, h] - o)
                assert (err <= tol).all(), (f"sequence {s} row {i} head {h}: {np.max(err / np.maximum(tol, 1e-300)):.3g} "
                                            f"of the tolerance, {out[i, h, :3]} for {o[:3]}")
                ref = t.max() + np.log(e.sum())
                assert abs(lse[i, h] - ref) <= 2.0 ** -24 * (16 * b + 128 + 4 * abs(ref)), f"lse of row {i} head {h}"


NAN_BYTES = np.array([0x7f, 0xff], np.uint8)


def nobody_has_page_0(p):
    free = np.setdiff1d(np.arange(p.pages), p.table[p.table >= 0])
    if 0 not in free:
        p.table[p.table == 0] = free[0]


@pytest.mark.parametrize("dtype,fmt,D", [("bf16", "e4m3", 128), ("f16", "e4m3", 64), ("f16", "int8", 128), ("f32", "e4m3", 64)])
@pytest.mark.parametrize("new", [1, 5, 90])
def test_keys_that_are_not_there_read_nothing(dtype, fmt, D, new):
    # behind the last token of a tile, and on pages outside the cache: zeros, whatever the bytes that
    # the cache begins with (its page 0 belongs to no sequence and was never written)
    p = Problem(40, [99, 150, 333], [new] * 3, dtype=dtype, fmt=fmt, D=D, Hq=8, P=32, G=4)
    nobody_has_page_0(p)
    p.table[1, 1], p.table[2, 3] = -1, p.pages
    r = np.random.RandomState(41)
    for c in (p.kc, p.vc):
        c[0] = r.choice(NAN_BYTES, c[0].shape)
    p.ks[0], p.vs[0] = np.nan, np.nan
    got = attend(p, p.cache())
    assert np.isfinite(to_f64(got[0])).all()
    close(p, got)


@pytest.mark.parametrize("dtype,D,G", [("bf16", 128, 16), ("f16", 64, 1), ("f16", 128, 4), ("f32", 64, 8)])
@pytest.mark.parametrize("new", [1, 5, 90])
def test_codes_7f_and_ff_are_480(dtype, D, G, new):
    # the two e4m3 codes that the writer never makes: +-480 to every reader, and nothing to a row
    # whose mask hides them
    from exact_scaled_dot_flash_gb300 import attn
    p = Problem(42, [99, 150, 333], [new] * 3, dtype=dtype, fmt="e4m3", D=D, Hq=8, P=32, G=G)
    r = np.random.RandomState(43)
    for c in (p.kc, p.vc):
        c[...] = np.where(r.rand(*c.shape) < 0.02, r.choice(NAN_BYTES, c.shape), c)
        c[p.table[1, 4], 20:22, :, 3] = 0xff  # tokens 148, 149 of sequence 1: only its last rows see them
    cache = p.cache()
    offs = gpu(np.concatenate([[0], np.cumsum(p.lens)]).astype(np.int32))
    rows = attn.kv8_read(*cache, offs, dtype=tdt(dtype))
    for got, c, s in zip(rows, (p.kc, p.vc), (p.ks, p.vs)):
        ref = R.read_rows(c, s, p.table, p.lens, offs.cpu().numpy(), int(p.lens.sum()), "e4m3")
        assert (np.abs(to_f64(got) - ref) <= (U[dtype] + 2.0 ** -24) * np.abs(ref) + 2.0 ** -25).all()
    got = attend(p, cache)
    assert np.isfinite(to_f64(got[0])).all()
    close(p, got)
    # only in places that no row but the last one sees
    q = Problem(44, [99, 150, 333], [new] * 3, dtype=dtype, fmt="e4m3", D=D, Hq=8, P=32, G=G)
    q.vc[q.table[1, 4], 21] = 0xff
    q.kc[q.table[2, 10], 12] = 0x7f
    close(q, attend(q, q.cache()))


@pytest.mark.parametrize("new", [1, 90])
def test_nan_scales_beside_codes_7f_and_ff(new):
    # NaN groups stay NaN, the rest stays finite
    p = Problem(45, [99, 150], [new, new], dtype="bf16", fmt="e4m3", D=128, Hq=8, P=32, G=4)
    r = np.random.RandomState(46)
    p.vc[...] = np.where(r.rand(*p.vc.shape) < 0.02, r.choice(NAN_BYTES, p.vc.shape), p.vc)
    p.vs[p.table[0, 0], 0, 0] = np.nan
    out = to_f64(attend(p, p.cache())[0])
    assert np.isnan(out[:new, :4]).all() and np.isfinite(out[:new, 4:]).all() and np.isfinite(out[new:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_groups_that_grow_over_codes_7f_and_ff(dtype):
    # tokens of an earlier call that hold the two codes are brought to a larger scale from +-480
    p = Problem(47, [40, 21, 70], [3, 2, 5], dtype=dtype, fmt="e4m3", G=16, loud=400.0)
    r = np.random.RandomState(48)
    for c in (p.kc, p.vc):
        c[...] = np.where(r.rand(*c.shape) < 0.2, r.choice(NAN_BYTES, c.shape), c)
    cache, want = p.cache(), p.written()
    write(p, cache)
    same_cache(p, cache, want)


def loud_key(p, s, j, code=16):
    """Key j of sequence s scores far above the others: its codes point along the (positive) queries."""
    p.kc[p.table[s, j // p.P], j % p.P] = code if p.fmt == "int8" else 0x58  # 16


@pytest.mark.parametrize("dtype,fmt,D,G", [("f16", "int8", 128, 1), ("bf16", "e4m3", 64, 4), ("f16", "e4m3", 128, 16),
                                           ("bf16", "int8", 128, 16), ("f32", "int8", 64, 4)])
@pytest.mark.parametrize("new", [1, 40, 90])
@pytest.mark.parametrize("down", [5, 8, 14, 24, 60, None])
def test_the_top_key_has_a_small_value_scale(dtype, fmt, D, G, new, down):
    # the key that takes nearly all of a row's probability holds values 2^-down of the others' (None:
    # zeros), so that the others' small probabilities count
    import torch
    p = Problem(50, [1500, 400], [new, new], dtype=dtype, fmt=fmt, D=D, G=G, P=32, Hq=4, H=1)
    p.q = p.q.abs()
    p.ks[...] = 0.01 if fmt == "int8" else 2.0 ** -8
    p.vs[...] = 2.0 ** -6
    for s, page in ((0, p.table[0, 0]), (1, p.table[1, 0])):
        p.kc[page, :G] = 0
        loud_key(p, s, 0)
        # the others' scores lie within some 2 of 0; the top one lies at 12 + log2(1500)
        t = 16 * p.q[p.offs[s]:p.offs[s + 1]].double().sum(-1).mean().item() / np.sqrt(D)
        p.ks[page, :, 0] = 19 * np.log(2.0) / t
        p.vs[page, :, 0] = 2.0 ** (-6 - down) if down else 0.0
    close(p, attend(p, p.cache()))


@pytest.mark.parametrize("dtype,fmt,D,G", [("f16", "int8", 128, 1), ("bf16", "e4m3", 64, 4), ("bf16", "e4m3", 128, 16),
                                           ("f32", "int8", 64, 4)])
@pytest.mark.parametrize("new", [2, 90, 200])
@pytest.mark.parametrize("up", [14, 25, 40, 100])
@pytest.mark.parametrize("mask", ["causal", "positions"])
def test_hidden_keys_of_large_value_scales(dtype, fmt, D, G, new, up, mask):
    # the values of the last group are 2^up of the others'; only the rows behind its first token see it
    p = Problem(51, [320, 416], [new, new], dtype=dtype, fmt=fmt, D=D, G=G, P=32, Hq=4, H=1)
    p.vs[...] = 2.0 ** -14
    for s, L in enumerate(p.lens):
        p.vs[p.table[s, (L - 1) // p.P], :, -1] = 2.0 ** (up - 14)
    seen = np.concatenate([np.arange(L - n, L) for L, n in zip(p.lens, p.new)]).astype(np.int32)
    last = np.concatenate([np.full(n, L - G) for L, n in zip(p.lens, p.new)])
    if mask == "positions":
        seen = np.concatenate([np.random.RandomState(52).permutation(a) for a in np.split(seen, [new])]).astype(np.int32)
    got = attend(p, p.cache(), seen if mask == "positions" else None)
    # in F16 the rows that see it may pass the type's range: they are not compared
    rows = seen < last if dtype == "f16" and up > 14 else None
    close(p, got, seen, rows=rows)


@pytest.mark.parametrize("loud", [1.0, 300.0])
def test_appending_at_a_scale_that_is_no_power_of_two(loud):
    # e4m3 groups that another program began: their scale divides, and their codes move to a larger
    # one, to the nearest code, ties to even, however near a quotient is to the border of two codes
    import torch
    p = Problem(53, [40, 21, 70, 13], [3, 2, 5, 1], dtype="f32", fmt="e4m3", G=16, H=3, loud=loud)
    r = np.random.RandomState(54)
    for s in (p.ks, p.vs):
        s *= r.uniform(1.0, 2.0, s.shape).astype(np.float32)
    border = (R.E4M3[:126] + R.E4M3[1:127]) / 2
    for x, sc in ((p.k, p.ks), (p.v, p.vs)):
        for s, (L, n) in enumerate(zip(p.lens, p.new)):
            for t in range(n):
                j = L - n + t
                S = sc[p.table[s, j // p.P], :, j % p.P // p.G].astype(np.float64)[:, None]  # [H, 1]
                y = (r.choice(border[20:110], (p.H, p.D)) * S * r.choice([-1, 1], (p.H, p.D))).astype(np.float32)
                y = np.nextafter(y, r.choice(np.array([-np.inf, 0, np.inf], np.float32), y.shape)) if t % 2 else y
                y[:, :4] = [0.0, -0.0, 1e-42, -3e-45]  # quotients that leave fp32's range
                x[p.offs[s] + t] = torch.from_numpy(y * np.float32(loud))
    cache, want = p.cache(), p.written()
    write(p, cache)
    same_cache(p, cache, want)
    write(p, cache)
    same_cache(p, cache, want, "second call: ")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("new", [1, 90])
def test_scores_far_below_zero(dtype, new):
    # every score is about -10^31, one of them half of the others: that key takes all
    import torch
    p = Problem(55, [200, 131], [new, new], dtype=dtype, fmt="int8", D=64, Hq=4, H=1, G=1)
    p.q = -torch.ones_like(p.q) * 512
    p.kc[...] = 64
    p.ks[...] = 2.0 ** 87
    best = [7, 3]
    for s, j in enumerate(best):
        p.ks[p.table[s, j // p.P], :, j % p.P] = 2.0 ** 86
    out, lse = attend(p, p.cache())
    v = R.read_all(p.vc, p.vs, "int8")
    for s, j in enumerate(best):
        ref = v[p.table[s, j // p.P], j % p.P]  # [1, D]
        assert (np.abs(to_f64(out[p.offs[s]:p.offs[s + 1]]) - ref) <= 2 * U[dtype] * np.abs(ref) + 2.0 ** -20).all()
        want = -512 * 64 * 64 * 2.0 ** 86 / 8
        assert (np.abs(lse[p.offs[s]:p.offs[s + 1]].cpu().numpy() / want - 1) <= 2.0 ** -20).all()


def test_a_nan_group_far_below_the_top_score():
    # 0 * NaN: a group without values makes its rows NaN however small its probability, also where the
    # key tiles are cut into runs and another run holds the scores that count
    import torch
    p = Problem(56, [3000], [80], dtype="bf16", fmt="int8", D=128, Hq=2, H=1, G=16, P=32)
    p.q = p.q.abs()
    p.kc[...] = 20
    p.ks[...] = 2.0 ** -20
    t = 20 * p.q.double().sum(-1).min().item() / np.sqrt(128) * 1.44
    for page in p.table[0, 80:]:
        p.ks[page] = 400 / t  # their scores lie 400 and more above, in powers of two
    clean = to_f64(attend(p, p.cache(), causal=False)[0])
    assert np.isfinite(clean).all()
    p.vs[p.table[0, 1], 0, 0] = np.nan
    assert np.isnan(to_f64(attend(p, p.cache(), causal=False)[0])).all()


@pytest.mark.parametrize("dtype,D,G", [("bf16", 128, 16), ("f16", 64, 1)])
@pytest.mark.parametrize("new,H,Hq", [(1, 2, 8), (3, 2, 10), (12, 1, 4), (70, 1, 2)])
def test_codes_7f_and_ff_in_cut_sequences(dtype, D, G, new, H, Hq):
    # the two codes and absent pages where the keys of a sequence are shared out over the GPU
    p = Problem(57, [2600, 40, 1313], [new] * 3, dtype=dtype, fmt="e4m3", D=D, Hq=Hq, H=H, P=32, G=G)
    nobody_has_page_0(p)
    r = np.random.RandomState(58)
    for c in (p.kc, p.vc):
        for s, page in ((0, 3), (0, 40), (0, 80), (2, 7)):  # a few pages of them, the others none
            at = p.table[s, page]
            c[at] = np.where(r.rand(*c[at].shape) < 0.3, r.choice(NAN_BYTES, c[at].shape), c[at])
        c[0] = 0xff
    p.table[0, 10], p.table[2, 20] = -1, p.pages + 3
    got = attend(p, p.cache())
    # of 70 rows of the sequence of 40 tokens the first 30 lie before its first token: no keys, NaN
    rows = np.concatenate([np.arange(L - n, L) >= 0 for L, n in zip(p.lens, p.new)])
    assert np.isfinite(to_f64(got[0])[rows]).all() and np.isnan(to_f64(got[0])[~rows]).all()
    close(p, got, rows=rows)
    again = attend(p, p.cache())
    assert all(a.cpu().float().numpy().tobytes() == b.cpu().float().numpy().tobytes() for a, b in zip(got, again))
