"""Rotary positions on the GPU (attn_rope) against 64 bits (kv8_ref.rope).

Tolerance of an element y = m (x1 cos a -+ x2 sin a): half a step of the type times |y|, and
2^-21 m (|x1| + |x2|) for fp32: the angle in half turns is one fp32 number in [-1, 1) (off by
2^-25, so a by pi 2^-25), sincospi by 2 units, three roundings of products and the sum; and the
fraction of a turn, position * 2^-52 of the product's rounding in double on either side."""
import numpy as np
import pytest

from tests import kv8_ref as R
from tests.gpu_util import to_f64

pytestmark = pytest.mark.gpu
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def tdt(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def near(got, x, pos, freq, layout, m, inverse, dtype):
    ref = R.rope(x, pos, freq, layout, m, inverse)
    mag = R.rope(np.abs(x), np.zeros_like(pos), freq, layout, m)  # m |x1|, m |x2|
    n = len(freq)
    i, j = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    both = mag.copy()
    both[..., i] = both[..., j] = mag[..., i] + mag[..., j]
    turn = 2.0 ** -21 + 2 * np.pi * np.abs(pos.astype(np.float64))[:, None, None] * 2.0 ** -52
    tol = U[dtype] * np.abs(ref) + turn * both + (2.0 ** -25 if dtype == "f16" else 0)
    tol[..., 2 * n:] = 0  # copied
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"worst {np.max(err - tol):.3e} over"


CASES = [
    dict(T=1, Hq=1, Hk=0, D=2, rot=2, dtype="f32"),
    dict(T=5, Hq=3, Hk=1, D=64, rot=64, dtype="bf16"),
    dict(T=64, Hq=32, Hk=8, D=128, rot=128, dtype="bf16"),
    dict(T=33, Hq=7, Hk=1, D=128, rot=64, dtype="f16"),
    dict(T=33, Hq=4, Hk=2, D=80, rot=20, dtype="bf16"),      # rows of 16 bytes, pairs that are not
    dict(T=17, Hq=2, Hk=2, D=18, rot=6, dtype="f16"),        # nothing on a boundary
    dict(T=9, Hq=2, Hk=1, D=512, rot=512, dtype="f32"),
    dict(T=9, Hq=2, Hk=1, D=512, rot=2, dtype="bf16"),
    dict(T=3001, Hq=4, Hk=1, D=96, rot=96, dtype="f16"),     # 4 tokens of a CTA, ragged
    dict(T=2600, Hq=2, Hk=2, D=64, rot=48, dtype="f32"),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("back", [False, True])
def test_rope(c, layout, back):
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    r = np.random.RandomState(c["T"])
    dt = tdt(c["dtype"])
    q = torch.from_numpy(r.randn(c["T"], c["Hq"], c["D"])).to(dt).cuda()
    k = torch.from_numpy(r.randn(c["T"], c["Hk"], c["D"])).to(dt).cuda() if c["Hk"] else None
    pos = r.randint(0, 1 << 20, c["T"]).astype(np.int32)
    pos[0] = 0
    freq, m = attn.rope_frequencies(c["rot"], scaling="by_parts", factor=3.0)
    f = attn.rope_bwd if back else attn.rope
    oq, ok = f(q, k, torch.from_numpy(pos).cuda(), freq.cuda(), layout=layout, mscale=m)
    near(to_f64(oq), to_f64(q), pos, freq.numpy(), layout, m, back, c["dtype"])
    if k is not None:
        near(to_f64(ok), to_f64(k), pos, freq.numpy(), layout, m, back, c["dtype"])
    else:
        assert ok is None


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_and_negative_positions(layout):
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    pos = np.array([0, 1, -1, -77777, (1 << 31) - 1, -(1 << 31), 123456789, 1 << 24], np.int32)
    x = np.random.RandomState(0).randn(8, 2, 64).astype(np.float32)
    # frequencies with few bits: position * frequency is exact in double, and so is the reference's angle
    freq = np.round(R.np.geomspace(1.0, 1e-4, 32) * 2 ** 20) / 2 ** 20
    got, _ = attn.rope(torch.from_numpy(x).cuda(), None, torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda(),
                       layout=layout)
    near(to_f64(got), x.astype(np.float64), pos, freq, layout, 1.0, False, "f32")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_dense_strided_and_in_place(layout):
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    B, Hq, Hk, S, D = 2, 4, 2, 37, 64
    r = np.random.RandomState(1)
    f = attn.rope_frequencies(32)[0].cuda()
    q = torch.from_numpy(r.randn(B, Hq, S, D)).to(torch.bfloat16).cuda()
    k = torch.from_numpy(r.randn(B, Hk, S, D)).to(torch.bfloat16).cuda()
    pos = torch.from_numpy(r.randint(0, 5000, (B, S)).astype(np.int32)).cuda()
    packed = lambda x: x.transpose(1, 2).reshape(B * S, -1, D)  # noqa: E731
    want = attn.rope(packed(q).contiguous(), packed(k).contiguous(), pos.view(-1), f, layout=layout)
    got = attn.rope(q, k, pos, f, layout=layout)               # dense, as the dense forward takes it
    for a, b in zip(got, want):
        assert torch.equal(packed(a), b)
    one = attn.rope(q, k, pos[0], f, layout=layout)            # one row of positions for every batch
    assert torch.equal(one[0][0], got[0][0]) and not torch.equal(one[0][1], got[0][1])
    fused = torch.cat([packed(q), packed(k), packed(k)], 1).contiguous()  # q, k, v of one projection
    for shift in (0, 1):
        buf = torch.zeros((B * S, Hq + 2 * Hk, D + shift), dtype=torch.bfloat16, device="cuda")
        buf[..., shift:] = fused
        qs, ks = buf[:, :Hq, shift:], buf[:, Hq:Hq + Hk, shift:]
        a = attn.rope(qs, ks, pos.view(-1), f, layout=layout)
        assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
        b = attn.rope(qs, ks, pos.view(-1), f, layout=layout, q_out=qs, k_out=ks)  # in place
        assert b[0] is qs and torch.equal(qs, want[0]) and torch.equal(ks, want[1])
        assert torch.equal(buf[:, Hq + Hk:, shift:], packed(k))                    # v untouched
        if shift:
            assert (buf[..., 0] == 0).all()
    with pytest.raises(attn.AttnError):
        attn.rope(buf[:, :Hq, 1:], buf[:, Hq:Hq + Hk, 1:], pos.view(-1), f, q_out=buf[:, 1:Hq + 1, 1:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient(layout):
    # rope_bwd(g) against central differences of <rope(x), g>, and as the transposed map:
    # <rope(x), g> = <x, rope_bwd(g)>
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    r = np.random.RandomState(2)
    freq, m = attn.rope_frequencies(24, scaling="by_parts", factor=8.0)
    f, pos = freq.cuda(), torch.from_numpy(r.randint(0, 9999, 11).astype(np.int32)).cuda()
    x, g = (torch.from_numpy(r.randn(11, 2, 32)).float().cuda() for _ in range(2))
    dx, _ = attn.rope_bwd(g, None, pos, f, layout=layout, mscale=m)
    run = lambda t: (attn.rope(t, None, pos, f, layout=layout, mscale=m)[0].double() * g.double()).sum().item()  # noqa: E731
    lhs, rhs = run(x), (x.double() * dx.double()).sum().item()
    size = (x.double().abs() * g.double().abs()).sum().item() * 2 * m
    assert abs(lhs - rhs) <= 2.0 ** -20 * size
    # the map is linear, so a wide step costs no truncation error
    for t, h, d in ((0, 0, 0), (3, 1, 11), (7, 0, 23), (10, 1, 24), (10, 1, 31), (5, 1, 12)):
        e = torch.zeros_like(x)
        e[t, h, d] = 1.0
        diff = (run(x + e) - run(x - e)) / 2
        assert abs(diff - dx[t, h, d].item()) <= 2.0 ** -20 * size


def test_graph_and_side_stream():
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    r = np.random.RandomState(3)
    f = attn.rope_frequencies(64)[0].cuda()
    q, k = (torch.from_numpy(r.randn(50, h, 64)).half().cuda() for h in (4, 2))
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    want = attn.rope(q, k, pos, f)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        outs = attn.rope(q, k, pos, f)
        back = attn.rope_bwd(*outs, pos, f)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    # two roundings of values of at most 8
    assert all((a.float() - b.float()).abs().max() <= 2.0 ** -9 * 8 for a, b in zip(back, (q, k)))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = attn.rope(q, k, pos, f, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("S", [1, 21])
def test_heads_of_one_dense_tensor_in_place(S):
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    r = np.random.RandomState(6)
    buf = torch.from_numpy(r.randn(3, 4 + 2 + 2, S, 64)).to(torch.float16).cuda()
    q, k, v = buf[:, :4], buf[:, 4:6], buf[:, 6:]
    f, pos = attn.rope_frequencies(64)[0].cuda(), torch.from_numpy(r.randint(0, 999, (3, S)).astype(np.int32)).cuda()
    want = attn.rope(q.contiguous(), k.contiguous(), pos, f)
    rest = v.clone()
    attn.rope(q, k, pos, f, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, rest)
    for out in (buf[:, 1:5], buf[:, 3:7]):  # shares heads with q or k
        with pytest.raises(attn.AttnError):
            attn.rope(q, k, pos, f, q_out=out)
