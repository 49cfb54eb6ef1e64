"""Rotary positions with several axes on the GPU (attn_rope_axes): each pair turns as attn_rope turns it
for the positions of its axis, so against 64 bits by the tolerance that test_rope_gpu.py derives,
pair by pair, and bit for bit where all axes have the same positions."""
import numpy as np
import pytest

from tests.gpu_util import to_f64
from tests.test_rope_gpu import U, tdt

pytestmark = pytest.mark.gpu


def reference(x, pos, axes, freq, layout, m, inverse):
    """y and m (|x1| + |x2|) of every element; pairs of other axes than those of pos: not turned."""
    y, both = x * 1.0, np.zeros_like(x)
    n = len(freq)
    for i in range(n):
        a, b = (i, n + i) if layout == "half" else (2 * i, 2 * i + 1)
        p = pos[axes[i]] if 0 <= axes[i] < len(pos) else np.zeros_like(pos[0])
        ang = (p.astype(np.longdouble) * np.longdouble(freq[i]))[..., None] * (-1 if inverse else 1)
        c, s = np.cos(ang).astype(np.float64), np.sin(ang).astype(np.float64)
        y[..., a] = m * (x[..., a] * c - x[..., b] * s)
        y[..., b] = m * (x[..., b] * c + x[..., a] * s)
        both[..., a] = both[..., b] = abs(m) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, both


def near(got, x, pos, axes, freq, layout, m, inverse, dtype):
    ref, both = reference(x, pos, axes, freq, layout, m, inverse)
    turn = 2.0 ** -21 + 2 * np.pi * float(np.abs(pos.astype(np.float64)).max()) * 2.0 ** -52
    tol = U[dtype] * np.abs(ref) + turn * both + (2.0 ** -25 if dtype == "f16" else 0)
    tol[..., 2 * len(freq):] = 0  # copied
    assert (np.abs(got - ref) <= tol).all()


CASES = [dict(T=1, Hq=1, Hk=0, D=2, rot=2, dtype="f32", A=1), dict(T=70, Hq=8, Hk=2, D=128, rot=128, dtype="bf16", A=3),
         dict(T=33, Hq=7, Hk=1, D=80, rot=20, dtype="f16", A=2), dict(T=17, Hq=2, Hk=2, D=18, rot=6, dtype="f32", A=4),
         dict(T=3001, Hq=4, Hk=1, D=96, rot=96, dtype="f16", A=3), dict(T=2600, Hq=2, Hk=2, D=64, rot=48, dtype="f32", A=2)]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("back", [False, True])
def test_axes(c, layout, back):
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    r = np.random.RandomState(c["T"])
    q = torch.from_numpy(r.randn(c["T"], c["Hq"], c["D"])).to(tdt(c["dtype"])).cuda()
    k = torch.from_numpy(r.randn(c["T"], c["Hk"], c["D"])).to(tdt(c["dtype"])).cuda() if c["Hk"] else None
    pos = r.randint(-1000, 1 << 20, (c["A"], c["T"])).astype(np.int32)
    axes = r.randint(0, c["A"], c["rot"] // 2).astype(np.int32)
    if len(axes) > 2:
        axes[1], axes[2] = -1, c["A"]  # of no axis
    freq = attn.rope_frequencies(c["rot"])[0]
    f = attn.rope_bwd if back else attn.rope
    m = 1.25
    got = f(q, k, torch.from_numpy(pos).cuda(), freq.cuda(), layout=layout, mscale=m, axes=torch.from_numpy(axes).cuda())
    for x, y in ((q, got[0]), (k, got[1])):
        if x is not None:
            near(to_f64(y), to_f64(x), pos, axes, freq.numpy(), layout, m, back, c["dtype"])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_equal_axes_turn_as_one(layout):
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    x = torch.randn((300, 12, 128), generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    pos = torch.arange(300, dtype=torch.int32, device="cuda") * 37
    f = attn.rope_frequencies(128)[0].cuda()
    axes = attn.rope_axes([16, 24, 24], cycle=True).cuda()
    a = attn.rope(x[:, :8], x[:, 8:], pos, f, layout=layout)
    b = attn.rope(x[:, :8], x[:, 8:], pos.expand(3, -1).contiguous(), f, layout=layout, axes=axes)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_dense_batches_strides_and_in_place():
    # [B, H, S, D], positions [axes, S] and [axes, B, S]; q and k turned in place inside one projection
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    r = np.random.RandomState(4)
    B, S, D = 3, 37, 64
    qkv = torch.from_numpy(r.randn(B, S, 8, D)).half().cuda()
    x = to_f64(qkv)
    freq = attn.rope_frequencies(D)[0]
    axes = attn.rope_axes([10, 11, 11])
    for shape in ((3, S), (3, B, S)):
        pos = r.randint(0, 5000, shape).astype(np.int32)
        full = pos if pos.ndim == 3 else np.repeat(pos[:, None], B, 1)
        t = qkv.clone()
        q, k = t[:, :, :4].transpose(1, 2), t[:, :, 4:6].transpose(1, 2)
        attn.rope(q, k, torch.from_numpy(pos).cuda(), freq.cuda(), axes=axes.cuda(), q_out=q, k_out=k)
        got = to_f64(t)
        near(got[:, :, :6], x[:, :, :6], full, axes.numpy(), freq.numpy(), "half", 1.0, False, "f16")
        assert np.array_equal(got[:, :, 6:], x[:, :, 6:])


def test_gradient_is_the_transposed_turn():
    # <rope(x), y> = <x, rope_bwd(y)>: in fp32, each element off by 2^-21 m (|x1| + |x2|)
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    g = torch.Generator().manual_seed(2)
    x, y = (torch.randn((50, 2, 64), generator=g).cuda() for _ in range(2))
    pos = torch.randint(0, 900, (2, 50), generator=g, dtype=torch.int32).cuda()
    f, axes = attn.rope_frequencies(64)[0].cuda(), attn.rope_axes([20, 12]).cuda()
    a = attn.rope(x, None, pos, f, axes=axes, mscale=0.7)[0].double() * y
    b = attn.rope_bwd(y, None, pos, f, axes=axes, mscale=0.7)[0].double() * x
    pair = lambda t: (t.abs() + t.abs().roll(32, -1)).double()  # noqa: E731
    assert abs(float(a.sum() - b.sum())) <= 2.0 ** -21 * 0.7 * float((pair(x) * y.abs() + pair(y) * x.abs()).sum())
