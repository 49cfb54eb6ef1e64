"""Values that are no numbers, and scores near the end of fp32, in attention of sequences that share a prefix
(attn_paged_prefix_fwd)."""
import numpy as np
import pytest

from tests.gpu_util import to_f64
from tests.pages_ref import Shared, near
from tests.test_prefix_gpu import BATCHES, FORMS, run
from tests.test_prefix_long_gpu import MANY, reference

pytestmark = pytest.mark.gpu


def ids(f):
    return "-".join(str(v) for v in f.values())


@pytest.mark.parametrize("form", FORMS, ids=ids)
@pytest.mark.parametrize("strange", [float("inf"), -float("inf")])
@pytest.mark.parametrize("name", ["drafts", "mixed", "prompts"])
def test_an_infinite_value_of_the_prefix(name, form, strange):
    # element 3 of the last value of the first group's prefix: every row of the group that sees it (all do) has a
    # weight of more than 0 for it, so that element of its output is infinite and no other one changes
    b = Shared(89, BATCHES[name], **form)
    ref = list(b.ref())
    pre, members = int(b.pre[0]), range(int(b.goff[0]), int(b.goff[1]))
    for s in members:
        b.vc[b.table[s, (pre - 1) // b.P], (pre - 1) % b.P, :, 3] = strange
    out, lse = run(b)
    o, z = to_f64(out), to_f64(lse)
    rows = np.concatenate([np.arange(b.offs[s], b.offs[s + 1]) for s in members])
    assert (o[rows][:, :, 3] == strange).all()
    o[rows, :, 3] = ref[0][rows, :, 3]
    near(o, z, ref, b.dtype, b.D)


# At most 16 rows of a kv head in the group and in each sequence
FEW = [dict(dtype="f16", D=64, P=16, H=1, Hq=7, n=2), dict(dtype="f16", D=128, P=16, H=2, Hq=2, n=4),
       dict(dtype="bf16", D=128, P=64, H=2, Hq=16, n=1), dict(dtype="bf16", D=64, P=24, H=1, Hq=4, n=4)]


@pytest.mark.parametrize("form", FEW, ids=ids)
@pytest.mark.parametrize("strange", [float("inf"), -float("inf")])
@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("where", [0, 77, 299, 300])
@pytest.mark.parametrize("share", [0.02, 1.0, 10.0])
def test_an_infinite_value_of_few_rows(share, where, wide, strange, form):
    # the value of one key of all members of the group: element 3 of each of their rows is infinite, whatever the key's weight
    # (from e^-9 or so of the largest one of a row to all of it)
    form = dict(form)
    b = Shared(101, [(300, [(5, 1)] * form.pop("n")), (77, [(30, 1)])], wide=wide, **form)
    scale = share * b.D ** -0.5
    if share == 10.0:  # the key outweighs all others of the last member's last head
        for s in range(int(b.goff[1])):
            b.kc[b.table[s, where // b.P], where % b.P, -1] = b.q[int(b.goff[1]) - 1, -1]
        scale = b.D ** -0.5
    ref = list(b.ref(scale=scale))
    for s in range(int(b.goff[1])):
        b.vc[b.table[s, where // b.P], where % b.P, :, 3] = strange
    out, lse = run(b, scale=scale)
    o, z = to_f64(out), to_f64(lse)
    rows = np.arange(b.offs[b.goff[1]])
    assert (o[rows][:, :, 3] == strange).all()
    o[rows, :, 3] = ref[0][rows, :, 3]
    near(o, z, ref, b.dtype, b.D)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("groups", [[(None, [(100000, 100)])], [(60000, [(40000, 100), (70, 60)])]])
@pytest.mark.parametrize("strange", [float("nan"), float("inf")])
@pytest.mark.parametrize("back", [99995, 101, 99, 64, 2])
def test_one_value_that_is_no_number_in_a_long_context(back, strange, groups, dtype, D):
    # 400 rows of 100000 keys; the value of the key `back` places from the end, which all rows see, or none but the last ones:
    # the same time and the same status as without it
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    b = Shared(103, groups, dtype=dtype, D=D, P=64, H=1, Hq=4, wide=False)
    d = b.device()
    ref = list(reference(b, d))
    j = int(b.lens[0]) - back
    d[2][b.table[0, j // b.P], j % b.P, :, 3] = strange
    out = torch.full_like(d[0], 768.0)
    attn.device_status(0, clear=True)
    times = []
    for _ in range(2):
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        e[0].record()
        out, lse = attn.paged_prefix_fwd(*d, max_queries=b.max_q, max_group_queries=b.max_gq, return_lse=True, out=out)
        e[1].record()
        torch.cuda.synchronize()
        times.append(e[0].elapsed_time(e[1]))
    assert attn.device_status(0, clear=True) == 0
    o, z = to_f64(out), to_f64(lse)
    sees = np.zeros(len(b.q), bool)
    seqs = [s for s in range(len(b.lens)) if b.table[s, j // b.P] == b.table[0, j // b.P]]
    for s in seqs:  # the keys that query i sees: L - n + i + 1
        n, L = int(b.new[s]), int(b.lens[s])
        sees[b.offs[s]:b.offs[s + 1]] = j < L - n + np.arange(n) + 1
    assert sees.sum() >= min(back, 100)
    at = o[sees][:, :, 3]
    assert (np.isnan(at) if np.isnan(strange) else at == strange).all()
    o[sees, :, 3] = ref[0][sees, :, 3]
    near(o, z, ref, dtype, D)
    assert min(times) < 20  # ms; 0.5 to 1.3 without it


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_values_that_are_no_numbers_all_over(causal, dtype, D):
    # rows that see anything from nothing to all of a long prefix, with such values spread over it and over the own keys: an
    # element of a row is a number unless the row sees one of them there
    b = Shared(107, MANY["unequal"][:2] + [(700, [(300, 200), (90, 80)])], dtype=dtype, D=D, P=64, H=8, Hq=32)
    r = np.random.RandomState(5)
    pos = r.randint(-2, 9100, len(b.q)).astype(np.int32) if causal else None
    d = b.device()
    ref = list(reference(b, d, pos, causal))
    hit = np.zeros((len(b.q), b.H, D), bool)
    for s in r.permutation(len(b.lens))[:12]:
        n, L, at = int(b.new[s]), int(b.lens[s]), slice(b.offs[s], b.offs[s + 1])
        for j in r.randint(0, L, 3):
            h, e = int(r.randint(b.H)), int(r.randint(D))
            page = b.table[s, j // b.P]
            d[2][page, j % b.P, h, e] = [float("nan"), float("inf"), -float("inf")][int(r.randint(3))]
            for s2 in np.flatnonzero(b.table[:, j // b.P] == page):
                rows = slice(b.offs[s2], b.offs[s2 + 1])
                if j < b.lens[s2]:
                    hit[rows, h, e] |= pos[rows] >= j if causal else True
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    out, lse = attn.paged_prefix_fwd(*d, positions=torch.from_numpy(pos).cuda() if causal else None, causal=causal,
                                     max_queries=b.max_q, max_group_queries=b.max_gq, return_lse=True)
    assert attn.device_status(0, clear=True) == 0
    o, z = to_f64(out), to_f64(lse)
    hit = np.repeat(hit, b.Hq // b.H, 1)
    assert hit.any() and not np.isfinite(o[hit]).any()
    o[hit] = ref[0][hit]
    near(o, z, ref, dtype, D)


@pytest.mark.parametrize("score", [-2.3e38, -2.2e38, -2.1e38, -1e38, -1e30])
@pytest.mark.parametrize("form", FORMS, ids=ids)
@pytest.mark.parametrize("new", [1, 2])
@pytest.mark.parametrize("pre", [0, 40])
def test_a_score_near_the_end_of_fp32(pre, new, form, score):
    # few rows, whose scores are all the same, in log2 units down to -3.33e38: the output is the mean of the values, the lse
    # the score itself (the log of the number of keys is far below its last bit)
    b = Shared(97, [(40, [(new, new)] * 2), (None, [(new + 7, new)])], **form)
    b.pre[:] = pre  # 0: all keys are the sequences' own
    f16 = b.dtype == "f16"
    q, k = (2.0 ** 15, -2.0 ** 15) if f16 else (2.0 ** 64, score / 2.0 ** 64)
    b.q.zero_()
    b.q[:, :, 0] = q
    b.kc[..., 0] = k
    scale = float(np.float32(score / (q * k))) if f16 else 1.0
    exact = q * float(b.kc[0, 0, 0, 0].double()) * scale
    out, lse = run(b, causal=False, scale=scale)
    ref = list(b.ref(None, False, 0.0))  # equal scores
    o, z = to_f64(out), to_f64(lse)
    # of it: the scale and its product with log2 e, the score, the way back with ln 2, each rounded, and the two constants
    assert np.abs(z / exact - 1).max() <= 6 * 2.0 ** -24
    ref[1] = z
    near(o, z, ref, b.dtype, b.D)
