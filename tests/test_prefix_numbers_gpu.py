"""Infinite values in attention of sequences that share a prefix (attn_paged_prefix_fwd)."""
import numpy as np
import pytest

from tests.gpu_util import to_f64
from tests.pages_ref import Shared, near
from tests.test_prefix_gpu import BATCHES, FORMS, run

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
