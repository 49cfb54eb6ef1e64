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

