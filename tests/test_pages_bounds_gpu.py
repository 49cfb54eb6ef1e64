"""The pages of a cache on the GPU (attn_pages_*) at the ends of their ranges."""
import numpy as np
import pytest

from tests.test_pages_gpu import Both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P,M", [(1000, 2147483), (1200000000, 1), (2147483647, 1)])
def test_fork_of_a_full_row(P, M):
    # rows of close to 2^31 tokens: the child names every page of its parent
    import torch
    from exact_scaled_dot_flash_gb300 import attn
    N = 7
    table = torch.full((2, M), -1, dtype=torch.int32, device="cuda")
    table[0] = torch.arange(M, device="cuda", dtype=torch.int32) % N
    refs = torch.bincount(table[0], minlength=N).int()
    for tokens in (M * P, M * P - 1, (M - 1) * P + 1, (M - 1) * P):
        lens = torch.tensor([tokens, 0], dtype=torch.int32, device="cuda")
        attn.pages_fork(table, lens, refs, lens.new_tensor([0]), lens.new_tensor([1]), page_size=P)
        held = -(-tokens // P)
        assert lens.tolist() == [tokens, tokens]
        assert torch.equal(table[1, :held], table[0, :held]) and bool((table[1, held:] == -1).all())
        assert torch.equal(torch.bincount(torch.cat([table[0], table[1, :held]]), minlength=N).int(), refs)
        attn.pages_free(table, lens, refs, lens.new_tensor([1]))
    assert torch.equal(torch.bincount(table[0], minlength=N).int(), refs)


@pytest.mark.parametrize("S,M,P,N", [(4097, 3, 4, 6000), (9000, 2, 8, 9100), (5000, 4, 3, 40000)])
def test_more_sequences_than_a_block_keeps(S, M, P, N):
    b = Both(S, M, P, N, [("i16", (P, 2))], seed=S)
    r = np.random.RandomState(S)
    for step in range(4):
        b.reserve(np.where(r.rand(S) < 0.4, r.randint(0, 2 * P, S), 0))
        kids = np.flatnonzero(b.ref.lens == 0)[:S // 8]
        parents = np.flatnonzero(b.ref.lens > 0)
        if len(kids) and len(parents):
            b.fork(r.choice(parents, len(kids)).tolist(), kids.tolist())
        b.reserve(r.randint(0, 2, S))
        b.free(r.permutation(S)[:S // 3].tolist())
        b.compact()
