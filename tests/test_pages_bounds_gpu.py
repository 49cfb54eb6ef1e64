"""The pages of a cache on the GPU (attn_pages_*) at the ends of their ranges."""
import pytest

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

