"""Buffers of the permutation wherever a caller may have them."""
import pytest
import torch

import moe_finalize_rmsnorm_gb300 as mf
from tests.test_experts_gpu import gen, permutation_ref

pytestmark = pytest.mark.gpu

GUARD = -77


def ids_of(T, K, E):
    return torch.randint(-1, E + 1, (T, K), generator=gen(T + K), dtype=torch.int32)


# one launch, two launches
@pytest.mark.parametrize("T,K,E", [(9, 4, 5), (1024, 4, 60), (1300, 4, 60), (40000, 4, 256)])
def test_permutation_in_one_allocation(cuda_lib, T, K, E):
    """The four buffers back to back."""
    ids = ids_of(T, K, E)
    n = T * K
    buf = torch.full((3 * n + E + 1,), GUARD, dtype=torch.int32, device="cuda")
    buf[:n] = ids.flatten().cuda()
    a, idx, tok, off = buf[:n].view(T, K), buf[n:2 * n].view(T, K), buf[2 * n:3 * n], buf[3 * n:]
    mf.moe_expert_permutation(a, E, expert_offsets=off, expanded_idx=idx, row_tokens=tok)
    for got, want in zip((off, idx, tok), permutation_ref(ids, E)):
        assert torch.equal(got.cpu(), want)
    assert torch.equal(a.cpu(), ids)
    with pytest.raises(mf.MoeFinalizeError):       # in place
        mf.moe_expert_permutation(a, E, expanded_idx=a)
    with pytest.raises(mf.MoeFinalizeError):       # two outputs in one place
        mf.moe_expert_permutation(a, E, expanded_idx=idx, row_tokens=idx.view(-1))
    assert torch.equal(a.cpu(), ids)
