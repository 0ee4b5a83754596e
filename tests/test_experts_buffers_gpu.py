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


@pytest.mark.parametrize("T,K,E", [(9, 1, 5), (700, 5, 33), (4097, 1, 60), (8211, 3, 100),
                                   (140001, 1, 256)])
def test_permutation_of_slices(cuda_lib, T, K, E):
    """A batch's ids from some token on, outputs at any word of a larger buffer."""
    ids = ids_of(T + 3, K, E)
    n = T * K
    whole = ids.cuda()
    for first in (1, 2, 3):
        part = whole[first:first + T]
        bufs = [torch.full((size + 8,), GUARD, dtype=torch.int32, device="cuda")
                for size in (E + 1, n, n)]
        off, idx, tok = (b[first:first + size] for b, size in zip(bufs, (E + 1, n, n)))
        mf.moe_expert_permutation(part, E, expert_offsets=off, expanded_idx=idx.view(T, K),
                                  row_tokens=tok)
        want = permutation_ref(ids[first:first + T], E)
        for b, out, ref in zip(bufs, (off, idx, tok), want):
            assert torch.equal(out.cpu(), ref.flatten())
            assert (b[:first] == GUARD).all() and (b[first + out.numel():] == GUARD).all()
