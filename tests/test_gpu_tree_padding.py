"""Padding of trees: tokens that are not computed must not be looked at, whatever their selections hold (bounds of
test_gpu_tree_attention.py)."""
import pytest
import torch

import _speculative as S
from test_gpu_tree_attention import Tree, outputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("B, N, k", [(1, 6, 300), (3, 8, 600), (20, 5, 100), (4, 4, 2048), (19, 2, 1500)])
# parts of a query, several and one; dealt out
def test_selections_of_padding_are_not_looked_at(cuda_lib, fmt, B, N, k):
    """Rows of padding hold what a caller's own selection left there: any count, any index."""
    csd, cap = cuda_lib, 2100
    c = Tree(csd, B, N, cap, "random", fmt, seed=30 + B)
    idx, cnt = c.select(k)
    c.pos[:, N // 2 + 1:] = -1
    c.pos[B - 1, 1:] = -(1 << 31)
    pad = c.pos < 0
    g = torch.Generator().manual_seed(31)
    idx[pad] = torch.randint(-(1 << 31), (1 << 31) - 1, (int(pad.sum()), k), generator=g).to(torch.int32)
    cnt[pad] = torch.randint(1, 1 << 30, (int(pad.sum()),), generator=g).to(torch.int32)
    out, lse = outputs(B, N)
    got = c.csa(idx, cnt, out=out, lse=lse, inverse_rope=True)
    assert csd.csa_read_device_error() == 0
    assert bool((got[0].cpu()[pad] == 7).all()) and bool((got[1].cpu()[pad] == 7).all())
    c.check(got, lambda b, i: idx[b, i, :int(cnt[b, i])].numpy(), 10000.0, rows={(0, 0), (0, N // 2), (B - 1, 0)})
