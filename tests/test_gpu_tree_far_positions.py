"""Trees at the end of the range of positions (bounds of test_gpu_tree_attention.py)."""
import numpy as np
import pytest
import torch

from test_gpu_tree_attention import Tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("W", [1, 8, 128])
def test_the_largest_positions(cuda_lib, fmt, W):
    """Tokens up to position 2^31 - 1: their window is still themselves, their ancestors and the ring."""
    B, N, cap = 2, 7, 300
    last = (1 << 31) - 1
    c = Tree(cuda_lib, B, N, cap, "chain", fmt, W=W, R=W + 3, seed=40, ctx=[last - (N - 1), last - 40])
    idx, cnt = c.select(200)
    got = c.csa(idx, cnt)
    c.check(got, lambda b, i: idx[b, i, :int(cnt[b, i])].numpy(), what="csa")
    got = c.hca(torch.tensor([cap, 7], dtype=torch.int32), 128)
    c.check(got, lambda b, i: np.arange((cap, 7)[b]), what="hca")
    assert cuda_lib.csa_read_device_error() == 0
