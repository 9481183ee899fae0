"""csa_verify_drafts: parents that are none, as padding has them, and the largest vocabulary."""
import numpy as np
import pytest
import torch

from test_gpu_verify_drafts import call, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q", [None, "fp32"])
def test_parents_that_are_none_are_never_reached(cuda_lib, q):
    """Entries outside [-1, i), and -1 itself, keep a token out of the walk; token 0's is not read."""
    x = make(24, 9, 600, "random", "fp32", q, seed=50)
    g = torch.Generator().manual_seed(51)
    out = torch.rand((24, 9), generator=g) < 0.3
    out[:, 0] = False
    x["parent"][out] = -1
    want = call(cuda_lib, x)
    check(x, want)
    i = torch.arange(9, dtype=torch.int32).expand(24, 9)
    none = torch.stack([i, i + 1, torch.full_like(i, 8), torch.full_like(i, -2), torch.full_like(i, (1 << 31) - 1),
                        torch.full_like(i, -(1 << 31))])
    pick = torch.randint(0, 6, (24, 9), generator=g)
    x["parent"][out] = none.gather(0, pick[None])[0][out]
    x["parent"][:, 0] = torch.randint(-(1 << 31), (1 << 31) - 1, (24,), generator=g).to(torch.int32)
    assert all(np.array_equal(a, b) for a, b in zip(call(cuda_lib, x), want))
    assert cuda_lib.csa_read_device_error() == 0


@pytest.mark.parametrize("q", [None, "bf16"])
def test_the_largest_vocabulary(cuda_lib, q):
    """2^24 tokens: a thread sums 4096 of them, 128 rounds of 32 (below 128 2^-24 = 8e-6 of the sum)."""
    x = make(1, 3, 1 << 24, "chain", "bf16", q, seed=52)
    check(x, call(cuda_lib, x))
    assert cuda_lib.csa_read_device_error() == 0
