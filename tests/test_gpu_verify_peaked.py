"""csa_verify_drafts where nearly all of the target is refused, against the definition in 64 bits.

What is left, R, is a sum of weights of up to 2^-44 of the largest: each is off by 44 2^-24 ln 2 (the
exponent's product) and as much for the rounding of the factor, together below 4e-6, and their fp32 sum by
less than 1e-6 of itself. The second or third sibling's uniform number is put 1e-4 beside the border u R = r.
"""
import numpy as np
import pytest
import torch

import _speculative as S
from test_gpu_verify_drafts import call, check

pytestmark = pytest.mark.gpu
MOST = 1 - 2.0 ** -24  # the largest uniform number


def peaked(B, V, rests, dtype, seed):
    """Stars of len(rests) + 1 drafts: draft i weighs 1 / rests[i] of all that comes after it, and the last one
    0.5 to 1.5 of the other tokens."""
    g = torch.Generator().manual_seed(seed)
    N = len(rests) + 2
    logits = torch.randn((B, 1, V), generator=g, dtype=torch.float64) * 0.5
    token = torch.stack([torch.randperm(V, generator=g)[:N] for _ in range(B)])
    for b in range(B):
        w = torch.exp(logits[b, 0])
        w[token[b, 1:]] = 0
        left = w.sum()
        logits[b, 0, token[b, N - 1]] = torch.log(left * float(0.5 + torch.rand((), generator=g)))
        left = left + torch.exp(logits[b, 0, token[b, N - 1]])
        for i in range(N - 2, 0, -1):
            logits[b, 0, token[b, i]] = torch.log(left / rests[i - 1])
            left = left + left / rests[i - 1]
    logits = logits.to(dtype).expand(B, N, V).contiguous()
    uniform = torch.full((B, N), MOST)
    for b in range(B):
        z = logits[b, 0].double()
        p = torch.softmax(z, 0)
        p[token[b, 1:N - 1]] = 0
        border = float(p[token[b, N - 1]] / p.sum())
        uniform[b, N - 1] = border * (1 + (1e-4 if b % 2 else -1e-4))
    return dict(logits=logits, tokens=token.to(torch.int32), parent=torch.tensor([-1] + [0] * (N - 1), dtype=torch.int32)
                .expand(B, N).contiguous(), uniform=uniform,
                noise=(-torch.log1p(-torch.rand((B, V), generator=g))).clamp(min=1e-9), draft_probs=None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [40, 4097, 32000, 131072])
@pytest.mark.parametrize("rests", [(0.5,), (0.1,), (1e-2,), (1e-4,), (3e-5,), (1e-3, 1e-3), (1e-4, 1e-2, 1e-2)])
def test_siblings_of_what_is_left(cuda_lib, rests, V, dtype):
    B = 16
    x = peaked(B, V, rests, dtype, seed=V + len(rests))
    got = call(cuda_lib, x)
    assert [int(n) for n in got[1]] == [1 if b % 2 else 2 for b in range(B)]
    check(x, got)
    assert cuda_lib.csa_read_device_error() == 0
