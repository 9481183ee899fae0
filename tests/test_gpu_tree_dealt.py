"""Dealt-out queries of a tree: E2M1 output, parents that are none (bounds of test_gpu_tree_attention.py)."""
import numpy as np
import pytest
import torch

import _speculative as S
from test_gpu_tree_attention import Tree

pytestmark = pytest.mark.gpu
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("B, N", [(4, 9), (19, 2), (3, 25)])
def test_e2m1_output(cuda_lib, fmt, B, N):
    """Codes of queries that are split and of some that are not, within half a step (at most 1, in units of the
    multiplier) of a value within the bound; padding keeps its rows."""
    csd, cap = cuda_lib, 3300
    c = Tree(csd, B, N, cap, "random", fmt, seed=60 + B)
    c.pos = (cap + S.depths(c.parent)).to(torch.int32)
    c.pos[B - 1, 1:] = -1
    n_comp = torch.full((B,), 3, dtype=torch.int32)
    n_comp[0], n_comp[B - 1] = cap, cap // 2
    codes = torch.full((B, N, 128, 256), 0x5A, dtype=torch.uint8, device="cuda")
    scale = torch.full((B, N, 128, 4), 7.0, device="cuda")
    lse = torch.full((B, N, 128), 7.0, device="cuda")
    c.hca(n_comp, 1, inverse_rope=True, fp4_out=True, out_fp4=codes, out_fp4_scale=scale, lse=lse)
    assert csd.csa_read_device_error() == 0
    pad = c.pos < 0
    code, sc = codes.cpu(), scale.cpu()
    assert bool((code[pad] == 0x5A).all()) and bool((sc[pad] == 7).all()) and bool((lse.cpu()[pad] == 7).all())
    code = np.stack([code.numpy() & 15, code.numpy() >> 4], -1).reshape(B, N, 128, 512)
    step = np.repeat(sc.double().numpy(), 128, axis=-1)
    val = np.where(code >= 8, -1.0, 1.0) * GRID[code & 7] * step
    for b, i in ((0, 0), (0, N - 1), (1, N - 1), (B - 1, 0)):
        o, l, bound, lbound = c.reference(b, i, np.arange(int(n_comp[b])), 10000.0)
        assert np.all(np.abs(val[b, i] - o) <= bound + step[b, i] * (1 + 1e-3))
        assert np.all(np.abs(lse[b, i].double().cpu().numpy() - l) <= lbound)


@pytest.mark.parametrize("fmt", [0, 1])
def test_bad_parents_are_reported_and_taken_as_none(cuda_lib, fmt):
    csd, B, N, cap = cuda_lib, 4, 9, 3300
    c = Tree(csd, B, N, cap, "chain", fmt, seed=70)
    n_comp = torch.tensor([cap, 9, 0, 1200], dtype=torch.int32)
    c.parent[0, 4], c.parent[2, 8], c.parent[3, 0] = 4, -3, 1 << 30
    c.pos = (cap + S.depths(c.parent)).to(torch.int32)
    got = c.hca(n_comp, 1)
    assert csd.csa_read_device_error() == csd.ERR_BAD_INDEX
    c.check(got, lambda b, i: np.arange(int(n_comp[b])), rows={(0, 3), (0, 4), (0, 8), (2, 7), (2, 8), (3, 0), (3, 8)})
