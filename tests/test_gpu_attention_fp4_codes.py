"""E2M1 codes of the attention over 4-bit records, each against the values that the
same call forms in BF16.

Bound, derived before the first run: the call forms the same fp32 value y for both
outputs. The BF16 one, o, is half a step off at most: |y - o| <= 2^-8 |o| (1 + 2^-8).
The code is E2M1's nearest to y / s: half the distance of the two codes around it,
s / 4 up to 2 s, s / 2 up to 4 s and s above (the largest value is 6 s, up to its
rounding), and 2^-20 of it for the quotient's fp32 roundings (at most four of
2^-24)."""
import numpy as np
import pytest

import _records as R
from test_gpu_attention_fp4 import Case

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8


def unpacked(codes):
    p = codes.cpu().numpy()
    code = np.stack([p & 15, p >> 4], -1).reshape(*p.shape[:-1], 512)
    return np.where(code >= 8, -1.0, 1.0) * R.E2M1[code & 7]


def check_codes(e2m1, out, what):
    codes, scale = e2m1
    s = np.repeat(scale.double().cpu().numpy(), 128, axis=-1)
    o = out.double().cpu().numpy()
    v = unpacked(codes) * s
    near = BF * (1 + BF) * np.abs(o)
    a = (np.abs(o) + near) / s
    half = np.where(a <= 2, 0.25, np.where(a <= 4, 0.5, 1.0)) * s
    bound = half * (1 + 2.0 ** -20) + near
    err = np.abs(v - o)
    assert np.all(err <= bound), f"{what}: {np.max(err / np.maximum(bound, 1e-300)):.3g} x bound"
    amax = np.abs(o).reshape(*o.shape[:-1], 4, 128).max(-1)
    m = scale.double().cpu().numpy()
    assert np.all(np.abs(m - np.where(amax > 0, amax / 6, 1)) <= BF * (1 + BF) * np.where(amax > 0, amax / 6, 1))
    # the codes of a random output use every magnitude
    assert np.all(np.bincount(np.searchsorted(R.E2M1, np.abs(unpacked(codes))).ravel(), minlength=8) > 0)


# rows over several pairs of CTAs (the codes formed where the splits are joined: one
# warp a head, and eight), and rows of one pair
@pytest.mark.parametrize("B,T,cap,n", [(1, 1, 1900, 1800), (1, 1, 500, 333), (24, 1, 700, 600), (40, 2, 80, 60), (90, 1, 300, 200)])
def test_codes_are_the_nearest(cuda_lib, B, T, cap, n):
    csd = cuda_lib
    c = Case(csd, B, T, cap, seed=71 + cap)
    counts = [[max(1, n - 7 * (b % 8) - t) for t in range(T)] for b in range(B)]
    idx, cnt = c.select(n, counts)
    for kw in (dict(), dict(inverse_rope=True, rope_theta=500000.0)):
        e2m1, lse = c.csa(idx, cnt, fp4_out=True, **kw)
        out, lse2 = c.csa(idx, cnt, **kw)
        assert np.array_equal(lse.cpu().numpy(), lse2.cpu().numpy())
        check_codes(e2m1, out, f"{B} x {T} rows of {n} {kw}")
    assert csd.csa_read_device_error() == 0


@pytest.mark.parametrize("B,n", [(1, 700), (24, 200), (90, 60)])  # eight warps a head, one, and no splits
def test_a_nan_of_the_output_is_not_hidden_by_its_codes(cuda_lib, B, n):
    """E2M1 has no NaN: the multiplier of a block of 128 dims that holds one is NaN."""
    csd = cuda_lib
    c = Case(csd, B, 1, n + 20, paged=False, seed=81)
    idx, cnt = c.select(n, [[n]] * B)
    (codes, scale), lse = c.csa(idx, cnt, fp4_out=True)
    assert np.all(np.isfinite(scale.cpu().numpy()))
    bad = B // 2
    at = bad * (n + 20) + int(idx[bad, 0, n // 2])
    c.pool[at, 224 + 2 * 9:224 + 2 * 9 + 2] = 255  # rope dim 9 of one selected record
    (codes2, scale2), _ = c.csa(idx, cnt, fp4_out=True)
    assert np.all(np.isnan(scale2[bad].cpu().numpy()))  # the score is NaN, so is the whole row
    rest = [b for b in range(B) if b != bad]
    assert np.array_equal(scale2[rest].cpu().numpy(), scale[rest].cpu().numpy())
    assert np.array_equal(codes2[rest].cpu().numpy(), codes[rest].cpu().numpy())
    c.pool[at, 224 + 2 * 9:224 + 2 * 9 + 2] = 0
    c.q[bad, 0, 77, 300] = float("nan")  # one head of the query
    _, s = c.csa(idx, cnt, fp4_out=True)[0]
    nan = np.isnan(s.cpu().numpy())
    assert np.all(nan[bad, 0, 77]) and nan.sum() == 4
    assert csd.csa_read_device_error() == 0
