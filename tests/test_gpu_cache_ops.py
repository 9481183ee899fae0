"""csa_head_norm_rope(_e4m3), csa_cache_append and csa_cache_read against the
64-bit restatement in _records.py.

Tolerances (derived before the first run). u = 2^-24 (fp32 half step).
* norm: the sum of D <= 512 squares is a chain of at most 16 fmas and 5 shuffle
  adds (relative error 21 u), rsqrt 2 ulp, two products: below 30 u = 1.8e-6
  relative. rotation: sine and cosine within 5e-7 absolute of the true angle
  (special function unit, angle to 2^-31 of a turn), so each value of a pair
  (a, b) moves by at most 5e-7 (|a| + |b|) + 3 u (|a| + |b|). Together REL =
  3e-6 of (|a| + |b|) (nope dims: of |a|).
* BF16 storage: half a step, 2^-8 of the value. E4M3 storage: 2^-4 of the
  value, or half its smallest step, 2^-10, in units of the scale. A scale is
  amax / 448: relative REL.
* 4-bit records without a norm: the inputs are floats that the reference sees
  unchanged, and the kernel decides as if exactly: bytes equal. With a norm the
  values carry REL, so a code or scale may fall on the other side of a midpoint:
  the stored value is then within one unit (the largest half step, 4..6) and the
  scale within one E4M3 step.
"""
import numpy as np
import pytest
import torch

import _records as R

pytestmark = pytest.mark.gpu
REL, BF16, E4M3 = 3e-6, 2.0 ** -8, 2.0 ** -4
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def cpu64(t):
    return t.double().cpu().numpy()


def pair_magnitude(y, x, rope_dim):
    """|a| + |b| of each value's pair (|y| outside the rotated dims)."""
    m = np.abs(y).copy()
    D = y.shape[-1]
    if rope_dim:
        s = np.abs(y[..., D - rope_dim::2]) + np.abs(y[..., D - rope_dim + 1::2])
        m[..., D - rope_dim::2] = m[..., D - rope_dim + 1::2] = 1.5 * s
    return m


def check(got, want, bound, what):
    err = np.abs(got - want)
    assert np.all(np.isfinite(got)), what
    worst = float(np.max(err / bound)) if err.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} x bound"


SHAPES = [  # B, T, H, D, rope_dim, sliced
    (1, 1, 1, 64, 64, False), (1, 1, 128, 512, 64, False), (3, 5, 7, 512, 64, True), (2, 3, 64, 128, 64, False),
    (1, 9, 3, 128, 0, True), (2, 2, 5, 192, 192, False), (1, 4, 2, 256, 256, True), (4, 1, 37, 72, 8, False),
    (1, 130, 1, 512, 64, False), (1, 1, 3, 8, 8, False), (2, 1, 2, 504, 128, True),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_head_norm_rope(cuda_lib, shape, dtype):
    csd = cuda_lib
    B, T, H, D, rope, sliced = shape
    g = torch.Generator(device="cuda").manual_seed(B + 7 * T + 11 * H + D)
    wide = torch.randn((B, T, H * D + (64 if sliced else 0)), generator=g, device="cuda").to(dtype)
    x = wide[..., :H * D].unflatten(-1, (H, D))
    pos = torch.randint(0, 1 << 21, (B, T), generator=g, device="cuda", dtype=torch.int32)
    pos[0, -1] = 2147483647
    w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    for norm, weight in ((True, w), (True, None), (False, None)):
        out = csd.csa_head_norm_rope(x, pos, weight=weight, norm=norm, eps=1e-6, rope_dim=rope, rope_theta=10000.0)
        codes, scale = csd.csa_head_norm_rope_e4m3(x, pos, weight=weight, norm=norm, rope_dim=rope)
        ww = None if not norm else (np.ones(D) if weight is None else cpu64(weight))
        y = R.norm_rope(cpu64(x), pos.cpu().numpy(), ww, float(np.float32(1e-6)), rope, 10000.0)
        m = pair_magnitude(y, None, rope)
        check(cpu64(out), y, BF16 * np.abs(y) + 1.01 * REL * m + 1e-30, f"bf16 {shape} {norm}")
        amax = np.abs(y).max(-1)
        s = cpu64(scale)
        check(s, amax / 448, 2 * REL * amax / 448 + 1e-30, f"scale {shape}")
        v = cpu64(codes.view(torch.float8_e4m3fn)) * s[..., None]
        check(v, y, E4M3 * np.abs(y) + 2.0 ** -10 * s[..., None] + 2 * REL * m + 1e-30, f"e4m3 {shape}")
    assert csd.csa_read_device_error() == 0


def test_head_norm_rope_in_place_padding_and_zero_rows(cuda_lib):
    csd = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((2, 6, 9, 512), generator=g, device="cuda").to(torch.bfloat16)
    x[0, 1, 4] = 0
    x[1, 2] = float("nan")  # a padded token's contents are not looked at
    pos = torch.arange(12, device="cuda", dtype=torch.int32).view(2, 6)
    pos[1, 2] = -1
    pos[0, 5] = -5
    want = csd.csa_head_norm_rope(x, pos, out=torch.full_like(x, 7.0))
    assert torch.all(want[1, 2] == 7) and torch.all(want[0, 5] == 7)
    assert torch.all(want[0, 1, 4] == 0) and torch.all(want[0, 0].float().abs() < 7)
    assert not torch.isnan(want).any()
    codes = torch.full((2, 6, 9, 512), 99, dtype=torch.uint8, device="cuda")
    scale = torch.full((2, 6, 9), 5.0, device="cuda")
    csd.csa_head_norm_rope_e4m3(x, pos, codes=codes, scale=scale)
    assert torch.all(codes[1, 2] == 99) and torch.all(scale[0, 5] == 5)
    assert torch.all(codes[0, 1, 4] == 0) and torch.all(scale[0, 1, 4] == 1)
    y = x.clone()
    assert csd.csa_head_norm_rope(y, pos, out=y) is y
    keep = want.clone()
    keep[1, 2], keep[0, 5] = x[1, 2], x[0, 5]
    assert torch.equal(y.view(torch.int16), keep.view(torch.int16))


def test_nan_and_infinity_stay_in_their_head(cuda_lib):
    csd = cuda_lib
    x = torch.randn((1, 1, 6, 128), device="cuda").to(torch.bfloat16)
    clean = csd.csa_head_norm_rope(x, torch.zeros((1, 1), dtype=torch.int32, device="cuda"))
    bad = x.clone()
    bad[0, 0, 2, 5] = float("nan")
    bad[0, 0, 4, 100] = float("inf")
    out = csd.csa_head_norm_rope(bad, torch.zeros((1, 1), dtype=torch.int32, device="cuda"))
    assert torch.isnan(out[0, 0, 2]).all()
    assert torch.isnan(out[0, 0, 4, 100]) and torch.all(out[0, 0, 4, :64] == 0)
    codes, scale = csd.csa_head_norm_rope_e4m3(bad, torch.zeros((1, 1), dtype=torch.int32, device="cuda"))
    assert torch.isnan(codes.view(torch.float8_e4m3fn)[0, 0, 2].float()).all() and torch.isnan(scale[0, 0, 2])
    for h in (0, 1, 3, 5):
        assert torch.equal(out[0, 0, h], clean[0, 0, h])


def make_cache(csd, fmt, B, cap, paged, page=4, extra=3, seed=0):
    """(description, pool, logical-to-record function)."""
    size = csd.FORMAT_BYTES[fmt]
    g = torch.Generator().manual_seed(seed)
    if not paged:
        pool = torch.full((B * cap + extra, size), 0xAB, dtype=torch.uint8, device="cuda")
        return csd.cache_desc(pool, cap, seq_stride=cap, fmt=fmt), pool, lambda b, e: b * cap + e
    pages = -(-cap // page)
    table = torch.randperm(B * pages + extra, generator=g)[:B * pages].to(torch.int32).view(B, pages)
    pool = torch.full(((B * pages + extra) * page, size), 0xAB, dtype=torch.uint8, device="cuda")
    d = csd.cache_desc(pool, cap, block_table=table.cuda(), page_records=page, fmt=fmt)
    return d, pool, lambda b, e: int(table[b, e // page]) * page + e % page


APPENDS = [  # B, T, cap, ring, paged, pos_stride, norm, keys
    (1, 1, 1, False, False, 1, False, False), (2, 5, 9, False, True, 4, False, True),
    (3, 17, 40, False, True, 128, True, True), (2, 3, 130, True, False, 1, True, False),
    (2, 40, 16, True, False, 1, False, False), (5, 9, 64, False, False, 4, True, True),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("case", APPENDS)
def test_append_and_read(cuda_lib, case, fmt, dtype):
    csd = cuda_lib
    B, T, cap, ring, paged, stride, norm, keys = case
    g = torch.Generator(device="cuda").manual_seed(T + cap)
    x = (torch.randn((B, T, 512), generator=g, device="cuda") *
         torch.exp(2 * torch.randn((B, T, 1), generator=g, device="cuda"))).to(dtype)
    x[0, 0, :448] = 0  # an all-zero record
    if T > 2:
        x[-1, 1, 16:448] = 0  # blocks far below the record's maximum, and zero ones
        x[-1, 1, 32:48] = 1e-6
        x[-1, 2, :448] = x[-1, 2, :448].sign() * 2.5  # quotients on halfway points
    first = torch.randint(0, (200 if ring else cap - T) + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    count = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    count[0], count[-1] = T, T
    w = 1 + 0.1 * torch.randn(512, generator=g, device="cuda") if norm else None
    d, pool, at = make_cache(csd, fmt, B, cap, paged)
    kw = {}
    if keys:
        key = torch.randn((B, T, 128), generator=g, device="cuda").to(dtype)
        k_idx = torch.full((B, cap, 128), 0xCD, dtype=torch.uint8, device="cuda")
        k_scale = torch.full((B, cap), -3.0, device="cuda")
        kw = dict(key=key, k_idx=k_idx, k_idx_scale=k_scale)
    csd.csa_cache_append(d, x, first, count, ring=ring, norm=norm, weight=w, pos_stride=stride, **kw)
    back = csd.csa_cache_read(d, first, count, T, ring=ring, out=torch.full((B, T, 512), 9.0, dtype=torch.bfloat16,
                                                                          device="cuda"))
    assert csd.csa_read_device_error() == 0
    pool_h, back_h = pool.cpu().numpy(), cpu64(back)
    untouched = np.ones(len(pool_h), bool)
    seen_keys = np.zeros((B, cap), bool)
    for b in range(B):
        f, n = int(first[b]), int(count[b])
        t0 = max(0, n - cap) if ring else 0
        assert np.all(back_h[b, :t0] == 9) and np.all(back_h[b, n:] == 9)
        if n == t0:
            continue
        e = f + np.arange(t0, n)
        r = np.array([at(b, int(i) % cap if ring else int(i)) for i in e])
        untouched[r] = False
        y = R.norm_rope(cpu64(x[b, t0:n]), e * stride, None if not norm else cpu64(w), float(np.float32(1e-6)), 64,
                        10000.0)
        m = pair_magnitude(y, None, 64)
        rec = pool_h[r]
        v = R.fp4_values(rec) if fmt else R.fp8_values(rec)
        check(v[:, 448:], y[:, 448:], BF16 * np.abs(y[:, 448:]) + REL * m[:, 448:] + 1e-30, "rope dims")
        if fmt:
            assert np.all(rec[:, 381:] == 0)
            unit = np.repeat(R.E4M3[rec[:, 352:380]] * 2.0 ** (rec[:, 380:381].astype(np.float64) - 127), 16, axis=1)
            for i in range(len(r)):
                codes, scales, E = R.fp4_record(y[i])
                if not norm:
                    got = np.stack([rec[i, :224] & 15, rec[i, :224] >> 4], -1).reshape(-1)
                    assert rec[i, 380] == E + 127, (b, i)
                    assert np.array_equal(rec[i, 352:380], scales), (b, i)
                    assert np.array_equal(got & 7, codes & 7), (b, i)
                    assert np.array_equal(got[codes & 7 > 0] >> 3, codes[codes & 7 > 0] >> 3), (b, i)
                else:
                    assert abs(int(rec[i, 380]) - (E + 127)) <= 1
            check(v[:, :448], y[:, :448], unit + 2.0 ** -10 * 6 * 2.0 ** (rec[:, 380:381] - 127.0) +
                  REL * np.abs(y[:, :448]) + 1e-30, "4-bit values")
            want = v
            assert np.array_equal(back_h[b, t0:n], want)
        else:
            mult = rec[:, 576:592].copy().view(np.float32).astype(np.float64)
            blocks = np.pad(np.abs(y[:, :448]), ((0, 0), (0, 64))).reshape(len(r), 4, 128).max(-1)
            want_m = np.where(blocks > 0, blocks / 448, 1.0)
            check(mult, want_m, 2 * REL * want_m, "multipliers")
            per = np.repeat(mult, 128, axis=1)[:, :448]
            check(v[:, :448], y[:, :448], E4M3 * np.abs(y[:, :448]) + 2.0 ** -10 * per + 2 * REL * np.abs(y[:, :448]) +
                  1e-30, "FP8 values")
            check(back_h[b, t0:n], v, BF16 * (1 + 1e-6) * np.abs(v) + 1e-30, "FP8 read back")
        if keys:
            k = R.norm_rope(cpu64(key[b, t0:n]), e * stride, None, 0, 64, 10000.0)
            km = pair_magnitude(k, None, 64)
            s = cpu64(k_scale[b, f:f + n])
            amax = np.abs(k).max(-1)
            check(s, amax / 448, 2 * REL * amax / 448, "key scale")
            kv = cpu64(k_idx[b, f:f + n].view(torch.float8_e4m3fn)) * s[:, None]
            check(kv, k, E4M3 * np.abs(k) + 2.0 ** -10 * s[:, None] + 2 * REL * km, "key codes")
            seen_keys[b, f:f + n] = True
    assert np.all(pool_h[untouched] == 0xAB), "a record that no token belongs to changed"
    if keys:
        assert np.all(k_idx.cpu().numpy()[~seen_keys] == 0xCD) and np.all(k_scale.cpu().numpy()[~seen_keys] == -3)


@pytest.mark.parametrize("fmt", [0, 1])
def test_entries_outside_the_cache_are_reported_and_skipped(cuda_lib, fmt):
    csd = cuda_lib
    x = torch.randn((2, 4, 512), device="cuda").to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")

    def run(first, count, **kw):
        d, pool, at = make_cache(csd, fmt, 2, 6, False)
        csd.csa_cache_append(d, x, torch.tensor(first, **i32), None if count is None else torch.tensor(count, **i32), **kw)
        back = csd.csa_cache_read(d, torch.tensor(first, **i32), None if count is None else torch.tensor(count, **i32), 4,
                                  ring=kw.get("ring", False))
        written = [int(r) for r in np.flatnonzero((pool.cpu().numpy() != 0xAB).any(1))]
        return csd.csa_read_device_error(), written, back

    assert run([0, 2], None)[:2] == (0, [0, 1, 2, 3, 8, 9, 10, 11])
    code, written, back = run([4, 0], None)  # entries 6 and 7 of sequence 0 are outside
    assert code == csd.ERR_BAD_INDEX and written == [4, 5, 6, 7, 8, 9]
    assert torch.all(back[0, 2:] == 0)
    assert run([-1, 0], None)[:2] == (csd.ERR_BAD_INDEX, [6, 7, 8, 9])
    assert run([0, 0], [-3, 1])[:2] == (csd.ERR_BAD_INDEX, [6])
    assert run([0, 0], [9, 0])[:2] == (csd.ERR_BAD_INDEX, [0, 1, 2, 3])
    assert run([2147483647, 0], [4, 1], ring=True)[0] == 0  # entry numbers past 32 bits wrap in the ring
    assert run([-2, 0], [4, 1], ring=True)[0] == csd.ERR_BAD_INDEX
    assert run([2147483647, 0], [4, 1])[:2] == (csd.ERR_BAD_INDEX, [6])
    # a block table's negative page, and one past the pool
    for page in (-1, 1 << 20):
        pool = torch.full((8, csd.FORMAT_BYTES[fmt]), 0xAB, dtype=torch.uint8, device="cuda")
        d = csd.cache_desc(pool, 8, block_table=torch.tensor([[0, page]], **i32), page_records=4, fmt=fmt)
        csd.csa_cache_append(d, x[:1], torch.tensor([2], **i32))
        assert csd.csa_read_device_error() == csd.ERR_BAD_INDEX
        assert np.flatnonzero((pool.cpu().numpy() != 0xAB).any(1)).tolist() == [2, 3]
    # indexer keys past their own capacity
    d, pool, _ = make_cache(csd, fmt, 2, 6, False)
    k_idx = torch.zeros((2, 3, 128), dtype=torch.uint8, device="cuda")
    ks = torch.zeros((2, 3), device="cuda")
    csd.csa_cache_append(d, x, torch.zeros(2, **i32), key=x[..., :128], k_idx=k_idx, k_idx_scale=ks)
    assert csd.csa_read_device_error() == csd.ERR_BAD_INDEX and torch.all(ks > 0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_latents_read_back_as_nan(cuda_lib, bad):
    csd = cuda_lib
    x = torch.randn((1, 3, 512), device="cuda").to(torch.bfloat16)
    x[0, 1, 200] = bad
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    for fmt in (0, 1):
        d, pool, _ = make_cache(csd, fmt, 1, 3, False)
        csd.csa_cache_append(d, x, zero, rope_theta=None)
        back = csd.csa_cache_read(d, zero, None, 3).float()
        hit = slice(0, 448) if fmt else slice(128, 256)
        assert torch.isnan(back[0, 1, hit]).all()
        if not fmt:
            assert torch.isfinite(back[0, 1, :128]).all() and torch.isfinite(back[0, 1, 256:]).all()
        assert torch.equal(back[0, 1, 448:], x[0, 1, 448:].float())
        assert torch.isfinite(back[0, 0]).all() and torch.isfinite(back[0, 2]).all()
    assert csd.csa_read_device_error() == 0


def test_values_at_the_ends_of_the_range(cuda_lib):
    """Latents near the largest and smallest fp32 values, against the reference
    bytes (4 bits) and the stored multiplier (FP8)."""
    csd = cuda_lib
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    rng = torch.Generator(device="cuda").manual_seed(1)
    base = torch.randn((1, 5, 512), generator=rng, device="cuda")
    size = torch.tensor([1e37, 1e-20, 1e-33, 1e-38, 1e-42], device="cuda")[None, :, None]
    x = base * size
    for fmt in (0, 1):
        d, pool, _ = make_cache(csd, fmt, 1, 5, False)
        csd.csa_cache_append(d, x, zero, rope_theta=None)
        rec = pool.cpu().numpy()[:5]
        for i in range(5):
            y = cpu64(x[0, i])
            if fmt:
                codes, scales, E = R.fp4_record(y)
                assert rec[i, 380] == E + 127 and np.array_equal(rec[i, 352:380], scales)
                got = np.stack([rec[i, :224] & 15, rec[i, :224] >> 4], -1).reshape(-1)
                assert np.array_equal(got & 7, codes & 7)
            else:
                v = R.fp8_values(rec[i:i + 1])[0, :448]
                mult = rec[i, 576:592].copy().view(np.float32).astype(np.float64)
                per = np.repeat(mult, 128)[:448]
                # a subnormal multiplier holds amax / 448 to half of 2^-149
                assert np.all(np.abs(v - y[:448]) <= E4M3 * np.abs(y[:448]) + 2.0 ** -10 * per +
                              448 * (2.0 ** -150 + 2.0 ** -24 * per))
    assert csd.csa_read_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("amax", [7.0, 6.5, 448.0, 0.0546875, 5.1875])
def test_e4m3_codes_of_16_bit_inputs_are_those_of_the_exact_quotients(cuda_lib, dtype, amax):
    """Values of few bits, many of whose quotients 448 y / amax are halfway points of
    the codes (a double holds those exactly, and its rounding of the others moves
    none across one): records, indexer keys and queries, not normalised."""
    csd = cuda_lib
    g = torch.Generator().manual_seed(int(amax * 64))
    unit = 2.0 ** np.floor(np.log2(amax) - 6)

    def values(*shape):
        x = torch.randint(-int(amax / unit), int(amax / unit) + 1, shape, generator=g).double() * unit
        x[..., 0] = amax
        for d in range(128, shape[-1], 128):  # the maximum of every 128-dim block
            x[..., d] = -amax
        return x.to(dtype)

    def codes_of(x):
        v = x.double().numpy() * 448 / amax
        return R.signed(R.nearest_code(v, R.E4M3), v, None, 128)

    x, key = values(2, 9, 512), values(2, 9, 128)
    cache = torch.zeros((18, 592), dtype=torch.uint8, device="cuda")
    k_idx = torch.zeros((2, 9, 128), dtype=torch.uint8, device="cuda")
    k_scale = torch.zeros((2, 9), device="cuda")
    csd.csa_cache_append(csd.cache_desc(cache, 9, seq_stride=9), x.cuda(), torch.zeros(2, dtype=torch.int32, device="cuda"),
                         rope_theta=None, key=key.cuda(), k_idx=k_idx, k_idx_scale=k_scale)
    assert np.array_equal(cache.cpu().numpy().reshape(2, 9, 592)[..., :448], codes_of(x)[..., :448])
    assert np.array_equal(k_idx.cpu().numpy(), codes_of(key))
    assert torch.all(k_scale.cpu() == np.float32(amax / 448))
    q = values(3, 5, 7, 128)
    codes, scale = csd.csa_head_norm_rope_e4m3(q.cuda(), torch.zeros((3, 5), dtype=torch.int32, device="cuda"), norm=False,
                                               rope_dim=0)
    assert np.array_equal(codes.cpu().numpy(), codes_of(q)) and torch.all(scale.cpu() == np.float32(amax / 448))
    assert csd.csa_read_device_error() == 0


def test_offsets_past_32_bits(cuda_lib):
    """A record beyond 4 GiB of the pool is written and read at its own place."""
    csd = cuda_lib
    n = (1 << 32) // 384 + 70000
    pool = torch.zeros((n, 384), dtype=torch.uint8, device="cuda")
    d = csd.cache_desc(pool, n, seq_stride=n, fmt=csd.FORMAT_FP4)
    x = torch.randn((1, 3, 512), device="cuda").to(torch.bfloat16)
    first = torch.tensor([n - 3], dtype=torch.int32, device="cuda")
    csd.csa_cache_append(d, x, first)
    got = csd.csa_cache_read(d, first, None, 3)
    small = torch.zeros((3, 384), dtype=torch.uint8, device="cuda")
    ds = csd.cache_desc(small, 3, fmt=csd.FORMAT_FP4)
    csd.csa_cache_append(ds, x, torch.zeros(1, dtype=torch.int32, device="cuda"), rope_theta=None)
    assert torch.equal(pool[-3:, :224], small[:, :224])
    assert torch.equal(pool[-3:, 352:], small[:, 352:])
    assert pool[:-3].count_nonzero() == 0
    assert got.float().abs().max() > 0 and csd.csa_read_device_error() == 0


def test_other_stream_and_graph_replay(cuda_lib):
    """The three calls on a stream of their own, captured and replayed on changed
    inputs, equal to direct calls."""
    csd = cuda_lib
    B, T = 2, 3
    x = torch.randn((B, T, 512), device="cuda").to(torch.bfloat16)
    q = torch.randn((B, T, 64, 128), device="cuda").to(torch.bfloat16)
    pos = torch.arange(B * T, device="cuda", dtype=torch.int32).view(B, T)
    first = torch.tensor([1, 4], dtype=torch.int32, device="cuda")
    pool = torch.zeros((2 * 16, 384), dtype=torch.uint8, device="cuda")
    d = csd.cache_desc(pool, 16, seq_stride=16, fmt=csd.FORMAT_FP4)
    codes, scale = csd.csa_head_norm_rope_e4m3(q, pos)
    out = torch.zeros((B, T, 512), dtype=torch.bfloat16, device="cuda")

    def step():
        csd.csa_head_norm_rope(x[:, :, None], pos, out=lat)
        csd.csa_cache_append(d, lat[:, :, 0], first, ring=True)
        csd.csa_cache_read(d, first, None, T, ring=True, out=out)
        csd.csa_head_norm_rope_e4m3(q, pos, codes=codes, scale=scale)

    lat = torch.empty((B, T, 1, 512), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    x.copy_(torch.randn((B, T, 512), device="cuda"))
    q.copy_(torch.randn((B, T, 64, 128), device="cuda"))
    pool.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (pool, out, codes, scale)]
    pool.zero_()
    step()
    torch.cuda.synchronize()
    for a, b in zip(got, (pool, out, codes, scale)):
        assert torch.equal(a, b)
    assert csd.csa_read_device_error() == 0


def test_outputs_made_for_a_named_stream(cuda_lib):
    """A call given a stream makes its output in that stream's order: the zeros
    behind a count, and nothing that the current stream still uses."""
    csd = cuda_lib
    pool = R.random_fp4_records(64, 3).cuda()
    cache = csd.cache_desc(pool, 64, seq_stride=64, fmt=csd.FORMAT_FP4)
    first = torch.tensor([0], dtype=torch.int32, device="cuda")
    count = torch.tensor([40], dtype=torch.int32, device="cuda")
    want = csd.csa_cache_read(cache, first, count, 64)
    x = torch.randn((1, 64, 4, 512), device="cuda")
    pos = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 64)
    want2, want3 = csd.csa_head_norm_rope(x, pos), csd.csa_head_norm_rope_e4m3(x, pos)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream):
        torch.full((64 << 20,), 7, device="cuda")  # freed at once, still being written
        got = csd.csa_cache_read(cache, first, count, 64, stream=s)
        got2, got3 = csd.csa_head_norm_rope(x, pos, stream=s), csd.csa_head_norm_rope_e4m3(x, pos, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.all(got[0, 40:] == 0) and torch.equal(got2, want2)
        assert torch.equal(got3[0], want3[0]) and torch.equal(got3[1], want3[1])
    assert csd.csa_read_device_error() == 0


def test_descriptions_that_do_not_fit_the_call_are_refused(cuda_lib):
    csd = cuda_lib
    pool = torch.zeros((4, 2, 384), dtype=torch.uint8, device="cuda")
    table = torch.arange(2, dtype=torch.int32, device="cuda").view(2, 1)
    first = torch.zeros(3, dtype=torch.int32, device="cuda")
    x = torch.zeros((3, 1, 512), dtype=torch.bfloat16, device="cuda")
    two = csd.cache_desc(pool, 4, block_table=table, page_records=4, fmt=csd.FORMAT_FP4)
    for call in (lambda: csd.csa_cache_append(two, x, first), lambda: csd.csa_cache_read(two, first, None, 1)):
        with pytest.raises(ValueError, match="2 rows for 3 sequences"):
            call()
    copy = csd.cache_desc(pool.transpose(0, 1), 4, seq_stride=4, fmt=csd.FORMAT_FP4)
    with pytest.raises(ValueError, match="not contiguous"):
        csd.csa_cache_append(copy, x[:1], first[:1])
    with pytest.raises(ValueError, match="go together"):
        csd.csa_cache_append(two, x[:2], first[:2], key=x[:2, :, :128])
    with pytest.raises(ValueError, match="status"):
        csd.csa_cache_append(two, x[:2], first[:2], status=torch.zeros(1, device="cuda"))
    assert csd.csa_read_device_error() == 0
