"""Calls large enough that a warp takes several tokens, records or heads one after
the other, against the same data sent in calls small enough for one each: every
byte has to be equal (an item's arithmetic does not depend on its neighbours), and
so have the places that no item writes. The small calls are tested against 64 bits
elsewhere. Tokens that do not count hold NaN."""
import pytest
import torch

import _records as R

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
WARPS = 4  # of a block: 128 threads, of which eight an SM are wanted before a warp takes a second item


def sm_count():
    return torch.cuda.get_device_properties(0).multi_processor_count


def pieces(B, items, most):
    """Ranges of sequences with fewer than `most` items (multiples of four, so that
    every slice starts on 16 bytes)."""
    n = max(4, (most - 1) // items // 4 * 4)
    assert n * items < most
    return [(b, min(B, b + n)) for b in range(0, B, n)]


def same(a, b, what):
    a, b = a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)
    assert torch.equal(a, b), f"{what}: {int((a != b).sum())} bytes differ"


class Tokens:
    """B x T tokens of which count[b] count, for a cache of `cap` entries a sequence,
    into which some sequences' last entries do not fit."""

    def __init__(self, csd, B, T, cap, dtype, fmt, paged, ring, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.csd, self.B, self.T, self.cap, self.fmt, self.ring = csd, B, T, cap, fmt, ring
        self.x = (torch.randn((B, T, 512), generator=g, device="cuda") *
                  torch.exp(2 * torch.randn((B, T, 1), generator=g, device="cuda"))).to(dtype)
        self.key = torch.randn((B, T, 128), generator=g, device="cuda").to(dtype)
        self.first = torch.randint(0, max(1, cap - T) + 2, (B,), generator=g, device="cuda", dtype=torch.int32)
        self.count = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        self.count[::3] = T
        self.first[0] = max(0, cap - T + 1)
        dead = torch.arange(T, device="cuda")[None] >= self.count[:, None]
        self.x[dead] = float("nan")
        self.key[dead] = float("nan")
        self.weight = 1 + 0.1 * torch.randn(512, generator=g, device="cuda")
        self.page = 4
        self.pages = -(-cap // self.page)
        self.table = (torch.randperm(B * self.pages, generator=g, device="cuda").to(torch.int32).view(B, self.pages)
                      if paged else None)
        size = csd.FORMAT_BYTES[fmt]
        self.shape = (B * self.pages * self.page if paged else B * cap, size)

    def desc(self, pool, b0, b1):
        if self.table is not None:
            return self.csd.cache_desc(pool, self.cap, block_table=self.table[b0:b1].clone(), page_records=self.page,
                                       fmt=self.fmt)
        return self.csd.cache_desc(pool[b0 * self.cap:b1 * self.cap], self.cap, seq_stride=self.cap, fmt=self.fmt)

    def append(self, ranges, norm, keys):
        pool = torch.full(self.shape, 0xAB, dtype=torch.uint8, device="cuda")
        k_idx = torch.full((self.B, self.cap, 128), 0xCD, dtype=torch.uint8, device="cuda")
        k_scale = torch.full((self.B, self.cap), -3.0, device="cuda")
        for b0, b1 in ranges:
            kw = dict(key=self.key[b0:b1], k_idx=k_idx[b0:b1], k_idx_scale=k_scale[b0:b1]) if keys else {}
            self.csd.csa_cache_append(self.desc(pool, b0, b1), self.x[b0:b1], self.first[b0:b1].clone(),
                                      self.count[b0:b1].clone(), ring=self.ring, norm=norm,
                                      weight=self.weight if norm else None, pos_stride=3, **kw)
        return pool, k_idx, k_scale

    def read(self, pool, ranges):
        out = torch.full((self.B, self.T, 512), 9.0, dtype=torch.bfloat16, device="cuda")
        for b0, b1 in ranges:
            self.csd.csa_cache_read(self.desc(pool, b0, b1), self.first[b0:b1].clone(), self.count[b0:b1].clone(),
                                    self.T, ring=self.ring, out=out[b0:b1])
        return out


# tokens a warp, tokens a sequence, capacity of a sequence, paged, ring
SHAPES = [(2, 5, 9, True, False), (3, 1009, 1020, False, False), (5, 1, 3, False, False), (8, 13, 14, True, False),
          (8, 401, 500, True, False), (7, 23, 16, False, True), (3, 2, 40, False, True)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_append_and_read_of_many_tokens(cuda_lib, shape, fmt, dtype):
    csd = cuda_lib
    per_warp, T, cap, paged, ring = shape
    unit = sm_count() * 8 * WARPS  # tokens at one a warp
    B = -(-(per_warp * unit + unit // 3) // T)
    if B * T % per_warp == 0:  # the last warp is to have fewer
        B += 1
    assert B * T // unit == per_warp and B * T % per_warp
    c = Tokens(csd, B, T, cap, dtype, fmt, paged, ring, seed=T + 10 * fmt)
    ranges = pieces(B, T, 2 * unit)
    assert len(ranges) > 1
    for norm in (False, True):
        for keys in ((False,) if ring else (False, True)):
            whole, parts = c.append([(0, B)], norm, keys), c.append(ranges, norm, keys)
            for a, b, what in zip(whole, parts, ("records", "key codes", "key scales")):
                same(a, b, f"{what}, norm {norm}, keys {keys}")
            if not keys:
                assert torch.all(whole[1] == 0xCD) and torch.all(whole[2] == -3)
        same(c.read(whole[0], [(0, B)]), c.read(whole[0], ranges), "read back")
    code = csd.csa_read_device_error()
    assert code == (0 if ring else csd.ERR_BAD_INDEX)
    # a sample of the rows against 64 bits: the whole chain of one sequence's first token
    live = torch.nonzero((c.count > 0) & (ring | (c.first < cap))).view(-1).cpu()[::max(1, B // 5)]
    back = c.read(whole[0], [(0, B)]).double().cpu().numpy()
    csd.csa_read_device_error()
    for b in live.tolist():
        t = max(0, int(c.count[b]) - cap) if ring else 0
        y = R.norm_rope(c.x[b, t:t + 1].double().cpu().numpy(), [(int(c.first[b]) + t) * 3],
                        c.weight.double().cpu().numpy(), 1e-6, 64, 10000.0)[0]
        # (formats' own steps: half of 2^-3 of the value and of the smallest step, in 4 bits
        # of an eighth of the block's maximum; the exact bounds are the small calls' tests')
        blocks = abs(y[:448]).reshape(-1, 16 if fmt else 64).max(-1).repeat(16 if fmt else 64)
        assert (abs(back[b, t, :448] - y[:448]) <= (0.25 if fmt else 0.08) * blocks + 2e-3 * abs(y[:448]).max()).all()
        assert (abs(back[b, t, 448:] - y[448:]) <= 2.0 ** -8 * abs(y[448:]) + 1e-5 * abs(y[448:]).max()).all()


# D, H, tokens a sequence, heads a group (16 at most), rope_dim
HEADS = [(512, 1, 7, 2, 64), (512, 37, 3, 3, 64), (512, 128, 11, 16, 64), (504, 2, 5, 16, 128), (256, 3, 9, 7, 256),
         (128, 64, 4, 5, 64), (128, 1, 1, 16, 128), (64, 1, 33, 16, 64), (72, 37, 6, 4, 0), (8, 5, 13, 2, 8)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("shape", HEADS, ids=str)
def test_norm_and_rotation_of_many_heads(cuda_lib, shape, dtype):
    csd = cuda_lib
    D, H, T, per_group, rope = shape
    groups = 4 if D > 128 else 8 if D > 64 else 16  # heads that a block of 128 threads holds at once
    unit = groups * 8 * sm_count()
    B = -(-(per_group * unit + unit // 3) // (T * H))
    if B * T * H % (per_group * groups) == 0:
        B += 1
    g = torch.Generator(device="cuda").manual_seed(D + H + T)
    wide = torch.randn((B, T, H * D + 64), generator=g, device="cuda", dtype=torch.float32).to(dtype)
    x = wide[..., :H * D].unflatten(-1, (H, D))
    pos = torch.randint(0, 1 << 20, (B, T), generator=g, device="cuda", dtype=torch.int32)
    dead = torch.rand((B, T), generator=g, device="cuda") < 0.3
    pos[dead] = -1
    x[dead] = float("nan")
    w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    ranges = pieces(B, T * H, 2 * unit)
    assert len(ranges) > 1 and B * T * H // unit >= per_group
    for norm in (True, False):
        kw = dict(weight=w if norm else None, norm=norm, rope_dim=rope)

        def run(ranges):
            out = torch.full((B, T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
            codes = torch.full((B, T, H, D), 99, dtype=torch.uint8, device="cuda")
            scale = torch.full((B, T, H), 5.0, device="cuda")
            for b0, b1 in ranges:
                p = pos[b0:b1].clone()
                csd.csa_head_norm_rope(x[b0:b1], p, out=out[b0:b1], **kw)
                csd.csa_head_norm_rope_e4m3(x[b0:b1], p, codes=codes[b0:b1], scale=scale[b0:b1], **kw)
            return out, codes, scale

        whole, parts = run([(0, B)]), run(ranges)
        for a, b, what in zip(whole, parts, ("BF16", "codes", "scales")):
            same(a, b, f"{what}, norm {norm}")
        out, codes, scale = whole
        assert torch.all(out[dead] == 7) and torch.all(codes[dead] == 99) and torch.all(scale[dead] == 5)
        assert not torch.isnan(out).any() and torch.all(scale > 0)
    # a sample against 64 bits (norm of the last pass: none; its rotation in 64 bits)
    b = B - 1
    y = R.norm_rope(torch.nan_to_num(x[b]).double().cpu().numpy(), pos[b].clamp_min(0).cpu().numpy(), None, 0, rope, 10000.0)
    alive = ~dead[b].cpu().numpy()
    assert (abs(out[b].double().cpu().numpy() - y)[alive] <= 2.0 ** -8 * abs(y[alive]) + 1e-5 * abs(y[alive]).max(initial=0)).all()
    assert csd.csa_read_device_error() == 0
