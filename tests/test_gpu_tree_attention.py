"""Attention of a tree's drafted tokens against its definition in 64 bits.

Bounds (derived before the first run), for head h, output dim d, with A_d =
sum_j p_j |x_jd| / den:
* scores: q is exact, 4-bit latents are exact in BF16, FP8 latents go in as their BF16
  value and the BF16 value of the rest, off by at most 2^-8 2^-8 of them; fp32
  accumulation of 512 (or 1024) products with a wide margin for the tensor core's
  alignment 2^-15: each score moves by at most B = (2^-15 + 2^-16) scale max_j sum_d
  |q_d x_jd|, each weight by e^{2B} - 1;
* the weights are rounded to BF16 (2^-8 of each), the latents that they multiply too
  (FP8 only, 2^-8 of each), and the output (2^-8 |o_d|);
* the partial outputs of a split are rounded to FP16 (2^-11 of each) in units of a
  power of two for 32 dims (2^-39 of the largest of them);
* fp32 exponentials and sums: below 1e-5.
So |err_d| <= A_d (3 2^-8 + 3 B + 1e-5) + 2^-39 G_d + 2^-8 |o_d|, for rotated dims with
A and |o| summed over the pair (+ 1e-6 of them for sine and cosine), and
|lse err| <= B + 1e-5 (1 + |lse|).
"""
import numpy as np
import pytest
import torch

import _speculative as S

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8


class Tree:
    """Random caches, drafts and positions of trees."""

    def __init__(self, csd, B, N, cap, kind, fmt, W=128, R=None, paged=True, page=32, seed=0, ctx=None, padded=False):
        g = torch.Generator().manual_seed(seed)
        self.csd, self.B, self.N, self.cap, self.W, self.fmt = csd, B, N, cap, W, fmt
        self.R = R or W
        self.bytes = csd.FORMAT_BYTES[fmt]
        pages = -(-cap // page)
        self.paged, self.page = paged, page
        self.pool = S.random_records(B * pages * page if paged else B * cap, fmt, seed + 1)
        self.ring = S.random_records(B * self.R, fmt, seed + 2).view(B, self.R, self.bytes)
        self.draft = S.random_records(B * N, fmt, seed + 3).view(B, N, self.bytes)
        self.table = torch.randperm(B * pages, generator=g).to(torch.int32).view(B, pages) if paged else None
        self.q = torch.randn((B, N, 128, 512), generator=g).to(torch.bfloat16)
        self.sink = torch.randn(128, generator=g)
        self.parent = S.random_tree(kind, B, N, g)
        self.ctx = torch.randint(0, 3 * cap + 2 * W, (B, 1), generator=g).int() if ctx is None else \
            torch.tensor(ctx, dtype=torch.int32).view(B, 1)
        self.pos = (self.ctx + S.depths(self.parent)).to(torch.int32)
        if padded:
            live = torch.randint(0, N + 1, (B, 1), generator=g)
            self.pos = torch.where(torch.arange(N)[None] < live, self.pos, -1).to(torch.int32)
        self.gen = g

    def where(self, b, e):
        e = np.asarray(e, dtype=np.int64)
        if not self.paged:
            return b * self.cap + e
        return self.table[b].numpy()[e // self.page].astype(np.int64) * self.page + e % self.page

    def select(self, k):
        """Random counts of distinct entries in ascending order, -1 behind them."""
        cnt = torch.randint(0, min(k, self.cap) + 1, (self.B, self.N), generator=self.gen).to(torch.int32)
        cnt[0, 0] = min(k, self.cap)
        idx = torch.full((self.B, self.N, k), -1, dtype=torch.int32)
        for b in range(self.B):
            for i in range(self.N):
                c = int(cnt[b, i])
                idx[b, i, :c] = torch.randperm(self.cap, generator=self.gen)[:c].sort().values.to(torch.int32)
        return idx, cnt

    def cache(self):
        self.d_pool = self.pool.cuda()
        return self.csd.cache_desc(self.d_pool, self.cap, seq_stride=0 if self.paged else self.cap,
                                   block_table=self.table.cuda() if self.paged else None,
                                   page_records=self.page if self.paged else 0, fmt=self.fmt)

    def csa(self, idx, cnt, **kw):
        r = self.csd.csa_tree_attention_decode(self.q.cuda(), self.sink.cuda(), S.SCALE, self.cache(), self.ring.cuda(),
                                               self.W, self.draft.cuda(), self.parent.cuda(), idx.cuda(), cnt.cuda(),
                                               self.pos.cuda(), **kw)
        torch.cuda.synchronize()
        return r

    def hca(self, n_comp, m, **kw):
        r = self.csd.hca_tree_attention_decode(self.q.cuda(), self.sink.cuda(), S.SCALE, self.cache(), n_comp.cuda(),
                                               self.ring.cuda(), self.W, self.draft.cuda(), self.parent.cuda(),
                                               self.pos.cuda(), m, **kw)
        torch.cuda.synchronize()
        return r

    def reference(self, b, i, entries, theta=None):
        """(o, lse, bound of o, bound of lse) of token i of sequence b."""
        p = int(self.pos[b, i])
        x = np.concatenate([
            S.values(self.pool.numpy()[self.where(b, entries)].reshape(-1, self.bytes), self.fmt),
            S.window(self.ring[b].numpy(), self.draft[b].numpy(), self.parent[b], i, p, self.W, self.fmt)])
        o, lse, A, size = S.attend(self.q[b, i].double().numpy(), self.sink.double().numpy(), x)
        Bz = (2.0 ** -15 + 2.0 ** -16) * size
        G = np.repeat(A.reshape(128, 16, 32).max(-1), 32, axis=-1)
        bound = A * (3 * BF + 3 * Bz[:, None] + 1e-5) + 2.0 ** -39 * G + BF * np.abs(o)
        if theta:
            s = bound[:, 448::2] + bound[:, 449::2] + 1e-6 * (A[:, 448::2] + A[:, 449::2])
            s = s + BF * (np.abs(o[:, 448::2]) + np.abs(o[:, 449::2]))
            bound = bound.copy()
            bound[:, 448::2] = bound[:, 449::2] = s
            o = S.turn_back(o, p, theta)
        return o, lse, bound, Bz + 1e-5 * (1 + np.abs(lse))

    def check(self, got, entries, theta=None, what="", rows=None):
        out, lse = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
        for b in range(self.B):
            for i in range(self.N):
                if int(self.pos[b, i]) < 0 or (rows is not None and (b, i) not in rows):
                    continue
                o, l, bound, lbound = self.reference(b, i, entries(b, i), theta)
                assert np.all(np.isfinite(out[b, i])), f"{what} {b},{i}"
                err = np.abs(out[b, i] - o)
                assert np.all(err <= bound + 1e-30), f"{what} {b},{i}: {np.max(err / (bound + 1e-30)):.3g} x bound"
                le = np.abs(lse[b, i] - l)
                assert np.all(le <= lbound), f"{what} {b},{i}: lse {le.max():.3g}"


def outputs(B, N, fill=7.0):
    return (torch.full((B, N, 128, 512), fill, dtype=torch.bfloat16, device="cuda"),
            torch.full((B, N, 128), fill, device="cuda"))


CSA = [  # B, N, cap, k, kind, W, R, paged, ctx
    (1, 1, 5, 1, "chain", 1, 1, False, None), (1, 8, 70, 64, "random", 128, 128, True, None),
    (2, 5, 300, 130, "forest", 128, 140, True, None), (3, 3, 900, 517, "star", 128, 128, False, None),
    (1, 2, 2100, 2048, "chain", 512, 600, True, None), (9, 13, 260, 200, "random", 128, 135, True, None),
    (2, 40, 64, 33, "random", 7, 9, True, None), (1, 128, 40, 16, "chain", 128, 128, True, [300]),
    (1, 128, 40, 16, "chain", 512, 512, False, [17]), (1, 128, 40, 16, "random", 5, 5, True, [0]),
    (3, 6, 40, 8, "random", 128, 128, True, [0, 1, 127]),
]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("case", CSA)
def test_tree_csa(cuda_lib, case, fmt):
    B, N, cap, k, kind, W, R, paged, ctx = case
    c = Tree(cuda_lib, B, N, cap, kind, fmt, W=W, R=R, paged=paged, ctx=ctx, seed=B * 100 + N)
    idx, cnt = c.select(k)
    theta = 10000.0 if N % 2 else None
    got = c.csa(idx, cnt, inverse_rope=theta is not None)
    assert cuda_lib.csa_read_device_error() == 0
    c.check(got, lambda b, i: idx[b, i, :int(cnt[b, i])].numpy(), theta, f"{case}")


HCA = [  # B, N, cap, m, kind, paged, ctx
    (1, 1, 1, 128, "chain", False, [0]), (1, 16, 900, 4, "random", True, None), (5, 7, 300, 128, "forest", True, None),
    (2, 3, 5000, 1, "chain", False, [4999, 9000]), (40, 2, 64, 3, "chain", True, None),
]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("case", HCA)
def test_tree_hca(cuda_lib, case, fmt):
    B, N, cap, m, kind, paged, ctx = case
    c = Tree(cuda_lib, B, N, cap, kind, fmt, paged=paged, ctx=ctx, seed=B * 10 + N, page=1 if paged else 32)
    n_comp = torch.randint(0, cap + 1, (B,), generator=c.gen).to(torch.int32)
    n_comp[0] = cap
    got = c.hca(n_comp, m, inverse_rope=True, rope_theta=1e6)
    assert cuda_lib.csa_read_device_error() == 0
    c.check(got, lambda b, i: np.arange(min(int(c.pos[b, i]) // m, int(n_comp[b]), cap)), 1e6, f"{case}")


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("B, N", [(1, 9), (2, 12), (30, 5)])  # many splits, a few, one
def test_padding_keeps_its_rows(cuda_lib, fmt, B, N):
    c = Tree(cuda_lib, B, N, 700, "random", fmt, padded=True, seed=3)
    c.pos[0, N // 2:] = -1
    idx, cnt = c.select(600)
    pad = c.pos < 0
    for hca in (False, True):
        out, lse = outputs(B, N)
        n_comp = torch.full((B,), 700, dtype=torch.int32)
        got = c.hca(n_comp, 2, out=out, lse=lse) if hca else c.csa(idx, cnt, out=out, lse=lse)
        assert bool((got[0].cpu()[pad] == 7).all()) and bool((got[1].cpu()[pad] == 7).all())
        rows = [(b, i) for b in range(min(B, 2)) for i in range(N)]
        c.check(got, (lambda b, i: np.arange(min(int(c.pos[b, i]) // 2, 700))) if hca else
                (lambda b, i: idx[b, i, :int(cnt[b, i])].numpy()), rows=rows)
    codes = torch.full((B, N, 128, 256), 0x5A, dtype=torch.uint8, device="cuda")
    scale = torch.full((B, N, 128, 4), 7.0, device="cuda")
    c.csa(idx, cnt, fp4_out=True, out_fp4=codes, out_fp4_scale=scale)
    assert bool((codes.cpu()[pad] == 0x5A).all()) and bool((scale.cpu()[pad] == 7).all())


def test_a_batch_of_padding_alone(cuda_lib):
    for fmt in (0, 1):
        c = Tree(cuda_lib, 2, 3, 50, "chain", fmt, seed=4)
        c.pos.fill_(-1)
        idx, cnt = c.select(20)
        out, lse = outputs(2, 3)
        c.csa(idx, cnt, out=out, lse=lse)
        assert bool((out == 7).all()) and bool((lse == 7).all()) and cuda_lib.csa_read_device_error() == 0


def test_a_chain_is_the_same_step_without_a_tree(cuda_lib):
    """Bit for bit the ordinary call whose ring holds the drafts (4-bit records; of so many queries that neither call
    splits one)."""
    csd, B, N = cuda_lib, 80, 4
    c = Tree(csd, B, N, 60, "chain", 1, R=140, seed=5)
    idx, cnt = c.select(50)
    got = c.csa(idx, cnt, inverse_rope=True)
    ring = c.ring.clone()
    for b in range(B):
        for i in range(N):
            ring[b, int(c.pos[b, i]) % 140] = c.draft[b, i]
    want = csd.csa_sink_attention_decode_fp4(c.q.cuda(), c.sink.cuda(), S.SCALE, c.cache(), ring.cuda(), c.W, idx.cuda(),
                                             cnt.cuda(), c.pos.cuda(), inverse_rope=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("B, N, live", [(19, 2, 2), (13, 3, 1), (1, 2, 1), (4, 9, 8), (3, 13, 13), (19, 4, 4), (11, 7, 5), (38, 4, 2), (3, 100, 9)])
def test_queries_of_very_different_lengths(cuda_lib, fmt, B, N, live):
    """One long query among short ones and padding: fewer and more queries than half of the CTA pairs, than all
    and twice as many."""
    c = Tree(cuda_lib, B, N, 2200, "random", fmt, seed=B, padded=False)
    c.pos[:, live:] = -1
    idx, cnt = c.select(2000)
    cnt[:, :] = torch.randint(0, 40, cnt.shape, generator=c.gen).to(torch.int32)
    cnt[0, 0], cnt[B // 2, 0] = 2000, 700
    for b in range(B):
        for i in range(N):
            idx[b, i, :int(cnt[b, i])] = torch.arange(int(cnt[b, i]), dtype=torch.int32) + b % 7
    out, lse = outputs(B, N)
    got = c.csa(idx, cnt, out=out, lse=lse, inverse_rope=True)
    rows = {(0, 0), (B // 2, 0), (B - 1, live - 1)} | {(b, (b * 3) % live) for b in range(0, B, 5)}
    c.check(got, lambda b, i: idx[b, i, :int(cnt[b, i])].numpy(), 10000.0, rows=rows)
    assert bool((got[0].cpu()[c.pos < 0] == 7).all()) and bool(torch.isfinite(got[0].float()).all())
    assert cuda_lib.csa_read_device_error() == 0


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("B, N, long", [(100, 1, 16400), (40, 1, 9000), (150, 2, 4000), (304, 1, 4000), (305, 1, 4000)])
def test_hca_queries_of_very_different_lengths(cuda_lib, fmt, B, N, long):
    """A query of up to 130 blocks among short ones, more queries than half of the pairs up to the most that are dealt
    out, and one more; all sequences' tables lead to the same pages."""
    cap, page = long + 100, 32
    c = Tree(cuda_lib, B, N, 32, "chain", fmt, seed=B, page=page)
    pages = -(-cap // page)
    c.cap, c.pool = cap, S.random_records(pages * page, fmt, 77)
    c.table = torch.randperm(pages, generator=c.gen).to(torch.int32).repeat(B, 1).contiguous()
    n_comp = torch.randint(0, 6, (B,), generator=c.gen).to(torch.int32)
    n_comp[B // 3], n_comp[B - 1] = long, long // 2
    c.pos += long - int(c.pos.min())
    got = c.hca(n_comp, 1, inverse_rope=True)
    assert cuda_lib.csa_read_device_error() == 0 and bool(torch.isfinite(got[0].float()).all())
    rows = {(b, N - 1) for b in (0, B // 3, B // 2, B - 1)}
    c.check(got, lambda b, i: np.arange(int(n_comp[b])), 10000.0, rows=rows)


@pytest.mark.parametrize("fmt", [0, 1])
def test_only_ancestors_and_committed_tokens_are_read(cuda_lib, fmt):
    """Latents that are NaN in every place that no token may look at."""
    csd, B, N, W = cuda_lib, 2, 10, 16
    c = Tree(csd, B, N, 60, "random", fmt, W=W, R=40, seed=6, ctx=[100, 37])
    idx, cnt = c.select(30)
    clean = c.csa(idx, cnt)
    nan = S.random_records(1, fmt, 9)[0]
    nan[-176 if fmt == 0 else 224:] = 0xFF
    nan[:224] = 0x7F if fmt == 0 else 0x77
    for b in range(B):  # ring: all but the W - 1 committed positions before the tree
        keep = {pos % 40 for pos in range(max(0, int(c.ctx[b]) - W + 1), int(c.ctx[b]))}
        for r in range(40):
            if r not in keep:
                c.ring[b, r] = nan
    used = {(b, int(e)) for b in range(B) for i in range(N) for e in c.where(b, idx[b, i, :int(cnt[b, i])].numpy())}
    for b in range(B):
        mine = {e for bb, e in used if bb == b}
        for e in c.where(b, np.arange(60)):
            if int(e) not in mine:
                c.pool[int(e)] = nan
    again = c.csa(idx, cnt)
    assert torch.equal(clean[0], again[0]) and torch.equal(clean[1], again[1])
    # a draft reaches itself and what follows it, and no other token
    c.draft[0, 3] = nan
    bad = c.csa(idx, cnt)
    for i in range(N):
        hit = 3 in S.chain_of(c.parent[0], i) and int(c.pos[0, i]) - int(c.pos[0, 3]) < W
        assert bool(torch.isnan(bad[0][0, i]).any()) == hit, i
        if not hit:
            assert torch.equal(bad[0][0, i], clean[0][0, i])
    assert torch.equal(bad[0][1], clean[0][1])


def test_bad_parents_are_reported_and_taken_as_none(cuda_lib):
    csd = cuda_lib
    c = Tree(csd, 1, 6, 60, "chain", 1, seed=7, ctx=[50])
    c.parent[0] = torch.tensor([-1, 0, 2, -5, 9, 1])  # token 2 its own parent, 3 and 4 out of range
    c.pos[0] = torch.tensor([50, 51, 50, 50, 50, 52])
    idx, cnt = c.select(20)
    got = c.csa(idx, cnt)
    assert csd.csa_read_device_error() == csd.ERR_BAD_INDEX
    c.check(got, lambda b, i: idx[b, i, :int(cnt[b, i])].numpy())
    c.parent[0] = torch.tensor([7, 0, 1, 2, 3, 4])  # of a token that is nobody's ancestor but its own
    c.pos[0] = 50 + torch.arange(6)
    got = c.csa(idx, cnt)
    assert csd.csa_read_device_error() == csd.ERR_BAD_INDEX
    c.check(got, lambda b, i: idx[b, i, :int(cnt[b, i])].numpy())


def test_entries_outside_the_cache_are_reported(cuda_lib):
    csd = cuda_lib
    for fmt in (0, 1):
        c = Tree(csd, 1, 3, 60, "chain", fmt, seed=8)
        idx, cnt = c.select(20)
        idx[0, 1, 0], cnt[0, 1] = 60, 5
        idx[0, 1, 1:5] = torch.tensor([1, 2, 3, 4], dtype=torch.int32)
        got = c.csa(idx, cnt)
        assert csd.csa_read_device_error() == csd.ERR_BAD_INDEX
        c.check(got, lambda b, i: [e for e in idx[b, i, :int(cnt[b, i])].tolist() if 0 <= e < 60])


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("B", [1, 39])
def test_e2m1_output(cuda_lib, fmt, B):
    """Codes within half a step (at most 1, in units of the multiplier) of a value within the bound."""
    c = Tree(cuda_lib, B, 2, 80, "chain", fmt, seed=11)
    idx, cnt = c.select(40)
    (codes, scale), lse = c.csa(idx, cnt, inverse_rope=True, fp4_out=True)
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    code = codes.cpu().numpy()
    code = np.stack([code & 15, code >> 4], -1).reshape(B, 2, 128, 512)
    step = np.repeat(scale.double().cpu().numpy(), 128, axis=-1)
    val = np.where(code >= 8, -1.0, 1.0) * grid[code & 7] * step
    for b in {0, B - 1}:
        for i in range(2):
            o, l, bound, lbound = c.reference(b, i, idx[b, i, :int(cnt[b, i])].numpy(), 10000.0)
            assert np.all(np.abs(val[b, i] - o) <= bound + step[b, i] * (1 + 1e-3))
            assert np.all(np.abs(lse[b, i].double().cpu().numpy() - l) <= lbound)


@pytest.mark.parametrize("fmt", [0, 1])
def test_offsets_past_32_bits(cuda_lib, fmt):
    """Pages whose records begin more than 2^32 bytes into the pool."""
    csd, cap, page = cuda_lib, 64, 32
    size = csd.FORMAT_BYTES[fmt]
    pages = (1 << 32) // (size * page) + 40
    pool = torch.zeros((pages * page, size), dtype=torch.uint8, device="cuda")
    rec = S.random_records(cap, fmt, 12)
    far = torch.tensor([[pages - 1, pages - 7]], dtype=torch.int32)
    for j in range(2):
        at = int(far[0, j]) * page
        pool[at:at + page] = rec[j * page:(j + 1) * page].cuda()
    c = Tree(csd, 1, 2, cap, "chain", fmt, seed=13, paged=False)
    c.pool = rec
    comp = csd.cache_desc(pool, cap, block_table=far.cuda(), page_records=page, fmt=fmt)
    idx, cnt = c.select(40)
    got = csd.csa_tree_attention_decode(c.q.cuda(), c.sink.cuda(), S.SCALE, comp, c.ring.cuda(), c.W, c.draft.cuda(),
                                        c.parent.cuda(), idx.cuda(), cnt.cuda(), c.pos.cuda())
    torch.cuda.synchronize()
    c.check(got, lambda b, i: idx[b, i, :int(cnt[b, i])].numpy())


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("B, N, cap", [(1, 1, 200), (2, 12, 2000)])  # many splits; two
def test_a_selected_nan_record_reaches_its_row_only(cuda_lib, fmt, B, N, cap):
    c = Tree(cuda_lib, B, N, cap, "random", fmt, seed=21)
    c.sink[3], c.sink[4] = -float("inf"), 80.0
    idx, cnt = c.select(min(cap, 1500))
    cnt[:, :] = idx.shape[2]
    for b in range(B):
        for i in range(N):
            idx[b, i] = torch.arange(idx.shape[2], dtype=torch.int32) + 1
    if idx.shape[2] >= cap:
        idx, cnt = idx[:, :, :cap - 1].contiguous(), cnt.clamp(max=cap - 1)
    clean = c.csa(idx, cnt)
    c.check(clean, lambda b, i: idx[b, i, :int(cnt[b, i])].numpy(), rows={(0, 0), (B - 1, N - 1)})
    rec = c.pool[int(c.where(B - 1, [0])[0])]
    rec[:] = 0xFF  # entry 0 of the last sequence: NaN in every place
    idx[B - 1, N - 1, 0] = 0
    got = c.csa(idx, cnt)
    assert bool(torch.isnan(got[0][B - 1, N - 1]).all()) and bool(torch.isnan(got[1][B - 1, N - 1]).all())
    keep = torch.ones((B, N), dtype=torch.bool)
    keep[B - 1, N - 1] = False
    keep = keep.cuda()
    assert torch.equal(got[0][keep], clean[0][keep]) and torch.equal(got[1][keep], clean[1][keep])


@pytest.mark.parametrize("fmt", [0, 1])
def test_dealt_out_queries_captured_and_replayed(cuda_lib, fmt):
    """Lengths that change between replays deal the queries out anew; two calls in one graph share a workspace."""
    csd, B, N, cap = cuda_lib, 4, 11, 4000
    c = Tree(csd, B, N, cap, "random", fmt, seed=22, page=1)
    c.pos = (4000 + S.depths(c.parent)).to(torch.int32)
    q, sink, ring, draft, parent, pos = (t.cuda() for t in (c.q, c.sink, c.ring, c.draft, c.parent, c.pos))
    comp = c.cache()
    n_comp = torch.tensor([4000, 10, 0, 2500], dtype=torch.int32, device="cuda")
    ws = csd.workspace(csd.OP_HCA_TREE_ATTENTION, B, N, cap, 0, "cuda")
    a, b = outputs(B, N), outputs(B, N)

    def calls(x, y):
        for o, l in (x, y):
            csd.hca_tree_attention_decode(q, sink, S.SCALE, comp, n_comp, ring, c.W, draft, parent, pos, 1, out=o, lse=l,
                                          ws=ws)

    calls(a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(a, b)
    for lengths, pad in (([4000, 10, 0, 2500], 0), ([3, 3999, 1200, 1], 5), ([0, 0, 0, 0], 0), ([4000] * 4, 11)):
        n_comp.copy_(torch.tensor(lengths, dtype=torch.int32))
        p = c.pos.clone()
        p[1, N - pad:] = -1
        pos.copy_(p)
        for t in (*a, *b):
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        assert bool((a[0].cpu()[p < 0] == 7).all()) and bool((a[1].cpu()[p < 0] == 7).all())
        keep, c.pos = c.pos, p
        c.check(a, lambda b_, i: np.arange(lengths[b_]), rows={(0, 0), (1, 0), (1, N - 1), (2, 5), (3, N - 1)})
        c.pos = keep
    assert csd.csa_read_device_error() == 0


@pytest.mark.parametrize("fmt", [0, 1])
def test_capture_replay_and_other_stream(cuda_lib, fmt):
    csd = cuda_lib
    c = Tree(csd, 2, 5, 400, "random", fmt, seed=14)
    idx, cnt = c.select(300)
    dev = [t.cuda() for t in (c.q, c.sink, c.ring, c.draft, c.parent, idx, cnt, c.pos)]
    q, sink, ring, draft, parent, didx, dcnt, pos = dev
    comp = c.cache()
    out, lse = outputs(2, 5)
    ws = csd.workspace(csd.OP_TREE_ATTENTION, 2, 5, 400, 300, "cuda")

    def call(o, l, stream=None):
        csd.csa_tree_attention_decode(q, sink, S.SCALE, comp, ring, c.W, draft, parent, didx, dcnt, pos, out=o, lse=l,
                                      ws=ws, stream=stream)

    call(out, lse)
    torch.cuda.synchronize()
    want = out.clone(), lse.clone()
    side = torch.cuda.Stream()
    o2, l2 = outputs(2, 5)
    side.wait_stream(torch.cuda.current_stream())
    call(o2, l2, side)
    side.synchronize()
    assert torch.equal(o2, want[0]) and torch.equal(l2, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, lse)
    q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(15)).to(torch.bfloat16))
    call(o2, l2)
    torch.cuda.synchronize()
    want = o2.clone(), l2.clone()
    for _ in range(2):
        out.fill_(3)
        lse.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("fmt", [0, 1])
def test_the_step_is_its_three_calls(cuda_lib, fmt):
    csd, B, N, cap, k, m = cuda_lib, 3, 7, 500, 130, 4
    c = Tree(csd, B, N, cap, "random", fmt, seed=16, ctx=[2100, 40, 900], padded=True)
    c.pos[0] = c.ctx[0] + S.depths(c.parent)[0]
    g = torch.Generator().manual_seed(17)
    q_idx = torch.randn((B, N, 64, 128), generator=g).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    k_idx = torch.randn((B, cap, 128), generator=g).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    qs, ks = torch.rand((B, N, 64), generator=g).cuda() + 0.1, torch.rand((B, cap), generator=g).cuda() + 0.1
    w = torch.randn((B, N, 64), generator=g).cuda()
    n_comp = torch.tensor([500, 10, 225], dtype=torch.int32, device="cuda")
    comp, pos = c.cache(), c.pos.cuda()
    rest = c.q.cuda(), c.sink.cuda(), S.SCALE, comp, c.ring.cuda(), c.W, c.draft.cuda(), c.parent.cuda()
    out, lse = outputs(B, N)
    ti = torch.empty((B, N, k), dtype=torch.int32, device="cuda")
    tc = torch.empty((B, N), dtype=torch.int32, device="cuda")
    csd.csa_tree_decode_step(q_idx, qs, w, k_idx, ks, *rest, pos, n_comp, m, k, out=out, lse=lse, topk_idx=ti, topk_cnt=tc,
                             inverse_rope=True)
    logits = csd.csa_indexer_logits(q_idx, qs, w, k_idx, ks, pos, n_comp, m)
    idx, cnt = csd.csa_topk(logits, pos, n_comp, m, k)
    o2, l2 = outputs(B, N)
    csd.csa_tree_attention_decode(*rest, idx, cnt, pos, out=o2, lse=l2, inverse_rope=True)
    torch.cuda.synchronize()
    assert torch.equal(ti, idx) and torch.equal(tc, cnt) and torch.equal(out, o2) and torch.equal(lse, l2)
    assert csd.csa_read_device_error() == 0


def test_expired_waits_are_reported(cuda_lib):
    """A wait limit of one nanosecond: the call ends with a status, and the next one is right."""
    csd = cuda_lib
    for fmt in (0, 1):
        c = Tree(csd, 2, 4, 700, "chain", fmt, seed=18)
        idx, cnt = c.select(600)
        csd.csa_debug_set_wait_limit_ns(1)
        try:
            c.csa(idx, cnt)
        finally:
            csd.csa_debug_set_wait_limit_ns(0)
        assert csd.csa_read_device_error() == csd.ERR_TIMEOUT
        c.check(c.csa(idx, cnt), lambda b, i: idx[b, i, :int(cnt[b, i])].numpy())
        assert csd.csa_read_device_error() == 0


def test_workspaces_are_checked(cuda_lib):
    csd = cuda_lib
    c = Tree(csd, 1, 2, 700, "chain", 0, seed=19)
    idx, cnt = c.select(600)
    need = csd.csa_workspace_bytes(csd.OP_TREE_ATTENTION, 1, 2, 700, 600)
    assert need > 0
    for ws in (torch.empty(need // 4, dtype=torch.uint8, device="cuda"),
               torch.empty(need + 512, dtype=torch.uint8, device="cuda")[16:]):
        with pytest.raises(csd.CsaError) as e:
            c.csa(idx, cnt, ws=ws)
        assert e.value.status == csd.ERR_WORKSPACE
        with pytest.raises(csd.CsaError) as e:
            c.hca(torch.full((1,), 700, dtype=torch.int32), 1, ws=ws)
        assert e.value.status == csd.ERR_WORKSPACE
