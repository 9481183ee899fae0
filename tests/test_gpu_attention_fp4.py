"""Attention over caches of 4-bit records against its definition in 64 bits.

Bounds (derived before the first run), for head h, output dim d, with A_d =
sum_j p_j |x_jd| / den the weighted magnitude of what is summed:
* the latents are exact in BF16; each score moves by at most B = 2^-15 scale
  max_j sum_d |q_d x_jd| (fp32 accumulation of 512 exact products, with a wide
  margin for the tensor core's alignment), so each weight by e^{2B} - 1;
* the weights are rounded to BF16 (2^-8 of each) and the output too (2^-8 |o_d|);
* the partial outputs of a split are rounded to FP16 (2^-11 of each, at most A_d
  together) in units u of a power of two for each 32 dims, whose largest value is
  at least 2^14 u; FP16's smallest step is 2^-24, so a value far below the largest
  of its 32 moves by up to 2^-25 u <= 2^-39 of that largest, which is at most the
  32 dims' largest share of A (summed over the splits: 2^-39 G_d, G_d = max A
  over the 32 dims);
* fp32 exponentials and sums: below 1e-5.
So |err_d| <= A_d (2 2^-8 + 3 B + 1e-5) + 2^-39 G_d + 2^-8 |o_d|, for rotated dims with A
and |o| summed over the pair (+ 1e-6 of them for sine and cosine), and
|lse err| <= B + 1e-5 (1 + |lse|).
"""
import math

import numpy as np
import pytest
import torch

import _records as R

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5
BF = 2.0 ** -8


class Case:
    """Random caches, queries and positions, and the definition in 64 bits."""

    def __init__(self, csd, B, T, cap, W=128, Rr=None, paged=True, page=32, seed=0, spread=1.0, extra=0):
        g = torch.Generator().manual_seed(seed)
        self.csd, self.B, self.T, self.cap, self.W = csd, B, T, cap, W
        self.R = Rr or W + T - 1
        pages = -(-cap // page)
        n = B * pages * page if paged else B * cap
        self.pool = R.random_fp4_records(n + extra, seed + 1, spread)
        self.ring = R.random_fp4_records(B * self.R, seed + 2, spread).view(B, self.R, 384)
        self.table = torch.randperm(B * pages, generator=g).to(torch.int32).view(B, pages) if paged else None
        self.page, self.paged = page, paged
        self.q = torch.randn((B, T, 128, 512), generator=g).to(torch.bfloat16)
        self.sink = torch.randn(128, generator=g)
        self.pos = (torch.randint(W, 2 * cap + W, (B, 1), generator=g) + torch.arange(T)).to(torch.int32)
        self.gen = g

    def where(self, b, e):
        e = np.asarray(e)
        if not self.paged:
            return b * self.cap + e
        return self.table[b].numpy()[e // self.page].astype(np.int64) * self.page + e % self.page

    def select(self, k, counts):
        """Distinct entries in ascending order, -1 behind each row's count."""
        idx = torch.full((self.B, self.T, k), -1, dtype=torch.int32)
        for b in range(self.B):
            for t in range(self.T):
                c = int(counts[b][t])
                idx[b, t, :c] = torch.randperm(self.cap, generator=self.gen)[:c].sort().values.to(torch.int32)
        return idx, torch.tensor(counts, dtype=torch.int32)

    def device(self):
        csd = self.csd
        self.d_pool = self.pool.cuda()
        self.comp = csd.cache_desc(self.d_pool, self.cap, seq_stride=0 if self.paged else self.cap,
                                   block_table=self.table.cuda() if self.paged else None,
                                   page_records=self.page if self.paged else 0, fmt=csd.FORMAT_FP4)
        return self.q.cuda(), self.sink.cuda(), SCALE, self.comp

    def csa(self, idx, cnt, **kw):
        q, sink, scale, comp = self.device()
        r = self.csd.csa_sink_attention_decode_fp4(q, sink, scale, comp, self.ring.cuda(), self.W, idx.cuda(),
                                                   cnt.cuda(), self.pos.cuda(), **kw)
        torch.cuda.synchronize()
        return r

    def hca(self, n_comp, m, **kw):
        q, sink, scale, comp = self.device()
        r = self.csd.hca_sink_attention_decode_fp4(q, sink, scale, comp, n_comp.cuda(), self.ring.cuda(), self.W,
                                                   self.pos.cuda(), m, **kw)
        torch.cuda.synchronize()
        return r

    def check(self, got, entries, theta=None, what=""):
        """got = (out, lse); entries(b, t) -> the compressed entries attended to."""
        out, lse = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
        worst = 0.0
        for b in range(self.B):
            for t in range(self.T):
                p = int(self.pos[b, t])
                win = np.arange(max(0, p - self.W + 1), p + 1) % self.R if p >= 0 else np.zeros(0, int)
                x = np.concatenate([R.fp4_values(self.pool.numpy()[self.where(b, entries(b, t))].reshape(-1, 384)),
                                    R.fp4_values(self.ring[b].numpy()[win])])
                ref, ref_lse, A, Bz = attend(self.q[b, t].double().numpy(), self.sink.double().numpy(), x)
                G = np.repeat(A.reshape(128, 16, 32).max(-1), 32, axis=-1)
                o, bound = ref, A * (2 * BF + 3 * Bz[:, None] + 1e-5) + 2.0 ** -39 * G + BF * np.abs(ref)
                if theta:
                    o = turn_back(ref, p, theta)
                    s = bound[:, 448::2] + bound[:, 449::2] + 1e-6 * (A[:, 448::2] + A[:, 449::2])
                    s = s + BF * (np.abs(ref[:, 448::2]) + np.abs(ref[:, 449::2]))
                    bound = bound.copy()
                    bound[:, 448::2] = bound[:, 449::2] = s
                assert np.all(np.isfinite(out[b, t])), f"{what} {b},{t}"
                err = np.abs(out[b, t] - o)
                assert np.all(err <= bound + 1e-30), f"{what} {b},{t}: {np.max(err / (bound + 1e-30)):.3g} x bound"
                worst = max(worst, float(np.max(err / (bound + 1e-30))))
                inf = np.isneginf(ref_lse)
                assert np.array_equal(inf, np.isneginf(lse[b, t])), f"{what} {b},{t}"
                le = np.abs(lse[b, t][~inf] - ref_lse[~inf])
                assert np.all(le <= Bz[~inf] + 1e-5 * (1 + np.abs(ref_lse[~inf]))), f"{what} {b},{t}: lse {le.max():.3g}"
        return worst


def attend(q, sink, x):
    """Definition in 64 bits -> (o, lse, A, B)."""
    z = SCALE * (q @ x.T)
    M = np.maximum(sink, z.max(1, initial=-np.inf))
    M0 = np.where(np.isneginf(M), 0.0, M)
    with np.errstate(divide="ignore"):
        p = np.exp(z - M0[:, None])
        den = p.sum(1) + np.exp(sink - M0)
        lse = M0 + np.log(den)
    d = np.where(den > 0, den, 1.0)[:, None]
    Bz = 2.0 ** -15 * SCALE * (np.abs(q) @ np.abs(x).T).max(1, initial=0.0)
    return p @ x / d, lse, p @ np.abs(x) / d, Bz


def turn_back(o, p, theta):
    o = o.copy()
    a = p * theta ** (-2.0 * np.arange(32) / 64)
    u, v = o[:, 448::2].copy(), o[:, 449::2].copy()
    o[:, 448::2] = u * np.cos(a) + v * np.sin(a)
    o[:, 449::2] = -u * np.sin(a) + v * np.cos(a)
    return o


CSA = [  # B, T, cap, k, counts of the rows, W, R, paged
    (1, 1, 5, 1, [[0]], 1, 1, False), (1, 1, 70, 64, [[64]], 128, 128, True), (2, 3, 300, 130, None, 128, 140, True),
    (3, 1, 900, 517, [[517], [0], [63]], 128, 128, False), (1, 2, 2100, 2048, [[2048, 2000]], 512, 600, True),
    (40, 2, 100, 33, None, 7, 9, True), (1, 1, 64, 65, [[64]], 64, 64, True), (9, 8, 260, 200, None, 128, 135, True),
]


@pytest.mark.parametrize("case", CSA)
def test_csa_fp4(cuda_lib, case):
    csd = cuda_lib
    B, T, cap, k, counts, W, Rr, paged = case
    c = Case(csd, B, T, cap, W, Rr, paged, seed=B + cap + k)
    if counts is None:
        counts = [[(17 * b + 5 * t + 3) % (min(k, cap) + 1) for t in range(T)] for b in range(B)]
    idx, cnt = c.select(k, counts)
    c.check(c.csa(idx, cnt), lambda b, t: idx[b, t, :counts[b][t]].numpy(), what="plain")
    got = c.csa(idx, cnt, inverse_rope=True, rope_theta=10000.0)
    c.check(got, lambda b, t: idx[b, t, :counts[b][t]].numpy(), theta=10000.0, what="inverse rope")
    assert csd.csa_read_device_error() == 0


@pytest.mark.parametrize("B,T,cap,m,vis", [(1, 1, 1, 128, [0]), (2, 1, 300, 128, [1, 300]), (3, 2, 200, 4, [63, 64, 65]),
                                           (64, 1, 600, 128, None), (1, 1, 8192, 128, [8192]), (5, 3, 129, 2, None)])
def test_hca_fp4(cuda_lib, B, T, cap, m, vis):
    csd = cuda_lib
    c = Case(csd, B, T, cap, page=1, seed=cap + m)
    vis = vis or [(29 * b + 11) % (cap + 1) for b in range(B)]
    n_comp = torch.tensor(vis, dtype=torch.int32)
    c.pos = (m * (cap + 1) + torch.arange(T)[None] + torch.arange(B)[:, None]).to(torch.int32)
    got = c.hca(n_comp, m, inverse_rope=True, rope_theta=1e6)
    c.check(got, lambda b, t: np.arange(vis[b]), theta=1e6, what="hca")
    # positions that cut the visible range
    c.pos = ((torch.arange(B)[:, None] * 37) % (m * cap + 1) + torch.arange(T)[None]).to(torch.int32)
    c.check(c.hca(n_comp, m), lambda b, t: np.arange(min(vis[b], int(c.pos[b, t]) // m)), what="hca early")
    assert csd.csa_read_device_error() == 0


def test_rows_without_candidates_and_minus_infinite_sinks(cuda_lib):
    csd = cuda_lib
    c = Case(csd, 3, 2, 50, seed=5)
    c.pos = torch.tensor([[-1, 0], [3, -7], [200, 201]], dtype=torch.int32)
    c.sink[::2] = -math.inf
    counts = [[0, 0], [0, 0], [20, 0]]
    idx, cnt = c.select(20, counts)
    got = c.csa(idx, cnt)
    c.check(got, lambda b, t: idx[b, t, :counts[b][t]].numpy())
    assert torch.all(got[0][0, 0] == 0) and torch.all(got[0][1, 1] == 0)
    assert torch.equal(got[1][0, 0].cpu()[1::2], c.sink[1::2]) and torch.all(torch.isneginf(got[1][0, 0, ::2]))
    cnt[0, 0], cnt[2, 1] = -4, 99  # counts outside [0, k] are clamped
    idx[2, 1] = torch.arange(20)
    c.check(c.csa(idx, cnt), lambda b, t: np.arange(20) if (b, t) == (2, 1) else idx[b, t, :counts[b][t]].numpy())
    big = torch.full((128,), 90.0)
    c.sink = big
    c.check(c.csa(idx, cnt), lambda b, t: np.arange(20) if (b, t) == (2, 1) else idx[b, t, :counts[b][t]].numpy(),
            what="large sink")


def test_growing_maxima_and_repeated_entries(cuda_lib):
    """Scores that grow by far more than the lazy rescale's threshold from chunk
    to chunk (and shrink again), one head at a time, and an entry selected often."""
    csd = cuda_lib
    c = Case(csd, 2, 1, 1500, paged=False, seed=8)
    scale = torch.arange(1500) // 100  # chunks' magnitudes: powers of two up to 2^7, then down
    e = torch.where(scale < 8, scale, 15 - scale).repeat(2)
    c.pool[:, 380] = (115 + e).to(torch.uint8)
    c.pool[:, 224:352] = 0
    c.q[:, :, ::3] *= 0.01
    c.q[:, :, 1::3] *= 4
    idx = torch.arange(1500, dtype=torch.int32).expand(2, 1, 1500).contiguous()
    idx[1, 0] = idx[1, 0].flip(0)
    cnt = torch.full((2, 1), 1500, dtype=torch.int32)
    c.check(c.csa(idx, cnt), lambda b, t: idx[b, t].numpy(), what="growth")
    idx[1, 0, :700] = 777
    c.check(c.csa(idx, cnt), lambda b, t: idx[b, t].numpy(), what="repeats")
    assert csd.csa_read_device_error() == 0


def test_bad_indices_are_reported_and_skipped_and_nan_records_unread(cuda_lib):
    csd = cuda_lib
    c = Case(csd, 2, 1, 100, paged=False, seed=11)
    c.pool[50:60, 380] = 255  # NaN records that nothing selects
    c.ring[:, :2] = 255
    c.pos = torch.tensor([[125], [129]], dtype=torch.int32)  # window: slots 0..125, and 2..127, 0, 1
    c.ring[1] = R.random_fp4_records(128, 99)
    c.ring[0, 126:] = 255
    c.ring[0, :2] = R.random_fp4_records(2, 98)
    idx = torch.arange(40, dtype=torch.int32).repeat(2, 1, 1)
    cnt = torch.full((2, 1), 40, dtype=torch.int32)
    good = c.csa(idx, cnt)
    assert csd.csa_read_device_error() == 0
    c.check(good, lambda b, t: np.arange(40))
    idx[0, 0, 7], idx[1, 0, 39], idx[1, 0, 0] = -1, 100, 2147483647
    got = c.csa(idx, cnt)
    assert csd.csa_read_device_error() == csd.ERR_BAD_INDEX
    keep = [np.delete(np.arange(40), 7), np.arange(1, 39)]
    c.check(got, lambda b, t: keep[b])


def test_fp4_output(cuda_lib):
    """E2M1 output against the 64-bit output: the multiplier is amax / 6 of what
    the kernel forms, each value within the code's half step (at most one unit)
    and the output's own bound."""
    csd = cuda_lib
    for B, T, cap, counts in ((1, 1, 400, [[333]]), (40, 2, 80, None)):
        c = Case(csd, B, T, cap, seed=21)
        counts = counts or [[(7 * b + t) % 81 for t in range(T)] for b in range(B)]
        idx, cnt = c.select(max(max(x) for x in counts), counts)
        (codes, s), lse = c.csa(idx, cnt, inverse_rope=True, fp4_out=True)
        out, lse2 = c.csa(idx, cnt, inverse_rope=True)
        assert torch.equal(lse, lse2)
        o = out.double().cpu().numpy()
        p, s = codes.cpu().numpy(), s.double().cpu().numpy()
        code = np.stack([p & 15, p >> 4], -1).reshape(*p.shape[:-1], 512)
        v = np.where(code >= 8, -1.0, 1.0) * R.E2M1[code & 7] * np.repeat(s, 128, axis=-1)
        amax = np.abs(o).reshape(*o.shape[:-1], 4, 128).max(-1)
        assert np.all(np.abs(s - np.where(amax > 0, amax / 6, 1)) <= BF * np.where(amax > 0, amax / 6, 1) * 1.001)
        assert np.all(np.abs(v - o) <= np.repeat(s, 128, axis=-1) * (1 + BF) + BF * np.abs(o))
        step = np.where(np.abs(v) >= 4 * np.repeat(s, 128, axis=-1), 1.0, 0.5) * np.repeat(s, 128, axis=-1)
        assert np.mean(np.abs(v - o) <= step * 0.51 + BF * np.abs(o)) > 0.5
    assert csd.csa_read_device_error() == 0


@pytest.mark.parametrize("sink, largest", [(20.0, -120), (30.0, -134)])
def test_fp4_output_of_tiny_values(cuda_lib, sink, largest):
    """Outputs near 2^-134, whose multiplier is a subnormal number: each value
    within its code's half step (at most one unit, and half a step of 2^-149 a
    unit for the multiplier's own rounding) of the 64-bit one."""
    csd = cuda_lib
    for B, T, cap, n in ((1, 1, 300, 280), (40, 2, 40, 30)):  # with and without splits
        c = Case(csd, B, T, cap, seed=23)
        for records in (c.pool, c.ring.view(-1, 384)):
            records[:, 380] = 20  # units 128 .. 448 times 2^-107: values near 2^-97
            records[:, 224:352] = 0
        c.sink = torch.full((128,), sink)  # the candidates' weight is about n e^-sink
        counts = [[n] * T for _ in range(B)]
        idx, cnt = c.select(n, counts)
        (codes, s), _ = c.csa(idx, cnt, fp4_out=True)
        p, s = codes.cpu().numpy(), s.double().cpu().numpy()
        code = np.stack([p & 15, p >> 4], -1).reshape(*p.shape[:-1], 512)
        v = np.where(code >= 8, -1.0, 1.0) * R.E2M1[code & 7] * np.repeat(s, 128, axis=-1)
        for b, t in ((0, 0), (B - 1, T - 1)):
            x = np.concatenate([R.fp4_values(c.pool.numpy()[c.where(b, idx[b, t, :n].numpy())]),
                                R.fp4_values(c.ring[b].numpy()[np.arange(int(c.pos[b, t]) - 127, int(c.pos[b, t]) + 1) % c.R])])
            o, _, A, _ = attend(c.q[b, t].double().numpy(), c.sink.double().numpy(), x)
            assert 2.0 ** (largest - 6) < np.abs(o).max() < 2.0 ** (largest + 2)
            sd = np.repeat(s[b, t], 128, axis=-1)
            assert np.all(np.abs(v[b, t] - o) <= sd * (1 + BF) + 3 * BF * A + 8 * 2.0 ** -149)
    assert csd.csa_read_device_error() == 0


@pytest.mark.parametrize("B,cap,n", [(2, 900, 700), (90, 40, 30)])  # with and without splits
def test_a_selected_nan_record_reaches_its_row_only(cuda_lib, B, cap, n):
    csd = cuda_lib
    c = Case(csd, B, 1, cap, paged=False, seed=33)
    idx, cnt = c.select(n, [[n]] * B)
    good = c.csa(idx, cnt)
    bad = B // 2
    c.pool[bad * cap + int(idx[bad, 0, n // 3]), 380] = 255
    out, lse = c.csa(idx, cnt)
    assert torch.all(torch.isnan(out[bad, :, :, :448])) and torch.all(torch.isnan(lse[bad]))
    keep = [b for b in range(B) if b != bad]
    assert torch.equal(out[keep], good[0][keep]) and torch.equal(lse[keep], good[1][keep])
    c.pool[bad * cap + int(idx[bad, 0, n // 3]), 380] = 127
    c.q[0, 0, 5, 9] = math.nan  # a head of the query
    out, lse = c.csa(idx, cnt)
    heads = [h for h in range(128) if h != 5]
    assert torch.all(torch.isnan(out[0, 0, 5])) and torch.isnan(lse[0, 0, 5])
    assert torch.all(torch.isfinite(out[0, 0, heads].float())) and torch.all(torch.isfinite(lse[0, 0, heads]))
    assert csd.csa_read_device_error() == 0


def test_expired_waits_are_reported_and_the_next_call_is_right(cuda_lib):
    csd = cuda_lib
    c = Case(csd, 3, 2, 700, seed=50)
    counts = [[600, 0], [130, 64], [1, 333]]
    idx, cnt = c.select(600, counts)
    first = c.csa(idx, cnt)
    c.check(first, lambda b, t: idx[b, t, :counts[b][t]].numpy())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    csd.csa_debug_set_wait_limit_ns(1)
    try:
        c.csa(idx, cnt, status=status)
        seen = csd.csa_read_device_error(status=status)
    finally:
        csd.csa_debug_set_wait_limit_ns(0)
    assert seen == csd.ERR_TIMEOUT
    again = c.csa(idx, cnt, status=status)
    assert csd.csa_read_device_error(status=status) == 0
    assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_offsets_past_32_bits(cuda_lib):
    csd = cuda_lib
    n = (1 << 32) // 384 + 5000
    small = R.random_fp4_records(200, 4)
    pool = torch.zeros((n, 384), dtype=torch.uint8, device="cuda")
    pool[-200:] = small.cuda()
    c = Case(csd, 1, 1, 200, paged=False, seed=30)
    c.pool = small
    idx, cnt = c.select(150, [[150]])
    want = c.csa(idx, cnt)
    comp = csd.cache_desc(pool, n, seq_stride=n, fmt=csd.FORMAT_FP4)
    got = csd.csa_sink_attention_decode_fp4(c.q.cuda(), c.sink.cuda(), SCALE, comp, c.ring.cuda(), c.W,
                                            torch.where(idx >= 0, idx + n - 200, idx).cuda(), cnt.cuda(), c.pos.cuda())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert csd.csa_read_device_error() == 0


def test_results_do_not_depend_on_the_run_or_the_workspace(cuda_lib):
    """The same call twice, with a workspace of its own full of NaN bytes, on
    another stream beside a second call, and from a replayed graph: equal bits."""
    csd = cuda_lib
    c = Case(csd, 4, 2, 700, seed=40)
    counts = [[(97 * b + 300 * t) % 601 for t in range(2)] for b in range(4)]
    idx, cnt = c.select(600, counts)
    first = c.csa(idx, cnt, inverse_rope=True)
    c.check(first, lambda b, t: idx[b, t, :counts[b][t]].numpy(), theta=10000.0)
    args = [*c.device(), c.ring.cuda(), c.W, idx.cuda(), cnt.cuda(), c.pos.cuda()]
    call = lambda **kw: csd.csa_sink_attention_decode_fp4(*args, inverse_rope=True, **kw)  # noqa: E731
    ws = csd.workspace(csd.OP_ATTENTION, 4, 2, c.cap, 600)
    assert ws is not None
    ws.fill_(255)
    outs = [call(ws=ws)]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (a, b):
        with torch.cuda.stream(s):
            outs.append(call())
    for s in (a, b, a.cuda_stream):  # and named by the call, which makes its outputs and workspace
        outs.append(call(stream=s))
    torch.cuda.synchronize()
    ws.fill_(255)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()  # two graphs that share a workspace
    held = []
    for g in (g1, g2):
        with torch.cuda.graph(g, stream=a):
            held.append(call(ws=ws))
    for _ in range(2):
        g1.replay()
        g2.replay()
    torch.cuda.synchronize()
    for o in outs + held:
        assert torch.equal(o[0], first[0]) and torch.equal(o[1], first[1])
    assert csd.csa_read_device_error() == 0


def test_one_layer_from_projections_to_attention(cuda_lib):
    """The operators as a decode loop uses them: a prompt's entries and window
    appended, then steps of prepared queries, append and csa_decode_step_fp4; each
    step's selection from the library, its attention against 64 bits on the
    records that the cache then holds; captured and replayed like the direct calls."""
    csd = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(77)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    B, T, m, k, W, cap, L = 3, 2, 4, 48, 128, 512, 700
    Rr = W + T - 1
    pages = cap // 32
    pool = torch.zeros((B * pages * 32, 384), dtype=torch.uint8, device="cuda")
    table = torch.randperm(B * pages, generator=g, device="cuda").to(torch.int32).view(B, pages).contiguous()
    comp = csd.cache_desc(pool, cap, block_table=table, page_records=32, fmt=csd.FORMAT_FP4)
    ring = torch.zeros((B, Rr, 384), dtype=torch.uint8, device="cuda")
    ring_desc = csd.cache_desc(ring, Rr, seq_stride=Rr, fmt=csd.FORMAT_FP4)
    k_idx = torch.zeros((B, cap, 128), dtype=torch.uint8, device="cuda")
    k_scale = torch.ones((B, cap), device="cuda")
    lens = torch.tensor([L, 130, 3], dtype=torch.int32, device="cuda")
    w = 1 + 0.1 * torch.randn(512, generator=g, device="cuda")
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    csd.csa_cache_append(ring_desc, rnd(B, L, 512), zero, lens, ring=True, norm=True, weight=w)
    csd.csa_cache_append(comp, rnd(B, L // m, 512), zero, lens // m, norm=True, weight=w, pos_stride=m,
                         key=rnd(B, L // m, 128), k_idx=k_idx, k_idx_scale=k_scale)
    kv, q_in, qi_in = rnd(B, T, 512), rnd(B, T, 128, 512), rnd(B, T, 64, 128)
    w_idx = torch.randn((B, T, 64), generator=g, device="cuda")
    sink = torch.randn(128, generator=g, device="cuda")
    pos = (lens[:, None] + torch.arange(T, device="cuda")).to(torch.int32).contiguous()
    n_comp = (lens // m).to(torch.int32)
    idx = torch.empty((B, T, k), dtype=torch.int32, device="cuda")
    cnt = torch.empty((B, T), dtype=torch.int32, device="cuda")
    out, lse = torch.empty((B, T, 128, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((B, T, 128), device="cuda")
    ws = csd.workspace(csd.OP_DECODE_STEP, B, T, cap, k)

    def step():
        csd.csa_cache_append(ring_desc, kv, pos[:, 0].contiguous(), ring=True, norm=True, weight=w)
        q = csd.csa_head_norm_rope(q_in, pos)
        qi, qs = csd.csa_head_norm_rope_e4m3(qi_in, pos, norm=False)
        csd.csa_decode_step_fp4(qi, qs, w_idx, k_idx, k_scale, q, sink, SCALE, comp, ring, W, pos, n_comp, m, k, out=out,
                                lse=lse, topk_idx=idx, topk_cnt=cnt, ws=ws, inverse_rope=True)
        return q

    q = step()
    torch.cuda.synchronize()
    assert csd.csa_read_device_error() == 0
    assert cnt.tolist() == [[48, 48], [32, 32], [0, 0]]
    c = Case.__new__(Case)
    c.B, c.T, c.cap, c.W, c.R, c.paged, c.page = B, T, cap, W, Rr, True, 32
    c.pool, c.ring, c.table, c.q, c.sink, c.pos = (t.cpu() for t in (pool, ring, table, q, sink, pos))
    c.check((out, lse), lambda b, t: idx[b, t, :int(cnt[b, t])].cpu().numpy(), theta=10000.0, what="step")
    direct = [t.clone() for t in (out, lse, idx, cnt, ring)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    out.zero_(), lse.zero_(), idx.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(direct, (out, lse, idx, cnt, ring)):
        assert torch.equal(a, b)
    assert csd.csa_read_device_error() == 0


def test_the_other_format_is_refused(cuda_lib):
    csd = cuda_lib
    c = Case(csd, 1, 1, 40, seed=1)
    idx, cnt = c.select(8, [[8]])
    q, sink, scale, comp = c.device()
    rest = (idx.cuda(), cnt.cuda(), c.pos.cuda())
    ring8 = torch.zeros((1, 128, 592), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="592-byte"):
        csd.csa_sink_attention_decode(q, sink, scale, comp, ring8, 128, *rest)
    with pytest.raises(ValueError, match="swa_ring"):
        csd.csa_sink_attention_decode_fp4(q, sink, scale, comp, ring8, 128, *rest)
    comp8 = csd.cache_desc(torch.zeros((40, 592), dtype=torch.uint8, device="cuda"), 40)
    with pytest.raises(ValueError, match="384-byte"):
        csd.csa_sink_attention_decode_fp4(q, sink, scale, comp8, c.ring.cuda(), 128, *rest)
