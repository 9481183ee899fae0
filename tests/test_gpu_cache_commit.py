"""csa_cache_commit: bytes where they belong and nowhere else; and a whole step of
speculative decoding, from drafts to the next step's cache."""
import numpy as np
import pytest
import torch

import _speculative as S

pytestmark = pytest.mark.gpu


def place(csd, pool, fmt, cap, ring, table=None, page=0):
    return csd.cache_desc(pool, cap, seq_stride=0 if table is not None else cap, block_table=table, page_records=page,
                          fmt=fmt)


def expected(pool, records, select, count, first, cap, ring, table, page):
    want = pool.clone()
    B, N = records.shape[:2]
    T = N if select is None else select.shape[1]
    for b in range(B):
        n = T if count is None else max(0, min(T, int(count[b])))
        for t in range(n):
            e = int(first[b]) + t
            node = t if select is None else int(select[b, t])
            if int(first[b]) < 0 or (ring and t < n - cap) or (not ring and e >= cap) or not 0 <= node < N:
                continue
            slot = e % cap if ring else e
            at = b * cap + slot if table is None else int(table[b, slot // page]) * page + slot % page
            want[at] = records[b, node]
    return want


CASES = [  # B, N, T, cap, ring, page, with select
    (1, 1, 1, 1, True, 0, True), (3, 8, 8, 128, True, 0, True), (2, 9, 9, 5, True, 0, True), (4, 16, 7, 40, False, 0, True),
    (5, 33, 33, 300, False, 32, True), (2, 6, 6, 30, False, 1, False), (70, 128, 128, 256, False, 64, True),
    (1, 3, 200, 64, True, 0, True), (2, 5, 4, 20, True, 0, False),
]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("case", CASES)
def test_records_land_where_they_belong(cuda_lib, case, fmt):
    csd = cuda_lib
    B, N, T, cap, ring, page, chosen = case
    g = torch.Generator().manual_seed(B + N)
    pages = -(-cap // page) if page else 0
    pool = S.random_records(B * pages * page if page else B * cap, fmt, 1)
    table = torch.randperm(B * pages, generator=g).to(torch.int32).view(B, pages) if page else None
    records = S.random_records(B * N, fmt, 2).view(B, N, -1)
    select = torch.randint(0, N, (B, T), generator=g).to(torch.int32) if chosen else None
    first = torch.randint(0, 100000 if ring else max(1, cap - T), (B,), generator=g).to(torch.int32)
    for counted in (True, False):
        if not chosen and T < N and not counted:
            continue
        count = torch.randint(0, T + 1, (B,), generator=g).to(torch.int32) if counted else None
        dev = pool.cuda()
        csd.csa_cache_commit(place(csd, dev, fmt, cap, ring, None if table is None else table.cuda(), page), records.cuda(),
                             None if select is None else select.cuda(), None if count is None else count.cuda(),
                             first.cuda(), ring=ring)
        torch.cuda.synchronize()
        if select is None:  # (the call takes every record of the sequence)
            want = expected(pool, records, None, count, first, cap, ring, table, page)
        else:
            want = expected(pool, records, select, count, first, cap, ring, table, page)
        assert torch.equal(dev.cpu(), want)
        bad = not ring and bool((first + (T if count is None else count) > cap).any())
        assert (csd.csa_read_device_error() == csd.ERR_BAD_INDEX) == bad


def test_what_does_not_fit_is_reported_and_left_out(cuda_lib):
    csd = cuda_lib
    for fmt in (0, 1):
        pool = S.random_records(3 * 10, fmt, 3)
        records = S.random_records(3 * 4, fmt, 4).view(3, 4, -1)
        for select, count, first in (
                ([[0, 1, 2, 3]] * 3, [4, 4, 4], [0, 8, 3]),          # sequence 1 passes the capacity
                ([[0, -1, 2, 4]] * 3, [4, 4, 4], [0, 1, 2]),         # nodes that are none
                ([[3, 2, 1, 0]] * 3, [1, 2, 3], [-1, 0, 0]),         # a negative entry
                ([[3, 2, 1, 0]] * 3, [-2, 9, 3], [0, 0, 0])):        # counts outside [0, T]
            select, count, first = (torch.tensor(v, dtype=torch.int32) for v in (select, count, first))
            dev = pool.cuda()
            csd.csa_cache_commit(place(csd, dev, fmt, 10, False), records.cuda(), select.cuda(), count.cuda(), first.cuda())
            assert csd.csa_read_device_error() == csd.ERR_BAD_INDEX
            assert torch.equal(dev.cpu(), expected(pool, records, select, count, first, 10, False, None, 0))
        # nodes behind the count are not looked at
        dev = pool.cuda()
        select = torch.tensor([[1, -1, 99, -1]] * 3, dtype=torch.int32)
        one = torch.ones(3, dtype=torch.int32)
        csd.csa_cache_commit(place(csd, dev, fmt, 10, False), records.cuda(), select.cuda(), one.cuda(), one.cuda())
        assert csd.csa_read_device_error() == 0
        assert torch.equal(dev.cpu(), expected(pool, records, select, one, one, 10, False, None, 0))


def test_block_tables_with_pages_that_are_none(cuda_lib):
    csd = cuda_lib
    pool = S.random_records(8, 1, 5)
    records = S.random_records(4, 1, 6).view(1, 4, -1)
    table = torch.tensor([[1, -1]], dtype=torch.int32)
    dev = pool.cuda()
    csd.csa_cache_commit(place(csd, dev, 1, 8, False, table.cuda(), 4), records.cuda(), None, None,
                         torch.tensor([2], dtype=torch.int32, device="cuda"))
    assert csd.csa_read_device_error() == csd.ERR_BAD_INDEX
    want = pool.clone()
    want[6:8] = records[0, :2]
    assert torch.equal(dev.cpu(), want)


@pytest.mark.parametrize("fmt", [0, 1])
def test_a_whole_speculative_step(cuda_lib, fmt):
    """Drafts in, attention over the tree, a path accepted and committed, and the next step's root sees it; all of it
    captured once and replayed on new drafts."""
    csd, B, N, cap, k, m, W, R, V = cuda_lib, 3, 7, 256, 60, 4, 32, 40, 1000
    size = csd.FORMAT_BYTES[fmt]
    g = torch.Generator().manual_seed(20)
    pool = S.random_records(B * cap, fmt, 21).cuda()
    ring0 = S.random_records(B * R, fmt, 22).view(B, R, size)
    comp = csd.cache_desc(pool, cap, seq_stride=cap, fmt=fmt)
    ring = ring0.clone().cuda()
    ring_cache = csd.cache_desc(ring, R, seq_stride=R, fmt=fmt)
    parent = S.random_tree("random", B, N, g)
    ctx = torch.tensor([900, 37, 500], dtype=torch.int32)
    pos = (ctx[:, None] + S.depths(parent)).to(torch.int32)
    n_comp = (ctx // m).clamp(max=cap).to(torch.int32).cuda()
    sink = torch.randn(128, generator=g).cuda()
    d = dict(parent=parent.cuda(), pos=pos.cuda(), ctx=ctx.cuda())
    state = {}

    def fill(seed):
        g = torch.Generator().manual_seed(seed)
        new = dict(kv=torch.randn((B, N, 1, 512), generator=g).to(torch.bfloat16),
                   q=torch.randn((B, N, 128, 512), generator=g).to(torch.bfloat16),
                   q_idx=torch.randn((B, N, 64, 128), generator=g).to(torch.bfloat16), w=torch.randn((B, N, 64), generator=g),
                   logits=torch.randn((B, N, V), generator=g) * 3, token=torch.randint(0, V, (B, N), generator=g).int(),
                   uniform=torch.rand((B, N), generator=g) * 0.2, noise=torch.rand((B, V), generator=g) + 1e-3)
        new["token"] = new["logits"].argmax(-1).gather(1, parent.long().clamp(min=0)).int()
        for key, v in new.items():
            if key in state:
                state[key].copy_(v)
            else:
                state[key] = v.cuda()

    fill(30)
    k_idx = torch.randn((B, cap, 128), generator=g).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    k_scale = (torch.rand((B, cap), generator=g) + 0.1).cuda()
    drafts = torch.zeros((B, N, size), dtype=torch.uint8, device="cuda")
    draft_cache = csd.cache_desc(drafts, N, seq_stride=N, fmt=fmt)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = csd.workspace(csd.OP_TREE_STEP, B, N, cap, k, "cuda")

    def step():
        kv = csd.csa_head_norm_rope(state["kv"], d["pos"])
        csd.csa_cache_append(draft_cache, kv[:, :, 0], zero, rope_theta=None)
        q = csd.csa_head_norm_rope(state["q"], d["pos"])
        q_idx, q_scale = csd.csa_head_norm_rope_e4m3(state["q_idx"], d["pos"], norm=False)
        out, lse = csd.csa_tree_decode_step(q_idx, q_scale, state["w"], k_idx, k_scale, q, sink, S.SCALE, comp, ring, W,
                                            drafts, d["parent"], d["pos"], n_comp, m, k, ws=ws, inverse_rope=True)
        path, accepted, nxt = csd.csa_verify_drafts(state["logits"], state["token"], d["parent"], state["uniform"],
                                                    state["noise"])
        csd.csa_cache_commit(ring_cache, drafts, path, accepted, d["ctx"], ring=True)
        return out, lse, path, accepted, nxt

    csd.status_word()
    first = [t.clone() for t in step()]
    torch.cuda.synchronize()
    ring.copy_(ring0.cuda())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, res))
    for seed in (31, 32):
        fill(seed)
        ring.copy_(ring0.cuda())
        graph.replay()
        torch.cuda.synchronize()
        path, accepted, nxt = (t.cpu().numpy() for t in res[2:])
        want = ring0.clone()
        for b in range(B):
            p, token, margin = S.verify(state["logits"][b].double().cpu().numpy(), state["token"][b].cpu().numpy(),
                                        parent[b].numpy(), state["uniform"][b].cpu().numpy(), state["noise"][b].cpu().numpy())
            assert margin > 1e-5 and list(path[b, :accepted[b]]) == p and int(nxt[b]) == token
            for t, node in enumerate(p):
                want[b, (int(ctx[b]) + t) % R] = drafts[b, node].cpu()
        assert int(accepted.max()) > 1 and torch.equal(ring.cpu(), want)
        # the next root, right behind the path, attends to the committed path as to any token
        root = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
        at = (d["ctx"] + res[3])[:, None].to(torch.int32).contiguous()
        n0 = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
        none = torch.full((B, 1, 1), -1, dtype=torch.int32, device="cuda")
        q1 = state["q"][:, :1].contiguous()
        mine = drafts[:, 1:2].contiguous()
        o, l = csd.csa_tree_attention_decode(q1, sink, S.SCALE, comp, ring, W, mine, root, none, n0, at)
        torch.cuda.synchronize()
        for b in range(B):
            x = S.window(want[b].numpy(), mine[b].cpu().numpy(), [-1], 0, int(at[b, 0]), W, fmt)
            ref, rl, A, size_ = S.attend(q1[b, 0].double().cpu().numpy(), sink.double().cpu().numpy(), x)
            # (the bounds of the attention's own tests: weights, latents and output in BF16, fp32 scores)
            assert np.all(np.abs(o[b, 0].double().cpu().numpy() - ref) <= A * (3 * 2.0 ** -8 + 2e-4 * size_.max()) +
                          2.0 ** -8 * np.abs(ref) + 1e-30)
    assert csd.csa_read_device_error() == 0
