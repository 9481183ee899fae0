"""The largest calls of speculative decoding: as many rows as the argument checks allow, bit for bit what small calls
give for the same rows."""
import pytest
import torch

import _speculative as S
from test_gpu_verify_drafts import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [0, 1])
def test_tree_attention_of_65408_tokens(cuda_lib, fmt):
    """511 trees of 128 tokens (offsets of q and out pass 2^32 bytes), every sequence one of three."""
    csd, B, N, cap, k, W = cuda_lib, 511, 128, 40, 5, 16
    g = torch.Generator().manual_seed(80)
    three = torch.arange(B) % 3
    pool, ring, draft = (S.random_records(3 * n, fmt, 81 + n).view(3, n, -1).cuda() for n in (cap, W, N))
    q = torch.randn((3, N, 128, 512), generator=g).to(torch.bfloat16).cuda()
    sink = torch.randn(128, generator=g).cuda()
    parent = S.random_tree("random", 3, N, g)
    pos = (torch.tensor([[0], [17], [900]]) + S.depths(parent)).to(torch.int32)
    idx = torch.stack([torch.randperm(cap, generator=g)[:k].sort().values for _ in range(3 * N)]).view(3, N, k).to(torch.int32)
    cnt = torch.randint(0, k + 1, (3, N), generator=g).to(torch.int32)

    def call(which):
        which = which.cuda()
        pick = [t.cuda()[which].contiguous() for t in (pool, ring, draft, q, parent, pos, idx, cnt)]
        comp = csd.cache_desc(pick[0], cap, seq_stride=cap, fmt=fmt)
        return csd.csa_tree_attention_decode(pick[3], sink, S.SCALE, comp, pick[1], W, pick[2], pick[4], pick[6], pick[7],
                                             pick[5], inverse_rope=True)

    want = call(torch.arange(3))
    got = call(three)
    for b in (0, 1, 2, 255, 256, B - 3, B - 2, B - 1):
        assert torch.equal(got[0][b], want[0][b % 3]) and torch.equal(got[1][b], want[1][b % 3]), b
    assert csd.csa_read_device_error() == 0


def test_verification_of_65535_sequences(cuda_lib):
    csd, B = cuda_lib, 65535
    for N, V in ((1, 33), (1, 64)):
        x = make(7, N, V, "chain", "bf16", seed=V)
        which = torch.arange(B) % 7
        small = [x[n].cuda() for n in ("logits", "tokens", "parent", "uniform", "noise")]
        want = csd.csa_verify_drafts(*small)
        got = csd.csa_verify_drafts(*[t[which.cuda()].contiguous() for t in small])
        assert all(torch.equal(a, b[which.cuda()]) for a, b in zip(got, want))
    assert csd.csa_read_device_error() == 0


@pytest.mark.parametrize("fmt", [0, 1])
def test_commit_of_as_many_entries_as_allowed(cuda_lib, fmt):
    """2^24 entries of 2^17 rings of two records: the last two of each stay."""
    csd, B, T, N = cuda_lib, 1 << 17, 128, 3
    size = csd.FORMAT_BYTES[fmt]
    g = torch.Generator(device="cuda").manual_seed(82)
    records = torch.randint(0, 256, (B, N, size), dtype=torch.uint8, device="cuda", generator=g)
    select = torch.randint(0, N, (B, T), dtype=torch.int32, device="cuda", generator=g)
    first = torch.randint(0, 1 << 20, (B,), dtype=torch.int32, device="cuda", generator=g)
    pool = torch.zeros((B, 2, size), dtype=torch.uint8, device="cuda")
    csd.csa_cache_commit(csd.cache_desc(pool, 2, seq_stride=2, fmt=fmt), records, select, None, first, ring=True)
    assert csd.csa_read_device_error() == 0
    b = torch.arange(B, device="cuda")
    for t in (T - 2, T - 1):
        assert torch.equal(pool[b, ((first + t) % 2).long()], records[b, select[:, t].long()])
