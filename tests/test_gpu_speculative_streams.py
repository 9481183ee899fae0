"""Calls of speculative decoding on two streams at once, each with buffers of its own."""
import pytest
import torch

import _speculative as S
from test_gpu_tree_attention import Tree
from test_gpu_verify_drafts import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [0, 1])
def test_two_streams_at_once(cuda_lib, fmt):
    """Trees that are dealt out and trees split in equal parts, verifications of two sizes: what each gives is what it
    gives alone, bit for bit, whatever runs beside it."""
    csd = cuda_lib
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    jobs = []
    for n, (B, N, cap) in enumerate(((4, 9, 3300), (3, 7, 500))):
        c = Tree(csd, B, N, cap, "random", fmt, seed=90 + n)
        x = {k: v.cuda() for k, v in make(6 + 40 * n, N, (40000, 5001)[n], "random", "bf16", seed=91 + n).items() if v is not None}
        c.pos = (cap + S.depths(c.parent)).to(torch.int32)
        t = [a.cuda() for a in (c.q, c.sink, c.ring, c.draft, c.parent, c.pos)]
        jobs.append((c, c.cache(), t, torch.full((B,), cap, dtype=torch.int32, device="cuda"), x))

    def run(n, stream):
        c, comp, (q, sink, ring, draft, parent, pos), n_comp, x = jobs[n]
        return [*csd.hca_tree_attention_decode(q, sink, S.SCALE, comp, n_comp, ring, c.W, draft, parent, pos, 1,
                                               stream=stream),
                *csd.csa_verify_drafts(x["logits"], x["tokens"], x["parent"], x["uniform"], x["noise"], stream=stream)]

    want = [run(n, None) for n in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for i in range(25):
        for n in range(2):
            got[n].append(run(n, side[(i + n) % 2]))
    torch.cuda.synchronize()
    for n in range(2):
        for r in got[n]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[n]))
    assert csd.csa_read_device_error() == 0
