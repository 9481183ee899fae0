"""Host-side refusals of the speculative-decoding entry points (no call reaches a
kernel), and pins of the plain restatement that the GPU tests compare with."""
import ctypes as C

import numpy as np
import pytest
import torch

import _speculative as S
import compressed_sparse_decode_gb300 as csd
from test_cache_desc_cpu import on_gpu

P = C.c_void_p
FAKE = P(0x1000)


@pytest.fixture(scope="module")
def lib():
    csd.build()
    return csd.load()


def desc(**kw):
    d = csd.csa_cache_desc()
    d.base, d.n_records, d.seq_stride, d.seq_capacity = 0x1000, 100, 50, 50
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def tree(records=0x1000, parent=0x1000):
    return C.byref(csd.csa_draft_tree(records, parent))


TREE = [
    (dict(q=None), 1), (dict(q=P(0x1008)), 1), (dict(sink=None), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
    (dict(cache=dict(base=None)), 1), (dict(cache=dict(seq_capacity=0)), 1), (dict(fmt=2), 1), (dict(fmt=-1), 1),
    (dict(ring=None), 1), (dict(R=64), 1), (dict(W=0), 1), (dict(W=513, R=600), 1), (dict(tree=None), 1),
    (dict(tree=(None, 0x1000)), 1), (dict(tree=(0x1000, None)), 1), (dict(tree=(0x1008, 0x1000)), 1),
    (dict(tree=(0x1000, 0x1002)), 1), (dict(pos=None), 1), (dict(B=0), 1), (dict(N=0), 1), (dict(N=129), 1),
    (dict(B=1000, N=128, cache=dict(seq_stride=64)), 1), (dict(out=None), 1), (dict(out=P(0x1004)), 1), (dict(lse=None), 1),
    (dict(status=P(0x1001)), 1), (dict(epi=csd.csa_attention_epilogue(1, 1.0, None, None)), 1),
    (dict(epi=csd.csa_attention_epilogue(0, 0.0, 0x1000, None)), 1),
]


@pytest.mark.parametrize("change, status", TREE)
def test_tree_attention_refuses(lib, change, status):
    a = dict(q=FAKE, sink=FAKE, scale=0.04, cache={}, fmt=1, ring=FAKE, R=128, W=128, tree=(0x1000, 0x1000), pos=FAKE, B=1,
             N=2, out=FAKE, lse=FAKE, epi=None, ws=(FAKE, 1 << 30), status=None)
    a.update(change)
    t = None if a["tree"] is None else tree(*a["tree"])
    e = None if a["epi"] is None else C.byref(a["epi"])
    d = desc(**a["cache"])
    assert lib.csa_tree_attention_decode(a["q"], a["sink"], a["scale"], d, a["fmt"], a["ring"], a["R"], a["W"], t, FAKE,
                                         FAKE, a["pos"], a["B"], a["N"], 64, a["out"], a["lse"], e, *a["ws"], a["status"],
                                         None) == status
    assert lib.hca_tree_attention_decode(a["q"], a["sink"], a["scale"], d, a["fmt"], FAKE, a["ring"], a["R"], a["W"], t,
                                         a["pos"], a["B"], a["N"], 128, a["out"], a["lse"], e, *a["ws"], a["status"],
                                         None) == status
    assert lib.csa_tree_decode_step(FAKE, FAKE, FAKE, FAKE, FAKE, a["q"], a["sink"], a["scale"], d, a["fmt"], a["ring"],
                                    a["R"], a["W"], t, a["pos"], FAKE, a["B"], a["N"], 50, 4, 20, a["out"], a["lse"], None,
                                    None, e, *a["ws"], a["status"], None) == status


@pytest.mark.parametrize("ws", [(None, 0), (P(0x1010), 1 << 30), (FAKE, 1000)])
def test_tree_step_refuses_bad_workspaces(lib, ws):
    assert lib.csa_tree_decode_step(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0.04, desc(), 1, FAKE, 128, 128, tree(), FAKE,
                                    FAKE, 1, 2, 50, 4, 20, FAKE, FAKE, None, None, None, *ws, None, None) == 3


@pytest.mark.parametrize("idx, cnt, k, status", [(None, FAKE, 64, 1), (FAKE, None, 64, 1), (FAKE, FAKE, 0, 1),
                                                 (FAKE, FAKE, 2049, 2)])
def test_tree_attention_refuses_bad_selections(lib, idx, cnt, k, status):
    assert lib.csa_tree_attention_decode(FAKE, FAKE, 0.04, desc(), 0, FAKE, 128, 128, tree(), idx, cnt, FAKE, 1, 1, k, FAKE,
                                         FAKE, None, FAKE, 1 << 30, None, None) == status


@pytest.mark.parametrize("change, status", [
    (dict(n_comp=None), 1), (dict(m=0), 1)])
def test_hca_tree_refuses(lib, change, status):
    a = dict(n_comp=FAKE, m=128)
    a.update(change)
    assert lib.hca_tree_attention_decode(FAKE, FAKE, 0.04, desc(), 0, a["n_comp"], FAKE, 128, 128, tree(), FAKE, 1, 1,
                                         a["m"], FAKE, FAKE, None, FAKE, 1 << 30, None, None) == status


@pytest.mark.parametrize("change, status", [
    (dict(logits=None), 1), (dict(logits=P(0x1001)), 1), (dict(logits=P(0x1002), dt=2), 1), (dict(dt=3), 1),
    (dict(sb=-1), 1), (dict(st=-8), 1), (dict(draft=P(0x1002)), 1), (dict(draft=FAKE, q_dt=5), 1), (dict(token=None), 1),
    (dict(parent=None), 1), (dict(uniform=None), 1), (dict(noise=None), 1), (dict(noise=P(0x1002)), 1),
    (dict(temperature=P(0x1001)), 1), (dict(B=0), 1), (dict(N=0), 1), (dict(N=129), 1), (dict(B=1000, N=128), 1),
    (dict(V=0), 1), (dict(path=None), 1), (dict(accepted=None), 1), (dict(next=None), 1), (dict(path=P(0x1002)), 1),
    (dict(status=P(0x1002)), 1), (dict(V=(1 << 24) + 1), 2),
])
def test_verify_refuses(lib, change, status):
    a = dict(logits=FAKE, dt=0, sb=8, st=8, draft=None, q_dt=2, token=FAKE, parent=FAKE, uniform=FAKE, noise=FAKE,
             temperature=None, B=1, N=1, V=8, path=FAKE, accepted=FAKE, next=FAKE, status=None)
    a.update(change)
    assert lib.csa_verify_drafts(a["logits"], a["dt"], a["sb"], a["st"], a["draft"], a["q_dt"], a["token"], a["parent"],
                                 a["uniform"], a["noise"], a["temperature"], a["B"], a["N"], a["V"], a["path"],
                                 a["accepted"], a["next"], None, 0, a["status"], None) == status


@pytest.mark.parametrize("change, status", [
    (dict(cache=dict(base=None)), 1), (dict(cache=dict(n_records=0)), 1), (dict(fmt=2), 1), (dict(records=None), 1),
    (dict(records=P(0x1008)), 1), (dict(N=0), 1), (dict(select=P(0x1004)), 1), (dict(first=None), 1),
    (dict(first=P(0x1004)), 1), (dict(count=P(0x1008)), 1), (dict(B=0), 1), (dict(T=0), 1), (dict(select=None, T=5), 1),
    (dict(status=P(0x1001)), 1), (dict(B=1 << 13, T=1 << 12, cache=dict(seq_stride=64)), 2),
])
def test_commit_refuses(lib, change, status):
    a = dict(cache={}, fmt=0, records=FAKE, N=4, select=FAKE, first=FAKE, count=None, B=1, T=4, status=None)
    a.update(change)
    assert lib.csa_cache_commit(desc(**a["cache"]), a["fmt"], 0, a["records"], a["N"], a["select"], a["first"], a["count"],
                                a["B"], a["T"], a["status"], None) == status


def test_binding_refuses_host_tensors():
    z = torch.zeros
    d = desc()
    with pytest.raises(ValueError, match="CUDA"):
        csd.csa_verify_drafts(z((1, 2, 8)), z((1, 2), dtype=torch.int32), z((1, 2), dtype=torch.int32), z((1, 2)), z((1, 8)))
    with pytest.raises(ValueError, match="CUDA"):
        csd.csa_cache_commit(d, z((1, 2, 592), dtype=torch.uint8), None, None, z(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        csd.hca_tree_attention_decode(z((1, 1, 128, 512), dtype=torch.bfloat16), z(128), 1.0, d, z(1, dtype=torch.int32),
                                      z((1, 128, 592), dtype=torch.uint8), 128, z((1, 1, 592), dtype=torch.uint8),
                                      z((1, 1), dtype=torch.int32), z((1, 1), dtype=torch.int32))


def test_commit_into_a_described_copy_is_refused(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    wide = on_gpu((4, 2, 592)).transpose(0, 1)
    d = csd.cache_desc(wide, 4, seq_stride=4)
    assert d._copied
    with pytest.raises(ValueError, match="copy"):
        csd.csa_cache_commit(d, on_gpu((1, 2, 592)), None, None, on_gpu((1,), torch.int32))


def test_workspaces(lib):
    for op in (csd.OP_TREE_ATTENTION, csd.OP_HCA_TREE_ATTENTION, csd.OP_TREE_STEP):
        assert csd.csa_workspace_bytes(op, 0, 1, 8, 8) == 0 and csd.csa_workspace_bytes(op, 1, 1, 1000, 8) >= 0
    assert csd.csa_workspace_bytes(csd.OP_TREE_STEP, 2, 8, 1000, 64) > 4 * 2 * 8 * 1000


# ---- the restatement against closed forms


def test_restated_verification_of_sure_cases():
    z = np.log(np.array([[0.5, 0.3, 0.2], [0.1, 0.1, 0.8], [1.0, 1.0, 1.0]]))
    ones = np.ones(3)
    # a guess of probability 0.5 is accepted below 0.5, and drawn tokens by the ratio of the probabilities
    assert S.verify(z, [0, 0, 2], [-1, 0, 1], [0, 0.49, 0.79], ones)[0] == [0, 1, 2]
    assert S.verify(z, [0, 0, 2], [-1, 0, 1], [0, 0.51, 0.0], ones)[:2] == ([0], 1)
    assert S.verify(z, [0, 0, 2], [-1, 0, 1], [0, 0.49, 0.81], ones)[:2] == ([0, 1], 0)
    q = np.array([[0.9, 0.05, 0.05]] * 3)
    assert S.verify(z, [0, 0, 2], [-1, 0, 1], [0, 0.55, 0.99], ones, draft=q)[0] == [0, 1, 2]
    assert S.verify(z, [0, 0, 2], [-1, 0, 1], [0, 0.56, 0.99], ones, draft=q)[:2] == ([0], 1)
    # siblings: the second is judged by what the first left, (0, 0.3, 0.2) / 0.5
    assert S.verify(z, [0, 0, 1], [-1, 0, 0], [0, 0.6, 0.59], ones)[0] == [0, 2]
    assert S.verify(z, [0, 0, 1], [-1, 0, 0], [0, 0.6, 0.61], ones)[:2] == ([0], 2)
    assert S.verify(z, [0, 0, 2], [-1, 0, 1], [0, 0, 0], ones, t=0.0)[:2] == ([0, 1, 2], 0)


def test_restated_verification_keeps_the_target():
    """Exactly, by adding up over a fine grid of the random number: one drawn draft."""
    p, q = np.array([0.5, 0.3, 0.2]), np.array([0.2, 0.7, 0.1])
    total, n = np.zeros(3), 2000
    for x in range(3):
        for u in (np.arange(n) + 0.5) / n:
            path, nxt, _ = S.verify(np.log(np.stack([p, p])), [0, x], [-1, 0], [0, u], np.ones(3), draft=np.stack([q, q]))
            if len(path) == 2:
                total[x] += q[x] / n
            else:
                r = np.maximum(p - q, 0)
                total += q[x] / n * r / r.sum()
                assert r[nxt] == r.max()
    assert np.allclose(total, p, atol=2 / n)
