"""csa_verify_drafts against its definition in 64 bits.

What decides are comparisons of numbers that carry fp32 roundings: a softmax weight (a few
2^-24 of its exponent, at most 20 in log2 units here, and of its sum: below 3e-6), products
and quotients of three of them. So sequences whose every decision has a relative margin
above 1e-5 in 64 bits have to come out equal (the others, about one in 10^4, are left
out), and at least nine in ten sequences must have it.
"""
import numpy as np
import pytest
import torch

import _speculative as S

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def make(B, N, V, kind, dtype, q=None, seed=0, sharp=3.0):
    """Logits with a few large ones, drafts that mostly follow them."""
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((B, N, V), generator=g) * 2
    few = min(V, 6)
    best = torch.stack([torch.randperm(V, generator=g)[:few] for _ in range(B * N)]).view(B, N, few)
    logits.scatter_(2, best, np.log(V) + 2 + sharp * torch.rand((B, N, few), generator=g))
    parent = S.random_tree(kind, B, N, g)
    draft = None
    token = torch.randint(0, V, (B, N), generator=g)
    if q:
        draft = torch.softmax(logits + torch.randn((B, N, V), generator=g), -1).to(DT[q])
    seen = {}
    for b in range(B):
        for i in range(1, N):
            up = max(0, int(parent[b, i]))
            n = seen[b, up] = seen.get((b, up), 0) + 1
            if q:
                token[b, i] = int(torch.multinomial(draft[b, up].float() + 1e-12, 1, generator=g))
            elif n <= few:
                token[b, i] = best[b, up, n - 1]
    return dict(logits=logits.to(DT[dtype]), tokens=token.to(torch.int32), parent=parent,
                uniform=torch.rand((B, N), generator=g), noise=(-torch.log1p(-torch.rand((B, V), generator=g))).clamp(min=1e-9),
                draft_probs=draft)


def call(csd, x, temperature=None, **kw):
    dev = {k: None if v is None else v.cuda() for k, v in x.items()}
    r = csd.csa_verify_drafts(dev["logits"], dev["tokens"], dev["parent"], dev["uniform"], dev["noise"],
                              temperature=None if temperature is None else temperature.cuda(),
                              draft_probs=dev["draft_probs"], **kw)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in r]


def check(x, got, temperature=None, least=0.9):
    B, N, V = x["logits"].shape
    path, accepted, nxt = got
    sure = 0
    for b in range(B):
        want, token, margin = S.verify(x["logits"][b].double().numpy(), x["tokens"][b].numpy(), x["parent"][b].numpy(),
                                       x["uniform"][b].numpy(), x["noise"][b].numpy(),
                                       1.0 if temperature is None else float(temperature[b]),
                                       None if x["draft_probs"] is None else x["draft_probs"][b].double().numpy())
        n = int(accepted[b])
        assert 1 <= n <= N and np.all(path[b, n:] == -1) and path[b, 0] == 0
        if margin <= 1e-5:
            continue
        sure += 1
        assert list(path[b, :n]) == want and int(nxt[b]) == token, f"{b}: {path[b, :n]} {nxt[b]} not {want} {token}"
    assert sure >= least * B, f"{sure} of {B} sequences are sure"


SIZES = [  # B, N, V, kind
    (1, 1, 1, "chain"), (3, 2, 2, "chain"), (5, 5, 7, "star"), (4, 9, 8, "random"), (2, 33, 33, "random"),
    (7, 12, 1000, "forest"), (3, 7, 4096, "random"), (3, 7, 4097, "random"), (2, 5, 32768, "chain"),
    (2, 5, 50001, "star"), (1, 128, 300, "random"), (2, 128, 64, "chain"), (40, 4, 9000, "chain"),
    (1, 3, 131072, "chain"), (200, 3, 100, "star"),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("q", [None, "fp32", "bf16", "fp16"])
def test_sizes(cuda_lib, dtype, q):
    for n, (B, N, V, kind) in enumerate(SIZES):
        x = make(B, N, V, kind, dtype, q, seed=n)
        check(x, call(cuda_lib, x))
    assert cuda_lib.csa_read_device_error() == 0


@pytest.mark.parametrize("q", [None, "fp32"])
def test_temperatures(cuda_lib, q):
    t = torch.tensor([0.0, 1.0, 0.3, 2.5, -1.0, float("nan"), 1e-3, 40.0])
    for V in (50, 5000):
        x = make(8, 9, V, "random", "fp32", q, seed=V)
        got = call(cuda_lib, x, t)
        # (in 64 bits a temperature of 40 is nearly flat, 1e-3 nearly greedy: both decide clearly)
        check(x, got, torch.where(torch.isnan(t), 0.0, t), least=0.8)


def test_extreme_temperatures_stay_defined(cuda_lib):
    x = make(4, 6, 500, "random", "bf16", seed=2)
    x["logits"][:, :, 7] = -float("inf")
    x["noise"][:, 7] = 1e-9  # (a weight of any size would win)
    path, accepted, nxt = call(cuda_lib, x, torch.tensor([1e-38, 1e-45, 3e38, float("inf")]))
    assert np.all((nxt >= 0) & (nxt < 500) & (nxt != 7)) and np.all(accepted >= 1)
    z = x["logits"].float().numpy()
    for b in (0, 1):  # the best token, as greedily
        assert z[b, path[b, accepted[b] - 1], nxt[b]] == z[b, path[b, accepted[b] - 1]].max()


def test_greedy_takes_the_lowest_of_equal_logits(cuda_lib):
    for V, at in ((700, (600, 40, 41)), (40000, (39999, 5000, 20000)), (9, (8, 3, 5))):
        x = make(2, 3, V, "chain", "bf16", seed=V)
        x["logits"][:] = -1
        for v in at:
            x["logits"][:, :, v] = 2
        x["tokens"][0, 1:] = min(at)
        x["tokens"][1, 1:] = max(at)
        path, accepted, nxt = call(cuda_lib, x, torch.zeros(2))
        assert list(accepted) == [3, 1] and list(nxt) == [min(at)] * 2 and list(path[0]) == [0, 1, 2]


def test_masked_rows_and_tokens(cuda_lib):
    inf, nan = float("inf"), float("nan")
    for V in (40, 6000):
        x = make(6, 4, V, "chain", "fp32", seed=V)
        x["uniform"][:] = 0  # accepts whatever has any weight
        x["tokens"][:] = 3
        x["logits"][:, :, 3] = 1.0
        x["logits"][0, 1, 3] = -inf           # the draft after token 1 is masked
        x["logits"][1, 2] = -inf              # nothing is left where token 2 is reached
        x["logits"][2, 0] = -inf              # nor at the root
        x["logits"][3, 1, V - 1] = nan
        x["logits"][4, 0, V // 2] = inf
        x["logits"][5, 3, 0] = nan            # the last token's row
        path, accepted, nxt = call(cuda_lib, x)
        assert list(accepted) == [2, 3, 1, 2, 1, 4]
        assert nxt[0] >= 0 and nxt[0] != 3 and list(nxt[1:]) == [-1] * 5
        greedy = call(cuda_lib, x, torch.zeros(6))
        assert list(greedy[2][1:5] == -1) == [list(greedy[0][b]).count(-1) == 4 - g and
                                             (b, int(greedy[0][b, g - 1])) in {(1, 2), (2, 0), (3, 1), (4, 0)}
                                             for b, g in list(enumerate(greedy[1]))[1:5]]
        assert cuda_lib.csa_read_device_error() == 0


def test_drafts_that_are_no_tokens(cuda_lib):
    csd = cuda_lib
    for q in (None, "fp32"):
        x = make(3, 6, 300, "star", "fp32", q, seed=4)
        x["tokens"][0, 2], x["tokens"][1, 1], x["tokens"][2, 5] = 300, -1, 1 << 30
        x["uniform"][:] = 1 - 2.0 ** -24
        got = call(csd, x)
        assert csd.csa_read_device_error() == csd.ERR_BAD_INDEX
        check(x, got)


def test_the_same_token_twice_among_siblings(cuda_lib):
    for q in (None, "bf16"):
        x = make(16, 6, 50, "star", "fp32", q, seed=5)
        x["tokens"][:, 1:] = x["tokens"][:, 1:2]
        x["uniform"][:, 1] = 1 - 2.0 ** -24
        check(x, call(cuda_lib, x))


def test_every_token_drafted_and_refused(cuda_lib):
    """Siblings that are the whole vocabulary: what rounding leaves of the distribution is nothing, or the last token."""
    V = 5
    x = make(8, V + 1, V, "star", "fp32", seed=6)
    x["tokens"][:, 1:] = torch.arange(V, dtype=torch.int32)
    x["uniform"][:] = 1.5  # outside [0, 1): refuses all there is (at 1 the last is a tie, which rounding decides)
    path, accepted, nxt = call(cuda_lib, x)
    assert np.all((nxt >= 0) & (nxt < V)) and np.all(accepted == 1)


def test_drafts_that_agree_are_accepted_and_a_zero_probability_is(cuda_lib):
    x = make(4, 5, 200, "chain", "fp32", "fp32", seed=7)
    x["draft_probs"] = torch.softmax(x["logits"], -1) * (1 - 1e-5)
    path, accepted, nxt = call(cuda_lib, x)
    assert np.all(accepted == 5)
    x["draft_probs"][:] = 0  # (such a token cannot have been drawn: it is accepted if the target allows it)
    assert np.all(call(cuda_lib, x)[1] == 5)


def test_strided_logits(cuda_lib):
    csd = cuda_lib
    for V, pad in ((512, 64), (501, 3), (512, 5)):
        x = make(3, 5, V, "random", "bf16", seed=V + pad)
        wide = torch.full((3, 7, V + pad), 30.0, dtype=torch.bfloat16, device="cuda")
        wide[:, 1:6, :V] = x["logits"].cuda()
        view = wide[:, 1:6, :V]
        want = call(csd, x)
        args = [x[k].cuda() for k in ("tokens", "parent", "uniform", "noise")]
        got = csd.csa_verify_drafts(view, *args)
        assert all(np.array_equal(a, b.cpu().numpy()) for a, b in zip(want, got))
        # one row for all tokens, one for all sequences
        one = x["logits"][:1, :1].cuda()
        got = csd.csa_verify_drafts(one.expand(3, 5, V), *args)
        want = csd.csa_verify_drafts(one.expand(3, 5, V).contiguous(), *args)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_buffers_streams_and_replay(cuda_lib):
    csd = cuda_lib
    x = {k: None if v is None else v.cuda() for k, v in make(6, 9, 5000, "random", "bf16", "fp32", seed=8).items()}
    out = [torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((6, 9), (6,), (6,))]

    def run(to, stream=None):
        return csd.csa_verify_drafts(x["logits"], x["tokens"], x["parent"], x["uniform"], x["noise"], path=to[0],
                                     accepted=to[1], next_token=to[2], draft_probs=x["draft_probs"], stream=stream)

    got = run(out)
    assert all(a is b for a, b in zip(got, out))
    want = [t.clone() for t in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = csd.csa_verify_drafts(x["logits"], x["tokens"], x["parent"], x["uniform"], x["noise"],
                                  draft_probs=x["draft_probs"], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out)
    x["uniform"].copy_(torch.rand((6, 9), generator=torch.Generator().manual_seed(9)))
    x["logits"].copy_(x["logits"].flip(0))
    want = [t.clone() for t in run([torch.empty_like(t) for t in out])]
    for t in out:
        t.fill_(77)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    # call after call the same, bit for bit
    assert all(torch.equal(a, b) for a, b in zip(run([torch.empty_like(t) for t in out]), want))


def test_expired_waits_end_and_the_next_call_is_right(cuda_lib):
    """A wait limit of one nanosecond: a cluster's CTAs give up, or were in time; either way the call ends."""
    csd = cuda_lib
    x = make(20, 5, 40000, "chain", "bf16", "bf16", seed=11)
    want = call(csd, x)
    csd.csa_debug_set_wait_limit_ns(1)
    try:
        for _ in range(3):
            call(csd, x)
    finally:
        csd.csa_debug_set_wait_limit_ns(0)
    assert csd.csa_read_device_error() in (0, csd.ERR_TIMEOUT)
    assert all(np.array_equal(a, b) for a, b in zip(call(csd, x), want))
    assert csd.csa_read_device_error() == 0


@pytest.mark.parametrize("q", [False, True])
def test_what_is_emitted_is_drawn_from_the_target(cuda_lib, q):
    """The first emitted token of 16000 sequences with one target: each token's share within five standard
    deviations of its probability, whatever the drafts."""
    csd, B, N, V = cuda_lib, 16000, 4, 6
    g = torch.Generator(device="cuda").manual_seed(10)
    logits = torch.tensor([1.0, 0.2, -0.5, 2.0, -3.0, 0.0], device="cuda")
    p = torch.softmax(logits.double(), 0).cpu().numpy()
    draft = torch.softmax(torch.tensor([0.0, 1.5, 0.1, 0.5, 0.0, -1.0], device="cuda"), 0)
    parent = torch.tensor([-1, 0, 0, 0], dtype=torch.int32, device="cuda").expand(B, N).contiguous()
    if q:
        token = torch.multinomial(draft.expand(B, V), N, replacement=True, generator=g).int()
    else:
        token = torch.rand((B, V), generator=g, device="cuda").argsort(1)[:, :N].int()
    path, accepted, nxt = csd.csa_verify_drafts(
        logits.expand(B, N, V), token.contiguous(), parent, torch.rand((B, N), generator=g, device="cuda"),
        -torch.log1p(-torch.rand((B, V), generator=g, device="cuda")),
        draft_probs=draft.expand(B, N, V).contiguous() if q else None)
    first = torch.where(accepted > 1, token.gather(1, path[:, 1:2].clamp(min=0).long())[:, 0], nxt)
    share = torch.bincount(first.long(), minlength=V).cpu().numpy() / B
    assert np.all(np.abs(share - p) <= 5 * np.sqrt(p * (1 - p) / B)), f"{share} {p}"
    assert 0.2 < float((accepted > 1).float().mean()) < 0.95
