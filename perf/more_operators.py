"""The speculative-decoding operators of the decode library: plain forms, the
library's own calls, and the cases they are measured on.

A step of speculative decoding runs the model over a tree of drafted tokens in
one go, keeps the path of it that the model agrees with, and puts that path's
latents into the cache. Three operators, used together around such a step:

* ``tree``     sink-merged attention of a tree's tokens: each attends to its top-k
               (or, HCA, every visible) compressed entries, to the committed tokens
               of its sliding window and to its own ancestors among the drafts.
               Caches of FP8 or 4-bit records.
* ``verify``   walks the tree from its root: a drafted child is accepted with the
               probability that leaves the target's distribution unchanged, given
               the random numbers; then the next token is drawn.
* ``commit``   the accepted path's records from the drafts into the ring or a
               paged cache, byte for byte.

Trees are arrays of parents: parent[b, i] < i, and -1 for a token that follows the
last committed one. A token at position -1 is padding.
"""
import math

import torch

own = False

NOPE, ROPE, DIM, HEADS = 448, 64, 512, 128
FP8_BYTES, FP4_BYTES = 592, 384
WINDOW = 128
THETA = 10000.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one user, a short context, eight drafted tokens: latency
        dict(name="tree_one_user", op="tree", kind="csa", fmt="fp8", B=1, N=8, cap=256, k=64, ctx=1024, tree="random",
             ragged=False, paged=False, inv=True),
        # eight sequences of 128K tokens, the 2048 best entries for each of eight drafts, 4-bit cache
        dict(name="tree_batch_128k", op="tree", kind="csa", fmt="fp4", B=8, N=8, cap=32768, k=2048, ctx=131072,
             tree="random", ragged=False, paged=True, inv=True),
        # lengths that differ, odd selection, thirteen nodes and padding, FP8 cache
        dict(name="tree_ragged", op="tree", kind="csa", fmt="fp8", B=6, N=13, cap=8192, k=517, ctx=32768,
             tree="forest", ragged=True, paged=True, inv=False),
        # wide trees at 1M tokens over every heavily compressed entry, 4-bit cache
        dict(name="tree_hca_1m", op="tree", kind="hca", fmt="fp4", B=4, N=32, cap=8192, k=0, ctx=1 << 20,
             tree="random", ragged=False, paged=True, inv=True),
        # chains of four drafts over every heavily compressed entry, FP8 cache
        dict(name="tree_hca_chain", op="tree", kind="hca", fmt="fp8", B=7, N=4, cap=2048, k=0, ctx=1 << 18,
             tree="chain", ragged=True, paged=False, inv=True),
        # one user's chain of drafts that have no probabilities (looked up in the prompt)
        dict(name="verify_one_user", op="verify", B=1, N=8, V=32000, tree="chain", dtype="bf16", q="", temp="one"),
        # a batch's chains against the draft model's probabilities
        dict(name="verify_chain", op="verify", B=32, N=6, V=131072, tree="chain", dtype="bf16", q="fp32", temp="one"),
        # trees whose siblings were drawn from the draft model, odd vocabulary, temperatures of their own
        dict(name="verify_tree_odd", op="verify", B=16, N=25, V=50001, tree="random", dtype="fp32", q="bf16",
             temp="mixed"),
        # large trees of the draft's best tokens for many users
        dict(name="verify_tree_large", op="verify", B=64, N=32, V=131072, tree="random", dtype="bf16", q="",
             temp="mixed"),
        # every sequence's accepted path into its sliding-window ring
        dict(name="commit_step", op="commit", fmt="fp4", B=32, N=8, cap=131, ring=True, page=32, last=131072),
        # long accepted drafts (text that repeats the prompt) into paged caches
        dict(name="commit_long", op="commit", fmt="fp8", B=64, N=128, cap=2048, ring=False, page=32, last=1900),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "verify", "verify", "commit"])
    tree = rng.choice(["chain", "random", "random", "forest"])
    if op == "commit":
        N = _log(rng, 1, 128)
        ring = rng.random() < 0.6
        cap = rng.randint(128, 160) if ring else rng.randint(N, 2048)
        return dict(op=op, fmt=rng.choice(["fp4", "fp8"]), B=_log(rng, 1, 64), N=N, cap=cap, ring=ring,
                    page=rng.choice([1, 32, 64]), last=_log(rng, 1, 131072) if ring else cap - N)
    if op == "verify":
        V = _log(rng, 700, 131072)
        B = _log(rng, 1, 64)
        N = _log(rng, 1, min(64, max(1, (1 << 28) // (B * V))))
        return dict(op=op, B=B, N=N, V=V, tree="random" if tree == "forest" else tree,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), q=rng.choice(["", "", "fp32", "bf16", "fp16"]),
                    temp=rng.choice(["one", "mixed"]))
    N = _log(rng, 1, 32)
    B = _log(rng, 1, max(1, 64 // N))
    case = dict(op=op, fmt=rng.choice(["fp4", "fp8"]), B=B, N=N, tree=tree, ragged=rng.random() < 0.6,
                paged=rng.random() < 0.6, inv=rng.random() < 0.5)
    if rng.random() < 0.6:
        cap = _log(rng, 40, 32768 if B * N <= 32 else 8192)
        return dict(case, kind="csa", cap=cap, k=min(cap, _log(rng, 1, 2048)), ctx=4 * cap)
    cap = _log(rng, 1, 8192)
    return dict(case, kind="hca", cap=cap, k=0, ctx=128 * cap)


def work(case):
    B, N = case["B"], case["N"]
    if case["op"] == "commit":
        moved = B * (N + 1) // 2 * (FP4_BYTES if case["fmt"] == "fp4" else FP8_BYTES)
        return dict(bytes=2 * moved, flops=0)
    if case["op"] == "verify":
        # the rows of the accepted path (two and a half on average), the draft's row where it ended, the noise
        rows = B * min(N, 2.5)
        size = {"bf16": 2, "fp16": 2, "fp32": 4}
        q = B * case["V"] * size[case["q"]] if case["q"] else 0
        return dict(bytes=int(rows * case["V"] * size[case["dtype"]] + q + 4 * B * case["V"]),
                    flops=int(rows * case["V"] * 4))
    rec = FP4_BYTES if case["fmt"] == "fp4" else FP8_BYTES
    rows, hca = B * N, case["kind"] == "hca"
    sel = min(case["cap"], case["ctx"] // 128) if hca else min(case["k"], case["ctx"] // 4)
    near = min(WINDOW, case["ctx"])
    if case["ragged"]:
        sel, rows = sel * 3 // 4, rows * 3 // 4
    # a sequence's tokens share the entries of HCA, the window and the drafts
    records = (B * sel if hca else rows * sel) + B * (near + N)
    return dict(bytes=records * rec + rows * (2 * HEADS * DIM * 2 + 4 * HEADS),
                flops=rows * (sel + near) * HEADS * DIM * 4)


# ---------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 6947 + 29)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)


def _randint(g, lo, hi, shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _random_records(g, n, fmt):
    """n records of about N(0,1) latents with a spread of magnitudes between them."""
    rope = _randn(g, n, ROPE).to(torch.bfloat16).view(torch.uint8)
    if fmt == "fp8":
        code = (_randn(g, n, NOPE) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        mult = (torch.exp(0.2 * _randn(g, n, 4)) / 100).view(torch.uint8)
        return torch.cat([code, rope, mult], 1)
    code = torch.randint(0, 256, (n, NOPE // 2), generator=g, device="cuda", dtype=torch.uint8)
    tail = torch.zeros((n, 32), dtype=torch.uint8, device="cuda")
    tail[:, :28] = (100 * torch.exp(0.2 * _randn(g, n, 28))).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8)
    tail[:, 28] = 119  # 2^-8
    return torch.cat([code, rope, tail], 1)


def _pages(g, B, n, page):
    """(block table, records in all): n logical entries a sequence in shuffled pages."""
    pages = -(-n // page)
    table = torch.randperm(B * pages, generator=g, device="cuda").to(torch.int32).view(B, pages).contiguous()
    return table, B * pages * page


def _tree(g, kind, B, N):
    """Parents [B, N]: a chain, a random tree under token 0, or several of them."""
    i = torch.arange(N, device="cuda", dtype=torch.int32)
    if kind == "chain":
        return (i - 1).expand(B, N).contiguous()
    back = (_rand(g, B, N) ** 2 * torch.clamp(i, max=12)).int()
    parent = i - 1 - torch.minimum(back, torch.clamp(i - 1, min=0))
    if kind == "forest":
        parent = torch.where(_rand(g, B, N) < 0.15, -1, parent)
    parent[:, 0] = -1
    return parent.to(torch.int32).contiguous()


def _depth(parent):
    depth = torch.zeros_like(parent)
    for i in range(parent.shape[1]):
        up = parent[:, i].long()
        depth[:, i] = torch.where(up < 0, 0, depth.gather(1, up.clamp(min=0)[:, None])[:, 0] + 1)
    return depth


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    B, N = case["B"], case["N"]
    if case["op"] == "commit":
        rec, cap = (FP4_BYTES if case["fmt"] == "fp4" else FP8_BYTES), case["cap"]
        s["table"], n = (None, B * cap) if case["ring"] else _pages(g, B, cap, case["page"])
        s["pool"] = torch.zeros((n, rec), dtype=torch.uint8, device="cuda")
        s["draft"] = _random_records(g, B * N, case["fmt"]).view(B, N, rec)
        # an accepted path is an ascending choice of nodes that begins with the root
        s["count"] = _randint(g, 1, N, (B,))
        order = torch.rand((B, N), generator=g, device="cuda")
        order[:, 0] = -1
        pick = order.argsort(dim=1).argsort(dim=1) < s["count"][:, None]
        node = torch.where(pick, torch.arange(N, device="cuda"), N).sort(dim=1).values
        s["path"] = torch.where(node < N, node, -1).to(torch.int32).contiguous()
        s["first"] = _randint(g, 0, case["last"], (B,))
        s["latents"] = torch.zeros((B, N, DIM), dtype=torch.bfloat16, device="cuda")
        if own:
            import compressed_sparse_decode_gb300 as csd
            s["cache"] = csd.cache_desc(s["pool"], cap, seq_stride=cap if case["ring"] else 0,
                                        block_table=s["table"], page_records=0 if case["ring"] else case["page"],
                                        fmt=csd.FORMAT_FP4 if case["fmt"] == "fp4" else csd.FORMAT_FP8)
        return s
    s["parent"] = _tree(g, case["tree"], B, N)
    if case["op"] == "verify":
        return _prepare_verify(s, case, g)
    cap, hca, fmt = case["cap"], case["kind"] == "hca", case["fmt"]
    m = 128 if hca else 4
    rec = FP4_BYTES if fmt == "fp4" else FP8_BYTES
    ctx = _randint(g, max(1, case["ctx"] // 2), case["ctx"], (B, 1)) if case["ragged"] else \
        torch.full((B, 1), case["ctx"], dtype=torch.int32, device="cuda")
    s["n_comp"] = torch.clamp(ctx[:, 0] // m, max=cap).to(torch.int32).contiguous()
    pos = ctx + _depth(s["parent"])
    if case["ragged"]:  # padding behind a sequence's own nodes
        live = _randint(g, max(1, N // 2), N, (B, 1))
        pos = torch.where(torch.arange(N, device="cuda") < live, pos, -1)
    s["pos"] = pos.to(torch.int32).contiguous()
    page = 1 if hca else 32
    s["table"], n = _pages(g, B, cap, page) if case["paged"] else (None, B * cap)
    s["page"] = page
    s["pool"] = _random_records(g, n, fmt)
    s["ring"] = _random_records(g, B * 160, fmt).view(B, 160, rec)
    s["draft"] = _random_records(g, B * N, fmt).view(B, N, rec)
    s["q"] = _randn(g, B, N, HEADS, DIM).to(torch.bfloat16)
    s["sink"] = _randn(g, HEADS)
    s["out"] = torch.zeros((B, N, HEADS, DIM), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros((B, N, HEADS), dtype=torch.float32, device="cuda")
    if not hca:
        # a random selection of the visible entries in ascending order, -1 behind it
        k = case["k"]
        vis = torch.minimum(s["pos"].clamp(min=0) // 4, s["n_comp"][:, None])
        key = torch.rand((B, N, cap), generator=g, device="cuda")
        key.masked_fill_(torch.arange(cap, device="cuda") >= vis[..., None], -1.0)
        top = key.topk(k, dim=-1)
        idx = torch.where(top.values >= 0, top.indices, cap).sort(dim=-1).values
        s["cnt"] = torch.clamp(vis, max=k).to(torch.int32).contiguous()
        s["idx"] = torch.where(idx < cap, idx, -1).to(torch.int32).contiguous()
    if own:
        import compressed_sparse_decode_gb300 as csd
        s["cache"] = csd.cache_desc(s["pool"], cap, seq_stride=0 if case["paged"] else cap, block_table=s["table"],
                                    page_records=page if case["paged"] else 0,
                                    fmt=csd.FORMAT_FP4 if fmt == "fp4" else csd.FORMAT_FP8)
        op = csd.OP_HCA_TREE_ATTENTION if hca else csd.OP_TREE_ATTENTION
        s["ws"] = csd.workspace(op, B, N, cap, case["k"], "cuda")
    return s


def _prepare_verify(s, c, g):
    """Target logits whose mass lies half on a few tokens of each row, drafts that
    agree with them more often than not."""
    B, N, V = c["B"], c["N"], c["V"]
    few = min(16, V)
    logits = torch.empty((B, N, V), dtype=DTYPES[c["dtype"]], device="cuda")
    draft = torch.empty((B, N, V), dtype=DTYPES[c["q"]], device="cuda") if c["q"] else None
    best = torch.empty((B, N, few), dtype=torch.long, device="cuda")
    drawn = torch.zeros((B, N), dtype=torch.long, device="cuda")
    level = math.log(V) + 2.0 + torch.linspace(4.0, -6.0, few, device="cuda")
    at = torch.arange(B, device="cuda")
    for i in range(N):
        row = 2.0 * _randn(g, B, V)
        best[:, i] = _rand(g, B, V).topk(few, dim=-1).indices
        top = level + 0.5 * _randn(g, B, few)
        row.scatter_(1, best[:, i], top)
        logits[:, i] = row.to(logits.dtype)
        if draft is not None:
            row = row + 1.2 * _randn(g, B, V)
            draft[:, i] = torch.softmax(row, -1).to(draft.dtype)
    ordinal = ((s["parent"][:, :, None] == s["parent"][:, None, :]) &
               (torch.arange(N, device="cuda")[None, None] < torch.arange(N, device="cuda")[None, :, None])).sum(-1)
    for i in range(N):
        up = s["parent"][:, i].long().clamp(min=0)
        if draft is None:  # the draft's best tokens, one for each sibling
            drawn[:, i] = torch.where(ordinal[:, i] < few, best[at, up, ordinal[:, i].clamp(max=few - 1)],
                                      torch.randint(0, V, (B,), generator=g, device="cuda"))
        else:  # a draw from the draft's distribution, for each sibling anew
            drawn[:, i] = (draft[at, up].float() / (-torch.log1p(-_rand(g, B, V))).clamp(min=1e-9)).argmax(-1)
    s["logits"], s["draft_probs"] = logits, draft
    s["tokens"] = drawn.to(torch.int32).contiguous()
    s["uniform"] = _rand(g, B, N)
    s["noise"] = (-torch.log1p(-_rand(g, B, V))).clamp(min=1e-9)
    s["temperature"] = None
    if c["temp"] == "mixed":  # about one in four takes the best token each time
        t = 0.5 + _rand(g, B)
        s["temperature"] = torch.where(_rand(g, B) < 0.25, 0.0, t).contiguous()
    if own:
        import compressed_sparse_decode_gb300 as csd
        s["ws"] = csd.workspace(csd.OP_VERIFY, B, N, V, 0, "cuda")
    return s


# ---------------------------------------------------------------- the pass


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"tree": _plain_tree, "verify": _plain_verify, "commit": _plain_commit}[case["op"]](state, case)


def _own(s, c):
    import compressed_sparse_decode_gb300 as csd
    if c["op"] == "commit":
        csd.csa_cache_commit(s["cache"], s["draft"], s["path"], s["count"], s["first"], ring=c["ring"])
        if c["fmt"] == "fp4":
            return csd.csa_cache_read(s["cache"], s["first"], s["count"], c["N"], ring=c["ring"], out=s["latents"])
        return _record_views(s["pool"])
    if c["op"] == "verify":
        return csd.csa_verify_drafts(s["logits"], s["tokens"], s["parent"], s["uniform"], s["noise"],
                                     temperature=s["temperature"], draft_probs=s["draft_probs"], ws=s["ws"])
    scale = DIM ** -0.5
    if c["kind"] == "csa":
        return csd.csa_tree_attention_decode(s["q"], s["sink"], scale, s["cache"], s["ring"], WINDOW, s["draft"],
                                             s["parent"], s["idx"], s["cnt"], s["pos"], out=s["out"], lse=s["lse"],
                                             ws=s["ws"], inverse_rope=c["inv"], rope_theta=THETA)
    return csd.hca_tree_attention_decode(s["q"], s["sink"], scale, s["cache"], s["n_comp"], s["ring"], WINDOW,
                                         s["draft"], s["parent"], s["pos"], 128, out=s["out"], lse=s["lse"],
                                         ws=s["ws"], inverse_rope=c["inv"], rope_theta=THETA)


def _record_views(pool):
    """FP8 records' codes, rope dims and multipliers, as they lie in them."""
    return [pool[:, :NOPE].view(torch.float8_e4m3fn), pool[:, NOPE:NOPE + 2 * ROPE].view(torch.bfloat16),
            pool[:, NOPE + 2 * ROPE:].view(torch.float32)]


# ---------------------------------------------------------------- plain forms


def _values(rec, fmt):
    """Records' bytes -> [..., 512] fp32."""
    if fmt == "fp8":
        code = rec[..., :NOPE].view(torch.float8_e4m3fn).float()
        mult = rec[..., 576:592].view(torch.float32).repeat_interleave(128, dim=-1)[..., :NOPE]
        return torch.cat([code * mult, rec[..., 448:576].view(torch.bfloat16).float()], -1)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=rec.device)
    packed = rec[..., :NOPE // 2]
    code = torch.stack([packed & 15, packed >> 4], -1).flatten(-2)
    unit = rec[..., 352:380].view(torch.float8_e4m3fn).float() * (rec[..., 380:381].int() << 23).view(torch.float32)
    nope = table[code.int()].unflatten(-1, (28, 16)) * unit[..., None]
    return torch.cat([nope.flatten(-2), rec[..., 224:352].view(torch.bfloat16).float()], -1)


def _at(s, c, entry):
    """Record numbers of logical entries [B, ...] of each sequence."""
    b = torch.arange(entry.shape[0], device=entry.device).view(-1, *[1] * (entry.dim() - 1))
    if s["table"] is None:
        return b * c["cap"] + entry
    page = s.get("page", c.get("page"))
    return s["table"][b, entry // page].long() * page + entry % page


def _turn_back(x, pos):
    """The last 64 dims as pairs (2i, 2i+1), pair i turned by -pos theta^(-2i/64) rad."""
    i = torch.arange(ROPE // 2, device=x.device, dtype=torch.float64)
    a = pos.double()[..., None, None] * THETA ** (-2 * i / ROPE)  # 64 bits: far positions
    cos, sin = a.cos().float(), a.sin().float()
    u, v = x[..., -ROPE::2], x[..., -ROPE + 1::2]
    return torch.cat([x[..., :-ROPE], torch.stack([u * cos + v * sin, v * cos - u * sin], -1).flatten(-2)], -1)


def _plain_tree(s, c):
    B, N, R, fmt = c["B"], c["N"], s["ring"].shape[1], c["fmt"]
    pos, q = s["pos"].long(), s["q"].float()
    # the chain of each token: itself, its parent, and so on
    node = torch.arange(N, device="cuda").expand(B, N)
    chain = []
    for _ in range(min(N, WINDOW)):
        chain.append(node)
        node = torch.where(node < 0, -1, s["parent"].long().gather(1, node.clamp(min=0)))
    length = torch.stack([a >= 0 for a in chain], -1).sum(-1)
    back = pos[..., None] - torch.arange(WINDOW, device="cuda")  # positions of the window
    committed = (torch.arange(WINDOW, device="cuda") >= length[..., None]) & (back >= 0)
    b = torch.arange(B, device="cuda")[:, None, None]
    near = _values(s["ring"], fmt)[b, back.clamp(min=0) % R]
    chain = torch.stack(chain, -1)
    drafted = _values(s["draft"], fmt)[b, chain.clamp(min=0)]
    x = torch.cat([near, drafted], 2)
    live = torch.cat([committed, chain >= 0], 2)
    z = torch.where(live[..., None, :], torch.matmul(q, x.transpose(-1, -2)) * DIM ** -0.5, -math.inf)
    if c["kind"] == "csa":
        sel = torch.arange(c["k"], device="cuda") < s["cnt"][..., None]
        far = _values(s["pool"][_at(s, c, s["idx"].long().clamp(min=0))], fmt)
    else:
        entry = torch.arange(c["cap"], device="cuda")
        sel = entry < torch.minimum(pos.clamp(min=0) // 128, s["n_comp"][:, None])[..., None]
        far = _values(s["pool"][_at(s, c, entry.expand(B, -1))], fmt)[:, None]  # shared by the tree
    zf = torch.where(sel[..., None, :], torch.matmul(q, far.transpose(-1, -2)) * DIM ** -0.5, -math.inf)
    sink = s["sink"][:, None]
    top = torch.maximum(torch.maximum(z.amax(-1, keepdim=True), zf.amax(-1, keepdim=True)), sink)
    w, wf = torch.exp(z - top), torch.exp(zf - top)
    den = w.sum(-1, keepdim=True) + wf.sum(-1, keepdim=True) + torch.exp(sink - top)
    o = (torch.matmul(w, x) + torch.matmul(wf, far)) / den
    if c["inv"]:
        o = _turn_back(o, pos)
    padding = pos < 0
    return (torch.where(padding[..., None, None], s["out"], o.to(torch.bfloat16)),
            torch.where(padding[..., None], s["lse"], (top + den.log())[..., 0]))


def _plain_verify(s, c):
    B, N, V = c["B"], c["N"], c["V"]
    dev = s["logits"].device
    at = torch.arange(B, device=dev)
    temp = torch.ones(B, device=dev) if s["temperature"] is None else s["temperature"]
    greedy = ~(temp > 0)
    x = s["logits"].float()
    top = x.amax(-1, keepdim=True)
    valid = torch.isfinite(top[..., 0])
    best = x.argmax(-1)
    e = torch.exp((x - top) / torch.where(greedy, 1.0, temp)[:, None, None])
    p = e / e.double().sum(-1, keepdim=True).float()  # 64 bits: a long sum
    cur = torch.zeros(B, dtype=torch.long, device=dev)
    path = torch.full((B, N), -1, dtype=torch.int32, device=dev)
    path[:, 0] = 0
    accepted = torch.ones(B, dtype=torch.int32, device=dev)
    left, mass = p[:, 0], torch.ones(B, device=dev)  # what the target has left, and its sum
    for i in range(1, N):
        child = s["parent"][:, i].long() == cur
        token = s["tokens"][:, i].long()
        q = s["draft_probs"][at, cur].float() if s["draft_probs"] is not None else None
        qx = q[at, token] if q is not None else torch.ones(B, device=dev)
        take = s["uniform"][:, i] * qx * mass < left[at, token]
        take = child & valid[at, cur] & torch.where(greedy, token == best[at, cur], take)
        refuse = child & ~take
        if q is not None:
            rest = left - mass[:, None] * q
        else:
            rest = left.clone()
            rest[at, token] = 0
        rest = torch.where(rest > 0, rest, 0)
        rest_mass = rest.double().sum(-1).float()  # 64 bits: a long sum
        cur = torch.where(take, i, cur)
        left = torch.where(take[:, None], p[:, i], torch.where(refuse[:, None], rest, left))
        mass = torch.where(take, 1.0, torch.where(refuse, rest_mass, mass))
        path[at, torch.where(take, accepted.long(), 0)] = torch.where(take, i, 0).int()
        accepted = accepted + take.int()
    left = torch.where((left > 0).any(-1)[:, None], left, p[at, cur])
    drawn = torch.where(left > 0, left / s["noise"], -1.0).argmax(-1)
    token = torch.where(greedy, best[at, cur], drawn)
    return path, accepted, torch.where(valid[at, cur], token, -1).int()


def _plain_commit(s, c):
    t = torch.arange(c["N"], device="cuda")[None]
    entry = s["first"][:, None].long() + t
    live = t < s["count"][:, None]
    b = torch.arange(c["B"], device="cuda")[:, None].expand_as(entry)
    if c["ring"]:
        slot = entry % c["cap"]
        live = live & (t >= s["count"][:, None] - c["cap"])
    else:
        slot = entry.clamp(max=c["cap"] - 1)
    at = _at(s, c, slot)
    s["pool"][at[live]] = s["draft"][b[live], s["path"].long()[live]]
    if c["fmt"] == "fp4":
        return torch.where(live[..., None], _values(s["pool"][at], "fp4").to(torch.bfloat16), s["latents"])
    return _record_views(s["pool"])


# ---------------------------------------------------------------- 64 bits


def _table_e4m3():
    """The values of the 256 E4M3 codes, from the format's definition."""
    v = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        mag = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        mag = math.nan if code & 127 == 127 else mag
        v.append(-mag if code & 128 else mag)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _two_to(e):
    """2^e for whole e, exactly (a power function may be a unit off)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(rec, fmt):
    """The 512 values of records, from their bytes."""
    r = rec.long()
    bits = r[..., -160:-32:2] + 256 * r[..., -159:-32:2] if fmt == "fp4" else r[..., 448:576:2] + 256 * r[..., 449:576:2]
    mag = torch.where((bits >> 7) % 256 == 0, (bits % 128).double() * 2.0 ** -133,
                      (1 + (bits % 128).double() / 128) * _two_to((bits >> 7) % 256 - 127))
    rope = torch.where(bits >= 32768, -mag, mag)
    e4m3 = _table_e4m3()
    d = torch.arange(NOPE, device=rec.device)
    if fmt == "fp8":
        mult = rec[..., 576:592].contiguous().view(torch.float32).double()
        nope = e4m3[r[..., :NOPE]] * mult[..., d // 128]
    else:
        code = (r[..., d // 2] >> (4 * (d % 2))) % 16
        grid = torch.tensor(E2M1, dtype=torch.float64, device=rec.device)
        nope = torch.where(code >= 8, -1.0, 1.0) * grid[code % 8] * e4m3[r[..., 352 + d // 16]] * \
            _two_to(r[..., 380:381] - 127)
    return torch.cat([nope, rope], -1)


def _place(s, c, b, entry):
    """Record numbers of entries of sequence b."""
    if s["table"] is None:
        return b * c["cap"] + entry
    page = s.get("page", c.get("page"))
    return s["table"][b].long()[entry // page] * page + entry % page


def exact(case, seed):
    s, c = prepare(case, seed), case
    return {"tree": _exact_tree, "verify": _exact_verify, "commit": _exact_commit}[c["op"]](s, c)


def _exact_tree(s, c):
    B, N, R, fmt = c["B"], c["N"], s["ring"].shape[1], c["fmt"]
    out = torch.zeros((B, N, HEADS, DIM), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, N, HEADS), dtype=torch.float64, device="cuda")
    freq = torch.tensor([THETA ** (-i / 32) for i in range(32)], dtype=torch.float64, device="cuda")
    parents, positions = s["parent"].tolist(), s["pos"].tolist()
    for b in range(B):
        ring, draft = _exact_values(s["ring"][b], fmt), _exact_values(s["draft"][b], fmt)
        everything = _exact_values(s["pool"][_place(s, c, b, torch.arange(c["cap"], device="cuda"))], fmt) \
            if c["kind"] == "hca" else None
        for i in range(N):
            p = positions[b][i]
            if p < 0:
                continue
            path = [i]
            while parents[b][path[-1]] >= 0:
                path.append(parents[b][path[-1]])
            oldest = max(0, p - WINDOW + 1)
            drafts = [n for d, n in enumerate(path) if p - d >= oldest]
            ringed = torch.arange(oldest, max(oldest, p - len(path) + 1), device="cuda") % R
            if c["kind"] == "csa":
                entry = s["idx"][b, i, :int(s["cnt"][b, i])].long()
                far = _exact_values(s["pool"][_place(s, c, b, entry)], fmt)
            else:
                far = everything[:min(p // 128, int(s["n_comp"][b]), c["cap"])]
            x = torch.cat([far, ring[ringed], draft[torch.tensor(drafts, device="cuda")]])
            z = torch.cat([s["sink"].double()[:, None], s["q"][b, i].double() @ x.T / math.sqrt(DIM)], 1)
            o = torch.softmax(z, 1)[:, 1:] @ x
            if c["inv"]:
                pair = torch.view_as_complex(o[:, NOPE:].unflatten(-1, (ROPE // 2, 2)).contiguous())
                o[:, NOPE:] = torch.view_as_real(pair * torch.polar(torch.ones_like(freq), -p * freq)).flatten(-2)
            out[b, i], lse[b, i] = o, torch.logsumexp(z, 1)
    return out, lse


def _exact_verify(s, c):
    B, N = c["B"], c["N"]
    path = torch.full((B, N), -1, dtype=torch.int32)
    accepted, following = torch.zeros(B, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    parents, tokens, uniform = s["parent"].tolist(), s["tokens"].tolist(), s["uniform"].double().tolist()
    for b in range(B):
        t = 1.0 if s["temperature"] is None else float(s["temperature"][b])
        node, n = 0, 0
        while True:
            path[b, n], n = node, n + 1
            x = s["logits"][b, node].double()
            p = torch.softmax(x / t, 0) if t > 0 else (torch.arange(c["V"], device="cuda") == x.argmax()).double()
            q = s["draft_probs"][b, node].double() if s["draft_probs"] is not None else None
            whole, mass, nxt = p, 1.0, -1
            for i in (j for j in range(node + 1, N) if parents[b][j] == node):
                v = tokens[b][i]
                if t > 0:
                    take = uniform[b][i] * (float(q[v]) if q is not None else 1.0) * mass < float(p[v])
                else:
                    take = float(p[v]) == 1.0
                if take:
                    nxt = i
                    break
                if t > 0:
                    hit = torch.zeros_like(p)
                    hit[v] = math.inf
                    p = (p - (mass * q if q is not None else hit)).clamp(min=0)
                    mass = float(p.sum())
            if nxt < 0:
                break
            node = nxt
        if not bool((p > 0).any()):
            p = whole
        accepted[b], following[b] = n, int((p / s["noise"][b].double()).argmax())
    return path.cuda(), accepted.cuda(), following.cuda()


def _exact_commit(s, c):
    B, N, cap = c["B"], c["N"], c["cap"]
    after, back = s["pool"].clone(), torch.zeros((B, N, DIM), dtype=torch.float64, device="cuda")
    for b in range(B):
        n, first = int(s["count"][b]), int(s["first"][b])
        for t in range(max(0, n - cap) if c["ring"] else 0, n):
            slot = (first + t) % cap if c["ring"] else first + t
            rec = s["draft"][b, int(s["path"][b, t])]
            after[int(_place(s, c, b, torch.tensor(slot, device="cuda")))] = rec
        if c["fmt"] == "fp4" and n:
            t = torch.arange(max(0, n - cap) if c["ring"] else 0, n, device="cuda")
            back[b, t] = _exact_values(s["draft"][b, s["path"][b, t].long()], "fp4")
    if c["fmt"] == "fp4":
        return back
    code = _table_e4m3()[after[:, :NOPE].long()]
    bits = after[:, 448:576:2].long() + 256 * after[:, 449:576:2].long()
    rope = (bits << 16).to(torch.int32).view(torch.float32).double()
    return [code, rope, after[:, 576:].contiguous().view(torch.float32).double()]
