"""The query, cache and 4-bit attention operators of the decode library: plain
forms, the library's own calls, and the cases they are measured on.

Four operators, used together around one decode step of a layer:

* ``norm_rope``   RMS norm of every head with the position rotation in the same
                  pass; BF16 output for the attention, E4M3 codes with a scale
                  per head for the indexer.
* ``append``      new latents (and the entries' indexer keys) into a paged or
                  ring cache of FP8 or 4-bit records, normalised and rotated on
                  the way.
* ``read``        a range of entries of such a cache back as BF16 latents.
* ``attention``   sink-merged attention over a cache of 4-bit records: top-k
                  entries and the sliding window (CSA), or every visible entry
                  and the window (HCA).

A 4-bit record (384 bytes) holds 448 E2M1 codes (dim 2i in the low nibble of
byte i), 64 BF16 rope dims, 28 E4M3 scales of 16 dims each, one power-of-two
multiplier (E8M0) and 3 zero bytes.
"""
import math

import torch

own = False

NOPE, ROPE, DIM, HEADS, IDX_DIM = 448, 64, 512, 128, 128
FP8_BYTES, FP4_BYTES = 592, 384
WINDOW = 128
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E2M1_EDGES = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # halfway points of the values above


def listed():
    return [
        # one user's single new token: all query heads of a layer, latency alone
        dict(name="query_one_token", op="norm_rope", B=1, T=1, H=128, D=512, dtype="bf16", out="bf16", norm=True,
             theta=10000.0, last=1024, padded=False, sliced=False),
        # a prompt chunk's query heads, a slice of a fused projection, an odd token count, padded rows
        dict(name="query_prompt", op="norm_rope", B=4, T=1027, H=128, D=512, dtype="bf16", out="bf16", norm=True,
             theta=10000.0, last=131072, padded=True, sliced=True),
        # indexer queries of a batched step with several tokens a sequence, at a far position
        dict(name="indexer_query_step", op="norm_rope", B=32, T=4, H=64, D=128, dtype="bf16", out="e4m3", norm=False,
             theta=10000.0, last=1 << 20, padded=False, sliced=False),
        # every sequence's new token into the sliding-window ring, 4-bit, read back as the window
        dict(name="append_step_fp4", op="append", fmt="fp4", B=32, T=1, cap=128, ring=True, paged=False, page=32,
             dtype="bf16", norm=True, idx=False, pos_stride=1, ragged=False, theta=10000.0, last=131072),
        # the compressed entries and indexer keys of eight prompts of up to 32K tokens, paged FP8
        dict(name="append_prompt_fp8", op="append", fmt="fp8", B=8, T=8192, cap=8192, ring=False, paged=True, page=32,
             dtype="bf16", norm=True, idx=True, pos_stride=4, ragged=True, theta=10000.0, last=0),
        # compressed entries in 32 bits from the compressor, odd counts, paged 4-bit with indexer keys
        dict(name="append_entries_fp4", op="append", fmt="fp4", B=16, T=1001, cap=4096, ring=False, paged=True,
             page=32, dtype="fp32", norm=False, idx=True, pos_stride=4, ragged=True, theta=10000.0, last=2048),
        # a batch's sliding windows back as latents
        dict(name="read_window_fp4", op="read", fmt="fp4", B=32, T=128, cap=131, ring=True, paged=False, page=32,
             ragged=False, last=131072),
        # eight prompts' compressed entries back as latents (a cache that moves to another format)
        dict(name="read_prompt_fp8", op="read", fmt="fp8", B=8, T=8192, cap=8192, ring=False, paged=True, page=32,
             ragged=True, last=0),
        # one user, a short context: latency
        dict(name="csa_one_user", op="attention", kind="csa", B=1, T=1, cap=256, k=64, ctx=1024, ragged=False,
             paged=False, inv=True),
        # the benchmark's step: 32 sequences of 128K tokens, the 2048 best entries and the window
        dict(name="csa_batch_128k", op="attention", kind="csa", B=32, T=1, cap=32768, k=2048, ctx=131072, ragged=False,
             paged=True, inv=True),
        # four tokens a sequence (speculative decoding), lengths that differ, odd selection
        dict(name="csa_tokens_ragged", op="attention", kind="csa", B=6, T=4, cap=8192, k=517, ctx=32768, ragged=True,
             paged=True, inv=False),
        # 64 sequences at 1M tokens over every heavily compressed entry
        dict(name="hca_batch_1m", op="attention", kind="hca", B=64, T=1, cap=8192, k=0, ctx=1 << 20, ragged=False,
             paged=True, inv=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "read", "attention", "attention"])
    if op == "norm_rope":
        e4m3 = rng.random() < 0.4
        D = 128 if e4m3 else rng.choice([64, 128, 192, 256, 512])
        H = rng.choice([1, 2, 8, 37, 64, 128])
        tokens = _log(rng, 1, 4096)
        B = min(tokens, _log(rng, 1, 64))
        return dict(op=op, B=B, T=max(1, tokens // B), H=H, D=D, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    out="e4m3" if e4m3 else "bf16", norm=rng.random() < 0.7, theta=rng.choice([10000.0, 1000000.0]),
                    last=_log(rng, 64, 1 << 20), padded=rng.random() < 0.5, sliced=rng.random() < 0.5)
    if op in ("append", "read"):
        B = _log(rng, 1, 64)
        T = _log(rng, 1, min(8192, 65536 // B))
        ring = rng.random() < 0.4
        cap = rng.randint(128, 160) if ring else T + rng.randint(0, 300)
        case = dict(op=op, fmt=rng.choice(["fp4", "fp8"]), B=B, T=T, cap=cap, ring=ring,
                    paged=not ring and rng.random() < 0.7, page=rng.choice([1, 32, 64]), ragged=rng.random() < 0.6,
                    last=_log(rng, 1, 131072) if ring else cap - T)
        if op == "append":
            # long prompts come normalised by the layer's own pass where they are kept in 4 bits
            case.update(dtype=rng.choice(["bf16", "fp16", "fp32"]), norm=rng.random() < 0.6 and
                        (case["fmt"] == "fp8" or B * T <= 256), idx=not ring and rng.random() < 0.6,
                        pos_stride=1 if ring else rng.choice([4, 128]), theta=rng.choice([10000.0, 1000000.0]))
        else:
            case["T"] = min(T, cap)
        return case
    if rng.random() < 0.6:
        T = rng.choice([1, 1, 2, 3, 4, 8])
        B = _log(rng, 1, 64 // T)
        cap = _log(rng, 40, 32768 if B * T <= 32 else 8192)
        return dict(op=op, kind="csa", B=B, T=T, cap=cap, k=min(cap, _log(rng, 1, 2048)), ctx=4 * cap,
                    ragged=rng.random() < 0.6, paged=rng.random() < 0.6, inv=rng.random() < 0.5)
    B, cap = _log(rng, 1, 64), _log(rng, 1, 8192)
    return dict(op=op, kind="hca", B=B, T=1, cap=cap, k=0, ctx=128 * cap, ragged=rng.random() < 0.6,
                paged=rng.random() < 0.6, inv=rng.random() < 0.5)


def work(case):
    if case["op"] == "norm_rope":
        n = case["B"] * case["T"] * case["H"]
        size = 4 if case["dtype"] == "fp32" else 2
        out = case["D"] * 2 if case["out"] == "bf16" else case["D"] + 4
        return dict(bytes=n * (case["D"] * size + out), flops=n * case["D"] * 6)
    rec = FP4_BYTES if case.get("fmt") == "fp4" else FP8_BYTES
    if case["op"] in ("append", "read"):
        n = case["B"] * case["T"]
        if case["ragged"]:
            n = n * 3 // 4
        if case["op"] == "read":
            return dict(bytes=n * (rec + 2 * DIM), flops=n * DIM)
        size = 4 if case["dtype"] == "fp32" else 2
        kept = min(n, case["B"] * case["cap"])
        b = kept * (DIM * size + rec)
        if case["idx"]:
            b += kept * (IDX_DIM * size + IDX_DIM + 4)
        if case["fmt"] == "fp4":  # the written entries read back as latents
            b += kept * (FP4_BYTES + 2 * DIM)
        return dict(bytes=b, flops=kept * DIM * 8)
    rows = case["B"] * case["T"]
    sel = min(case["k"], case["ctx"] // 4) if case["kind"] == "csa" else min(case["cap"], case["ctx"] // 128)
    if case["ragged"]:
        sel = sel * 3 // 4
    n = sel + min(WINDOW, case["ctx"])
    return dict(bytes=rows * (n * FP4_BYTES + 2 * HEADS * DIM * 2 + 4 * HEADS), flops=rows * n * HEADS * DIM * 4)


# ---------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _randint(g, lo, hi, shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _random_records(g, n, fmt):
    """n records of N(0,1) latents with a spread of magnitudes between records."""
    parts = []
    for s in range(0, n, 1 << 16):
        m = min(n, s + (1 << 16)) - s
        x = (_randn(g, m, DIM) * torch.exp(0.2 * _randn(g, m, 1))).to(torch.bfloat16).float()
        nope = _fp4_bytes(x[:, :NOPE]) if fmt == "fp4" else _fp8_bytes(x[:, :NOPE])
        rope = x[:, NOPE:].to(torch.bfloat16).view(torch.uint8)
        parts.append(torch.cat([nope[0], rope, nope[1]], 1))
    return torch.cat(parts)


def _pages(g, case, n):
    """(records, block table or None, records a sequence): n logical entries for
    each sequence, in shuffled pages or one after the other."""
    B = case["B"]
    if not case["paged"]:
        return B * n, None
    page = case.get("page", 32)
    pages = -(-n // page)
    table = torch.randperm(B * pages, generator=g, device="cuda").to(torch.int32).view(B, pages).contiguous()
    return B * pages * page, table


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    B, T = case["B"], case["T"]
    if case["op"] == "norm_rope":
        H, D, dt = case["H"], case["D"], DTYPES[case["dtype"]]
        wide = _randn(g, B, T, H * D + (256 if case["sliced"] else 0)) * torch.exp(0.3 * _randn(g, B, T, 1))
        wide = wide.to(dt)
        s["x"] = wide[..., :H * D].unflatten(-1, (H, D))
        s["weight"] = 1 + 0.1 * _randn(g, D) if case["norm"] else None
        first = _randint(g, 0, case["last"], (B, 1))
        pos = first + torch.arange(T, device="cuda", dtype=torch.int32)
        if case["padded"]:
            live = _randint(g, max(1, T // 2), T, (B, 1))
            pos = torch.where(torch.arange(T, device="cuda")[None] < live, pos, -1)
        s["pos"] = pos.to(torch.int32).contiguous()
        if case["out"] == "bf16":
            s["out"] = torch.zeros((B, T, H, D), dtype=torch.bfloat16, device="cuda")
        else:
            s["codes"] = torch.zeros((B, T, H, D), dtype=torch.uint8, device="cuda")
            s["scale"] = torch.zeros((B, T, H), dtype=torch.float32, device="cuda")
        return s
    if case["op"] in ("append", "read"):
        rec = FP4_BYTES if case["fmt"] == "fp4" else FP8_BYTES
        cap = case["cap"]
        n, s["table"] = _pages(g, case, cap)
        s["pool"] = _random_records(g, n, case["fmt"]) if case["op"] == "read" else \
            torch.zeros((n, rec), dtype=torch.uint8, device="cuda")
        s["first"] = _randint(g, 0, case["last"], (B,))
        s["count"] = _randint(g, T // 2, T, (B,)) if case["ragged"] else torch.full((B,), T, dtype=torch.int32,
                                                                                    device="cuda")
        s["latents"] = torch.zeros((B, T, DIM), dtype=torch.bfloat16, device="cuda")
        if case["op"] == "append":
            dt = DTYPES[case["dtype"]]
            s["x"] = (_randn(g, B, T, DIM) * torch.exp(0.3 * _randn(g, B, T, 1))).to(dt)
            s["weight"] = 1 + 0.1 * _randn(g, DIM) if case["norm"] else None
            if case["idx"]:
                s["key"] = _randn(g, B, T, IDX_DIM).to(dt)
                s["k_idx"] = torch.zeros((B, cap, IDX_DIM), dtype=torch.uint8, device="cuda")
                s["k_idx_scale"] = torch.zeros((B, cap), dtype=torch.float32, device="cuda")
        if own:
            import compressed_sparse_decode_gb300 as csd
            fmt = csd.FORMAT_FP4 if case["fmt"] == "fp4" else csd.FORMAT_FP8
            s["cache"] = csd.cache_desc(s["pool"], cap, seq_stride=0 if case["paged"] else cap,
                                        block_table=s["table"], page_records=case["page"] if case["paged"] else 0,
                                        fmt=fmt)
        return s
    cap, hca = case["cap"], case["kind"] == "hca"
    m = 128 if hca else 4
    ctx = _randint(g, case["ctx"] // 2, case["ctx"], (B, 1)) if case["ragged"] else \
        torch.full((B, 1), case["ctx"], dtype=torch.int32, device="cuda")
    s["pos"] = (ctx + torch.arange(T, device="cuda", dtype=torch.int32)).contiguous()
    s["n_comp"] = torch.clamp(ctx[:, 0] // m, max=cap).to(torch.int32).contiguous()
    n, s["table"] = _pages(g, dict(case, page=1 if hca else 32), cap)
    s["pool"] = _random_records(g, n, "fp4")
    R = WINDOW + T - 1
    s["ring"] = _random_records(g, B * R, "fp4").view(B, R, FP4_BYTES)
    s["q"] = _randn(g, B, T, HEADS, DIM).to(torch.bfloat16)
    s["sink"] = _randn(g, HEADS)
    s["out"] = torch.empty((B, T, HEADS, DIM), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty((B, T, HEADS), dtype=torch.float32, device="cuda")
    if not hca:
        # a random selection of the visible entries in ascending order, -1 behind it
        k = case["k"]
        vis = torch.minimum(s["pos"] // 4, s["n_comp"][:, None])
        key = torch.rand((B, T, cap), generator=g, device="cuda")
        key.masked_fill_(torch.arange(cap, device="cuda") >= vis[..., None], -1.0)
        top = key.topk(k, dim=-1)
        idx = torch.where(top.values >= 0, top.indices, cap).sort(dim=-1).values
        s["cnt"] = torch.clamp(vis, max=k).to(torch.int32).contiguous()
        s["idx"] = torch.where(idx < cap, idx, -1).to(torch.int32).contiguous()
    if own:
        import compressed_sparse_decode_gb300 as csd
        s["cache"] = csd.cache_desc(s["pool"], cap, seq_stride=0 if case["paged"] else cap, block_table=s["table"],
                                    page_records=(1 if hca else 32) if case["paged"] else 0, fmt=csd.FORMAT_FP4)
        op = csd.OP_HCA_ATTENTION if hca else csd.OP_ATTENTION
        s["ws"] = csd.workspace(op, B, T, cap, case["k"], "cuda")
    return s


# ---------------------------------------------------------------- the pass


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"norm_rope": _plain_norm_rope, "append": _plain_append, "read": _plain_read,
            "attention": _plain_attention}[case["op"]](state, case)


def _own(s, c):
    import compressed_sparse_decode_gb300 as csd
    if c["op"] == "norm_rope":
        if c["out"] == "bf16":
            return csd.csa_head_norm_rope(s["x"], s["pos"], weight=s["weight"], norm=c["norm"], eps=EPS,
                                          rope_dim=ROPE, rope_theta=c["theta"], out=s["out"])
        codes, scale = csd.csa_head_norm_rope_e4m3(s["x"], s["pos"], weight=s["weight"], norm=c["norm"], eps=EPS,
                                                   rope_dim=ROPE, rope_theta=c["theta"], codes=s["codes"],
                                                   scale=s["scale"])
        return codes.view(torch.float8_e4m3fn), scale
    if c["op"] == "append":
        idx = dict(key=s["key"], k_idx=s["k_idx"], k_idx_scale=s["k_idx_scale"]) if c["idx"] else {}
        csd.csa_cache_append(s["cache"], s["x"], s["first"], s["count"], ring=c["ring"], norm=c["norm"],
                             weight=s["weight"], eps=EPS, rope_theta=c["theta"], pos_stride=c["pos_stride"], **idx)
        if c["fmt"] == "fp4":
            first, count, T = s["first"], s["count"], c["T"]
            return _with_index(s, c, [csd.csa_cache_read(s["cache"], first, count, T, ring=c["ring"],
                                                         out=s["latents"])])
        return _with_index(s, c, _record_views(s["pool"]))
    if c["op"] == "read":
        return csd.csa_cache_read(s["cache"], s["first"], s["count"], c["T"], ring=c["ring"], out=s["latents"])
    scale = DIM ** -0.5
    if c["kind"] == "csa":
        return csd.csa_sink_attention_decode_fp4(s["q"], s["sink"], scale, s["cache"], s["ring"], WINDOW, s["idx"],
                                                 s["cnt"], s["pos"], out=s["out"], lse=s["lse"], ws=s["ws"],
                                                 inverse_rope=c["inv"], rope_theta=10000.0)
    return csd.hca_sink_attention_decode_fp4(s["q"], s["sink"], scale, s["cache"], s["n_comp"], s["ring"], WINDOW,
                                             s["pos"], 128, out=s["out"], lse=s["lse"], ws=s["ws"],
                                             inverse_rope=c["inv"], rope_theta=10000.0)


def _record_views(pool):
    """An FP8 cache's codes, rope dims and multipliers, as they lie in the records."""
    return [pool[:, :NOPE].view(torch.float8_e4m3fn), pool[:, NOPE:NOPE + 2 * ROPE].view(torch.bfloat16),
            pool[:, NOPE + 2 * ROPE:].view(torch.float32)]


def _with_index(s, c, outs):
    if c["idx"]:
        outs = outs + [s["k_idx"].view(torch.float8_e4m3fn), s["k_idx_scale"]]
    return outs


# ---------------------------------------------------------------- plain forms


def _rotate(x, pos, theta):
    """The last 64 dims as pairs (2i, 2i+1), pair i turned by pos theta^(-2i/64) rad."""
    i = torch.arange(ROPE // 2, device=x.device, dtype=torch.float64)
    a = pos.double()[..., None] * theta ** (-2 * i / ROPE)  # 64 bits: far positions
    cos, sin = a.cos().float(), a.sin().float()
    if x.dim() == pos.dim() + 2:
        cos, sin = cos.unsqueeze(-2), sin.unsqueeze(-2)
    u, v = x[..., -ROPE::2], x[..., -ROPE + 1::2]
    turned = torch.stack([u * cos - v * sin, u * sin + v * cos], dim=-1).flatten(-2)
    return torch.cat([x[..., :-ROPE], turned], dim=-1)


def _rms(x, weight):
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return y * weight


def _e4m3(x):
    """(codes as E4M3, one scale for the last dim): scale = amax / 448, 1 where all is zero."""
    amax = x.abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn), scale[..., 0]


def _power(byte):
    """2^(byte - 127), from its bits."""
    return (byte.int() << 23).view(torch.float32)


def _fp8_bytes(nope):
    """[n, 448] fp32 -> (code bytes, multiplier bytes)."""
    blocks = torch.nn.functional.pad(nope, (0, 64)).unflatten(-1, (4, 128))
    codes, scale = _e4m3(blocks)
    return codes.flatten(-2)[..., :NOPE].view(torch.uint8), scale.contiguous().view(torch.uint8)


def _fp4_bytes(nope):
    """[n, 448] fp32 -> (code bytes, bytes of the 28 scales, the power of two and padding)."""
    n = nope.shape[0]
    amax = nope.abs().amax(-1)
    mant, ex = torch.frexp(amax)  # mant in [0.5, 1): amax = 2 mant 2^(ex - 1)
    e = ex - 1 - 11 + (2 * mant > 1.3125).int()  # the smallest e with amax <= 6 448 2^e
    e = torch.where(amax > 0, e.clamp(min=-111), 0)
    two = _power(e + 127).double()[:, None]
    blocks = nope.double().unflatten(-1, (28, 16))  # 64 bits: values next to a border
    sb = (blocks.abs().amax(-1) / 6 / two).clamp(max=448).float().to(torch.float8_e4m3fn)
    unit = (sb.double() * two)[..., None]
    r = torch.where(unit > 0, blocks.abs() / torch.where(unit > 0, unit, 1), torch.zeros_like(blocks))
    code = torch.zeros_like(r, dtype=torch.int32)
    edges = torch.tensor(E2M1_EDGES, device=r.device, dtype=torch.float64)
    code = torch.bucketize(r, edges, right=False).int()  # an edge itself falls below
    tie = (r[..., None] == edges[1::2]).any(-1)  # edges whose even neighbour is the one above
    code = code + tie.int() + ((blocks < 0) & (unit > 0)).int() * 8
    code = code.flatten(-2)
    packed = (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)
    tail = torch.zeros((n, 32), dtype=torch.uint8, device=nope.device)
    tail[:, :28] = sb.view(torch.uint8)
    tail[:, 28] = (e + 127).to(torch.uint8)
    return packed, tail


def _fp4_values(rec):
    """[..., 384] bytes -> [..., 512] fp32."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=rec.device)
    packed = rec[..., :NOPE // 2]
    code = torch.stack([packed & 15, packed >> 4], -1).flatten(-2)
    unit = rec[..., 352:380].view(torch.float8_e4m3fn).float() * _power(rec[..., 380:381].int())
    nope = table[code.int()].unflatten(-1, (28, 16)) * unit[..., None]
    return torch.cat([nope.flatten(-2), rec[..., 224:352].view(torch.bfloat16).float()], -1)


def _fp8_values(rec):
    """[..., 592] bytes -> [..., 512] fp32."""
    code = rec[..., :NOPE].view(torch.float8_e4m3fn).float()
    mult = rec[..., 576:592].view(torch.float32).repeat_interleave(128, dim=-1)[..., :NOPE]
    return torch.cat([code * mult, rec[..., 448:576].view(torch.bfloat16).float()], -1)


def _records(s, c, entry):
    """Record numbers of logical entries [B, n] of each sequence."""
    b = torch.arange(entry.shape[0], device=entry.device)[:, None]
    if s["table"] is None:
        return b * c["cap"] + entry
    page = c.get("page", 1 if c.get("kind") == "hca" else 32)
    return s["table"][b, entry // page].long() * page + entry % page


def _plain_norm_rope(s, c):
    x = s["x"].float()
    y = _rms(x, s["weight"]) if c["norm"] else x
    y = _rotate(y, s["pos"], c["theta"])
    live = (s["pos"] >= 0)[..., None, None]
    if c["out"] == "bf16":
        return torch.where(live, y.to(torch.bfloat16), s["out"])
    codes, scale = _e4m3(y)
    return (torch.where(live, codes.view(torch.uint8), s["codes"]).view(torch.float8_e4m3fn),
            torch.where(live[..., 0], scale, s["scale"]))


def _range(s, c):
    """(logical slot [B, T], whether token t of sequence b counts)."""
    t = torch.arange(c["T"], device="cuda")[None]
    entry = s["first"][:, None].long() + t
    live = t < s["count"][:, None]
    if c["ring"]:
        return entry, entry % c["cap"], live & (t >= s["count"][:, None] - c["cap"])
    return entry, entry, live


def _plain_append(s, c):
    entry, slot, live = _range(s, c)
    x = s["x"].float()
    if c["norm"]:
        x = _rms(x, s["weight"])
    pos = entry * c["pos_stride"]
    y = _rotate(x, pos, c["theta"])
    y = y[live]
    nope = _fp4_bytes(y[:, :NOPE]) if c["fmt"] == "fp4" else _fp8_bytes(y[:, :NOPE])
    rope = y[:, NOPE:].to(torch.bfloat16).view(torch.uint8)
    s["pool"][_records(s, c, slot.clamp(max=c["cap"] - 1))[live]] = torch.cat([nope[0], rope, nope[1]], 1)
    if c["idx"]:
        codes, scale = _e4m3(_rotate(s["key"].float(), pos, c["theta"])[live])
        b = torch.arange(c["B"], device="cuda")[:, None].expand_as(slot)[live]
        s["k_idx"][b, slot[live]] = codes.view(torch.uint8)
        s["k_idx_scale"][b, slot[live]] = scale
    if c["fmt"] == "fp4":
        return _with_index(s, c, [_plain_read(s, c)])
    return _with_index(s, c, _record_views(s["pool"]))


def _plain_read(s, c):
    _, slot, live = _range(s, c)
    rec = s["pool"][_records(s, c, slot.clamp(max=c["cap"] - 1))]
    x = _fp4_values(rec) if c["fmt"] == "fp4" else _fp8_values(rec)
    return torch.where(live[..., None], x.to(torch.bfloat16), s["latents"])


def _candidates(s, c):
    """(records [B, T, n, 384], which of them count [B, T, n])."""
    B, T, R = c["B"], c["T"], s["ring"].shape[1]
    if c["kind"] == "csa":
        n = c["k"]
        entry = s["idx"].long()
        live = torch.arange(n, device="cuda") < s["cnt"][..., None]
    else:
        n = c["cap"]
        entry = torch.arange(n, device="cuda").expand(B, T, n)
        live = entry < torch.minimum(s["pos"] // 128, s["n_comp"][:, None])[..., None]
    at = _records(s, c, entry.clamp(min=0).reshape(B, T * n)).view(B, T, n)
    back = s["pos"][..., None].long() - torch.arange(WINDOW - 1, -1, -1, device="cuda")
    slot = back.clamp(min=0) % R
    near = s["ring"][torch.arange(B, device="cuda")[:, None, None], slot]
    return torch.cat([s["pool"][at], near], 2), torch.cat([live, back >= 0], 2)


def _plain_attention(s, c):
    rec, live = _candidates(s, c)
    x = _fp4_values(rec)
    z = torch.matmul(s["q"].float(), x.transpose(-1, -2)) * DIM ** -0.5
    z = torch.where(live[..., None, :], z, -math.inf)
    sink = s["sink"][:, None]
    top = torch.maximum(z.amax(-1, keepdim=True), sink)
    p = torch.exp(z - top)
    den = p.sum(-1, keepdim=True) + torch.exp(sink - top)
    o = torch.matmul(p, x) / den
    if c["inv"]:
        o = _rotate(o, -s["pos"], 10000.0)
    return o.to(torch.bfloat16), (top + den.log())[..., 0]


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


def _nearest(x, grid):
    """x >= 0 on an ascending grid whose first value is even, ties to the even place, saturating."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    lo = hi - 1
    down, up = x - grid[lo], grid[hi] - x
    take_up = (up < down) | ((up == down) & (hi % 2 == 0))
    return grid[torch.where(take_up, hi, lo)]


def _exact_turn(x, pos, theta):
    """Rotation of the last 64 dims as a product with unit complex numbers."""
    z = torch.view_as_complex(x[..., -ROPE:].unflatten(-1, (ROPE // 2, 2)).contiguous())
    freq = torch.tensor([theta ** (-i / 32) for i in range(32)], dtype=torch.float64, device=x.device)
    angle = pos.double()[..., None] * freq
    w = torch.polar(torch.ones_like(angle), angle)
    while w.dim() < z.dim():
        w = w.unsqueeze(-2)
    x = x.clone()
    x[..., -ROPE:] = torch.view_as_real(z * w).flatten(-2)
    return x


def _exact_norm(x, weight):
    return x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()


def _exact_e4m3(x):
    """(values on the E4M3 grid, scale) of x over its last dim."""
    top = x.abs().max(-1, keepdim=True).values
    scale = torch.where(top == 0, 1.0, top / 448)
    return x.sign() * _nearest((x / scale).abs(), _table_e4m3()[:127]), scale[..., 0]


def _two_to(e):
    """2^e for whole e, exactly (a power function may be a unit off)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_nope4(y):
    """[n, 448] -> the values that its 4-bit record stands for."""
    top = y.abs().max(-1).values
    e = torch.log2(top.clamp(min=2.0 ** -140)) - math.log2(2688)
    e = torch.ceil(e)  # then corrected against the definition: the smallest e with top <= 2688 2^e
    e = torch.where(top <= 2688 * _two_to(e - 1), e - 1, torch.where(top > 2688 * _two_to(e), e + 1, e))
    two = torch.where(top > 0, _two_to(e.clamp(min=-111)), 1.0)[:, None]
    blocks = y.view(-1, 28, 16)
    sb = _nearest(blocks.abs().max(-1).values / (6 * two), _table_e4m3()[:127])
    unit = (sb * two)[..., None]
    grid = torch.tensor(E2M1, dtype=torch.float64, device=y.device)
    code = _nearest(torch.where(unit > 0, blocks.abs() / unit.clamp(min=2.0 ** -300), 0.0), grid)
    return (blocks.sign() * code * unit).view(-1, NOPE)


def _exact_record(rec, fmt):
    """The 512 values of records, from their bytes."""
    r = rec.long()
    bits = r[..., -160:-32:2] + 256 * r[..., -159:-32:2] if fmt == "fp4" else r[..., 448:576:2] + 256 * r[..., 449:576:2]
    mag = torch.where((bits >> 7) % 256 == 0, (bits % 128) * 2.0 ** -133,
                      (1 + (bits % 128) / 128.0).double() * _two_to((bits >> 7) % 256 - 127))
    rope = torch.where(bits >= 32768, -mag, mag)
    e4m3 = _table_e4m3()
    if fmt == "fp8":
        mult = rec[..., 576:592].contiguous().view(torch.float32).double()
        nope = e4m3[r[..., :NOPE]] * mult[..., torch.arange(NOPE, device=rec.device) // 128]
    else:
        grid = torch.tensor(E2M1, dtype=torch.float64, device=rec.device)
        d = torch.arange(NOPE, device=rec.device)
        code = (r[..., d // 2] >> (4 * (d % 2))) % 16
        value = torch.where(code >= 8, -1.0, 1.0) * grid[code % 8]
        nope = value * e4m3[r[..., 352 + d // 16]] * _two_to(r[..., 380:381] - 127)
    return torch.cat([nope, rope], -1)


def _where(s, c, b, entry):
    """Record numbers of entries of sequence b."""
    if s["table"] is None:
        return b * c["cap"] + entry
    page = c.get("page", 1 if c.get("kind") == "hca" else 32)
    return s["table"][b].long()[entry // page] * page + entry % page


def _spans(s, c):
    """For each sequence: (tokens that count, their entries, their slots)."""
    for b in range(c["B"]):
        f, n = int(s["first"][b]), int(s["count"][b])
        t = torch.arange(max(0, n - c["cap"]) if c["ring"] else 0, n, device="cuda")
        yield b, t, f + t, (f + t) % c["cap"] if c["ring"] else f + t


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "norm_rope":
        y = s["x"].double()
        if c["norm"]:
            y = _exact_norm(y, s["weight"])
        y = _exact_turn(y, s["pos"], c["theta"])
        live = s["pos"] >= 0
        if c["out"] == "bf16":
            return y * live[..., None, None]
        value, scale = _exact_e4m3(y)
        return value * live[..., None, None], scale * live[..., None]
    if c["op"] == "read":
        out = torch.zeros((c["B"], c["T"], DIM), dtype=torch.float64, device="cuda")
        for b, t, _, slot in _spans(s, c):
            out[b, t] = _exact_record(s["pool"][_where(s, c, b, slot)], c["fmt"])
        return out
    if c["op"] == "append":
        back = torch.zeros((c["B"], c["T"], DIM), dtype=torch.float64, device="cuda")
        code = torch.zeros((s["pool"].shape[0], NOPE), dtype=torch.float64, device="cuda")
        rope = torch.zeros((s["pool"].shape[0], ROPE), dtype=torch.float64, device="cuda")
        mult = torch.zeros((s["pool"].shape[0], 4), dtype=torch.float64, device="cuda")
        keys = torch.zeros((c["B"], c["cap"], IDX_DIM), dtype=torch.float64, device="cuda")
        key_scale = torch.zeros((c["B"], c["cap"]), dtype=torch.float64, device="cuda")
        for b, t, entry, slot in _spans(s, c):
            x = s["x"][b, t].double()
            if c["norm"]:
                x = _exact_norm(x, s["weight"])
            turned = _exact_turn(x, entry * c["pos_stride"], c["theta"])
            y = turned[:, :NOPE]
            at = _where(s, c, b, slot)
            if c["fmt"] == "fp4":
                back[b, t] = torch.cat([_exact_nope4(y), turned[:, NOPE:]], -1)
            else:
                parts = [_exact_e4m3(p) for p in y.split(128, dim=-1)]
                code[at] = torch.cat([p[0] for p in parts], -1)
                mult[at] = torch.stack([p[1] for p in parts], -1)
                rope[at] = turned[:, NOPE:]
            if c["idx"]:
                keys[b, slot], key_scale[b, slot] = _exact_e4m3(
                    _exact_turn(s["key"][b, t].double(), entry * c["pos_stride"], c["theta"]))
        outs = [back] if c["fmt"] == "fp4" else [code, rope, mult]
        return outs + [keys, key_scale] if c["idx"] else outs
    B, T, R = c["B"], c["T"], s["ring"].shape[1]
    out = torch.zeros((B, T, HEADS, DIM), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, T, HEADS), dtype=torch.float64, device="cuda")
    for b in range(B):
        for t in range(T):
            p = int(s["pos"][b, t])
            if c["kind"] == "csa":
                entry = s["idx"][b, t, :int(s["cnt"][b, t])].long()
            else:
                entry = torch.arange(min(p // 128, int(s["n_comp"][b]), c["cap"]), device="cuda")
            near = torch.arange(max(0, p - WINDOW + 1), p + 1, device="cuda") % R
            x = _exact_record(torch.cat([s["pool"][_where(s, c, b, entry)], s["ring"][b, near]]), "fp4")
            z = s["q"][b, t].double() @ x.T / math.sqrt(DIM)
            z = torch.cat([s["sink"].double()[:, None], z], 1)
            w = torch.softmax(z, 1)
            out[b, t], lse[b, t] = w[:, 1:] @ x, torch.logsumexp(z, 1)
            if c["inv"]:
                out[b, t] = _exact_turn(out[b, t], torch.tensor(-p, device="cuda"), 10000.0)
    return out, lse
