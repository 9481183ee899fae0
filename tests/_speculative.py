"""Plain 64-bit restatement (numpy, CPU) of the speculative-decoding calls from the
formulas in include/csa.h: loops over sequences and tokens, no code of the library."""
from __future__ import annotations

import numpy as np
import torch

import _records as R

SCALE = 512 ** -0.5


def random_fp8_records(n: int, seed: int, spread: float = 1.0) -> torch.Tensor:
    """n records of about N(0, spread) latents (CPU uint8)."""
    g = torch.Generator().manual_seed(seed)
    code = (torch.randn((n, 448), generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    rope = (torch.randn((n, 64), generator=g) * spread).to(torch.bfloat16).view(torch.uint8)
    mult = (torch.exp(0.3 * torch.randn((n, 4), generator=g)) * (spread / 100)).view(torch.uint8)
    return torch.cat([code, rope, mult], 1)


def random_records(n: int, fmt: int, seed: int) -> torch.Tensor:
    return R.random_fp4_records(n, seed) if fmt else random_fp8_records(n, seed)


def values(rec: np.ndarray, fmt: int) -> np.ndarray:
    return R.fp4_values(rec) if fmt else R.fp8_values(rec)


def random_tree(kind: str, B: int, N: int, g: torch.Generator) -> torch.Tensor:
    """Parents [B, N]: "chain", "star" (all follow token 0), "random" or "forest"."""
    parent = torch.full((B, N), -1, dtype=torch.int32)
    for b in range(B):
        for i in range(1, N):
            if kind == "chain":
                parent[b, i] = i - 1
            elif kind == "random" or (kind == "forest" and float(torch.rand((), generator=g)) > 0.2):
                parent[b, i] = int(torch.randint(0, i, (), generator=g))
            elif kind == "star":
                parent[b, i] = 0
    return parent


def chain_of(parent, i: int) -> list:
    """Token i and its ancestors, the youngest first; a parent that is none ends it."""
    path = [i]
    while 0 <= int(parent[path[-1]]) < path[-1]:
        path.append(int(parent[path[-1]]))
    return path


def depths(parent: torch.Tensor) -> torch.Tensor:
    B, N = parent.shape
    return torch.tensor([[len(chain_of(parent[b], i)) - 1 for i in range(N)] for b in range(B)], dtype=torch.int32)


def window(ring: np.ndarray, draft: np.ndarray, parent, i: int, p: int, W: int, fmt: int) -> np.ndarray:
    """Latents of the window of token i at position p: ring [R, bytes], draft [N, bytes]."""
    path = chain_of(parent, i)
    rec = []
    for pos in range(max(0, p - W + 1), p + 1):
        back = p - pos
        rec.append(draft[path[back]] if back < len(path) else ring[pos % len(ring)])
    return values(np.stack(rec), fmt)


def attend(q, sink, x):
    """Definition of the attention in 64 bits -> (o, lse, weighted magnitude A of what is
    summed, largest sum of |q x| of a score times the scale)."""
    z = SCALE * (q @ x.T)
    M = np.maximum(sink, z.max(1, initial=-np.inf))
    M0 = np.where(np.isneginf(M), 0.0, M)
    with np.errstate(divide="ignore"):
        p = np.exp(z - M0[:, None])
        den = p.sum(1) + np.exp(sink - M0)
        lse = M0 + np.log(den)
    d = np.where(den > 0, den, 1.0)[:, None]
    size = SCALE * (np.abs(q) @ np.abs(x).T).max(1, initial=0.0)
    return p @ x / d, lse, p @ np.abs(x) / d, size


def turn_back(o, p, theta):
    o = o.copy()
    a = p * theta ** (-2.0 * np.arange(32) / 64)
    u, v = o[:, 448::2].copy(), o[:, 449::2].copy()
    o[:, 448::2] = u * np.cos(a) + v * np.sin(a)
    o[:, 449::2] = -u * np.sin(a) + v * np.cos(a)
    return o


def verify(logits, token, parent, uniform, noise, t=1.0, draft=None):
    """One sequence: logits [N, V], token, parent, uniform [N], noise [V], draft [N, V] or
    None, all numpy. Returns (path, next token, smallest relative margin of a decision)."""
    N, V = logits.shape
    path, margin, node = [], np.inf, 0

    def near(a, b):
        return abs(a - b) / max(abs(a), abs(b), 1e-300)

    while True:
        path.append(node)
        z = logits[node].astype(np.float64)
        top = z.max()
        if not np.isfinite(top):
            return path, -1, margin
        kids = [i for i in range(node + 1, N) if parent[i] == node]
        if not t > 0:
            best = int(np.argmax(z))
            hit = [i for i in kids if token[i] == best]
            if not hit:
                return path, best, margin
            node = hit[0]
            continue
        with np.errstate(over="ignore", under="ignore"):
            w = np.where(np.isneginf(z), 0.0, np.exp((z - top) / np.float64(t)))
        p = w / w.sum()
        r, mass, nxt = p.copy(), 1.0, None
        for i in kids:
            x = int(token[i])
            if not 0 <= x < V:
                continue
            q = float(draft[node, x]) if draft is not None else 1.0
            a = float(uniform[i]) * q * mass
            if a > 0 or r[x] > 0:
                margin = min(margin, near(a, r[x]))
            if a < r[x]:
                nxt = i
                break
            if draft is not None:
                full = r - mass * draft[node].astype(np.float64)
                r = np.where(full > 0, full, 0.0)
            else:
                r[x] = 0.0
            mass = r.sum()
        if nxt is not None:
            node = nxt
            continue
        if not (r > 0).any():
            r = p
        ratio = np.where(r > 0, r / noise.astype(np.float64), -1.0)
        best = int(np.argmax(ratio))
        rest = np.delete(ratio, best)
        if rest.size and rest.max() > 0:
            margin = min(margin, near(ratio[best], rest.max()))
        return path, best, margin
