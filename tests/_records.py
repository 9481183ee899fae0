"""Plain 64-bit restatement (numpy) of the row operators: norm, rotation, the
record formats and their quantisers, from the formulas in include/csa.h. Loops
over formats' tables, no code of the library."""
from __future__ import annotations

import numpy as np
import torch

NOPE, ROPE, DIM = 448, 64, 512
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def e4m3_table() -> np.ndarray:
    """The finite non-negative E4M3 values in the order of their codes 0..126."""
    return np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                     for e in range(16) for m in range(8)][:127])


E4M3 = e4m3_table()


def nearest_code(v, grid) -> np.ndarray:
    """Code of the grid value nearest to |v|, ties to the even code, saturating."""
    v = np.abs(np.asarray(v, dtype=np.float64))
    mid = (grid[1:] + grid[:-1]) / 2
    below, above = np.searchsorted(mid, v, side="left"), np.searchsorted(mid, v, side="right")
    return np.where(below % 2 == 0, below, above)  # equal unless v is a midpoint


def signed(code, v, grid, bit) -> np.ndarray:
    return (code + bit * np.signbit(v)).astype(np.uint8)


def norm_rope(x, pos, weight, eps, rope_dim, theta) -> np.ndarray:
    """x [..., D] float64, pos [...] -> normalised (weight not None) and rotated."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * weight
    if rope_dim:
        D = y.shape[-1]
        a = np.asarray(pos, dtype=np.float64)[..., None] * theta ** (-2.0 * np.arange(rope_dim // 2) / rope_dim)
        while a.ndim < y.ndim:
            a = a[..., None, :]
        u, v = y[..., D - rope_dim::2].copy(), y[..., D - rope_dim + 1::2].copy()
        y[..., D - rope_dim::2] = u * np.cos(a) - v * np.sin(a)
        y[..., D - rope_dim + 1::2] = u * np.sin(a) + v * np.cos(a)
    return y


def fp4_record(y):
    """y [512] float64 -> (codes [448], block scale codes [28], E)."""
    nope = np.asarray(y[:NOPE], dtype=np.float64)
    amax = np.abs(nope).max()
    E = 0
    if amax > 0:
        E = int(np.floor(np.log2(amax / 2688))) - 1
        while amax > 2688 * 2.0 ** E:
            E += 1
        E = max(E, -111)
    codes, scales = np.zeros(NOPE, np.uint8), np.zeros(28, np.uint8)
    for i in range(28):
        blk = nope[16 * i:16 * i + 16]
        # amax / 6 against the midpoints, without dividing
        s = int(nearest_code(np.abs(blk).max() * 2.0 ** -E, 6 * E4M3))
        scales[i] = s
        if s:
            unit = E4M3[s] * 2.0 ** E
            codes[16 * i:16 * i + 16] = signed(nearest_code(blk, E2M1 * unit), blk, None, 8)
    return codes, scales, E


def fp4_values(rec: np.ndarray) -> np.ndarray:
    """[n, 384] uint8 -> [n, 512] float64."""
    rec = np.asarray(rec)
    code = np.stack([rec[:, :224] & 15, rec[:, :224] >> 4], -1).reshape(len(rec), NOPE)
    val = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7]
    e4m3 = np.concatenate([E4M3, [np.nan]])
    sc = rec[:, 352:380]
    unit = np.where(sc >= 128, -1.0, 1.0) * e4m3[sc & 127]
    with np.errstate(invalid="ignore", over="ignore"):
        power = np.where(rec[:, 380] == 255, np.inf, 2.0 ** (rec[:, 380].astype(np.float64) - 127))
        nope = val * np.repeat(unit, 16, axis=1) * power[:, None]
    return np.concatenate([nope, bf16(rec[:, 224:352])], 1)


def fp8_values(rec: np.ndarray) -> np.ndarray:
    """[n, 592] uint8 -> [n, 512] float64."""
    rec = np.ascontiguousarray(rec)
    code = torch.from_numpy(rec[:, :NOPE].copy()).view(torch.float8_e4m3fn).double().numpy()
    mult = rec[:, 576:592].copy().view(np.float32).astype(np.float64)
    return np.concatenate([code * np.repeat(mult, 128, axis=1)[:, :NOPE], bf16(rec[:, 448:576])], 1)


def bf16(b: np.ndarray) -> np.ndarray:
    """[n, 128] bytes -> [n, 64] float64."""
    bits = b[:, 0::2].astype(np.uint32) | (b[:, 1::2].astype(np.uint32) << 8)
    return (bits << 16).view(np.float32).astype(np.float64)


def random_fp4_records(n: int, seed: int, spread: float = 1.0) -> torch.Tensor:
    """n records with random codes, block scales and rope dims around 1 (CPU uint8)."""
    g = torch.Generator().manual_seed(seed)
    rec = torch.zeros((n, 384), dtype=torch.uint8)
    rec[:, :224] = torch.randint(0, 256, (n, 224), generator=g, dtype=torch.uint8)
    rec[:, 224:352] = (torch.randn((n, 64), generator=g) * spread).to(torch.bfloat16).view(torch.uint8)
    rec[:, 352:380] = torch.randint(0x70, 0x7F, (n, 28), generator=g, dtype=torch.uint8)  # 128 .. 448
    rec[:, 380] = torch.randint(117, 120, (n,), generator=g, dtype=torch.uint8)  # 2^-10 .. 2^-8
    return rec
