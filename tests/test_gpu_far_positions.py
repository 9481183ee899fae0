"""Rotation at positions up to the largest that a call can ask for (entry 2^31 - 1
times a stride of 65536: 2^47), against angles computed with 80 decimal digits.

Tolerance, derived before the first run: a pair's fraction of a turn is a 64-bit
number, half a unit off at most, so position p has its angle to p * 2^-65 turns; the
product is cut at 2^-32 turns; sine and cosine are within 2 u of their angle's and
the two products and the sum each round once (u = 2^-24, at most 4 u of |a| + |b|
together); the BF16 result is half a step off, 2^-8 of the value. So a value of the
pair (a, b) may be off by (2 pi (p 2^-65 + 2^-32) + 6 u) (|a| + |b|), and by 2^-8 of
what comes of that."""
import decimal
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
THETAS = [10000.0, 500000.0, 1.5, 1e30]
U, BF16 = 2.0 ** -24, 2.0 ** -8


def angles(p, theta, rope_dim):
    """p * theta^(-2i/rope_dim) modulo a turn, in radians (float64), for positions p."""
    with decimal.localcontext() as c:
        c.prec = 80
        base = decimal.Decimal(float(np.float32(theta)))
        out = []
        for i in range(rope_dim // 2):
            turn = (base.ln() * (decimal.Decimal(-2 * i) / rope_dim)).exp() / (2 * PI)
            out.append([float((int(v) * turn) % 1 * 2 * PI) for v in p])
    return np.array(out).T


def check(got, x, p, theta, rope_dim, what):
    """got, x [n, rope_dim] float64: the rotated and the given values at positions p."""
    a = angles(p, theta, rope_dim)
    u, v = x[:, 0::2], x[:, 1::2]
    want = np.stack([u * np.cos(a) - v * np.sin(a), u * np.sin(a) + v * np.cos(a)], -1).reshape(x.shape)
    pair = np.repeat(np.abs(u) + np.abs(v), 2, axis=1)
    off = (2 * math.pi * (np.asarray(p, dtype=np.float64) * 2.0 ** -65 + 2.0 ** -32) + 6 * U)[:, None] * pair
    bound = off + BF16 * (np.abs(want) + off)
    worst = (np.abs(got - want) / bound).max()
    assert worst <= 1, f"{what}: {worst:.3g} x bound"


@pytest.mark.parametrize("theta", THETAS)
@pytest.mark.parametrize("pos_stride", [1, 4, 65536])
@pytest.mark.parametrize("fmt", [0, 1])
def test_append_far_entries(cuda_lib, fmt, pos_stride, theta):
    csd = cuda_lib
    B, T, cap = 12, 5, 7
    g = torch.Generator(device="cuda").manual_seed(pos_stride + fmt)
    x = torch.randn((B, T, 512), generator=g, device="cuda")
    first = torch.randint(1 << 24, (1 << 31) - T, (B,), generator=g, device="cuda").to(torch.int32)
    first[0] = 2147483647 - T + 1
    pool = torch.zeros((B * cap, csd.FORMAT_BYTES[fmt]), dtype=torch.uint8, device="cuda")
    ring = csd.cache_desc(pool, cap, seq_stride=cap, fmt=fmt)
    csd.csa_cache_append(ring, x, first, ring=True, rope_theta=theta, pos_stride=pos_stride)
    got = csd.csa_cache_read(ring, first, None, T, ring=True)
    p = [(int(e) + t) * pos_stride for e in first.tolist() for t in range(T)]
    check(got[..., 448:].double().cpu().numpy().reshape(-1, 64), x[..., 448:].double().cpu().numpy().reshape(-1, 64), p,
          theta, 64, f"entries {min(p)} .. {max(p)}")
    assert csd.csa_read_device_error() == 0


@pytest.mark.parametrize("theta", THETAS)
@pytest.mark.parametrize("rope_dim", [64, 200])
def test_heads_at_far_positions(cuda_lib, rope_dim, theta):
    csd = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(rope_dim)
    pos = torch.randint(1 << 24, 1 << 31, (2, 9), generator=g, device="cuda").to(torch.int32)
    pos[1, 8], pos[0, 0] = 2147483647, 0
    x = torch.randn((2, 9, 1, 200), generator=g, device="cuda")
    out = csd.csa_head_norm_rope(x, pos, norm=False, rope_dim=rope_dim, rope_theta=theta)
    check(out[..., 200 - rope_dim:].double().cpu().numpy().reshape(-1, rope_dim),
          x[..., 200 - rope_dim:].double().cpu().numpy().reshape(-1, rope_dim), pos.view(-1).tolist(), theta, rope_dim,
          "heads")


def test_calls_that_take_turns_with_their_bases(cuda_lib):
    """More (base, rope_dim) pairs than are kept: each call has its own."""
    csd = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((1, 3, 2, 72), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.tensor([[7, 100003, 1999999]], dtype=torch.int32, device="cuda")
    hows = [(t, r) for t in (10000.0, 160000.0, 1e6) for r in (64, 8, 0)]
    alone = []
    for i in range(3):
        for theta, rope in hows:
            out = csd.csa_head_norm_rope(x, pos, norm=False, rope_dim=rope, rope_theta=theta)
            if i == 0:
                alone.append(out)
                if rope:
                    check(out[..., 72 - rope:].double().cpu().numpy().reshape(-1, rope),
                          x[..., 72 - rope:].double().cpu().numpy().reshape(-1, rope),
                          [p for p in pos.view(-1).tolist() for _ in range(2)], theta, rope, f"{theta} {rope}")
            else:
                assert torch.equal(out, alone[hows.index((theta, rope))])
