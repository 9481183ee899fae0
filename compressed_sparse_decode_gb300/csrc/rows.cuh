// rows.cuh -- device helpers of the kernels that normalise, rotate, quantise
// and unpack rows of latents and heads (norm_rope.cu, cache.cu): eight
// consecutive values ("an octet") a lane, whatever the element type.
#pragma once

#include <cmath>

#include "common.cuh"
#include "ptx.cuh"

namespace csa {

constexpr int kFp4Bytes = CSA_FP4_RECORD_BYTES;
constexpr int kFp4RopeOffset = kNope / 2;                     // 224
constexpr int kFp4ScaleOffset = kFp4RopeOffset + 2 * kRope;   // 352
constexpr int kFp4Block = 16;
constexpr int kFp4Blocks = kNope / kFp4Block;                 // 28
constexpr int kFp4PowerOffset = kFp4ScaleOffset + kFp4Blocks; // 380
constexpr int kFp4MinExponent = -111;  // keeps every product code * scale * 2^E a normal number
constexpr int kMaxRopePairs = 128;

// Normalisation and rotation of a row, as the kernels take it. turn[i] is the
// angle of rope pair i per position in turns, as a 64-bit fixed-point
// fraction.
struct RowOps {
    const float *weight;
    float eps;
    int norm;
    int rope_dim;
    uint64_t turn[kMaxRopePairs];
};

inline bool finite_above(float v, float lo) { return std::isfinite(v) && v > lo; }

// Host side: the checks of csa_norm_rope for rows of D values, and its
// parameters. turn = theta^(-2i/rope_dim) / (2 pi) * 2^64 (below 2^62, so it
// fits).
inline bool make_row_ops(const csa_norm_rope *how, int D, RowOps *o) {
    if (!how) return false;
    o->norm = how->norm ? 1 : 0;
    o->weight = how->weight;
    o->eps = how->eps;
    o->rope_dim = how->rope_dim;
    if (!o->norm && how->weight) return false;
    if (reinterpret_cast<uintptr_t>(how->weight) & 15u) return false;
    if (o->norm && !(how->eps >= 0.f && std::isfinite(how->eps))) return false;
    if (how->rope_dim < 0 || how->rope_dim % 8 || how->rope_dim > D || how->rope_dim > 2 * kMaxRopePairs) return false;
    const int pairs = how->rope_dim / 2;
    if (pairs && !finite_above(how->rope_theta, 1.f)) return false;
    // the table of the last (theta, rope_dim) of this thread: 32 pow calls cost
    // more than the rest of a call
    struct Cached {
        float theta;
        int rope_dim;
        uint64_t turn[kMaxRopePairs];
    };
    static thread_local Cached c = {0.f, 0, {0}};
    if (pairs && (c.theta != how->rope_theta || c.rope_dim != how->rope_dim)) {
        for (int i = 0; i < pairs; ++i) {
            const double f = std::pow((double)how->rope_theta, -2.0 * i / how->rope_dim);
            c.turn[i] = (uint64_t)std::ldexp(f / 6.283185307179586476925287, 64);
        }
        c.theta = how->rope_theta;
        c.rope_dim = how->rope_dim;
    }
    for (int i = 0; i < pairs; ++i) o->turn[i] = c.turn[i];
    return true;
}

// cos and sin of position p's angle for a pair: p * turn modulo one turn is a
// 64-bit integer product, exact but for the fraction's own rounding (2^-65 of
// a turn a position), so far positions keep their angle and no double
// arithmetic runs (this GPU does two fp64 FMAs a clock and SM). The upper 32
// bits as a signed number are the angle in (-1/2, 1/2] turn; the special
// function unit's sine and cosine are off by about 4e-7 there.
__device__ __forceinline__ float2 turn_cos_sin(int64_t p, uint64_t turn) {
    const int32_t part = (int32_t)(((uint64_t)p * turn) >> 32);
    float sn, cs;
    __sincosf((float)part * 1.4629180792671596e-9f, &sn, &cs);  // 2 pi / 2^32
    return make_float2(cs, sn);
}

// Eight consecutive elements: loaded as 16-byte vectors, read as fp32. (Plain
// loads, not the read-only path: a row may be overwritten in place.)
template <int DT>
struct Octet;

template <>
struct Octet<CSA_BF16> {
    uint4 v;
    __device__ __forceinline__ void load(const void *base, int64_t at) {
        v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + at);
    }
    __device__ __forceinline__ void floats(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};

template <>
struct Octet<CSA_FP16> {
    uint4 v;
    __device__ __forceinline__ void load(const void *base, int64_t at) {
        v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + at);
    }
    __device__ __forceinline__ void floats(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        }
    }
};

template <>
struct Octet<CSA_FP32> {
    uint4 v, u;
    __device__ __forceinline__ void load(const void *base, int64_t at) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + at);
        v = p[0];
        u = p[1];
    }
    __device__ __forceinline__ void floats(float (&f)[8]) const {
        const uint32_t w[8] = {v.x, v.y, v.z, v.w, u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}

__device__ __forceinline__ uint4 pack_bf16_octet(const float (&f)[8]) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// Four values -> four E4M3 codes (round to nearest even, saturating; NaN kept).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Largest |f| of an octet as its bits: the order of the bits is the order of
// the magnitudes, and a NaN is above them all (a float maximum would drop it).
__device__ __forceinline__ uint32_t amax_bits(const float (&f)[8], uint32_t m = 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    return m;
}

// amax / 448 as a multiplier: 1 for an all-zero block.
__device__ __forceinline__ float e4m3_scale(uint32_t amax) {
    return amax ? __fdiv_rn(__uint_as_float(amax), 448.f) : 1.f;
}

// x / s correctly rounded for ordinary sizes, given inv = 1 / s (rounded):
// one Newton step on the quotient. A scale so small that 1 / s or the
// remainder leaves the normal range is divided by.
__device__ __forceinline__ float quotient(float x, float s, float inv) {
    if (s < 1e-30f) return __fdiv_rn(x, s);
    const float q = x * inv;
    return fmaf(fmaf(-q, s, x), inv, q);
}

// The same with a sticky last bit: if x / s is not a float, the result is the
// neighbour with an odd last bit on the true side, so a later rounding to a
// short format sees on which side of its halfway point the quotient lies.
__device__ __forceinline__ float sticky_quotient(float x, float s, float inv) {
    const float q = quotient(x, s, inv);
    const float r = fmaf(-q, s, x);  // exact
    if (r == 0.f || !(fabsf(q) < INFINITY)) return q;
    // away from zero when the remainder has q's sign, else towards it
    const uint32_t b = __float_as_uint(q);
    const bool up = (__float_as_uint(r) ^ b) >> 31 == 0;
    return __uint_as_float((up ? b : b - 1u) | 1u);
}

// y_d = x_d * inv_rms * w_d for one octet.
__device__ __forceinline__ void scale_octet(float (&f)[8], float inv_rms, const float *weight, int at) {
    if (weight) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(weight + at));
        const float4 b = __ldg(reinterpret_cast<const float4 *>(weight + at) + 1);
        const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * inv_rms * w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= inv_rms;
    }
}

// Turns the four pairs of an octet.
__device__ __forceinline__ void turn_octet(float (&f)[8], const float2 (&cs)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = f[2 * i], y = f[2 * i + 1];
        f[2 * i] = fmaf(x, cs[i].x, -y * cs[i].y);
        f[2 * i + 1] = fmaf(x, cs[i].y, y * cs[i].x);
    }
}

// 2^(byte - 127) of a 4-bit record (byte 0: the subnormal 2^-127; 255: infinity).
__device__ __forceinline__ float fp4_power(uint32_t byte) {
    return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// Launch configuration shared by these kernels: programmatic stream
// serialisation (a kernel may be set up while its predecessor drains; it
// waits for it before touching memory).
struct PdlLaunch {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg;
    PdlLaunch(dim3 grid, dim3 block, cudaStream_t stream) : cfg() {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = grid;
        cfg.blockDim = block;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    PdlLaunch(const PdlLaunch &) = delete;
    PdlLaunch &operator=(const PdlLaunch &) = delete;
};

}  // namespace csa
