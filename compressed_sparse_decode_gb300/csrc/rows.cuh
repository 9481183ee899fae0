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
// fits), to the nearest whole number: in long double, since a double's own 53 bits
// would leave the 64-bit fraction wrong by hundreds of units (2^-56 of a turn a
// position, 0.009 radians at position 2^47).
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
    if (!pairs) return true;
    // the tables of this thread's last four (theta, rope_dim), since a model's layers
    // may take turns with theirs (a pow of 113 bits for each pair of a table made in
    // every call took 47 us; its ratio alone, and products, 2 us)
    struct Cached {
        float theta;
        int rope_dim;
        uint64_t turn[kMaxRopePairs];
    };
    constexpr int kTables = 4;
    static thread_local Cached tables[kTables] = {};
    static thread_local int oldest = 0;
    int at = 0;
    while (at < kTables && (tables[at].theta != how->rope_theta || tables[at].rope_dim != how->rope_dim)) ++at;
    if (at == kTables) {
        at = oldest;
        oldest = (oldest + 1) % kTables;
        Cached &c = tables[at];
        const long double two_pi = 8 * std::atan(1.0L);
        const long double ratio = std::pow((long double)how->rope_theta, -2.0L / how->rope_dim);
        long double f = std::ldexp(1 / two_pi, 64);
        for (int i = 0; i < pairs; ++i, f *= ratio) c.turn[i] = (uint64_t)(f + 0.5L);
        c.theta = how->rope_theta;
        c.rope_dim = how->rope_dim;
    }
    for (int i = 0; i < pairs; ++i) o->turn[i] = tables[at].turn[i];
    return true;
}

// cos and sin of position p's angle for a pair: p * turn modulo one turn is a
// 64-bit integer product, exact but for the fraction's own rounding (2^-65 of
// a turn a position), so far positions keep their angle and no double
// arithmetic runs (this GPU does two fp64 FMAs a clock and SM). The upper 32
// bits are taken to the nearest quarter turn; on the rest, |x| <= pi / 4, the
// Taylor polynomials to x^9 and x^10 are within 4e-9 and 2e-10 of sine and
// cosine, below the fp32 rounding of the sum (the special function unit's are
// off by 4e-7, which changes an E4M3 code now and then).
__device__ __forceinline__ float2 turn_cos_sin(int64_t p, uint64_t turn) {
    const uint32_t part = (uint32_t)(((uint64_t)p * turn) >> 32);
    const uint32_t quarter = (part + 0x20000000u) >> 30;  // modulo 4
    const float x = (float)(int32_t)(part - (quarter << 30)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    const float y = x * x;
    float s = fmaf(y, 1.f / 362880.f, -1.f / 5040.f), c = fmaf(y, -1.f / 3628800.f, 1.f / 40320.f);
    s = fmaf(s, y, 1.f / 120.f);
    c = fmaf(c, y, -1.f / 720.f);
    s = fmaf(s, y, -1.f / 6.f);
    c = fmaf(c, y, 1.f / 24.f);
    s = fmaf(s * y, x, x);
    c = fmaf(c, y, -0.5f);
    c = fmaf(c, y, 1.f);
    const float cs = (quarter & 1u) ? s : c, sn = (quarter & 1u) ? c : s;
    return make_float2((quarter + 1u) & 2u ? -cs : cs, quarter & 2u ? -sn : sn);
}

// Eight consecutive elements: loaded as 16-byte vectors, read as fp32. (Plain
// loads, not the read-only path: a row may be overwritten in place.)
template <int DT>
struct Octet;

template <>
struct Octet<CSA_BF16> {
    uint4 v;
    __device__ __forceinline__ void clear() { v = make_uint4(0, 0, 0, 0); }
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
    __device__ __forceinline__ void clear() { v = make_uint4(0, 0, 0, 0); }
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
    __device__ __forceinline__ void clear() { v = u = make_uint4(0, 0, 0, 0); }
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

// Largest |f| of an octet, NaN if one is (a plain maximum would drop it).
__device__ __forceinline__ float amax_octet(const float (&f)[8], float m = 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(f[i])));
    return m;
}
// As bits, whose order is that of the magnitudes, with NaN above them all.
__device__ __forceinline__ uint32_t amax_bits(float amax) { return __float_as_uint(amax) & 0x7FFFFFFFu; }

// x / s to one of the two floats around it (itself if it is one), given inv = 1 / s
// rounded: the quotient's residual r = x - q s, exact in an FMA, corrects it (P. W.
// Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", IBM J. Res. Dev. 34, 1990). s is in the middle of the range (see
// fp4_codes).
__device__ __forceinline__ float quotient(float x, float s, float inv) {
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

// amax / 448 as a multiplier: 1 for an all-zero block.
__device__ __forceinline__ float e4m3_scale(uint32_t amax) {
    return amax ? quotient(__uint_as_float(amax), 448.f, 1.f / 448.f) : 1.f;
}

// 448 f / amax for the E4M3 codes of an octet. With a Newton step (kExact) a quotient
// that is a halfway point of the codes comes out as that, and for values with up to
// 21 bits (448 f is exact) every other on its own side of it, so the codes of 16-bit
// inputs are those of the exact quotients. Others go without: values that a norm has
// rounded already, and fp32 inputs as they are, whose 448 f would round too. Their
// quotient is within two roundings, 2^-23, of the exact one, so that a value that
// near to a halfway point, where either code is half a step off, may take either.
// (All times a power of two where a product or remainder would leave the range.)
template <bool kExact>
__device__ __forceinline__ void e4m3_quotients(const float (&f)[8], uint32_t amax, float (&q)[8]) {
    float up = 1.f;
    if (amax < 0x0DA24260u) up = 1.152921504606846976e18f;  // below 1e-30: 2^60
    if (amax > 0x7149F2CAu) up = 8.673617379884035e-19f;    // above 1e30: 2^-60
    const float t = amax ? __uint_as_float(amax) * up : 448.f, inv = __frcp_rn(t);
    const float2 k = make_float2(448.f * up, 448.f * up), ii = make_float2(inv, inv), tt = make_float2(-t, -t);
    const float2 quick = make_float2(quotient(448.f, t, inv), quotient(448.f, t, inv));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float2 x = make_float2(f[2 * e], f[2 * e + 1]);
        if (kExact) {
            x = __fmul2_rn(x, k);
            const float2 a = __fmul2_rn(x, ii);
            x = __ffma2_rn(__ffma2_rn(a, tt, x), ii, a);
        } else {
            x = __fmul2_rn(x, quick);
        }
        q[2 * e] = x.x;
        q[2 * e + 1] = x.y;
    }
    if (!kExact && up != 1.f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] *= up;
    }
}

// Sum of the squares of an octet, added to two running sums.
__device__ __forceinline__ void square_octet(const float (&f)[8], float2 &sum) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 v = make_float2(f[2 * e], f[2 * e + 1]);
        sum = __ffma2_rn(v, v, sum);
    }
}

// The norm's weights of an octet (ones without any).
__device__ __forceinline__ void load_weights(float (&w)[8], const float *weight, int at) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.f;
    if (!weight) return;
    const float4 a = __ldg(reinterpret_cast<const float4 *>(weight + at));
    const float4 b = __ldg(reinterpret_cast<const float4 *>(weight + at) + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}

// (mean + eps)^(-1/2) with a Newton step (the function's 2 ulp would be half of a
// normalised value's error, which decides E4M3 codes): e = 1 - a r^2, with what
// a r loses kept. Where a r^2 has no value (a zero or infinite) r stays.
__device__ __forceinline__ float inverse_rms(float sum, float inv_d, float eps) {
    const float a = fmaf(sum, inv_d, eps), r = rsqrtf(a);
    const float p = a * r, lost = fmaf(a, r, -p);
    const float e = fmaf(-lost, r, fmaf(-p, r, 1.f));
    return fabsf(e) < 1e-3f ? fmaf(0.5f * r, e, r) : r;
}

// y_d = x_d * inv_rms * w_d for one octet.
__device__ __forceinline__ void scale_octet(float (&f)[8], float inv_rms, const float (&w)[8]) {
    const float2 r = make_float2(inv_rms, inv_rms);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 v = __fmul2_rn(__fmul2_rn(make_float2(f[2 * e], f[2 * e + 1]), r), make_float2(w[2 * e], w[2 * e + 1]));
        f[2 * e] = v.x;
        f[2 * e + 1] = v.y;
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
