// cache.cu -- writing latents into a cache and reading them back
// (csa_cache_append, csa_cache_read), and whole records into it (csa_cache_commit): FP8 and
// 4-bit records, contiguous, paged or ring.
//
// One warp a token (several, one after the other, in large calls); lane l holds
// dims [16 l, 16 l + 16): lanes 0..27 the nope dims (one 4-bit scale block each,
// eight lanes an FP8 block), lanes 28..31 the rope dims. So the 4-bit block
// maximum needs no shuffle, and a record is written with one vector store a lane.
//
// Appending is bound by instructions: 8 x up to 8192 tokens, normalised, into FP8
// records with indexer keys take 480 instructions a token, two thirds of the issue
// slots, 31 us (97 MB: 0.46 of the measured copy rate); 16 x 1001 FP32 tokens into 4-bit
// records 15 us; one token of 32 sequences 2.5 us, a launch. Reading 8 x up to 8192
// FP8 records back: 77 MB in 18.0 us, 0.63 of the copy rate.
#include <cuda_fp4.h>

#include "rows.cuh"

namespace csa {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kNopeLanes = kNope / 16;  // 28
constexpr uint32_t kAll = 0xffffffffu;

// Which entry token t of sequence b is.
struct Span {
    CacheView cache;
    int ring;
    const int32_t *first, *count;
    int B, T;
};

struct Slot {
    int64_t entry;   // first + t
    int64_t record;  // -1: the token does not count, or its entry is outside the cache
};

// Slot of token t of sequence b. Reports what lies outside the cache.
__device__ __forceinline__ Slot find_slot(const Span &s, int b, int t, int *err) {
    Slot o = {0, -1};
    int n = s.count ? __ldg(s.count + b) : s.T;
    const int first = __ldg(s.first + b);
    if (n < 0 || n > s.T) {
        if (t == 0) report_error(err, CSA_ERR_BAD_INDEX);
        n = n < 0 ? 0 : s.T;
    }
    if (t >= n) return o;
    o.entry = (int64_t)first + t;
    int64_t slot = o.entry;
    if (s.ring) {
        if (t < n - s.cache.seq_capacity) return o;  // overwritten by a later token of this call
        if (first >= 0) slot = o.entry % s.cache.seq_capacity;
    }
    if (first >= 0 && slot < s.cache.seq_capacity) o.record = record_index(s.cache, b, (int)slot);
    if (o.record < 0) report_error(err, CSA_ERR_BAD_INDEX);
    return o;
}

// A warp's tokens [t0, t0 + n): lane j looks token t0 + j up, all at once.
__device__ __forceinline__ Slot find_slots(const Span &s, int t0, int n, int lane, int *err) {
    const int token = t0 + lane;
    Slot o = {0, -1};
    if (lane < n && token < s.B * s.T) o = find_slot(s, token / s.T, token % s.T, err);
    return o;
}
// Tokens a warp: as many as leave every SM eight blocks, up to `most`. (A warp's
// tokens share the look-up, the norm's weights and the rotation's table, and the
// next one's loads run under the current one. Reading has less to share: 49k FP8
// records took 19.5 us with one, 17.9 with two, 18.3 with four, 19.0 with eight.)
constexpr int kAppendTokens = 8, kReadTokens = 2;
int tokens_per_warp(int tokens, int most) {
    const int n = tokens / (cached_sm_count() * 8 * kWarps);
    return n < 1 ? 1 : n > most ? most : n;
}

struct AppendParams {
    Span span;
    const void *x;
    int64_t seq_stride, token_stride;
    int pos_stride;
    RowOps ops;
    uint8_t *base;
    const void *key;  // indexer keys, or null
    int64_t key_seq_stride, key_token_stride;
    uint8_t *k_idx;
    float *k_idx_scale;
    int idx_cap;
    int per_warp;
    int *err;
};

// 16 values of a nope lane as E2M1 codes of unit s = sb * 2^E (4 significant
// bits). A quotient of a 16-bit input is a halfway point of the codes or 2^-12 of
// it away, so rounding it to fp32 decides nothing; other values need the sticky
// bit. (s is at least 2^-69 and the values of its size: the caller has multiplied
// tiny ones by 2^64, so that the remainders stay normal numbers.)
template <bool kSticky>
__device__ __forceinline__ uint2 fp4_codes(const float (&f)[2][8], float s) {
    uint32_t w[2];
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = kSticky ? sticky_quotient(f[o][e], s, inv) : quotient(f[o][e], s, inv);
        w[o] = e2m1x4(q[0], q[1], q[2], q[3]) | (e2m1x4(q[4], q[5], q[6], q[7]) << 16);
    }
    return make_uint2(w[0], w[1]);
}

// Exponent of a 4-bit record: the smallest E with amax <= 6 * 448 * 2^E =
// 1.3125 * 2^(E + 11), from the bits of amax; at least kFp4MinExponent.
__device__ __forceinline__ int fp4_exponent(uint32_t amax) {
    const int ex = (int)(amax >> 23) - 127;
    const int e = ex - 11 + ((amax & 0x7FFFFFu) > 0x280000u ? 1 : 0);  // 0.3125 * 2^23
    return amax ? max(e, kFp4MinExponent) : 0;
}

// Six blocks an SM, 80 registers (with blocks of twice the size, two an SM, an FP8
// prompt of up to 64k tokens with keys took 36 us when six took 32). FP32 input, whose
// loads are twice as long, takes seven, 72 registers: 16 x 1001 ragged tokens into 4-bit
// records with keys, and back, 19 us, with five 20.6; 8 x 8192 normalised ones into FP8
// records 32.3, with six 34.0. But with the norm and keys together seven spill: the
// 8 x 8192 tokens 56 us, with six 49.7, into 4-bit records 64 and 58.
template <int DT, int FMT, bool KEYS, bool NORM>
__global__ void __launch_bounds__(kThreads, DT == CSA_FP32 && !(NORM && KEYS) ? 7 : 6)
append_kernel(const __grid_constant__ AppendParams P) {
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int t0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * P.per_warp;
    if (t0 >= P.span.B * P.span.T) return;
    const Slot mine = find_slots(P.span, t0, P.per_warp, lane, P.err);
    // The indexer keys of two tokens at once, 16 lanes each (one at a time: 4 % more):
    // lane hl of a half holds octet hl of the key of token j + half (j even).
    const int half = lane >> 4, hl = lane & 15;
    const bool turn = P.ops.rope_dim > 0;
    __shared__ __align__(16) float2 warp_cs[kWarps][2][32];  // of the warp's current two tokens
    float2(*pair_cs)[32] = warp_cs[threadIdx.x >> 5];
    const uint64_t pair_turn = turn ? P.ops.turn[lane] : 0;
    float w[2][8];  // the norm's weights of this lane's dims
    load_weights(w[0], NORM ? P.ops.weight : nullptr, 16 * lane);
    load_weights(w[1], NORM ? P.ops.weight : nullptr, 16 * lane + 8);
    struct {
        Octet<DT> x[2];
        int64_t record;
    } now, next;
    Octet<DT> key, next_key;
    int key_b = 0, next_key_b = 0;
    int nb = t0 / P.span.T, nt = t0 - nb * P.span.T;  // the token to fetch
    auto fetch = [&](int j, auto &o) {
        const int b = nb, t = nt;
        if (++nt == P.span.T) nt = 0, ++nb;
        if (KEYS && !(j & 1)) {
            next_key_b = half ? nb : b;
            if (__shfl_sync(kAll, mine.record, j + half) >= 0)
                next_key.load(P.key, next_key_b * P.key_seq_stride + (half ? nt : t) * P.key_token_stride + 8 * hl);
        }
        o.record = __shfl_sync(kAll, mine.record, j);
        if (o.record < 0) return;
        const int64_t at = b * P.seq_stride + t * P.token_stride + 16 * lane;
        o.x[0].load(P.x, at);
        o.x[1].load(P.x, at + 8);
    };
    fetch(0, next);
#pragma unroll 1
    for (int j = 0; j < P.per_warp; ++j) {
        now = next;
        if (KEYS && !(j & 1)) {
            key = next_key;
            key_b = next_key_b;
        }
        if (j + 1 < P.per_warp) fetch(j + 1, next);
        if (now.record >= 0) {
            if (turn) {
                const int64_t entry = __shfl_sync(kAll, mine.entry, j);
                __syncwarp();
                pair_cs[j & 1][lane] = turn_cos_sin(entry * P.pos_stride, pair_turn);
                __syncwarp();
            }

            float f[2][8];
            now.x[0].floats(f[0]);
            now.x[1].floats(f[1]);
            if (NORM) {
                float2 two = make_float2(0.f, 0.f);
                square_octet(f[0], two);
                square_octet(f[1], two);
                float sum = two.x + two.y;
#pragma unroll
                for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
                const float inv_rms = inverse_rms(sum, 1.f / kDim, P.ops.eps);
                scale_octet(f[0], inv_rms, w[0]);
                scale_octet(f[1], inv_rms, w[1]);
            }
            const bool rope_lane = lane >= kNopeLanes;
            if (turn && rope_lane) {
                const float2 *cs = pair_cs[j & 1] + 8 * (lane - kNopeLanes);
                turn_octet(f[0], *reinterpret_cast<const float2(*)[4]>(cs));
                turn_octet(f[1], *reinterpret_cast<const float2(*)[4]>(cs + 4));
            }
            const uint32_t amax = rope_lane ? 0u : amax_bits(amax_octet(f[1], amax_octet(f[0])));
            uint8_t *rec = P.base + now.record * (FMT == CSA_FORMAT_FP4 ? kFp4Bytes : kRecBytes);
            if (FMT == CSA_FORMAT_FP4) {
                const uint32_t top = __reduce_max_sync(kAll, amax);
                const bool bad = top >= 0x7F800000u;  // an infinity or NaN: the whole record reads as NaN
                const int E = bad ? 128 : fp4_exponent(top);
                if (rope_lane) {
                    uint4 *dst = reinterpret_cast<uint4 *>(rec + kFp4RopeOffset + 32 * (lane - kNopeLanes));
                    dst[0] = pack_bf16_octet(f[0]);
                    dst[1] = pack_bf16_octet(f[1]);
                    if (lane == kNopeLanes)
                        *reinterpret_cast<uint32_t *>(rec + kFp4PowerOffset) = (uint32_t)(E + 127);
                } else {
                    // block scale: e4m3(amax / 6 * 2^-E), its halfway cases decided exactly
                    const float ratio = sticky_quotient(__uint_as_float(amax), 6.f, 1.f / 6.f) *
                                        __uint_as_float((uint32_t)(127 - E) << 23);
                    const uint32_t sb = bad ? 0u : e4m3x4(ratio, 0.f, 0.f, 0.f) & 0xFFu;
                    uint2 codes = make_uint2(0u, 0u);
                    if (sb) {
                        float unit = e4m3x2_to_float2((uint16_t)sb).x * __uint_as_float((uint32_t)(E + 127) << 23);
                        if (E < -60) {
                            constexpr float kUp = 18446744073709551616.f;
                            unit *= kUp;
#pragma unroll
                            for (int e = 0; e < 8; ++e) f[0][e] *= kUp, f[1][e] *= kUp;
                        }
                        codes = fp4_codes<DT == CSA_FP32 || NORM>(f, unit);
                    }
                    *reinterpret_cast<uint2 *>(rec + 8 * lane) = codes;
                    rec[kFp4ScaleOffset + lane] = (uint8_t)sb;
                }
            } else {
                uint32_t top = amax;  // over the eight lanes of a 128-dim block (rope lanes hold 0)
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(kAll, top, o));
                if (rope_lane) {
                    uint4 *dst = reinterpret_cast<uint4 *>(rec + kRopeOffset + 32 * (lane - kNopeLanes));
                    dst[0] = pack_bf16_octet(f[0]);
                    dst[1] = pack_bf16_octet(f[1]);
                } else {
                    const float s = e4m3_scale(top);
                    float q[2][8];
                    e4m3_quotients<DT != CSA_FP32 && !NORM>(f[0], top, q[0]);
                    e4m3_quotients<DT != CSA_FP32 && !NORM>(f[1], top, q[1]);
                    *reinterpret_cast<uint4 *>(rec + 16 * lane) =
                        make_uint4(e4m3x4(q[0][0], q[0][1], q[0][2], q[0][3]), e4m3x4(q[0][4], q[0][5], q[0][6], q[0][7]),
                               e4m3x4(q[1][0], q[1][1], q[1][2], q[1][3]), e4m3x4(q[1][4], q[1][5], q[1][6], q[1][7]));
                    if ((lane & 7) == 0) *reinterpret_cast<float *>(rec + kScaleOffset + 4 * (lane >> 3)) = s;
                }
            }
        }
        if (KEYS && ((j & 1) || j + 1 == P.per_warp)) {
            const int from = (j & ~1) + half;
            const bool live = __shfl_sync(kAll, mine.record, from) >= 0;
            const int64_t entry = __shfl_sync(kAll, mine.entry, from);
            float g[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = 0.f;
            if (live) key.floats(g);
            // octets 8..15 are the key's rope dims: pairs 4 (hl - 8) ..
            if (turn && live && hl >= 8)
                turn_octet(g, *reinterpret_cast<const float2(*)[4]>(pair_cs[half] + 4 * (hl - 8)));
            uint32_t top = amax_bits(amax_octet(g));
#pragma unroll
            for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(kAll, top, o));
            if (live && entry >= P.idx_cap) {
                if (hl == 0) report_error(P.err, CSA_ERR_BAD_INDEX);
            } else if (live) {
                const float s = e4m3_scale(top);
                const int64_t row = (int64_t)key_b * P.idx_cap + entry;
                e4m3_quotients<DT != CSA_FP32>(g, top, g);
                *reinterpret_cast<uint2 *>(P.k_idx + row * kIdxDim + 8 * hl) =
                    make_uint2(e4m3x4(g[0], g[1], g[2], g[3]), e4m3x4(g[4], g[5], g[6], g[7]));
                if (hl == 0) P.k_idx_scale[row] = s;
            }
        }
    }
}

struct ReadParams {
    Span span;
    uint4 *out;
    int per_warp;
    int *err;
};

template <int FMT>
__global__ void __launch_bounds__(kThreads)
read_kernel(const __grid_constant__ ReadParams P) {
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int t0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * P.per_warp;
    if (t0 >= P.span.B * P.span.T) return;
    const Slot mine = find_slots(P.span, t0, P.per_warp, lane, P.err);
    const bool rope_lane = lane >= kNopeLanes;
    // a lane's bytes of a record: 16 codes (8 or 16 bytes) and their scale, or 32
    // bytes of rope dims
    struct {
        uint4 a, b;
        uint32_t scale, power;
        int64_t record;
    } now, next;
    auto fetch = [&](int j, auto &o) {
        o.record = __shfl_sync(kAll, mine.record, j);
        if (o.record < 0) return;
        const uint8_t *rec = P.span.cache.base + o.record * (FMT == CSA_FORMAT_FP4 ? kFp4Bytes : kRecBytes);
        if (rope_lane) {
            const uint4 *src = reinterpret_cast<const uint4 *>(
                rec + (FMT == CSA_FORMAT_FP4 ? kFp4RopeOffset : kRopeOffset) + 32 * (lane - kNopeLanes));
            o.a = src[0];
            o.b = src[1];
        } else if (FMT == CSA_FORMAT_FP4) {
            const uint2 c = *reinterpret_cast<const uint2 *>(rec + 8 * lane);
            o.a.x = c.x;
            o.a.y = c.y;
            o.scale = rec[kFp4ScaleOffset + lane];
            o.power = rec[kFp4PowerOffset];
        } else {
            o.a = *reinterpret_cast<const uint4 *>(rec + 16 * lane);
            o.scale = *reinterpret_cast<const uint32_t *>(rec + kScaleOffset + 4 * (lane >> 3));
        }
    };
    fetch(0, next);
#pragma unroll 1
    for (int j = 0; j < P.per_warp; ++j) {
        now = next;
        if (j + 1 < P.per_warp) fetch(j + 1, next);
        if (now.record < 0) continue;
        uint4 lo = now.a, hi = now.b;
        if (!rope_lane) {
            const uint32_t w[4] = {now.a.x, now.a.y, now.a.z, now.a.w};
            float f[2][8];
            if (FMT == CSA_FORMAT_FP4) {
                const float s = e4m3x2_to_float2((uint16_t)now.scale).x * fp4_power(now.power);
#pragma unroll
                for (int o = 0; o < 2; ++o)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(w[o] >> (8 * e)), __NV_E2M1);
                        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                        f[o][2 * e] = v.x * s;
                        f[o][2 * e + 1] = v.y * s;
                    }
            } else {
                const float s = __uint_as_float(now.scale);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 u = e4m3x2_to_float2((uint16_t)(w[i] & 0xFFFFu));
                    const float2 v = e4m3x2_to_float2((uint16_t)(w[i] >> 16));
                    f[i >> 1][4 * (i & 1)] = u.x * s;
                    f[i >> 1][4 * (i & 1) + 1] = u.y * s;
                    f[i >> 1][4 * (i & 1) + 2] = v.x * s;
                    f[i >> 1][4 * (i & 1) + 3] = v.y * s;
                }
            }
            lo = pack_bf16_octet(f[0]);
            hi = pack_bf16_octet(f[1]);
        }
        uint4 *dst = P.out + (int64_t)(t0 + j) * (kDim / 8) + 2 * lane;
        dst[0] = lo;
        dst[1] = hi;
    }
}

struct CommitParams {
    Span span;
    const uint4 *records;
    const int32_t *select;
    int N, words;  // records a sequence, 16-byte words a record
    uint4 *base;
    int *err;
};

// A warp a token: 24 or 37 words of 16 bytes, one or two a lane. Bound by its three trips
// to memory in a row (count and first; page and number; the record): 64 x up to 128 FP8
// records 2.8 us, a launch of nothing 2.
__global__ void __launch_bounds__(kThreads) commit_kernel(const __grid_constant__ CommitParams P) {
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int token = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (token >= P.span.B * P.span.T) return;
    const int b = token / P.span.T, t = token - b * P.span.T;
    // every lane looks the token up (the same addresses); one of them reports
    int *const err = lane == 0 ? P.err : nullptr;
    const Slot to = find_slot(P.span, b, t, err);
    if (to.record < 0) return;
    const int from = P.select ? __ldg(P.select + token) : t;
    if (from < 0 || from >= P.N) {
        report_error(err, CSA_ERR_BAD_INDEX);
        return;
    }
    const uint4 *src = P.records + ((int64_t)b * P.N + from) * P.words;
    uint4 *dst = P.base + to.record * P.words;
    const bool more = lane + 32 < P.words;
    uint4 v, w;
    if (lane < P.words) v = __ldg(src + lane);
    if (more) w = __ldg(src + lane + 32);
    if (lane < P.words) dst[lane] = v;
    if (more) dst[lane + 32] = w;
}

bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// The checks that both calls share, and their span.
csa_status_t make_span(const csa_cache_desc &cache, csa_format_t fmt, int ring, const int32_t *first,
                       const int32_t *count, int B, int T, const int32_t *status, Span *s) {
    if (fmt != CSA_FORMAT_FP8 && fmt != CSA_FORMAT_FP4) return CSA_ERR_INVALID_ARG;
    if (!first || misaligned(first) || misaligned(count) || B < 1 || T < 1 || !valid_cache(cache, B) ||
        !valid_status_word(status))
        return CSA_ERR_INVALID_ARG;
    if ((int64_t)B * T > (1 << 24)) return CSA_ERR_UNSUPPORTED;
    s->cache = make_view(cache);
    s->ring = ring ? 1 : 0;
    s->first = first;
    s->count = count;
    s->B = B;
    s->T = T;
    return CSA_OK;
}

template <int DT, int FMT>
cudaError_t launch_append(const AppendParams &P, PdlLaunch &l) {
    if (P.ops.norm)
        return P.key ? cudaLaunchKernelEx(&l.cfg, append_kernel<DT, FMT, true, true>, P)
                     : cudaLaunchKernelEx(&l.cfg, append_kernel<DT, FMT, false, true>, P);
    return P.key ? cudaLaunchKernelEx(&l.cfg, append_kernel<DT, FMT, true, false>, P)
                 : cudaLaunchKernelEx(&l.cfg, append_kernel<DT, FMT, false, false>, P);
}

template <int DT>
cudaError_t launch_append(const AppendParams &P, csa_format_t fmt, PdlLaunch &l) {
    return fmt == CSA_FORMAT_FP4 ? launch_append<DT, CSA_FORMAT_FP4>(P, l) : launch_append<DT, CSA_FORMAT_FP8>(P, l);
}

}  // namespace

}  // namespace csa

extern "C" CSA_API csa_status_t csa_cache_append(csa_cache_desc cache, csa_format_t fmt, int ring, const void *x,
                                                 csa_dtype_t x_dtype, int64_t x_seq_stride, int64_t x_token_stride,
                                                 const int32_t *first, const int32_t *count, int B, int T,
                                                 int pos_stride, const csa_norm_rope *how, const csa_index_append *idx,
                                                 int32_t *status, cudaStream_t stream) {
    using namespace csa;
    AppendParams P;
    const csa_status_t a = make_span(cache, fmt, ring, first, count, B, T, status, &P.span);
    if (a != CSA_OK) return a;
    if (x_dtype != CSA_BF16 && x_dtype != CSA_FP16 && x_dtype != CSA_FP32) return CSA_ERR_INVALID_ARG;
    const int64_t per16 = x_dtype == CSA_FP32 ? 4 : 8;
    if (!x || misaligned(x) || x_seq_stride < 0 || x_token_stride < 0 || x_seq_stride % per16 ||
        x_token_stride % per16 || pos_stride < 1 || pos_stride > 65536)
        return CSA_ERR_INVALID_ARG;
    if (!make_row_ops(how, kDim, &P.ops) || (P.ops.rope_dim != 0 && P.ops.rope_dim != kRope)) return CSA_ERR_INVALID_ARG;
    P.key = nullptr;
    P.key_seq_stride = P.key_token_stride = 0;
    P.k_idx = nullptr;
    P.k_idx_scale = nullptr;
    P.idx_cap = 0;
    if (idx) {
        if (ring || !idx->key || !idx->k_idx || !idx->k_idx_scale || misaligned(idx->key) || misaligned(idx->k_idx) ||
            misaligned(idx->k_idx_scale) || idx->Ncap < 1 || idx->seq_stride < 0 || idx->token_stride < 0 ||
            idx->seq_stride % per16 || idx->token_stride % per16)
            return CSA_ERR_INVALID_ARG;
        P.key = idx->key;
        P.key_seq_stride = idx->seq_stride;
        P.key_token_stride = idx->token_stride;
        P.k_idx = idx->k_idx;
        P.k_idx_scale = idx->k_idx_scale;
        P.idx_cap = idx->Ncap;
    }
    P.x = x;
    P.seq_stride = x_seq_stride;
    P.token_stride = x_token_stride;
    P.pos_stride = pos_stride;
    P.base = static_cast<uint8_t *>(const_cast<void *>(cache.base));
    P.err = status;
    P.per_warp = tokens_per_warp(B * T, kAppendTokens);
    PdlLaunch l(dim3((B * T + kWarps * P.per_warp - 1) / (kWarps * P.per_warp)), dim3(kThreads), stream);
    count_launch();
    const cudaError_t e = x_dtype == CSA_BF16   ? launch_append<CSA_BF16>(P, fmt, l)
                          : x_dtype == CSA_FP16 ? launch_append<CSA_FP16>(P, fmt, l)
                                                : launch_append<CSA_FP32>(P, fmt, l);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

extern "C" CSA_API csa_status_t csa_cache_read(csa_cache_desc cache, csa_format_t fmt, int ring, const int32_t *first,
                                               const int32_t *count, int B, int T, void *out, int32_t *status,
                                               cudaStream_t stream) {
    using namespace csa;
    ReadParams P;
    const csa_status_t a = make_span(cache, fmt, ring, first, count, B, T, status, &P.span);
    if (a != CSA_OK) return a;
    if (!out || misaligned(out)) return CSA_ERR_INVALID_ARG;
    P.out = static_cast<uint4 *>(out);
    P.err = status;
    P.per_warp = tokens_per_warp(B * T, kReadTokens);
    PdlLaunch l(dim3((B * T + kWarps * P.per_warp - 1) / (kWarps * P.per_warp)), dim3(kThreads), stream);
    count_launch();
    const cudaError_t e = fmt == CSA_FORMAT_FP4 ? cudaLaunchKernelEx(&l.cfg, read_kernel<CSA_FORMAT_FP4>, P)
                                                : cudaLaunchKernelEx(&l.cfg, read_kernel<CSA_FORMAT_FP8>, P);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

extern "C" CSA_API csa_status_t csa_cache_commit(csa_cache_desc cache, csa_format_t fmt, int ring, const void *records,
                                                 int N, const int32_t *select, const int32_t *first,
                                                 const int32_t *count, int B, int T, int32_t *status,
                                                 cudaStream_t stream) {
    using namespace csa;
    CommitParams P;
    const csa_status_t a = make_span(cache, fmt, ring, first, count, B, T, status, &P.span);
    if (a != CSA_OK) return a;
    if (!records || misaligned(records) || misaligned(select) || N < 1 || (!select && T > N)) return CSA_ERR_INVALID_ARG;
    P.records = static_cast<const uint4 *>(records);
    P.select = select;
    P.N = N;
    P.words = (fmt == CSA_FORMAT_FP4 ? kFp4Bytes : kRecBytes) / 16;
    P.base = static_cast<uint4 *>(const_cast<void *>(cache.base));
    P.err = status;
    PdlLaunch l(dim3((B * T + kWarps - 1) / kWarps), dim3(kThreads), stream);
    count_launch();
    const cudaError_t e = cudaLaunchKernelEx(&l.cfg, commit_kernel, P);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}
