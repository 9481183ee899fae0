// attention_fp4.cu -- sink-merged attention over caches of 4-bit records
// (csa_sink_attention_decode_fp4, hca_sink_attention_decode_fp4).
//
// For head h over candidates j (x_j the dequantised latent):
//   z_j = scale * q_h . x_j,  o_h = sum_j e^{z_j-M} x_j / (e^{sink_h-M} + sum_j e^{z_j-M}),
//   lse_h = M + ln(den),  M = max(sink_h, max_j z_j).
//
// One CTA a (query token, 16 heads); candidates in chunks of 32, dequantised to
// fp32 in shared memory, a running maximum and sum for each head.
#include <cuda_fp4.h>

#include "rows.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;
constexpr int kHeadGroup = 16;
constexpr int kChunk = 32;
constexpr int kXStride = kDim + 4;

struct Params {
    const __nv_bfloat16 *q;
    const float *sink;
    float scale;
    CacheView comp;
    const uint8_t *ring;
    int R, W;
    const int32_t *topk_idx, *topk_cnt, *n_comp, *q_pos;
    int m_hca, hca, T, k;
    __nv_bfloat16 *out;
    float *lse;
    uint8_t *out_fp4;
    float *out_fp4_scale;
    int inv_rope;
    uint64_t turn[kRope / 2];
    int *err;
};

struct Smem {
    float x[kChunk][kXStride];
    float q[kHeadGroup][kDim];
    float p[kHeadGroup][kChunk];
    float m[kHeadGroup], l[kHeadGroup], alpha[kHeadGroup];
    float amax[kHeadGroup][kThreads / 32];
    int valid[kChunk];
};

__global__ void __launch_bounds__(kThreads)
attention_fp4_kernel(const __grid_constant__ Params P) {
    extern __shared__ uint8_t raw[];
    Smem &s = *reinterpret_cast<Smem *>(raw);
    const int tid = threadIdx.x, r = blockIdx.y, b = r / P.T, h0 = blockIdx.x * kHeadGroup;
    const int p = P.q_pos[r];
    int n_sel;
    if (P.hca) {
        n_sel = visible_entries(p, P.m_hca, P.n_comp[b], P.comp.seq_capacity);
    } else {
        const int c = P.topk_cnt[r];
        n_sel = c < 0 ? 0 : (c > P.k ? P.k : c);
    }
    const int j0 = max(0, p - P.W + 1);
    const int n = n_sel + (p >= 0 ? p - j0 + 1 : 0);
    for (int i = tid; i < kHeadGroup * kDim; i += kThreads)
        s.q[i / kDim][i % kDim] = __bfloat162float(P.q[((size_t)r * kHeads + h0) * kDim + i]) * P.scale;
    if (tid < kHeadGroup) {
        s.m[tid] = P.sink[h0 + tid];
        s.l[tid] = s.m[tid] == -INFINITY ? 0.f : 1.f;
    }
    float2 acc[kHeadGroup];
#pragma unroll
    for (int h = 0; h < kHeadGroup; ++h) acc[h] = make_float2(0.f, 0.f);
    for (int c0 = 0; c0 < n; c0 += kChunk) {
        __syncthreads();
        {  // eight threads a candidate
            const int c = tid >> 3, part = tid & 7, i = c0 + c;
            const uint8_t *rec = nullptr;
            if (i < n_sel) {
                const int e = P.hca ? i : P.topk_idx[(size_t)r * P.k + i];
                const int64_t ri = record_index(P.comp, b, e);
                if (ri >= 0) rec = P.comp.base + ri * kFp4Bytes;
                else if (part == 0 && blockIdx.x == 0) report_error(P.err, CSA_ERR_BAD_INDEX);
            } else if (i < n) {
                rec = P.ring + ((int64_t)b * P.R + (j0 + i - n_sel) % P.R) * kFp4Bytes;
            }
            if (part == 0) s.valid[c] = rec != nullptr;
            for (int d = part * 64; d < part * 64 + 64; ++d) {
                float v = 0.f;
                if (rec) {
                    if (d >= kNope) {
                        v = bf16_bits_to_float(reinterpret_cast<const uint16_t *>(rec + kFp4RopeOffset)[d - kNope]);
                    } else {
                        const __half2_raw two = __nv_cvt_fp4x2_to_halfraw2(rec[d >> 1], __NV_E2M1);
                        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&two));
                        const float sb = e4m3x2_to_float2(rec[kFp4ScaleOffset + d / kFp4Block]).x;
                        v = ((d & 1) ? f.y : f.x) * sb * fp4_power(rec[kFp4PowerOffset]);
                    }
                }
                s.x[c][d] = v;
            }
        }
        __syncthreads();
        const int h = tid >> 4;  // 16 threads a head, two candidates each
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int c = (tid & 15) + 16 * e;
            float z = 0.f;
            for (int d = 0; d < kDim; d += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(&s.q[h][d]);
                const float4 x = *reinterpret_cast<const float4 *>(&s.x[c][d]);
                z = fmaf(a.x, x.x, fmaf(a.y, x.y, fmaf(a.z, x.z, fmaf(a.w, x.w, z))));
            }
            s.p[h][c] = s.valid[c] ? z : -INFINITY;
        }
        __syncthreads();
        if (tid < kHeadGroup) {
            float m = s.m[tid];
            for (int c = 0; c < kChunk; ++c) m = fmaxf(m, s.p[tid][c]);
            const float ref = m == -INFINITY ? 0.f : m, al = s.m[tid] == -INFINITY ? 0.f : expf(s.m[tid] - ref);
            float l = s.l[tid] * al;
            for (int c = 0; c < kChunk; ++c) {
                const float e = expf(s.p[tid][c] - ref);
                s.p[tid][c] = e;
                l += e;
            }
            s.m[tid] = m;
            s.l[tid] = l;
            s.alpha[tid] = al;
        }
        __syncthreads();
#pragma unroll
        for (int g = 0; g < kHeadGroup; ++g) {
            float2 a = make_float2(acc[g].x * s.alpha[g], acc[g].y * s.alpha[g]);
            for (int c = 0; c < kChunk; ++c) {
                const float w = s.p[g][c];
                a.x = fmaf(w, s.x[c][2 * tid], a.x);
                a.y = fmaf(w, s.x[c][2 * tid + 1], a.y);
            }
            acc[g] = a;
        }
    }
    __syncthreads();
    // thread t holds dims 2t, 2t + 1 of every head: a rope pair from t = 224 on
    float2 cs = make_float2(1.f, 0.f);
    if (P.inv_rope && tid >= kNope / 2) cs = turn_cos_sin(p, P.turn[tid - kNope / 2]);
#pragma unroll
    for (int g = 0; g < kHeadGroup; ++g) {
        const float inv = s.l[g] > 0.f ? 1.f / s.l[g] : 0.f;
        const float x = acc[g].x * inv, y = acc[g].y * inv;
        acc[g] = make_float2(fmaf(x, cs.x, y * cs.y), fmaf(-x, cs.y, y * cs.x));
        const size_t row = (size_t)r * kHeads + h0 + g;
        if (P.out_fp4) {
            float a = fmaxf(fabsf(acc[g].x), fabsf(acc[g].y));
            for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
            if ((tid & 31) == 0) s.amax[g][tid >> 5] = a;
        } else {
            reinterpret_cast<uint32_t *>(P.out)[row * (kDim / 2) + tid] = pack_bf16(acc[g].x, acc[g].y);
        }
        if (tid == 0) P.lse[row] = s.l[g] > 0.f ? s.m[g] + logf(s.l[g]) : -INFINITY;
    }
    if (!P.out_fp4) return;
    __syncthreads();
    for (int g = 0; g < kHeadGroup; ++g) {
        const size_t row = (size_t)r * kHeads + h0 + g;
        const float a = fmaxf(s.amax[g][(tid >> 5) & ~1], s.amax[g][tid >> 5 | 1]);
        const float sc = a > 0.f ? a / 6.f : 1.f, inv = 1.f / sc;
        P.out_fp4[row * (kDim / 2) + tid] = (uint8_t)e2m1x4(acc[g].x * inv, acc[g].y * inv, 0.f, 0.f);
        if ((tid & 63) == 0) P.out_fp4_scale[row * 4 + (tid >> 6)] = sc;
    }
}

}  // namespace

// `k` = the top-k row length (CSA) or the per-sequence capacity (HCA).
cudaError_t launch_attention_fp4(const void *q, const float *sink, float scale, const csa_cache_desc &comp,
                                 const void *ring, int R, int W, const int32_t *topk_idx, const int32_t *topk_cnt,
                                 const int32_t *n_comp, int m_hca, const int32_t *q_pos, int B, int T, int k, bool hca,
                                 void *out, float *lse, const csa_attention_epilogue *epi, void *, size_t, int *err,
                                 cudaStream_t stream) {
    Params P = {};
    P.q = static_cast<const __nv_bfloat16 *>(q);
    P.sink = sink;
    P.scale = scale;
    P.comp = make_view(comp);
    P.ring = static_cast<const uint8_t *>(ring);
    P.R = R;
    P.W = W;
    P.topk_idx = topk_idx;
    P.topk_cnt = topk_cnt;
    P.n_comp = n_comp;
    P.q_pos = q_pos;
    P.m_hca = m_hca;
    P.hca = hca ? 1 : 0;
    P.T = T;
    P.k = hca ? 0 : k;
    P.out = static_cast<__nv_bfloat16 *>(out);
    P.lse = lse;
    P.err = err;
    if (epi) {
        P.out_fp4 = epi->out_fp4;
        P.out_fp4_scale = epi->out_fp4_scale;
        if (epi->inverse_rope) {
            RowOps o;
            const csa_norm_rope how = {0, 0.f, nullptr, kRope, epi->rope_theta};
            if (!make_row_ops(&how, kDim, &o)) return cudaErrorInvalidValue;
            P.inv_rope = 1;
            for (int i = 0; i < kRope / 2; ++i) P.turn[i] = o.turn[i];
        }
    }
    const cudaError_t e = set_max_dynamic_smem_once(reinterpret_cast<const void *>(attention_fp4_kernel), sizeof(Smem));
    if (e != cudaSuccess) return e;
    count_launch();
    attention_fp4_kernel<<<dim3(kHeads / kHeadGroup, B * T), kThreads, sizeof(Smem), stream>>>(P);
    return cudaGetLastError();
}

}  // namespace csa
