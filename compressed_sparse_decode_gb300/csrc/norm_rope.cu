// norm_rope.cu -- RMS norm of every head with the position rotation in the
// same pass (csa_head_norm_rope, csa_head_norm_rope_e4m3).
//
// For the D values x of a head at position p:
//   y = x * (mean x^2 + eps)^(-1/2) * w;  the last rope_dim values of y turned
//   pairwise by p * theta^(-2i/rope_dim);  out = bf16(y), or e4m3(y / s) with
//   s = amax |y| / 448.
#include "rows.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;

struct NormRopeParams {
    const void *x;
    int64_t seq_stride, token_stride, head_stride;  // elements
    const int32_t *pos;
    int T, H, D, rows;
    void *out;       // BF16 values or E4M3 codes
    float *scale;    // E4M3 only
    RowOps ops;
};

// A group of G lanes holds a head (NV octets a lane); each group takes R
// consecutive heads, whose loads are all issued before the first is used.
template <int DT, int G, int NV, int R, bool E4M3>
__global__ void __launch_bounds__(kThreads)
norm_rope_kernel(const __grid_constant__ NormRopeParams P) {
    ptx::griddep_wait();
    const int gl = threadIdx.x & (G - 1);
    const int r0 = (blockIdx.x * (kThreads / G) + threadIdx.x / G) * R;
    const int octets = P.D >> 3;
    const int rope_octet = (P.D - P.ops.rope_dim) >> 3;

    Octet<DT> in[R][NV];
    int pos[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = r0 + i;
        pos[i] = -1;
        if (r < P.rows) {
            const int token = r / P.H, h = r - token * P.H;
            pos[i] = __ldg(P.pos + token);
            if (pos[i] >= 0) {
                const int b = token / P.T;
                const int64_t at = b * P.seq_stride + (int64_t)(token - b * P.T) * P.token_stride + h * P.head_stride;
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    if (gl + G * v < octets) in[i][v].load(P.x, at + 8 * (gl + G * v));
            }
        }
    }

    float2 cs[NV][4];
    int turned = -1;  // the position that cs holds
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int p = pos[i];
        float f[NV][8];
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (p >= 0 && gl + G * v < octets) {
                in[i][v].floats(f[v]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[v][e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(f[v][e], f[v][e], sum);
        }
        if (P.ops.norm) {
#pragma unroll
            for (int o = G / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float inv_rms = rsqrtf(sum / P.D + P.ops.eps);
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (gl + G * v < octets) scale_octet(f[v], inv_rms, P.ops.weight, 8 * (gl + G * v));
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int o = gl + G * v;
            if (o >= rope_octet && o < octets && p >= 0) {
                if (p != turned) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) cs[v][e] = turn_cos_sin(p, P.ops.turn[4 * (o - rope_octet) + e]);
                }
                turn_octet(f[v], cs[v]);
            }
        }
        turned = p;
        const int64_t row = r0 + i;
        if (!E4M3) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (p >= 0 && gl + G * v < octets)
                    reinterpret_cast<uint4 *>(P.out)[row * octets + gl + G * v] = pack_bf16_octet(f[v]);
        } else {
            uint32_t amax = 0;
#pragma unroll
            for (int v = 0; v < NV; ++v) amax = amax_bits(f[v], amax);
#pragma unroll
            for (int o = G / 2; o; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const float s = e4m3_scale(amax), inv = 1.f / s;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (p >= 0 && gl + G * v < octets) {
                    float q[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) q[e] = quotient(f[v][e], s, inv);
                    reinterpret_cast<uint2 *>(P.out)[row * octets + gl + G * v] =
                        make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
                }
            }
            if (p >= 0 && gl == 0) P.scale[row] = s;
        }
    }
}

template <int DT, int G, int NV, bool E4M3>
cudaError_t launch_rows(const NormRopeParams &P, cudaStream_t stream) {
    constexpr int kGroups = kThreads / G;
    const int ctas = (P.rows + kGroups - 1) / kGroups;
    PdlLaunch l(dim3(ctas), dim3(kThreads), stream);
    count_launch();
    return cudaLaunchKernelEx(&l.cfg, norm_rope_kernel<DT, G, NV, 1, E4M3>, P);
}

template <int DT, bool E4M3>
cudaError_t launch_type(const NormRopeParams &P, cudaStream_t stream) {
    if (P.D <= 64) return launch_rows<DT, 8, 1, E4M3>(P, stream);
    if (P.D <= 128) return launch_rows<DT, 16, 1, E4M3>(P, stream);
    if (P.D <= 256) return launch_rows<DT, 32, 1, E4M3>(P, stream);
    return launch_rows<DT, 32, 2, E4M3>(P, stream);
}

template <bool E4M3>
csa_status_t run(const void *x, csa_dtype_t dt, int64_t seq_stride, int64_t token_stride, int64_t head_stride,
                 const int32_t *pos, int B, int T, int H, int D, const csa_norm_rope *how, void *out, float *scale,
                 const int32_t *status, cudaStream_t stream) {
    if (dt != CSA_BF16 && dt != CSA_FP16 && dt != CSA_FP32) return CSA_ERR_INVALID_ARG;
    if (!x || !pos || !how || !out || (E4M3 && !scale) || !valid_status_word(status)) return CSA_ERR_INVALID_ARG;
    const uintptr_t all = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(pos) |
                          reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(scale);
    if (all & 15u) return CSA_ERR_INVALID_ARG;
    if (B < 1 || T < 1 || H < 1 || D < 8) return CSA_ERR_INVALID_ARG;
    const int64_t per16 = dt == CSA_FP32 ? 4 : 8;
    if (seq_stride < 0 || token_stride < 0 || head_stride < 0 || seq_stride % per16 || token_stride % per16 ||
        head_stride % per16)
        return CSA_ERR_INVALID_ARG;
    if (D % 8 || D > kDim || (int64_t)B * T > (1 << 24) || (int64_t)B * T * H >= ((int64_t)1 << 31))
        return CSA_ERR_UNSUPPORTED;
    NormRopeParams P;
    if (!make_row_ops(how, D, &P.ops)) return CSA_ERR_INVALID_ARG;
    P.x = x;
    P.seq_stride = seq_stride;
    P.token_stride = token_stride;
    P.head_stride = head_stride;
    P.pos = pos;
    P.T = T;
    P.H = H;
    P.D = D;
    P.rows = B * T * H;
    P.out = out;
    P.scale = scale;
    const cudaError_t e = dt == CSA_BF16   ? launch_type<CSA_BF16, E4M3>(P, stream)
                          : dt == CSA_FP16 ? launch_type<CSA_FP16, E4M3>(P, stream)
                                           : launch_type<CSA_FP32, E4M3>(P, stream);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

}  // namespace

}  // namespace csa

extern "C" CSA_API csa_status_t csa_head_norm_rope(const void *x, csa_dtype_t x_dtype, int64_t x_seq_stride,
                                                   int64_t x_token_stride, int64_t x_head_stride, const int32_t *pos,
                                                   int B, int T, int H, int D, const csa_norm_rope *how, void *out,
                                                   int32_t *status, cudaStream_t stream) {
    return csa::run<false>(x, x_dtype, x_seq_stride, x_token_stride, x_head_stride, pos, B, T, H, D, how, out, nullptr,
                           status, stream);
}

extern "C" CSA_API csa_status_t csa_head_norm_rope_e4m3(const void *x, csa_dtype_t x_dtype, int64_t x_seq_stride,
                                                        int64_t x_token_stride, int64_t x_head_stride,
                                                        const int32_t *pos, int B, int T, int H, int D,
                                                        const csa_norm_rope *how, uint8_t *codes, float *scale,
                                                        int32_t *status, cudaStream_t stream) {
    return csa::run<true>(x, x_dtype, x_seq_stride, x_token_stride, x_head_stride, pos, B, T, H, D, how, codes, scale,
                          status, stream);
}
