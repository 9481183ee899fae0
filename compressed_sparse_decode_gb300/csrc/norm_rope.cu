// norm_rope.cu -- RMS norm of every head with the position rotation in the
// same pass (csa_head_norm_rope, csa_head_norm_rope_e4m3).
//
// For the D values x of a head at position p:
//   y = x * (mean x^2 + eps)^(-1/2) * w;  the last rope_dim values of y turned
//   pairwise by p * theta^(-2i/rope_dim);  out = bf16(y), or e4m3(y / s) with
//   s = amax |y| / 448.
//
// One pass: a head is read once into registers and written once. 4 x 1027 tokens of
// 128 heads of 512 BF16 values (77 % of them not padding): 824 MB in 132 us, 6.2
// TB/s or 0.92 of the measured copy rate, with two thirds of the issue slots busy.
// One token of 128 heads: 2.5 us, a launch and two trips to memory.
#include "rows.cuh"

namespace csa {

namespace {

constexpr int kThreads = 128;

struct NormRopeParams {
    const void *x;
    int64_t seq_stride, token_stride, head_stride;  // elements
    const int32_t *pos;
    int T, H, D, rows;
    void *out;       // BF16 values or E4M3 codes
    float *scale;    // E4M3 only
    int per_group;   // heads a group, one after the other
    RowOps ops;
};

// A group of G lanes holds a head (NV octets a lane) and takes per_group
// consecutive heads, the next one's loads under the current one (two heads ahead
// needs registers that cost warps: 139 us instead of 132). What bounds the pass is
// DRAM only if a head costs few instructions: the rotation's sines and cosines are
// computed once a token and block, into shared memory (each head for itself took
// 120 of 390 instructions), the norm's weights stay in registers.
template <int DT, int G, int NV, bool E4M3>
__global__ void __launch_bounds__(kThreads, DT == CSA_FP32 ? 4 : 8)
norm_rope_kernel(const __grid_constant__ NormRopeParams P) {
    extern __shared__ float2 turns[];  // [tokens of the block][rope pairs]
    ptx::griddep_wait();
    constexpr int kGroups = kThreads / G;
    const int gl = threadIdx.x & (G - 1);
    const int block0 = blockIdx.x * kGroups * P.per_group;  // (rows < 2^31 - 2^20)
    const int r0 = block0 + threadIdx.x / G * P.per_group;
    const int octets = P.D >> 3;
    const int rope_octet = (P.D - P.ops.rope_dim) >> 3, pairs = P.ops.rope_dim >> 1;
    const int token0 = block0 / P.H;

    // the group's position in the tensor: token (b, t), head h
    int token = r0 / P.H, h = r0 - token * P.H, b = token / P.T, t = token - b * P.T;
    struct Head {
        Octet<DT> x[NV];
        int pos, token;
    } now, next;
    auto fetch = [&](int i, Head &o) {
        o.pos = -1;
        if (i >= P.per_group || r0 + i >= P.rows) return;
        o.token = token;
        o.pos = __ldg(P.pos + token);
        const int64_t at = b * P.seq_stride + t * P.token_stride + h * P.head_stride;
        if (++h == P.H) {
            h = 0;
            ++token;
            if (++t == P.T) t = 0, ++b;
        }
        if (o.pos < 0) return;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (gl + G * v < octets) o.x[v].load(P.x, at + 8 * (gl + G * v));
    };
#pragma unroll
    for (int v = 0; v < NV; ++v) next.x[v].clear();  // (octets past D stay so)
    fetch(0, next);

    if (pairs) {
        const int last = min(block0 + kGroups * P.per_group, P.rows) - 1;
        const int n = (last / P.H - token0 + 1) * pairs;
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const int tk = i / pairs, pair = i - tk * pairs;
            turns[i] = turn_cos_sin(__ldg(P.pos + token0 + tk), P.ops.turn[pair]);
        }
    }
    float w[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v)
        load_weights(w[v], P.ops.norm && gl + G * v < octets ? P.ops.weight : nullptr, 8 * (gl + G * v));
    const float inv_d = 1.f / P.D;
    __syncthreads();

    auto finish = [&](int i, const Head &now) {
        const bool live = now.pos >= 0;
        float f[NV][8];
        float2 two = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            now.x[v].floats(f[v]);  // (a head that does not count: whatever was there)
            square_octet(f[v], two);
        }
        if (P.ops.norm) {
            float sum = two.x + two.y;
#pragma unroll
            for (int o = G / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float inv_rms = inverse_rms(sum, inv_d, P.ops.eps);
#pragma unroll
            for (int v = 0; v < NV; ++v) scale_octet(f[v], inv_rms, w[v]);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int o = gl + G * v;
            if (o >= rope_octet && o < octets && live) {
                const float4 *cs = reinterpret_cast<const float4 *>(turns + (now.token - token0) * pairs + 4 * (o - rope_octet));
                const float4 c0 = cs[0], c1 = cs[1];
                const float2 c[4] = {make_float2(c0.x, c0.y), make_float2(c0.z, c0.w), make_float2(c1.x, c1.y),
                                     make_float2(c1.z, c1.w)};
                turn_octet(f[v], c);
            }
        }
        const int64_t row = r0 + i;
        if (!E4M3) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (live && gl + G * v < octets)
                    reinterpret_cast<uint4 *>(P.out)[row * octets + gl + G * v] = pack_bf16_octet(f[v]);
        } else {
            float m = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v) m = amax_octet(f[v], m);
            uint32_t amax = amax_bits(m);
#pragma unroll
            for (int o = G / 2; o; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const float s = e4m3_scale(amax);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (live && gl + G * v < octets) {
                    float q[8];
                    if (DT != CSA_FP32 && !P.ops.norm) e4m3_quotients<true>(f[v], amax, q);
                    else e4m3_quotients<false>(f[v], amax, q);
                    reinterpret_cast<uint2 *>(P.out)[row * octets + gl + G * v] =
                        make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
                }
            }
            if (live && gl == 0) P.scale[row] = s;
        }
    };
#pragma unroll 1
    for (int i = 0; i < P.per_group; ++i) {
        now = next;
        fetch(i + 1, next);
        if (G < 32 || now.pos >= 0) finish(i, now);
    }
}

// Heads a group: as many as leave every SM eight blocks, up to 16.
template <int DT, int G, int NV, bool E4M3>
cudaError_t launch_rows(NormRopeParams &P, cudaStream_t stream) {
    constexpr int kGroups = kThreads / G;
    const int n = P.rows / (kGroups * 8 * cached_sm_count());
    P.per_group = n < 1 ? 1 : n > 16 ? 16 : n;
    // the rotation of the block's tokens (at most this many) has 48 KB
    auto turn_bytes = [&]() {
        return (size_t)((kGroups * P.per_group - 1) / P.H + 2) * (P.ops.rope_dim / 2) * sizeof(float2);
    };
    while (P.per_group > 1 && turn_bytes() > 48 * 1024) --P.per_group;
    const int per_block = kGroups * P.per_group;
    PdlLaunch l(dim3((P.rows + per_block - 1) / per_block), dim3(kThreads), stream);
    l.cfg.dynamicSmemBytes = turn_bytes();
    count_launch();
    return cudaLaunchKernelEx(&l.cfg, norm_rope_kernel<DT, G, NV, E4M3>, P);
}

template <int DT, bool E4M3>
cudaError_t launch_type(NormRopeParams &P, cudaStream_t stream) {
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
    if (D % 8 || D > kDim || (int64_t)B * T > (1 << 24) || (int64_t)B * T * H >= ((int64_t)1 << 31) - (1 << 20))
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
