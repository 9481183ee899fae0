// verify.cu -- verification of a tree's drafted tokens against the target's
// distribution (csa_verify_drafts).
//
// With p = softmax(z / t) of the current token's logits, the walk tests the
// children x_1, x_2, .. of the current token in turn:
//   accept x_k  if  u_k q(x_k) R_k < r_k(x_k),    else go on with r_k+1, R_k+1;
// since max(max(a - b, 0) - c, 0) = max(a - b - c, 0) for c >= 0, all residuals of a
// token are r_k = max(p - S_k q, 0) with S_k = R_1 + .. + R_k-1: a rejection
// changes one number, and only R_k+1, where another child asks for it, takes a pass
// over the row. (Without q: r_k is p without the tokens rejected so far.) At the end
// of the walk the next token is argmax r(v) / noise(v), one more pass. Everything is
// kept without the softmax's denominator: p stands for e^{(z - max) / t}, R_1 for its
// sum.
//
// One cluster of up to eight CTAs a sequence, each with a slice of the vocabulary;
// only rows on the accepted path are read. All CTAs take every decision from the
// same numbers in the same order, so they walk together without a leader; partial
// results go to every CTA of the cluster through distributed shared memory, one
// cluster barrier a pass.
#include <cmath>

#include "rows.cuh"

namespace csa {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxNodes = CSA_MAX_TOKENS_PER_SEQ;
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLog2e = 1.44269502f, kLog2eRest = 1.92596303e-8f;  // log2(e) in two floats
constexpr int kNoDraft = -1;  // draft type: none

// What a pass over a row leaves: a value, its index and a sum.
struct alignas(16) Found {
    float value;  // the largest (NaN if one is)
    int32_t index;
    float sum;
    uint32_t unused;
};

struct VerifyParams {
    const void *logits, *draft;
    int64_t seq_stride, token_stride;
    const int32_t *token, *parent;
    const float *uniform, *noise, *temperature;
    int N, V, slice;  // slice: tokens a CTA, a multiple of 8
    int32_t *path, *accepted, *next;
    int *err;
};

template <int DT>
__device__ __forceinline__ float element(const void *base, int64_t at) {
    if (DT == CSA_FP32) return __ldg(static_cast<const float *>(base) + at);
    if (DT == CSA_FP16) return __half2float(__ldg(static_cast<const __half *>(base) + at));
    return __bfloat162float(__ldg(static_cast<const __nv_bfloat16 *>(base) + at));
}

// A thread's U units of W consecutive elements, kThreads units apart, all loaded before any
// is used. W is 8 where rows begin on 16 bytes, else 1.
template <int DT, int W, int U>
struct Units;
template <int DT, int U>
struct Units<DT, 8, U> {
    Octet<DT> o[U];
    __device__ __forceinline__ void load(const void *base, int64_t row, int v, int v1) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v + u * kThreads * 8 < v1) o[u].load(base, row + v + u * kThreads * 8);
    }
    __device__ __forceinline__ void get(int u, float (&f)[8]) const { o[u].floats(f); }
};
template <int DT, int U>
struct Units<DT, 1, U> {
    float o[U];
    __device__ __forceinline__ void load(const void *base, int64_t row, int v, int v1) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v + u * kThreads < v1) o[u] = element<DT>(base, row + v + u * kThreads);
    }
    __device__ __forceinline__ void get(int u, float (&f)[1]) const { f[0] = o[u]; }
};

__device__ __forceinline__ void store_remote(uint32_t addr, const Found &f) {
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(__float_as_uint(f.value)),
                 "r"((uint32_t)f.index), "r"(__float_as_uint(f.sum)), "r"(0u)
                 : "memory");
}

// The larger value, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
    return a;
}

// Order of the values: -0 is 0, a NaN (of any bits) above all.
__device__ __forceinline__ uint32_t value_key(float v) {
    return v != v ? 0xFFFFFFFFu : v == 0.f ? 0x80000000u : order_key(v);
}
__device__ __forceinline__ float key_value(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}

// How the parts of a pass are joined: the largest value (a NaN is the largest of all) with
// its lowest index, and the sum. Of a softmax the sums are of 2^{(z - value) k} and scaled
// to the largest value (a part whose value is -inf has the sum 0).
struct Join {
    float k;  // 0: plain sums
    __device__ __forceinline__ float factor(float value, float top) const {
        return k == 0.f ? 1.f : value > -INFINITY ? exp2f((value - top) * k) : 0.f;
    }
    // the parts of a warp's first `lanes` lanes (a power of two; the others hold them again)
    __device__ __forceinline__ Found warp(const Found &f, int lanes) const {
        Found r;
        const uint32_t key = value_key(f.value), top = __reduce_max_sync(kAll, key);
        r.value = key_value(top);
        r.index = (int32_t)__reduce_min_sync(kAll, key == top ? (uint32_t)f.index : 0x7FFFFFFFu);
        r.sum = f.sum * factor(f.value, r.value);
        for (int o = lanes / 2; o; o >>= 1) r.sum += __shfl_xor_sync(kAll, r.sum, o);
        r.unused = 0;
        return r;
    }
};

// 2^{d (k + k_rest)} for the tokens that decide: the product's own rounding, which at
// d k = -20 would be 1e-6 of the weight, is put right.
__device__ __forceinline__ float weight_of(float d, float k, float k_rest) {
    const float a = d * k;
    const float rest = fmaf(d, k_rest, fmaf(d, k, -a));
    const float e = exp2f(a);
    return fabsf(rest) < 1.f ? fmaf(e, rest * 0.69314718f, e) : e;  // (d = -inf has no rest)
}

// A sum that tokens are taken from, in two floats: what is left after most of it
// has gone keeps its bits.
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair less(const Pair &a, float v) {
    const float s = a.hi - v, back = s - a.hi;
    const float lo = a.lo + ((a.hi - (s - back)) + (-v - back));
    Pair r;
    r.hi = fmaxf(s + lo, 0.f);
    r.lo = lo - (r.hi - s);
    return r;
}

struct Smem {
    Found warps[kWarps];
    Found ctas[2][kMaxCluster];  // by the parity of the pass
    int32_t parent[kMaxNodes], token[kMaxNodes];
    float uniform[kMaxNodes];
    float logit[kMaxNodes], draft[kMaxNodes];  // of the children of the current token
    int32_t out[kMaxNodes];                    // rejected tokens of the current token (no draft probabilities)
};

// Joins every thread's part over the cluster; the same result, bit for bit, in
// all threads of it.
__device__ __forceinline__ Found join_cluster(Smem &s, Found f, int ctas, int rank, int &pass, const Join &join) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    f = join.warp(f, 32);
    if (lane == 0) s.warps[warp] = f;
    __syncthreads();
    if (warp == 0) {
        f = join.warp(s.warps[lane % kWarps], kWarps);
        if (lane < ctas) store_remote(ptx::mapa(ptx::smem_u32(&s.ctas[pass & 1][rank]), lane), f);
    }
    // (A slot is written again two passes later, behind the next pass's barrier,
    // which every thread enters after it has read this pass's slots.)
    ptx::cluster_sync();
    const Found r = join.warp(s.ctas[pass & 1][lane & (ctas - 1)], ctas);
    ++pass;
    return r;
}

template <int DT, int QT, int W>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const __grid_constant__ VerifyParams P, int ctas) {
    __shared__ Smem s;
    ptx::griddep_wait();
    const int b = blockIdx.x / ctas, rank = blockIdx.x - b * ctas;
    const int tid = threadIdx.x, lane = tid & 31;
    constexpr bool kDraft = QT != kNoDraft;
    constexpr int kQ = kDraft ? QT : CSA_FP32;
    constexpr int kRow = W == 1 ? 16 : DT == CSA_FP32 ? 2 : 4;              // units of a row in flight
    constexpr int kRows = W == 1 ? 8 : DT == CSA_FP32 || kDraft ? 1 : 2;  // of two or three rows
    if (tid < P.N) {
        const int64_t at = (int64_t)b * P.N + tid;
        s.parent[tid] = __ldg(P.parent + at);
        s.token[tid] = __ldg(P.token + at);
        s.uniform[tid] = __ldg(P.uniform + at);
    }
    const float t = P.temperature ? __ldg(P.temperature + b) : 1.f;
    const bool greedy = !(t > 0.f);
    // 1 / t in units of log2, in two floats; in (0, inf) for any t, so that a largest
    // logit's weight stays 1 and a masked token's 0
    float k = kLog2e, k_rest = kLog2eRest;
    if (!greedy) {
        k = fminf(fmaxf(kLog2e / t, 1e-30f), 1e38f);
        const float rest = (fmaf(-k, t, kLog2e) + kLog2eRest) / t;
        k_rest = fabsf(rest) < k ? rest : 0.f;  // (where k was clamped it has none)
    }
    const int v0 = rank * P.slice, v1 = min(P.V, v0 + P.slice);  // this CTA's tokens
    const int mine = v0 + tid * W;                               // this thread's first
    const int64_t noise_row = (int64_t)b * P.V;
    if (!greedy)  // (read at the end of the walk)
        for (int v = v0 + tid * 32; v < v1; v += kThreads * 32)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(P.noise + noise_row + v));
    // every CTA has started before anything is stored into it
    ptx::cluster_sync();

    int cur = 0, n = 0, pass = 0;
    if (rank == 0 && tid == 0) P.path[(int64_t)b * P.N] = 0;
    int next_token = -1;
    while (true) {
        ++n;
        const int64_t row = b * P.seq_stride + cur * P.token_stride;
        const int64_t qrow = ((int64_t)b * P.N + cur) * P.V;
        // what the children's tests will ask for, under way with the row
        const bool child_here = tid < P.N && tid > cur && s.parent[tid] == cur;
        float child_logit = 0.f, child_q = 1.f;
        if (child_here) {
            const int x = s.token[tid];
            if (x >= 0 && x < P.V) {
                child_logit = element<DT>(P.logits, row + x);
                if (kDraft) child_q = element<kQ>(P.draft, qrow + x);
            }
        }
        // ---- the row's largest logit and softmax sum
        Found f = {-INFINITY, INT32_MAX, 0.f, 0u};
        for (int v = mine; v < v1; v += kThreads * W * kRow) {
            Units<DT, W, kRow> z;
            z.load(P.logits, row, v, v1);
            float m = f.value;
#pragma unroll
            for (int u = 0; u < kRow; ++u)
                if (v + u * kThreads * W < v1) {
                    float x[W];
                    z.get(u, x);
#pragma unroll
                    for (int e = 0; e < W; ++e) m = max_nan(m, x[e]);
                }
            if (greedy) {
                if (m != f.value) {  // (its first place; no sum is needed)
                    f.value = m;
#pragma unroll
                    for (int u = kRow - 1; u >= 0; --u)
                        if (v + u * kThreads * W < v1) {
                            float x[W];
                            z.get(u, x);
#pragma unroll
                            for (int e = W - 1; e >= 0; --e)
                                if (x[e] == m) f.index = v + u * kThreads * W + e;
                        }
                }
                continue;
            }
            if (!(m > -INFINITY)) {  // (nothing yet, or a NaN)
                f.value = m;
                continue;
            }
            f.sum = f.value > -INFINITY ? f.sum * exp2f((f.value - m) * k) : 0.f;
            f.value = m;
            float part[2] = {0.f, 0.f};
#pragma unroll
            for (int u = 0; u < kRow; ++u)
                if (v + u * kThreads * W < v1) {
                    float x[W];
                    z.get(u, x);
#pragma unroll
                    for (int e = 0; e < W; ++e) part[(u * W + e) & 1] += ptx::ex2_approx((x[e] - m) * k);
                }
            f.sum += part[0] + part[1];
        }
        if (child_here) {
            s.logit[tid] = child_logit;
            s.draft[tid] = child_q;
        }
        f = join_cluster(s, f, ctas, rank, pass, Join{k});
        const float top = f.value;
        const int best = f.index;
        if (!(fabsf(top) < INFINITY)) break;  // no distribution
        // ---- its children
        float S = 0.f;
        Pair R = {f.sum, 0.f};
        bool stale = false;  // R is that of the rejections before the last
        int gone = 0;        // rejected tokens in s.out
        int last = cur, taken = -1;
        auto weight = [&](float z, float q) {  // of a token in the residual, rejected tokens aside
            const float p = ptx::ex2_approx((z - top) * k);
            return kDraft ? p - S * q : p;
        };
        while (taken < 0) {
            int child = kMaxNodes;
            for (int i0 = 0; i0 < P.N && child == kMaxNodes; i0 += 32) {
                const int i = i0 + lane;
                const uint32_t hit = __ballot_sync(kAll, i < P.N && i > last && s.parent[i] == cur);
                if (hit) child = i0 + __ffs(hit) - 1;
            }
            if (child == kMaxNodes) break;
            last = child;
            const int x = s.token[child];
            if (x < 0 || x >= P.V) {
                if (rank == 0 && tid == 0) report_error(P.err, CSA_ERR_BAD_INDEX);
                continue;
            }
            if (greedy) {
                if (x == best) taken = child;
                continue;
            }
            if (kDraft && stale) {  // the sum of what is left
                Found g = {0.f, 0, 0.f, 0u};
                for (int v = mine; v < v1; v += kThreads * W * kRows) {
                    Units<DT, W, kRows> z;
                    Units<kQ, W, kRows> q;
                    z.load(P.logits, row, v, v1);
                    q.load(P.draft, qrow, v, v1);
#pragma unroll
                    for (int u = 0; u < kRows; ++u)
                        if (v + u * kThreads * W < v1) {
                            float x[W], y[W];
                            z.get(u, x);
                            q.get(u, y);
#pragma unroll
                            for (int e = 0; e < W; ++e) g.sum += fmaxf(weight(x[e], y[e]), 0.f);
                        }
                }
                R = {join_cluster(s, g, ctas, rank, pass, Join{0.f}).sum, 0.f};
                stale = false;
            }
            const float p = weight_of(s.logit[child] - top, k, k_rest);
            const float q = s.draft[child];
            float r = p;
            if (kDraft) {
                r = fmaxf(fmaf(-S, q, p), 0.f);
            } else {
                for (int i = 0; i < gone; ++i)
                    if (s.out[i] == x) r = 0.f;
            }
            if (s.uniform[child] * q * R.hi < r) {
                taken = child;
            } else if (kDraft) {
                S += R.hi;
                stale = true;
            } else if (r > 0.f) {
                R = less(R, p);
                __syncthreads();
                if (tid == 0) s.out[gone] = x;
                ++gone;
                __syncthreads();
            }
        }
        if (taken >= 0) {
            if (rank == 0 && tid == 0) P.path[(int64_t)b * P.N + n] = taken;
            cur = taken;
            continue;
        }
        // ---- the next token
        if (greedy) {
            next_token = best;
            break;
        }
        for (int from_p = 0; from_p < 2; ++from_p) {  // the second time from p itself
            if (from_p) S = 0.f, gone = 0;
            Found g = {-1.f, INT32_MAX, 0.f, 0u};
            for (int v = mine; v < v1; v += kThreads * W * kRows) {
                Units<DT, W, kRows> z;
                Units<kQ, W, kRows> q;
                Units<CSA_FP32, W, kRows> e;
                z.load(P.logits, row, v, v1);
                if (kDraft) q.load(P.draft, qrow, v, v1);
                e.load(P.noise, noise_row, v, v1);
                uint32_t out = 0;  // which of these tokens were rejected
                if (!kDraft)
                    for (int o = 0; o < gone; ++o) {
                        const int at = s.out[o] - v;
#pragma unroll
                        for (int u = 0; u < kRows; ++u)
                            if ((uint32_t)(at - u * kThreads * W) < (uint32_t)W) out |= 1u << (u * W + at - u * kThreads * W);
                    }
#pragma unroll
                for (int u = 0; u < kRows; ++u)
                    if (v + u * kThreads * W < v1) {
                        float x[W], y[W], d[W];
                        z.get(u, x);
                        if (kDraft) q.get(u, y);
                        e.get(u, d);
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            const float r = weight(x[i], kDraft ? y[i] : 0.f);
                            const bool in = r > 0.f && (kDraft || !(out >> (u * W + i) & 1u));
                            const float ratio = in ? __fdividef(r, d[i]) : -1.f;
                            if (ratio > g.value) g.value = ratio, g.index = v + u * kThreads * W + i;
                        }
                    }
            }
            g = join_cluster(s, g, ctas, rank, pass, Join{0.f});
            if (g.value >= 0.f) {
                next_token = g.index;
                break;
            }
        }
        break;
    }
    if (rank == 0) {
        if (tid == 0) {
            P.accepted[b] = n;
            P.next[b] = next_token;
        }
        if (tid >= n && tid < P.N) P.path[(int64_t)b * P.N + tid] = -1;
    }
}

struct Plan {
    int ctas, slice;
};
// CTAs a sequence, a power of two up to eight: as many as have 2048 tokens each, while all
// sequences' fit on the SMs at once (two an SM).
Plan make_plan(int B, int V) {
    Plan p;
    p.ctas = 1;
    while (p.ctas < kMaxCluster && V > p.ctas * 2048 && B * p.ctas * 2 <= 2 * cached_sm_count()) p.ctas *= 2;
    p.slice = ((V + p.ctas - 1) / p.ctas + 7) / 8 * 8;
    return p;
}

template <int DT, int QT>
cudaError_t launch_verify(const VerifyParams &P, int ctas, bool wide, const cudaLaunchConfig_t &cfg) {
    return wide ? cudaLaunchKernelEx(&cfg, verify_kernel<DT, QT, 8>, P, ctas)
                : cudaLaunchKernelEx(&cfg, verify_kernel<DT, QT, 1>, P, ctas);
}

template <int DT>
cudaError_t launch_verify(const VerifyParams &P, int draft_dtype, int ctas, bool wide, const cudaLaunchConfig_t &cfg) {
    if (!P.draft) return launch_verify<DT, kNoDraft>(P, ctas, wide, cfg);
    return draft_dtype == CSA_BF16   ? launch_verify<DT, CSA_BF16>(P, ctas, wide, cfg)
           : draft_dtype == CSA_FP16 ? launch_verify<DT, CSA_FP16>(P, ctas, wide, cfg)
                                     : launch_verify<DT, CSA_FP32>(P, ctas, wide, cfg);
}

bool valid_dtype(int d) { return d == CSA_BF16 || d == CSA_FP16 || d == CSA_FP32; }
bool off(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

}  // namespace

size_t verify_workspace_bytes(int, int, int) { return 0; }

}  // namespace csa

extern "C" CSA_API csa_status_t csa_verify_drafts(const void *logits, csa_dtype_t logits_dtype, int64_t seq_stride,
                                                  int64_t token_stride, const void *draft_probs,
                                                  csa_dtype_t draft_dtype, const int32_t *token,
                                                  const int32_t *parent, const float *uniform, const float *noise,
                                                  const float *temperature, int B, int N, int V, int32_t *path,
                                                  int32_t *accepted, int32_t *next_token, void *workspace,
                                                  size_t workspace_bytes, int32_t *status, cudaStream_t stream) {
    using namespace csa;
    (void)workspace;
    (void)workspace_bytes;
    if (!logits || !token || !parent || !uniform || !noise || !path || !accepted || !next_token)
        return CSA_ERR_INVALID_ARG;
    if (!valid_dtype(logits_dtype) || (draft_probs && !valid_dtype(draft_dtype)) || !valid_status_word(status))
        return CSA_ERR_INVALID_ARG;
    if (!valid_dims(B, N) || V < 1 || seq_stride < 0 || token_stride < 0) return CSA_ERR_INVALID_ARG;
    const int size = logits_dtype == CSA_FP32 ? 4 : 2, q_size = draft_dtype == CSA_FP32 ? 4 : 2;
    if (off(logits, size) || (draft_probs && off(draft_probs, q_size)) || off(noise, 4) || off(token, 4) ||
        off(parent, 4) || off(uniform, 4) || off(temperature, 4) || off(path, 4) || off(accepted, 4) ||
        off(next_token, 4))
        return CSA_ERR_INVALID_ARG;
    if (V > (1 << 24)) return CSA_ERR_UNSUPPORTED;
    VerifyParams P;
    P.logits = logits;
    P.draft = draft_probs;
    P.seq_stride = seq_stride;
    P.token_stride = token_stride;
    P.token = token;
    P.parent = parent;
    P.uniform = uniform;
    P.noise = noise;
    P.temperature = temperature;
    P.N = N;
    P.V = V;
    P.path = path;
    P.accepted = accepted;
    P.next = next_token;
    P.err = status;
    const Plan plan = make_plan(B, V);
    P.slice = plan.slice;
    // eight elements a load where every row that is read begins on 16 bytes
    const bool wide = V % 8 == 0 && seq_stride % 8 == 0 && token_stride % 8 == 0 && !off(logits, 16) &&
                      !off(draft_probs, 16) && !off(noise, 16);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = plan.ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(B * plan.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    count_launch();
    const cudaError_t e = logits_dtype == CSA_BF16   ? launch_verify<CSA_BF16>(P, draft_dtype, plan.ctas, wide, cfg)
                          : logits_dtype == CSA_FP16 ? launch_verify<CSA_FP16>(P, draft_dtype, plan.ctas, wide, cfg)
                                                     : launch_verify<CSA_FP32>(P, draft_dtype, plan.ctas, wide, cfg);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}
