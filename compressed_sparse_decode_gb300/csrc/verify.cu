// verify.cu -- verification of a tree's drafted tokens against the target's
// distribution (csa_verify_drafts).
//
// With p = softmax(z / t) of the current token's logits, the walk tests the
// children x_1, x_2, .. of the current token in turn:
//   accept x_k  if  u_k q(x_k) R_k < r_k(x_k),    else go on with r_k+1, R_k+1;
// since max(max(a - b, 0) - c, 0) = max(a - b - c, 0) for c >= 0, all residuals of a
// token are r_k = max(p - S_k q, 0) with S_k = R_1 + .. + R_k-1: a rejection
// changes one number, and only R_k+1, where another child asks for it, takes a pass
// over the row. (Without q: r_k is p without the tokens rejected so far, and R_k+1 is
// R_k - r_k(x_k), with a pass where that is little of R_k.) At the end
// of the walk the next token is argmax r(v) / noise(v), one more pass. Everything is
// kept without the softmax's denominator: p stands for e^{(z - max) / t}, R_1 for its
// sum.
//
// One cluster of up to eight CTAs a sequence, each with a slice of the vocabulary;
// only rows on the accepted path are read. All CTAs take every decision from the
// same numbers in the same order, so they walk together without a leader; every CTA's
// part of a pass goes to all CTAs of the cluster through distributed shared memory.
//
// Measured (mean path 2.5 of the tokens): 64 trees of 32 tokens over 131072 BF16 logits 35.8
// us (75 MB of rows and noise: 0.31 of the copy rate), 32 chains of 6 with an FP32 draft
// 23.6, 16 trees of 25 over 50001 FP32 logits 17.3, one chain of 8 over 32000 5.3. The
// longest walk of a batch decides: a row takes 1.3 us (its latency, and 32 exponentials a
// thread), the join 1.0, the children's tests 0.4.
#include <cmath>
#include <type_traits>

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
    uint32_t ok;  // (of the joined parts: they have all come)
};

struct VerifyParams {
    const void *logits, *draft;
    int64_t seq_stride, token_stride;
    const int32_t *token, *parent;
    const float *uniform, *noise, *temperature;
    int N, V, slice;  // slice: tokens a CTA, a multiple of 8
    int32_t *path, *accepted, *next;
    int *err;
    uint64_t wait_ns;  // limit of each bounded wait
};

template <int DT>
__device__ __forceinline__ float element(const void *base, int64_t at) {
    if (DT == CSA_FP32) return __ldg(static_cast<const float *>(base) + at);
    if (DT == CSA_FP16) return __half2float(__ldg(static_cast<const __half *>(base) + at));
    return __bfloat162float(__ldg(static_cast<const __nv_bfloat16 *>(base) + at));
}

// A thread's U units of W consecutive elements, kThreads units apart, all loaded before any
// is used (behind v1: `fill`). W is 8 where rows begin on 16 bytes, else 1.
template <int DT>
constexpr uint32_t kMinusInf = DT == CSA_FP32 ? 0xFF800000u : DT == CSA_FP16 ? 0xFC00FC00u : 0xFF80FF80u;
template <int DT, int W, int U>
struct Units;
template <int DT, int U>
struct Units<DT, 8, U> {
    Octet<DT> o[U];
    __device__ __forceinline__ void load(const void *base, int64_t row, int v, int v1, uint32_t fill) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            o[u].v = make_uint4(fill, fill, fill, fill);
            if constexpr (DT == CSA_FP32) o[u].u = o[u].v;
            if (v + u * kThreads * 8 < v1) o[u].load(base, row + v + u * kThreads * 8);
        }
    }
    __device__ __forceinline__ void get(int u, float (&f)[8]) const { o[u].floats(f); }
};
template <int DT, int U>
struct Units<DT, 1, U> {
    float o[U];
    __device__ __forceinline__ void load(const void *base, int64_t row, int v, int v1, uint32_t fill) {
        const float f = DT == CSA_FP32 ? __uint_as_float(fill) : fill ? -INFINITY : 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) o[u] = v + u * kThreads < v1 ? element<DT>(base, row + v + u * kThreads) : f;
    }
    __device__ __forceinline__ void get(int u, float (&f)[1]) const { f[0] = o[u]; }
};

// The larger value, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
    return a;
}

// The largest element of the units, NaN if one is (16-bit elements two at a time).
template <int DT, int W, int U>
__device__ __forceinline__ float largest(const Units<DT, W, U> &z) {
    if constexpr (W == 8 && DT != CSA_FP32) {
        using Two = std::conditional_t<DT == CSA_BF16, __nv_bfloat162, __half2>;
        Two m[2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t w[4] = {z.o[u].v.x, z.o[u].v.y, z.o[u].v.z, z.o[u].v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const Two x = *reinterpret_cast<const Two *>(&w[i]);
                m[i & 1] = u == 0 && i < 2 ? x : __hmax2_nan(m[i & 1], x);
            }
        }
        const Two t = __hmax2_nan(m[0], m[1]);
        return max_nan((float)t.x, (float)t.y);
    } else {
        float m[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[W];
            z.get(u, x);
#pragma unroll
            for (int e = 0; e < W; ++e) m[(u * W + e) & 1] = max_nan(m[(u * W + e) & 1], x[e]);
        }
        return max_nan(m[0], m[1]);
    }
}

// A thread's part of the pass over tokens [mine, v1) of a row: the largest logit and the
// softmax sum, or, greedy, the largest logit and its first place.
template <int DT, int W>
__device__ __forceinline__ Found scan_row(const void *logits, int64_t row, int mine, int v1, float k, bool greedy) {
    constexpr int U = W == 1 ? 16 : DT == CSA_FP32 ? 2 : 4;  // units in flight
    Found f = {-INFINITY, INT32_MAX, 0.f, 1u};
    for (int v = mine; v < v1; v += kThreads * W * U) {
        Units<DT, W, U> z;
        z.load(logits, row, v, v1, kMinusInf<DT>);
        const float m = max_nan(f.value, largest(z));
        if (greedy) {
            if (m == f.value) continue;
            f.value = m;
#pragma unroll
            for (int u = U - 1; u >= 0; --u) {
                float x[W];
                z.get(u, x);
#pragma unroll
                for (int e = W - 1; e >= 0; --e)
                    if (x[e] == m) f.index = v + u * kThreads * W + e;
            }
            continue;
        }
        if (!(m > -INFINITY)) {  // (nothing yet, or a NaN)
            f.value = m;
            continue;
        }
        f.sum = f.value > -INFINITY ? f.sum * exp2f((f.value - m) * k) : 0.f;
        f.value = m;
        if constexpr (W == 1) {
            float part[2] = {0.f, 0.f};
#pragma unroll
            for (int u = 0; u < U; ++u) part[u & 1] += ptx::ex2_approx((z.o[u] - m) * k);
            f.sum += part[0] + part[1];
        } else {
            float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[W];
                z.get(u, x);
#pragma unroll
                for (int e = 0; e < W / 2; ++e) {
                    float2 d = __fadd2_rn(make_float2(x[2 * e], x[2 * e + 1]), make_float2(-m, -m));
                    d = __fmul2_rn(d, make_float2(k, k));
                    part[e & 1] = __fadd2_rn(part[e & 1], make_float2(ptx::ex2_approx(d.x), ptx::ex2_approx(d.y)));
                }
            }
            f.sum += (part[0].x + part[0].y) + (part[1].x + part[1].y);
        }
    }
    return f;
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
        r.ok = 1;
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

// A sum that tokens are taken from, in two floats: taking them off adds no rounding to the
// sum's own error. What is left carries that error whole, so when less than kLeast of the last
// sum is left, and another child asks for it, it is summed anew (R off by up to 1e-6 / kLeast
// of itself; with one token of 1 - 1e-5 refused it would be off by a hundredth, and below
// 1e-7 nothing would be left of it). The pass takes 1.1 us over 32000 tokens of one sequence,
// 4.2 over 131072 of 64 (with 0.23 of the row left 8.5 and 20.4 us a call, with a third 7.4 and
// 16.2); 1 / 16 for kLeast changed no time of the usual drafts.
constexpr float kLeast = 0.25f;
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

// A sequence's 1 / temperature in units of log2, in two floats; in (0, inf) for any
// temperature, so that a largest logit's weight stays 1 and a masked token's 0.
struct Scale {
    bool greedy;
    float k, k_rest;
    __device__ __forceinline__ Scale(const VerifyParams &P, int b) {
        const float t = P.temperature ? __ldg(P.temperature + b) : 1.f;
        greedy = !(t > 0.f);
        k = kLog2e;
        k_rest = kLog2eRest;
        if (greedy) return;
        k = fminf(fmaxf(kLog2e / t, 1e-30f), 1e38f);
        const float rest = (fmaf(-k, t, kLog2e) + kLog2eRest) / t;
        k_rest = fabsf(rest) < k ? rest : 0.f;  // (where k was clamped it has none)
    }
};

struct Smem {
    Found warps[kWarps];
    Found ctas[2][kMaxCluster];  // by the parity of the pass
    Found all;
    uint64_t full[2];
    int32_t parent[kMaxNodes], token[kMaxNodes];
    float uniform[kMaxNodes];
    float logit[kMaxNodes], draft[kMaxNodes];  // of the drafts: their logit and probability, in their parents' rows
    uint8_t out[kWarps][kMaxNodes];            // a warp's list of the current token's rejected children (no draft)
};

// Joins every thread's part over the cluster; the same result, bit for bit, in
// all threads of it. The first warp of each CTA sends the CTA's part to all of them,
// counted on a barrier there. (Slots and barriers are two by turns: those of pass p are
// sent to again in pass p + 2, after a wait for pass p + 1, to which every CTA sends after
// it has read pass p's.) False, for the whole CTA, after a wait that expired.
__device__ __forceinline__ bool join_cluster(Smem &s, Found &f, int ctas, int rank, int &pass, const Join &join,
                                             uint64_t wait_ns) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, now = pass & 1;
    f = join.warp(f, 32);
    if (lane == 0) s.warps[warp] = f;
    __syncthreads();
    if (warp == 0) {
        f = join.warp(s.warps[lane % kWarps], kWarps);
        uint64_t *full = &s.full[now];
        if (lane < ctas) {
            const uint32_t v[4] = {__float_as_uint(f.value), (uint32_t)f.index, __float_as_uint(f.sum), 0u};
            ptx::store4_to_peer(ptx::mapa(ptx::smem_u32(&s.ctas[now][rank]), lane), v,
                                ptx::mapa(ptx::smem_u32(full), lane));
        }
        if (lane == 0) ptx::mbar_arrive_expect_tx(full, ctas * sizeof(Found));
        const uint32_t parity = (pass >> 1) & 1;
        const bool poll = wait_ns < ptx::kPollOnlyBelowNs;  // (a diagnostic limit: no suspension outlasts it)
        const uint64_t t0 = ptx::globaltimer_ns();
        bool here;
        do here = (!poll || ptx::mbar_test_wait(full, parity)) && ptx::try_wait_cluster(full, parity);
        while (!here && ptx::globaltimer_ns() - t0 <= wait_ns);
        const bool all = __all_sync(kAll, here);
        f = join.warp(s.ctas[now][lane & (ctas - 1)], ctas);
        f.ok = all;
        if (lane == 0) s.all = f;
    }
    __syncthreads();
    f = s.all;
    ++pass;
    return f.ok;
}

template <int DT, int QT, int W>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const __grid_constant__ VerifyParams P, int ctas) {
    __shared__ Smem s;
    const int b = blockIdx.x / ctas, rank = blockIdx.x - b * ctas;
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) ptx::mbar_init(&s.full[i], 1);  // (and all CTAs' bytes)
        ptx::fence_mbar_init();
    }
    __syncthreads();
    // every CTA's barriers exist before anything is sent to it (waited for behind the
    // first row's loads)
    ptx::cluster_arrive();
    ptx::griddep_wait();
    constexpr bool kDraft = QT != kNoDraft;
    constexpr int kQ = kDraft ? QT : CSA_FP32;
    constexpr int kRows = W == 1 ? 8 : DT == CSA_FP32 || kDraft ? 1 : 2;  // units of two or three rows in flight
    if (tid < P.N) {
        const int64_t at = (int64_t)b * P.N + tid;
        const int parent = __ldg(P.parent + at), x = __ldg(P.token + at);
        s.parent[tid] = parent;
        s.token[tid] = x;
        s.uniform[tid] = __ldg(P.uniform + at);
        float logit = 0.f, q = 1.f;
        if (parent >= 0 && parent < tid && x >= 0 && x < P.V) {
            logit = element<DT>(P.logits, b * P.seq_stride + parent * P.token_stride + x);
            if (kDraft) q = element<kQ>(P.draft, (at - tid + parent) * P.V + x);
        }
        s.logit[tid] = logit;
        s.draft[tid] = q;
    }
    const Scale scale(P, b);
    const bool greedy = scale.greedy;
    const float k = scale.k;
    const int v0 = rank * P.slice, v1 = min(P.V, v0 + P.slice);  // this CTA's tokens
    const int mine = v0 + tid * W;                               // this thread's first
    const int64_t noise_row = (int64_t)b * P.V;
    uint8_t *out_list = s.out[tid >> 5];
    __syncthreads();

    int cur = 0, n = 0, pass = 0;
    bool ok = true;
    if (rank == 0 && tid == 0) P.path[(int64_t)b * P.N] = 0;
    int next_token = -1;
    // the current token's next child behind token `last` (kMaxNodes: none)
    auto next_child = [&](int last) {
        for (int i0 = last & ~31; i0 < P.N; i0 += 32) {
            const int i = i0 + lane;
            const uint32_t hit = __ballot_sync(kAll, i < P.N && i > last && s.parent[i] == cur);
            if (hit) return i0 + __ffs(hit) - 1;
        }
        return kMaxNodes;
    };
    while (true) {
        ++n;
        const int64_t row = b * P.seq_stride + cur * P.token_stride;
        const int64_t qrow = ((int64_t)b * P.N + cur) * P.V;
        // ---- the row's largest logit and softmax sum
        Found f = scan_row<DT, W>(P.logits, row, mine, v1, k, greedy);
        if (n == 1) {
            // the noise, read at the end of the walk, comes into L2 behind the first row
            if (!greedy)
                for (int v = v0 + tid * 32; v < v1; v += kThreads * 32)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(P.noise + noise_row + v));
            __syncwarp();  // (the loops' trips differ between lanes, and the wait takes a converged warp)
            ptx::cluster_wait();
        }
        ok = join_cluster(s, f, ctas, rank, pass, Join{k}, P.wait_ns);
        if (!ok) break;
        const float top = f.value;
        const int best = f.index;
        if (!(fabsf(top) < INFINITY)) break;  // no distribution
        // ---- its children
        float S = 0.f;
        Pair R = {f.sum, 0.f};
        float whole = f.sum;  // the sum that R comes from
        bool stale = false;   // R is to be summed: it is that of the rejections before the last, or too little of `whole`
        int gone = 0;         // children in out_list
        int last = cur, taken = -1;
        auto weight = [&](float z, float q) {  // of a token in the residual, rejected tokens aside
            const float p = ptx::ex2_approx((z - top) * k);
            return kDraft ? p - S * q : p;
        };
        auto rejected = [&](int v) {  // which of a thread's tokens from v on, bit u W + e (no draft)
            uint32_t out = 0;
            if (!kDraft)
                for (int o = 0; o < gone; ++o) {
                    const int at = s.token[out_list[o]] - v;
#pragma unroll
                    for (int u = 0; u < kRows; ++u)
                        if ((uint32_t)(at - u * kThreads * W) < (uint32_t)W) out |= 1u << (u * W + at - u * kThreads * W);
                }
            return out;
        };
        while (taken < 0) {
            const int child = next_child(last);
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
            if (stale) {  // the sum of what is left
                Found g = {0.f, 0, 0.f, 0u};
                for (int v = mine; v < v1; v += kThreads * W * kRows) {
                    Units<DT, W, kRows> z;
                    Units<kQ, W, kRows> q;
                    z.load(P.logits, row, v, v1, kMinusInf<DT>);
                    if (kDraft) q.load(P.draft, qrow, v, v1, 0u);
                    const uint32_t out = rejected(v);
#pragma unroll
                    for (int u = 0; u < kRows; ++u) {
                        float x[W], y[W];
                        z.get(u, x);
                        if (kDraft) q.get(u, y);
#pragma unroll
                        for (int e = 0; e < W; ++e)
                            if (kDraft || !(out >> (u * W + e) & 1u)) g.sum += fmaxf(weight(x[e], kDraft ? y[e] : 0.f), 0.f);
                    }
                }
                ok = join_cluster(s, g, ctas, rank, pass, Join{0.f}, P.wait_ns);
                if (!ok) break;
                R = {g.sum, 0.f};
                whole = g.sum;
                stale = false;
            }
            const float p = weight_of(s.logit[child] - top, k, scale.k_rest);
            const float q = s.draft[child];
            float r = p;
            if (kDraft) {
                r = fmaxf(fmaf(-S, q, p), 0.f);
            } else {
                for (int i = 0; i < gone; ++i)
                    if (s.token[out_list[i]] == x) r = 0.f;
            }
            if (s.uniform[child] * q * R.hi < r) {
                taken = child;
            } else if (kDraft) {
                S += R.hi;
                stale = true;
            } else if (r > 0.f) {
                R = less(R, p);
                stale = R.hi < kLeast * whole;
                if (lane == 0) out_list[gone] = (uint8_t)child;
                ++gone;
                __syncwarp();
            }
        }
        if (!ok) break;
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
                z.load(P.logits, row, v, v1, kMinusInf<DT>);
                if (kDraft) q.load(P.draft, qrow, v, v1, 0u);
                e.load(P.noise, noise_row, v, v1, 0x3F800000u);
                const uint32_t out = rejected(v);
#pragma unroll
                for (int u = 0; u < kRows; ++u) {
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
            ok = join_cluster(s, g, ctas, rank, pass, Join{0.f}, P.wait_ns);
            if (!ok) break;
            if (g.value >= 0.f) {
                next_token = g.index;
                break;
            }
        }
        break;
    }
    if (!ok) {
        // given up: what was sent to another CTA (16 bytes a pass) lands long before this
        // bounded pause ends, and none has left before the others' has
        if (tid == 0) report_error(P.err, CSA_ERR_TIMEOUT);
        const uint64_t t0 = ptx::globaltimer_ns();
        while (ptx::globaltimer_ns() - t0 < 100000ull) {}
        __syncwarp();
        ptx::cluster_sync();
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

}  // namespace csa

extern "C" CSA_API csa_status_t csa_verify_drafts(const void *logits, csa_dtype_t logits_dtype, int64_t seq_stride,
                                                  int64_t token_stride, const void *draft_probs,
                                                  csa_dtype_t draft_dtype, const int32_t *token,
                                                  const int32_t *parent, const float *uniform, const float *noise,
                                                  const float *temperature, int B, int N, int V, int32_t *path,
                                                  int32_t *accepted, int32_t *next_token, void *workspace,
                                                  size_t workspace_bytes, int32_t *status, cudaStream_t stream) {
    using namespace csa;
    (void)workspace;  // (none is needed)
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
    P.wait_ns = wait_limit_ns();
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
