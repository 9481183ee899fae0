// attention_fp4.cu -- sink-merged attention over caches of 4-bit records
// (csa_sink_attention_decode_fp4, hca_sink_attention_decode_fp4), and of a tree's
// drafted tokens over 4-bit or FP8 records (csa_tree_attention_decode,
// hca_tree_attention_decode), on the tensor cores.
//
// For head h over candidates j (x_j the dequantised latent):
//   z_j = scale * q_h . x_j,  o_h = sum_j e^{z_j-M} x_j / (e^{sink_h-M} + sum_j e^{z_j-M}),
//   lse_h = M + ln(den),  M = max(sink_h, max_j z_j).
//
// Work unit = (query token, candidate split), on a cluster of two CTAs. The
// 128 x 512 fp32 output fills all of one SM's tensor memory, so CTA r keeps
// dims [256 r, 256 r + 256) of everything: of the query (in tensor memory), of the
// latents and of the output. Per block of 128 candidates, 64 of which are a CTA's
// own, each CTA runs
//   QK   S = Q[:, own dims] X[:, own dims]^T   M = 128 heads, N = 128, K = 256
//   PV   O += P X[:, own dims]                 M = 128, N = 256 dims, K = 128
// and each latent is unpacked once a pair. Between them the pair exchanges, through
// distributed shared memory: the scores' partial sums (fp32, each sends those of
// the other's own candidates, 32 KB), every head's largest own score (512 B), and
// the softmax weights of the own candidates (BF16, 16 KB). Both scale the weights
// by the same reference maximum: they apply the same rule to the pair of maxima
// (the reference moves only when they exceed it by more than 2^8, log2 domain), so
// neither has to look at the other's decision. The weights are computed with the
// old reference while the maxima travel, and the next block's partial sums travel
// while PV runs.
//
// The weights are BF16 because the latents are: an MMA takes both operands in one
// type, and FP16 would not hold every latent. Their sum adds the unrounded ones, so
// the log-sum is free of that rounding; the output's error against 64 bits is 0.0019
// (its norm over the output's), of which its own BF16 is 0.0017.
//
// Warps: one resolves the records and fetches their lines into L2; eight unpack
// them, exactly (see csa_format_t), from global memory into the MMA's layout in
// two buffers of a block, the next block's bytes in registers meanwhile;
// one issues the MMAs, QK(i + 1) before PV(i); eight do the softmax and the
// epilogue, two threads a head.
//
// Measured: 32 queries of 2176 candidates 44.1 us (414 TFLOP/s, 0.22 of the cuBLAS
// rate; FP8 records: 57), 64 queries of 8320 candidates 198 us (703 TFLOP/s, 0.38;
// FP8 records: 313), 24 ragged queries 20.5 us, one query of 192 candidates 14.3.
// A block takes 5700 cycles, of which the tensor core works a third. What sets the
// pace is the way of a block through its buffer, two of which are all that fits:
// unpacking 2 x 950 cycles, QK 1300, the exchange of the partial sums 1700, softmax
// 2500, the weights' way to the other CTA 1000, PV 1300. (Scores split by candidate,
// which need no partial sums but 64-column MMAs and one and a half times the
// unpacking, took 222 us; more warps for the unpacking, the softmax or the exchange
// cost registers, and all were slower.)
//
// A tree's token differs in its window alone: the pointer warp walks up its ancestors
// and takes their records from the drafts. 8 x 8 tokens of 2176 candidates take 62 us,
// 4 x 32 of 8320 382 in equal parts and 389 dealt out (see deal_units_kernel).
//
// FP8 latents (a code times an fp32 multiplier of 128 dims) do not fit BF16. Rounded
// once, they move each score by 10^-3 and the log-sums by 4 10^-5 of their value, so the
// scores take them as two BF16 numbers, the rounded value and the rest (2^-17 of it is
// lost): q . x = q . bf16(x) + q . bf16(x - bf16(x)). PV takes the rounded ones, whose
// error there is of the size of the weights'. The rests, 64 candidates x 64 dims at a time,
// pass through a ring of three 8 KB buffers, all that fits. That makes a block 9000
// cycles: 7 x 4 ragged chains over 2048 entries, two parts each, 48.2 us (with rounded
// latents 38.7; dealt out 38.3). Tried on the two parts: the rests of a whole block before
// its rounded values in the same buffer, unpacked twice, 61.2 us; one buffer of 64 dims of
// the block 50.8; issuing PV as soon as its weights are there, between the pieces of QK, no
// change. Tried on the dealt ones: both chunks' pieces behind one fence 38.9; buffers of 32
// dims of both chunks, whose MMAs are 128 columns wide, 40.2.
#include <cuda_fp4.h>

#include "rows.cuh"

namespace csa {

namespace {

constexpr int kChunk = 64;                 // candidates of a block that a CTA owns
constexpr int kBlock = 2 * kChunk;         // candidates a block
constexpr int kHalf = 256;                 // output dims per CTA
constexpr int kConvWarps = 8;              // unpacking: warps 0..7, four threads a candidate, 64 at a time
constexpr int kSoftWarps = 8;              // softmax and epilogue: warps 8..15, two threads a head
constexpr int kPtrWarp = 16;               // record pointers
constexpr int kMmaWarp = 17;               // MMA issuer, TMEM owner
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kSoftCols = kChunk / 2;      // scores per softmax thread
constexpr int kAtom = kBlock * 128;        // 128 candidates x 64 dims, 128-byte swizzled rows
constexpr int kBlockBytes = 4 * kAtom;     // 128 candidates x 256 dims, 64 KB
constexpr int kPtrRing = 4;                // blocks of resolved record pointers
constexpr int kRests = 3;                  // buffers of rests (FP8)
constexpr int kDealtRows = 304;            // the most queries that are dealt out
constexpr int kMaxSplits = 96;             // the most units of a query
constexpr uint32_t kWarp = 0xffffffffu;
constexpr int kPieces = kHalf / 32 / 2;    // 32-column pieces of the output per softmax thread
constexpr int kFp4RowBytes = kDim / 2;     // E2M1 output bytes per head
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.f;               // the reference moves only by more than 2^8

constexpr uint32_t kColQ = 0;    // 128 columns: the own dims of Q, BF16 pairs
constexpr uint32_t kColS = 128;  // 128 columns: scores, own candidates first
constexpr uint32_t kColO = 256;  // 256 columns: O half, fp32
constexpr uint32_t kTmemCols = 512;

// (The rests take their 24 KB with FP8 records alone: the longest 4-bit calls took 198.6 us
// instead of 198.0 with them. With 4-bit records their place is 1 KB, so that what follows
// stays on its 128-byte lines: off them, behind 16 bytes, the same calls took 204.)
template <int FMT>
struct AttSmem {
    alignas(1024) uint8_t x[2][kBlockBytes];
    alignas(1024) uint8_t p[kHeads * 128];     // own weights (K-major 128-byte rows)
    alignas(1024) uint8_t pp[kHeads * 128];    // the other CTA's weights
    alignas(1024) uint8_t rest[FMT == CSA_FORMAT_FP8 ? kRests : 1][FMT == CSA_FORMAT_FP8 ? kAtom / 2 : 1024];
                                               // what rounding left of 64 candidates x 64 dims
    float4 part[2][kSoftCols / 4][kHeads];     // the other CTA's part of the own scores
    float pmax[2][4][kHeads];                  // maxima: own CTA's halves, the other CTA's halves
    const uint8_t *rec[kPtrRing][kBlock];      // records: the own chunk's, then the other CTA's (nullptr: none)
    uint32_t vmask[kPtrRing][2];               // which own candidates exist
    uint64_t x_full[2], x_empty[2][2];         // of a buffer; of its chunks
    uint64_t rest_full[kRests], rest_empty[kRests];
    uint64_t ptr_full[kPtrRing], ptr_empty[kPtrRing];
    uint64_t s_full, s_free, part_full, p_full, pp_full, max_full[2], o_done, q_ready, mma_done, pair[4];
    uint8_t chain[CSA_MAX_TOKENS_PER_SEQ];  // a tree's token and its ancestors, the youngest first
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(AttSmem<CSA_FORMAT_FP8>) + 1024 <= 232448, "shared memory plan exceeds the per-CTA limit");

struct Params {
    const __nv_bfloat16 *q;
    const float *sink;
    float scale_log2;  // softmax scale * log2(e)
    CacheView comp;
    const uint8_t *ring;
    int R, W;
    const int32_t *topk_idx, *topk_cnt, *n_comp, *q_pos;
    int m_hca, hca, T, k, n_split;
    __nv_bfloat16 *out;
    float *lse;
    __half *part_o;         // [units, 128, 512] FP16 of split queries, each 32 dims to a power of two:
    uint8_t *part_ex;       // [units, 128, 16] their exponents (see part_unit)
    float2 *part_ml;        // [units, 128] (max, sum) in log2 units
    uint8_t *out_fp4;       // null: BF16 output
    float *out_fp4_scale;
    int inv_rope;
    uint64_t turn[kRope / 2];
    const uint8_t *draft;   // [B, T] records of a tree's tokens, and their parents (null: no tree)
    const int32_t *parent;
    int4 *dealt;            // [pairs] units as deal_units_kernel makes them (query, split, splits of the
    int2 *row_units;        // query, blocks), [rows] a query's first unit and how many it has; else null
    int rows, pairs, round;  // queries, pairs launched, pairs that run at once
    int *err;
    uint64_t wait_ns;  // limit of each bounded wait (drains keep kDrainWaitNs)
};

// Queries of an ordinary call, and a tree's, split in equal parts or as dealt out.
enum Plan { kNoTree, kTree, kTreeDealt };

// Selected entries of query r (of sequence b), and its candidates with the window's. (A tree's
// padding has none, whatever the caller's selection left in its rows. The attention passes the
// b that it has: a second division ahead of these loads made its calls 0.2 us longer.)
struct Candidates {
    int p, n_sel, n;
    __device__ __forceinline__ Candidates(const Params &P, int r, int b, bool tree) {
        p = __ldg(P.q_pos + r);
        if (P.hca) {
            n_sel = visible_entries(p, P.m_hca, __ldg(P.n_comp + b), P.comp.seq_capacity);
        } else {
            const int c = tree && p < 0 ? 0 : __ldg(P.topk_cnt + r);
            n_sel = c < 0 ? 0 : (c > P.k ? P.k : c);
        }
        n = n_sel + (p >= 0 ? p - max(0, p - P.W + 1) + 1 : 0);
    }
};

// The candidates of a work unit: [cb, ce) of the row's selected entries
// followed by its window.
struct Unit {
    int r, b, p, n_sel, j0, cb, ce, n_blocks;
};

template <Plan PLAN>
__device__ __forceinline__ Unit make_unit(const Params &P) {
    Unit u;
    const int pair = blockIdx.x >> 1;
    int split, per;
    if (PLAN == kTreeDealt) {
        const int4 d = P.dealt[pair];
        u.r = max(d.x, 0);
        split = d.x < 0 ? -1 : d.y;
        per = d.w * kBlock;
    } else {
        u.r = pair / P.n_split;
        split = pair % P.n_split;
    }
    u.b = u.r / P.T;
    const Candidates c(P, u.r, u.b, PLAN != kNoTree);
    u.p = c.p;
    u.n_sel = c.n_sel;
    u.j0 = max(0, u.p - P.W + 1);
    if (PLAN != kTreeDealt) per = ((c.n + P.n_split - 1) / P.n_split + kBlock - 1) / kBlock * kBlock;
    if (PLAN == kTreeDealt && split < 0) u.p = -1, split = 0, per = 0;  // a pair without a unit: as padding
    u.cb = min(c.n, split * per);
    u.ce = min(c.n, u.cb + per);
    u.n_blocks = (u.ce - u.cb + kBlock - 1) / kBlock;
    return u;
}

// Deals out the queries of a tree step, whose lengths differ (positions, selections, padding),
// to the pairs: units of up to c blocks, the smallest c with which they fill w rounds of all
// pairs, w and c for the least w (c + kUnitCost), a unit costing that many blocks besides
// its own, and the combine of what is split. (Equal parts, pairs / queries rounded down
// a query, leave pairs idle: 7 x 4 ragged HCA chains took 48.2 us with two parts each, 38.2
// dealt out; 5 x 8 of 65 blocks 190 whole and 156 dealt out, ragged ones 177 and 90. Done at the
// start of each CTA instead, the registers that it takes made every block 12 % longer.)
// One warp, kEach queries a lane.
constexpr float kUnitCost = 2.5f, kPartCost = 0.015f;
template <int kEach>
__global__ void __launch_bounds__(32) deal_units_kernel(const __grid_constant__ Params P) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the attention sets up meanwhile)
    ptx::griddep_wait();
    const int lane = threadIdx.x;
    int blocks[kEach], most = 1, live = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        blocks[j] = 0;
        if (32 * j + lane < P.rows) {
            const int r = 32 * j + lane;
            const Candidates c(P, r, r / P.T, true);
            if (c.p >= 0) blocks[j] = max(1, (c.n + kBlock - 1) / kBlock);  // (one without candidates has its output)
        }
        most = max(most, blocks[j]);
        live += blocks[j] > 0;
    }
    most = __reduce_max_sync(kWarp, most);
    live = __reduce_add_sync(kWarp, live);
    auto parts = [](int b, float of_c, int c) {  // ceil(b / c): within one by floats (b <= 2^24), then as whole numbers
        int q = (int)((float)(b + c - 1) * of_c);
        q += q * c < b ? 1 : 0;
        return q - ((q - 1) * c >= b ? 1 : 0);
    };
    auto units = [&](int c) {
        const float of_c = 1.f / (float)c;
        int n = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) n += parts(blocks[j], of_c, c);
        return (int)__reduce_add_sync(kWarp, n);
    };
    int best = most;
    float least = INFINITY;
    for (int w = max(1, (live + P.round - 1) / P.round); w * P.round <= P.pairs; ++w) {
        int lo = (most + kMaxSplits - 1) / kMaxSplits, hi = most;
        while (lo < hi) {
            const int c = (lo + hi) >> 1;
            if (units(c) <= w * P.round) hi = c;
            else lo = c + 1;
        }
        const int n = units(lo);
        const float time = w * (lo + kUnitCost) + (n > live ? kPartCost * n : 0.f);
        if (time < least) least = time, best = lo;
    }
    int next = 0;
    const float of_best = 1.f / (float)best;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int n = parts(blocks[j], of_best, best);
        int end = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kWarp, end, o);
            if (lane >= o) end += v;
        }
        end += next;
        const int r = 32 * j + lane;
        if (r < P.rows) P.row_units[r] = make_int2(end - n, n);
        for (int i = 0; i < n; ++i) P.dealt[end - n + i] = make_int4(r, i, n, best);
        next = __shfl_sync(kWarp, end, 31);
    }
    for (int i = next + lane; i < P.pairs; i += 32) P.dealt[i] = make_int4(-1, 0, 1, 0);
}

// The larger magnitude, NaN if one is (a plain maximum would drop it).
__device__ __forceinline__ float max_magnitude(float m, float v) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v)));
    return m;
}

// E2M1 multiplier of values of this largest magnitude: 1 when all are zero, NaN when
// one is (E2M1 has no code for it).
__device__ __forceinline__ float e2m1_scale(float amax) { return amax == 0.f ? 1.f : amax / 6.f; }

// A factor for values of this magnitude so that the reciprocal of their E2M1
// multiplier stays in range.
__device__ __forceinline__ float upscale(float amax) { return amax < 7.9e-31f ? 1.2676506002282294e30f : 1.f; }

// A split's output is kept as FP16 with a power of two for every 32 dims, their
// amax's exponent field ex: value = half * part_unit(ex), the halves below 2^15. So
// the detour costs 2^-12 of a value (BF16 made it 2^-9, half of the whole call's
// error) at any magnitude, and fp32 would double the bytes. (From ex = 32 up, so
// that the unit is a normal number: the halves then end 2^-133, as BF16 does.)
__device__ __forceinline__ uint32_t part_exponent(float amax) { return max(__float_as_uint(amax) >> 23, 32u); }
__device__ __forceinline__ float part_unit(uint32_t ex) { return __uint_as_float((ex - 14u) << 23); }
__device__ __forceinline__ float part_factor(uint32_t ex) { return __uint_as_float((268u - ex) << 23); }

// 16-byte chunk cc of row `row` of a swizzled block of 128-byte rows.
__device__ __forceinline__ uint4 *sw128(uint8_t *block, int row, int cc) {
    return reinterpret_cast<uint4 *>(block + row * 128 + ((cc ^ (row & 7)) << 4));
}

// ---------------------------------------------------------------- PTX of the pair

// One lane of a converged warp, the same for every call.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}

// Arrive on the barrier at this offset in both CTAs of the pair when the MMAs
// issued so far by this thread are done.
__device__ __forceinline__ void commit_both(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            ptx::smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// Store into the other CTA, counted (4 bytes) on a barrier there. (A store and a
// releasing arrive would make the warp wait for the store's way there.)
__device__ __forceinline__ void store_to_peer(uint32_t addr, float v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
                 "r"(__float_as_uint(v)), "r"(bar)
                 : "memory");
}
// Copy into the other CTA, counted on a barrier there.
__device__ __forceinline__ void copy_to_peer(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "r"(ptx::smem_u32(src)), "r"(bytes), "r"(bar)
        : "memory");
}

// Bounded wait of a whole warp: true when the phase is complete for every lane,
// and what the other CTA stored before it arrived is visible. One (suspending)
// try is in line, the rest out of it (in line at every wait, the roles' loops take
// more of the instruction cache: 203 us instead of 198 for the longest calls).
__device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort, uint64_t limit_ns) {
    return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, abort, limit_ns) && ptx::try_wait_cluster(bar, parity)) != 0;
}

// ---------------------------------------------------------------- unpacking

// 8 E2M1 codes times s -> 8 BF16 values (exact).
__device__ __forceinline__ uint4 unpack8(uint32_t w, float2 s) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(w >> (8 * i)), __NV_E2M1);
        const float2 v = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2 *>(&h)), s);
        o[i] = pack_bf16(v.x, v.y);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// A thread's quarter of a record's own half, as it lies in the record: four units
// of 16 dims, 64 apart (the last unit of the upper half is 16 rope dims).
template <int FMT>
struct Quarter;

template <>
struct Quarter<CSA_FORMAT_FP4> {
    uint2 code[4];
    uint4 rope[2];
    uint4 scale;  // byte hq of word i: unit i's
    uint32_t power;
    __device__ __forceinline__ void load(const uint8_t *rec, int rank, int hq) {
#pragma unroll
        for (int i = 0; i < 4; ++i) code[i] = make_uint2(0, 0);
        rope[0] = rope[1] = scale = make_uint4(0, 0, 0, 0);  // no record: zero latents
        power = 0;
        if (!rec) return;
        const uint8_t *own = rec + rank * (kHalf / 2) + 8 * hq;
#pragma unroll
        for (int i = 0; i < 3; ++i) code[i] = __ldcs(reinterpret_cast<const uint2 *>(own + 32 * i));
        scale = __ldcs(reinterpret_cast<const uint4 *>(rec + kFp4ScaleOffset + 16 * rank));
        if (rank == 0) {
            code[3] = __ldcs(reinterpret_cast<const uint2 *>(own + 96));
            power = __ldcs(reinterpret_cast<const uint32_t *>(rec + kFp4PowerOffset));
        } else {
            const uint4 *r = reinterpret_cast<const uint4 *>(rec + kFp4RopeOffset + 32 * hq);
            rope[0] = __ldcs(r);
            rope[1] = __ldcs(r + 1);
            power = scale.w;  // (bytes 380..383)
        }
    }
    // to column block i of a row at lo / hi (16-byte chunks 2 hq and 2 hq + 1)
    __device__ __forceinline__ void unpack(int rank, int hq, uint4 *lo, uint4 *hi) const {
        constexpr int kStep = kAtom / 16;
        const float pw = fp4_power(power & 0xFFu);
        const uint32_t sw[4] = {scale.x, scale.y, scale.z, scale.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i == 3 && rank == 1) {
                lo[i * kStep] = rope[0];
                hi[i * kStep] = rope[1];
                break;
            }
            const float s = e4m3x2_to_float2((uint16_t)((sw[i] >> (8 * hq)) & 0xFFu)).x * pw;
            lo[i * kStep] = unpack8(code[i].x, make_float2(s, s));
            hi[i * kStep] = unpack8(code[i].y, make_float2(s, s));
        }
    }
};

// 8 E4M3 codes times a multiplier: as BF16 (rounded once), and what that rounding left, as
// BF16.
__device__ __forceinline__ void unpack8_e4m3(uint32_t w0, uint32_t w1, float s, uint4 &whole, uint4 &rest) {
    const uint32_t w[2] = {w0, w1};
    uint32_t o[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint16_t two = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        const float2 a = __fmul2_rn(e4m3x2_to_float2(two), make_float2(s, s));
        o[i] = pack_bf16(a.x, a.y);
        l[i] = pack_bf16(a.x - __uint_as_float(o[i] << 16), a.y - __uint_as_float(o[i] & 0xFFFF0000u));
    }
    whole = make_uint4(o[0], o[1], o[2], o[3]);
    rest = make_uint4(l[0], l[1], l[2], l[3]);
}

template <>
struct Quarter<CSA_FORMAT_FP8> {
    uint4 piece[5];  // the units' codes; of the upper half three units', and its rope dims
    float2 mult;     // multipliers of the half's two 128-dim blocks
    __device__ __forceinline__ void load(const uint8_t *rec, int rank, int hq) {
#pragma unroll
        for (int i = 0; i < 5; ++i) piece[i] = make_uint4(0, 0, 0, 0);  // no record: zero latents
        mult = make_float2(0.f, 0.f);
        if (!rec) return;
        const uint4 *own = reinterpret_cast<const uint4 *>(rec + rank * kHalf) + hq;
#pragma unroll
        for (int i = 0; i < 3; ++i) piece[i] = __ldcs(own + 4 * i);
        const uint4 *last = rank == 0 ? own + 12 : reinterpret_cast<const uint4 *>(rec + kRopeOffset) + 2 * hq;
        piece[3] = __ldcs(last);
        if (rank == 1) piece[4] = __ldcs(last + 1);
        mult = __ldcs(reinterpret_cast<const float2 *>(rec + kScaleOffset) + rank);
    }
    // unit i's two 16-byte chunks, to lo and hi, and their rests (rope dims are BF16:
    // none)
    __device__ __forceinline__ void unpack(int i, int rank, uint4 *lo, uint4 *hi, uint4 (&rest)[2]) const {
        if (i == 3 && rank == 1) {
            *lo = piece[3];
            *hi = piece[4];
            return;
        }
        const float s = i < 2 ? mult.x : mult.y;
        uint4 whole[2];
        unpack8_e4m3(piece[i].x, piece[i].y, s, whole[0], rest[0]);
        unpack8_e4m3(piece[i].z, piece[i].w, s, whole[1], rest[1]);
        *lo = whole[0];
        *hi = whole[1];
    }
};

// ---------------------------------------------------------------- the kernel

template <int FMT, Plan PLAN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
attention_fp4_kernel(const __grid_constant__ Params P) {
    constexpr int kRecordBytes = FMT == CSA_FORMAT_FP4 ? kFp4Bytes : kRecBytes;
    constexpr bool kFp8 = FMT == CSA_FORMAT_FP8;  // (whose latents BF16 does not hold)
    constexpr bool TREE = PLAN != kNoTree;
    extern __shared__ uint8_t smem_raw[];
    AttSmem<FMT> &s = *reinterpret_cast<AttSmem<FMT> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x & 1;  // = the CTA's rank in its cluster
    volatile int *abort = &s.abort_flag;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&s.x_full[i], 2 * kConvWarps);  // both chunks of a block
            for (int c = 0; c < 2; ++c) ptx::mbar_init(&s.x_empty[i][c], 1);
        }
        for (int i = 0; i < kPtrRing; ++i) {
            ptx::mbar_init(&s.ptr_full[i], 32);  // every lane of the pointer warp
            ptx::mbar_init(&s.ptr_empty[i], kConvWarps + kSoftWarps);
        }
        for (int i = 0; kFp8 && i < kRests; ++i) {
            ptx::mbar_init(&s.rest_full[i], kConvWarps);
            ptx::mbar_init(&s.rest_empty[i], 1);
        }
        ptx::mbar_init(&s.s_full, 1);
        ptx::mbar_init(&s.s_free, kSoftWarps);
        ptx::mbar_init(&s.part_full, kSoftWarps);  // (and the other CTA's bytes)
        ptx::mbar_init(&s.p_full, kSoftWarps);
        ptx::mbar_init(&s.pp_full, 1);
        for (int i = 0; i < 2; ++i) ptx::mbar_init(&s.max_full[i], kSoftWarps);  // (and the other CTA's bytes)
        ptx::mbar_init(&s.o_done, 2);  // both CTAs' PV of a block
        for (int i = 0; i < 4; ++i) ptx::mbar_init(&s.pair[i], 2);
        ptx::mbar_init(&s.q_ready, kSoftWarps);
        ptx::mbar_init(&s.mma_done, 1);
        s.abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == kMmaWarp) ptx::tmem_alloc(&s.tmem_base, kTmemCols);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();  // the other CTA's barriers exist before anything is sent to it
    ptx::tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    ptx::griddep_wait();
    const Unit u = make_unit<PLAN>(P);

    auto fail = [&]() {
        report_error(P.err, CSA_ERR_TIMEOUT);
        *abort = 1;
    };
    const bool poll = P.wait_ns < ptx::kPollOnlyBelowNs;  // (a diagnostic limit: no suspension outlasts it)
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        const bool now = poll ? ptx::mbar_test_wait(bar, parity) : ptx::mbar_try_wait(bar, parity);
        return __all_sync(0xffffffffu, now) || wait_slow(bar, parity, abort, P.wait_ns);
    };
    auto wait_peer = [&](uint64_t *bar, uint32_t parity) {
        const bool now = !poll && ptx::try_wait_cluster(bar, parity);
        return __all_sync(0xffffffffu, now) || wait_slow(bar, parity, abort, P.wait_ns);
    };
    if (warp == kPtrWarp) {
        // ------------------------------------------------------------ record pointers
        // Lane L resolves candidates L, L + 32, .. of a block (own chunk first) in
        // three stages, one block apart, so that no stage waits for the load it
        // started: entry (top-k list), page (block table), record.
        // Of a tree's window the last `own` positions are its token and the token's
        // ancestors, found by walking up from it while the first entries and pages are
        // under way: lane L holds the parents of tokens L, L + 32, ..
        int own = 0;
        const bool walk = TREE && u.ce > u.n_sel;
        int up[CSA_MAX_TOKENS_PER_SEQ / 32];
#pragma unroll
        for (int j = 0; j < CSA_MAX_TOKENS_PER_SEQ / 32; ++j)
            up[j] = walk && 32 * j + lane < P.T ? __ldg(P.parent + (int64_t)u.b * P.T + 32 * j + lane) : -1;
        auto cand = [&](int i, int e) {
            return u.cb + i * kBlock + (e < 2 ? rank : rank ^ 1) * kChunk + (e & 1) * 32 + lane;
        };
        auto load_entry = [&](int i, int e) {
            const int c = cand(i, e);
            if (P.hca || c >= u.ce || c >= u.n_sel) return c;
            return __ldg(P.topk_idx + (size_t)u.r * P.k + c);
        };
        // the physical page of an entry, -1 for none (0 without a block table)
        auto load_page = [&](int i, int e, int entry) {
            const int c = cand(i, e);
            if (c >= u.ce || c >= u.n_sel) return 0;
            if (entry < 0 || entry >= P.comp.seq_capacity) return -1;
            if (!P.comp.block_table) return 0;
            const int page = entry / P.comp.page_records;
            return page < P.comp.max_pages ? __ldg(P.comp.block_table + (int64_t)u.b * P.comp.max_pages + page) : -1;
        };
        auto record = [&](int i, int e, int entry, int page) -> const uint8_t * {
            const int c = cand(i, e);
            if (c >= u.ce) return nullptr;
            if (c >= u.n_sel) {
                const int pos = u.j0 + (c - u.n_sel);
                if (TREE && u.p - pos < own)
                    return P.draft + ((int64_t)u.b * P.T + s.chain[u.p - pos]) * kRecordBytes;
                return P.ring + ((int64_t)u.b * P.R + pos % P.R) * kRecordBytes;
            }
            const int64_t ri = P.comp.block_table ? (int64_t)page * P.comp.page_records + entry % P.comp.page_records
                                                  : (int64_t)u.b * P.comp.seq_stride + entry;
            if (page >= 0 && ri < P.comp.n_records) return P.comp.base + ri * kRecordBytes;
            if (rank == 0) report_error(P.err, CSA_ERR_BAD_INDEX);
            return nullptr;
        };
        int entry[4], page[4], next_entry[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) entry[e] = u.n_blocks > 0 ? load_entry(0, e) : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) next_entry[e] = u.n_blocks > 1 ? load_entry(1, e) : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) page[e] = u.n_blocks > 0 ? load_page(0, e, entry[e]) : 0;
        if (walk) {
            const int most = min(min(P.W - 1, u.p) + 1, P.T);  // (position 2^31 - 1 has a window too)
#pragma unroll 1
            for (int node = u.r - u.b * P.T; node >= 0 && own < most; ++own) {
                if (lane == 0) s.chain[own] = (uint8_t)node;
                int next = -1;
#pragma unroll
                for (int j = 0; j < CSA_MAX_TOKENS_PER_SEQ / 32; ++j) {
                    const int v = __shfl_sync(0xffffffffu, up[j], node & 31);
                    if (node >> 5 == j) next = v;
                }
                if (next >= node || next < -1) {  // (a parent comes before its children: the walk ends)
                    if (rank == 0 && lane == 0) report_error(P.err, CSA_ERR_BAD_INDEX);
                    next = -1;
                }
                node = next;
            }
            __syncwarp();
        }
#pragma unroll 1
        for (int i = 0; i < u.n_blocks; ++i) {
            const int pr = i % kPtrRing;
            if (!wait(&s.ptr_empty[pr], ((i / kPtrRing) & 1) ^ 1)) { fail(); break; }
            uint32_t have[2];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint8_t *rec = record(i, e, entry[e], page[e]);
                s.rec[pr][e * 32 + lane] = rec;
                // into L2 while the block is up to kPtrRing blocks away (each CTA
                // its own candidates: the pair reads both; one line a prefetch,
                // since a bulk prefetch takes as long as a bulk copy)
                if (e < 2 && rec) {
#pragma unroll
                    for (int b = 0; b < kRecordBytes; b += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(rec + b));
                    // (an FP8 record need not begin with a line: its last one)
                    if (kRecordBytes % 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(rec + kRecordBytes - 16));
                }
                if (e < 2) have[e] = __ballot_sync(0xffffffffu, rec != nullptr);
                entry[e] = next_entry[e];
                if (i + 1 < u.n_blocks) page[e] = load_page(i + 1, e, entry[e]);
                if (i + 2 < u.n_blocks) next_entry[e] = load_entry(i + 2, e);
            }
            if (lane == 0) {
                s.vmask[pr][0] = have[0];
                s.vmask[pr][1] = have[1];
            }
            ptx::mbar_arrive(&s.ptr_full[pr]);
        }
    } else if (warp < kConvWarps) {
        // ------------------------------------------------------------ unpack
        // Of every block 64 own candidates and 64 of the other CTA's, four threads a
        // candidate; the bytes of a chunk are under way while the block before it is
        // unpacked.
        const int row = threadIdx.x >> 2, hq = threadIdx.x & 3;
        Quarter<FMT> own, other;
        auto fetch = [&](int i, int chunk, Quarter<FMT> &q) {
            q.load(s.rec[i % kPtrRing][chunk * kChunk + row], rank, hq);
        };
        auto unpack = [&](int i, int chunk, const Quarter<FMT> &q) {
            if constexpr (!kFp8) {
                const int r = chunk * kChunk + row, b = i & 1;
                q.unpack(rank, hq, sw128(s.x[b], r, 2 * hq), sw128(s.x[b], r, 2 * hq + 1));
                ptx::fence_proxy_async_smem();  // generic-proxy stores -> MMA (async proxy) reads
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&s.x_full[b]);
            }
        };
        // FP8: 64 dims of a chunk at a time, and their rests, which go into the scores from
        // a ring of buffers
        int slot = 0;
        uint32_t turn = 1;  // parity of the ring's last turn
        auto unpack_dims = [&](int i, int a, int chunk, const Quarter<FMT> &q) {
            if constexpr (kFp8) {
                uint8_t *x = s.x[i & 1] + a * kAtom;
                uint4 rest[2];
                q.unpack(a, rank, sw128(x, chunk * kChunk + row, 2 * hq), sw128(x, chunk * kChunk + row, 2 * hq + 1), rest);
                if (!wait(&s.rest_empty[slot], turn)) return false;
                if (a < 3 || rank == 0) {
                    *sw128(s.rest[slot], row, 2 * hq) = rest[0];
                    *sw128(s.rest[slot], row, 2 * hq + 1) = rest[1];
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&s.rest_full[slot]);
                if (++slot == kRests) slot = 0, turn ^= 1;
            }
            return true;
        };
        bool ok = true;
        if (u.n_blocks > 0) {
            ok = wait(&s.ptr_full[0], 0);
            if (ok) fetch(0, 0, own);
            if (ok) fetch(0, 1, other);
        }
#pragma unroll 1
        for (int i = 0; i < u.n_blocks && ok; ++i) {
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&s.ptr_empty[i % kPtrRing]);  // (both chunks' pointers have been read)
            const int n = i + 1;
            const bool more = n < u.n_blocks;
            ok = !more || wait(&s.ptr_full[n % kPtrRing], n / kPtrRing & 1);
            ok = ok && wait(&s.x_empty[i & 1][0], (i >> 1 & 1) ^ 1);
            if (!ok) break;
            unpack(i, 0, own);
            ok = wait(&s.x_empty[i & 1][1], (i >> 1 & 1) ^ 1);
            if (!ok) break;
            unpack(i, 1, other);
            if (kFp8) {
#pragma unroll
                for (int a = 0; a < 4; ++a) ok = ok && unpack_dims(i, a, 0, own) && unpack_dims(i, a, 1, other);
                if (!ok) break;
            }
            if (more) {
                fetch(n, 0, own);
                fetch(n, 1, other);
            }
        }
        if (!ok) fail();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA issuer
        constexpr uint32_t kIdescQK = ptx::idesc_f32acc(1, 1, 128, kBlock);
        constexpr uint32_t kIdescPV = ptx::idesc_f32acc(1, 1, 128, kHalf, 1);
        const uint32_t leader = elect_one();
        bool ok = u.n_blocks == 0 || wait(&s.q_ready, 0);
        auto pv = [&](const uint8_t *w, const uint8_t *x, bool first) {
            const uint64_t ad = ptx::desc_kmajor_sw128(ptx::smem_u32(w));
            const uint64_t bd = ptx::desc_mnmajor_sw128(ptx::smem_u32(x), kAtom, 1024);
            if (!leader) return;
#pragma unroll
            for (int k = 0; k < kChunk / 16; ++k)
                ptx::mma_f16(tmem + kColO, ad + (uint64_t)(k * 32 >> 4), bd + (uint64_t)(k * 2048 >> 4), kIdescPV,
                             !(first && k == 0));
        };
        int slot = 0;       // of the rests' ring (FP8), and
        uint32_t turn = 0;  // the parity of its turn
#pragma unroll 1
        for (int i = 0; i <= u.n_blocks && ok; ++i) {
            if (i < u.n_blocks) {  // QK(i)
                const uint64_t xd = ptx::desc_kmajor_sw128(ptx::smem_u32(s.x[i & 1]));
                auto qk = [&](int k) {  // dims [16 k, 16 k + 16)
                    ptx::mma_f16_ts(tmem + kColS, tmem + kColQ + k * 8,
                                    xd + (uint64_t)(((k >> 2) * kAtom + (k & 3) * 32) >> 4), kIdescQK, kFp8 || k > 0);
                };
                if (kFp8) {
                    // the rests of a chunk's 64 dims into its half of the scores, then, both
                    // chunks' being there, the 64 dims themselves
                    constexpr uint32_t kIdescRest = ptx::idesc_f32acc(1, 1, 128, kChunk);
#pragma unroll 1
                    for (int dims = 0; dims < 4 && ok; ++dims) {
#pragma unroll
                        for (int chunk = 0; chunk < 2; ++chunk) {
                            ok = ok && wait(&s.rest_full[slot], turn) &&
                                 (dims + chunk > 0 || i == 0 || wait(&s.s_free, (i & 1) ^ 1));
                            if (!ok) break;
                            ptx::tc_fence_after();
                            if (leader) {
                                if (dims < 3 || rank == 0) {  // (the last 64 dims of rank 1 are rope: no rests)
                                    const uint64_t rd = ptx::desc_kmajor_sw128(ptx::smem_u32(s.rest[slot]));
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        ptx::mma_f16_ts(tmem + kColS + chunk * kChunk, tmem + kColQ + (4 * dims + k) * 8,
                                                        rd + k * 2, kIdescRest, dims > 0 || k > 0);
                                }
                                ptx::mma_commit(&s.rest_empty[slot]);
                                if (chunk == 1) {
#pragma unroll
                                    for (int k = 0; k < 4; ++k) qk(4 * dims + k);
                                }
                            }
                            __syncwarp();
                            if (++slot == kRests) slot = 0, turn ^= 1;
                        }
                    }
                    if (!ok) break;
                } else {
                    ok = wait(&s.x_full[i & 1], i >> 1 & 1) && (i == 0 || wait(&s.s_free, (i & 1) ^ 1));
                    if (!ok) break;
                    ptx::tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < kHalf / 16; ++k) qk(k);
                    }
                }
                if (leader) ptx::mma_commit(&s.s_full);
                __syncwarp();
            }
            if (i > 0) {  // PV(i - 1): the own, then the other CTA's candidates
                const uint32_t ph = (i & 1) ^ 1;
                const uint8_t *x = s.x[ph];
                ok = wait(&s.p_full, ph);
                if (!ok) break;
                ptx::tc_fence_after();
                pv(s.p, x, i == 1);
                if (leader) {
                    ptx::mma_commit(&s.x_empty[ph][0]);
                    ptx::mbar_arrive_expect_tx(&s.pp_full, kHeads * 128);
                }
                __syncwarp();
                ok = wait_peer(&s.pp_full, ph);
                if (!ok) break;
                ptx::tc_fence_after();
                pv(s.pp, x + kChunk * 128, false);
                if (leader) {
                    ptx::mma_commit(&s.x_empty[ph][1]);
                    commit_both(&s.o_done);
                }
                __syncwarp();
            }
        }
        if (!ok) fail();
        if (leader) ptx::mma_commit(&s.mma_done);
        __syncwarp();
        // every MMA issued has finished with tensor and shared memory before the
        // CTA frees them (not cut short by the abort flag)
        if (!__all_sync(0xffffffffu, ptx::mbar_wait_drain(&s.mma_done, 0, kDrainWaitNs)))
            report_error(P.err, CSA_ERR_TIMEOUT);
        if (!ok || *abort) {
            // given up: arrivals and copies that were sent to the other CTA (a few
            // KB, microseconds) land long before this bounded pause ends
            const uint64_t t0 = ptx::globaltimer_ns();
            while (ptx::globaltimer_ns() - t0 < 100000ull) {}
        }
    } else {
        // ------------------------------------------------------------ softmax / epilogue
        // Two threads a head: warps 8..11 the first half of the block's scores (and
        // of the output columns), warps 12..15 the second; a warp's TMEM lanes
        // are 32 (warp % 4) ..
        const int quarter = warp & 3, half = (warp - kConvWarps) >> 2;
        const int h = quarter * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t peer_max = ptx::mapa(ptx::smem_u32(&s.pmax[0][2 + half][h]), rank ^ 1);
        const uint32_t peer_max_full = ptx::mapa(ptx::smem_u32(&s.max_full[0]), rank ^ 1);
        const uint32_t peer_part = ptx::mapa(ptx::smem_u32(&s.part[half][0][h]), rank ^ 1);
        const uint32_t peer_part_full = ptx::mapa(ptx::smem_u32(&s.part_full), rank ^ 1);
        const uint32_t peer_pp = ptx::mapa(ptx::smem_u32(s.pp), rank ^ 1);
        const uint32_t peer_pp_full = ptx::mapa(ptx::smem_u32(&s.pp_full), rank ^ 1);
        const bool final_out = PLAN == kTreeDealt ? P.dealt[blockIdx.x >> 1].z == 1 : P.n_split == 1;
        // this thread's maximum of block i (or, at the end, its sum) to the other
        // three threads of the head
        auto send = [&](int i, float v) {
            store_to_peer(peer_max + (i & 1) * (4 * kHeads * 4), v, peer_max_full + (i & 1) * 8);
            s.pmax[i & 1][half][h] = v;
            __syncwarp();
            // (each warp expects the bytes of the other CTA's warp like it)
            if (lane == 0) ptx::mbar_arrive_expect_tx(&s.max_full[i & 1], 32 * 4);
        };
        auto received = [&](int i, int from) { return *reinterpret_cast<volatile float *>(&s.pmax[i & 1][from][h]); };
        bool ok = true;
        if (u.n_blocks > 0) {
            // The own dims of Q -> TMEM (BF16 pairs, lane = head), 64 dims a piece, two
            // of the four pieces a thread. A load takes four heads' 128 bytes (a head a
            // lane would touch 32 lines); the warp's 4 KB of the weights' buffers, not
            // used yet, turn them into a head a lane.
            const int r4 = lane >> 3, c = lane & 7;
            const uint4 *qg = reinterpret_cast<const uint4 *>(
                P.q + ((size_t)u.r * kHeads + quarter * 32 + r4) * kDim + rank * kHalf) + c;
            uint8_t *turn = half ? s.pp + quarter * 4096 : s.p + quarter * 4096;
            const uint64_t policy = ptx::l2_policy_evict_first();
#pragma unroll 1
            for (int pc = 2 * half; pc < 2 * half + 2; ++pc) {
                uint4 w[8];
#pragma unroll
                for (int g = 0; g < 8; ++g) w[g] = ptx::ldg_v4_policy(qg + (size_t)4 * g * (kDim / 8) + 8 * pc, policy);
#pragma unroll
                for (int g = 0; g < 8; ++g) *sw128(turn, 4 * g + r4, c) = w[g];
                __syncwarp();
                uint32_t regs[32];
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                    const uint4 x = *sw128(turn, lane, v);
                    regs[4 * v] = x.x;
                    regs[4 * v + 1] = x.y;
                    regs[4 * v + 2] = x.z;
                    regs[4 * v + 3] = x.w;
                }
                ptx::tmem_st32(lane_base + kColQ + pc * 32, regs);
                __syncwarp();
            }
            ptx::tmem_st_wait();
            ptx::fence_proxy_async_smem();  // the turning buffers -> the other CTA's copies into them
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&s.q_ready);
        }
        // this CTA's part of the other's scores of block i, when QK(i) is done
        auto send_part = [&](int i) {
            if (!wait(&s.s_full, i & 1)) return false;
            ptx::tc_fence_after();
            uint32_t v[kSoftCols];
            ptx::tmem_ld32(lane_base + kColS + kChunk + half * kSoftCols, v);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < kSoftCols / 4; ++c)
                ptx::store4_to_peer(peer_part + c * (kHeads * 16), v + 4 * c, peer_part_full);
            __syncwarp();
            // (each warp expects the bytes of the other CTA's warp like it)
            if (lane == 0) ptx::mbar_arrive_expect_tx(&s.part_full, 32 * 4 * kSoftCols);
            return true;
        };
        if (u.n_blocks > 0 && !send_part(0)) { fail(); ok = false; }
        float m = -INFINITY, l = 0.f;  // reference and own sum, log2 domain, sink not included
#pragma unroll 1
        for (int i = 0; i < u.n_blocks && ok; ++i) {
            const int pr = i % kPtrRing;
            if (!wait(&s.ptr_full[pr], (i / kPtrRing) & 1)) { fail(); ok = false; break; }
            const uint32_t mask = *reinterpret_cast<volatile uint32_t *>(&s.vmask[pr][half]);
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&s.ptr_empty[pr]);
            float z[kSoftCols];  // raw scores, -inf where there is no candidate
            {
                uint32_t sv[kSoftCols];
                ptx::tmem_ld32(lane_base + kColS + half * kSoftCols, sv);
                ptx::tmem_ld_wait();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&s.s_free);
                // (the buffer is free for block i + 1 once this CTA's maxima are sent:
                // the other CTA sends its parts after it has those of block i)
                if (!wait_peer(&s.part_full, i & 1)) { fail(); ok = false; break; }
#pragma unroll
                for (int c = 0; c < kSoftCols / 4; ++c) {
                    const float4 o = s.part[half][c][h];
                    z[4 * c] = __uint_as_float(sv[4 * c]) + o.x;
                    z[4 * c + 1] = __uint_as_float(sv[4 * c + 1]) + o.y;
                    z[4 * c + 2] = __uint_as_float(sv[4 * c + 2]) + o.z;
                    z[4 * c + 3] = __uint_as_float(sv[4 * c + 3]) + o.w;
                }
            }
            if (mask != 0xffffffffu) {
#pragma unroll
                for (int c = 0; c < kSoftCols; ++c)
                    if (!((mask >> c) & 1u)) z[c] = -INFINITY;
            }
            float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < kSoftCols; ++c) mx4[c & 3] = fmaxf(mx4[c & 3], z[c]);
            const float own = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * P.scale_log2;  // (scale > 0)
            // buffer i % 2 is free: every thread of the head sent its maximum of
            // block i - 1 after it had read those of block i - 2
            send(i, own);
            // the weights with the reference as it stands, while the maxima travel
            uint32_t w[kSoftCols / 2];
            float sum;
            auto weights = [&]() {
                const float mref = (m == -INFINITY) ? 0.f : m;  // every z is -inf while m is (or they come again)
                const float2 sc = make_float2(P.scale_log2, P.scale_log2), mm = make_float2(-mref, -mref);
                float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < kSoftCols / 2; ++c) {
                    float2 e = __ffma2_rn(make_float2(z[2 * c], z[2 * c + 1]), sc, mm);
                    e.x = ptx::ex2_approx(e.x);
                    e.y = ptx::ex2_approx(e.y);
                    ps[c & 1] = __fadd2_rn(ps[c & 1], e);
                    w[c] = pack_bf16(e.x, e.y);
                }
                sum = (ps[0].x + ps[0].y) + (ps[1].x + ps[1].y);
            };
            weights();
            if (!wait_peer(&s.max_full[i & 1], (i >> 1) & 1)) { fail(); ok = false; break; }
            const float mx = fmaxf(fmaxf(received(i, 0), received(i, 1)), fmaxf(received(i, 2), received(i, 3)));
            // Both CTAs' PV of block i - 1 is done: O holds the blocks before
            // this one, the own weights have been read here and copied there.
            if (i > 0) {
                if (!wait_peer(&s.o_done, (i - 1) & 1)) { fail(); ok = false; break; }
                ptx::tc_fence_after();
            }
            // Lazy rescale, the same decision in both CTAs. It is per head (lane)
            // but the TMEM accesses are warp-collective, so the whole warp
            // enters when any lane needs it; other lanes use a factor of 1.
            const bool need = mx > m + kLazy || (m == -INFINITY && mx > -INFINITY);
            if (__any_sync(0xffffffffu, need)) {
                const float alpha = need ? ptx::ex2_approx(m - mx) : 1.f;  // 0 when m = -inf
                if (i > 0) {
#pragma unroll 1
                    for (int piece = half * kPieces; piece < half * kPieces + kPieces; ++piece) {
                        uint32_t o[32];
                        ptx::tmem_ld32(lane_base + kColO + piece * 32, o);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        ptx::tmem_st32(lane_base + kColO + piece * 32, o);
                    }
                    ptx::tmem_st_wait();
                    ptx::tc_fence_before();
                }
                l *= alpha;
                if (need) m = mx;
                weights();
            }
            l += sum;
#pragma unroll
            for (int c8 = 0; c8 < kSoftCols / 8; ++c8)
                *sw128(s.p, h, half * (kSoftCols / 8) + c8) = make_uint4(w[4 * c8], w[4 * c8 + 1], w[4 * c8 + 2], w[4 * c8 + 3]);
            ptx::fence_proxy_async_smem();  // weights -> the copy's and PV's (async proxy) reads
            // two warps (the halves) fill the rows of a quarter; the first of them
            // copies it (4 KB) when both have
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(&s.p_full);
                ptx::mbar_arrive(&s.pair[quarter]);
            }
            if (half == 0) {
                if (!wait(&s.pair[quarter], i & 1)) { fail(); ok = false; break; }
                if (lane == 0)
                    copy_to_peer(peer_pp + quarter * 32 * 128, s.p + quarter * 32 * 128, 32 * 128, peer_pp_full);
            }
            if (i + 1 < u.n_blocks && !send_part(i + 1)) { fail(); ok = false; }
        }
        // both halves' warps of a quarter have staged their output columns (the
        // phase before this one is complete: the sums came after it)
        auto rows_staged = [&]() {
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&s.pair[quarter]);
            if (wait(&s.pair[quarter], u.n_blocks & 1)) return true;
            fail();
            return false;
        };
        // the sums travel like one more block's maxima; added in one order by all
        if (ok && u.n_blocks > 0) {
            const int i = u.n_blocks;
            send(i, l);
            if (!wait_peer(&s.max_full[i & 1], (i >> 1) & 1) || !wait_peer(&s.o_done, (i - 1) & 1)) {
                fail();
                ok = false;
            } else {
                const float here = received(i, 0) + received(i, 1), there = received(i, 2) + received(i, 3);
                l = here + there;
            }
            ptx::tc_fence_after();
        }
        // ---------------- epilogue: O half (and LSE) out
        if (ok && !(TREE && u.p < 0)) {  // (a tree's padding keeps its rows)
            const int r = u.r;
            float factor, lse_out = 0.f;
            const float2 ml = make_float2(m, l);
            if (final_out) {
                const float sk = __ldg(P.sink + h) * kLog2e;
                const float M = fmaxf(sk, m);
                const float es = (sk == -INFINITY) ? 0.f : exp2f(sk - M);
                const float eo = (m == -INFINITY) ? 0.f : exp2f(m - M);
                const float den = es + l * eo;
                factor = den > 0.f ? eo / den : 0.f;
                lse_out = l != 0.f ? (M + log2f(den)) * kLn2 : __ldg(P.sink + h);  // no candidates: the sink itself
            } else {
                factor = l != 0.f ? 1.f / l : 0.f;  // (NaN stays)
            }
            const bool rope_here = final_out && P.inv_rope && rank == 1;
            float2 cs = make_float2(1.f, 0.f);  // lane i: cos, sin of rope pair i
            if (rope_here) cs = turn_cos_sin(u.p, P.turn[lane]);
            // piece (32 dims) of this head's O half, normalised and turned back
            auto piece_values = [&](int piece, float (&v)[32]) {
                if (u.n_blocks > 0) {
                    uint32_t o[32];
                    ptx::tmem_ld32(lane_base + kColO + piece * 32, o);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(o[e]) * factor;
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.f;
                }
                if (rope_here && piece >= (kNope - kHalf) / 32) {  // latent dims 448..511
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int pair = (piece - (kNope - kHalf) / 32) * 16 + e;
                        const float c = __shfl_sync(0xffffffffu, cs.x, pair);
                        const float sn = __shfl_sync(0xffffffffu, cs.y, pair);
                        const float x = v[2 * e], y = v[2 * e + 1];
                        v[2 * e] = fmaf(x, c, y * sn);
                        v[2 * e + 1] = fmaf(-x, sn, y * c);
                    }
                }
            };
            // Rows are staged in shared memory (the pieces' buffers are free once
            // every PV is done), then each warp writes its 32 head rows whole.
            // Chunk c (16 B) of row h sits at position c ^ (h & 7).
            uint8_t *ostage = s.x[0];
            if (!(final_out && P.out_fp4)) {
                uint8_t *srow = ostage + h * (kHalf * 2);
                const size_t part = (size_t)(blockIdx.x >> 1) * kHeads;  // (units are numbered in the order of their queries)
                uint32_t exponents = 0;
#pragma unroll 1
                for (int piece = half * kPieces; piece < half * kPieces + kPieces; ++piece) {
                    float v[32];
                    piece_values(piece, v);
                    uint32_t w[16];
                    if (final_out) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
                    } else {
                        float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int e = 0; e < 32; ++e) a[e & 3] = fmaxf(a[e & 3], fabsf(v[e]));
                        const uint32_t ex = part_exponent(fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])));
                        const float f = part_factor(ex);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const __half2 p = __floats2half2_rn(v[2 * e] * f, v[2 * e + 1] * f);
                            w[e] = *reinterpret_cast<const uint32_t *>(&p);
                        }
                        exponents = exponents >> 8 | ex << 24;
                    }
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) {
                        const int c = piece * 4 + q4;
                        *reinterpret_cast<uint4 *>(srow + ((c ^ (h & 7)) << 4)) =
                            make_uint4(w[4 * q4], w[4 * q4 + 1], w[4 * q4 + 2], w[4 * q4 + 3]);
                    }
                }
                static_assert(kPieces == 4, "a thread's exponents are one word");
                if (!final_out) reinterpret_cast<uint32_t *>(P.part_ex)[(part + h) * 4 + rank * 2 + half] = exponents;
                const bool staged = rows_staged();
                const uint64_t policy = ptx::l2_policy_evict_first();
                uint16_t *dst0 = (final_out ? reinterpret_cast<uint16_t *>(P.out) + (size_t)r * kHeads * kDim
                                            : reinterpret_cast<uint16_t *>(P.part_o) + part * kDim) + rank * kHalf;
#pragma unroll 4
                for (int i = 0; i < 16 && staged; ++i) {
                    const int hr = quarter * 32 + 16 * half + i;  // a head row of this warp pair
                    const uint4 v = *reinterpret_cast<const uint4 *>(ostage + hr * (kHalf * 2) + ((lane ^ (hr & 7)) << 4));
                    if (final_out)
                        reinterpret_cast<uint4 *>(dst0 + (size_t)hr * kDim)[lane] = v;
                    else  // split partials are read once, by the combine: evict-first
                        ptx::stg_v4_policy(reinterpret_cast<uint4 *>(dst0 + (size_t)hr * kDim) + lane, v, policy);
                }
            } else {
                // E2M1: two 128-dim blocks per half, each scaled by its amax / 6
                // (a first pass over TMEM finds the amax); 128 B per head row
                uint8_t *frow = ostage + h * (kFp4RowBytes / 2);
                {
                    const int bl = half;
                    float amax = 0.f;
#pragma unroll 1
                    for (int pp = 0; pp < 4; ++pp) {
                        float v[32];
                        piece_values(4 * bl + pp, v);
#pragma unroll
                        for (int e = 0; e < 32; ++e) amax = max_magnitude(amax, v[e]);
                    }
                    const float sc = e2m1_scale(amax);
                    const float up = upscale(amax), inv = 1.f / (sc * up);
                    auto q = [&](float x) { return x * up * inv; };
#pragma unroll 1
                    for (int pp = 0; pp < 4; ++pp) {
                        float v[32];
                        piece_values(4 * bl + pp, v);
                        uint32_t w[4];
#pragma unroll
                        for (int q4 = 0; q4 < 4; ++q4)
                            w[q4] = e2m1x4(q(v[8 * q4]), q(v[8 * q4 + 1]), q(v[8 * q4 + 2]), q(v[8 * q4 + 3])) |
                                    (e2m1x4(q(v[8 * q4 + 4]), q(v[8 * q4 + 5]), q(v[8 * q4 + 6]), q(v[8 * q4 + 7]))
                                     << 16);
                        const int c = 4 * bl + pp;
                        *reinterpret_cast<uint4 *>(frow + ((c ^ (h & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    P.out_fp4_scale[((size_t)r * kHeads + h) * 4 + rank * 2 + bl] = sc;
                }
                const bool staged = rows_staged();
#pragma unroll 2
                for (int i = 0; i < 4 && staged; ++i) {
                    const int hr = quarter * 32 + 16 * half + i * 4 + (lane >> 3);  // 8 lanes per 128-byte row
                    const int c = lane & 7;
                    const uint4 v = *reinterpret_cast<const uint4 *>(ostage + hr * (kFp4RowBytes / 2) + ((c ^ (hr & 7)) << 4));
                    reinterpret_cast<uint4 *>(P.out_fp4 + ((size_t)r * kHeads + hr) * kFp4RowBytes +
                                              rank * (kFp4RowBytes / 2))[c] = v;
                }
            }
            if (rank == 0 && half == 0) {
                if (final_out)
                    P.lse[(size_t)r * kHeads + h] = lse_out;
                else
                    P.part_ml[(size_t)(blockIdx.x >> 1) * kHeads + h] = ml;
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, kTmemCols);
    ptx::cluster_sync();  // nothing is on its way to a CTA that has left
}

// Folds the per-split normalised partials and the sink (log2 domain):
//   M = max(sink, m_s), den = e^{sink-M} + sum_s l_s e^{m_s-M},
//   out = sum_s l_s e^{m_s-M} o_s / den, lse = M + ln den.
// kWarps warps per (row, head), each every kWarps'th split, 16 dims per lane; the
// splits' weights are computed once, a split a lane. It is a chain of loads from L2
// (four splits' at once), so many splits are spread over eight warps, whose sums
// are added in their order: 9, 18 and 76 splits of one query took 16.1, 16.2 and
// 18.8 us a call, and with one warp 16.9, 18.2 and 28.7; two splits of 32 queries
// took 46 us with one warp, with eight 68.
constexpr int kCombineBatch = 4;
template <int kWarps, Plan PLAN>
__global__ void __launch_bounds__(256, 3)
combine_fp4_kernel(const __grid_constant__ Params P) {
    static_assert(kWarps == 1 || kWarps == 8, "one head a warp, or one a block");
    __shared__ float4 sums[kWarps > 1 ? kWarps : 1][kWarps > 1 ? kDim / 4 : 1];
    // The next kernel of the stream may be set up now (it waits for this one's end
    // before it touches memory): 0.4 us a call where the next is this attention.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    ptx::griddep_wait();
    const int r = blockIdx.y;
    if (PLAN != kNoTree && __ldg(P.q_pos + r) < 0) return;  // a tree's padding keeps its rows
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x * (8 / kWarps) + warp / kWarps, part = warp % kWarps;
    int n_split = P.n_split;
    int64_t unit = (int64_t)r * n_split;
    if (PLAN == kTreeDealt) {
        const int2 mine = P.row_units[r];
        unit = mine.x;
        n_split = mine.y;
        if (n_split == 1) return;  // (written by its unit)
    }
    const size_t row0 = (size_t)unit * kHeads + h, row_stride = kHeads;  // of the splits' rows
    const uint64_t policy = ptx::l2_policy_evict_first();
    const float sk = __ldg(P.sink + h) * kLog2e;
    // four splits' rows (all splits have written theirs)
    uint32_t ex[kCombineBatch];
    Octet<CSA_FP16> v[kCombineBatch][2];
    auto load = [&](int s0) {
#pragma unroll
        for (int q = 0; q < kCombineBatch; ++q) {
            const int s = s0 + q * kWarps;
            ex[q] = 32;
            v[q][0].clear();
            v[q][1].clear();
            if (s >= n_split) continue;
            const size_t at = row0 + s * row_stride;
            const uint4 *o = reinterpret_cast<const uint4 *>(P.part_o + at * kDim) + lane * 2;
            ex[q] = P.part_ex[at * 16 + (lane >> 1)];
            v[q][0].v = ptx::ldg_v4_policy(o, policy);
            v[q][1].v = ptx::ldg_v4_policy(o + 1, policy);
        }
    };
    float2 ml[kMaxSplits / 32];
#pragma unroll
    for (int j = 0; j < kMaxSplits / 32; ++j) {
        ml[j] = make_float2(-INFINITY, 0.f);
        if (32 * j + lane < n_split) ml[j] = P.part_ml[row0 + (32 * j + lane) * row_stride];
    }
    load(part);  // (while the weights are computed)
    float w[kMaxSplits / 32], M = sk, den = 0.f;
    // (a split without candidates has the sum 0; one with a NaN among them counts)
#pragma unroll
    for (int j = 0; j < kMaxSplits / 32; ++j)
        if (ml[j].y != 0.f) M = fmaxf(M, ml[j].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
    for (int j = 0; j < kMaxSplits / 32; ++j) {
        w[j] = ml[j].y != 0.f ? ml[j].y * exp2f(ml[j].x - M) : 0.f;
        den += w[j];
    }
    float acc[2][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[0][e] = acc[1][e] = 0.f;
#pragma unroll 1
    for (int s0 = part;;) {
#pragma unroll
        for (int q = 0; q < kCombineBatch; ++q) {
            const int s = s0 + q * kWarps;
            float ws = 0.f;
#pragma unroll
            for (int j = 0; j < kMaxSplits / 32; ++j) {
                const float x = __shfl_sync(0xffffffffu, w[j], s & 31);
                if (s >> 5 == j) ws = x;
            }
            if (ws == 0.f) continue;  // (a split that counts for nothing, whatever its row holds)
            const float wu = ws * part_unit(ex[q]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float f[8];
                v[q][e].floats(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[e][i] = fmaf(wu, f[i], acc[e][i]);
            }
        }
        s0 += kCombineBatch * kWarps;
        if (s0 >= n_split) break;
        load(s0);
    }
    if (kWarps > 1) {
        float4 *mine = &sums[part][lane * 4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mine[i] = make_float4(acc[i >> 1][4 * (i & 1)], acc[i >> 1][4 * (i & 1) + 1], acc[i >> 1][4 * (i & 1) + 2],
                                  acc[i >> 1][4 * (i & 1) + 3]);
        __syncthreads();
        if (part != 0) return;
#pragma unroll
        for (int p = 1; p < kWarps; ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 a = sums[p][lane * 4 + i];
                float *to = &acc[i >> 1][4 * (i & 1)];
                to[0] += a.x, to[1] += a.y, to[2] += a.z, to[3] += a.w;
            }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    const bool none = den == 0.f;  // no candidates: lse is the sink itself
    den += (sk == -INFINITY) ? 0.f : exp2f(sk - M);
    const float inv = den > 0.f ? 1.f / den : 0.f;
    float2 cs = make_float2(1.f, 0.f);  // lane i: cos, sin of rope pair i
    if (P.inv_rope) cs = turn_cos_sin(__ldg(P.q_pos + r), P.turn[lane]);
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[e][i] *= inv;
    // lanes 28..31 hold the rope dims 448..511, 8 pairs each
    if (P.inv_rope) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float2 back[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int pair = ((lane - kNope / 16) & 3) * 8 + 4 * e + i;
                back[i].x = __shfl_sync(0xffffffffu, cs.x, pair);
                back[i].y = -__shfl_sync(0xffffffffu, cs.y, pair);
            }
            if (lane >= kNope / 16) turn_octet(acc[e], back);
        }
    }
    const size_t row = (size_t)r * kHeads + h;
    if (P.out_fp4) {
        // E2M1 with one multiplier per 128 dims = 8 lanes
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = max_magnitude(amax, acc[e][i]);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) amax = max_magnitude(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float sc = e2m1_scale(amax);
        const float up = upscale(amax), inv_sc = 1.f / (sc * up);
        auto q = [&](float x) { return x * up * inv_sc; };
        uint32_t w[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            w[e] = e2m1x4(q(acc[e][0]), q(acc[e][1]), q(acc[e][2]), q(acc[e][3])) |
                   (e2m1x4(q(acc[e][4]), q(acc[e][5]), q(acc[e][6]), q(acc[e][7])) << 16);
        reinterpret_cast<uint2 *>(P.out_fp4 + row * kFp4RowBytes)[lane] = make_uint2(w[0], w[1]);
        if ((lane & 7) == 0) P.out_fp4_scale[row * 4 + (lane >> 3)] = sc;
    } else {
        uint4 *dst = reinterpret_cast<uint4 *>(P.out + row * kDim) + lane * 2;
        ptx::stg_v4_policy(dst, pack_bf16_octet(acc[0]), policy);
        ptx::stg_v4_policy(dst + 1, pack_bf16_octet(acc[1]), policy);
    }
    if (lane == 0) P.lse[row] = none ? __ldg(P.sink + h) : (M + log2f(den)) * kLn2;
}

// Splits per query so that about one CTA pair per two SMs is busy.
// `max_candidates` bounds the candidates of any query (selected + window).
int choose_splits(int rows, int64_t max_candidates) {
    const int blocks = (int)((max_candidates + kBlock - 1) / kBlock);
    int n = cached_sm_count() / 2 / (rows > 0 ? rows : 1);
    if (n > blocks) n = blocks;
    if (n > kMaxSplits) n = kMaxSplits;
    return n < 1 ? 1 : n;
}

}  // namespace

namespace {
// The partials of this many units: values, exponents, (max, sum).
size_t part_bytes(int units) { return (size_t)units * kHeads * (kDim * sizeof(__half) + 16 + sizeof(float2)); }

// Pairs launched for a tree's queries that are dealt out: as many times all pairs as the
// queries fill them, and once more where that leaves a choice; 0 where they are not dealt
// out. Dealing costs 3 us, half a block's time, and pairs that get no unit 1 us a round: six
// queries of 17 blocks, twelve parts each, take 22.2 us without and 24.7 with it. So it is
// done where equal parts have more than four blocks and, of more queries than half of the
// pairs, which would go unsplit, more than 24.
int dealt_units(int rows, int64_t max_candidates) {
    const int pairs = cached_sm_count() / 2, parts = choose_splits(rows, max_candidates);
    const int64_t blocks = (max_candidates + kBlock - 1) / kBlock;
    if (rows > kDealtRows || pairs < 1) return 0;
    if (2 * rows <= pairs) return blocks > 4 * parts ? pairs : 0;
    return blocks > 24 ? pairs * ((rows + pairs - 1) / pairs + 1) : 0;
}
size_t dealt_bytes(int rows, int units) { return (size_t)units * sizeof(int4) + (size_t)rows * sizeof(int2); }
}  // namespace

size_t attention_fp4_workspace_bytes(int B, int T, int max_selected, int W) {
    const int n = choose_splits(B * T, (int64_t)max_selected + W);
    return n == 1 ? 0 : part_bytes(B * T * n);
}

// `k` = the top-k row length (CSA) or the per-sequence capacity (HCA). The
// workspace holds the splits' partials, their exponents and their (max, sum).
namespace {
template <int FMT, Plan PLAN>
cudaError_t launch_pairs(const void *q, const float *sink, float scale, const csa_cache_desc &comp, const void *ring,
                         int R, int W, const csa_draft_tree &tree, const int32_t *topk_idx, const int32_t *topk_cnt,
                         const int32_t *n_comp, int m_hca, const int32_t *q_pos, int B, int T, int k, bool hca,
                         void *out, float *lse, const csa_attention_epilogue *epi, void *ws, size_t ws_bytes, int *err,
                         cudaStream_t stream) {
    Params P = {};
    P.draft = static_cast<const uint8_t *>(tree.records);
    P.parent = tree.parent;
    P.q = static_cast<const __nv_bfloat16 *>(q);
    P.sink = sink;
    P.scale_log2 = scale * kLog2e;
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
    P.wait_ns = wait_limit_ns();
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
    P.rows = B * T;
    P.n_split = choose_splits(P.rows, (int64_t)k + W);
    P.pairs = PLAN == kTreeDealt ? dealt_units(P.rows, (int64_t)k + W) : P.rows * P.n_split;
    P.round = cached_sm_count() / 2;
    if (P.n_split > 1 || PLAN == kTreeDealt) {
        if (!ws || ws_bytes < part_bytes(P.pairs) + (PLAN == kTreeDealt ? dealt_bytes(P.rows, P.pairs) : 0))
            return cudaErrorInvalidValue;
        const size_t parts = (size_t)P.pairs * kHeads;
        P.part_o = static_cast<__half *>(ws);
        P.part_ex = static_cast<uint8_t *>(ws) + parts * kDim * sizeof(__half);
        P.part_ml = reinterpret_cast<float2 *>(P.part_ex + parts * 16);
        if (PLAN == kTreeDealt) {
            P.dealt = reinterpret_cast<int4 *>(P.part_ml + parts);
            P.row_units = reinterpret_cast<int2 *>(P.dealt + P.pairs);
        }
    }
    constexpr size_t smem = sizeof(AttSmem<FMT>) + 1024;
    cudaError_t e = set_max_dynamic_smem_once(reinterpret_cast<const void *>(attention_fp4_kernel<FMT, PLAN>), (int)smem);
    if (e != cudaSuccess) return e;
    if (PLAN == kTreeDealt) {
        PdlLaunch d(dim3(1), dim3(32), stream);
        count_launch();
        e = P.rows <= 64 ? cudaLaunchKernelEx(&d.cfg, deal_units_kernel<2>, P)
                         : cudaLaunchKernelEx(&d.cfg, deal_units_kernel<(kDealtRows + 31) / 32>, P);
        if (e != cudaSuccess) return e;
    }
    PdlLaunch l(dim3(2 * P.pairs), dim3(kThreads), stream);
    l.cfg.dynamicSmemBytes = smem;
    count_launch();
    e = cudaLaunchKernelEx(&l.cfg, attention_fp4_kernel<FMT, PLAN>, P);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess || (P.n_split == 1 && PLAN != kTreeDealt)) return e;
    // Eight warps a head instead of one. For trees' queries up to three alone: one of 17
    // splits takes 17.2 us a call with eight and 19.4 with one, three 18.7 and 19.6, four 21.6
    // and 20.1, eight of nine splits 30.6 and 24.9.
    const bool spread = P.n_split > kCombineBatch && (PLAN == kNoTree || P.rows <= 3);
    PdlLaunch c(dim3(spread ? kHeads : kHeads / 8, P.rows), dim3(256), stream);
    count_launch();
    e = spread ? cudaLaunchKernelEx(&c.cfg, combine_fp4_kernel<8, PLAN>, P)
               : cudaLaunchKernelEx(&c.cfg, combine_fp4_kernel<1, PLAN>, P);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_attention_fp4(const void *q, const float *sink, float scale, const csa_cache_desc &comp,
                                 const void *ring, int R, int W, const int32_t *topk_idx, const int32_t *topk_cnt,
                                 const int32_t *n_comp, int m_hca, const int32_t *q_pos, int B, int T, int k, bool hca,
                                 void *out, float *lse, const csa_attention_epilogue *epi, void *ws, size_t ws_bytes,
                                 int *err, cudaStream_t stream) {
    return launch_pairs<CSA_FORMAT_FP4, kNoTree>(q, sink, scale, comp, ring, R, W, csa_draft_tree{}, topk_idx, topk_cnt,
                                               n_comp, m_hca, q_pos, B, T, k, hca, out, lse, epi, ws, ws_bytes, err,
                                               stream);
}

size_t tree_attention_workspace_bytes(int B, int N, int max_selected, int W) {
    const int units = dealt_units(B * N, (int64_t)max_selected + W);
    return units ? part_bytes(units) + dealt_bytes(B * N, units) : attention_fp4_workspace_bytes(B, N, max_selected, W);
}

// The tokens of a tree, over either record format.
cudaError_t launch_tree_attention(const void *q, const float *sink, float scale, const csa_cache_desc &comp,
                                  csa_format_t fmt, const void *ring, int R, int W, const csa_draft_tree &tree,
                                  const int32_t *topk_idx, const int32_t *topk_cnt, const int32_t *n_comp, int m_hca,
                                  const int32_t *q_pos, int B, int N, int k, bool hca, void *out, float *lse,
                                  const csa_attention_epilogue *epi, void *ws, size_t ws_bytes, int *err,
                                  cudaStream_t stream) {
    const bool dealt = dealt_units(B * N, (int64_t)k + W) > 0;
    const auto launch = fmt == CSA_FORMAT_FP4
                            ? (dealt ? launch_pairs<CSA_FORMAT_FP4, kTreeDealt> : launch_pairs<CSA_FORMAT_FP4, kTree>)
                            : (dealt ? launch_pairs<CSA_FORMAT_FP8, kTreeDealt> : launch_pairs<CSA_FORMAT_FP8, kTree>);
    return launch(q, sink, scale, comp, ring, R, W, tree, topk_idx, topk_cnt, n_comp, m_hca, q_pos, B, N, k, hca, out,
                  lse, epi, ws, ws_bytes, err, stream);
}

}  // namespace csa
