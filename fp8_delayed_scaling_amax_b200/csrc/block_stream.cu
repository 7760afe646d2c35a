// Block-scaled products of a few rows: the weight streams through once and the tensor cores take it as
// the M operand (128 weight rows per tile), the tokens as N (16 to 64 columns).  Serves
//   fp8_gemm_block / linear_forward_fp8_block with at most 64 rows, and
//   moe_forward_fp8_block: a mixture-of-experts layer for at most 64 tokens, in two launches (more than 16
//   tokens are quantized by one before).
//
//     product:  out[j][i] = RN_bf16( sum_b RN32(sw(i,b) sx(j,b)) (sum_{k in b} W[i][k] x[j][k]) + bias[i] )
//     experts:  for every (token t, slot s) with e = ids[t][s] in 0 .. experts - 1:
//                 g, u = rows of W13[e] . q(x[t]);  h = g / (1 + exp(-g)) * u  (fp32);  hq = q(h), 1 x 128 blocks
//                 out[t] = RN_bf16( sum_s weight[t][s] * (W2[e] . hq) )
//
// Bound by reading the weight from HBM (once per launch; an expert's once per 16 of its pairs, then from L2), for the
// smallest sizes by latency:
//  * a ring of stages, each a 128 x 128 weight tile (gate and up: two), a token tile, its scales and a TMEM
//    buffer: warp 0 streams the weights by TMA, warp 1 issues the MMAs, three to five warps build the
//    token tiles (FP8 rows come by TMA, the experts' hidden rows are copied, bf16 rows quantized on the
//    way: 1 x 128 blocks never leave a tile) and fetch the scales, four or eight add the blocks with their
//    scales in fp32 registers (a thread owns one weight row).  One commit per stage frees it for the producer
//    and hands it to the adders.  (With rings and commits of their own for weights, tokens and TMEM the issuer took
//    longer over a unit than the unit's bytes take from HBM.)
//  * two CTAs per SM for up to 16 columns: 100 to 190 KB per SM are in flight;
//  * the contraction is cut over a cluster of up to 8 CTAs; their fp32 sums meet in distributed shared
//    memory and are added in range order, so results do not depend on timing and no workspace is needed.
//  * experts: each CTA sorts the (token, slot) pairs by expert itself (a few hundred ids), so there is no
//    routing launch; only experts that are asked for are read.  The first launch forms h and quantizes
//    it; the second multiplies by W2 and adds a token's experts, all in one cluster per 128 outputs, in
//    expert order.  Launched with programmatic dependence, the second fills its ring with weights while the
//    first still runs, and waits only before it reads hq.
//  * every wait is bounded, as in the per-tensor GEMM.
//
// Measured (GB/s of 6551), weights from HBM: one row of FP8 tokens by 4096 x 1024 5.2 us (4.5 from L2), by 8192 x 8192
// 14.6 us (4600), 64 rows by 8192 x 2048 8.7 us, by 8192 x 8192 16.9; 8 bf16 rows by 1024 x 4096 7.2 us, by 8192 x 8192
// 18.5 us.  Experts: one token x 2 of 8 (1024, 4096) 15.3 us, 16 x 8 of 64 (2048, 1024) 70 us (5070), 61 x 4 of 16
// (4096, 1360) 76 us, 64 x 8 of 64 95 us.  The smallest are latency: 1 us from the launch to the first copy, 1.3 us to its
// arrival, 1.5 us from the last block to the output over the cluster.  Tried and dropped for the second launch, whose 16 tiles of 2048 outputs give
// 128 CTAs: clusters of 16 (7 fit at one CTA per SM, so 14 of the 16 needed at two); a whole SM's memory each (15
// clusters of 8 fit then: 73 -> 95 us); two clusters per tile whose sums meet in global memory (73 -> 74 us).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>
#include <string>

#include "internal.h"

namespace fp8dsa {
namespace {

constexpr int kBM = 128;       // weight rows per tile (TMEM lanes)
constexpr int kBK = 128;       // K per block
constexpr int kUmmaK = 32;
constexpr int kTileBytes = kBM * kBK;
constexpr int kFirstBuilder = 2;
constexpr int kMaxStages = 12;
constexpr int kBarBytes = 512;
constexpr int kMaxSplit = 8;

// kUp: the first expert launch on bf16 tokens, kUpFp8: on tokens quantized before, kDown: the second launch.
enum Mode : int { kDenseFp8 = 0, kDenseBf16 = 1, kUp = 2, kDown = 3, kUpFp8 = 4 };
constexpr bool is_up(int mode) { return mode == kUp || mode == kUpFp8; }

// Two CTAs per SM (96 registers per thread, 112 KB each) for up to 16 columns; the instance of 64 columns takes an SM
// alone (stages of 24 KB and 64 columns of TMEM).
constexpr int ctas_per_sm(int nmax) { return nmax == 16 ? 2 : 1; }
constexpr int smem_budget(int nmax) { return ctas_per_sm(nmax) == 2 ? 112 * 1024 : 224 * 1024; }
constexpr int tmem_cols(int nmax) { return 512 / ctas_per_sm(nmax); }
// A short product's ring is small: a launch takes this much shared memory all the same, so that no more CTAs share
// an SM than its TMEM serves.
constexpr int smem_least(int nmax) { return tmem_cols(nmax) <= 256 ? kTmemHalfSmem : kTmemWholeSmem; }
static_assert(smem_least(16) <= smem_budget(16) && smem_least(64) <= smem_budget(64), "shared memory");
constexpr int builders(int nmax) { return nmax == 16 ? 3 : 5; }
// Four adders, one per quarter of the weight rows; of 64 columns each of eight takes 32.  (64 rows of 8192 x
// 2048: 11.3 us with four, 10.6 with eight.)
constexpr int adders(int nmax) { return nmax == 16 ? 4 : 8; }
constexpr int threads_of(int nmax) { return 32 * (kFirstBuilder + builders(nmax) + adders(nmax)); }
// A builder waits for a stage's last use without having seen the uses between.  Units complete in order (one
// thread issues all MMAs, and a unit's builder arrives before it), so with at least as many stages as
// builders none of them can be a whole phase behind or ahead of a barrier.
constexpr int min_stages(int nmax) { return builders(nmax); }
constexpr int tiles_of(int mode) { return is_up(mode) ? 2 : 1; }
constexpr int stage_bytes(int mode, int nmax) { return tiles_of(mode) * kTileBytes + nmax * kBK; }
constexpr int max_stages(int mode, int nmax) {
    return tmem_cols(nmax) / (tiles_of(mode) * nmax) < kMaxStages ? tmem_cols(nmax) / (tiles_of(mode) * nmax) : kMaxStages;
}

struct StreamArgs {
    int splits;       // CTAs per cluster
    int stages;       // ring
    int k_blocks;     // blocks of the contraction
    int row_tiles;    // 128-row tiles of the weight
    uint32_t idesc;   // without N
    int fmt;          // of the tokens (quantizing modes)
    // product
    int ncols, rows;            // tokens, weight rows
    int64_t k;
    const void* x;              // FP8 bytes or bf16
    int64_t ldx, x_batch;       // elements
    int x_vec;                  // rows are 16-byte aligned
    int w_mn, w_batched, x_batched;
    BlockScales sw, sx;
    const uint16_t* bias;
    uint16_t* out;
    int64_t ldo, stride_o;
    int out_vec;                // four outputs of a row are 8-byte aligned
    // experts
    const int* ids;
    const float* weights;
    const float* w_scale;
    int tokens, pairs, experts, hidden, inter;
    uint32_t topk_inv;          // 2^16 / topk, rounded up
    const uint8_t* xq;          // [tokens][hidden] quantized before (more than 16 tokens)
    const float* sxq;           // [blocks of hidden][tokens]
    uint8_t* hq;                // [pairs][inter]
    float* sh;                  // [blocks of inter][pairs]
    int off_table, off_out;     // byte offsets in shared memory
    int off_recv;               // of the cluster's sums; 0: over the ring
    WaitCtl wait;
};

struct Entry {  // up to kRun pairs of one expert
    int expert, start, n;
};
// Runs of 16 with two CTAs per SM.  An expert with more pairs has its weights read again, mostly from L2, for
// every further run: 61 tokens x 4 over 16 experts took 94 us so, and 132 us in runs of 32 with an SM to itself.
constexpr int kRun = 16;
// as stored: 10, 11 and 4 bits
__device__ __forceinline__ uint32_t pack_entry(int expert, int start, int n) {
    return static_cast<uint32_t>(expert | (start << 10) | ((n - 1) << 21));
}
__device__ __forceinline__ Entry unpack_entry(uint32_t v) {
    return Entry{static_cast<int>(v & 1023u), static_cast<int>((v >> 10) & 2047u), static_cast<int>(v >> 21) + 1};
}
static_assert(FP8DSA_MOE_MAX_EXPERTS <= 1024 && FP8DSA_MOE_MAX_TOKENS * FP8DSA_MOE_MAX_TOPK <= 2048 && kRun <= 16, "entries");

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Pairs sorted by expert (stable), and the entries: runs of at most kRun pairs of one expert.
struct Table {
    int* total;         // entries
    uint16_t* sorted;   // [pairs] the pair at a sorted position
    uint32_t* entries;
    float* weight;      // [pairs] its weight (second launch)
};

__host__ __device__ constexpr int max_entries(int pairs, int experts) {
    return (pairs < experts ? pairs : experts) + pairs / kRun;
}
__host__ __device__ constexpr int table_bytes(int pairs, int experts, bool weights) {
    const int p8 = (pairs + 7) / 8 * 8;
    return 16 + p8 * 2 + (max_entries(pairs, experts) + 3) / 4 * 16 + (weights ? p8 * 4 : 0);
}

__device__ __forceinline__ Table table_at(uint8_t* base, const StreamArgs& g) {
    Table t;
    t.total = reinterpret_cast<int*>(base);
    t.sorted = reinterpret_cast<uint16_t*>(base + 16);
    t.entries = reinterpret_cast<uint32_t*>(t.sorted + (g.pairs + 7) / 8 * 8);
    t.weight = reinterpret_cast<float*>(t.entries + (max_entries(g.pairs, g.experts) + 3) / 4 * 4);
    return t;
}

// pair / topk: topk_inv is 2^16 / topk, rounded up, which is exact for up to 2048 pairs and 32 slots
__device__ __forceinline__ int token_of(const StreamArgs& g, int pair) {
    return static_cast<int>((static_cast<uint32_t>(pair) * g.topk_inv) >> 16);
}

// The pairs are dealt to the warps in runs; a thread's first one, loaded before the table is built (a load waits
// long while the first launch streams its weights).
struct FirstPair {
    int id;
    float weight;
};
__device__ __forceinline__ int pairs_per_warp(const StreamArgs& g, int warps) { return ((g.pairs + 31) / 32 + warps - 1) / warps * 32; }
template <bool kWeights, int kThreads>
__device__ __forceinline__ FirstPair load_first(const StreamArgs& g) {
    const int run = pairs_per_warp(g, kThreads / 32);
    const int p = static_cast<int>(threadIdx.x >> 5) * run + static_cast<int>(threadIdx.x & 31);
    FirstPair f{-1, 0.0f};
    if (p < g.pairs) {
        f.id = __ldg(g.ids + p);
        if (kWeights) f.weight = __ldg(g.weights + p);
    }
    return f;
}

// Whole CTA.  Deterministic: ranks follow the pairs' order.  `scratch` (build_scratch bytes) is the ring, which
// nothing fills yet.  Ends with a barrier.
constexpr int build_scratch(int threads) {
    return threads / 32 * FP8DSA_MOE_MAX_EXPERTS * 2 + FP8DSA_MOE_MAX_EXPERTS * 4 + 2 * FP8DSA_MOE_MAX_TOKENS * FP8DSA_MOE_MAX_TOPK * 2;
}
template <bool kWeights, int kThreads>
__device__ __forceinline__ void build_table(const Table& t, const StreamArgs& g, uint8_t* scratch, const FirstPair& first) {
    const int tid = threadIdx.x, lane = tid & 31;
    auto place = [&](int pos, int p, float w) {
        t.sorted[pos] = static_cast<uint16_t>(p);
        if (kWeights) t.weight[pos] = w;
    };
    if (g.pairs <= 32) {
        // one warp, in registers: a pair's position is the number of pairs with a smaller expert, found bit by bit, and
        // of those before it with the same one
        if (tid < 32) {
            const int e0 = first.id;
            const bool valid = e0 >= 0 && e0 < g.experts;
            uint32_t less = 0u, same = __ballot_sync(0xFFFFFFFFu, valid);
#pragma unroll 1
            for (int bit = 31 - __clz(g.experts - 1); bit >= 0; --bit) {
                const bool one = (e0 >> bit & 1) != 0;
                const uint32_t ones = __ballot_sync(0xFFFFFFFFu, one);
                if (one) less |= same & ~ones;
                same &= one ? ones : ~ones;
            }
            const int rank = __popc(same & ((1u << lane) - 1u)), pos = __popc(less) + rank;
            const bool leader = valid && rank % kRun == 0;  // the first pair of an entry
            const uint32_t leaders = __ballot_sync(0xFFFFFFFFu, leader);
            if (leader) t.entries[__popc(leaders & less) + rank / kRun] = pack_entry(e0, pos, min(kRun, __popc(same) - rank));
            if (valid) place(pos, lane, first.weight);
            if (lane == 0) *t.total = __popc(leaders);
        }
        __syncthreads();
        return;
    }
    // Every warp ranks a run of consecutive pairs within itself and counts them by expert in a row of its own;
    // then a thread per expert sums the rows, and one warp the experts.
    // (One warp ranking all pairs, and counting, for each pair, the pairs before it, took microseconds for a few
    // hundred of them.)
    constexpr int kWarps = kThreads / 32;
    const int warp = tid >> 5, run = pairs_per_warp(g, kWarps);
    const int rows = (g.pairs + run - 1) / run, e4 = (g.experts + 3) / 4 * 4;
    const int p_begin = warp * run, p_end = min(g.pairs, p_begin + run);
    int* start = reinterpret_cast<int*>(scratch);                         // [experts] pairs, then the first position
    uint16_t* counts = reinterpret_cast<uint16_t*>(start + e4);           // [warp][experts]
    uint16_t* ids = counts + kWarps * e4;                                 // [pairs] expert or 0xFFFF
    uint16_t* ranks = ids + FP8DSA_MOE_MAX_TOKENS * FP8DSA_MOE_MAX_TOPK;  // [pairs] position among its warp's
    uint16_t* mine = counts + warp * e4;
    for (int i = tid; i < rows * e4 / 2; i += kThreads) reinterpret_cast<uint32_t*>(counts)[i] = 0u;
    __syncthreads();
    int next = first.id;
    for (int p0 = p_begin; p0 < p_end; p0 += 32) {
        const int p = p0 + lane, v = next;
        uint32_t e = 0xFFFFu;
        if (p + 32 < p_end) next = __ldg(g.ids + p + 32);
        if (p < p_end) {
            if (v >= 0 && v < g.experts) e = static_cast<uint32_t>(v);
            ids[p] = static_cast<uint16_t>(e);
        }
        const uint32_t mask = __match_any_sync(0xFFFFFFFFu, e);
        const int before = __popc(mask & ((1u << lane) - 1u));
        int base = 0;
        if (e != 0xFFFFu) {
            base = mine[e];
            ranks[p] = static_cast<uint16_t>(base + before);
        }
        __syncwarp();
        if (e != 0xFFFFu && before == 0) mine[e] = static_cast<uint16_t>(base + __popc(mask));
        __syncwarp();
    }
    __syncthreads();
    for (int e = tid; e < g.experts; e += kThreads) {
        int before = 0;
        for (int r = 0; r < rows; ++r) {
            const int c = counts[r * e4 + e];
            counts[r * e4 + e] = static_cast<uint16_t>(before);
            before += c;
        }
        start[e] = before;
    }
    __syncthreads();
    if (tid < 32) {
        int pos = 0, ent = 0;
        for (int e0 = 0; e0 < g.experts; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < g.experts ? start[e] : 0;
            const int ne = (c + kRun - 1) / kRun;
            int both = c | (ne << 16);  // pairs and entries: 2048 each at most
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, both, o);
                if (lane >= o) both += v;
            }
            const int first = pos + (both & 0xFFFF) - c, ent0 = ent + (both >> 16) - ne;
            if (e < g.experts) start[e] = first;
            for (int q = 0; q < ne; ++q)
                t.entries[ent0 + q] = pack_entry(e, first + q * kRun, min(kRun, c - q * kRun));
            const int all = __shfl_sync(0xFFFFFFFFu, both, 31);
            pos += all & 0xFFFF;
            ent += all >> 16;
        }
        if (lane == 0) *t.total = ent;
    }
    __syncthreads();
    for (int p = p_begin + lane; p < p_end; p += 32) {
        const uint32_t e = ids[p];
        if (e != 0xFFFFu) place(start[e] + mine[e] + ranks[p], p, !kWeights ? 0.0f : p < p_begin + 32 ? first.weight : __ldg(g.weights + p));
    }
    fence_proxy_async_smem();  // the ring is TMA's from here on
    __syncthreads();
}

// One K block of 2 * kPairs bf16 rows, 16 lanes per row (lane l16 holds elements 8 l16 .. of rows 2 r + lane / 16,
// r = 0 .. kPairs - 1): quantized into the 128-byte-swizzled rows j0 .. of a token tile, with the scales.  The
// maxima's shuffles run side by side, and each lane forms one row's scale and reciprocal for all.
template <int kFmt, int kPairs>
__device__ __forceinline__ void quant_rows(uint8_t* tile, float* sc, int j0, int lane, const uint4* v) {
    const int l16 = lane & 15, half = lane >> 4;
    float am[kPairs], mine = 0.0f;
#pragma unroll
    for (int r = 0; r < kPairs; ++r) {
        const uint32_t m = max_abs_bf16x2(max_abs_bf16x2(0u, v[r].x), max_abs_bf16x2(v[r].y, max_abs_bf16x2(v[r].z, v[r].w)));
        am[r] = fmaxf(fabsf(__uint_as_float(m << 16)), fabsf(__uint_as_float(m & 0xFFFF0000u)));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < kPairs; ++r) am[r] = fmaxf(am[r], __shfl_xor_sync(0xFFFFFFFFu, am[r], o));
#pragma unroll
    for (int r = 0; r < kPairs; ++r)
        if (l16 == r) mine = am[r];
    const float s = block_step(mine, kFmt);
    const float inv_mine = __frcp_rn(s);
    if (l16 < kPairs) sc[j0 + 2 * l16 + half] = s;
#pragma unroll
    for (int r = 0; r < kPairs; ++r) {
        const float inv = __shfl_sync(0xFFFFFFFFu, inv_mine, (half << 4) | r);
        const uint32_t w[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            mul2_rn(f[2 * i], f[2 * i + 1], inv);
        }
        const int j = j0 + 2 * r + half;
        *reinterpret_cast<uint2*>(tile + j * 128 + (((l16 >> 1) ^ (j & 7)) << 4) + (l16 & 1) * 8) =
            make_uint2(cvt_fp8x4<kFmt>(f[0], f[1], f[2], f[3]), cvt_fp8x4<kFmt>(f[4], f[5], f[6], f[7]));
    }
}

// gate / (1 + exp(-gate)) * up in fp32
__device__ __forceinline__ float gated(float gate, float up) { return __fdiv_rn(gate, 1.0f + expf(-gate)) * up; }

// One warp: h of pair p in the 128 values of tile `tile`, from the ranges' sums (`ranges` parts `range_step`
// floats apart, the up sums `up_step` behind the gate sums, column `j`), its block scale and its bytes.
__device__ __forceinline__ void form_h(const StreamArgs& g, const float* recv, int ranges, int range_step, int up_step, int j,
                                       int p, int tile, int lane) {
    float v[2][4] = {};
    for (int s = 0; s < ranges; ++s) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const float4 a = *reinterpret_cast<const float4*>(recv + s * range_step + t * up_step + j * kBM + 4 * lane);
            v[t][0] += a.x;
            v[t][1] += a.y;
            v[t][2] += a.z;
            v[t][3] += a.w;
        }
    }
    const int i = tile * kBM + 4 * lane;  // inter is a multiple of 16: four rows are in or out
    float h[4], am = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        h[e] = i < g.inter ? gated(v[0][e], v[1][e]) : 0.0f;
        am = fmaxf(am, fabsf(h[e]));
    }
    am = warp_max(am);
    const float s = block_step(am, g.fmt);
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = __fmul_rn(h[e], inv);
    const uint32_t bytes = g.fmt == 0 ? cvt_fp8x4<0>(h[0], h[1], h[2], h[3]) : cvt_fp8x4<1>(h[0], h[1], h[2], h[3]);
    if (i < g.inter) *reinterpret_cast<uint32_t*>(g.hq + static_cast<int64_t>(p) * g.inter + i) = bytes;
    if (lane == 0) g.sh[static_cast<int64_t>(tile) * g.pairs + p] = s;
}

// Position in a CTA's sequence of units: K block `kb` of entry (experts) or tile `ent`.
struct Cursor {
    int ent, kb;
    __device__ __forceinline__ void advance(int step, int k_blocks) {
        kb += step;
        while (kb >= k_blocks) {
            kb -= k_blocks;
            ++ent;
        }
    }
};

// (first launch) the columns of an entry that one CTA of the cluster forms h of, at most
__host__ __device__ __forceinline__ int own_columns(const StreamArgs& g, int split_log) {
    return ((g.pairs < kRun ? g.pairs : kRun) + (1 << split_log) - 1) >> split_log;
}

// Column j of packed sums, by comparison (indexing would put them in memory).
template <int kPairs>
__device__ __forceinline__ float column(const uint64_t (&acc)[kPairs], int j) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        float lo, hi;
        unpack_f32x2(acc[k], lo, hi);
        if (2 * k == j) v = lo;
        if (2 * k + 1 == j) v = hi;
    }
    return v;
}
template <int kPairs>
__device__ __forceinline__ void set_column(uint64_t (&acc)[kPairs], int j, float v) {
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        float lo, hi;
        unpack_f32x2(acc[k], lo, hi);
        acc[k] = pack_f32x2(2 * k == j ? v : lo, 2 * k + 1 == j ? v : hi);
    }
}

// (the experts' modes have 16 columns and four adders)
template <int kMode, int NMAX>
__global__ void __launch_bounds__(threads_of(NMAX), ctas_per_sm(NMAX))
    block_stream_kernel(const __grid_constant__ CUtensorMap tma_w, const __grid_constant__ CUtensorMap tma_x,
                        const __grid_constant__ StreamArgs g) {
    constexpr int kBuilders = builders(NMAX), kFirstEpi = kFirstBuilder + kBuilders, kThreads = threads_of(NMAX);
    constexpr int kAdders = adders(NMAX), kOwn = 4 * NMAX / kAdders;  // kOwn: columns per adder
    constexpr bool kIsUp = is_up(kMode);
    constexpr bool kMoe = kIsUp || kMode == kDown;
    constexpr int kTiles = kIsUp ? 2 : 1;   // weight tiles per K block (gate and up)
    constexpr int kStage = stage_bytes(kMode, NMAX);
    constexpr int kCols = tmem_cols(NMAX);
    extern __shared__ __align__(1024) uint8_t smem[];
    // stage st: weight tiles [128][128] each, then the token tile [NMAX][128]; behind the ring (its length
    // is the launch's) the tokens' scales and the barriers
    uint8_t* tail = smem + g.stages * kStage;
    // The scales' ring is twice as long: a stage is built again once its MMAs are done, when those of the unit
    // before that have been read.
    float* xs = reinterpret_cast<float*>(tail);                // [2 stages][NMAX] the tokens' scales
    float* ws = xs + 2 * g.stages * NMAX;                      // [2 kMaxStages][2] the weight tiles' scales
    uint64_t* full = reinterpret_cast<uint64_t*>(ws + 4 * kMaxStages);  // weights landed and tokens written
    uint64_t* done = full + kMaxStages;                        // MMAs complete
    uint64_t* drain = done + kMaxStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((2 * kMaxStages + 1) * 8 + 8 + 4 * kMaxStages * 4 <= kBarBytes, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const int R = g.stages;
    if constexpr (!kIsUp) pdl_trigger();

    // The second expert launch reads only ids and weights before its wait: the first one has waited for
    // whatever wrote them before it let this launch start.
    FirstPair mine{-1, 0.0f};
    if constexpr (kMode == kDown) mine = load_first<true, kThreads>(g);
    if (warp == 0) {
        if (lane < R) {  // (a lane each: one after the other they are on every launch's path)
            mbar_init(full + lane, 2 + kAdders);  // the weights, the tokens, and the adders of the unit a ring ago
            mbar_init(done + lane, 2);  // the MMAs' commit, and the builder (whose scales the adders read)
            fence_mbar_init();
            mbar_arrive_many(full + lane, kAdders);  // nothing is there to be added at first
        }
        if (lane == 0) {
            mbar_init(drain, 1);
            *abort_flag = 0;
            fence_mbar_init();
            prefetch_tensormap(&tma_w);
        }
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kCols);
        tmem_relinquish();
    }
    float* outacc = reinterpret_cast<float*>(smem + g.off_out);  // second launch: [tokens][128]
    if constexpr (kMode == kDown)
        for (int i = threadIdx.x; i < g.tokens * kBM; i += kThreads) outacc[i] = 0.0f;
    if constexpr (kMode != kDown) pdl_wait();
    if constexpr (kIsUp) {
        pdl_trigger();
        mine = load_first<false, kThreads>(g);
    }
    Table table{};
    if constexpr (kMoe) {
        table = table_at(smem + g.off_table, g);
        build_table<kMode == kDown, kThreads>(table, g, smem, mine);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    // Where the sums of the cluster's CTAs come to lie: over the ring, once every CTA is through with its own, or apart,
    // where a peer only has to have started.
    const bool apart = g.off_recv != 0;
    const int split_log = 31 - __clz(g.splits);  // splits is 1, 2, 4 or 8
    if (apart) cluster_arrive();

    // This CTA's units.  A cluster takes one item (a 128-row tile of the product, of one entry's gate and up,
    // or of the second launch's outputs) and cuts its units over its CTAs; without clusters the first
    // expert launch's CTAs walk all items.
    const int cluster_id = static_cast<int>(blockIdx.x) / g.splits;
    const int clusters = static_cast<int>(gridDim.x) / g.splits;
    int items = 1, total = g.k_blocks;
    if constexpr (kIsUp) {
        const int all = *table.total * g.row_tiles;
        items = cluster_id < all ? (all - 1 - cluster_id) / clusters + 1 : 0;  // with clusters: one or none
    }
    if constexpr (kMode == kDown) total = *table.total * g.k_blocks;
    const int u0 = static_cast<int>((static_cast<int64_t>(rank) * total) / g.splits);
    const int u1 = static_cast<int>((static_cast<int64_t>(rank + 1) * total) / g.splits);
    const int per_item = u1 - u0;       // with items > 1 the CTA has whole items
    const int units = items * per_item;
    // first cursor, and what a cursor stands for
    auto first = [&](int skip) {
        Cursor c{0, 0};
        if constexpr (kMode == kDown) {
            c.ent = u0 / g.k_blocks;
            c.kb = u0 - c.ent * g.k_blocks;
        } else {
            c.kb = u0;
        }
        if (skip > 0) c.advance(skip, g.k_blocks);
        return c;
    };
    // (first launch) item of cursor entry i: expert-major, so that CTAs side by side read one expert
    auto item_of = [&](int ent) { return cluster_id + ent * clusters; };
    auto tile_of = [&](int ent) { return kIsUp ? item_of(ent) % g.row_tiles : cluster_id % g.row_tiles; };
    auto entry_at = [&](int ent) { return unpack_entry(table.entries[kIsUp ? item_of(ent) / g.row_tiles : ent]); };
    const int batch = kMoe ? 0 : cluster_id / g.row_tiles;

    if (warp == 0) {
        // ------------------------------------------------------------------ weights
        if (lane == 0) {
            int st = 0, ent = -1, row = 0, e = 0;
            uint32_t phase = 0, issued = 0, parity = 0;
            bool ok = true;
            Cursor c = first(0);
            for (int i = 0; i < units; ++i, c.advance(1, g.k_blocks)) {
                if (c.ent != ent) {
                    ent = c.ent;
                    row = tile_of(ent) * kBM;
                    e = kMoe ? entry_at(ent).expert : (g.w_batched ? batch : 0);
                }
                if (!mbar_wait_bounded(done + st, phase ^ 1u, g.wait, abort_flag, kStatusWaitProducer)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(full + st, kTiles * kTileBytes + (kMode == kDenseFp8 ? NMAX * kBK : 0));
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    const int r = row + t * g.inter;  // up rows follow the gate rows
                    tma_load_3d(smem + st * kStage + t * kTileBytes, &tma_w, full + st, g.w_mn ? r : c.kb * kBK,
                                g.w_mn ? c.kb * kBK : r, e);
                }
                if constexpr (kMode == kDenseFp8)  // FP8 rows come by TMA (rows from ncols on are zeros)
                    tma_load_3d(smem + st * kStage + kTiles * kTileBytes, &tma_x, full + st, c.kb * kBK, 0, g.x_batched ? batch : 0);
                issued |= 1u << st;
                parity = (parity & ~(1u << st)) | (phase << st);
                if (++st == R) {
                    st = 0;
                    phase ^= 1u;
                }
            }
            // Every copy in flight lands before the CTA can exit.  (A stage's barrier also counts its token
            // tile, which may never come: one wait that runs out has covered the other copies as well.)
            if (!ok)
                for (int s = 0; s < R; ++s)
                    if ((issued & (1u << s)) != 0 &&
                        !mbar_wait_bounded(full + s, (parity >> s) & 1u, g.wait, nullptr, kStatusWaitDrain))
                        break;
        }
        __syncwarp();
        if (!apart) cluster_arrive();
        cluster_wait();
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMA issuer
        if (elect_one()) {
            int st = 0, ent = -1;
            uint32_t phase = 0, idesc = g.idesc;
            bool ready = false;  // the unit's barrier, looked at before the last unit's MMAs were issued
            Cursor c = first(0);
            for (int i = 0; i < units; ++i, c.advance(1, g.k_blocks)) {
                if (c.ent != ent) {
                    ent = c.ent;
                    const int n = kMoe ? entry_at(ent).n : g.ncols;
                    idesc = g.idesc | (static_cast<uint32_t>((n + 15) / 16 * 2) << 17);  // N = n up to a multiple of 16
                }
                if (!ready && !mbar_wait_bounded(full + st, phase, g.wait, abort_flag, kStatusWaitMma)) break;
                tc_fence_after_sync();
                const uint32_t a_base = smem_addr(smem) + static_cast<uint32_t>(st * kStage);
                const uint32_t b_base = a_base + kTiles * kTileBytes;
                const uint32_t d = tmem_base + static_cast<uint32_t>(st * kTiles * NMAX);
                const int st_next = st + 1 == R ? 0 : st + 1;
                const uint32_t phase_next = st_next == 0 ? phase ^ 1u : phase;
                ready = i + 1 < units && mbar_test_wait(full + st_next, phase_next);
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
#pragma unroll
                    for (int kk = 0; kk < kBK / kUmmaK; ++kk) {
                        const uint32_t a = a_base + t * kTileBytes;
                        const uint64_t ad = g.w_mn ? smem_desc(a + kk * kUmmaK * 128, kTileBytes, 1024)
                                                   : smem_desc(a + kk * kUmmaK, 16, 1024);
                        umma_f8f6f4(d + t * NMAX, ad, smem_desc(b_base + kk * kUmmaK, 16, 1024), idesc, kk != 0 ? 1u : 0u);
                    }
                }
                umma_commit(done + st);
                st = st_next;
                phase = phase_next;
            }
            // every MMA this thread issued must complete before TMEM is released
            umma_commit(drain);
            mbar_wait_bounded(drain, 0, g.wait, nullptr, kStatusWaitDrain);
        }
        __syncwarp();
        if (!apart) cluster_arrive();
        cluster_wait();
    } else if (warp < kFirstEpi) {
        // ------------------------------------------------------------------ token tiles
        // The builders take the units in turn.  Columns from n on are left as they are: a column of the
        // product depends on its own token only.  A unit's first rows are loaded before its stage is waited for.
        if constexpr (kMode == kDown) pdl_wait();  // hq is the first launch's
        constexpr bool kQuant = kMode == kDenseBf16 || kMode == kUp;
        // quantizing: 16 lanes per row, 8 elements each; copying: 8 lanes per row, 16 bytes each (a product's
        // FP8 rows come by TMA: only their scales are copied)
        constexpr int kRowsAtOnce = kQuant ? 2 : 4;
        constexpr int kUnroll = kMode == kDenseFp8 ? 1 : NMAX / 4;
        static_assert(kQuant || kMode == kDenseFp8 || NMAX <= kRun, "a copied tile is one batch");
        constexpr int kBatch = kMode == kDenseFp8 ? NMAX : kRowsAtOnce * kUnroll;
        constexpr int kScales = kQuant ? 1 : (NMAX + 31) / 32;  // copying: scales per lane
        const int lrow = kQuant ? lane >> 4 : lane >> 3;        // row within kRowsAtOnce
        const int lcol = kQuant ? (lane & 15) * 8 : (lane & 7) * 16;
        const int64_t klen = kIsUp ? g.hidden : kMode == kDown ? g.inter : g.k;
        struct Batch {
            uint4 v[kUnroll];
        } cur;
        float sc_cur[kScales], sw_cur = 0.0f;
        auto columns = [&](int ent) { return kMoe ? entry_at(ent).n : g.ncols; };
        auto load = [&](Cursor c, int n, int j0, Batch& out, float (&scale)[kScales], float& w_scale) {
            if (j0 == 0 && lane < kTiles) {
                // the weight tile's scale (128 x 128 blocks), with the tokens': it may come from HBM, and the
                // adders, a block ahead at most, would wait for it
                if constexpr (kMoe)
                    w_scale = __ldg(g.w_scale + ((static_cast<int64_t>(entry_at(c.ent).expert) * kTiles + lane) * g.row_tiles +
                                                 tile_of(c.ent)) * g.k_blocks + c.kb);
                else if (g.sw.shift != 0)
                    w_scale = __ldg(g.sw.p + static_cast<int64_t>(tile_of(0)) * g.sw.s_mn + c.kb * g.sw.s_kb + batch * g.sw.s_b);
            }
            const int pos = kMoe ? entry_at(c.ent).start : 0;
            const int64_t col = static_cast<int64_t>(c.kb) * kBK + lcol;
#pragma unroll
            for (int r = 0; r < (kMode == kDenseFp8 ? 0 : kUnroll); ++r) {
                const int j = j0 + kRowsAtOnce * r + lrow;
                out.v[r] = make_uint4(0u, 0u, 0u, 0u);
                if (j >= n || col >= klen) continue;
                if constexpr (kQuant) {
                    const uint16_t* row = static_cast<const uint16_t*>(g.x) +
                                          (kMode == kUp ? token_of(g, table.sorted[pos + j]) * g.ldx : batch * g.x_batch + j * g.ldx);
                    if (g.x_vec) {  // k % 8 == 0: the eight elements are all inside
                        out.v[r] = __ldg(reinterpret_cast<const uint4*>(row + col));
                    } else {
                        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (col + e < klen) w[e >> 1] |= static_cast<uint32_t>(__ldg(row + col + e)) << (16 * (e & 1));
                        out.v[r] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {  // (hidden and inter are multiples of 16)
                    const uint8_t* row = kMode == kDown ? g.hq + static_cast<int64_t>(table.sorted[pos + j]) * g.inter
                                                        : g.xq + static_cast<int64_t>(token_of(g, table.sorted[pos + j])) * g.hidden;
                    out.v[r] = __ldcg(reinterpret_cast<const uint4*>(row + col));
                }
            }
            if (!kQuant && j0 == 0) {
#pragma unroll
                for (int q = 0; q < kScales; ++q) {
                    const int j = lane + 32 * q;
                    scale[q] = 0.0f;
                    if (j < n)
                        scale[q] = kMode == kDown
                                       ? __ldcg(g.sh + static_cast<int64_t>(c.kb) * g.pairs + table.sorted[pos + j])
                                   : kMode == kUpFp8
                                       ? __ldcg(g.sxq + static_cast<int64_t>(c.kb) * g.tokens + token_of(g, table.sorted[pos + j]))
                                       : __ldg(g.sx.p + static_cast<int64_t>(j >> g.sx.shift) * g.sx.s_mn + c.kb * g.sx.s_kb +
                                               batch * g.sx.s_b);
                }
            }
        };
        int i = warp - kFirstBuilder, st = i % R, slot = i % (2 * R), n = 0;
        uint32_t phase = static_cast<uint32_t>(i / R) & 1u;
        Cursor c = first(i);
        if (i < units) {
            n = columns(c.ent);
            load(c, n, 0, cur, sc_cur, sw_cur);
        }
        while (i < units) {
            Cursor cn = c;
            cn.advance(kBuilders, g.k_blocks);
            const bool more = i + kBuilders < units;
            const int nn = more ? (cn.ent == c.ent ? n : columns(cn.ent)) : 0;
            bool ok = mbar_wait_bounded(done + st, phase ^ 1u, g.wait, abort_flag, kStatusWaitProducer);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            uint8_t* dst = smem + st * kStage + kTiles * kTileBytes;
            float* sc = xs + slot * NMAX;
            if (lane < kTiles) ws[2 * slot + lane] = sw_cur;
            for (int j0 = 0; j0 < n; j0 += kBatch) {
                if (!kQuant && j0 == 0) {
#pragma unroll
                    for (int q = 0; q < kScales; ++q)
                        if (lane + 32 * q < n) sc[lane + 32 * q] = sc_cur[q];
                }
                if constexpr (kQuant) {
                    // one pair of rows, or the whole batch: the rows from n on are zeros and lie below NMAX
                    if (j0 + 2 >= n) {
                        if (g.fmt == 0)
                            quant_rows<0, 1>(dst, sc, j0, lane, cur.v);
                        else
                            quant_rows<1, 1>(dst, sc, j0, lane, cur.v);
                    } else if (g.fmt == 0) {
                        quant_rows<0, kUnroll>(dst, sc, j0, lane, cur.v);
                    } else {
                        quant_rows<1, kUnroll>(dst, sc, j0, lane, cur.v);
                    }
                } else if constexpr (kMode != kDenseFp8) {
#pragma unroll
                    for (int r = 0; r < kUnroll; ++r) {
                        const int j = j0 + kRowsAtOnce * r + lrow;
                        // 16-byte chunk c of row j sits at chunk c ^ (j % 8)
                        if (j < n) *reinterpret_cast<uint4*>(dst + j * 128 + (((lane & 7) ^ (j & 7)) << 4)) = cur.v[r];
                    }
                }
                // (loading these ahead as well took registers that spilled: 17.1 -> 18.5 us for one row of 8192 x 8192)
                if (j0 + kBatch < n) load(c, n, j0 + kBatch, cur, sc_cur, sw_cur);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(done + st);  // before `full`: the commit stays the last arrival of a phase
                mbar_arrive(full + st);
            }
            // only now: the proxy fence above waits for every load the thread has under way
            if (more) load(cn, nn, 0, cur, sc_cur, sw_cur);
            i += kBuilders;
            c = cn;
            n = nn;
            st += kBuilders;
            while (st >= R) {
                st -= R;
                phase ^= 1u;
            }
            slot += kBuilders;
            if (slot >= 2 * R) slot -= 2 * R;
        }
        __syncwarp();
        if (!apart) cluster_arrive();
        cluster_wait();
    } else {
        // ------------------------------------------------------------------ blocks added with their scales
        // Two sums at a time: two units of one weight tile each, or a unit's gate and up.  A round is mostly latency, so the
        // two barriers are looked at together and the scales are multiplied while TMEM is read (with a wait per unit, the
        // scales after the sums and scalar adds the experts' 16 tokens x 8 of 64 took 83 us instead of 73).  Loops over
        // columns outside the K loop are rolled: little code, little of it fetched.
        constexpr int kAtOnce = kTiles == 1 ? 2 : 1;
        const int q = warp & 3;
        const int row = q * 32 + lane;               // of the tile
        const int col0 = kOwn == NMAX ? 0 : (warp - kFirstEpi) / 4 * kOwn;
        const uint32_t tmem_mine = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(col0);
        uint64_t acc2[kTiles][kOwn / 2];             // pairs of columns
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int j = 0; j < kOwn / 2; ++j) acc2[t][j] = 0u;
        // a product whose weight has a scale per row: this thread's, loaded a round ahead
        const bool row_scales = !kMoe && g.sw.shift == 0;
        const float* sw_at = nullptr;
        float sw_row[2] = {0.0f, 0.0f};
        Cursor c = first(0);
        if (row_scales && units > 0) {
            const int grow = min(tile_of(0) * kBM + row, g.rows - 1);  // rows past the end are never stored
            sw_at = g.sw.p + static_cast<int64_t>(grow) * g.sw.s_mn + batch * g.sw.s_b + c.kb * g.sw.s_kb;
#pragma unroll
            for (int p = 0; p < 2; ++p)
                if (p < units) sw_row[p] = ldg_pinned(sw_at + p * g.sw.s_kb);
        }
        int st = 0, slot = 0, n = g.ncols;
        uint32_t phase = 0;
        bool ok = true;
        for (int i = 0; i < units;) {
            // the units of one entry (or this CTA's part of them)
            const int ent = c.ent, len = min(units - i, g.k_blocks - c.kb);
            Entry here{};
            if constexpr (kMoe) {
                here = entry_at(ent);
                n = here.n;
            }
            for (int r = 0; r < len; r += kAtOnce) {
                const bool two = kAtOnce == 2 && r + 1 < len;
                int st1 = st, slot1 = slot;
                uint32_t phase1 = phase;
                if (two) {
                    if (++st1 == R) {
                        st1 = 0;
                        phase1 ^= 1u;
                    }
                    if (++slot1 == 2 * R) slot1 = 0;
                }
                // (scales and sums come with `done`)  A warp that gave up runs on without waiting or adding, so that
                // the barrier at the end of an item still finds all of them.
                if (ok) {
                    const bool done0 = mbar_test_wait(done + st, phase), done1 = mbar_test_wait(done + st1, phase1);
                    if (!(done0 && done1))
                        ok = mbar_wait_bounded(done + st, phase, g.wait, abort_flag, kStatusWaitEpilogue) &&
                             mbar_wait_bounded(done + st1, phase1, g.wait, abort_flag, kStatusWaitEpilogue);
                }
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (ok) {
                    tc_fence_after_sync();
                    float sw0 = ws[2 * slot], sw1 = ws[kTiles == 2 ? 2 * slot + 1 : 2 * slot1];
                    if (row_scales) {
                        sw0 = sw_row[0];
                        sw1 = sw_row[1];
#pragma unroll
                        for (int p = 0; p < 2; ++p)
                            if (r + 2 + p < len) sw_row[p] = ldg_pinned(sw_at + (r + 2 + p) * g.sw.s_kb);
                    }
                    const uint64_t sw_pair[2] = {pack_f32x2(sw0, sw0), pack_f32x2(sw1, sw1)};
                    const uint32_t sum0 = tmem_mine + static_cast<uint32_t>(st * kTiles * NMAX);
                    const uint32_t sum1 = kTiles == 2 ? sum0 + NMAX : tmem_mine + static_cast<uint32_t>(st1 * NMAX);
                    const float* sc0 = xs + slot * NMAX + col0;  // columns from n on: never stored
                    const float* sc1 = kTiles == 2 ? sc0 : xs + slot1 * NMAX + col0;
#pragma unroll
                    for (int cc = 0; cc < kOwn; cc += 16) {
                        if (col0 + cc >= n) break;
                        uint32_t d0[16], d1[16];
                        tmem_load_16cols(sum0 + cc, d0);
                        tmem_load_16cols(sum1 + cc, d1);
                        uint64_t f0[8], f1[8];
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const float4 a = *reinterpret_cast<const float4*>(sc0 + cc + 2 * e);
                            const float4 b = *reinterpret_cast<const float4*>(sc1 + cc + 2 * e);
                            f0[e] = mul_f32x2(sw_pair[0], pack_f32x2(a.x, a.y));
                            f0[e + 1] = mul_f32x2(sw_pair[0], pack_f32x2(a.z, a.w));
                            f1[e] = mul_f32x2(sw_pair[1], pack_f32x2(b.x, b.y));
                            f1[e + 1] = mul_f32x2(sw_pair[1], pack_f32x2(b.z, b.w));
                        }
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e) fma_f32x2(acc2[0][cc / 2 + e], pack_b32x2(d0[2 * e], d0[2 * e + 1]), f0[e]);
                        if (two || kTiles == 2) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                fma_f32x2(acc2[kTiles - 1][cc / 2 + e], pack_b32x2(d1[2 * e], d1[2 * e + 1]), f1[e]);
                        }
                    }
                    // the stages' sums and scales are read
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(full + st);
                        if (two) mbar_arrive(full + st1);
                    }
                }
                st = st1 + 1;
                phase = phase1;
                if (st == R) {
                    st = 0;
                    phase ^= 1u;
                }
                slot = slot1 + 1 == 2 * R ? 0 : slot1 + 1;
            }
            i += len;
            ++c.ent;
            c.kb = 0;
            if constexpr (kMode == kDown) {
                // add the entry to its tokens' rows, which only this thread touches
#pragma unroll 1
                for (int j = 0; j < n; ++j) {
                    const float v = column(acc2[0], j);
                    const int at = here.start + j;
                    float* dst = outacc + token_of(g, table.sorted[at]) * kBM + row;
                    *dst = fmaf(table.weight[at], v, *dst);
                }
#pragma unroll
                for (int k = 0; k < kOwn / 2; ++k) acc2[0][k] = 0u;
            }
            if constexpr (kIsUp) {
                // Without a cluster the item is complete here: a thread has its row's gate and up sums, the
                // block's maximum goes over the four warps.
                if (g.splits == 1) {
                    float* most = reinterpret_cast<float*>(smem + g.off_out) + (ent & 1) * 4 * NMAX;  // [warp][column]
                    const int tile = tile_of(ent), at = tile * kBM + row;
                    // Rolled loops that pick a column's registers by comparison: this code runs once per item, and
                    // unrolled it would first have to be fetched from a memory system that is busy with weights.
#pragma unroll 1
                    for (int j = 0; j < n; ++j) {
                        const float h = at < g.inter ? gated(column(acc2[0], j), column(acc2[1], j)) : 0.0f;
                        set_column(acc2[0], j, h);
                        const float am = warp_max(fabsf(h));
                        if (lane == 0) most[q * NMAX + j] = am;
                    }
                    named_barrier(1, 32 * kAdders);
#pragma unroll 1
                    for (int j = 0; j < n; ++j) {
                        const float h = column(acc2[0], j);
                        const float am = fmaxf(fmaxf(most[j], most[NMAX + j]), fmaxf(most[2 * NMAX + j], most[3 * NMAX + j]));
                        const float s = block_step(am, g.fmt);
                        const float v = __fmul_rn(h, __frcp_rn(s));
                        const int p = table.sorted[here.start + j];
                        const uint32_t byte = g.fmt == 0 ? cvt_fp8x2<0>(v, 0.0f) : cvt_fp8x2<1>(v, 0.0f);
                        if (at < g.inter) g.hq[static_cast<int64_t>(p) * g.inter + at] = static_cast<uint8_t>(byte);
                        if (row == 0) g.sh[static_cast<int64_t>(tile) * g.pairs + p] = s;
                    }
#pragma unroll
                    for (int j = 0; j < kOwn / 2; ++j) acc2[0][j] = acc2[1][j] = 0u;
                }
            }
        }
        float acc[kTiles][kOwn];
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int j = 0; j < kOwn / 2; ++j) unpack_f32x2(acc2[t][j], acc[t][2 * j], acc[t][2 * j + 1]);
        // The sums go to the CTAs of the cluster that write them out: rows to row / (128 / splits), or a pair's h (which needs its whole block) to
        // column % splits.
        __syncwarp();
        if (!apart) cluster_arrive();
        cluster_wait();
        if (ok && units > 0 && !(kIsUp && g.splits == 1)) {
            const uint32_t recv = smem_addr(smem + g.off_recv);
            if constexpr (kIsUp) {  // [range][tile][own column][row]
                const int per = own_columns(g, split_log);
#pragma unroll
                for (int j = 0; j < NMAX; ++j) {
                    if (j >= n) break;
                    const int own = j & (g.splits - 1), at = (rank * kTiles * per + (j >> split_log)) * kBM + row;
#pragma unroll
                    for (int t = 0; t < kTiles; ++t)
                        st_cluster_f32(mapa_shared(recv + static_cast<uint32_t>(at + t * per * kBM) * 4, own), acc[t][j]);
                }
            } else if constexpr (kMode != kDown) {  // [range][column][own row]
                const int per = kBM >> split_log, own = row >> (7 - split_log);
                const uint32_t at = mapa_shared(recv + static_cast<uint32_t>(rank * g.ncols * per + (row & (per - 1))) * 4, own);
#pragma unroll
                for (int j = 0; j < kOwn; ++j) {
                    if (col0 + j >= g.ncols) break;
                    st_cluster_f32(at + static_cast<uint32_t>((col0 + j) * per) * 4, acc[0][j]);
                }
            }
        }
        if constexpr (kMode == kDown) {  // (zeros, too, from a CTA that had no unit)
            const int per = kBM >> split_log, own = row >> (7 - split_log);
            const uint32_t at = mapa_shared(smem_addr(smem + g.off_recv) +
                                            static_cast<uint32_t>(rank * g.tokens * per + (row & (per - 1))) * 4, own);
            for (int j = 0; j < g.tokens; ++j) st_cluster_f32(at + static_cast<uint32_t>(j * per) * 4, outacc[j * kBM + row]);
        }
    }

    // ---------------------------------------------------------------------- sums over the cluster
    __syncwarp();
    cluster_arrive();
    cluster_wait();  // every range's sums are here; nothing of this CTA's is read or written by a peer after it
    const float* recv = reinterpret_cast<const float*>(smem + g.off_recv);
    if constexpr (kIsUp) {
        if (items > 0 && g.splits > 1) {
            const Entry en = entry_at(0);
            const int per = own_columns(g, split_log);
            for (int jj = warp; jj * g.splits + rank < en.n; jj += kThreads / 32)
                form_h(g, recv, g.splits, kTiles * per * kBM, per * kBM, jj, table.sorted[en.start + jj * g.splits + rank],
                       tile_of(0), lane);
        }
    } else {
        // this CTA's rows of the tile for every column (product) or token (experts), four rows per item
        const int per = kBM >> split_log, quad_log = 5 - split_log;
        const int cols = kMode == kDown ? g.tokens : g.ncols;
        const int rows = kMode == kDown ? g.hidden : g.rows;
        for (int i = threadIdx.x; i < cols << quad_log; i += kThreads) {
            const int j = i >> quad_log, r = 4 * (i & ((1 << quad_log) - 1));
            const int row = tile_of(0) * kBM + rank * per + r;
            if (row >= rows) continue;
            float v[4] = {};
            for (int s = 0; s < g.splits; ++s) {
                const float4 a = *reinterpret_cast<const float4*>(recv + (s * cols + j) * per + r);
                v[0] += a.x;
                v[1] += a.y;
                v[2] += a.z;
                v[3] += a.w;
            }
            uint16_t* dst = g.out + batch * g.stride_o + static_cast<int64_t>(j) * g.ldo + row;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (kMode != kDown && g.bias != nullptr && row + e < rows) v[e] += bf16_bits_to_float(__ldg(g.bias + row + e));
            if (g.out_vec && row + 4 <= rows) {
                *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (row + e < rows) dst[e] = __bfloat16_as_ushort(__float2bfloat16_rn(v[e]));
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 1) tmem_dealloc(tmem_base, kCols);
}

template <int kMode, int NMAX>
cudaError_t kernel_setup() {
    static std::once_flag once[kMaxDevices];
    static cudaError_t errs[kMaxDevices];
    const int dev = current_device();
    std::call_once(once[dev], [dev] {
        errs[dev] = cudaFuncSetAttribute(block_stream_kernel<kMode, NMAX>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         smem_budget(NMAX));
    });
    return errs[dev];
}

// Shared memory: the ring, scales, barriers, then the table and `out_size` bytes (the second expert launch's
// outputs, the first one's block maxima); as many stages as the budget and TMEM hold.
template <int kMode, int NMAX>
constexpr int stages_for(int table_size, int out_size) {
    const int n = std::min(max_stages(kMode, NMAX),
                           (smem_budget(NMAX) - kBarBytes - table_size - out_size) / (stage_bytes(kMode, NMAX) + 2 * NMAX * 4));
    return n >= min_stages(NMAX) ? n : 0;
}

template <int kMode, int NMAX>
int launch_stream(const CUtensorMap& map_w, const CUtensorMap& map_x, StreamArgs& g, int table_size, int out_size,
                  int64_t units, int64_t grid, cudaStream_t stream) {
    // the sums' exchange lies over the ring
    static_assert(min_stages(NMAX) * stage_bytes(kMode, NMAX) >= tiles_of(kMode) * NMAX * kBM * 4, "exchange");
    static_assert(kMode >= kUp || stages_for<kMode, NMAX>(0, 0) > 0, "shared memory");
    static_assert(kMode < kUp || min_stages(NMAX) * stage_bytes(kMode, NMAX) >= build_scratch(threads_of(NMAX)), "table");
    static_assert(kMode != kDown || min_stages(NMAX) * stage_bytes(kMode, NMAX) >= FP8DSA_MOE_MAX_TOKENS * kBM * 4, "exchange");
    const cudaError_t se = kernel_setup<kMode, NMAX>();
    if (se != cudaSuccess) return fail(FP8DSA_ERR_CUDA, std::string("cudaFuncSetAttribute: ") + cudaGetErrorString(se));
    const int split_log = g.splits == 8 ? 3 : g.splits == 4 ? 2 : g.splits - 1;
    const int recv = (kMode == kDown ? g.tokens : is_up(kMode) ? tiles_of(kMode) * own_columns(g, split_log) * g.splits : g.ncols) * kBM * 4;
    // no more stages than a CTA has units; the sums' room apart, where that does not cost a stage (one token
    // 4.9 -> 4.5 us)
    g.stages = stages_for<kMode, NMAX>(table_size, out_size);
    g.stages = static_cast<int>(std::max<int64_t>(min_stages(NMAX), std::min<int64_t>(g.stages, units)));
    g.off_table = g.stages * (stage_bytes(kMode, NMAX) + 2 * NMAX * 4) + kBarBytes;
    g.off_out = g.off_table + table_size;
    size_t bytes = static_cast<size_t>(g.off_out + out_size);
    g.off_recv = 0;
    if (bytes + static_cast<size_t>(recv) <= static_cast<size_t>(smem_budget(NMAX))) {
        g.off_recv = static_cast<int>(bytes);
        bytes += static_cast<size_t>(recv);
    }
    bytes = std::max(bytes, static_cast<size_t>(smem_least(NMAX)));
    const int rc = wait_ctl(&g.wait);
    if (rc) return rc;
    const cudaError_t e = launch_ex(block_stream_kernel<kMode, NMAX>, dim3(static_cast<unsigned>(grid)), dim3(threads_of(NMAX)),
                                    bytes, stream, g.splits, map_w, map_x, g);
    if (e != cudaSuccess) return fail(FP8DSA_ERR_CUDA, std::string("block stream launch: ") + cudaGetErrorString(e));
    return FP8DSA_OK;
}

// K ranges per tile: clusters double while all CTAs are resident at once and every range keeps two blocks.
int split_for(int64_t tiles, int64_t k_blocks, int ctas) {
    int s = 1;
    while (s < kMaxSplit && 2 * s * tiles <= ctas * sm_count() && k_blocks >= 4 * s) s *= 2;
    return s;
}

}  // namespace

int block_stream_gemm(const BlockGemmDesc& d, bool x_is_bf16, cudaStream_t stream) {
    const int64_t row_tiles = (d.n + kBM - 1) / kBM;
    const int64_t tiles = row_tiles * d.batch;
    if (tiles > (int64_t(1) << 26)) return fail(FP8DSA_ERR_UNSUPPORTED, "too many output tiles");
    const bool b_bat = d.stride_b != 0 && d.batch > 1;
    const int64_t outer = d.b_mn ? d.k : d.n;
    CUtensorMap map;
    int rc = encode_tensor_map(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, d.b, d.b_mn ? d.n : d.k, outer, b_bat ? d.batch : 1,
                               d.ldb, b_bat ? d.stride_b : d.ldb * outer, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
    CUtensorMap map_x = map;
    const bool a_bat = d.stride_a != 0 && d.batch > 1;
    if (!x_is_bf16) {
        rc = encode_tensor_map(&map_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, d.a, d.k, d.m, a_bat ? d.batch : 1, d.lda,
                               a_bat ? d.stride_a : d.lda * d.m, 128, d.m <= 16 ? 16 : 64, CU_TENSOR_MAP_SWIZZLE_128B);
        if (rc) return rc;
    }
    StreamArgs g{};
    g.x_batched = a_bat;
    g.k_blocks = static_cast<int>((d.k + kBK - 1) / kBK);
    g.row_tiles = static_cast<int>(row_tiles);
    g.splits = split_for(tiles, g.k_blocks, ctas_per_sm(d.m <= 16 ? 16 : 64));
    g.idesc = (1u << 4) | (static_cast<uint32_t>(d.fmt_b) << 7) | (static_cast<uint32_t>(d.fmt_a) << 10) |
              (static_cast<uint32_t>(d.b_mn) << 15) | (static_cast<uint32_t>(kBM >> 4) << 24);
    g.fmt = d.fmt_a;
    g.ncols = static_cast<int>(d.m);
    g.rows = static_cast<int>(d.n);
    g.k = d.k;
    g.x = d.a;
    g.ldx = d.lda;
    g.x_batch = d.stride_a;
    g.x_vec = aligned16(d.a) && d.lda % 8 == 0 && d.stride_a % 8 == 0 && d.k % 8 == 0;
    g.w_mn = d.b_mn;
    g.w_batched = b_bat;
    g.sw = scales_of(d.sb);
    g.sx = scales_of(d.sa);
    g.bias = static_cast<const uint16_t*>(d.bias);
    g.out = static_cast<uint16_t*>(d.out);
    g.ldo = d.ldo;
    g.stride_o = d.stride_o;
    g.out_vec = (reinterpret_cast<uintptr_t>(d.out) & 7) == 0 && d.ldo % 4 == 0 && (d.batch == 1 || d.stride_o % 4 == 0);
    const int64_t grid = tiles * g.splits, units = (g.k_blocks + g.splits - 1) / g.splits;
    launch_begin(kKindGemm, stream);
    if (x_is_bf16)
        rc = launch_stream<kDenseBf16, 16>(map, map, g, 0, 0, units, grid, stream);
    else if (d.m <= 16)
        rc = launch_stream<kDenseFp8, 16>(map, map_x, g, 0, 0, units, grid, stream);
    else
        rc = launch_stream<kDenseFp8, 64>(map, map_x, g, 0, 0, units, grid, stream);
    if (rc) return rc;
    launch_end(kKindGemmSingle, stream, 2.0 * static_cast<double>(d.m) * d.n * d.k * d.batch);
    return check_launch("block stream kernel");
}

namespace {

constexpr int64_t kMaxTokens = FP8DSA_MOE_MAX_TOKENS, kMaxTopk = FP8DSA_MOE_MAX_TOPK, kMaxExperts = FP8DSA_MOE_MAX_EXPERTS;

struct MoeLayout {
    size_t hq, sh, xq, sxq, total;
};
MoeLayout moe_layout(int64_t tokens, int64_t topk, int64_t hidden, int64_t inter) {
    MoeLayout L;
    const size_t pairs = static_cast<size_t>(tokens) * topk;
    L.hq = 0;
    L.sh = align_up(pairs * static_cast<size_t>(inter), 256);
    L.xq = align_up(L.sh + pairs * static_cast<size_t>((inter + 127) / 128) * sizeof(float), 256);
    L.sxq = align_up(L.xq + static_cast<size_t>(tokens) * hidden, 256);
    L.total = align_up(L.sxq + static_cast<size_t>(tokens) * static_cast<size_t>((hidden + 127) / 128) * sizeof(float), 256);
    return L;
}

bool moe_sizes_ok(int64_t tokens, int64_t topk, int64_t experts, int64_t hidden, int64_t inter) {
    return tokens >= 0 && tokens <= kMaxTokens && topk >= 1 && topk <= kMaxTopk && experts >= 1 && experts <= kMaxExperts &&
           hidden >= 16 && inter >= 16 && hidden % 16 == 0 && inter % 16 == 0 && hidden <= (1 << 24) && inter <= (1 << 24);
}

// More tokens than this are quantized by a launch of their own: it costs one token 2.3 us, and sixteen nothing;
// without it 61 tokens x 4 over 16 experts take 92 us instead of 85.
constexpr int64_t kQuantizeBefore = 16;

constexpr int kMaximaBytes = 2 * 4 * kRun * 4;  // two items, four warps

// The largest tables fit beside the smallest ring.
constexpr int table_bytes_max(bool weights) {
    return table_bytes(FP8DSA_MOE_MAX_TOKENS * FP8DSA_MOE_MAX_TOPK, FP8DSA_MOE_MAX_EXPERTS, weights);
}
static_assert(stages_for<kUp, kRun>(table_bytes_max(false), kMaximaBytes) > 0, "shared memory");
static_assert(stages_for<kDown, kRun>(table_bytes_max(true), FP8DSA_MOE_MAX_TOKENS * kBM * 4) > 0, "shared memory");

int moe_launch(StreamArgs g, const uint8_t* w13, const float* w13_scale, const uint8_t* w2, const float* w2_scale,
               const void* x, void* out, cudaStream_t stream) {
    const int hb = (g.hidden + kBK - 1) / kBK, ib = (g.inter + kBK - 1) / kBK;
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    CUtensorMap m13, m2;
    int rc = encode_tensor_map(&m13, u8, w13, g.hidden, 2 * static_cast<int64_t>(g.inter), g.experts, g.hidden,
                               2 * static_cast<int64_t>(g.inter) * g.hidden, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
    rc = encode_tensor_map(&m2, u8, w2, g.inter, g.hidden, g.experts, g.inter, static_cast<int64_t>(g.hidden) * g.inter, 128,
                           128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
    const int entries = max_entries(g.pairs, g.experts);
    const int table = table_bytes(g.pairs, g.experts, false);
    const double row_flops = 2.0 * g.pairs * static_cast<double>(g.hidden) * g.inter;

    StreamArgs a = g;
    a.x = x;
    a.ldx = g.hidden;
    a.x_vec = aligned16(x);
    if (g.xq != nullptr) {  // the tokens are quantized once, not by every CTA that reads them
        BlockQuantJob j;
        j.x = x;
        j.rows = g.tokens;
        j.cols = g.hidden;
        j.fmt = static_cast<fp8_fmt_t>(g.fmt);
        j.out_row = const_cast<uint8_t*>(g.xq);
        j.scale_row = const_cast<float*>(g.sxq);
        rc = launch_block_quantize(j, stream);
        if (rc) return rc;
    }
    a.k_blocks = hb;
    a.row_tiles = ib;
    a.w_scale = w13_scale;
    // `entries` is the most there can be; without clusters as many CTAs as run at once walk what there is
    a.splits = split_for(static_cast<int64_t>(entries) * ib, hb, ctas_per_sm(kRun));
    int64_t grid = static_cast<int64_t>(entries) * ib * a.splits;
    if (a.splits == 1) grid = std::min<int64_t>(grid, static_cast<int64_t>(ctas_per_sm(kRun)) * sm_count());
    int64_t units = a.splits > 1 ? (hb + a.splits - 1) / a.splits : int64_t(entries) * ib * hb;  // of a CTA, at most
    launch_begin(kKindGemm, stream);
    rc = g.xq != nullptr ? launch_stream<kUpFp8, kRun>(m13, m13, a, table, kMaximaBytes, units, grid, stream)
                         : launch_stream<kUp, kRun>(m13, m13, a, table, kMaximaBytes, units, grid, stream);
    if (rc) return rc;
    launch_end(kKindGemmSingle, stream, 2.0 * row_flops);

    StreamArgs b = g;
    b.k_blocks = ib;
    b.row_tiles = hb;
    b.w_scale = w2_scale;
    b.out = static_cast<uint16_t*>(out);
    b.ldo = g.hidden;
    b.out_vec = (reinterpret_cast<uintptr_t>(out) & 7) == 0;
    b.splits = split_for(hb, static_cast<int64_t>(std::min(g.pairs, g.experts)) * ib, ctas_per_sm(kRun));
    launch_begin(kKindGemm, stream);
    units = (int64_t(entries) * ib + b.splits - 1) / b.splits;
    rc = launch_stream<kDown, kRun>(m2, m2, b, table_bytes(g.pairs, g.experts, true), g.tokens * kBM * 4, units,
                                  static_cast<int64_t>(hb) * b.splits, stream);
    if (rc) return rc;
    launch_end(kKindGemmSingle, stream, row_flops);
    return check_launch("block stream kernel");
}

}  // namespace
}  // namespace fp8dsa

using namespace fp8dsa;

extern "C" size_t moe_forward_fp8_block_workspace_size(int64_t tokens, int64_t topk, int64_t experts, int64_t hidden,
                                                       int64_t inter) {
    if (!moe_sizes_ok(tokens, topk, experts, hidden, inter)) return 0;
    return moe_layout(tokens, topk, hidden, inter).total;
}

extern "C" int moe_forward_fp8_block(const void* x, const int* ids, const float* weights, int64_t tokens, int64_t topk,
                                     int64_t experts, int64_t hidden, int64_t inter, fp8_fmt_t fmt, const uint8_t* w13,
                                     const float* w13_scale, const uint8_t* w2, const float* w2_scale, void* workspace,
                                     size_t workspace_bytes, void* out, cudaStream_t stream) {
    clear_error();
    if (!valid_fmt(fmt)) return fail(FP8DSA_ERR_INVALID_ARG, "fmt must be FP8_E4M3 or FP8_E5M2");
    if (tokens < 0 || topk < 1 || experts < 1 || hidden < 1 || inter < 1)
        return fail(FP8DSA_ERR_INVALID_ARG, "tokens must be >= 0, topk, experts, hidden and inter >= 1");
    if (!moe_sizes_ok(tokens, topk, experts, hidden, inter))
        return fail(FP8DSA_ERR_UNSUPPORTED,
                    "tokens <= 64, topk <= 32, experts <= 1024; hidden and inter multiples of 16 up to 2^24");
    if (w13 == nullptr || w13_scale == nullptr || w2 == nullptr || w2_scale == nullptr)
        return fail(FP8DSA_ERR_INVALID_ARG, "w13, w2 and their scales are required");
    if (!aligned16(w13) || !aligned16(w2)) return fail(FP8DSA_ERR_UNSUPPORTED, "w13 and w2 must be 16-byte aligned");
    if (((reinterpret_cast<uintptr_t>(w13_scale) | reinterpret_cast<uintptr_t>(w2_scale)) & 3) != 0)
        return fail(FP8DSA_ERR_UNSUPPORTED, "scales must be 4-byte aligned");
    if (tokens > 0) {
        if (x == nullptr || ids == nullptr || weights == nullptr || out == nullptr)
            return fail(FP8DSA_ERR_INVALID_ARG, "x, ids, weights and out are required");
        if (((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) & 1) != 0 ||
            ((reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(weights)) & 3) != 0)
            return fail(FP8DSA_ERR_UNSUPPORTED, "x, out, ids and weights must be aligned to their element sizes");
        if (workspace == nullptr) return fail(FP8DSA_ERR_INVALID_ARG, "workspace is required");
        if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
            return fail(FP8DSA_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
        if (workspace_bytes < moe_layout(tokens, topk, hidden, inter).total)
            return fail(FP8DSA_ERR_WORKSPACE, "workspace too small: see moe_forward_fp8_block_workspace_size");
    }
    int rc = check_device();
    if (rc) return rc;
    if (tokens == 0) return FP8DSA_OK;
    const MoeLayout L = moe_layout(tokens, topk, hidden, inter);
    StreamArgs g{};
    g.idesc = (1u << 4) | (static_cast<uint32_t>(fmt) << 7) | (static_cast<uint32_t>(fmt) << 10) |
              (static_cast<uint32_t>(kBM >> 4) << 24);
    g.fmt = fmt;
    g.ids = ids;
    g.weights = weights;
    g.tokens = static_cast<int>(tokens);
    g.topk_inv = static_cast<uint32_t>((65536 + topk - 1) / topk);
    g.pairs = static_cast<int>(tokens * topk);
    g.experts = static_cast<int>(experts);
    g.hidden = static_cast<int>(hidden);
    g.inter = static_cast<int>(inter);
    g.hq = static_cast<uint8_t*>(workspace) + L.hq;
    g.sh = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + L.sh);
    if (tokens > kQuantizeBefore) {
        g.xq = static_cast<uint8_t*>(workspace) + L.xq;
        g.sxq = reinterpret_cast<const float*>(static_cast<uint8_t*>(workspace) + L.sxq);
    }
    return moe_launch(g, w13, w13_scale, w2, w2_scale, x, out, stream);
}
