// Block-scaled products of a few rows: the weight streams through once and the tensor cores take it as
// the M operand (128 weight rows per tile), the tokens as N (16 to 64 columns).  Serves
//   fp8_gemm_block / linear_forward_fp8_block with at most 64 rows, and
//   moe_forward_fp8_block: a mixture-of-experts layer for at most 64 tokens, in two launches.
//
//     product:  out[j][i] = RN_bf16( sum_b RN32(sw(i,b) sx(j,b)) (sum_{k in b} W[i][k] x[j][k]) + bias[i] )
//     experts:  for every (token t, slot s) with e = ids[t][s] in 0 .. experts - 1:
//                 g, u = rows of W13[e] . q(x[t]);  h = g / (1 + exp(-g)) * u  (fp32);  hq = q(h), 1 x 128 blocks
//                 out[t] = RN_bf16( sum_s weight[t][s] * (W2[e] . hq) )
//
// Bound by reading the weight from HBM (every byte once per launch), for the smallest sizes by latency:
//  * warp 0 streams 128 x 128 weight tiles by TMA into a ring of 16 KB slots; 100 to 190 KB per SM are in
//    flight;
//  * warps 2-5 build the token tiles (one K block each in turn, so their latencies overlap): FP8 rows are
//    copied with their scales, bf16 rows are quantized on the way (1 x 128 blocks never leave a tile);
//  * warp 1 issues the MMAs, one TMEM buffer per K block; warps 6-9 add the blocks with their scales in
//    fp32 registers (a thread owns one weight row);
//  * the contraction is cut over a cluster of up to 8 CTAs; their fp32 sums meet in distributed shared
//    memory and are added in range order, so results do not depend on timing and no workspace is needed.
//  * experts: each CTA sorts the (token, slot) pairs by expert itself (a few hundred ids), so there is no
//    routing launch; only experts that are asked for are read.  The first launch forms h and quantizes
//    it; the second multiplies by W2 and adds a token's experts, all in one cluster per 128 outputs, in
//    expert order.  Launched with programmatic dependence, the second fills its ring with weights while the
//    first still runs, and waits only before it reads hq.
//  * every wait is bounded, as in the per-tensor GEMM.
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
constexpr int kSlotBytes = kBM * kBK;
constexpr int kBuilders = 4;
constexpr int kFirstBuilder = 2, kFirstEpi = 6;
constexpr int kThreads = 320;
constexpr int kTmemCols = 256;   // two CTAs share an SM's 512 columns
constexpr int kXSlots = 4;       // token tiles in flight
constexpr int kMaxWSlots = 12;
constexpr int kMaxBufs = 8;
constexpr int kScaleSlots = 12;  // >= kXSlots + kMaxBufs: a slot is reused only after its block was added
constexpr int kBarBytes = 512;
constexpr int kMaxSplit = 8;

enum Mode : int { kDenseFp8 = 0, kDenseBf16 = 1, kUp = 2, kDown = 3 };

// Two CTAs per SM (96 registers per thread, 112 KB each) where a thread's sums are few; the wide
// instances keep 64 sums per thread and take an SM alone.
constexpr int ctas_per_sm(int mode, int nmax) { return (mode == kUp ? 2 : 1) * nmax <= 32 ? 2 : 1; }
constexpr int smem_budget(int ctas) { return ctas == 2 ? 112 * 1024 : 224 * 1024; }

struct Scales {
    const float* p;
    int64_t s_mn, s_kb, s_b;
    int shift;
};

struct StreamArgs {
    int splits;       // CTAs per cluster
    int w_slots;      // weight ring
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
    int w_mn, w_batched;
    Scales sw, sx;
    const uint16_t* bias;
    uint16_t* out;
    int64_t ldo, stride_o;
    // experts
    const int* ids;
    const float* weights;
    const float* w_scale;
    int tokens, pairs, topk, experts, hidden, inter;
    uint8_t* hq;                // [pairs][inter]
    float* sh;                  // [blocks of inter][pairs]
    int off_table, off_out;     // byte offsets in shared memory
    WaitCtl wait;
};

struct Entry {  // up to NMAX pairs of one expert
    uint16_t expert, start, n, pad;
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Pairs sorted by expert (stable), and the entries: runs of at most nmax pairs of one expert.
struct Table {
    int* start;         // [experts] first sorted position (scratch before)
    uint16_t* id;       // [pairs] expert or 0xFFFF
    uint16_t* rank;     // [pairs] position among the expert's pairs
    uint16_t* sorted;   // [pairs]
    Entry* entries;
    int* total;
};

__host__ __device__ inline int max_entries(int pairs, int experts, int nmax) {
    return (pairs < experts ? pairs : experts) + pairs / nmax;
}
__host__ __device__ inline int table_bytes(int pairs, int experts, int nmax) {
    const int p8 = (pairs + 7) / 8 * 8;
    return 16 + ((experts + 3) / 4 * 4) * 4 + 3 * p8 * 2 + max_entries(pairs, experts, nmax) * 8;
}

__device__ __forceinline__ Table table_at(uint8_t* base, const StreamArgs& g, int nmax) {
    Table t;
    const int p8 = (g.pairs + 7) / 8 * 8;
    t.total = reinterpret_cast<int*>(base);
    t.start = reinterpret_cast<int*>(base + 16);
    t.id = reinterpret_cast<uint16_t*>(t.start + (g.experts + 3) / 4 * 4);
    t.rank = t.id + p8;
    t.sorted = t.rank + p8;
    t.entries = reinterpret_cast<Entry*>(t.sorted + p8);
    (void)nmax;
    return t;
}

// Whole CTA.  Deterministic: ranks follow the pairs' order.
__device__ __forceinline__ void build_table(const Table& t, const StreamArgs& g, int nmax) {
    const int tid = threadIdx.x, lane = tid & 31;
    for (int e = tid; e < g.experts; e += kThreads) t.start[e] = 0;
    for (int p = tid; p < g.pairs; p += kThreads) {
        const int e = __ldg(g.ids + p);
        t.id[p] = e >= 0 && e < g.experts ? static_cast<uint16_t>(e) : 0xFFFFu;
    }
    __syncthreads();
    if (tid < 32) {
        for (int p0 = 0; p0 < g.pairs; p0 += 32) {
            const int p = p0 + lane;
            const uint32_t e = p < g.pairs ? t.id[p] : 0xFFFFu;
            const uint32_t mask = __match_any_sync(0xFFFFFFFFu, e);
            const int before = __popc(mask & ((1u << lane) - 1u));
            int base = 0;
            if (e != 0xFFFFu) {
                base = t.start[e];
                t.rank[p] = static_cast<uint16_t>(base + before);
            }
            __syncwarp();
            if (e != 0xFFFFu && before == 0) t.start[e] = base + __popc(mask);
            __syncwarp();
        }
        int pos = 0, ent = 0;
        for (int e0 = 0; e0 < g.experts; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < g.experts ? t.start[e] : 0;
            const int ne = (c + nmax - 1) / nmax;
            int ci = c, ni = ne;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(0xFFFFFFFFu, ci, o), b = __shfl_up_sync(0xFFFFFFFFu, ni, o);
                if (lane >= o) {
                    ci += a;
                    ni += b;
                }
            }
            const int first = pos + ci - c, ent0 = ent + ni - ne;
            if (e < g.experts) t.start[e] = first;
            for (int q = 0; q < ne; ++q)
                t.entries[ent0 + q] = Entry{static_cast<uint16_t>(e), static_cast<uint16_t>(first + q * nmax),
                                            static_cast<uint16_t>(min(nmax, c - q * nmax)), 0};
            pos += __shfl_sync(0xFFFFFFFFu, ci, 31);
            ent += __shfl_sync(0xFFFFFFFFu, ni, 31);
        }
        if (lane == 0) *t.total = ent;
    }
    __syncthreads();
    for (int p = tid; p < g.pairs; p += kThreads) {
        const uint32_t e = t.id[p];
        if (e != 0xFFFFu) t.sorted[t.start[e] + t.rank[p]] = static_cast<uint16_t>(p);
    }
    __syncthreads();
}

// One K block of a bf16 row, 16 lanes per row (lane l16 holds elements 8 l16 ..): quantized into the
// 128-byte-swizzled row `j` of a token tile; returns the block's scale.
template <int kFmt>
__device__ __forceinline__ float quant_row(uint8_t* tile, int j, int l16, const uint32_t (&w)[4]) {
    uint32_t m = max_abs_bf16x2(max_abs_bf16x2(0u, w[0]), max_abs_bf16x2(w[1], max_abs_bf16x2(w[2], w[3])));
    float am = fmaxf(fabsf(__uint_as_float(m << 16)), fabsf(__uint_as_float(m & 0xFFFF0000u)));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
    const float s = fmaxf(__fdiv_rn(am, kFmt == 0 ? 448.0f : 57344.0f), 1e-12f);
    const float inv = __frcp_rn(s);
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        mul2_rn(f[2 * i], f[2 * i + 1], inv);
    }
    const uint2 q = make_uint2(cvt_fp8x4<kFmt>(f[0], f[1], f[2], f[3]), cvt_fp8x4<kFmt>(f[4], f[5], f[6], f[7]));
    *reinterpret_cast<uint2*>(tile + j * 128 + (((l16 >> 1) ^ (j & 7)) << 4) + (l16 & 1) * 8) = q;
    return s;
}

template <int kMode, int NMAX>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(kMode, NMAX))
    block_stream_kernel(const __grid_constant__ CUtensorMap tma_w, const __grid_constant__ StreamArgs g) {
    constexpr bool kMoe = kMode == kUp || kMode == kDown;
    constexpr int kTiles = kMode == kUp ? 2 : 1;   // weight tiles per K block (gate and up)
    constexpr int kBufCols = kTiles * NMAX;
    constexpr int kBufs = kTmemCols / kBufCols < kMaxBufs ? kTmemCols / kBufCols : kMaxBufs;
    static_assert(kXSlots + kBufs <= kScaleSlots, "scale ring");
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* sX = smem;                                        // [kXSlots][NMAX][128]
    uint8_t* sW = smem + kXSlots * NMAX * kBK;                 // [w_slots][128][128]
    // behind the weight ring (its size is the launch's)
    uint8_t* tail = sW + g.w_slots * kSlotBytes;
    float* xs = reinterpret_cast<float*>(tail);                // [kScaleSlots][NMAX]
    uint64_t* wfull = reinterpret_cast<uint64_t*>(tail + kScaleSlots * NMAX * 4);
    uint64_t* wempty = wfull + kMaxWSlots;
    uint64_t* sfull = wempty + kMaxWSlots;
    uint64_t* xempty = sfull + kScaleSlots;
    uint64_t* acc_full = xempty + kXSlots;
    uint64_t* acc_empty = acc_full + kMaxBufs;
    uint64_t* drain = acc_empty + kMaxBufs;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((2 * kMaxWSlots + kScaleSlots + kXSlots + 2 * kMaxBufs + 1) * 8 + 8 <= kBarBytes, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const int item = static_cast<int>(blockIdx.x) / g.splits;
    if constexpr (kMode != kUp) pdl_trigger();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxWSlots; ++i) {
            mbar_init(wfull + i, 1);
            mbar_init(wempty + i, 1);
        }
        for (int i = 0; i < kScaleSlots; ++i) mbar_init(sfull + i, 1);
        for (int i = 0; i < kXSlots; ++i) mbar_init(xempty + i, 1);
        for (int i = 0; i < kMaxBufs; ++i) {
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tma_w);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    float* outacc = reinterpret_cast<float*>(smem + g.off_out);  // down: [tokens][128]
    if constexpr (kMode == kDown)
        for (int i = threadIdx.x; i < g.tokens * kBM; i += kThreads) outacc[i] = 0.0f;
    // The second expert launch reads only ids and weights before its wait: the first one has waited for
    // whatever wrote them before it let this launch start.
    if constexpr (kMode != kDown) pdl_wait();
    if constexpr (kMode == kUp) pdl_trigger();
    Table table{};
    if constexpr (kMoe) {
        table = table_at(smem + g.off_table, g, NMAX);
        build_table(table, g, NMAX);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;

    // This CTA's work: units u0 .. u1 - 1, unit u = K block u % k_blocks of entry u / k_blocks.
    int batch = 0, tile = 0;
    int total = g.k_blocks;
    bool idle = false;
    if constexpr (kMode == kUp) {
        idle = item / g.row_tiles >= *table.total;  // fewer entries than the grid allows for
        batch = item / g.row_tiles;                 // the entry
        tile = item % g.row_tiles;
    } else if constexpr (kMode == kDown) {
        tile = item;
        total = *table.total * g.k_blocks;
    } else {
        batch = item / g.row_tiles;
        tile = item % g.row_tiles;
    }
    if (idle) total = 0;
    const int u0 = static_cast<int>((static_cast<int64_t>(rank) * total) / g.splits);
    const int u1 = static_cast<int>((static_cast<int64_t>(rank + 1) * total) / g.splits);
    // entry of unit u (experts)
    auto entry_of = [&](int u) { return table.entries[kMode == kUp ? batch : u / g.k_blocks]; };
    auto block_of = [&](int u) { return kMode == kDown ? u % g.k_blocks : u; };

    if (warp == 0) {
        // ------------------------------------------------------------------ weights
        if (lane == 0) {
            int slot = 0;
            uint32_t phase = 0, issued = 0, parity = 0;
            bool ok = true;
            for (int u = u0; u < u1 && ok; ++u) {
                const int kb = block_of(u);
                const int e = kMoe ? entry_of(u).expert : (g.w_batched ? batch : 0);
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    if (!mbar_wait_bounded(wempty + slot, phase ^ 1u, g.wait, abort_flag, kStatusWaitProducer)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(wfull + slot, kSlotBytes);
                    const int row = tile * kBM + t * g.inter;  // up rows follow the gate rows
                    tma_load_3d(sW + slot * kSlotBytes, &tma_w, wfull + slot, g.w_mn ? row : kb * kBK,
                                g.w_mn ? kb * kBK : row, e);
                    issued |= 1u << slot;
                    parity = (parity & ~(1u << slot)) | (phase << slot);
                    if (++slot == g.w_slots) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok)  // every copy in flight lands before the CTA can exit
                for (int s = 0; s < g.w_slots; ++s)
                    if (issued & (1u << s))
                        mbar_wait_bounded(wfull + s, (parity >> s) & 1u, g.wait, nullptr, kStatusWaitDrain);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            int slot = 0, xslot = 0, sslot = 0, buf = 0;
            uint32_t wphase = 0, sphase = 0, bphase = 0;
            for (int u = u0; u < u1; ++u) {
                const int n = kMoe ? static_cast<int>(entry_of(u).n) : g.ncols;
                const uint32_t idesc = g.idesc | (static_cast<uint32_t>((n + 15) / 16 * 2) << 17);  // N = n up to a multiple of 16
                if (!mbar_wait_bounded(acc_empty + buf, bphase ^ 1u, g.wait, abort_flag, kStatusWaitMma) ||
                    !mbar_wait_bounded(sfull + sslot, sphase, g.wait, abort_flag, kStatusWaitMma))
                    break;
                bool ok = true;
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    if (!mbar_wait_bounded(wfull + slot, wphase, g.wait, abort_flag, kStatusWaitMma)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t a_base = smem_addr(sW + slot * kSlotBytes);
                    const uint32_t b_base = smem_addr(sX + xslot * NMAX * kBK);
                    const uint32_t d = tmem_base + static_cast<uint32_t>(buf * kBufCols + t * NMAX);
#pragma unroll
                    for (int kk = 0; kk < kBK / kUmmaK; ++kk) {
                        const uint64_t ad = g.w_mn ? smem_desc(a_base + kk * kUmmaK * 128, kSlotBytes, 1024)
                                                   : smem_desc(a_base + kk * kUmmaK, 16, 1024);
                        umma_f8f6f4(d, ad, smem_desc(b_base + kk * kUmmaK, 16, 1024), idesc, kk != 0 ? 1u : 0u);
                    }
                    umma_commit(wempty + slot);
                    if (++slot == g.w_slots) {
                        slot = 0;
                        wphase ^= 1u;
                    }
                }
                if (!ok) break;
                umma_commit(xempty + xslot);
                umma_commit(acc_full + buf);
                if (++xslot == kXSlots) xslot = 0;
                if (++sslot == kScaleSlots) {
                    sslot = 0;
                    sphase ^= 1u;
                }
                if (++buf == kBufs) {
                    buf = 0;
                    bphase ^= 1u;
                }
            }
            // every MMA this thread issued must complete before TMEM is released
            umma_commit(drain);
            mbar_wait_bounded(drain, 0, g.wait, nullptr, kStatusWaitDrain);
        }
        __syncwarp();
    } else if (warp < kFirstEpi) {
        // ------------------------------------------------------------------ token tiles
        // Warp w builds blocks w - 2, w + 2, ...: four blocks' loads are under way at once.  Columns from n
        // on are left as they are: a column of the product depends on its own token only.
        if constexpr (kMode == kDown) pdl_wait();  // hq is the first launch's
        for (int i = warp - kFirstBuilder; u0 + i < u1; i += kBuilders) {
            const int u = u0 + i, kb = block_of(u);
            const int xslot = i % kXSlots, sslot = i % kScaleSlots;
            bool ok = mbar_wait_bounded(xempty + xslot, ((i / kXSlots) & 1) ^ 1u, g.wait, abort_flag, kStatusWaitProducer);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            uint8_t* dst = sX + xslot * NMAX * kBK;
            float* sc = xs + sslot * NMAX;
            int n = g.ncols;
            const uint16_t* pairs = nullptr;
            if constexpr (kMoe) {
                const Entry en = entry_of(u);
                n = en.n;
                pairs = table.sorted + en.start;
            }
            if constexpr (kMode == kDenseBf16 || kMode == kUp) {
                const int half = lane >> 4, l16 = lane & 15;
                const int64_t klen = kMode == kUp ? g.hidden : g.k;
                const int64_t col = static_cast<int64_t>(kb) * kBK + 8 * l16;
                constexpr int kUnroll = 4;  // row pairs whose loads are under way together
                for (int j0 = 0; j0 < n; j0 += 2 * kUnroll) {
                    uint32_t w[kUnroll][4];
#pragma unroll
                    for (int r = 0; r < kUnroll; ++r) {
                        const int j = j0 + 2 * r + half;
#pragma unroll
                        for (int v = 0; v < 4; ++v) w[r][v] = 0u;
                        if (j < n && col < klen) {
                            const uint16_t* row =
                                static_cast<const uint16_t*>(g.x) +
                                (kMode == kUp ? static_cast<int64_t>(pairs[j] / g.topk) * g.ldx : batch * g.x_batch + j * g.ldx);
                            if (g.x_vec) {  // k % 8 == 0: the eight elements are all inside
                                const uint4 a = __ldg(reinterpret_cast<const uint4*>(row + col));
                                w[r][0] = a.x;
                                w[r][1] = a.y;
                                w[r][2] = a.z;
                                w[r][3] = a.w;
                            } else {
#pragma unroll
                                for (int v = 0; v < 8; ++v)
                                    if (col + v < klen) w[r][v >> 1] |= static_cast<uint32_t>(__ldg(row + col + v)) << (16 * (v & 1));
                            }
                        }
                    }
#pragma unroll
                    for (int r = 0; r < kUnroll; ++r) {
                        if (j0 + 2 * r >= n) break;  // uniform: both halves run, the shuffles need all lanes
                        const int j = min(j0 + 2 * r + half, NMAX - 1);
                        const float s = g.fmt == 0 ? quant_row<0>(dst, j, l16, w[r]) : quant_row<1>(dst, j, l16, w[r]);
                        if (l16 == 0) sc[j] = s;
                    }
                }
            } else {
                // 16-byte chunk c of row j sits at chunk c ^ (j % 8)
                const int64_t klen = kMode == kDown ? g.inter : g.k;
                const int c = lane & 7;
                const int64_t col = static_cast<int64_t>(kb) * kBK + 16 * c;
                constexpr int kUnroll = NMAX / 4 < 8 ? NMAX / 4 : 8;
                for (int j0 = 0; j0 < n; j0 += 4 * kUnroll) {
                    uint4 v[kUnroll];
#pragma unroll
                    for (int r = 0; r < kUnroll; ++r) {
                        const int j = j0 + 4 * r + (lane >> 3);
                        v[r] = make_uint4(0u, 0u, 0u, 0u);
                        if (j < n && col < klen) {
                            const uint8_t* row = kMode == kDown ? g.hq + static_cast<int64_t>(pairs[j]) * g.inter
                                                                : static_cast<const uint8_t*>(g.x) + batch * g.x_batch + j * g.ldx;
                            if (col + 16 <= klen) {  // rows are 16-byte aligned
                                v[r] = kMode == kDown ? __ldcg(reinterpret_cast<const uint4*>(row + col))
                                                      : __ldg(reinterpret_cast<const uint4*>(row + col));
                            } else {
                                uint32_t b[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                                for (int e = 0; e < 15; ++e)
                                    if (col + e < klen) b[e >> 2] |= static_cast<uint32_t>(row[col + e]) << (8 * (e & 3));
                                v[r] = make_uint4(b[0], b[1], b[2], b[3]);
                            }
                        }
                    }
#pragma unroll
                    for (int r = 0; r < kUnroll; ++r) {
                        const int j = j0 + 4 * r + (lane >> 3);
                        if (j < n) *reinterpret_cast<uint4*>(dst + j * 128 + ((c ^ (j & 7)) << 4)) = v[r];
                    }
                }
                for (int j = lane; j < n; j += 32)
                    sc[j] = kMode == kDown ? __ldcg(g.sh + static_cast<int64_t>(kb) * g.pairs + pairs[j])
                                           : __ldg(g.sx.p + static_cast<int64_t>(j >> g.sx.shift) * g.sx.s_mn + kb * g.sx.s_kb +
                                                   batch * g.sx.s_b);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(sfull + sslot);
        }
    } else {
        // ------------------------------------------------------------------ blocks added with their scales
        const int q = warp & 3;
        const int row = q * 32 + lane;               // of the tile
        const int grow = tile * kBM + row;           // of the weight
        float acc[kTiles][NMAX];
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int j = 0; j < NMAX; ++j) acc[t][j] = 0.0f;
        // scale of unit u's weight tile t for this thread's row
        const int tiles_k = g.k_blocks;
        auto weight_scale = [&](int u, int t) -> float {
            const int kb = block_of(u);
            if constexpr (kMode == kUp)
                return ldg_pinned(g.w_scale + ((static_cast<int64_t>(entry_of(u).expert) * 2 + t) * g.row_tiles + tile) * tiles_k + kb);
            else if constexpr (kMode == kDown)
                return ldg_pinned(g.w_scale + (static_cast<int64_t>(entry_of(u).expert) * g.row_tiles + tile) * tiles_k + kb);
            else
                return grow < g.rows ? ldg_pinned(g.sw.p + static_cast<int64_t>(grow >> g.sw.shift) * g.sw.s_mn + kb * g.sw.s_kb +
                                                  batch * g.sw.s_b)
                                     : 0.0f;
        };
        float next[kTiles];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) next[t] = u0 < u1 ? weight_scale(u0, t) : 0.0f;
        int buf = 0, sslot = 0;
        uint32_t bphase = 0, sphase = 0;
        bool ok = true;
        for (int u = u0; u < u1; ++u) {
            float sw[kTiles];
#pragma unroll
            for (int t = 0; t < kTiles; ++t) sw[t] = next[t];
            if (u + 1 < u1) {
#pragma unroll
                for (int t = 0; t < kTiles; ++t) next[t] = weight_scale(u + 1, t);
            }
            const int n = kMoe ? static_cast<int>(entry_of(u).n) : g.ncols;
            ok = mbar_wait_bounded(sfull + sslot, sphase, g.wait, abort_flag, kStatusWaitEpilogue) &&
                 mbar_wait_bounded(acc_full + buf, bphase, g.wait, abort_flag, kStatusWaitEpilogue);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after_sync();
            const float* sc = xs + sslot * NMAX;
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(buf * kBufCols);
#pragma unroll
            for (int c = 0; c < NMAX; c += 16) {
                if (c < n) {
                    uint32_t d[kTiles][16];
#pragma unroll
                    for (int t = 0; t < kTiles; ++t) tmem_load_16cols(taddr + t * NMAX + c, d[t]);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(sc + c + e);  // columns from n on: never stored
#pragma unroll
                        for (int t = 0; t < kTiles; ++t) {
                            acc[t][c + e] = fmaf(__uint_as_float(d[t][e]), __fmul_rn(sw[t], f.x), acc[t][c + e]);
                            acc[t][c + e + 1] = fmaf(__uint_as_float(d[t][e + 1]), __fmul_rn(sw[t], f.y), acc[t][c + e + 1]);
                            acc[t][c + e + 2] = fmaf(__uint_as_float(d[t][e + 2]), __fmul_rn(sw[t], f.z), acc[t][c + e + 2]);
                            acc[t][c + e + 3] = fmaf(__uint_as_float(d[t][e + 3]), __fmul_rn(sw[t], f.w), acc[t][c + e + 3]);
                        }
                    }
                }
            }
            // the buffer and the scales are read
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty + buf);
            if (++buf == kBufs) {
                buf = 0;
                bphase ^= 1u;
            }
            if (++sslot == kScaleSlots) {
                sslot = 0;
                sphase ^= 1u;
            }
            if constexpr (kMode == kDown) {
                // the entry (or this CTA's part of it) is done: add it to its tokens' rows, which only
                // this thread touches
                if (u + 1 == u1 || block_of(u) + 1 == g.k_blocks) {
                    const Entry en = entry_of(u);
#pragma unroll
                    for (int j = 0; j < NMAX; ++j) {
                        if (j < en.n) {
                            const int p = table.sorted[en.start + j];
                            float* dst = outacc + (p / g.topk) * kBM + row;
                            *dst = fmaf(__ldg(g.weights + p), acc[0][j], *dst);
                        }
                        acc[0][j] = 0.0f;
                    }
                }
            }
        }
        if constexpr (kMode != kDown) {
            // [tile][column][row] over the rings: this CTA's MMAs and copies are all done
            float* red = reinterpret_cast<float*>(smem);
            const int n = kMoe ? (idle ? 0 : static_cast<int>(entry_of(u0).n)) : g.ncols;
            if (ok) {
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
#pragma unroll
                    for (int j = 0; j < NMAX; ++j)
                        if (j < n) red[(t * NMAX + j) * kBM + row] = acc[t][j];
            }
        }
    }

    // ---------------------------------------------------------------------- sums over the cluster
    __syncwarp();
    cluster_sync();
    if constexpr (kMode == kUp) {
        if (!idle) {
            // one warp per pair, all of its 128 values: h, its block scale and bytes
            const Entry en = table.entries[batch];
            for (int j = rank + g.splits * warp; j < en.n; j += g.splits * (kThreads / 32)) {
                float v[2][4] = {};
                for (int s = 0; s < g.splits; ++s) {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const float4 a = ld_cluster_f4(mapa_shared(
                            smem_addr(smem) + static_cast<uint32_t>(((t * NMAX + j) * kBM + 4 * lane) * 4), static_cast<uint32_t>(s)));
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
                    h[e] = i < g.inter ? __fdiv_rn(v[0][e], 1.0f + expf(-v[0][e])) * v[1][e] : 0.0f;
                    am = fmaxf(am, fabsf(h[e]));
                }
                am = warp_max(am);
                const float s = fmaxf(__fdiv_rn(am, g.fmt == 0 ? 448.0f : 57344.0f), 1e-12f);
                const float inv = __frcp_rn(s);
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = __fmul_rn(h[e], inv);
                const uint32_t bytes = g.fmt == 0 ? cvt_fp8x4<0>(h[0], h[1], h[2], h[3]) : cvt_fp8x4<1>(h[0], h[1], h[2], h[3]);
                const int p = table.sorted[en.start + j];
                if (i < g.inter) *reinterpret_cast<uint32_t*>(g.hq + static_cast<int64_t>(p) * g.inter + i) = bytes;
                if (lane == 0) g.sh[static_cast<int64_t>(tile) * g.pairs + p] = s;
            }
        }
    } else {
        // rows r0 .. r1 - 1 of the tile for every column (product) or token (experts)
        const int r0 = (rank * kBM) / g.splits, r1 = ((rank + 1) * kBM) / g.splits;
        const int cols = kMode == kDown ? g.tokens : g.ncols;
        const int rows = kMode == kDown ? g.hidden : g.rows;
        const uint32_t src = smem_addr(smem) + (kMode == kDown ? static_cast<uint32_t>(g.off_out) : 0u);
        for (int i = threadIdx.x; i < cols * (r1 - r0); i += kThreads) {
            const int j = i / (r1 - r0), r = r0 + i % (r1 - r0);
            const int row = tile * kBM + r;
            if (row >= rows) continue;
            float v = 0.0f;
            for (int s = 0; s < g.splits; ++s)
                v += ld_cluster_f32(mapa_shared(src + static_cast<uint32_t>((j * kBM + r) * 4), static_cast<uint32_t>(s)));
            if (kMode != kDown && g.bias != nullptr) v += bf16_bits_to_float(__ldg(g.bias + row));
            g.out[batch * g.stride_o + static_cast<int64_t>(j) * g.ldo + row] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
        }
    }
    cluster_sync();  // nobody's shared memory goes away while it is read

    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 1) tmem_dealloc(tmem_base, kTmemCols);
}

template <int kMode, int NMAX>
cudaError_t kernel_setup() {
    static std::once_flag once[kMaxDevices];
    static cudaError_t errs[kMaxDevices];
    const int dev = current_device();
    std::call_once(once[dev], [dev] {
        errs[dev] = cudaFuncSetAttribute(block_stream_kernel<kMode, NMAX>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         smem_budget(ctas_per_sm(kMode, NMAX)));
    });
    return errs[dev];
}

// Shared memory: token tiles, weight ring, scales, barriers, then `extra` bytes (the tables and, for the
// second expert launch, the outputs); as many weight slots as the budget holds.
template <int kMode, int NMAX>
int launch_stream(const CUtensorMap& map, StreamArgs& g, int extra_table, int extra_out, int64_t grid, cudaStream_t stream) {
    const cudaError_t se = kernel_setup<kMode, NMAX>();
    if (se != cudaSuccess) return fail(FP8DSA_ERR_CUDA, std::string("cudaFuncSetAttribute: ") + cudaGetErrorString(se));
    constexpr int kTiles = kMode == kUp ? 2 : 1;
    const int fixed = kXSlots * NMAX * kBK + kScaleSlots * NMAX * 4 + kBarBytes;
    const int extra = static_cast<int>(align_up(static_cast<size_t>(extra_table), 16)) + extra_out;
    const int slots = std::min(kMaxWSlots, (smem_budget(ctas_per_sm(kMode, NMAX)) - fixed - extra) / kSlotBytes);
    // the sums' exchange lies over the token tiles and the weight ring
    if (slots < kTiles || (kMode != kDown && kTiles * NMAX * kBM * 4 > kXSlots * NMAX * kBK + slots * kSlotBytes))
        return fail(FP8DSA_ERR_UNSUPPORTED, "shared memory: too many tokens, experts or slots");
    g.w_slots = slots;
    g.off_table = fixed + slots * kSlotBytes;
    g.off_out = g.off_table + static_cast<int>(align_up(static_cast<size_t>(extra_table), 16));
    const int rc = wait_ctl(&g.wait);
    if (rc) return rc;
    const cudaError_t e = launch_ex(block_stream_kernel<kMode, NMAX>, dim3(static_cast<unsigned>(grid)), dim3(kThreads),
                                    static_cast<size_t>(g.off_out + extra_out), stream, g.splits, map, g);
    if (e != cudaSuccess) return fail(FP8DSA_ERR_CUDA, std::string("block stream launch: ") + cudaGetErrorString(e));
    return FP8DSA_OK;
}

// K ranges per tile: clusters double while all CTAs are resident at once and every range keeps two blocks.
int split_for(int64_t tiles, int64_t k_blocks, int ctas) {
    int s = 1;
    while (s < kMaxSplit && 2 * s * tiles <= ctas * sm_count() && k_blocks >= 4 * s) s *= 2;
    return s;
}

Scales scales_of(const fp8_block_scale_t& s) {
    return Scales{s.scale, s.stride_mn, s.stride_kb, s.stride_batch, s.block_mn == 128 ? 7 : 0};
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
    StreamArgs g{};
    g.k_blocks = static_cast<int>((d.k + kBK - 1) / kBK);
    g.row_tiles = static_cast<int>(row_tiles);
    g.splits = split_for(tiles, g.k_blocks, ctas_per_sm(kDenseFp8, d.m <= 16 ? 16 : 64));
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
    const int64_t grid = tiles * g.splits;
    launch_begin(kKindGemm, stream);
    if (d.m <= 16)
        rc = x_is_bf16 ? launch_stream<kDenseBf16, 16>(map, g, 0, 0, grid, stream)
                       : launch_stream<kDenseFp8, 16>(map, g, 0, 0, grid, stream);
    else
        rc = x_is_bf16 ? launch_stream<kDenseBf16, 64>(map, g, 0, 0, grid, stream)
                       : launch_stream<kDenseFp8, 64>(map, g, 0, 0, grid, stream);
    if (rc) return rc;
    launch_end(kKindGemmSingle, stream, 2.0 * static_cast<double>(d.m) * d.n * d.k * d.batch);
    return check_launch("block stream kernel");
}

namespace {

constexpr int64_t kMaxTokens = FP8DSA_MOE_MAX_TOKENS, kMaxTopk = FP8DSA_MOE_MAX_TOPK, kMaxExperts = FP8DSA_MOE_MAX_EXPERTS;

struct MoeLayout {
    size_t hq, sh, total;
};
MoeLayout moe_layout(int64_t tokens, int64_t topk, int64_t inter) {
    MoeLayout L;
    const size_t pairs = static_cast<size_t>(tokens) * topk;
    L.hq = 0;
    L.sh = align_up(pairs * static_cast<size_t>(inter), 256);
    L.total = align_up(L.sh + pairs * static_cast<size_t>((inter + 127) / 128) * sizeof(float), 256);
    return L;
}

bool moe_sizes_ok(int64_t tokens, int64_t topk, int64_t experts, int64_t hidden, int64_t inter) {
    return tokens >= 0 && tokens <= kMaxTokens && topk >= 1 && topk <= kMaxTopk && experts >= 1 && experts <= kMaxExperts &&
           hidden >= 16 && inter >= 16 && hidden % 16 == 0 && inter % 16 == 0 && hidden <= (1 << 24) && inter <= (1 << 24);
}

template <int NMAX>
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
    const int entries = max_entries(g.pairs, g.experts, NMAX);
    const int table = table_bytes(g.pairs, g.experts, NMAX);
    const double row_flops = 2.0 * g.pairs * static_cast<double>(g.hidden) * g.inter;

    StreamArgs a = g;
    a.x = x;
    a.ldx = g.hidden;
    a.x_vec = aligned16(x);
    a.k_blocks = hb;
    a.row_tiles = ib;
    a.w_scale = w13_scale;
    a.splits = split_for(static_cast<int64_t>(entries) * ib, hb, ctas_per_sm(kUp, NMAX));
    launch_begin(kKindGemm, stream);
    rc = launch_stream<kUp, NMAX>(m13, a, table, 0, static_cast<int64_t>(entries) * ib * a.splits, stream);
    if (rc) return rc;
    launch_end(kKindGemmSingle, stream, 2.0 * row_flops);

    StreamArgs b = g;
    b.k_blocks = ib;
    b.row_tiles = hb;
    b.w_scale = w2_scale;
    b.out = static_cast<uint16_t*>(out);
    b.ldo = g.hidden;
    b.splits = split_for(hb, static_cast<int64_t>(std::min(g.pairs, g.experts)) * ib, ctas_per_sm(kDown, NMAX));
    launch_begin(kKindGemm, stream);
    rc = launch_stream<kDown, NMAX>(m2, b, table, g.tokens * kBM * 4, static_cast<int64_t>(hb) * b.splits, stream);
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
    return moe_layout(tokens, topk, inter).total;
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
        if (workspace_bytes < moe_layout(tokens, topk, inter).total)
            return fail(FP8DSA_ERR_WORKSPACE, "workspace too small: see moe_forward_fp8_block_workspace_size");
    }
    int rc = check_device();
    if (rc) return rc;
    if (tokens == 0) return FP8DSA_OK;
    const MoeLayout L = moe_layout(tokens, topk, inter);
    StreamArgs g{};
    g.idesc = (1u << 4) | (static_cast<uint32_t>(fmt) << 7) | (static_cast<uint32_t>(fmt) << 10) |
              (static_cast<uint32_t>(kBM >> 4) << 24);
    g.fmt = fmt;
    g.ids = ids;
    g.weights = weights;
    g.tokens = static_cast<int>(tokens);
    g.topk = static_cast<int>(topk);
    g.pairs = static_cast<int>(tokens * topk);
    g.experts = static_cast<int>(experts);
    g.hidden = static_cast<int>(hidden);
    g.inter = static_cast<int>(inter);
    g.hq = static_cast<uint8_t*>(workspace) + L.hq;
    g.sh = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + L.sh);
    // at most `tokens` pairs of an expert unless a token names it twice: runs of 16 where that is enough
    return tokens <= 16 ? moe_launch<16>(g, w13, w13_scale, w2, w2_scale, x, out, stream)
                        : moe_launch<32>(g, w13, w13_scale, w2, w2_scale, x, out, stream);
}
