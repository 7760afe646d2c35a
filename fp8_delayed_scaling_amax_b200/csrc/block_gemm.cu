// FP8 x FP8 -> bf16 matrix product of operands that carry one fp32 scale for each block of 128
// along the contraction, on the sm_100a tensor cores.
//
//     out[i][j] = RN_bf16( sum_b RN32(sa(i, b) * sb(j, b)) * (sum_{k in block b} A[i][k] * B[k][j]) + bias[j] )
//
// sa(i, b) is given per row of A or per 128 rows, sb(j, b) per column of the product or per 128.  A
// 128-deep sum of fp8 products is formed by four tcgen05.mma (kind::f8f6f4, K = 32 each) in TMEM;
// the scales differ from block to block, so every block's sum is then read back and added in fp32
// registers: acc = fma(d, sa * sb, acc).
//
// Structure (as the per-tensor GEMM, whose helpers it shares):
//  * warp 0 = TMA producer, warps 1 and 2 = MMA issuers, 8 warps promote and write the output;
//  * a stage holds one K block (128 bytes) of both operands; each K block goes to a TMEM buffer of its
//    own (accumulate = 0 for its first MMA), handed over with one commit; the promotion of block b
//    overlaps the MMAs of the blocks after it.  The tile's fp32 sums live in registers for the whole K
//    loop: 128 per thread for 256-wide tiles.
//  * 256 x 256 tiles on CTA pairs (M = 256 MMA across two SMs, each SM loads half of B), or
//    128 x 128 tiles on single CTAs, which may split K over a cluster of up to 8 CTAs, whose sums are
//    added through distributed shared memory in a fixed order (no workspace, no atomics).  A model
//    of the launch's time chooses (choose_plan).  (Splitting K over pairs measured no faster than either:
//    2048 x 1024 x 4096 20.4 us against 18.7 on 128 x 128 tiles; the exchange of 256 x 256 sums eats it.)
//  * a thread owns one row of the tile: its sa is one register per K block.  With sb per 128 columns
//    the product sa * sb is one more; with sb per column each promotion warp keeps its own columns'
//    scales of the current block in shared memory and reads them back as broadcasts.
//  * every wait is bounded, as in the per-tensor GEMM.
//
// Bound by the promotion: a 256 x 256 pair block takes 0.48 us with one scale per thread and 0.73 with a
// scale per column (a multiply more for each sum; the slopes of 2048 x 2048 over K = 4096 and 8192), its MMAs 0.26
// (512 cycles).  Measured: 8192^3 470 to 563 us by the inputs' power (2000 TFLOP/s; the tensor pipe is 55% busy at
// 4096^3, 67 to 70 us), 8192^3 with a scale per column on both sides 797 to 816 us.
// Tried there and slower: a TMEM load shape that gives a thread four rows and a quarter of the columns, with
// a quarter of the reads of the scales (4096^3 107 -> 110 us); the next block's first sums loaded before
// the last ones are added (spills 54 registers: 70 -> 107 us); barriers, buffers and an issuer for each half of
// the columns (70 -> 80 us); scalar adds (70 -> 77 us).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>
#include <string>

#include "internal.h"

namespace fp8dsa {
namespace {

constexpr int kBM = 128;    // rows of a CTA's tile (TMEM lanes)
constexpr int kBK = 128;    // K per stage: one scale block, one 128-byte swizzle row
constexpr int kUmmaK = 32;
constexpr int kIssuers = 2;  // MMA-issuing warps
constexpr int kEpiWarps = 8;
constexpr int kEpiThreads = 32 * kEpiWarps;

// Promotion of a 256-wide tile needs more than the 168 registers that eleven warps leave a thread
// (128 sums and 64 values in flight): its warps are two whole warpgroups that take over registers of
// the first one (warp 3 only fills that).  384 threads launch with 168 each, 64,512 in all;
// 128 x 56 + 256 x 224 = 64,512.  Spills are dear: with all but 28 KB of an SM's L1 used as
// shared memory, they go to L2 (8192^3 with 136 bytes of spills: 1357 against 1850 TFLOP/s).  ptxas reports none but for
// the 256-wide instance with a scale per column, which stores 24 bytes and loads 48 (gone without the bias's code,
// which a tile runs once; larger shares of the registers do not change them).
template <bool kRegSplit>
struct Roles {
    static constexpr int kFirstEpiWarp = kRegSplit ? 4 : 1 + kIssuers;
    static constexpr int kThreads = 32 * kFirstEpiWarp + kEpiThreads;
};
constexpr int kOtherRegs = 56, kEpiRegs = 224;
static_assert(128 * kOtherRegs + kEpiThreads * kEpiRegs <= Roles<true>::kThreads * 168, "registers a launch has");

constexpr int kChunk = 32;  // columns per TMEM load
constexpr int kOutBox = 64;                       // output columns per TMA store
constexpr int kOutStageBytes = 32 * kOutBox * 2;  // one warp's 32 rows x 64 columns
constexpr int kSmemLimit = 232448;
constexpr int kMaxStages = 8;
constexpr int kGroupM = 16;     // tile rows per group of the grouped raster
constexpr int kMaxSplit = 8;    // portable cluster size
constexpr int kRedPad = 4;      // floats between rows of the split-K exchange (bank spread)

template <int BN, bool kPair>
struct Cfg {
    static constexpr int kTileM = kPair ? 2 * kBM : kBM;
    static constexpr int kBRows = kPair ? BN / 2 : BN;
    static constexpr int kAStage = kBM * kBK;
    static constexpr int kBStage = kBRows * kBK;
    static constexpr int kAccBufs = 512 / BN;               // TMEM buffers of one K block each
    static constexpr int kEpiCols = BN / (kEpiWarps / 4);   // columns per promotion warp
    static constexpr int kBoxes = kEpiCols / kOutBox;       // output boxes per promotion warp
    static constexpr int kOutBytes = kEpiWarps * kBoxes * kOutStageBytes;
    static_assert(3 * kEpiCols * 4 <= kOutBytes / kEpiWarps, "per-column scales (double-buffered) and bias lie in the output boxes");
    static constexpr int kBarBytes = 512;
    static constexpr int kFixed = kOutBytes + kBarBytes;
    static constexpr int kStagesFit = (kSmemLimit - kFixed) / (kAStage + kBStage);
    static constexpr int kStages = kStagesFit < kMaxStages ? kStagesFit : kMaxStages;
    static constexpr int kSmem = kFixed + kStages * (kAStage + kBStage);
    static constexpr uint32_t kTxBytes = (kPair ? 2u : 1u) * (kAStage + kBStage);
    static_assert(kStages >= 4, "too few pipeline stages");
    static_assert(kBM * (BN + kRedPad) * 4 <= kStages * (kAStage + kBStage), "split-K exchange exceeds the stages");
    static_assert((2 * kStages + 2 * kAccBufs + 2) * 8 <= kBarBytes, "barrier area");
    static_assert(kSmem >= kTmemWholeSmem, "a CTA shares its SM's TMEM with no other");
};

struct BlockGemmArgs {
    int m, n, k_blocks;
    int tiles_m, tiles_n, num_tiles;
    int splits;  // K ranges per tile = cluster size (split instance)
    int a_batched, b_batched, a_mn, b_mn;
    uint32_t idesc;
    uint16_t* out;
    int64_t ldo, stride_o;
    int vec_out, tma_out;
    const uint16_t* bias;
    BlockScales sa, sb;
    WaitCtl wait;
};

__device__ __forceinline__ void decode_tile(int tile, const BlockGemmArgs& g, int& b, int& tm, int& tn) {
    const int per = g.tiles_m * g.tiles_n;
    b = tile / per;
    const int r = tile - b * per;
    const int group = kGroupM * g.tiles_n;
    const int gi = r / group;
    const int first_m = gi * kGroupM;
    const int gm = min(g.tiles_m - first_m, kGroupM);
    const int within = r - gi * group;
    tm = first_m + within % gm;
    tn = within / gm;
}

__device__ __forceinline__ void st_cluster_2xb64(uint32_t addr, uint64_t a, uint64_t b) {
    asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(addr), "l"(a), "l"(b) : "memory");
}

template <int BN, bool kPair, bool kColScale, bool kSplit>
__global__ void __launch_bounds__(Roles<kPair>::kThreads, 1)
    block_gemm_kernel(const __grid_constant__ CUtensorMap tma_a, const __grid_constant__ CUtensorMap tma_b,
                      const __grid_constant__ CUtensorMap tma_o, const __grid_constant__ BlockGemmArgs g) {
    using C = Cfg<BN, kPair>;
    constexpr bool kRegSplit = kPair;
    constexpr int kFirstEpiWarp = Roles<kRegSplit>::kFirstEpiWarp;
    constexpr int S = C::kStages;
    constexpr int kBufs = C::kAccBufs;
    static_assert(!(kPair && kSplit), "pairs do not split K");
    // 1024-byte aligned by declaration (the swizzle's period): every address below is a constant, which
    // the promotion warps' register budget needs
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* sA = smem;
    uint8_t* sB = smem + S * C::kAStage;
    uint8_t* sOut = sB + S * C::kBStage;
    uint64_t* full = reinterpret_cast<uint64_t*>(sOut + C::kOutBytes);
    uint64_t* empty = full + S;
    uint64_t* acc_full = empty + S;
    uint64_t* acc_empty = acc_full + kBufs;
    uint64_t* drain = acc_empty + kBufs;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    pdl_trigger();
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = kPair ? cluster_ctarank() : 0u;                     // half of the pair
    const int range = kSplit ? static_cast<int>(cluster_ctarank()) : 0;       // K range
    const bool leader = rank == 0;
    const int group = kPair ? 2 : (kSplit ? g.splits : 1);                    // CTAs that share a tile
    const int unit = static_cast<int>(blockIdx.x) / group;
    const int units = static_cast<int>(gridDim.x) / group;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int a = 0; a < kBufs; ++a) {
            mbar_init(acc_full + a, 1);
            mbar_init(acc_empty + a, kEpiWarps * (kPair ? 2 : 1));  // one arrival per promotion warp
        }
        mbar_init(drain, kIssuers);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tma_a);
        prefetch_tensormap(&tma_b);
        if (g.tma_out) prefetch_tensormap(&tma_o);
    }
    if (warp == 1) {
        if constexpr (kPair) {
            tmem_alloc_pair(tmem_slot, 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, 512);
            tmem_relinquish();
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (kPair) cluster_sync();  // the peer's loads target the leader's initialised barriers
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();

    // this CTA's K blocks: all of them, or its range of the split
    const int kb0 = kSplit ? static_cast<int>((static_cast<int64_t>(range) * g.k_blocks) / g.splits) : 0;
    const int kb1 = kSplit ? static_cast<int>((static_cast<int64_t>(range + 1) * g.k_blocks) / g.splits) : g.k_blocks;

    if (warp < kFirstEpiWarp) {
        if constexpr (kRegSplit) regs_release<kOtherRegs>();
        if (warp == 0) {
            // ------------------------------------------------------------------ TMA producer
            if (lane == 0) {
                int stage = 0;
                uint32_t phase = 0;
                uint32_t issued = 0, issued_parity = 0;
                bool ok = true;
                for (int t = unit; t < g.num_tiles && ok; t += units) {
                    int b, tm, tn;
                    decode_tile(t, g, b, tm, tn);
                    const int ba = g.a_batched ? b : 0;
                    const int bb = g.b_batched ? b : 0;
                    const int arow = tm * C::kTileM + (kPair ? static_cast<int>(rank) * kBM : 0);
                    const int brow = tn * BN + (kPair ? static_cast<int>(rank) * C::kBRows : 0);
                    for (int kb = kb0; kb < kb1; ++kb) {
                        if (!mbar_wait_bounded(empty + stage, phase ^ 1u, g.wait, abort_flag, kStatusWaitProducer)) {
                            ok = false;
                            break;
                        }
                        if (leader) mbar_arrive_expect_tx(full + stage, C::kTxBytes);
                        uint8_t* a_dst = sA + stage * C::kAStage;
                        uint8_t* b_dst = sB + stage * C::kBStage;
                        const int ac0 = g.a_mn ? arow : kb * kBK, ac1 = g.a_mn ? kb * kBK : arow;
                        const int bc0 = g.b_mn ? brow : kb * kBK, bc1 = g.b_mn ? kb * kBK : brow;
                        if constexpr (kPair) {
                            const uint32_t fb = mapa_shared(smem_addr(full + stage), 0);
                            tma_load_3d_pair(a_dst, &tma_a, fb, ac0, ac1, ba);
                            tma_load_3d_pair(b_dst, &tma_b, fb, bc0, bc1, bb);
                        } else {
                            tma_load_3d(a_dst, &tma_a, full + stage, ac0, ac1, ba);
                            tma_load_3d(b_dst, &tma_b, full + stage, bc0, bc1, bb);
                        }
                        issued |= 1u << stage;
                        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                        if (++stage == S) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
                if (!ok && leader) {
                    // every copy in flight lands before the CTAs can exit
                    for (int s = 0; s < S; ++s)
                        if (issued & (1u << s))
                            mbar_wait_bounded(full + s, (issued_parity >> s) & 1u, g.wait, nullptr, kStatusWaitDrain);
                }
            }
            __syncwarp();
        } else if (warp <= kIssuers) {
            // ------------------------------------------------------------------ MMA issuers (leader)
            // Two threads take the K blocks in turn, each with half of the TMEM buffers: one block's waits
            // and commits run beside the other's MMAs.
            if (leader && lane == 0) {
                const int first = warp - 1;
                const int64_t my_tiles = (g.num_tiles - 1 - unit) / units + 1;
                const int64_t blocks = unit < g.num_tiles ? my_tiles * (kb1 - kb0) : 0;
                int stage = first, buf = first;
                uint32_t phase = 0, buf_phase = 0;
                for (int64_t i = first; i < blocks; i += kIssuers) {
                    if (!mbar_wait_bounded(acc_empty + buf, buf_phase ^ 1u, g.wait, abort_flag, kStatusWaitMma) ||
                        !mbar_wait_bounded(full + stage, phase, g.wait, abort_flag, kStatusWaitMma))
                        break;
                    tc_fence_after_sync();
                    const uint32_t a_base = smem_addr(sA + stage * C::kAStage);
                    const uint32_t b_base = smem_addr(sB + stage * C::kBStage);
                    const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * BN);
#pragma unroll
                    for (int kk = 0; kk < kBK / kUmmaK; ++kk) {
                        // K-major: step 32 bytes along the swizzled row; MN-major: step 32 rows
                        const uint64_t ad = g.a_mn ? smem_desc(a_base + kk * kUmmaK * 128, C::kAStage, 1024)
                                                   : smem_desc(a_base + kk * kUmmaK, 16, 1024);
                        const uint64_t bd = g.b_mn ? smem_desc(b_base + kk * kUmmaK * 128, C::kBStage, 1024)
                                                   : smem_desc(b_base + kk * kUmmaK, 16, 1024);
                        if constexpr (kPair)
                            umma_f8f6f4_pair(d_tmem, ad, bd, g.idesc, kk != 0 ? 1u : 0u);
                        else
                            umma_f8f6f4(d_tmem, ad, bd, g.idesc, kk != 0 ? 1u : 0u);
                    }
                    if constexpr (kPair) {
                        umma_commit_pair_multicast(acc_full + buf, 0x3);
                        umma_commit_pair_multicast(empty + stage, 0x3);
                    } else {
                        umma_commit(acc_full + buf);
                        umma_commit(empty + stage);
                    }
                    stage += kIssuers;
                    if (stage >= S) {
                        stage -= S;
                        phase ^= 1u;
                    }
                    buf += kIssuers;
                    if (buf >= kBufs) {
                        buf -= kBufs;
                        buf_phase ^= 1u;
                    }
                }
                // every MMA the issuers sent off must complete before TMEM is released
                if constexpr (kPair)
                    umma_commit_pair(drain);
                else
                    umma_commit(drain);
                mbar_wait_bounded(drain, 0, g.wait, nullptr, kStatusWaitDrain);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------------ promotion and output
        if constexpr (kRegSplit) regs_take<kEpiRegs>();
        uint64_t acc[C::kEpiCols / 2];  // the tile's sums of this thread's row, two columns each
        // Warp w reads TMEM lanes 32 (w % 4) .. + 31, i.e. rows 32 (w % 4) + lane of the CTA's tile;
        // warps w and w + 4 split its columns.
        const int ew = warp - kFirstEpiWarp;
        const int q = warp & 3;
        const int cbase = (ew >> 2) * C::kEpiCols;
        const uint32_t tmem_mine = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(cbase);
        uint8_t* my_stage = sOut + ew * C::kBoxes * kOutStageBytes;
        float* my_scale = reinterpret_cast<float*>(my_stage);  // per-column scales share the output boxes
        const uint32_t acc_empty_leader = kPair ? mapa_shared(smem_addr(acc_empty), 0) : 0u;
        // a buffer is in registers: the MMAs of a later block may overwrite it
        auto hand_back = [&](int which) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if (kPair && !leader)
                    mbar_arrive_remote(acc_empty_leader + static_cast<uint32_t>(which * sizeof(uint64_t)));
                else
                    mbar_arrive(acc_empty + which);
            }
        };
        int buf = 0, flip = 0;
        uint32_t buf_phase = 0;
        bool ok = true;
        for (int t = unit; t < g.num_tiles && ok; t += units) {
            int b, tm, tn;
            decode_tile(t, g, b, tm, tn);
            const int row0 = tm * C::kTileM + (kPair ? static_cast<int>(rank) * kBM : 0) + q * 32;
            const int row = row0 + lane;
            const int col0 = tn * BN + cbase;
#pragma unroll
            for (int c = 0; c < C::kEpiCols / 2; ++c) acc[c] = 0u;
            // The next K block's scales are on their way a block ahead of their use (loads that stay where they are
            // written).  Scales outside the matrix are never read: their products are never stored.
            constexpr int kNb = kColScale ? C::kEpiCols / 32 : 1;  // kColScale: columns col0 + lane + 32 i
            const int sb_col = col0 + (kColScale ? lane : 0);
            const bool pa_in = row < g.m, sb_in = sb_col < g.n;
            const float* pa = g.sa.p + static_cast<int64_t>(row >> g.sa.shift) * g.sa.s_mn + b * g.sa.s_b + kb0 * g.sa.s_kb;
            const float* pb = g.sb.p + static_cast<int64_t>(sb_col >> g.sb.shift) * g.sb.s_mn + b * g.sb.s_b + kb0 * g.sb.s_kb;
            float sa_next = 0.0f, sb_next = 0.0f;
            auto fetch = [&]() {
                sa_next = pa_in ? ldg_pinned(pa) : 0.0f;
                if constexpr (kColScale) {
                    // straight into this warp's half of shared memory that the last block has been added from
                    const uint32_t dst = smem_addr(my_scale + flip * C::kEpiCols + lane);
#pragma unroll
                    for (int i = 0; i < kNb; ++i) {
                        const bool in = sb_col + 32 * i < g.n;
                        cp_async_f32(dst + 128 * i, in ? pb + i * 32 * g.sb.s_mn : g.sb.p, in);
                    }
                    cp_async_commit();
                } else {
                    sb_next = sb_in ? ldg_pinned(pb) : 0.0f;
                }
                pa += g.sa.s_kb;
                pb += g.sb.s_kb;
            };
            if constexpr (kColScale) {
                if (lane == 0) bulk_wait_group_read<0>();  // the last tile's stores have read the box
                __syncwarp();
            }
            if (kb0 < kb1) fetch();

            for (int kb = kb0; kb < kb1; ++kb) {
                const float sa = sa_next;
                uint64_t s2 = 0;  // RN32(sa * sb), twice
                const uint32_t cs_addr = smem_addr(my_scale + flip * C::kEpiCols);
                float4 f[2][2];  // kColScale: the scales of 8 columns
                flip ^= 1;
                if constexpr (kColScale) {
                    cp_async_wait_all();
                    __syncwarp();
#pragma unroll
                    for (int v = 0; v < 2; ++v) f[0][v] = lds_f32x4(cs_addr + 16 * v);
                } else {
                    const float s = __fmul_rn(sa, sb_next);
                    s2 = pack_f32x2(s, s);
                }
                if (kb + 1 < kb1) fetch();
                if (!mbar_wait_bounded(acc_full + buf, buf_phase, g.wait, abort_flag, kStatusWaitEpilogue)) {
                    ok = false;
                }
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t taddr = tmem_mine + static_cast<uint32_t>(buf * BN);
                if constexpr (kColScale) {
                    // 16 columns at a time; the next 16 columns' sums, and the next 8 columns' scales, are loaded while
                    // these are added
                    constexpr int kChunks = C::kEpiCols / 16;
                    uint32_t d[2][16];
                    tmem_load_16cols(taddr, d[0]);
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        tmem_wait_ld();
                        if (c + 1 < kChunks)
                            tmem_load_16cols(taddr + 16 * (c + 1), d[(c + 1) & 1]);
                        else
                            hand_back(buf);
                        const uint32_t(&dc)[16] = d[c & 1];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (c + 1 < kChunks || h == 0) {
#pragma unroll
                                for (int v = 0; v < 2; ++v) f[1 - h][v] = lds_f32x4(cs_addr + (16 * c + 8 * (h + 1) + 4 * v) * 4);
                            }
#pragma unroll
                            for (int v = 0; v < 2; ++v) {
                                // RN32(sa * sb), then one fma
                                float4 m = f[h][v];
                                mul2_rn(m.x, m.y, sa);
                                mul2_rn(m.z, m.w, sa);
                                const int e = 8 * h + 4 * v;
                                fma_f32x2(acc[8 * c + e / 2], pack_b32x2(dc[e], dc[e + 1]), pack_f32x2(m.x, m.y));
                                fma_f32x2(acc[8 * c + e / 2 + 1], pack_b32x2(dc[e + 2], dc[e + 3]), pack_f32x2(m.z, m.w));
                            }
                        }
                    }
                } else {
                    // two 32-column loads in flight; a chunk's registers are loaded again as soon as it is added
                    uint32_t d[2][kChunk];
                    auto add = [&](int c, const uint32_t(&dc)[kChunk]) {
#pragma unroll
                        for (int e = 0; e < kChunk; e += 2)
                            fma_f32x2(acc[(kChunk * c + e) / 2], pack_b32x2(dc[e], dc[e + 1]), s2);
                    };
                    constexpr int kChunks = C::kEpiCols / kChunk;
                    static_assert(kChunks % 2 == 0, "chunks in pairs");
                    tmem_load_32cols(taddr, d[0]);
                    tmem_load_32cols(taddr + kChunk, d[1]);
#pragma unroll
                    for (int c = 0; c < kChunks; c += 2) {
                        tmem_wait_ld();
                        const bool last = c + 2 == kChunks;
                        if (last) hand_back(buf);
                        add(c, d[0]);
                        if (!last) tmem_load_32cols(taddr + kChunk * (c + 2), d[0]);
                        add(c + 1, d[1]);
                        if (!last) tmem_load_32cols(taddr + kChunk * (c + 3), d[1]);
                    }
                }
                if (++buf == kBufs) {
                    buf = 0;
                    buf_phase ^= 1u;
                }
            }
            if (!ok) break;

            if constexpr (!kSplit) {
                // ---------------------------------------------------------- output of the whole tile
                // Compact code: it runs once per tile, and instruction fetches are most of its time (moving the
                // bias and the direct stores out of the unrolled loop took 2048 x 4096 x 1024 from 17.6 to
                // 15.0 us).
                if (lane == 0) bulk_wait_group_read<0>();  // the last tile's stores have read the boxes
                __syncwarp();
                if (g.bias != nullptr) {
                    float* bs = reinterpret_cast<float*>(my_stage) + 2 * C::kEpiCols;  // clear of the scales
#pragma unroll
                    for (int i = 0; i < C::kEpiCols / 32; ++i) {
                        const int col = col0 + lane + 32 * i;
                        bs[lane + 32 * i] = col < g.n ? bf16_bits_to_float(__ldg(g.bias + col)) : 0.0f;
                    }
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < C::kEpiCols; c += 4) {
                        const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(bs + c);
                        acc[c / 2] = add_f32x2(acc[c / 2], f.x);
                        acc[c / 2 + 1] = add_f32x2(acc[c / 2 + 1], f.y);
                    }
                    __syncwarp();
                }
#pragma unroll
                for (int c = 0; c < C::kEpiCols; c += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float lo, hi;
                        unpack_f32x2(acc[c / 2 + e], lo, hi);
                        w[e] = pack_bf16x2(lo, hi);
                    }
                    // 128-byte swizzle: 16-byte chunk j of row r sits at chunk j ^ (r % 8)
                    *reinterpret_cast<uint4*>(my_stage + (c / kOutBox) * kOutStageBytes + lane * 128 +
                                              (((c % kOutBox / 8) ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (g.tma_out) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && row0 < g.m) {
#pragma unroll
                        for (int i = 0; i < C::kBoxes; ++i)
                            if (col0 + i * kOutBox < g.n)
                                tma_store_3d(&tma_o, my_stage + i * kOutStageBytes, col0 + i * kOutBox, row0, b);
                        bulk_commit_group();
                    }
                } else {
                    // rows a tensor map cannot describe: each lane writes two columns of a row
                    __syncwarp();
                    for (int r = 0; r < 32 && row0 + r < g.m; ++r) {
                        uint16_t* orow = g.out + static_cast<int64_t>(b) * g.stride_o + static_cast<int64_t>(row0 + r) * g.ldo;
#pragma unroll
                        for (int i = 0; i < C::kBoxes; ++i) {
                            const int col = col0 + i * kOutBox + 2 * lane;
                            const uint32_t v = *reinterpret_cast<const uint32_t*>(
                                my_stage + i * kOutStageBytes + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
                            if (col < g.n) orow[col] = static_cast<uint16_t>(v);
                            if (col + 1 < g.n) orow[col + 1] = static_cast<uint16_t>(v >> 16);
                        }
                    }
                    __syncwarp();
                }
            }
        }
        if (lane == 0) bulk_wait_group_all();
        __syncwarp();
        if constexpr (kSplit) {
            // Once every range's MMAs and copies are done (the last block's commit covers a CTA's own), its sums
            // go to the range that writes their row: [range][row of its share][column] over the stages there,
            // rows kRedPad floats further apart than a power of two.
            cluster_sync();
            if (ok) {
                const int per = kBM / g.splits, r = q * 32 + lane;
                const uint32_t dst = mapa_shared(
                    smem_addr(smem) + static_cast<uint32_t>(((range * per + r % per) * (BN + kRedPad) + cbase) * 4),
                    static_cast<uint32_t>(r / per));
#pragma unroll
                for (int c = 0; c < C::kEpiCols; c += 4) st_cluster_2xb64(dst + c * 4, acc[c / 2], acc[c / 2 + 1]);
            }
            __syncwarp();
        }
    }

    if constexpr (kSplit) {
        if (warp < kFirstEpiWarp) cluster_sync();  // (the barrier above)
        cluster_sync();  // all sums have arrived, and nobody's shared memory is written after this
        if (warp >= kFirstEpiWarp) {
            int b, tm, tn;
            decode_tile(unit, g, b, tm, tn);
            const int et = static_cast<int>(threadIdx.x) - 32 * kFirstEpiWarp;
            const int per = kBM / g.splits;
            constexpr int kVec = BN / 8;  // eight columns per item
            for (int i = et; i < per * kVec; i += kEpiThreads) {
                const int rr = i / kVec, cc = (i % kVec) * 8;
                const int row = tm * kBM + range * per + rr, col = tn * BN + cc;
                if (row >= g.m || col >= g.n) continue;
                float v[8] = {};
                const float* src = reinterpret_cast<const float*>(smem) + rr * (BN + kRedPad) + cc;
                for (int s = 0; s < g.splits; ++s, src += per * (BN + kRedPad)) {  // in range order
                    const float4 x = *reinterpret_cast<const float4*>(src), y = *reinterpret_cast<const float4*>(src + 4);
                    v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
                    v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
                }
                uint16_t* dst = g.out + static_cast<int64_t>(b) * g.stride_o + static_cast<int64_t>(row) * g.ldo + col;
                if (g.bias != nullptr) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (col + e < g.n) v[e] += bf16_bits_to_float(__ldg(g.bias + col + e));
                }
                if (g.vec_out && col + 8 <= g.n) {
                    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                                pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (col + e < g.n) dst[e] = __bfloat16_as_ushort(__float2bfloat16_rn(v[e]));
                }
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if constexpr (kPair) cluster_sync();  // neither CTA releases TMEM or exits while the peer still uses it
    tc_fence_after_sync();
    if (warp == 1) {
        if constexpr (kPair)
            tmem_dealloc_pair(tmem_base, 512);
        else
            tmem_dealloc(tmem_base, 512);
    }
}

// k == 0: the product is empty; out = bias or 0.
__global__ void block_fill_kernel(uint16_t* out, int64_t m, int64_t n, int64_t ldo, int64_t stride_o, int64_t batch,
                                  const uint16_t* bias) {
    pdl_trigger();
    pdl_wait();
    const int64_t total = batch * m * n;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t j = i % n, r = (i / n) % m, b = i / (n * m);
        out[b * stride_o + r * ldo + j] = bias != nullptr ? bias[j] : 0;
    }
}

// Shared-memory limit of an instance, and how many groups of `group` CTAs (clusters) run at once.
template <int BN, bool kPair, bool kColScale, bool kSplit>
cudaError_t kernel_setup(int group, int* units_out) {
    using C = Cfg<BN, kPair>;
    static std::once_flag once[kMaxDevices];
    static cudaError_t errs[kMaxDevices];
    static int units[kMaxDevices][4];  // by log2(group)
    const int dev = current_device();
    std::call_once(once[dev], [dev] {
        auto kernel = block_gemm_kernel<BN, kPair, kColScale, kSplit>;
        errs[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (errs[dev] != cudaSuccess) return;
        for (int i = 0; i < 4; ++i) {
            units[dev][i] = sm_count() >> i;
            if (i == 0) continue;
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = 1u << i;
            at[0].val.clusterDim.y = 1;
            at[0].val.clusterDim.z = 1;
            cfg.gridDim = dim3(static_cast<unsigned>((sm_count() >> i) << i), 1, 1);
            cfg.blockDim = dim3(Roles<kPair>::kThreads, 1, 1);
            cfg.dynamicSmemBytes = C::kSmem;
            cfg.attrs = at;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0) units[dev][i] = n;
            cudaGetLastError();
        }
    });
    *units_out = units[dev][group == 1 ? 0 : group == 2 ? 1 : group == 4 ? 2 : 3];
    return errs[dev];
}

template <int BN, bool kPair, bool kColScale, bool kSplit>
int launch_cfg(const CUtensorMap (&maps)[3], const BlockGemmArgs& g, cudaStream_t stream) {
    using C = Cfg<BN, kPair>;
    const int group = kPair ? 2 : (kSplit ? g.splits : 1);
    int units = 0;
    cudaError_t e = kernel_setup<BN, kPair, kColScale, kSplit>(group, &units);
    if (e != cudaSuccess) return fail(FP8DSA_ERR_CUDA, std::string("cudaFuncSetAttribute: ") + cudaGetErrorString(e));
    // a split launch has one cluster per tile; the others walk the tiles
    const int64_t grid = static_cast<int64_t>(kSplit ? g.num_tiles : std::min(g.num_tiles, units)) * group;
    e = launch_ex(block_gemm_kernel<BN, kPair, kColScale, kSplit>, dim3(static_cast<unsigned>(grid)),
                  dim3(Roles<kPair>::kThreads),
                  C::kSmem, stream, group, maps[0], maps[1], maps[2], g);
    if (e != cudaSuccess) return fail(FP8DSA_ERR_CUDA, std::string("block gemm launch: ") + cudaGetErrorString(e));
    return FP8DSA_OK;
}

// Tile shape and K ranges of a launch: the modelled time of every choice, in us, fitted to B200 measurements of
// these kernels.  A K block costs 0.51 us on a pair's 256 x 256 tile (0.76 with per-column scales) and 0.50
// (0.58) on a 128 x 128 tile, whose shared memory fills at the same rate; a pair launch has 6.0 us around
// that (cluster launch, first load, last output), a single one 1.6; the exchange of split sums 2.0 and 0.4
// per range.  Both sides measured: 2048 x 4096 x 1024 15.8 us on pairs, 18.8 on single CTAs; 2048 x 1024 x
// 4096 22.8 and 18.7; 128 x 1024 x 8192 27.0 us unsplit, 18.6, 13.2 and 11.8 in 2, 4 and 8 ranges.
struct Plan {
    bool pair;
    int splits;
};

Plan choose_plan(const BlockGemmDesc& d, int64_t k_blocks, bool col) {
    auto tiles_of = [&](int64_t edge) { return ((d.m + edge - 1) / edge) * ((d.n + edge - 1) / edge) * d.batch; };
    auto walk_us = [&](int64_t tiles, int64_t units, double kb_us, double out_us) {
        return static_cast<double>((tiles + units - 1) / units) * (static_cast<double>(k_blocks) * kb_us + out_us);
    };
    Plan best{true, 1};
    double best_us = 6.0 + walk_us(tiles_of(256), sm_count() / 2, col ? 0.76 : 0.51, 0.7);
    const double kb_us = col ? 0.58 : 0.50;
    const int64_t tiles = tiles_of(128);
    for (int s = 1; s <= kMaxSplit; s *= 2) {
        if (s > 1 && (tiles * s > sm_count() || k_blocks < 2 * s)) break;
        const double us = s == 1 ? 1.6 + walk_us(tiles, sm_count(), kb_us, 0.6)
                                 : 1.6 + static_cast<double>((k_blocks + s - 1) / s) * kb_us + 2.0 + 0.4 * s;
        if (us < best_us) {
            best_us = us;
            best = Plan{false, s};
        }
    }
    return best;
}

}  // namespace

int block_gemm_launch(const BlockGemmDesc& d, cudaStream_t stream) {
    if (d.m == 0 || d.n == 0 || d.batch == 0) return FP8DSA_OK;
    if (d.k == 0) {
        const int64_t total = d.batch * d.m * d.n;
        const int blocks = static_cast<int>(std::min<int64_t>((total + 255) / 256, sm_count() * 8));
        launch_begin(kKindOther, stream);
        launch_ex(block_fill_kernel, dim3(blocks), dim3(256), 0, stream, 1, static_cast<uint16_t*>(d.out), d.m, d.n,
                  d.ldo, d.stride_o, d.batch, static_cast<const uint16_t*>(d.bias));
        launch_end(kKindOther, stream, static_cast<double>(total) * 2);
        return check_launch("block fill kernel");
    }
    if (d.m <= kStreamMaxRows && !d.a_mn) return block_stream_gemm(d, false, stream);
    const int64_t k_blocks = (d.k + kBK - 1) / kBK;
    const bool col = d.sb.block_mn == 1;
    const Plan plan = choose_plan(d, k_blocks, col);
    const bool pair = plan.pair;
    const int splits = plan.splits;
    const int bn = pair ? 256 : 128;
    const int64_t tiles = ((d.m + bn - 1) / bn) * ((d.n + bn - 1) / bn) * d.batch;
    if (tiles > (int64_t(1) << 28)) return fail(FP8DSA_ERR_UNSUPPORTED, "too many output tiles");

    const bool a_bat = d.stride_a != 0 && d.batch > 1;
    const bool b_bat = d.stride_b != 0 && d.batch > 1;
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    CUtensorMap maps[3];
    const int64_t a_outer = d.a_mn ? d.k : d.m, b_outer = d.b_mn ? d.k : d.n;
    int rc = encode_tensor_map(&maps[0], u8, d.a, d.a_mn ? d.m : d.k, a_outer, a_bat ? d.batch : 1, d.lda,
                               a_bat ? d.stride_a : d.lda * a_outer, 128, kBM, sw);
    if (rc) return rc;
    // pairs: each CTA's half of the columns, 128; single CTAs: all 128
    rc = encode_tensor_map(&maps[1], u8, d.b, d.b_mn ? d.n : d.k, b_outer, b_bat ? d.batch : 1, d.ldb,
                           b_bat ? d.stride_b : d.ldb * b_outer, 128, 128, sw);
    if (rc) return rc;
    const bool rows16 = aligned16(d.out) && d.ldo % 8 == 0 && (d.batch == 1 || d.stride_o % 8 == 0);
    if (rows16) {
        rc = encode_tensor_map(&maps[2], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d.out, d.n, d.m, d.batch, d.ldo * 2,
                               d.batch > 1 ? d.stride_o * 2 : d.ldo * 2 * d.m, kOutBox, 32, sw);
        if (rc) return rc;
    } else {
        maps[2] = maps[0];  // unused
    }

    BlockGemmArgs g{};
    g.m = static_cast<int>(d.m);
    g.n = static_cast<int>(d.n);
    g.k_blocks = static_cast<int>(k_blocks);
    g.tiles_m = static_cast<int>((d.m + bn - 1) / bn);
    g.tiles_n = static_cast<int>((d.n + bn - 1) / bn);
    g.num_tiles = static_cast<int>(tiles);
    g.splits = splits;
    g.a_batched = a_bat;
    g.b_batched = b_bat;
    g.a_mn = d.a_mn;
    g.b_mn = d.b_mn;
    g.idesc = (1u << 4) | (static_cast<uint32_t>(d.fmt_a) << 7) | (static_cast<uint32_t>(d.fmt_b) << 10) |
              (static_cast<uint32_t>(d.a_mn) << 15) | (static_cast<uint32_t>(d.b_mn) << 16) |
              (static_cast<uint32_t>(bn >> 3) << 17) | (static_cast<uint32_t>((pair ? 256 : 128) >> 4) << 24);
    g.out = static_cast<uint16_t*>(d.out);
    g.ldo = d.ldo;
    g.stride_o = d.stride_o;
    g.vec_out = rows16;
    g.tma_out = rows16 && splits == 1;
    g.bias = static_cast<const uint16_t*>(d.bias);
    g.sa = scales_of(d.sa);
    g.sb = scales_of(d.sb);
    rc = wait_ctl(&g.wait);
    if (rc) return rc;

    launch_begin(kKindGemm, stream);
    if (pair)
        rc = col ? launch_cfg<256, true, true, false>(maps, g, stream) : launch_cfg<256, true, false, false>(maps, g, stream);
    else if (splits > 1)
        rc = col ? launch_cfg<128, false, true, true>(maps, g, stream) : launch_cfg<128, false, false, true>(maps, g, stream);
    else
        rc = col ? launch_cfg<128, false, true, false>(maps, g, stream) : launch_cfg<128, false, false, false>(maps, g, stream);
    if (rc) return rc;
    launch_end(pair ? kKindGemmPair : kKindGemmSingle, stream, 2.0 * static_cast<double>(d.m) * d.n * d.k * d.batch);
    return check_launch("block gemm kernel");
}

}  // namespace fp8dsa

using namespace fp8dsa;

namespace {

int check_scale(const fp8_block_scale_t* s, const char* name) {
    const std::string n(name);
    if (s == nullptr || s->scale == nullptr) return fail(FP8DSA_ERR_INVALID_ARG, n + " is required");
    if (s->block_mn != 1 && s->block_mn != 128) return fail(FP8DSA_ERR_INVALID_ARG, n + ".block_mn must be 1 or 128");
    if (s->stride_mn < 0 || s->stride_kb < 0 || s->stride_batch < 0)
        return fail(FP8DSA_ERR_INVALID_ARG, n + " has a negative stride");
    if ((reinterpret_cast<uintptr_t>(s->scale) & 3) != 0) return fail(FP8DSA_ERR_UNSUPPORTED, n + " must be 4-byte aligned");
    return FP8DSA_OK;
}

}  // namespace

extern "C" int fp8_gemm_block(const uint8_t* a, const uint8_t* b, fp8_fmt_t fmt_a, fp8_fmt_t fmt_b, fp8_layout_t layout,
                              int64_t m, int64_t n, int64_t k, int64_t lda, int64_t ldb, int64_t ldo, int64_t batch,
                              int64_t stride_a, int64_t stride_b, int64_t stride_o, const fp8_block_scale_t* scale_a,
                              const fp8_block_scale_t* scale_b, const void* bias, void* out, cudaStream_t stream) {
    clear_error();
    if (!valid_fmt(fmt_a) || !valid_fmt(fmt_b)) return fail(FP8DSA_ERR_INVALID_ARG, "fmt must be FP8_E4M3 or FP8_E5M2");
    if (layout < FP8_LAYOUT_NT || layout > FP8_LAYOUT_TT) return fail(FP8DSA_ERR_INVALID_ARG, "bad layout");
    if (m < 0 || n < 0 || k < 0 || batch < 0) return fail(FP8DSA_ERR_INVALID_ARG, "negative size");
    if (m > 0x7FFFFF00 || n > 0x7FFFFF00 || k > 0x7FFFFF00 || batch > 0x7FFFFF00)
        return fail(FP8DSA_ERR_UNSUPPORTED, "sizes must be below 2^31 - 256");
    const bool empty_out = m == 0 || n == 0 || batch == 0;
    if (out == nullptr && !empty_out) return fail(FP8DSA_ERR_INVALID_ARG, "out is required");
    if ((reinterpret_cast<uintptr_t>(out) & 1) != 0 || (reinterpret_cast<uintptr_t>(bias) & 1) != 0)
        return fail(FP8DSA_ERR_UNSUPPORTED, "out and bias must be 2-byte aligned");
    if (ldo < n) return fail(FP8DSA_ERR_INVALID_ARG, "ldo must be >= n");
    constexpr int64_t kMaxStride = int64_t(1) << 38;  // within what a tensor map can describe
    if (lda > kMaxStride || ldb > kMaxStride || ldo > kMaxStride || stride_a > kMaxStride || stride_b > kMaxStride ||
        stride_o > kMaxStride)
        return fail(FP8DSA_ERR_UNSUPPORTED, "strides must be at most 2^38");
    if (batch > 1 && !empty_out && static_cast<__int128>(ldo) * (m - 1) + n > stride_o)
        return fail(FP8DSA_ERR_INVALID_ARG, "stride_o overlaps batches");
    const int a_mn = (layout == FP8_LAYOUT_TN || layout == FP8_LAYOUT_TT) ? 1 : 0;
    const int b_mn = (layout == FP8_LAYOUT_NN || layout == FP8_LAYOUT_TN) ? 1 : 0;
    if (!empty_out && k > 0) {
        if (a == nullptr || b == nullptr) return fail(FP8DSA_ERR_INVALID_ARG, "a and b are required");
        int rc = check_scale(scale_a, "scale_a");
        if (rc) return rc;
        rc = check_scale(scale_b, "scale_b");
        if (rc) return rc;
        if (lda < (a_mn ? m : k)) return fail(FP8DSA_ERR_INVALID_ARG, "lda too small for the layout");
        if (ldb < (b_mn ? n : k)) return fail(FP8DSA_ERR_INVALID_ARG, "ldb too small for the layout");
        if (lda % 16 != 0 || ldb % 16 != 0)
            return fail(FP8DSA_ERR_UNSUPPORTED, "lda and ldb must be multiples of 16 (TMA row strides)");
        if (!aligned16(a) || !aligned16(b)) return fail(FP8DSA_ERR_UNSUPPORTED, "a and b must be 16-byte aligned");
        if (stride_a < 0 || stride_b < 0) return fail(FP8DSA_ERR_INVALID_ARG, "negative batch stride");
        if (stride_a % 16 != 0 || stride_b % 16 != 0)
            return fail(FP8DSA_ERR_UNSUPPORTED, "batch strides must be multiples of 16");
    }
    int rc = check_device();
    if (rc) return rc;
    BlockGemmDesc d{a, b, fmt_a, fmt_b, a_mn, b_mn, m, n, k, lda, ldb, ldo, batch, stride_a, stride_b, stride_o,
                    {}, {}, bias, out};
    if (!empty_out && k > 0) {
        d.sa = *scale_a;
        d.sb = *scale_b;
    }
    return block_gemm_launch(d, stream);
}
