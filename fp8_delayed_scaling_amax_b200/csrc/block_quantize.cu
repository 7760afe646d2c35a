// FP8 quantize with one scale per block of 128: rows of 1 x 128, columns of 128 x 1, both from one
// read, or 128 x 128 blocks.
//
// For a block S of x (any subset of the elements of one 128 x 128 tile):
//     s = max(RN32(max_S |x| / FP8_MAX), 1e-12),   q = RN_fp8(RN32(x * RN32(1/s))), saturating,
// the formula of the dynamic step (fp8_amax_scale with margin 0) and of fp8_quantize, per block.
//
// Every mode walks 128 x 128 tiles, one per 256-thread CTA: a tile holds whole blocks of either
// orientation, so no reduction ever leaves the CTA and no scratch or atomic is needed.  Thread
// (tx, ty) holds columns 8 tx .. 8 tx + 7 of rows ty + 16 r, r = 0 .. 7, in registers (a warp reads
// two 256-byte row pieces of bf16 per load, all eight loads in flight): a row's maximum is a
// 16-lane shuffle, a column's one shuffle and an 8-warp shared-memory maximum.  x is read once for
// both orientations, and the column sums of the tile (the bias gradient's partial sums) come
// from the same registers.  Bound by HBM: 2 bytes in and 1 out per bf16 element and orientation.
// Measured, 8192^2 (GB/s of 6551 measured): bf16 rows 6290, columns 6300, both 5540, squares 6420; fp32 rows 6060 to 6560,
// both 5770 to 6230, squares 6660.  With
// the elements unpacked in registers (two CTAs per SM, 128 registers) and bounds checks on every row it
// was 1870 to 2100; 2048 x 1024 takes 2.6 to 4.4 us, mostly the launch and one HBM round trip.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <string>

#include "internal.h"

namespace fp8dsa {
namespace {

constexpr int kB = 128;         // block and tile edge
constexpr int kThreads = 256;
constexpr int kRowsPer = 8;     // rows per thread
constexpr int kColsPer = 8;     // columns per thread

struct BlockQuantArgs {
    const void* x;
    int64_t rows, cols;
    int64_t tiles_c;
    uint8_t* out_row;   // 1 x 128 blocks (or 128 x 128 blocks in kSquare)
    float* scale_row;   // [tiles_c][rows] (kSquare: [tiles_r][tiles_c])
    uint8_t* out_col;   // 128 x 1 blocks
    float* scale_col;   // [tiles_r][cols]
    float* colsum;      // [tiles_r][cols] column sums of each tile, or null
    int vec_in;         // 16-byte loads
    int vec_row, vec_col;  // 8-byte stores
    int vec_all;           // all of these
};

// Eight consecutive elements as they are stored: 16-bit types stay packed (4 registers), so a thread's 64
// elements leave room for three CTAs per SM.
template <int kIn>
struct Raw8 {
    uint32_t w[kIn == FP8_IN_F32 ? 8 : 4];
    static constexpr int kWords = kIn == FP8_IN_F32 ? 8 : 4;

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    // Forget what was derived from the words: unpacked values are not kept (64 registers) between uses.
    __device__ __forceinline__ void opaque() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) asm volatile("" : "+r"(w[i]));
    }
    __device__ __forceinline__ void unpack(float (&f)[8]) const {
        if constexpr (kIn == FP8_IN_F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (kIn == FP8_IN_BF16) {
                    f[2 * i] = __uint_as_float(w[i] << 16);
                    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
                } else {
                    f[2 * i] = __half2float(__ushort_as_half(static_cast<uint16_t>(w[i] & 0xFFFFu)));
                    f[2 * i + 1] = __half2float(__ushort_as_half(static_cast<uint16_t>(w[i] >> 16)));
                }
            }
        }
    }
};

// Packed running maximum of magnitudes (NaN does not enter): word by word, then its value(s).
template <int kIn>
__device__ __forceinline__ uint32_t word_max(uint32_t a, uint32_t v) {
    if constexpr (kIn == FP8_IN_BF16) return max_abs_bf16x2(a, v);
    if constexpr (kIn == FP8_IN_F16) return max_abs_f16x2(a, v);
    return __float_as_uint(fmaxf(fabsf(__uint_as_float(a)), fabsf(__uint_as_float(v))));
}
template <int kIn>
__device__ __forceinline__ void word_abs(uint32_t a, float& lo, float& hi) {
    if constexpr (kIn == FP8_IN_BF16) {
        lo = fabsf(__uint_as_float(a << 16));
        hi = fabsf(__uint_as_float(a & 0xFFFF0000u));
    } else if constexpr (kIn == FP8_IN_F16) {
        lo = fabsf(__half2float(__ushort_as_half(static_cast<uint16_t>(a & 0xFFFFu))));
        hi = fabsf(__half2float(__ushort_as_half(static_cast<uint16_t>(a >> 16))));
    } else {
        lo = hi = fabsf(__uint_as_float(a));
    }
}

// A thread's eight elements of row row0 + 16 r, zeros outside the tensor.  kFull: the tile lies wholly
// inside and rows are 16-byte aligned; `p` is the thread's first element.
template <int kIn, bool kFull>
__device__ __forceinline__ void load8(const BlockQuantArgs& g, const uint8_t* p, int r, int64_t row, int64_t col, Raw8<kIn>& v) {
    constexpr int kSize = kIn == FP8_IN_F32 ? 4 : 2;
    const uint8_t* q = p + static_cast<int64_t>(16 * r) * g.cols * kSize;
    if (kFull || (g.vec_in && row + 16 * r < g.rows && col < g.cols)) {  // vec_in: cols % 8 == 0
#pragma unroll
        for (int i = 0; i < Raw8<kIn>::kWords / 4; ++i) {
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(q) + i);
            v.w[4 * i] = a.x;
            v.w[4 * i + 1] = a.y;
            v.w[4 * i + 2] = a.z;
            v.w[4 * i + 3] = a.w;
        }
        return;
    }
    v.clear();
    if (g.vec_in || row + 16 * r >= g.rows) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (col + i < g.cols) {
            if constexpr (kIn == FP8_IN_F32)
                v.w[i] = __ldg(reinterpret_cast<const uint32_t*>(q) + i);
            else
                v.w[i >> 1] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(q) + i)) << (16 * (i & 1));
        }
    }
}

// Eight bytes of row row0 + 16 r; `p` is the thread's first byte.
template <bool kFull>
__device__ __forceinline__ void store8(uint8_t* p, const BlockQuantArgs& g, int vec, int r, int64_t row, int64_t col,
                                       uint32_t lo, uint32_t hi) {
    uint8_t* q = p + static_cast<int64_t>(16 * r) * g.cols;
    if (kFull) {
        *reinterpret_cast<uint2*>(q) = make_uint2(lo, hi);
        return;
    }
    if (row + 16 * r >= g.rows || col >= g.cols) return;
    if (vec) {
        *reinterpret_cast<uint2*>(q) = make_uint2(lo, hi);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (col + i < g.cols) q[i] = static_cast<uint8_t>((i < 4 ? lo : hi) >> (8 * (i & 3)));
}

// One tile.  kSquare: one scale per tile.  Otherwise kRow / kCol name the orientations wanted.
template <int kIn, int kFmt, bool kRow, bool kCol, bool kSquare, bool kFull>
__device__ __forceinline__ void quant_tile(const BlockQuantArgs& g, int64_t tr, int64_t tc, float (&red)[8][kB],
                                           float (&inv_col)[kB]) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row0 = tr * kB + ty, col0 = tc * kB + tx * kColsPer;

    const int64_t at = row0 * g.cols + col0;
    const uint8_t* px = static_cast<const uint8_t*>(g.x) + at * (kIn == FP8_IN_F32 ? 4 : 2);
    Raw8<kIn> v[kRowsPer];
#pragma unroll
    for (int r = 0; r < kRowsPer; ++r) load8<kIn, kFull>(g, px, r, row0, col0, v[r]);
    constexpr int kWords = Raw8<kIn>::kWords;

    if constexpr (kSquare) {
        uint32_t wm = 0u;
#pragma unroll
        for (int r = 0; r < kRowsPer; ++r)
#pragma unroll
            for (int c = 0; c < kWords; ++c) wm = word_max<kIn>(wm, v[r].w[c]);
        float am, hi;
        word_abs<kIn>(wm, am, hi);
        am = warp_max(fmaxf(am, hi));
        if (lane == 0) red[0][warp] = am;
        __syncthreads();
        am = red[0][0];
#pragma unroll
        for (int w = 1; w < 8; ++w) am = fmaxf(am, red[0][w]);
        const float s = block_step(am, kFmt), inv = __frcp_rn(s);
        if (threadIdx.x == 0) g.scale_row[tr * g.tiles_c + tc] = s;
#pragma unroll
        for (int r = 0; r < kRowsPer; ++r) {
            float f[kColsPer];
            v[r].unpack(f);
#pragma unroll
            for (int c = 0; c < kColsPer; c += 2) mul2_rn(f[c], f[c + 1], inv);
            store8<kFull>(g.out_row + at, g, g.vec_row, r, row0, col0, cvt_fp8x4<kFmt>(f[0], f[1], f[2], f[3]),
                   cvt_fp8x4<kFmt>(f[4], f[5], f[6], f[7]));
        }
        return;
    }

    if constexpr (kRow) {
        float mine = 0.0f;  // lane tx = r keeps the scale of row r
#pragma unroll
        for (int r = 0; r < kRowsPer; ++r) {
            if (!kFull && tr * kB + 2 * warp + 16 * r >= g.rows) break;  // neither of the warp's two rows exists
            uint32_t wm = 0u;
#pragma unroll
            for (int c = 0; c < kWords; ++c) wm = word_max<kIn>(wm, v[r].w[c]);
            float am, hi;
            word_abs<kIn>(wm, am, hi);
            am = fmaxf(am, hi);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
            const float s = block_step(am, kFmt), inv = __frcp_rn(s);
            if (tx == r) mine = s;
            float f[kColsPer];
            v[r].unpack(f);
#pragma unroll
            for (int c = 0; c < kColsPer; c += 2) mul2_rn(f[c], f[c + 1], inv);
            store8<kFull>(g.out_row + at, g, g.vec_row, r, row0, col0, cvt_fp8x4<kFmt>(f[0], f[1], f[2], f[3]),
                   cvt_fp8x4<kFmt>(f[4], f[5], f[6], f[7]));
        }
        const int64_t row = row0 + 16 * tx;
        if (tx < kRowsPer && row < g.rows) g.scale_row[tc * g.rows + row] = mine;
    }

    if constexpr (kCol) {
#pragma unroll
        for (int r = 0; r < kRowsPer; ++r) v[r].opaque();
        float am[kColsPer];
#pragma unroll
        for (int c = 0; c < kWords; ++c) {
            uint32_t wm = 0u;
#pragma unroll
            for (int r = 0; r < kRowsPer; ++r) wm = word_max<kIn>(wm, v[r].w[c]);
            wm = word_max<kIn>(wm, __shfl_xor_sync(0xFFFFFFFFu, wm, 16));
            if constexpr (kIn == FP8_IN_F32) {
                am[c] = fabsf(__uint_as_float(wm));
            } else {
                word_abs<kIn>(wm, am[2 * c], am[2 * c + 1]);
            }
        }
        if (lane < 16) {
            float4* dst = reinterpret_cast<float4*>(&red[warp][tx * kColsPer]);
            dst[0] = make_float4(am[0], am[1], am[2], am[3]);
            dst[1] = make_float4(am[4], am[5], am[6], am[7]);
        }
        __syncthreads();
        if (threadIdx.x < kB) {
            const int c = threadIdx.x;
            float a = red[0][c];
#pragma unroll
            for (int w = 1; w < 8; ++w) a = fmaxf(a, red[w][c]);
            const float s = block_step(a, kFmt), inv = __frcp_rn(s);
            inv_col[c] = inv;
            const int64_t col = tc * kB + c;
            if (col < g.cols) g.scale_col[tr * g.cols + col] = s;
        }
        __syncthreads();
        const float4 i0 = *reinterpret_cast<const float4*>(&inv_col[tx * kColsPer]);
        const float4 i1 = *reinterpret_cast<const float4*>(&inv_col[tx * kColsPer + 4]);
#pragma unroll
        for (int r = 0; r < kRowsPer; ++r) {
            float f[kColsPer];
            v[r].opaque();
            v[r].unpack(f);
            mul2_pair_rn(f[0], f[1], i0.x, i0.y);
            mul2_pair_rn(f[2], f[3], i0.z, i0.w);
            mul2_pair_rn(f[4], f[5], i1.x, i1.y);
            mul2_pair_rn(f[6], f[7], i1.z, i1.w);
            store8<kFull>(g.out_col + at, g, g.vec_col, r, row0, col0, cvt_fp8x4<kFmt>(f[0], f[1], f[2], f[3]),
                   cvt_fp8x4<kFmt>(f[4], f[5], f[6], f[7]));
        }
        if (g.colsum != nullptr) {
            // column sums in a fixed order: a thread's rows, the two half-warps, the warps
            float sum[kColsPer] = {};
#pragma unroll
            for (int r = 0; r < kRowsPer; ++r) {
                float f[kColsPer];
                v[r].opaque();
                v[r].unpack(f);
#pragma unroll
                for (int c = 0; c < kColsPer; ++c) sum[c] += f[c];
            }
#pragma unroll
            for (int c = 0; c < kColsPer; ++c) sum[c] += __shfl_xor_sync(0xFFFFFFFFu, sum[c], 16);
            // every thread is past its reads of `red` (the second barrier above)
            if (lane < 16) {
                float4* dst = reinterpret_cast<float4*>(&red[warp][tx * kColsPer]);
                dst[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
                dst[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
            }
            __syncthreads();
            const int64_t col = tc * kB + threadIdx.x;
            if (threadIdx.x < kB && col < g.cols) {
                float a = red[0][threadIdx.x];
#pragma unroll
                for (int w = 1; w < 8; ++w) a += red[w][threadIdx.x];
                g.colsum[tr * g.cols + col] = a;
            }
        }
    }
}

// CTAs per SM.  Squares of 16-bit types fit in 64 registers (8192^2: 32.8 us with three, 31.9 with four); the other modes
// spill there (2048 x 1024 in both orientations: 4.2 us with three, 4.7 with four).  With three, 80 registers, both
// orientations of 16-bit types spill 16 bytes a thread, the other modes nothing; fp32, whose elements take 64 registers,
// has two.
constexpr int ctas_per_sm(int in, bool square) { return in == FP8_IN_F32 ? 2 : square ? 4 : 3; }

template <int kIn, int kFmt, bool kRow, bool kCol, bool kSquare>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(kIn, kSquare)) block_quant_kernel(const __grid_constant__ BlockQuantArgs g) {
    __shared__ float red[8][kB];
    __shared__ float inv_col[kB];
    pdl_trigger();
    pdl_wait();
    const int64_t tr = blockIdx.x / g.tiles_c, tc = blockIdx.x - tr * g.tiles_c;
    if (g.vec_all && (tr + 1) * kB <= g.rows && (tc + 1) * kB <= g.cols)
        quant_tile<kIn, kFmt, kRow, kCol, kSquare, true>(g, tr, tc, red, inv_col);
    else
        quant_tile<kIn, kFmt, kRow, kCol, kSquare, false>(g, tr, tc, red, inv_col);
}

template <int kIn, int kFmt>
cudaError_t launch_fmt(const BlockQuantArgs& g, unsigned grid, bool square, cudaStream_t stream) {
    if (square) return launch_ex(block_quant_kernel<kIn, kFmt, false, false, true>, dim3(grid), dim3(kThreads), 0, stream, 1, g);
    if (g.out_row != nullptr && g.out_col != nullptr)
        return launch_ex(block_quant_kernel<kIn, kFmt, true, true, false>, dim3(grid), dim3(kThreads), 0, stream, 1, g);
    if (g.out_row != nullptr)
        return launch_ex(block_quant_kernel<kIn, kFmt, true, false, false>, dim3(grid), dim3(kThreads), 0, stream, 1, g);
    return launch_ex(block_quant_kernel<kIn, kFmt, false, true, false>, dim3(grid), dim3(kThreads), 0, stream, 1, g);
}

template <int kIn>
cudaError_t launch_in(const BlockQuantArgs& g, fp8_fmt_t fmt, unsigned grid, bool square, cudaStream_t stream) {
    return fmt == FP8_E4M3 ? launch_fmt<kIn, 0>(g, grid, square, stream) : launch_fmt<kIn, 1>(g, grid, square, stream);
}

}  // namespace

int launch_block_quantize(const BlockQuantJob& j, cudaStream_t stream) {
    if (j.rows <= 0 || j.cols <= 0) return FP8DSA_OK;
    BlockQuantArgs g{};
    g.x = j.x;
    g.rows = j.rows;
    g.cols = j.cols;
    g.tiles_c = (j.cols + kB - 1) / kB;
    const int64_t tiles_r = (j.rows + kB - 1) / kB;
    if (tiles_r > 0x7FFFFFFF / g.tiles_c) return fail(FP8DSA_ERR_UNSUPPORTED, "block quantize: too many 128 x 128 tiles");
    g.out_row = j.out_row;
    g.scale_row = j.scale_row;
    g.out_col = j.out_col;
    g.scale_col = j.scale_col;
    g.colsum = j.colsum;
    g.vec_in = aligned16(j.x) && j.cols % 8 == 0;
    g.vec_row = j.cols % 8 == 0 && (reinterpret_cast<uintptr_t>(j.out_row) & 7) == 0;
    g.vec_col = j.cols % 8 == 0 && (reinterpret_cast<uintptr_t>(j.out_col) & 7) == 0;
    g.vec_all = g.vec_in && g.vec_row && g.vec_col;
    const unsigned grid = static_cast<unsigned>(tiles_r * g.tiles_c);
    const double elems = static_cast<double>(j.rows) * j.cols;
    launch_begin(kKindQuantize, stream);
    cudaError_t e;
    switch (j.in_type) {
        case FP8_IN_BF16: e = launch_in<FP8_IN_BF16>(g, j.fmt, grid, j.square, stream); break;
        case FP8_IN_F16: e = launch_in<FP8_IN_F16>(g, j.fmt, grid, j.square, stream); break;
        default: e = launch_in<FP8_IN_F32>(g, j.fmt, grid, j.square, stream); break;
    }
    if (e != cudaSuccess) return fail(FP8DSA_ERR_CUDA, std::string("block quantize launch: ") + cudaGetErrorString(e));
    launch_end(kKindQuantize, stream,
               elems * (in_type_bytes(j.in_type) + (j.out_row != nullptr ? 1 : 0) + (j.out_col != nullptr ? 1 : 0)));
    return check_launch("block quantize kernel");
}

}  // namespace fp8dsa

using namespace fp8dsa;

extern "C" int fp8_quantize_block(const void* x, fp8_in_t in_type, int64_t rows, int64_t cols, fp8_fmt_t fmt,
                                  uint8_t* out_row, float* scale_row, uint8_t* out_col, float* scale_col,
                                  cudaStream_t stream) {
    clear_error();
    if (!valid_in_type(in_type)) return fail(FP8DSA_ERR_INVALID_ARG, "bad in_type");
    if (!valid_fmt(fmt)) return fail(FP8DSA_ERR_INVALID_ARG, "fmt must be FP8_E4M3 or FP8_E5M2");
    if (rows < 0 || cols < 0) return fail(FP8DSA_ERR_INVALID_ARG, "negative size");
    if (rows > 0 && cols > 0) {
        if (x == nullptr) return fail(FP8DSA_ERR_INVALID_ARG, "x is required");
        if (out_row == nullptr && out_col == nullptr) return fail(FP8DSA_ERR_INVALID_ARG, "out_row or out_col is required");
        if ((out_row == nullptr) != (scale_row == nullptr) || (out_col == nullptr) != (scale_col == nullptr))
            return fail(FP8DSA_ERR_INVALID_ARG, "out_row and scale_row, out_col and scale_col go together");
        if (reinterpret_cast<uintptr_t>(x) % in_type_bytes(in_type) != 0)
            return fail(FP8DSA_ERR_UNSUPPORTED, "x must be aligned to its element size");
        if ((reinterpret_cast<uintptr_t>(scale_row) & 3) != 0 || (reinterpret_cast<uintptr_t>(scale_col) & 3) != 0)
            return fail(FP8DSA_ERR_UNSUPPORTED, "scales must be 4-byte aligned");
    }
    int rc = check_device();
    if (rc) return rc;
    BlockQuantJob j;
    j.x = x;
    j.in_type = in_type;
    j.rows = rows;
    j.cols = cols;
    j.fmt = fmt;
    j.out_row = out_row;
    j.scale_row = scale_row;
    j.out_col = out_col;
    j.scale_col = scale_col;
    return launch_block_quantize(j, stream);
}

extern "C" int fp8_quantize_block128(const void* x, fp8_in_t in_type, int64_t rows, int64_t cols, fp8_fmt_t fmt,
                                     uint8_t* out, float* scale, cudaStream_t stream) {
    clear_error();
    if (!valid_in_type(in_type)) return fail(FP8DSA_ERR_INVALID_ARG, "bad in_type");
    if (!valid_fmt(fmt)) return fail(FP8DSA_ERR_INVALID_ARG, "fmt must be FP8_E4M3 or FP8_E5M2");
    if (rows < 0 || cols < 0) return fail(FP8DSA_ERR_INVALID_ARG, "negative size");
    if (rows > 0 && cols > 0) {
        if (x == nullptr || out == nullptr || scale == nullptr)
            return fail(FP8DSA_ERR_INVALID_ARG, "x, out and scale are required");
        if (reinterpret_cast<uintptr_t>(x) % in_type_bytes(in_type) != 0)
            return fail(FP8DSA_ERR_UNSUPPORTED, "x must be aligned to its element size");
        if ((reinterpret_cast<uintptr_t>(scale) & 3) != 0)
            return fail(FP8DSA_ERR_UNSUPPORTED, "scale must be 4-byte aligned");
    }
    int rc = check_device();
    if (rc) return rc;
    BlockQuantJob j;
    j.x = x;
    j.in_type = in_type;
    j.rows = rows;
    j.cols = cols;
    j.fmt = fmt;
    j.out_row = out;
    j.scale_row = scale;
    j.square = true;
    return launch_block_quantize(j, stream);
}
