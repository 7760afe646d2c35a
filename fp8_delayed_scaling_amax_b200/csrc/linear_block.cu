// FP8 linear layer with block scaling (one scale for each block of 128 along the contraction): the forward,
// and the backward's grad_x, grad_w and grad_b, composed from the block quantizer and the block-scaled
// products.
//
//     y      [m][n] = x8 . w8^T + bias     x in 1 x 128 blocks along k, w in 128 x 128 blocks
//     grad_x [m][k] = g8 . w8              g in 1 x 128 blocks along n, w's bytes and scales as they are
//     grad_w [n][k] = g8c^T . x8c          g and x in 128 x 1 blocks along the tokens
//     grad_b [n]    = sum over the tokens of g
//
// A block's scale has to run along the contraction of the product that uses it, so x and g have two
// quantizations (along the row, and down the column), formed from one read of each; the column form of x
// is left by the forward for the backward.  Nothing is transposed: the tensor cores read w8 and the
// column forms as MN-major operands.
//
// Launches: forward 2 (x, product) + 1 when w is bf16; one in all for at most kStreamMaxBf16Rows rows of
// an FP8 weight, where the product quantizes x itself.  Backward 1 (g) + 1 per product + 1 for grad_b.
#include <cuda_runtime.h>

#include <string>

#include "internal.h"

namespace fp8dsa {
namespace {

constexpr size_t kAlign = 256;

int64_t blocks_of(int64_t n) { return (n + 127) / 128; }

struct FwdLayout {
    size_t x8, sx, w8, sw, total;
};
FwdLayout fwd_layout(int64_t m, int64_t k, int64_t n) {
    FwdLayout L;
    size_t off = 0;
    L.x8 = off;
    off = align_up(off + static_cast<size_t>(m) * k, kAlign);
    L.sx = off;
    off = align_up(off + sizeof(float) * static_cast<size_t>(m) * blocks_of(k), kAlign);
    L.w8 = off;
    off = align_up(off + static_cast<size_t>(n) * k, kAlign);
    L.sw = off;
    off = align_up(off + sizeof(float) * static_cast<size_t>(blocks_of(n)) * blocks_of(k), kAlign);
    L.total = off;
    return L;
}

// Whether x is quantized by a launch of its own: for its column form, or for a product of more than
// kStreamMaxBf16Rows rows (with fewer the product quantizes x itself: one launch).
bool quantizes_x(int64_t m, int64_t k, int64_t n, const uint8_t* x8c_out) {
    return m > 0 && k > 0 && (x8c_out != nullptr || (n > 0 && m > kStreamMaxBf16Rows));
}

// What a call touches of its layout: all of it where w is quantized into the workspace, x8 with its scales (which
// lie first) where only x is.
size_t fwd_need(int64_t m, int64_t k, int64_t n, bool w8_elsewhere, const uint8_t* x8c_out) {
    const FwdLayout L = fwd_layout(m, k, n);
    return !w8_elsewhere && n > 0 ? L.total : quantizes_x(m, k, n, x8c_out) ? L.w8 : 0;
}

struct BwdLayout {
    size_t g8, sg, g8c, sgc, colsum, total;
};
BwdLayout bwd_layout(int64_t m, int64_t n) {
    BwdLayout L;
    size_t off = 0;
    const size_t mn = static_cast<size_t>(m) * n;
    L.g8 = off;
    off = align_up(off + mn, kAlign);
    L.sg = off;
    off = align_up(off + sizeof(float) * static_cast<size_t>(m) * blocks_of(n), kAlign);
    L.g8c = off;
    off = align_up(off + mn, kAlign);
    L.sgc = off;
    off = align_up(off + sizeof(float) * static_cast<size_t>(blocks_of(m)) * n, kAlign);
    L.colsum = off;
    off = align_up(off + sizeof(float) * static_cast<size_t>(blocks_of(m)) * n, kAlign);
    L.total = off;
    return L;
}

bool sizes_ok(int64_t m, int64_t k, int64_t n) {
    constexpr int64_t kMax = 0x7FFFFF00;
    return m >= 0 && k >= 0 && n >= 0 && m <= kMax && k <= kMax && n <= kMax;
}

int check_common(int64_t m, int64_t k, int64_t n, const void* workspace, size_t bytes, size_t need) {
    if (m < 0 || k < 0 || n < 0) return fail(FP8DSA_ERR_INVALID_ARG, "negative size");
    if (!sizes_ok(m, k, n)) return fail(FP8DSA_ERR_UNSUPPORTED, "sizes must be below 2^31 - 256");
    if (k % 16 != 0 || n % 16 != 0) return fail(FP8DSA_ERR_UNSUPPORTED, "k and n must be multiples of 16");
    if (need == 0) return FP8DSA_OK;
    if (workspace == nullptr) return fail(FP8DSA_ERR_INVALID_ARG, "workspace is required");
    if ((reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0)
        return fail(FP8DSA_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
    if (bytes < need) return fail(FP8DSA_ERR_WORKSPACE, "workspace too small");
    return FP8DSA_OK;
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

BlockGemmDesc product(const uint8_t* a, const uint8_t* b, int fmt_a, int fmt_b, int a_mn, int b_mn, int64_t m, int64_t n,
                      int64_t k, const fp8_block_scale_t& sa, const fp8_block_scale_t& sb, const void* bias, void* out) {
    return BlockGemmDesc{a, b, fmt_a, fmt_b, a_mn, b_mn, m, n, k, a_mn ? m : k, b_mn ? n : k, n, 1, 0, 0, m * n, sa, sb, bias, out};
}

}  // namespace
}  // namespace fp8dsa

using namespace fp8dsa;

extern "C" size_t linear_forward_fp8_block_workspace_size(int64_t m, int64_t k, int64_t n) {
    return sizes_ok(m, k, n) ? fwd_layout(m, k, n).total : 0;
}

extern "C" int linear_forward_fp8_block(const void* x, const void* w, int w_is_fp8, const float* w_scale, const void* bias,
                                        int64_t m, int64_t k, int64_t n, fp8_fmt_t fmt, uint8_t* w8_out,
                                        float* w_scale_out, uint8_t* x8c_out, float* x8c_scale_out, void* workspace,
                                        size_t workspace_bytes, void* y, cudaStream_t stream) {
    clear_error();
    if (!valid_fmt(fmt)) return fail(FP8DSA_ERR_INVALID_ARG, "fmt must be FP8_E4M3 or FP8_E5M2");
    int rc = check_common(m, k, n, workspace, workspace_bytes,
                          sizes_ok(m, k, n) ? fwd_need(m, k, n, w_is_fp8 || w8_out != nullptr, x8c_out) : 0);
    if (rc) return rc;
    const bool has_x = m > 0 && k > 0, has_w = n > 0 && k > 0, has_y = m > 0 && n > 0;
    if ((has_x && x == nullptr) || (has_w && w == nullptr) || (has_y && y == nullptr))
        return fail(FP8DSA_ERR_INVALID_ARG, "x, w and y are required");
    if (w_is_fp8 && has_w && w_scale == nullptr) return fail(FP8DSA_ERR_INVALID_ARG, "an fp8 w needs w_scale");
    if (w_is_fp8 && (w8_out != nullptr || w_scale_out != nullptr))
        return fail(FP8DSA_ERR_INVALID_ARG, "w8_out is for a bf16 w");
    if ((w8_out == nullptr) != (w_scale_out == nullptr) || (x8c_out == nullptr) != (x8c_scale_out == nullptr))
        return fail(FP8DSA_ERR_INVALID_ARG, "w8_out and w_scale_out, x8c_out and x8c_scale_out go together");
    if (misaligned(x, 2) || misaligned(y, 2) || misaligned(bias, 2) || misaligned(w, w_is_fp8 ? 16 : 2) ||
        misaligned(w8_out, 16) || misaligned(x8c_out, 16) || misaligned(w_scale, 4) || misaligned(w_scale_out, 4) ||
        misaligned(x8c_scale_out, 4))
        return fail(FP8DSA_ERR_UNSUPPORTED, "bf16 tensors must be 2-byte, scales 4-byte and fp8 tensors 16-byte aligned");
    rc = check_device();
    if (rc) return rc;

    const FwdLayout L = fwd_layout(m, k, n);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const uint8_t* w8 = static_cast<const uint8_t*>(w);
    const float* sw = w_scale;
    if (!w_is_fp8 && has_w) {
        BlockQuantJob j;
        j.x = w;
        j.rows = n;
        j.cols = k;
        j.fmt = fmt;
        j.square = true;
        j.out_row = w8_out != nullptr ? w8_out : ws + L.w8;
        j.scale_row = w8_out != nullptr ? w_scale_out : reinterpret_cast<float*>(ws + L.sw);
        rc = launch_block_quantize(j, stream);
        if (rc) return rc;
        w8 = j.out_row;
        sw = j.scale_row;
    }
    const fp8_block_scale_t sb{sw, 128, blocks_of(k), 1, 0};
    const bool with_x8 = quantizes_x(m, k, n, x8c_out);
    if (has_x && has_y && !with_x8) {
        const BlockGemmDesc d = product(static_cast<const uint8_t*>(x), w8, fmt, fmt, 0, 0, m, n, k, {}, sb, bias, y);
        return block_stream_gemm(d, true, stream);
    }
    uint8_t* x8 = ws + L.x8;
    float* sx = reinterpret_cast<float*>(ws + L.sx);
    if (with_x8) {
        BlockQuantJob j;
        j.x = x;
        j.rows = m;
        j.cols = k;
        j.fmt = fmt;
        j.out_row = x8;
        j.scale_row = sx;
        j.out_col = x8c_out;
        j.scale_col = x8c_scale_out;
        rc = launch_block_quantize(j, stream);
        if (rc) return rc;
    }
    return block_gemm_launch(product(x8, w8, fmt, fmt, 0, 0, m, n, k, {sx, 1, 1, m, 0}, sb, bias, y), stream);
}

extern "C" size_t linear_backward_fp8_block_workspace_size(int64_t m, int64_t k, int64_t n) {
    return sizes_ok(m, k, n) ? bwd_layout(m, n).total : 0;
}

extern "C" int linear_backward_fp8_block(const void* g, const uint8_t* x8c, const float* x8c_scale, const uint8_t* w8,
                                         const float* w_scale, int64_t m, int64_t k, int64_t n, fp8_fmt_t fmt_g,
                                         fp8_fmt_t fmt, int need_grad_x, int need_grad_w, int need_grad_b, void* workspace,
                                         size_t workspace_bytes, void* grad_x, void* grad_w, void* grad_b,
                                         cudaStream_t stream) {
    clear_error();
    if (!valid_fmt(fmt) || !valid_fmt(fmt_g)) return fail(FP8DSA_ERR_INVALID_ARG, "fmt must be FP8_E4M3 or FP8_E5M2");
    int rc = check_common(m, k, n, workspace, workspace_bytes, linear_backward_fp8_block_workspace_size(m, k, n));
    if (rc) return rc;
    const bool has_g = m > 0 && n > 0, has_x = m > 0 && k > 0, has_w = n > 0 && k > 0;
    const bool any = need_grad_x || need_grad_w || need_grad_b;
    if (any && has_g && g == nullptr) return fail(FP8DSA_ERR_INVALID_ARG, "g is required");
    if (need_grad_x && ((has_w && has_x && (w8 == nullptr || w_scale == nullptr)) || (has_x && grad_x == nullptr)))
        return fail(FP8DSA_ERR_INVALID_ARG, "grad_x needs w8, w_scale and grad_x");
    if (need_grad_w && ((has_x && has_w && (x8c == nullptr || x8c_scale == nullptr)) || (has_w && grad_w == nullptr)))
        return fail(FP8DSA_ERR_INVALID_ARG, "grad_w needs x8c, x8c_scale and grad_w");
    if (need_grad_b && n > 0 && grad_b == nullptr) return fail(FP8DSA_ERR_INVALID_ARG, "grad_b is required");
    if (misaligned(g, 2) || misaligned(grad_x, 2) || misaligned(grad_w, 2) || misaligned(grad_b, 2) || misaligned(x8c, 16) ||
        misaligned(w8, 16) || misaligned(x8c_scale, 4) || misaligned(w_scale, 4))
        return fail(FP8DSA_ERR_UNSUPPORTED, "bf16 tensors must be 2-byte, scales 4-byte and fp8 tensors 16-byte aligned");
    rc = check_device();
    if (rc) return rc;
    if (!any) return FP8DSA_OK;

    const BwdLayout L = bwd_layout(m, n);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    BlockQuantJob j;
    j.x = g;
    j.rows = m;
    j.cols = n;
    j.fmt = fmt_g;
    if (need_grad_x) {
        j.out_row = ws + L.g8;
        j.scale_row = reinterpret_cast<float*>(ws + L.sg);
    }
    if (need_grad_w || need_grad_b) {  // the column sums come with the column form
        j.out_col = ws + L.g8c;
        j.scale_col = reinterpret_cast<float*>(ws + L.sgc);
    }
    if (need_grad_b) j.colsum = reinterpret_cast<float*>(ws + L.colsum);
    rc = launch_block_quantize(j, stream);
    if (rc) return rc;
    if (need_grad_x) {
        rc = block_gemm_launch(product(j.out_row, w8, fmt_g, fmt, 0, 1, m, k, n, {j.scale_row, 1, 1, m, 0},
                                       {w_scale, 128, 1, blocks_of(k), 0}, nullptr, grad_x), stream);
        if (rc) return rc;
    }
    if (need_grad_w) {
        rc = block_gemm_launch(product(j.out_col, x8c, fmt_g, fmt, 1, 1, n, k, m, {j.scale_col, 1, 1, n, 0},
                                       {x8c_scale, 1, 1, k, 0}, nullptr, grad_w), stream);
        if (rc) return rc;
    }
    if (need_grad_b && n > 0) {
        if (m > 0) return launch_colsum_finalize(j.colsum, blocks_of(m), n, grad_b, stream);
        const cudaError_t e = cudaMemsetAsync(grad_b, 0, sizeof(uint16_t) * static_cast<size_t>(n), stream);
        if (e != cudaSuccess) return fail(FP8DSA_ERR_CUDA, std::string("memset grad_b: ") + cudaGetErrorString(e));
    }
    return FP8DSA_OK;
}
