// C ABI of the operators around a projection (declared in include/nvfp4.h):
// argument checks, device check and launches.  Like every entry point, a call
// is refused before any device work, nothing is allocated and nothing
// synchronises.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_checks.h"
#include "block_ops.h"
#include "nvfp4.h"

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Elements from row to row of a [rows, cols] array: whole 16-byte vectors,
// rows that do not overlap, and offsets that stay inside 2^60 elements.
bool stride_ok(int64_t stride, int64_t rows, int64_t cols) {
    return stride >= cols && stride % 8 == 0 && stride <= (int64_t(1) << 60) / (rows > 0 ? rows : 1);
}

bool vector_ok(const void *p, int64_t stride, int64_t groups, int64_t cols) {
    return p == nullptr || stride == 0 || stride_ok(stride, groups, cols);
}

bool norm_ok(int kind, float eps, const void *weight, const void *bias) {
    if (kind == NVFP4_NORM_NONE) return weight == nullptr && bias == nullptr;
    if (kind != NVFP4_NORM_RMS && kind != NVFP4_NORM_LAYER) return false;
    return std::isfinite(eps) && eps >= 0.0f;
}

// The status of a launch; a refused one leaves no error behind for others to find.
nvfp4_status launched(cudaError_t e) {
    if (e == cudaSuccess) return NVFP4_OK;
    cudaGetLastError();
    return NVFP4_ERR_LAUNCH;
}

bool lora_sizes_ok(int64_t rows, int64_t k, int64_t n, int64_t rank) {
    return rows >= 0 && rows <= (int64_t(1) << 27) && k >= 16 && k <= (1 << 20) && k % 16 == 0 &&
           n >= 16 && n <= (1 << 20) && n % 8 == 0 && rank >= 16 && rank <= 128 && rank % 16 == 0;
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_residual_norm(const nvfp4_residual_norm_args *args, nvfp4_stream_t stream) {
    if (args == nullptr) return NVFP4_ERR_INVALID_ARG;
    const nvfp4_residual_norm_args &a = *args;
    if (a.rows < 0 || a.rows > (int64_t(1) << 31) - 256 || a.cols < 16 || a.cols > 32768 ||
        a.cols % 16 != 0)
        return NVFP4_ERR_INVALID_ARG;
    if ((a.stream_dtype != NVFP4_BF16 && a.stream_dtype != NVFP4_F32) ||
        (a.vector_dtype != NVFP4_BF16 && a.vector_dtype != NVFP4_F32))
        return NVFP4_ERR_INVALID_ARG;
    if (!norm_ok(a.post_norm, a.post_eps, a.post_weight, a.post_bias) ||
        !norm_ok(a.pre_norm, a.pre_eps, a.pre_weight, a.pre_bias))
        return NVFP4_ERR_INVALID_ARG;
    if (!std::isfinite(a.residual_scale) || !std::isfinite(a.branch_scale))
        return NVFP4_ERR_INVALID_ARG;
    if (a.groups < 1 || a.groups > (int64_t(1) << 31) ||
        (a.row_group == nullptr && a.rows % a.groups != 0))
        return NVFP4_ERR_INVALID_ARG;
    const bool normed = a.out != nullptr || a.q != nullptr;
    // Rows that are empty have arrays that may be NULL.
    if (a.rows > 0) {
        if (a.residual == nullptr || (a.h == nullptr && !normed)) return NVFP4_ERR_INVALID_ARG;
        if (a.y == nullptr && (a.h != nullptr || a.gate != nullptr || a.post_norm != NVFP4_NORM_NONE))
            return NVFP4_ERR_INVALID_ARG;
        if (normed && a.pre_norm == NVFP4_NORM_NONE) return NVFP4_ERR_INVALID_ARG;
        if (!normed && (a.pre_norm != NVFP4_NORM_NONE || a.scale != nullptr || a.shift != nullptr))
            return NVFP4_ERR_INVALID_ARG;
        if (a.q != nullptr ? (a.sf == nullptr || a.s_dec_rows == nullptr)
                           : (a.sf != nullptr || a.s_dec_rows != nullptr || a.amax_rows != nullptr))
            return NVFP4_ERR_INVALID_ARG;
    }
    if (!stride_ok(a.residual_stride, a.rows, a.cols) ||
        (a.y != nullptr && !stride_ok(a.y_stride, a.rows, a.cols)) ||
        (a.h != nullptr && !stride_ok(a.h_stride, a.rows, a.cols)) ||
        (a.out != nullptr && !stride_ok(a.out_stride, a.rows, a.cols)) ||
        !vector_ok(a.gate, a.gate_stride, a.groups, a.cols) ||
        !vector_ok(a.scale, a.scale_stride, a.groups, a.cols) ||
        !vector_ok(a.shift, a.shift_stride, a.groups, a.cols))
        return NVFP4_ERR_INVALID_ARG;
    // In place only row on row: the same type and stride.
    const bool f32 = a.stream_dtype == NVFP4_F32;
    const auto over = [&](const void *out, int64_t out_stride, const void *in, int64_t in_stride, bool types) {
        return out != nullptr && out == in && (types || (a.rows > 1 && out_stride != in_stride));
    };
    if (over(a.h, a.h_stride, a.residual, a.residual_stride, false) || over(a.h, a.h_stride, a.y, a.y_stride, f32) ||
        over(a.out, a.out_stride, a.y, a.y_stride, false) ||
        over(a.out, a.out_stride, a.residual, a.residual_stride, f32))
        return NVFP4_ERR_INVALID_ARG;
    const void *wide[] = {a.residual, a.y,    a.h,     a.out,   a.post_weight, a.post_bias, a.pre_weight,
                          a.pre_bias, a.gate, a.scale, a.shift, a.q,           a.sf};
    for (const void *p : wide)
        if (!aligned(p, 16)) return NVFP4_ERR_MISALIGNED;
    if (!aligned(a.row_group, 4) || !aligned(a.s_dec_rows, 4) || !aligned(a.amax_rows, 4))
        return NVFP4_ERR_MISALIGNED;
    int sms = 0;
    const nvfp4_status st = nvfp4::current_device(&sms);
    if (st != NVFP4_OK) return st;
    if (a.rows == 0) return NVFP4_OK;
    return launched(nvfp4::launch_residual_norm(a, sms, stream));
}

size_t nvfp4_lora_workspace_bytes(int64_t rows, int64_t k, int64_t n, int64_t rank) {
    if (!lora_sizes_ok(rows, k, n, rank)) return 0;
    return nvfp4::lora_workspace_bytes(rows, k, n, rank);
}

nvfp4_status nvfp4_lora(const nvfp4_lora_args *args, nvfp4_stream_t stream) {
    if (args == nullptr) return NVFP4_ERR_INVALID_ARG;
    const nvfp4_lora_args &p = *args;
    if (!lora_sizes_ok(p.rows, p.k, p.n, p.rank)) return NVFP4_ERR_INVALID_ARG;
    const int64_t widest = p.k > p.n ? p.k : p.n;
    if (p.slots < 1 || p.slots >= (int64_t(1) << 31) / (widest > p.rank ? widest : p.rank))
        return NVFP4_ERR_INVALID_ARG;
    if (p.a == nullptr || p.b == nullptr || p.scale == nullptr) return NVFP4_ERR_INVALID_ARG;
    if (p.rows > 0 && (p.x == nullptr || p.y == nullptr || p.out == nullptr || p.out == p.x))
        return NVFP4_ERR_INVALID_ARG;
    // (A tensor map takes strides below 2^40 bytes.)
    const int64_t strides[] = {p.x_stride, p.y_stride, p.out_stride};
    for (const int64_t s : strides)
        if (s >= int64_t(1) << 39) return NVFP4_ERR_INVALID_ARG;
    if (!stride_ok(p.x_stride, p.rows, p.k) || !stride_ok(p.y_stride, p.rows, p.n) ||
        !stride_ok(p.out_stride, p.rows, p.n))
        return NVFP4_ERR_INVALID_ARG;
    if (p.out == p.y && p.out_stride != p.y_stride) return NVFP4_ERR_INVALID_ARG;
    const bool needs_workspace = nvfp4::lora_workspace_bytes(p.rows, p.k, p.n, p.rank) > 0;
    if (needs_workspace && p.workspace == nullptr) return NVFP4_ERR_INVALID_ARG;
    const void *wide[] = {p.x, p.y, p.out, p.a, p.b, p.workspace};
    for (const void *q : wide)
        if (!aligned(q, 16)) return NVFP4_ERR_MISALIGNED;
    if (!aligned(p.scale, 4) || !aligned(p.row_slot, 4)) return NVFP4_ERR_MISALIGNED;
    int sms = 0;
    const nvfp4_status st = nvfp4::current_device(&sms);
    if (st != NVFP4_OK) return st;
    if (p.rows == 0) return NVFP4_OK;
    return launched(nvfp4::launch_lora(p, stream));
}

}  // extern "C"
