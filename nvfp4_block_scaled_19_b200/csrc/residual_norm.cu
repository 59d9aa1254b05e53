// The norms before and after a block, fused with its gate, its residual scale
// and the quantization of the next projection's input.  Per row r of request g:
//   z   = post(y)                              (none, RMS or layer norm)
//   h   = residual_scale * residual + branch_scale * gate[g] * z
//   out = pre(h) * (1 + scale[g]) + shift[g]   (bf16)
// and, when codes are wanted, the per-row NVFP4 quantization of that bf16 out.
//
// Mathematics: RMS x * rsqrt(mean(x^2) + eps); layer norm with the mean taken
// off first and the variance summed over the differences, both from values
// held in registers, so nothing cancels.  All of it is fp32; h feeds the pre
// norm unrounded and is rounded once, when it is stored.  Codes are computed
// from the bf16-rounded out, so they are bit for bit those of
// quantize_rowwise on it.
//
// What bounds it: memory.  Each of residual, y, h and out crosses HBM once;
// the vectors (weights, gate, scale, shift) are re-read per row from L1/L2.
// One row per group of T threads keeps the whole row in registers, so the
// chain of row reductions (at most five: two of a layer norm on either side
// and the row amax) needs no second pass over memory; the loads of a row are
// all issued before its first reduction, and several CTAs per SM overlap one
// row's reductions with another's loads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "block_ops.h"
#include "nvfp4_math.cuh"

namespace nvfp4 {
namespace {

__device__ __forceinline__ uint4 ld_stream_16B(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

__device__ __forceinline__ void unpack8(uint4 v, float *f) {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x);
    f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z);
    f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

__device__ __forceinline__ uint4 pack8(const float *f) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// Eight elements, starting at element `at`, of a weight or modulation vector.
__device__ __forceinline__ void load_vec8(const void *p, bool f32, int64_t at, float *f) {
    if (f32) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
        const float4 a = __ldg(q), b = __ldg(q + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        unpack8(__ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at)), f);
    }
}

// Reductions over the T threads of a row.  Two buffers alternate: a thread
// writes one again only after a barrier that follows every read of it.
template <int T>
struct RowReduce {
    float *red;  // [2][32] shared floats (unused for T == 32)
    int turn = 0;

    template <class Op>
    __device__ __forceinline__ float run(float v, Op op) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
        if (T == 32) return v;
        float *b = red + 32 * turn;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = v;
        __syncthreads();
        v = b[0];
#pragma unroll
        for (int w = 1; w < T / 32; ++w) v = op(v, b[w]);
        return v;
    }
    __device__ __forceinline__ float sum(float v) {
        return run(v, [](float a, float b) { return a + b; });
    }
    // Of non-negative floats, by their bits (as the quantize kernels take it).
    __device__ __forceinline__ float max(float v) {
        return run(v, [](float a, float b) {
            return __uint_as_float(::max(__float_as_uint(a), __float_as_uint(b)));
        });
    }
};

// x <- norm(x) * weight + bias over the row's V x 8 values per thread.
template <int T, int V>
__device__ __forceinline__ void norm_row(float (&x)[V][8], int kind, float eps, const void *weight,
                                         const void *bias, bool vec_f32, float inv_cols, int tx,
                                         int nvec, RowReduce<T> &rr) {
    if (kind == NVFP4_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += x[i][j];
        const float mean = rr.sum(s) * inv_cols;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * T + tx < nvec) {  // the others stay zero
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] -= mean;
            }
    }
    float s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s2 = fmaf(x[i][j], x[i][j], s2);
    const float inv = rsqrtf(fmaf(rr.sum(s2), inv_cols, eps));
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int vec = i * T + tx;
        if (vec >= nvec) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i][j] *= inv;
        if (weight != nullptr) {
            float w[8];
            load_vec8(weight, vec_f32, int64_t(vec) * 8, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] *= w[j];
        }
        if (bias != nullptr) {
            float b[8];
            load_vec8(bias, vec_f32, int64_t(vec) * 8, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] += b[j];
        }
    }
}

// T threads per row, V vectors of 8 elements per thread (vector i of thread t
// is number i * T + t of the row), ROWS rows per CTA (more than one only for
// a warp per row, which needs no CTA barrier).
template <int T, int V, int ROWS, bool kStreamF32>
__global__ void __launch_bounds__(T *ROWS) residual_norm_kernel(const nvfp4_residual_norm_args a,
                                                                const int64_t rows_per_group) {
    __shared__ float red[64];
    const int tx = threadIdx.x % T;
    const int64_t r = int64_t(blockIdx.x) * ROWS + threadIdx.x / T;
    const int nvec = static_cast<int>(a.cols >> 3);
    const int64_t kb4 = (a.cols + 63) >> 6;  // scale words per row
    if (r >= a.rows) {
        // Padding rows of the tiled scales.
        if (a.q != nullptr && r < ((a.rows + 127) & ~int64_t(127)))
            for (int64_t c = tx; c < kb4; c += T)
                *reinterpret_cast<uint32_t *>(a.sf + sf_offset(r, 4 * c, kb4)) = 0u;
        return;
    }
    const int64_t g = a.row_group != nullptr ? int64_t(__ldg(a.row_group + r)) : r / rows_per_group;
    if (g < 0 || g >= a.groups) return;  // a padding row: left as it is
    const bool vec_f32 = a.vector_dtype == NVFP4_F32;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    RowReduce<T> rr{red};

    uint4 yv[V];
    uint4 rv[kStreamF32 ? 2 * V : V];
    const uint16_t *yrow = static_cast<const uint16_t *>(a.y) + r * a.y_stride;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int vec = i * T + tx;
        yv[i] = make_uint4(0, 0, 0, 0);
        if (a.y != nullptr && vec < nvec) yv[i] = ld_stream_16B(yrow + vec * 8);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int vec = i * T + tx;
        if (kStreamF32) {
            const float *p = static_cast<const float *>(a.residual) + r * a.residual_stride + vec * 8;
            rv[2 * i] = rv[2 * i + 1] = make_uint4(0, 0, 0, 0);
            if (vec < nvec) {
                rv[2 * i] = ld_stream_16B(p);
                rv[2 * i + 1] = ld_stream_16B(p + 4);
            }
        } else {
            const uint16_t *p =
                static_cast<const uint16_t *>(a.residual) + r * a.residual_stride + vec * 8;
            rv[i] = make_uint4(0, 0, 0, 0);
            if (vec < nvec) rv[i] = ld_stream_16B(p);
        }
    }

    float x[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) unpack8(yv[i], x[i]);
    if (a.post_norm != NVFP4_NORM_NONE)
        norm_row<T, V>(x, a.post_norm, a.post_eps, a.post_weight, a.post_bias, vec_f32, inv_cols,
                       tx, nvec, rr);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int vec = i * T + tx;
        if (vec >= nvec) continue;
        float res[8];
        if (kStreamF32) {
            const uint4 lo = rv[2 * i], hi = rv[2 * i + 1];
            res[0] = __uint_as_float(lo.x); res[1] = __uint_as_float(lo.y);
            res[2] = __uint_as_float(lo.z); res[3] = __uint_as_float(lo.w);
            res[4] = __uint_as_float(hi.x); res[5] = __uint_as_float(hi.y);
            res[6] = __uint_as_float(hi.z); res[7] = __uint_as_float(hi.w);
        } else {
            unpack8(rv[i], res);
        }
        if (a.y != nullptr) {
            if (a.gate != nullptr) {
                float gt[8];
                load_vec8(a.gate, vec_f32, g * a.gate_stride + int64_t(vec) * 8, gt);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] *= gt[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[i][j] = fmaf(a.residual_scale, res[j], a.branch_scale * x[i][j]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] = a.residual_scale * res[j];
        }
        if (a.h != nullptr) {
            if (kStreamF32) {
                float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(a.h) + r * a.h_stride +
                                                       vec * 8);
                p[0] = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
                p[1] = make_float4(x[i][4], x[i][5], x[i][6], x[i][7]);
            } else {
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.h) + r * a.h_stride + vec * 8) =
                    pack8(x[i]);
            }
        }
    }
    if (a.pre_norm == NVFP4_NORM_NONE) return;
    norm_row<T, V>(x, a.pre_norm, a.pre_eps, a.pre_weight, a.pre_bias, vec_f32, inv_cols, tx, nvec,
                   rr);
    uint4 o[V];
    uint32_t mx[V];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int vec = i * T + tx;
        o[i] = make_uint4(0, 0, 0, 0);
        if (vec < nvec) {
            if (a.scale != nullptr) {
                float s[8];
                load_vec8(a.scale, vec_f32, g * a.scale_stride + int64_t(vec) * 8, s);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] = fmaf(x[i][j], s[j], x[i][j]);
            }
            if (a.shift != nullptr) {
                float s[8];
                load_vec8(a.shift, vec_f32, g * a.shift_stride + int64_t(vec) * 8, s);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] += s[j];
            }
            o[i] = pack8(x[i]);
            if (a.out != nullptr)
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + r * a.out_stride +
                                           vec * 8) = o[i];
        }
        mx[i] = absmax_bf16x8(o[i]);
        m = max(m, mx[i]);
    }
    if (a.q == nullptr) return;

    // Per-row quantization: lanes 2j and 2j + 1 hold a block of 16, eight
    // lanes a 4-byte word of block scales.  Vectors past the row are zero, so
    // the padding blocks of its last word get zero scales.
    const float amax = rr.max(__uint_as_float(m << 16));
    const float s_enc = tensor_encode_scale(amax);
    if (tx == 0) {
        a.s_dec_rows[r] = __fdiv_rn(1.0f, s_enc);
        if (a.amax_rows != nullptr) a.amax_rows[r] = amax;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int vec = i * T + tx;
        const uint32_t mb = max(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], 1));
        const BlockScale bs = block_scale_direct(__uint_as_float(mb << 16), s_enc);
        if (vec < nvec)
            *reinterpret_cast<uint32_t *>(a.q + r * (a.cols >> 1) + vec * 4) =
                quantize_bf16x8(o[i], bs.inv);
        const uint32_t sfc = vec < nvec ? bs.sf : 0u;
        const uint32_t s1 = __shfl_down_sync(0xFFFFFFFFu, sfc, 2);
        const uint32_t s2 = __shfl_down_sync(0xFFFFFFFFu, sfc, 4);
        const uint32_t s3 = __shfl_down_sync(0xFFFFFFFFu, sfc, 6);
        if ((tx & 7) == 0 && vec < nvec)
            *reinterpret_cast<uint32_t *>(a.sf + sf_offset(r, int64_t(vec >> 1), kb4)) =
                sfc | (s1 << 8) | (s2 << 16) | (s3 << 24);
    }
}

template <int T, int V, int ROWS>
cudaError_t launch(const nvfp4_residual_norm_args &a, cudaStream_t stream) {
    const int64_t rows = a.q != nullptr ? (a.rows + 127) / 128 * 128 : a.rows;
    const unsigned grid = static_cast<unsigned>((rows + ROWS - 1) / ROWS);
    const int64_t per_group = (a.rows + a.groups - 1) / a.groups;
    if (a.stream_dtype == NVFP4_F32)
        residual_norm_kernel<T, V, ROWS, true><<<grid, T * ROWS, 0, stream>>>(a, per_group);
    else
        residual_norm_kernel<T, V, ROWS, false><<<grid, T * ROWS, 0, stream>>>(a, per_group);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_residual_norm(const nvfp4_residual_norm_args &a, int num_sms,
                                 cudaStream_t stream) {
    const int64_t c = a.cols;
    // Few rows: one vector per thread, the shortest chain.  Many: two or four,
    // so that a row's reductions cost fewer threads.
    const bool few = a.rows <= 2 * int64_t(num_sms);
    if (c <= 256) return launch<32, 1, 4>(a, stream);
    if (few) {
        if (c <= 1024) return launch<128, 1, 1>(a, stream);
        if (c <= 2048) return launch<256, 1, 1>(a, stream);
        if (c <= 4096) return launch<512, 1, 1>(a, stream);
        if (c <= 8192) return launch<1024, 1, 1>(a, stream);
    }
    if (c <= 512) return launch<32, 2, 4>(a, stream);
    if (c <= 1024) return launch<32, 4, 4>(a, stream);
    if (c <= 2048) return launch<128, 2, 1>(a, stream);
    if (c <= 4096) return launch<256, 2, 1>(a, stream);
    if (c <= 8192) return launch<256, 4, 1>(a, stream);
    if (c <= 16384) return launch<512, 4, 1>(a, stream);
    return launch<1024, 4, 1>(a, stream);
}

}  // namespace nvfp4
