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
// The threads of a row keep all of it in registers, so the chain of row
// reductions (at most five: two of a layer norm on either side and the row
// amax) needs no second pass over memory.  Two forms: a CTA per row for few of
// them and for wide ones (residual_norm_kernel: 1 x 4096 2.5 us, 93 x 5120 5.0 us;
// 2^27 values in rows of 12288 3.3 TB/s, 16384 3.8, 32768 4.0), and persistent CTAs
// with prefetched rows (residual_norm_rows_kernel).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "block_ops.h"
#include "block_waits.cuh"
#include "gemm.h"
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

// Codes and block scale of vector `vec` of row r (eight bf16 values `o` whose
// largest magnitude has the bits mx): lanes 2j and 2j + 1 hold a block of 16,
// eight lanes a 4-byte word of block scales.  All lanes of a warp call;
// vectors past the row are zero, so the padding blocks of its last word get
// zero scales.
__device__ __forceinline__ void quantize_vec(const nvfp4_residual_norm_args &a, int64_t r, int vec,
                                             int nvec, uint4 o, uint32_t mx, float s_enc) {
    const uint32_t mb = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
    const BlockScale bs = block_scale_direct(__uint_as_float(mb << 16), s_enc);
    if (vec < nvec)
        *reinterpret_cast<uint32_t *>(a.q + r * (a.cols >> 1) + vec * 4) = quantize_bf16x8(o, bs.inv);
    const uint32_t sfc = vec < nvec ? bs.sf : 0u;
    const uint32_t s1 = __shfl_down_sync(0xFFFFFFFFu, sfc, 2);
    const uint32_t s2 = __shfl_down_sync(0xFFFFFFFFu, sfc, 4);
    const uint32_t s3 = __shfl_down_sync(0xFFFFFFFFu, sfc, 6);
    if ((vec & 7) == 0 && vec < nvec)
        *reinterpret_cast<uint32_t *>(a.sf + sf_offset(r, int64_t(vec >> 1), (a.cols + 63) >> 6)) =
            sfc | (s1 << 8) | (s2 << 16) | (s3 << 24);
}

// RN(a / 6) of a non-negative bf16 value in three fp32 operations.  Why it is
// exact: c = RN(1/6) puts q = RN(a c) within two units of its last place of
// a / 6, so a - 6 q is a small multiple of that unit and the fma gives it
// without rounding; adding its sixth, computed to 24 bits, makes the value that
// is rounded at the end agree with a / 6 to 2^-22 units, and a / 6 of a bf16 a
// is 0, 1/3 or 2/3 of a unit above a representable number, at least 1/6 from
// where rounding changes.  Values whose quotient could be subnormal (below 2^-100),
// infinity and NaN take the double product of nvfp4_math.cuh.
__device__ __forceinline__ float sixth(float a) {
    constexpr uint32_t least = 27u << 23 /* 2^-100 */, inf = 0x7F800000u;
    if (__float_as_uint(a) - least >= inf - least) return div6_short(a);
    const float c = 1.0f / 6.0f;
    const float q = __fmul_rn(a, c);
    return __fmaf_rn(__fmaf_rn(-6.0f, q, a), c, q);
}

// Value of an E4M3 code by the conversion instructions (every one is a half); of
// NaN's code (an infinite block under S_enc = 0) 480, as e4m3_decode reads it.
__device__ __forceinline__ float e4m3_value(uint32_t code) {
    float v;
    asm("{\n\t.reg .b32 h2;\n\t.reg .b16 c, lo, hi;\n\t"
        "cvt.u16.u32 c, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 h2, c;\n\t"
        "mov.b32 {lo, hi}, h2;\n\t"
        "cvt.f32.f16 %0, lo;\n\t}\n"
        : "=f"(v)
        : "r"(code));
    return code == 0x7Fu ? 480.0f : v;
}

// Codes and block scales of two vectors of a thread, as quantize_vec gives them
// for each: `q0` and `q1` are where their codes go, `sf` where the word of block
// scales goes that this thread may have to write (see sf_word).  The two lanes
// that share a block share its scale: the even one computes the first vector's,
// the odd one the second's, one division each.
__device__ __forceinline__ void quantize_two(uint8_t *q0, uint8_t *q1, uint8_t *sf, bool second, uint4 o0,
                                             uint4 o1, uint32_t m0, uint32_t m1, float s_enc) {
    const bool odd = threadIdx.x & 1;
    m0 = max(m0, __shfl_xor_sync(0xFFFFFFFFu, m0, 1));
    m1 = max(m1, __shfl_xor_sync(0xFFFFFFFFu, m1, 1));
    const uint32_t code = e4m3_encode(__fmul_rn(sixth(__uint_as_float((odd ? m1 : m0) << 16)), s_enc));
    const float value = e4m3_value(code);
    float inv = 0.0f;
    if (value != 0.0f) {
        inv = __fdiv_rn(s_enc, value);
        if (!isfinite(inv)) inv = FLT_MAX;
    }
    const float other = __shfl_xor_sync(0xFFFFFFFFu, inv, 1);
    *reinterpret_cast<uint32_t *>(q0) = quantize_bf16x8(o0, odd ? other : inv);
    if (second) *reinterpret_cast<uint32_t *>(q1) = quantize_bf16x8(o1, odd ? inv : other);
    // Four blocks (eight lanes) a word: lane 0 of the eight gathers the first
    // vector's, lane 1 the second's.
    const uint32_t s0 = odd && !second ? 0u : code;
    const uint32_t s1 = __shfl_down_sync(0xFFFFFFFFu, s0, 2);
    const uint32_t s2 = __shfl_down_sync(0xFFFFFFFFu, s0, 4);
    const uint32_t s3 = __shfl_down_sync(0xFFFFFFFFu, s0, 6);
    if ((threadIdx.x & 6) == 0 && (!odd || second))
        *reinterpret_cast<uint32_t *>(sf) = s0 | (s1 << 8) | (s2 << 16) | (s3 << 24);
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

    const float amax = rr.max(__uint_as_float(m << 16));
    const float s_enc = tensor_encode_scale(amax);
    if (tx == 0) {
        a.s_dec_rows[r] = __fdiv_rn(1.0f, s_enc);
        if (a.amax_rows != nullptr) a.amax_rows[r] = amax;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) quantize_vec(a, r, i * T + tx, nvec, o[i], mx[i], s_enc);
}

// ---------------------------------------------------------------- many rows

constexpr int kMaxStages = 8;
constexpr int kRingBytes = 160 * 1024;
// Of a CTA: half the ring's bytes (two CTAs at least share an SM), or two rows of
// the widest kind, 8192 columns of bf16 y and fp32 residual.
constexpr int kMaxRowBytes = 8192 * (2 + 4);
constexpr int kMaxSmem = 2 * kMaxRowBytes > kRingBytes / 2 ? 2 * kMaxRowBytes : kRingBytes / 2;
constexpr int kTimeoutTag = 48;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ void unpack4(uint4 v, float2 (&f)[4]) {
    f[0] = make_float2(bf16_lo(v.x), bf16_hi(v.x));
    f[1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
    f[2] = make_float2(bf16_lo(v.z), bf16_hi(v.z));
    f[3] = make_float2(bf16_lo(v.w), bf16_hi(v.w));
}

__device__ __forceinline__ uint4 pack4(const float2 (&f)[4]) {
    return make_uint4(pack2(f[0].x, f[0].y), pack2(f[1].x, f[1].y), pack2(f[2].x, f[2].y),
                      pack2(f[3].x, f[3].y));
}

// A weight or modulation vector's eight elements at `vec`, as loaded and as
// four pairs.  `p` may be NULL (then `f` is not touched).
template <bool kF32>
struct RawVec {
    uint4 w[kF32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *p, int vec) {
        if (p == nullptr) return;
        const uint4 *q = static_cast<const uint4 *>(p) + vec * (kF32 ? 2 : 1);
        w[0] = __ldg(q);
        if (kF32) w[kF32 ? 1 : 0] = __ldg(q + 1);
    }
    __device__ __forceinline__ void get(float2 (&f)[4]) const {
        if (kF32) {
            const uint4 b = w[kF32 ? 1 : 0];
            f[0] = make_float2(__uint_as_float(w[0].x), __uint_as_float(w[0].y));
            f[1] = make_float2(__uint_as_float(w[0].z), __uint_as_float(w[0].w));
            f[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
            f[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
        } else {
            unpack4(w[0], f);
        }
    }
};

constexpr int kVecs = 2;  // vectors of 8 columns per thread

// Persistent CTAs of T = blockDim.x threads, two vectors per thread, rows
// blockIdx.x, + gridDim.x, ...  y and the residual arrive by bulk copies,
// `stages` rows ahead of the arithmetic, so the bytes in flight depend neither
// on occupancy nor on a row's reductions.  What is left to keep small is the
// instruction count: a row's fixed cost (barriers, reductions, addresses) is
// shared by 16 columns per thread (8 took 1.4 times the time; 32 spill), and the
// arithmetic takes fp32 pairs.  64 registers, so that 1024 threads share an SM.
// Measured: 33792 x 4096, layer norm with gate and modulation, 181 us (1.11 GB,
// 6.1 TB/s; the measured copy 6.5); 8192 x 8192 with an fp32 stream and norms on
// both sides 148 us (5.4 TB/s); 4571 x 2560 21 us (4.4 TB/s: 5 rows per CTA);
// 4608 x 4096 into codes 39 us (3.2 TB/s: its 718 instructions per warp and row,
// a third of them for the codes, are 23 us at full issue, and the issue slots are
// 58 % busy: three barriers a row, 8 rounds of 7.8 rows per CTA and the start-up
// are the rest).  2^27 values of a bf16 stream: 1152 columns 4.3 TB/s, 2880 5.4, 5376
// 5.1.  fp32 vectors spill 40 to 104 bytes a thread (4096 columns 5.9 -> 4.8 TB/s).
template <bool kFull, bool kQuant, bool kStreamF32, bool kVecF32>
__global__ void __launch_bounds__(512, 2)
    residual_norm_rows_kernel(const nvfp4_residual_norm_args a, const uint32_t per_group,
                              const int stages, int *err) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) uint64_t bars[kMaxStages];
    __shared__ __align__(16) float red[2][16];
    __shared__ int abort_flag;
    constexpr int V = kVecs;
    const int T = blockDim.x, tx = threadIdx.x, lane = tx & 31, warp = tx >> 5;
    const int nvec = static_cast<int>(a.cols) >> 3;
    // The first vector is always in the row.  Where the second is not, its place
    // holds the row's last one, made zero wherever it would count.
    const bool second = kFull || T + tx < nvec;
    const int place[V] = {tx, kFull ? T + tx : min(T + tx, nvec - 1)};
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    const uint32_t y_bytes = a.y != nullptr ? static_cast<uint32_t>(a.cols) * 2 : 0;
    const uint32_t slot_bytes = y_bytes + static_cast<uint32_t>(a.cols) * (kStreamF32 ? 4 : 2);
    const uint32_t ring_a = s32(ring), bar_a = s32(bars);
    const Abort ab{&abort_flag, err};
    const size_t vec_size = kVecF32 ? 4 : 2;
    if (tx == 0) {
        for (int s = 0; s < stages; ++s)
            bar_init(bar_a + 8 * s, 1);
        abort_flag = 0;
        bar_init_fence();
    }
    if (tx < 32) red[tx >> 4][tx & 15] = 0.0f;  // the entries past the last warp stay 0

    auto fetch = [&](int64_t r, int slot) __attribute__((always_inline)) {
        const uint32_t bar = bar_a + 8 * slot, dst = ring_a + slot * slot_bytes;
        bar_expect(bar, slot_bytes);
        if (y_bytes) bulk_load(dst, static_cast<const uint16_t *>(a.y) + r * a.y_stride, y_bytes, bar);
        bulk_load(dst + y_bytes,
                  static_cast<const uint8_t *>(a.residual) + r * a.residual_stride * (kStreamF32 ? 4 : 2),
                  slot_bytes - y_bytes, bar);
    };
    int turn = 0;
    // `v` is the warp's already.
    auto reduce_warps = [&](float v, auto op) __attribute__((always_inline)) {
        if (lane == 0) red[turn][warp] = v;
        __syncthreads();
        const float4 *b = reinterpret_cast<const float4 *>(red[turn]);
        turn ^= 1;
        const float4 u = b[0], w = b[1];
        v = op(op(op(u.x, u.y), op(u.z, u.w)), op(op(w.x, w.y), op(w.z, w.w)));
        if (T > 256) {
            const float4 y = b[2], z = b[3];
            v = op(v, op(op(op(y.x, y.y), op(y.z, y.w)), op(op(z.x, z.y), op(z.z, z.w))));
        }
        return v;
    };
    auto add = [](float u, float v) __attribute__((always_inline)) { return u + v; };
    auto sum = [&](float v) __attribute__((always_inline)) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        return reduce_warps(v, add);
    };
    auto larger = [](float u, float v) __attribute__((always_inline)) {
        return __uint_as_float(::max(__float_as_uint(u), __float_as_uint(v)));
    };
    auto only_in_row = [&](float2 (&v)[4]) __attribute__((always_inline)) {
        if (!kFull)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = make_float2(second ? v[j].x : 0.0f, second ? v[j].y : 0.0f);
    };
    // x <- x - mean for a layer norm; returns 1 / sqrt(mean(x^2) + eps).
    auto centred_inverse = [&](float2 (&x)[V][4], int kind, float eps) __attribute__((always_inline)) {
        if (kind == NVFP4_NORM_LAYER) {
            float2 s = both(0.0f);
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s = __fadd2_rn(s, x[i][j]);
            const float2 mean = both(-sum(s.x + s.y) * inv_cols);
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] = __fadd2_rn(x[i][j], mean);
            only_in_row(x[1]);
        }
        float2 s2 = both(0.0f);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s2 = __ffma2_rn(x[i][j], x[i][j], s2);
        return rsqrtf(fmaf(sum(s2.x + s2.y), inv_cols, eps));
    };
    auto group_of = [&](int64_t r) __attribute__((always_inline)) {
        return a.row_group != nullptr ? int64_t(__ldg(a.row_group + r))
                                      : int64_t(static_cast<uint32_t>(r) / per_group);
    };
    // x <- x * vector (or x + vector) where there is one.
    auto times = [&](float2 (&x)[V][4], const void *p) __attribute__((always_inline)) {
        if (p == nullptr) return;
        RawVec<kVecF32> raw[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            raw[i].load(p, place[i]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float2 f[4];
            raw[i].get(f);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i][j] = __fmul2_rn(x[i][j], f[j]);
        }
    };
    auto plus = [&](float2 (&x)[V][4], const void *p) __attribute__((always_inline)) {
        if (p == nullptr) return;
        RawVec<kVecF32> raw[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            raw[i].load(p, place[i]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float2 f[4];
            raw[i].get(f);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i][j] = __fadd2_rn(x[i][j], f[j]);
        }
    };

    const int64_t step = gridDim.x;
    int64_t r = blockIdx.x, issued = 0;  // issued: rows asked for (thread 0)
    if (tx == 0)
        for (; issued < stages && r + issued * step < a.rows; ++issued)
            fetch(r + issued * step, static_cast<int>(issued));
    __syncthreads();
    int64_t next = r < a.rows ? group_of(r) : -1;
    int slot = 0;
    uint32_t parity = 0;
    // This thread's first vector of the current row of h and out.
    uint8_t *hp = static_cast<uint8_t *>(a.h) + (r * a.h_stride + tx * 8) * (kStreamF32 ? 4 : 2);
    uint8_t *op = static_cast<uint8_t *>(a.out) + (r * a.out_stride + tx * 8) * 2;
    const int64_t h_step = step * a.h_stride * (kStreamF32 ? 4 : 2), o_step = step * a.out_stride * 2;
    // Of the codes; and the word of block scales that the thread may write (the
    // first vector's for an even one, the second's for an odd one), in row 0.
    uint8_t *qp = a.q + r * (a.cols >> 1) + tx * 4;
    const int64_t q_step = step * (a.cols >> 1), sf_step = ((a.cols + 63) >> 6) * 512;
    uint8_t *sf_word = a.sf + ((tx & 1 ? T + tx - 1 : tx) >> 3) * 512;
    for (; r < a.rows; r += step, hp += h_step, op += o_step, qp += q_step) {
        const int64_t group = next;
        if (r + step < a.rows) next = group_of(r + step);
        const bool live = group >= 0 && group < a.groups;
        // A wait that gives up says so, and the row is worked on with whatever the slot
        // holds, as are all later ones at once: the threads of the CTA stay together, and
        // the call ends with the error word set.
        bar_wait(bar_a + 8 * slot, parity, ab, kTimeoutTag);
        const uint32_t ys = ring_a + slot * slot_bytes, rs = ys + y_bytes;
        uint4 yv[V], rv[kStreamF32 ? 2 * V : V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            yv[i] = y_bytes ? ld_shared_16B(ys + place[i] * 16) : make_uint4(0, 0, 0, 0);
            if (kStreamF32) {
                rv[i] = ld_shared_16B(rs + place[i] * 32);
                rv[(kStreamF32 ? V : 0) + i] = ld_shared_16B(rs + place[i] * 32 + 16);
            } else {
                rv[i] = ld_shared_16B(rs + place[i] * 16);
            }
        }
        // The slot is free, and asked to hold a later row, once every thread has
        // read it: at the row's first reduction, or here where none comes.
        const bool abandoned = *static_cast<volatile int *>(&abort_flag);
        auto refill = [&]() __attribute__((always_inline)) {
            if (tx == 0 && r + stages * step < a.rows && !abandoned) {
                fetch(r + stages * step, slot);
                ++issued;
            }
        };
        if (!live || (a.post_norm == NVFP4_NORM_NONE && a.pre_norm == NVFP4_NORM_NONE)) {
            __syncthreads();
            refill();
        }
        if (live) {
            float2 x[V][4];
#pragma unroll
            for (int i = 0; i < V; ++i) unpack4(yv[i], x[i]);
            only_in_row(x[1]);
            if (a.post_norm != NVFP4_NORM_NONE) {
                const float2 inv = both(centred_inverse(x, a.post_norm, a.post_eps));
                refill();
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[i][j] = __fmul2_rn(x[i][j], inv);
                times(x, a.post_weight);
                plus(x, a.post_bias);
            }
            const float2 rscale = both(a.residual_scale);
            if (a.branch_scale != 1.0f) {
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[i][j] = __fmul2_rn(x[i][j], both(a.branch_scale));
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float2 res[4], gf[4];
                if (kStreamF32) {
                    const uint4 lo = rv[i], hi = rv[(kStreamF32 ? V : 0) + i];
                    res[0] = make_float2(__uint_as_float(lo.x), __uint_as_float(lo.y));
                    res[1] = make_float2(__uint_as_float(lo.z), __uint_as_float(lo.w));
                    res[2] = make_float2(__uint_as_float(hi.x), __uint_as_float(hi.y));
                    res[3] = make_float2(__uint_as_float(hi.z), __uint_as_float(hi.w));
                } else {
                    unpack4(rv[i], res);
                }
                if (a.gate != nullptr) {
                    RawVec<kVecF32> gate;
                    gate.load(static_cast<const uint8_t *>(a.gate) + group * a.gate_stride * vec_size, place[i]);
                    gate.get(gf);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[i][j] = __fmul2_rn(x[i][j], gf[j]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[i][j] = __ffma2_rn(rscale, res[j], x[i][j]);
                if (a.h != nullptr && (i == 0 || second)) {
                    if (kStreamF32) {
                        float4 *o = reinterpret_cast<float4 *>(hp + i * T * 32);
                        o[0] = make_float4(x[i][0].x, x[i][0].y, x[i][1].x, x[i][1].y);
                        o[1] = make_float4(x[i][2].x, x[i][2].y, x[i][3].x, x[i][3].y);
                    } else {
                        *reinterpret_cast<uint4 *>(hp + i * T * 16) = pack4(x[i]);
                    }
                }
            }
            only_in_row(x[1]);
            if (a.pre_norm != NVFP4_NORM_NONE) {
                const float2 inv = both(centred_inverse(x, a.pre_norm, a.pre_eps));
                if (a.post_norm == NVFP4_NORM_NONE) refill();
                const uint8_t *sp = static_cast<const uint8_t *>(a.scale) + group * a.scale_stride * vec_size;
                const uint8_t *tp = static_cast<const uint8_t *>(a.shift) + group * a.shift_stride * vec_size;
                if (a.pre_weight == nullptr && a.pre_bias == nullptr) {
                    // x * (inv + inv * scale) + shift
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        RawVec<kVecF32> s, t;
                        float2 f[4];
                        if (a.scale != nullptr) s.load(sp, place[i]);
                        if (a.shift != nullptr) t.load(tp, place[i]);
                        if (a.scale != nullptr) {
                            s.get(f);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                x[i][j] = __fmul2_rn(x[i][j], __ffma2_rn(f[j], inv, inv));
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j) x[i][j] = __fmul2_rn(x[i][j], inv);
                        }
                        if (a.shift != nullptr) {
                            t.get(f);
#pragma unroll
                            for (int j = 0; j < 4; ++j) x[i][j] = __fadd2_rn(x[i][j], f[j]);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[i][j] = __fmul2_rn(x[i][j], inv);
                    times(x, a.pre_weight);
                    plus(x, a.pre_bias);
                    if (a.scale != nullptr) {
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            RawVec<kVecF32> raw;
                            float2 f[4];
                            raw.load(sp, place[i]);
                            raw.get(f);
#pragma unroll
                            for (int j = 0; j < 4; ++j) x[i][j] = __ffma2_rn(x[i][j], f[j], x[i][j]);
                        }
                    }
                    if (a.shift != nullptr) plus(x, tp);
                }
                uint4 o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    o[i] = pack4(x[i]);
                    if (!kFull && i > 0 && !second) o[i] = make_uint4(0, 0, 0, 0);
                    if (a.out != nullptr && (i == 0 || second))
                        *reinterpret_cast<uint4 *>(op + i * T * 16) = o[i];
                }
                if (kQuant) {
                    const uint32_t m0 = absmax_bf16x8(o[0]), m1 = absmax_bf16x8(o[1]);
                    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, ::max(m0, m1));
                    const float amax = reduce_warps(__uint_as_float(m << 16), larger);
                    const float s_enc = tensor_encode_scale(amax);
                    if (tx == 0) {
                        a.s_dec_rows[r] = __fdiv_rn(1.0f, s_enc);
                        if (a.amax_rows != nullptr) a.amax_rows[r] = amax;
                    }
                    const uint32_t r32 = static_cast<uint32_t>(r);
                    uint8_t *sfp = sf_word + (r >> 7) * sf_step + (r32 & 31) * 16 + ((r32 >> 5) & 3) * 4;
                    quantize_two(qp, qp + T * 4, sfp, second, o[0], o[1], m0, m1, s_enc);
                }
            }
        }
        if (++slot == stages) {
            slot = 0;
            parity ^= 1;
        }
    }
    if (tx == 0 && *static_cast<volatile int *>(&abort_flag)) {  // copies still in flight
        const uint64_t deadline = timer_ns() + kBlockTimeoutNs;
        for (int64_t k = issued > stages ? issued - stages : 0; k < issued; ++k)
            bar_drain(bar_a + 8 * static_cast<int>(k % stages), (k / stages) & 1, deadline);
    }
    if (kQuant) {  // padding rows of the tiled scales
        const int64_t rows_pad = (a.rows + 127) & ~int64_t(127), kb4 = (a.cols + 63) >> 6;
        for (int64_t z = a.rows + blockIdx.x; z < rows_pad; z += step)
            for (int64_t c = tx; c < kb4; c += T)
                *reinterpret_cast<uint32_t *>(a.sf + sf_offset(z, 4 * c, kb4)) = 0u;
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

template <bool kFull, bool kQuant, bool kStreamF32, bool kVecF32>
cudaError_t launch_rows_as(const nvfp4_residual_norm_args &a, int num_sms, cudaStream_t stream) {
    auto *kernel = residual_norm_rows_kernel<kFull, kQuant, kStreamF32, kVecF32>;
    int *err = device_error_word();
    if (err == nullptr) return cudaErrorUnknown;
    const int threads = static_cast<int>((a.cols / 8 + kVecs - 1) / kVecs + 31) / 32 * 32;
    const int64_t slot = a.cols * ((a.y != nullptr ? 2 : 0) + (kStreamF32 ? 4 : 2));
    // 1024 threads per SM by registers, in at most 16 CTAs; kRingBytes of rows
    // in flight between them.
    int per_sm = 1024 / threads;
    if (per_sm > 16) per_sm = 16;
    int64_t stages = kRingBytes / per_sm / slot;
    stages = stages < 2 ? 2 : stages > kMaxStages ? kMaxStages : stages;
    const int smem = static_cast<int>(stages * slot);
    // The limit belongs to the kernel, whichever host thread sets it: once per device,
    // to the most that any width takes, or a call of narrow rows could lower it
    // between another thread's setting and launch.
    static std::atomic<int> configured[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev].load(std::memory_order_acquire)) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return e;
        configured[dev].store(1, std::memory_order_release);
    }
    const int64_t grid = static_cast<int64_t>(num_sms) * per_sm;
    kernel<<<static_cast<unsigned>(grid < a.rows ? grid : a.rows), threads, smem, stream>>>(
        a, static_cast<uint32_t>((a.rows + a.groups - 1) / a.groups), static_cast<int>(stages), err);
    return cudaGetLastError();
}

template <bool kFull, bool kQuant>
cudaError_t launch_rows_of(const nvfp4_residual_norm_args &a, int num_sms, cudaStream_t stream) {
    const bool v32 = a.vector_dtype == NVFP4_F32;
    if (a.stream_dtype == NVFP4_F32)
        return v32 ? launch_rows_as<kFull, kQuant, true, true>(a, num_sms, stream)
                   : launch_rows_as<kFull, kQuant, true, false>(a, num_sms, stream);
    return v32 ? launch_rows_as<kFull, kQuant, false, true>(a, num_sms, stream)
               : launch_rows_as<kFull, kQuant, false, false>(a, num_sms, stream);
}

cudaError_t launch_rows(const nvfp4_residual_norm_args &a, int num_sms, cudaStream_t stream) {
    // Whole warps of whole vectors need no bounds checks (4096 columns with / without
    // them: into codes 3.66 / 3.85 TB/s, fp32 vectors 4.2 / 4.8).
    if (a.cols % (32 * 8 * kVecs) == 0)
        return a.q != nullptr ? launch_rows_of<true, true>(a, num_sms, stream)
                              : launch_rows_of<true, false>(a, num_sms, stream);
    return a.q != nullptr ? launch_rows_of<false, true>(a, num_sms, stream)
                          : launch_rows_of<false, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_residual_norm(const nvfp4_residual_norm_args &a, int num_sms,
                                 cudaStream_t stream) {
    const int64_t c = a.cols;
    // The persistent form from 2^21 values on, and from a row per SM where a row
    // needs more than 512 threads of the other (us, layer norm with gate and
    // modulation, one CTA per row / persistent: 1200 x 1024 3.7 / 4.1, 2400 x 1024
    // 6.5 / 5.9; 600 x 2048 3.9 / 4.1, 1200 x 2048 6.6 / 6.0; 444 x 4096 5.0 / 5.1,
    // 8000 x 4096 64 / 46; 148 x 8192 4.6 / 4.4, 8000 x 8192 185 / 91).  Rows of 256
    // columns are a warp each.
    if (c > 256 && c <= 8192 && (c <= 4096 ? a.rows * c > (1 << 21) : a.rows > num_sms))
        return launch_rows(a, num_sms, stream);
    // One CTA per row, one vector per thread: the shortest chain.
    if (c <= 256) return launch<32, 1, 4>(a, stream);
    if (c <= 1024) return launch<128, 1, 1>(a, stream);
    if (c <= 2048) return launch<256, 1, 1>(a, stream);
    if (c <= 4096) return launch<512, 1, 1>(a, stream);
    if (c <= 8192) return launch<1024, 1, 1>(a, stream);
    if (c <= 16384) return launch<512, 4, 1>(a, stream);
    return launch<1024, 4, 1>(a, stream);
}

}  // namespace nvfp4
