// Low-rank adapters of many requests beside a projection.  Row m with adapter
// s = row_slot[m] (A[s]: rank x K, B[s]: N x rank, both bf16):
//   t      = scale[s] * A[s] x[m]          (fp32)
//   out[m] = bf16(y[m] + B[s] t)           (fp32, one rounding at the end)
// and out[m] = y[m] for a row whose slot is not in [0, slots).
//
// A cluster of CTAs per row.  Each CTA takes a slice of K for every rank (a
// warp per rank, so a row of A is read in whole lines), the partial sums go to
// every CTA of the cluster through distributed shared memory, and after one
// cluster barrier each CTA adds its slice of N: two outputs per thread, whose
// rows of B are one contiguous piece.  B's slice is asked into L2 before the
// first product, so its latency passes behind it.
// What bounds it: the adapters' bytes, rank * (K + N) * 2 per row, from HBM
// where rows have adapters of their own and from L2 where they share them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "block_ops.h"
#include "nvfp4_math.cuh"

namespace nvfp4 {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kCluster = 8;
constexpr int kMaxRank = 128;

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// Stores v at the address of `p` in CTA `rank` of the cluster.
__device__ __forceinline__ void st_cluster_f32(float *p, uint32_t rank, float v) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %0, %1;\n\t"
        "st.shared::cluster.f32 [a], %2;\n\t}\n" ::"r"(smem_u32(p)),
        "r"(rank), "f"(v)
        : "memory");
}

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// acc + a . b over eight bf16 pairs, in order.
__device__ __forceinline__ float dot8(uint4 a, uint4 b, float acc) {
    acc = fmaf(bf16_lo(a.x), bf16_lo(b.x), acc);
    acc = fmaf(bf16_hi(a.x), bf16_hi(b.x), acc);
    acc = fmaf(bf16_lo(a.y), bf16_lo(b.y), acc);
    acc = fmaf(bf16_hi(a.y), bf16_hi(b.y), acc);
    acc = fmaf(bf16_lo(a.z), bf16_lo(b.z), acc);
    acc = fmaf(bf16_hi(a.z), bf16_hi(b.z), acc);
    acc = fmaf(bf16_lo(a.w), bf16_lo(b.w), acc);
    return fmaf(bf16_hi(a.w), bf16_hi(b.w), acc);
}

// acc + t . b over eight values.
__device__ __forceinline__ float dot8(const float *t, uint4 b, float acc) {
    acc = fmaf(t[0], bf16_lo(b.x), acc);
    acc = fmaf(t[1], bf16_hi(b.x), acc);
    acc = fmaf(t[2], bf16_lo(b.y), acc);
    acc = fmaf(t[3], bf16_hi(b.y), acc);
    acc = fmaf(t[4], bf16_lo(b.z), acc);
    acc = fmaf(t[5], bf16_hi(b.z), acc);
    acc = fmaf(t[6], bf16_lo(b.w), acc);
    return fmaf(t[7], bf16_hi(b.w), acc);
}

__global__ void __launch_bounds__(kRowThreads) __cluster_dims__(kCluster, 1, 1)
    lora_rows_kernel(const nvfp4_lora_args p) {
    __shared__ __align__(16) float part[kCluster][kMaxRank];
    __shared__ __align__(16) float t[kMaxRank];
    const int64_t row = blockIdx.x / kCluster;
    const int c = static_cast<int>(blockIdx.x % kCluster);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(p.rank);
    const uint32_t *yrow =
        reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p.y) + row * p.y_stride);
    uint32_t *orow = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) + row * p.out_stride);
    // This CTA's pairs of outputs.
    const int64_t pairs = p.n >> 1;
    const int64_t p0 = pairs * c / kCluster, p1 = pairs * (c + 1) / kCluster;
    const int64_t slot = p.row_slot != nullptr ? int64_t(__ldg(p.row_slot + row)) : 0;
    if (slot < 0 || slot >= p.slots) {  // the same in every CTA of the cluster
        if (p.out != p.y)
            for (int64_t i = p0 + threadIdx.x; i < p1; i += kRowThreads) orow[i] = yrow[i];
        return;
    }
    cluster_arrive();  // this CTA runs: its shared memory may be written
    const uint16_t *a = static_cast<const uint16_t *>(p.a) + slot * rank * p.k;
    const uint8_t *b = static_cast<const uint8_t *>(p.b) + slot * p.n * rank * 2;
    const int64_t pair_bytes = 4 * int64_t(rank);
    for (int64_t o = p0 * pair_bytes + threadIdx.x * 128; o < p1 * pair_bytes; o += kRowThreads * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(b + o));

    // t's partial sums over this CTA's slice of K.
    const int64_t nk = p.k >> 3;
    const int64_t k0 = nk * c / kCluster, k1 = nk * (c + 1) / kCluster;
    const uint4 *xrow =
        reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.x) + row * p.x_stride);
    bool peers_run = false;
    for (int r = warp; r < rank; r += 2 * kRowWarps) {  // two ranks of a warp at a time
        const uint4 *a0 = reinterpret_cast<const uint4 *>(a + r * p.k);
        const uint4 *a1 = reinterpret_cast<const uint4 *>(a + (r + kRowWarps) * p.k);
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 2
        for (int64_t k = k0 + lane; k < k1; k += 32) {
            const uint4 xv = __ldg(xrow + k);
            const uint4 v0 = __ldg(a0 + k), v1 = __ldg(a1 + k);
            s0 = dot8(xv, v0, s0);
            s1 = dot8(xv, v1, s1);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s0 += __shfl_xor_sync(0xFFFFFFFFu, s0, o);
            s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, o);
        }
        if (!peers_run) {
            cluster_wait();
            peers_run = true;
        }
        if (lane < kCluster) {
            st_cluster_f32(&part[c][r], lane, s0);
            st_cluster_f32(&part[c][r + kRowWarps], lane, s1);
        }
    }
    cluster_arrive();
    cluster_wait();
    if (threadIdx.x < rank) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kCluster; ++i) s += part[i][threadIdx.x];
        t[threadIdx.x] = s * __ldg(p.scale + slot);
    }
    __syncthreads();

    const int vecs = rank >> 3;
    for (int64_t i = p0 + threadIdx.x; i < p1; i += kRowThreads) {
        const uint4 *b0 = reinterpret_cast<const uint4 *>(b + i * pair_bytes);
        const uint4 *b1 = b0 + vecs;
        float lo = 0.0f, hi = 0.0f;
#pragma unroll 4
        for (int v = 0; v < vecs; ++v) {
            lo = dot8(t + 8 * v, __ldg(b0 + v), lo);
            hi = dot8(t + 8 * v, __ldg(b1 + v), hi);
        }
        const uint32_t yv = yrow[i];
        const __nv_bfloat162 o = __floats2bfloat162_rn(bf16_lo(yv) + lo, bf16_hi(yv) + hi);
        orow[i] = *reinterpret_cast<const uint32_t *>(&o);
    }
}

}  // namespace

// Rows from which the tiles are taken.
constexpr int64_t kTileFromRows = 97;

size_t lora_workspace_bytes(int64_t rows, int64_t k, int64_t n, int64_t rank) {
    (void)n;
    return rows < kTileFromRows ? 0 : lora_tile_workspace_bytes(rows, k, rank);
}

cudaError_t launch_lora(const nvfp4_lora_args &p, cudaStream_t stream) {
    if (p.rows >= kTileFromRows) return launch_lora_tile(p, stream);
    lora_rows_kernel<<<static_cast<unsigned>(p.rows * kCluster), kRowThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace nvfp4
