// Low-rank adapters of many requests beside a projection.  Row m with adapter
// s = row_slot[m] (A[s]: rank x K, B[s]: N x rank, both bf16):
//   t      = scale[s] * A[s] x[m]          (fp32)
//   out[m] = bf16(y[m] + B[s] t)           (fp32, one rounding at the end)
// and out[m] = y[m] for a row whose slot is not in [0, slots).
//
// A cluster of CTAs per row.  Each CTA takes a slice of K for every rank (a
// warp per rank, so a row of A is read in whole lines), the partial sums go to
// every CTA of the cluster through distributed shared memory, and after one
// cluster barrier each CTA adds its slice of N.  B's slice is asked into L2 as
// soon as A has arrived, behind the reductions and the barrier; asked for before
// A it delays A, which everything waits for (61 rows, rank 32, K 4096, N 12288:
// 18.8 us against 16.5; behind A's loads, before they arrive, 17.6).
// What bounds it: the adapters' bytes, rank * (K + N) * 2 per row, from HBM
// where rows have adapters of their own and from L2 where they share them.
// Measured: one row, rank 16, 4096 x 4096 3.5 us; 61 rows with 61 adapters of rank
// 32, K 4096, N 12288 14.9 us (67 MB, 4.5 TB/s: 7 us until A is summed up, then B at
// 6.9 TB/s).
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

// A load that is issued where it stands.
__device__ __forceinline__ uint4 ld_nc_16B(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
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

// Rank 16 * R16.  In the second product L lanes share an output's row of B, V
// 16-byte pieces each, so that a warp reads whole lines; a batch is 32 outputs
// of a warp, and U batches are in flight at a time.
template <int R16>
__global__ void __launch_bounds__(kRowThreads, R16 <= 2 ? 4 : R16 == 4 ? 3 : 2) __cluster_dims__(kCluster, 1, 1)
    lora_rows_kernel(const nvfp4_lora_args p, const int *crowded) {
    constexpr int rank = 16 * R16;
    constexpr int L = R16 == 8 ? 16 : R16 == 4 ? 8 : R16 % 2 == 0 ? 4 : 2;
    constexpr int V = rank / 8 / L;
    constexpr int U = rank <= 16 ? 4 : rank <= 48 ? 2 : 1;
    __shared__ __align__(16) float part[kCluster][rank];
    __shared__ __align__(16) float t[rank];
    const int64_t row = blockIdx.x / kCluster;
    const int c = static_cast<int>(blockIdx.x % kCluster);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // Beside the tile kernels: only the rows of the tiles they left out.
    if (crowded != nullptr && __ldg(crowded + (row >> 7)) == 0) return;
    const uint16_t *yrow = static_cast<const uint16_t *>(p.y) + row * p.y_stride;
    uint16_t *orow = static_cast<uint16_t *>(p.out) + row * p.out_stride;
    // This CTA's outputs.
    const int64_t n0 = (p.n >> 3) * c / kCluster * 8, n1 = (p.n >> 3) * (c + 1) / kCluster * 8;
    const int64_t slot = p.row_slot != nullptr ? int64_t(__ldg(p.row_slot + row)) : 0;
    if (slot < 0 || slot >= p.slots) {  // the same in every CTA of the cluster
        if (p.out != p.y)
            for (int64_t n = n0 + 8 * threadIdx.x; n < n1; n += 8 * kRowThreads)
                *reinterpret_cast<uint4 *>(orow + n) = *reinterpret_cast<const uint4 *>(yrow + n);
        return;
    }
    cluster_arrive();  // this CTA runs: its shared memory may be written
    const uint16_t *a = static_cast<const uint16_t *>(p.a) + slot * rank * p.k;
    const uint8_t *b = static_cast<const uint8_t *>(p.b) + slot * p.n * (rank * 2);

    // t's partial sums over this CTA's slice of K, up to four ranks of a warp
    // at a time.
    const int64_t nk = p.k >> 3;
    const int64_t k0 = nk * c / kCluster, k1 = nk * (c + 1) / kCluster;
    const uint4 *xrow =
        reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.x) + row * p.x_stride);
    constexpr int kRanks = rank / kRowWarps;  // of a warp: warp, warp + 8, ...
#pragma unroll 1
    for (int i0 = 0; i0 < kRanks; i0 += 4) {
        constexpr int G = kRanks < 4 ? kRanks : 4;
        float s[G];
#pragma unroll
        for (int i = 0; i < G; ++i) s[i] = 0.0f;
        for (int64_t k = k0 + lane; k < k1; k += 64) {
            // Two steps' loads together.
            uint4 xv[2], v[2][G];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = k + 32 * h < k1;
                xv[h] = in ? ld_nc_16B(xrow + k + 32 * h) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < G; ++i)
                    v[h][i] = in && i0 + i < kRanks
                                  ? ld_nc_16B(reinterpret_cast<const uint4 *>(
                                                  a + (warp + (i0 + i) * kRowWarps) * p.k) +
                                              k + 32 * h)
                                  : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < G; ++i) s[i] = dot8(xv[h], v[h][i], s[i]);
        }
        if (i0 + 4 >= kRanks)  // A is here: HBM's next work, behind the reductions and the barrier
            for (int64_t o = n0 * (rank * 2) + threadIdx.x * 128; o < n1 * (rank * 2); o += kRowThreads * 128)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(b + o), "f"(s[0]));
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s[i] += __shfl_xor_sync(0xFFFFFFFFu, s[i], o);
        if (i0 == 0) cluster_wait();
        if (lane < kCluster)
#pragma unroll
            for (int i = 0; i < G; ++i)
                if (i0 + i < kRanks) st_cluster_f32(&part[c][warp + (i0 + i) * kRowWarps], lane, s[i]);
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

    const int l = lane % L, group = lane / L;
    float tv[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) tv[v][j] = t[(v * L + l) * 8 + j];
    for (int64_t base = n0 + warp * (32 * U); base < n1; base += kRowWarps * 32 * U) {
        uint4 bv[U][L][V];
        uint16_t yv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const int64_t n = base + u * 32 + j * (32 / L) + group;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (n < n1)
                        bv[u][j][v] = __ldg(reinterpret_cast<const uint4 *>(b + n * (rank * 2)) + v * L + l);
            }
            const int64_t n = base + u * 32 + l * (32 / L) + group;
            if (n < n1) yv[u] = yrow[n];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float acc[L];
#pragma unroll
            for (int j = 0; j < L; ++j) {
                acc[j] = 0.0f;
#pragma unroll
                for (int v = 0; v < V; ++v) acc[j] = dot8(tv[v], bv[u][j][v], acc[j]);
            }
            // The L lanes' sums meet, each lane keeping the output of its number.
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
                for (int j = 0; j < o; ++j) {
                    const bool upper = l & o;
                    const float other = __shfl_xor_sync(0xFFFFFFFFu, upper ? acc[j] : acc[j + o], o);
                    acc[j] = (upper ? acc[j + o] : acc[j]) + other;
                }
            const int64_t n = base + u * 32 + l * (32 / L) + group;
            if (n < n1)
                orow[n] = __bfloat16_as_ushort(
                    __float2bfloat16_rn(__uint_as_float(static_cast<uint32_t>(yv[u]) << 16) + acc[0]));
        }
    }
}

template <int R16>
cudaError_t launch_rows_as(const nvfp4_lora_args &p, const int *crowded, cudaStream_t stream) {
    lora_rows_kernel<R16><<<static_cast<unsigned>(p.rows * kCluster), kRowThreads, 0, stream>>>(p, crowded);
    return cudaGetLastError();
}

cudaError_t launch_rows(const nvfp4_lora_args &p, const int *crowded, cudaStream_t stream) {
    switch (p.rank / 16) {
        case 1: return launch_rows_as<1>(p, crowded, stream);
        case 2: return launch_rows_as<2>(p, crowded, stream);
        case 3: return launch_rows_as<3>(p, crowded, stream);
        case 4: return launch_rows_as<4>(p, crowded, stream);
        case 5: return launch_rows_as<5>(p, crowded, stream);
        case 6: return launch_rows_as<6>(p, crowded, stream);
        case 7: return launch_rows_as<7>(p, crowded, stream);
        default: return launch_rows_as<8>(p, crowded, stream);
    }
}

// Whether a cluster per row is taken (us measured with it / on tiles, K = 4096):
//   rows x rank x (K + N) up to 2^25    rank 16, 64 rows, N 12288: 8.1 / 11.3;
//     128 rows: 14.3 / 11.5 with one adapter, 14.3 / 15.1 with four;
//     rank 64, 32 rows, N 12288: 11.2 / 12.9, 64 rows: 24.4 / 13.0
//   up to 2^26 where many adapters are held: a tile's cost grows with the
//     adapters among its rows (rank 16, 128 rows with one each: 15.5 / 163),
//     which the host cannot see
//   at most 256 rows: each is a cluster, whatever its size.
bool by_rows(int64_t rows, int64_t k, int64_t n, int64_t rank, bool many_adapters) {
    return rows <= 256 && rows * rank * (k + n) <= (int64_t(1) << (many_adapters ? 26 : 25));
}

}  // namespace

size_t lora_workspace_bytes(int64_t rows, int64_t k, int64_t n, int64_t rank) {
    return by_rows(rows, k, n, rank, false) ? 0 : lora_tile_workspace_bytes(rows, rank);
}

cudaError_t launch_lora(const nvfp4_lora_args &p, cudaStream_t stream) {
    if (by_rows(p.rows, p.k, p.n, p.rank, p.slots > 8)) return launch_rows(p, nullptr, stream);
    // A tile of D adapters costs about as much as D / 10 tiles row by row (us, 128
    // rows with an adapter each, by rows / on a tile: rank 16 10 / 158, rank 64
    // 30 / 276, rank 128 56 / 488), and tiles run side by side: up to 12 of them,
    // those with more than ten adapters for each tile of the call go row by row.
    const int64_t tiles = (p.rows + 127) / 128;
    const int most = static_cast<int>(10 * tiles < 128 ? 10 * tiles : 128);
    const int *crowded = nullptr;
    const cudaError_t e = launch_lora_tile(p, most, &crowded, stream);
    if (e != cudaSuccess || most == 128 || p.slots <= most) return e;
    return launch_rows(p, crowded, stream);
}

}  // namespace nvfp4
