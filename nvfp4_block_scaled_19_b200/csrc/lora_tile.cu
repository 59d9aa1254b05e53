// Low-rank adapters for many rows (the mathematics is stated in lora.cu): two
// launches on 128-row tiles, both tcgen05 with TMA-fed shared memory.
//
// lora_shrink_kernel   t[m] = scale[s] * A[s] x[m].
//   A cluster of `splits` CTAs per row tile, each over its share of K (where there
//   are few tiles, several clusters, each for a part of the tile's adapters).  A stage
//   is the tile's 128 x 64 piece of x and, side by side as one B operand, the
//   matching rank x 64 pieces of up to G = 256 / rank different adapters, so a
//   tile whose rows belong to G requests still reads x once; each row's
//   epilogue thread keeps its own adapter's columns.  The splits' fp32 sums meet
//   through distributed shared memory (in the workspace where a tile has more
//   adapters than a pass takes, as the ring is then still in use): after a
//   cluster barrier each CTA adds up its share of the rows, in the order of the
//   splits, so the result does not depend on timing.
//   t is written as the sum of two bf16 (hi + lo, 16 mantissa bits, see split_t), as
//   the expand's MMA takes it.
// lora_expand_kernel   out[m][n] = bf16(y[m][n] + B[s] t[m]).
//   A CTA keeps t of its row tile in shared memory and walks over units of 64
//   columns: y by TMA into a ring, B's 64 x rank piece by TMA, the product in
//   tensor memory (two MMAs per 16 ranks, for hi and lo, so that it keeps nearly
//   fp32 accuracy while B, which is bf16 already, needs no second copy), added
//   to y in place in the ring, out by TMA.  A tile with rows of several adapters
//   makes one product per adapter, each row taking its own adapter's: nothing of
//   another adapter, not even NaN, reaches a row.  The launch overlaps the
//   shrink's (programmatic dependence): only t waits for it.
//
// What bounds them: HBM (x once; y and out once).  Rank 128 is 64 flops per byte
// of x, above what the register-operand MMAs sustain beside the loads and far
// below tcgen05's rate.  Measured, both launches: 16896 rows, rank 16, K 4096, N
// 12288 176 us (0.97 GB, 5.5 TB/s; 35 us of it the shrink, which shares HBM with
// the write-back of what ran before); 4608 rows, rank 128, K 12288, N 4096, three
// adapters 61 us (40 and 21); 1337 rows of six requests, rank 64, 5120 x 5120
// 24 us, most of it start-up, sums over the cluster and tiles of two or three
// requests.
//
// Roles of both: the first and last warp TMA producers (x or y; the adapters:
// a copy costs the thread that issues it a few hundred cycles), warp 1 MMA
// issuer, the warps between epilogue (one 32-lane quadrant each; in the expand
// two to a quadrant, for half a unit's columns each).  Every wait is bounded; on a
// timeout the kernel records NVFP4_ERR_TIMEOUT (tags 40-47), all roles stop,
// copies and MMAs in flight are drained with bounded waits and tensor memory is
// freed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "api_checks.h"
#include "block_ops.h"
#include "block_waits.cuh"
#include "gemm.h"
#include "nvfp4_math.cuh"

namespace nvfp4 {
namespace {

constexpr int kTileRows = 128;
constexpr int kThreads = 224;
constexpr uint32_t kXBytes = kTileRows * 128;  // 128 rows x 64 bf16
constexpr int kMaxSplits = 8;  // CTAs of a shrink cluster, over K

// ---------------------------------------------------------------- PTX

__device__ __forceinline__ void load_2d(const CUtensorMap *m, uint32_t bar, uint32_t dst, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

__device__ __forceinline__ void prefetch_2d(const CUtensorMap *m, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(m), "r"(x),
                 "r"(y)
                 : "memory");
}

__device__ __forceinline__ void store_2d(const CUtensorMap *m, uint32_t src, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(m),
        "r"(src), "r"(x), "r"(y)
        : "memory");
}

__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
    // K-major, 128-byte swizzle: 8-row groups of 1024 bytes.
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFF) | (1ull << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// kind::f16 with bf16 operands, both K-major, fp32 accumulator.
__device__ __forceinline__ uint32_t bf16_idesc(int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(kTileRows >> 4) << 24);
}

__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ void fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

template <int k>
__device__ __forceinline__ void tmem_ld16_part(uint32_t addr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[k]), "=r"(r[k + 1]), "=r"(r[k + 2]), "=r"(r[k + 3]), "=r"(r[k + 4]), "=r"(r[k + 5]),
          "=r"(r[k + 6]), "=r"(r[k + 7]), "=r"(r[k + 8]), "=r"(r[k + 9]), "=r"(r[k + 10]),
          "=r"(r[k + 11]), "=r"(r[k + 12]), "=r"(r[k + 13]), "=r"(r[k + 14]), "=r"(r[k + 15])
        : "r"(addr + k)
        : "memory");
}

// The first min(n16, 4) x 16 columns of this warp's 32 lanes, complete on return.
__device__ __forceinline__ void tmem_ld_up_to_64(uint32_t addr, uint32_t (&r)[64], int n16) {
    tmem_ld16_part<0>(addr, r);
    if (n16 > 1) tmem_ld16_part<16>(addr, r);
    if (n16 > 2) tmem_ld16_part<32>(addr, r);
    if (n16 > 3) tmem_ld16_part<48>(addr, r);
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    // No use of the values moves above the wait.
#pragma unroll
    for (int i = 0; i < 64; ++i) asm volatile("" : "+r"(r[i]));
}

// 64 or 32 columns of this warp's 32 lanes, complete on return.
__device__ __forceinline__ void tmem_ld_cols(uint32_t addr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_ld_cols(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}

// The pair of bf16 in w plus two fp32 values, rounded once.
__device__ __forceinline__ uint32_t add_pair(uint32_t w, uint32_t lo, uint32_t hi) {
    const __nv_bfloat162 o =
        __floats2bfloat162_rn(bf16_lo(w) + __uint_as_float(lo), bf16_hi(w) + __uint_as_float(hi));
    return *reinterpret_cast<const uint32_t *>(&o);
}

__device__ __forceinline__ void st_shared_16B(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

// 16 bytes at this CTA's shared address `a`, of CTA `rank` of the cluster.
__device__ __forceinline__ float4 ld_cluster_16B(uint32_t a, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .b32 r;\n\t"
        "mapa.shared::cluster.u32 r, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [r];\n\t}\n"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(a), "r"(rank)
        : "memory");
    return v;
}

// ---------------------------------------------------------------- the tile's adapters

struct alignas(16) TileSlots {
    int row[kTileRows];       // each row's adapter, as its place in `list`, or -1
    int list[kTileRows];      // the different adapters, in order of first use
    int count;
    int warp_count[4];
};

// Fills `ts` for rows [m0, m0 + 128) (all threads call; ends with a barrier).
__device__ __forceinline__ void find_slots(TileSlots &ts, const nvfp4_lora_args &p, int64_t m0) {
    const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
    int slot = -1;
    if (i < kTileRows) {
        if (m0 + i < p.rows) {
            slot = p.row_slot != nullptr ? __ldg(p.row_slot + m0 + i) : 0;
            if (slot < 0 || slot >= p.slots) slot = -1;
        }
        ts.row[i] = slot;
    }
    __syncthreads();
    bool first = false;
    unsigned firsts = 0;
    if (i < kTileRows) {
        const unsigned same = __match_any_sync(0xFFFFFFFFu, slot);
        first = slot >= 0 && lane == __ffs(same) - 1;
        if (first) {  // and in no earlier warp
            const int4 *rows = reinterpret_cast<const int4 *>(ts.row);
            bool seen = false;
#pragma unroll 8
            for (int j = 0; j < 8 * warp; ++j) {
                const int4 v = rows[j];
                seen |= v.x == slot || v.y == slot || v.z == slot || v.w == slot;
            }
            first = !seen;
        }
        __syncwarp();
        firsts = __ballot_sync(0xFFFFFFFFu, first);
        if (lane == 0) ts.warp_count[warp] = __popc(firsts);
    }
    __syncthreads();
    if (i < kTileRows) {
        int at = __popc(firsts & ((1u << lane) - 1u));
        for (int w = 0; w < warp; ++w) at += ts.warp_count[w];
        if (first) ts.list[at] = slot;
        if (i == 0) ts.count = ts.warp_count[0] + ts.warp_count[1] + ts.warp_count[2] + ts.warp_count[3];
    }
    __syncthreads();
    if (i < kTileRows && slot >= 0) {
        int d = 0;
        while (ts.list[d] != slot) ++d;  // it is in the list
        ts.row[i] = d;
    }
    __syncthreads();
}

// How t is laid out for a rank: rows of 64-element (128-byte) groups, hi's
// groups first, then lo's; up to rank 32 both share one group, lo from its
// 32nd element on.
struct TLayout {
    int groups;     // 128-byte groups of a row
    int lo_at;      // element where lo starts
    __host__ __device__ explicit TLayout(int rank)
        : groups(rank <= 32 ? 1 : rank <= 64 ? 2 : 4), lo_at(rank <= 32 ? 32 : groups * 32) {}
};

// t as the sum of two bf16 values (returned in fp32).  Both have t's sign and
// neither is zero unless t is (from |t| = 2^-110 on), so that an infinity in B makes
// two infinities of one sign, as t itself would: hi is t cut off, not rounded, to 8
// bits, lo the rest rounded to 8 (off by 2^-16 of t at most); a t of no more than 8
// bits is halved, and one that is not finite stands in both.
__device__ __forceinline__ void split_t(float t, float &hi, float &lo) {
    hi = __uint_as_float(__float_as_uint(t) & 0xFFFF0000u);
    lo = t - hi;
    if (!isfinite(t)) {
        hi = lo = t;
    } else if (lo == 0.0f && fabsf(hi) >= 2.3509887e-38f /* 2^-125: halves are exact */) {
        hi = lo = 0.5f * hi;
    }
}

// Eight values of t as hi and lo, 16 bytes each.
__device__ __forceinline__ void store_t8(const float *t, uint16_t *hi_dst, uint16_t *lo_dst) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float h0, l0, h1, l1;
        split_t(t[2 * j], h0, l0);
        split_t(t[2 * j + 1], h1, l1);
        const __nv_bfloat162 h = __floats2bfloat162_rn(h0, h1), l = __floats2bfloat162_rn(l0, l1);
        hi[j] = *reinterpret_cast<const uint32_t *>(&h);
        lo[j] = *reinterpret_cast<const uint32_t *>(&l);
    }
    *reinterpret_cast<uint4 *>(hi_dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4 *>(lo_dst) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

struct alignas(64) ShrinkMaps {
    CUtensorMap x, a;
};

struct alignas(64) ExpandMaps {
    CUtensorMap y, b, out, t;
};

// ---------------------------------------------------------------- shrink

constexpr int kAccCols = 256;  // tensor memory of a CTA of either kernel: two fit an SM

// Two rings, of x's 128 x 64 pieces and of the adapters' pieces of a pass, with
// as many slots as fit for the tile's adapters.  What bounds the stream of x is
// bytes in flight: a box of 128 rows takes about 2 us from HBM, so 96 KB of x in
// flight are worth 48 GB/s of an SM.  192 KB where a CTA has its SM alone, else
// 96 KB and two CTAs per SM.
constexpr uint32_t kLargeRings = 192 * 1024, kSmallRings = 96 * 1024;
constexpr int kMaxSlots = 8;

__global__ void __launch_bounds__(kThreads)
    lora_shrink_kernel(const __grid_constant__ ShrinkMaps maps, const nvfp4_lora_args p,
                       const int splits, const int parts, const uint32_t ring_bytes,
                       const int most_adapters, int *crowded, float *partial, uint16_t *t, int *err) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ TileSlots ts;
    __shared__ float scales[kTileRows];
    __shared__ __align__(8) uint64_t bars[2 * kMaxSlots + 3];
    __shared__ uint32_t tmem_holder;
    __shared__ int abort_flag;
    const uint32_t x_ring = (s32(smem_raw) + 1023u) & ~1023u;
    const uint32_t full = s32(bars), empty = full + 8 * kMaxSlots;  // of both rings' slots
    const uint32_t acc_full = empty + 8 * kMaxSlots, acc_empty = acc_full + 8, drain = acc_empty + 8;
    const Abort ab{&abort_flag, err};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = blockIdx.x / (splits * parts), split = blockIdx.x % splits;
    const int part = blockIdx.x / splits % parts;
    const int64_t m0 = int64_t(tile) * kTileRows;
    const int rank = static_cast<int>(p.rank);
    const int k_blocks = static_cast<int>((p.k + 63) / 64);
    const int kb0 = static_cast<int>(int64_t(k_blocks) * split / splits);
    const int kbs = static_cast<int>(int64_t(k_blocks) * (split + 1) / splits) - kb0;
    // Pieces of x asked for before the tile's adapters are known: the slots that
    // there are with the most adapters of a pass (32 KB a slot).
    const int early = min(static_cast<int>(ring_bytes / (kXBytes + 32 * 1024)), kbs);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxSlots; ++s) {
            bar_init(full + 8 * s, 2);  // the two producers
            bar_init(empty + 8 * s, 1);
        }
        bar_init(acc_full, 1);
        bar_init(acc_empty, 4);
        bar_init(drain, 1);
        abort_flag = 0;
        bar_init_fence();
        for (int i = 0; i < early; ++i) {
            bar_expect(full + 8 * i, kXBytes);
            load_2d(&maps.x, full + 8 * i, x_ring + i * kXBytes, (kb0 + i) * 64, static_cast<int>(m0));
        }
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         s32(&tmem_holder)),
                     "r"(kAccCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        fence_before();
    }
    find_slots(ts, p, m0);
    fence_after();
    // The expand may start its prologue once every CTA here holds its tensor memory.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = tmem_holder;
    // A crowded tile is left to the kernel of single rows.
    const int all = ts.count <= most_adapters ? ts.count : 0;
    if (split == 0 && part == 0 && threadIdx.x == 64) crowded[tile] = ts.count > most_adapters;
    const int begin = all * part / parts, end = all * (part + 1) / parts;  // this cluster's adapters
    const int count = end - begin;
    const int group = max(1, min(kAccCols / rank, count));  // adapters per pass over x
    const int passes = (count + group - 1) / group;          // 0: no row has an adapter
    const uint32_t a_slot = group * rank * 128;              // at most 32 KB
    const int slots = min(kMaxSlots, static_cast<int>(ring_bytes / (kXBytes + a_slot)));
    const uint32_t a_ring = x_ring + slots * kXBytes;
    const int steps = passes * kbs;

    if (warp == 0) {
        if (lane == 0) {
            int slot = early % slots, issued = early;
            uint32_t phase = early == slots ? 1 : 0;
            bool ok = passes > 0;
            // A ring shortened by wide adapters keeps too little of x in flight:
            // L2 then fetches what the full ring would hold.
            const int ahead = splits > 1 ? kMaxSlots : 0;
            for (int i = early; i < steps && ok; ++i) {
                if (!bar_wait(empty + 8 * slot, phase ^ 1, ab, 40)) {
                    ok = false;
                    break;
                }
                bar_expect(full + 8 * slot, kXBytes);
                load_2d(&maps.x, full + 8 * slot, x_ring + slot * kXBytes, (kb0 + i % kbs) * 64,
                        static_cast<int>(m0));
                if (ahead > slots && i + ahead - slots < kbs)
                    prefetch_2d(&maps.x, (kb0 + i + ahead - slots) * 64, static_cast<int>(m0));
                if (issued < slots) ++issued;
                if (++slot == slots) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            if (!ok) {  // given up, or nothing to multiply: the copies in flight land first
                const uint64_t deadline = timer_ns() + kBlockTimeoutNs;
                if (passes == 0)
                    for (int i = 0; i < early; ++i) bar_arrive(full + 8 * i);  // the other producer's part
                for (int i = 0; i < issued; ++i) {
                    if (--slot < 0) {
                        slot = slots - 1;
                        phase ^= 1;
                    }
                    bar_drain(full + 8 * slot, phase, deadline);
                }
            }
        }
    } else if (warp == 6) {
        if (lane == 0) {
            int slot = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int q = 0; q < passes && ok; ++q) {
                const int d0 = begin + q * group, d1 = min(end, d0 + group);
                for (int kb = kb0; kb < kb0 + kbs; ++kb) {
                    if (!bar_wait(empty + 8 * slot, phase ^ 1, ab, 40)) {
                        ok = false;
                        break;
                    }
                    bar_expect(full + 8 * slot, (d1 - d0) * rank * 128);
                    for (int d = d0; d < d1; ++d)
                        load_2d(&maps.a, full + 8 * slot, a_ring + slot * a_slot + (d - d0) * rank * 128,
                                kb * 64, ts.list[d] * rank);
                    if (issued < slots) ++issued;
                    if (++slot == slots) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok) {
                const uint64_t deadline = timer_ns() + kBlockTimeoutNs;
                for (int i = 0; i < issued; ++i) {
                    if (--slot < 0) {
                        slot = slots - 1;
                        phase ^= 1;
                    }
                    bar_drain(full + 8 * slot, phase, deadline);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int slot = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int q = 0; q < passes && ok; ++q) {
                const int d0 = begin + q * group, d1 = min(end, d0 + group);
                const uint32_t idesc = bf16_idesc((d1 - d0) * rank);
                if (!bar_wait(acc_empty, (q & 1) ^ 1, ab, 41)) break;
                fence_after();
                for (int kb = 0; kb < kbs; ++kb) {
                    if (!bar_wait(full + 8 * slot, phase, ab, 42)) {
                        ok = false;
                        break;
                    }
                    fence_after();
                    const uint64_t a = operand_desc(x_ring + slot * kXBytes);
                    const uint64_t b = operand_desc(a_ring + slot * a_slot);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_bf16(tmem, a + 2 * j, b + 2 * j, idesc, (kb > 0 || j > 0) ? 1u : 0u);
                    mma_commit(empty + 8 * slot);
                    if (++slot == slots) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                if (ok) mma_commit(acc_full);
            }
            mma_commit(drain);
        }
        __syncwarp();
    } else {
        const int quad = warp & 3, row = quad * 32 + lane;
        const int mine = ts.row[row];
        const TLayout tl(rank);
        float *dst = partial + (int64_t(split) * p.rows + m0 + row) * rank;
        uint16_t *tdst = t + (m0 + row) * (tl.groups * 64);
        if (row < all) scales[row] = __ldg(p.scale + ts.list[row]);
        const float c = mine >= 0 ? __ldg(p.scale + ts.list[mine]) : 0.0f;
        for (int q = 0; q < passes; ++q) {
            const int d0 = begin + q * group, d1 = min(end, d0 + group);
            if (!bar_wait_warp(acc_full, q & 1, ab, 43)) break;
            fence_after();
            const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16);
            for (int d = d0; d < d1; ++d) {
                if (!__any_sync(0xFFFFFFFFu, mine == d)) continue;  // none of this warp's rows
                for (int r0 = 0; r0 < rank; r0 += 64) {
                    uint32_t f[64];
                    tmem_ld_up_to_64(acc + (d - d0) * rank + r0, f, (rank - r0) >> 4);
                    if (mine == d) {  // never a row past the last one
#pragma unroll
                        for (int h = 0; h < 64; h += 8) {
                            const int r = r0 + h;
                            if (r >= rank) break;
                            if (splits == 1) {
                                float v[8];
#pragma unroll
                                for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(f[h + j]) * c;
                                store_t8(v, tdst + r, tdst + tl.lo_at + r);
                            } else if (passes == 1) {  // x's ring is free: all of it has been multiplied
                                const uint32_t at = x_ring + ((r >> 2) * kTileRows + row) * 16;
                                st_shared_16B(at, make_uint4(f[h], f[h + 1], f[h + 2], f[h + 3]));
                                st_shared_16B(at + kTileRows * 16,
                                              make_uint4(f[h + 4], f[h + 5], f[h + 6], f[h + 7]));
                            } else {
                                uint4 *o = reinterpret_cast<uint4 *>(dst + r);
                                o[0] = make_uint4(f[h], f[h + 1], f[h + 2], f[h + 3]);
                                o[1] = make_uint4(f[h + 4], f[h + 5], f[h + 6], f[h + 7]);
                            }
                        }
                    }
                    __syncwarp();
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(acc_empty);
        }
    }
    if (splits == 1) {
        __syncthreads();
    } else {
        // Every split's sums are written: this CTA's share of the rows, eight
        // ranks per thread at a time, in the order of the splits.
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                         : "memory");
        const TLayout tl(rank);
        const int share = (kTileRows + splits - 1) / splits;
        for (int i = threadIdx.x; i < share * (rank >> 3); i += kThreads) {
            const int row = split * share + i % share, r = i / share * 8;
            const int d = row < kTileRows && passes > 0 ? ts.row[row] : -1;
            if (d < begin || d >= end) continue;
            float4 w[kMaxSplits][2];  // asked for together
            if (passes == 1) {
                const uint32_t at = x_ring + ((r >> 2) * kTileRows + row) * 16;
#pragma unroll
                for (int s = 0; s < kMaxSplits; ++s)
                    if (s < splits) {
                        w[s][0] = ld_cluster_16B(at, s);
                        w[s][1] = ld_cluster_16B(at + kTileRows * 16, s);
                    }
            } else {
                const float *src = partial + (m0 + row) * rank + r;
#pragma unroll
                for (int s = 0; s < kMaxSplits; ++s)
                    if (s < splits) {
                        const float4 *o = reinterpret_cast<const float4 *>(src + s * p.rows * rank);
                        w[s][0] = o[0];
                        w[s][1] = o[1];
                    }
            }
            float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < kMaxSplits; ++s)
                if (s < splits) {
                    v[0] += w[s][0].x; v[1] += w[s][0].y; v[2] += w[s][0].z; v[3] += w[s][0].w;
                    v[4] += w[s][1].x; v[5] += w[s][1].y; v[6] += w[s][1].z; v[7] += w[s][1].w;
                }
            const float c = scales[d];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= c;
            uint16_t *o = t + (m0 + row) * (tl.groups * 64) + r;
            store_t8(v, o, o + tl.lo_at);
        }
        // No CTA of the cluster leaves while another reads its shared memory.
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                         : "memory");
    }
    if (warp == 1) {
        if (lane == 0) bar_drain(drain, 0, timer_ns() + kBlockTimeoutNs);  // every MMA has completed
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kAccCols)
                     : "memory");
    }
}

// ---------------------------------------------------------------- expand

// Shared-memory plan of an expand launch, from the rank.  Up to rank 64 two CTAs
// fit an SM (104 KB each) on units of 64 columns; above, t alone is 64 KB, and
// one CTA takes units of 128: an MMA of 64 columns costs the tensor core about
// as much as one of 128.
struct ExpandPlan {
    int y_slots, b_slots;     // ring depths
    uint32_t b_bytes;         // a unit's B: `unit` rows x (64 ranks x chunks)
    uint32_t lo_offset;       // bytes from t's hi part to its lo part
    uint32_t t_bytes;
    int chunks;               // 64-rank chunks
    uint32_t smem_bytes;
};

constexpr int kMaxYSlots = 4, kMaxBSlots = 3;
constexpr uint32_t kBoxBytes = kTileRows * 128;  // 128 rows x 64 columns

constexpr int kUnitsPerCta = 32;

int expand_unit(int64_t rank) { return rank <= 64 ? 64 : 128; }

constexpr int kExpandEpiWarps = 8;
constexpr int kExpandThreads = 32 * (3 + kExpandEpiWarps);

ExpandPlan expand_plan(int64_t rank) {
    const TLayout tl(static_cast<int>(rank));
    const int unit = expand_unit(rank);
    ExpandPlan e;
    e.chunks = rank > 64 ? 2 : 1;
    e.b_bytes = e.chunks * unit * 128;
    e.lo_offset = rank <= 32 ? 64 : tl.groups / 2 * kBoxBytes;
    e.t_bytes = tl.groups * kBoxBytes;
    e.y_slots = rank <= 32 ? 4 : 3;
    e.b_slots = rank <= 64 ? 3 : 2;
    e.smem_bytes = e.t_bytes + e.y_slots * (unit / 64 * kBoxBytes) + e.b_slots * e.b_bytes + 1024;
    return e;
}

// The launch's units, row tile by row tile, are dealt out evenly: each CTA takes
// a run of them, parts of one or a few tiles.  Where there are few tiles the
// shares are weighed, as a tile with rows of several adapters takes longer: a
// unit costs 10 with one adapter and 7 more for each other (1.6 and 2.7 us
// measured).  Weighing takes about 2 us before a CTA's first copies: with 8 units
// per CTA it pays (4608 rows, rank 128, three adapters 63.7 -> 61.7 us), with 3 it
// does not (1337 rows of six requests 26.6 -> 28.6).
constexpr int kWeighedTiles = 128, kWeighedUnits = 6;

// The tiles' costs, and where two places in their sum are.
struct Shares {
    int prefix[kWeighedTiles + 1];  // unit costs of the tiles before each
    long long first, last;          // this CTA's units, counted through the tiles
};

// Fills `sh` for CTA i of n (all threads call; ends with a barrier).  A tile's cost
// goes by its different adapters, in whatever order its rows have them; one that
// is left to the kernel of single rows (more than most_adapters) costs nothing
// here.  A unit of tile t starts at units * prefix[t] and its unit cost apart; a
// CTA's units are those that start in its n-th of the sum.
__device__ __forceinline__ void share_out(Shares &sh, const nvfp4_lora_args &p, int tiles, int units,
                                          int most_adapters, unsigned i, unsigned n) {
    constexpr int kBatch = 4;  // tiles of a warp at a time, their slots loaded together
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int t0 = threadIdx.x >> 5; t0 < tiles; t0 += kBatch * warps) {
        int slot[kBatch][4];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t row = int64_t(t0 + b * warps) * kTileRows + 32 * q + lane;
                const int s = row < p.rows ? __ldg(p.row_slot + row) : -1;
                slot[b][q] = s >= 0 && s < p.slots ? s : -1;
            }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            // One adapter after the other is counted and struck out of every lane.
            const int t = t0 + b * warps;
            int count = 0;
            while (count <= most_adapters) {
                const int next = __reduce_max_sync(
                    0xFFFFFFFFu, max(max(slot[b][0], slot[b][1]), max(slot[b][2], slot[b][3])));
                if (next < 0) break;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (slot[b][q] == next) slot[b][q] = -1;
                ++count;
            }
            if (lane == 0 && t < tiles)
                sh.prefix[t + 1] = count > most_adapters ? 0 : count > 0 ? 3 + 7 * count : p.out == p.y ? 0 : 8;
        }
    }
    __syncthreads();
    if (threadIdx.x < 32) {  // four tiles per lane
        int c[4], sum = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int t = 4 * lane + k;
            sum += t < tiles ? sh.prefix[t + 1] : 0;
            c[k] = sum;
        }
        int upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += v;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (4 * lane + k < tiles) sh.prefix[4 * lane + k + 1] = upto - sum + c[k];
        if (lane == 0) {
            sh.prefix[0] = 0;
            sh.first = sh.last = static_cast<long long>(tiles) * units;  // unless found below
        }
    }
    __syncthreads();
    const int t = threadIdx.x;
    if (t < tiles) {
        const int64_t all = int64_t(units) * sh.prefix[tiles], begin = int64_t(units) * sh.prefix[t];
        const int cost = sh.prefix[t + 1] - sh.prefix[t];
        const int64_t end = begin + int64_t(units) * cost;
        const int64_t at0 = all * i / n, at1 = all * (i + 1) / n;
        if (begin <= at0 && at0 < end) sh.first = int64_t(t) * units + (at0 - begin + cost - 1) / cost;
        if (begin <= at1 && at1 < end) sh.last = int64_t(t) * units + (at1 - begin + cost - 1) / cost;
    }
    __syncthreads();
}

template <int kUnit, bool kWeighed>
__global__ void __launch_bounds__(kExpandThreads, kUnit == 64 ? 2 : 1)
    lora_expand_kernel(const __grid_constant__ ExpandMaps maps, const nvfp4_lora_args p,
                       const ExpandPlan plan, const int most_adapters, int *err) {
    constexpr uint32_t kYBytes = kUnit / 64 * kBoxBytes;
    constexpr int kAccs = kAccCols / kUnit;
    constexpr int kEpiWarps = kExpandEpiWarps;
    constexpr int kCols = 4 * kUnit / kEpiWarps;  // columns of an epilogue warp: 32 or 64
    constexpr int kBWarp = 2 + kEpiWarps;         // loads B
    extern __shared__ uint8_t smem_raw[];
    __shared__ TileSlots ts;
    __shared__ __align__(8) uint64_t bars[2 * kMaxYSlots + 2 * kMaxBSlots + 2 * kAccs + 2];
    __shared__ uint32_t tmem_holder;
    __shared__ int abort_flag;
    const uint32_t t_base = (s32(smem_raw) + 1023u) & ~1023u;
    const uint32_t y_ring = t_base + plan.t_bytes, b_ring = y_ring + plan.y_slots * kYBytes;
    const uint32_t y_full = s32(bars), y_empty = y_full + 8 * kMaxYSlots;
    const uint32_t b_full = y_empty + 8 * kMaxYSlots, b_empty = b_full + 8 * kMaxBSlots;
    const uint32_t d_full = b_empty + 8 * kMaxBSlots, d_empty = d_full + 8 * kAccs;
    const uint32_t t_full = d_empty + 8 * kAccs, drain = t_full + 8;
    const Abort ab{&abort_flag, err};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(p.rank);
    const int units = static_cast<int>((p.n + kUnit - 1) / kUnit);  // of a row tile
    const int64_t tiles = (p.rows + kTileRows - 1) / kTileRows, total = tiles * units;

    if (threadIdx.x == 0) {
        for (int s = 0; s < plan.y_slots; ++s) {
            bar_init(y_full + 8 * s, 1);
            bar_init(y_empty + 8 * s, kUnit / 16);  // the stores of a unit
        }
        for (int s = 0; s < plan.b_slots; ++s) {
            bar_init(b_full + 8 * s, 1);
            bar_init(b_empty + 8 * s, 1);
        }
        for (int s = 0; s < kAccs; ++s) {
            bar_init(d_full + 8 * s, 1);
            bar_init(d_empty + 8 * s, kEpiWarps);
        }
        bar_init(t_full, 1);
        bar_init(drain, 1);
        abort_flag = 0;
        bar_init_fence();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         s32(&tmem_holder)),
                     "r"(kAccCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_holder;

    int64_t g0 = total * blockIdx.x / gridDim.x, g1 = total * (blockIdx.x + 1) / gridDim.x;
    if (kWeighed) {
        __shared__ Shares shares;
        share_out(shares, p, static_cast<int>(tiles), units, most_adapters, blockIdx.x, gridDim.x);
        g0 = shares.first;
        g1 = shares.last;
    }

    // Ring positions, of whichever role the thread has; they go on from tile
    // to tile.
    int ys = 0, bs = 0, acc = 0, y_issued = 0, b_issued = 0, prev = -1;
    uint32_t yph = 0, bph = 0, aph = 0, tph = 0;
    bool waited = false, t_issued = false;

    for (int64_t g = g0; g < g1;) {
        const int64_t tile = g / units;
        const int u0 = static_cast<int>(g - tile * units);
        const int u1 = static_cast<int>(min(g1 - tile * units, int64_t(units)));
        const int64_t m0 = tile * kTileRows;
        g += u1 - u0;
        find_slots(ts, p, m0);  // begins after every role's end of the last tile, see below
        const int count = ts.count;
        if (count == 0 && p.out == p.y) continue;  // nothing to add and nothing to copy
        if (count > most_adapters) continue;       // left to the kernel of single rows

        if (warp == 0) {
            if (lane == 0)
                for (int u = u0; u < u1; ++u) {
                    if (!bar_wait(y_empty + 8 * ys, yph ^ 1, ab, 44)) break;
                    bar_expect(y_full + 8 * ys, kYBytes);
#pragma unroll
                    for (int h = 0; h < kUnit; h += 64)
                        load_2d(&maps.y, y_full + 8 * ys, y_ring + ys * kYBytes + h * (kTileRows * 2),
                                u * kUnit + h, static_cast<int>(m0));
                    if (y_issued < plan.y_slots) ++y_issued;
                    if (++ys == plan.y_slots) {
                        ys = 0;
                        yph ^= 1;
                    }
                }
        } else if (warp == kBWarp) {
            if (lane == 0) {
                bool ok = true;
                for (int u = u0; u < u1 && ok; ++u)
                    for (int d = 0; d < count; ++d) {
                        if (!bar_wait(b_empty + 8 * bs, bph ^ 1, ab, 45)) {
                            ok = false;
                            break;
                        }
                        bar_expect(b_full + 8 * bs, plan.b_bytes);
                        const int row = static_cast<int>(ts.list[d] * p.n + u * kUnit);
                        for (int c = 0; c < plan.chunks; ++c)
                            load_2d(&maps.b, b_full + 8 * bs, b_ring + bs * plan.b_bytes + c * (kUnit * 128),
                                    c * 64, row);
                        if (b_issued < plan.b_slots) ++b_issued;
                        if (++bs == plan.b_slots) {
                            bs = 0;
                            bph ^= 1;
                        }
                    }
            }
        } else if (warp == 1) {
            if (lane == 0 && count > 0) {
                // t, the one thing here that waits for the shrink.
                if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
                waited = true;
                bar_expect(t_full, plan.t_bytes);
                for (uint32_t o = 0; o < plan.t_bytes; o += kBoxBytes)
                    load_2d(&maps.t, t_full, t_base + o, static_cast<int>(o / (kTileRows * 2)),
                            static_cast<int>(m0));
                t_issued = true;
                constexpr uint32_t n_field = static_cast<uint32_t>(kUnit >> 3) << 17;
                const uint32_t idesc = bf16_idesc(0) | n_field;
                int64_t left = int64_t(u1 - u0) * count;
                if (!bar_wait(t_full, tph, ab, 46)) left = 0;
                if (left > 0) {
                    tph ^= 1;
                    t_issued = false;  // landed
                }
                for (; left > 0; --left) {
                    if (!bar_wait(b_full + 8 * bs, bph, ab, 46)) break;
                    if (!bar_wait(d_empty + 8 * acc, aph ^ 1, ab, 46)) break;
                    fence_after();
                    const uint32_t d = tmem + acc * kUnit;
                    for (int r = 0; r < rank; r += 16) {
                        const uint32_t chunk = r >> 6, in = (r & 63) * 2;
                        const uint64_t hi = operand_desc(t_base + chunk * kBoxBytes + in);
                        const uint64_t b = operand_desc(b_ring + bs * plan.b_bytes + chunk * (kUnit * 128) + in);
                        mma_bf16(d, hi, b, idesc, r > 0 ? 1u : 0u);
                        mma_bf16(d, hi + (plan.lo_offset >> 4), b, idesc, 1u);
                    }
                    mma_commit(b_empty + 8 * bs);
                    mma_commit(d_full + 8 * acc);
                    if (++bs == plan.b_slots) {
                        bs = 0;
                        bph ^= 1;
                    }
                    if (++acc == kAccs) {
                        acc = 0;
                        aph ^= 1;
                    }
                }
            }
            __syncwarp();
        } else {
            const int quad = warp & 3, row = quad * 32 + lane, first = (warp - 2) / 4 * kCols;
            const int h = first & ~63;  // the 64-column box of its columns
            const bool storer = (first & 63) == 0;
            const int mine = ts.row[row];
            const uint32_t swz = (row & 7) << 4;
            const uint32_t col_bytes = (first & 63) * 2;
            const bool stored = m0 + quad * 32 < p.rows;  // a box of this warp's rows
            bool ok = true;
            for (int u = u0; u < u1; ++u) {
                if (!bar_wait_warp(y_full + 8 * ys, yph, ab, 47)) {
                    ok = false;
                    break;
                }
                const uint32_t box = y_ring + ys * kYBytes + h * (kTileRows * 2);
                for (int d = 0; d < count; ++d) {
                    if (!bar_wait_warp(d_full + 8 * acc, aph, ab, 47)) {
                        ok = false;
                        break;
                    }
                    fence_after();
                    const uint32_t src = tmem + acc * kUnit + (static_cast<uint32_t>(quad * 32) << 16);
                    const bool any = count == 1 || __any_sync(0xFFFFFFFFu, mine == d);  // rows of it
                    uint32_t f[kCols];
                    if (any) tmem_ld_cols(src + first, f);
                    fence_before();  // read: back to the MMA thread
                    __syncwarp();
                    if (lane == 0) bar_arrive(d_empty + 8 * acc);
                    if (mine == d) {
#pragma unroll
                        for (int c = 0; c < kCols / 8; ++c) {
                            const uint32_t at = box + row * 128 + ((col_bytes + 16 * c) ^ swz);
                            uint4 v = ld_shared_16B(at);
                            v.x = add_pair(v.x, f[8 * c], f[8 * c + 1]);
                            v.y = add_pair(v.y, f[8 * c + 2], f[8 * c + 3]);
                            v.z = add_pair(v.z, f[8 * c + 4], f[8 * c + 5]);
                            v.w = add_pair(v.w, f[8 * c + 6], f[8 * c + 7]);
                            st_shared_16B(at, v);
                        }
                    }
                    __syncwarp();
                    if (++acc == kAccs) {
                        acc = 0;
                        aph ^= 1;
                    }
                }
                if (!ok) break;
                // A box of 32 rows and 64 columns goes out, by the warp of its first
                // columns; the slot of the unit before is free once its store has
                // read it.
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                if (kCols == 32) {
                    // The two warps of a box meet.  One that gives up says so first
                    // and arrives below, so the other is not left waiting.
                    if (__shfl_sync(0xFFFFFFFFu, *ab.flag, 0)) {
                        ok = false;
                        break;
                    }
                    asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory");
                } else {
                    __syncwarp();
                }
                if (lane == 0 && storer) {
                    if (stored && u * kUnit + h < p.n)
                        store_2d(&maps.out, box + quad * 4096, u * kUnit + h, static_cast<int>(m0) + quad * 32);
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                    if (prev >= 0) bar_arrive(y_empty + 8 * prev);
                }
                prev = ys;
                if (++ys == plan.y_slots) {
                    ys = 0;
                    yph ^= 1;
                }
            }
            if (kCols == 32 && !ok) asm volatile("bar.arrive %0, 64;" ::"r"(1 + quad) : "memory");
        }
        // Every role is done with this tile (its t, its adapters), and every
        // product of it has been read.
        __syncthreads();
        if (abort_flag) break;
    }

    if (lane == 0 && abort_flag) {  // copies still in flight
        const uint64_t deadline = timer_ns() + kBlockTimeoutNs;
        for (int i = 0; i < y_issued; ++i) {
            if (--ys < 0) {
                ys = plan.y_slots - 1;
                yph ^= 1;
            }
            bar_drain(y_full + 8 * ys, yph, deadline);
        }
        for (int i = 0; i < b_issued; ++i) {
            if (--bs < 0) {
                bs = plan.b_slots - 1;
                bph ^= 1;
            }
            bar_drain(b_full + 8 * bs, bph, deadline);
        }
    }
    if (warp >= 2 && warp < kBWarp && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");  // this grid never ends before the shrink
    if (warp == 1) {
        if (lane == 0) {  // every MMA, and t's copies, have completed
            const uint64_t deadline = timer_ns() + kBlockTimeoutNs;
            mma_commit(drain);
            bar_drain(drain, 0, deadline);
            if (abort_flag && t_issued) bar_drain(t_full, tph, deadline);
        }
        __syncwarp();
    }
    __syncthreads();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kAccCols)
                     : "memory");
}

// ---------------------------------------------------------------- host

// [rows, cols] bf16 with `stride` elements from row to row, boxes of 64
// columns (128 bytes, swizzled) x box_rows rows.
bool encode_map(CUtensorMap *m, const void *base, int64_t cols, int64_t rows, int64_t stride,
                uint32_t box_rows) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (enc == nullptr) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
    cuuint32_t box[2] = {64, box_rows};
    cuuint32_t one[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box,
               one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kSms = 148;  // a B200's; another count would cost speed, not results

int64_t row_tiles(int64_t rows) { return (rows + kTileRows - 1) / kTileRows; }

// (`bytes` is the same in every call for a kernel: an expand of 64-column units
// takes 105 KB at any rank, one of 128 225 KB.)
template <class K>
cudaError_t allow_smem(K kernel, uint32_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(bytes));
}

cudaLaunchConfig_t shrink_config(int64_t clusters, int splits, uint32_t rings, cudaLaunchAttribute *attr,
                                 cudaStream_t stream) {
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = static_cast<unsigned>(splits);
    attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = rings + 1024;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// How many clusters of `splits` CTAs run at once on the current device, one CTA
// per SM.  (Not the SMs divided by the size: a cluster stays inside a group of
// SMs, so larger ones leave some idle.)  Asked once; atomic, as host threads may
// make their first calls at the same time.
int clusters_at_once(int splits) {
    static std::atomic<int> known[64][kMaxSplits + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = known[dev][splits].load(std::memory_order_relaxed);
    if (n == 0) {
        cudaLaunchAttribute attr;
        const cudaLaunchConfig_t cfg = shrink_config(1, splits, kLargeRings, &attr, nullptr);
        if (cudaOccupancyMaxActiveClusters(&n, lora_shrink_kernel, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        known[dev][splits].store(n > 0 ? n : -1, std::memory_order_relaxed);
    }
    return n > 0 ? n : 0;
}

// CTAs of a shrink cluster: the most of which every row tile's cluster runs at
// once with one CTA per SM, and each has 4 blocks of 64 at least.  (Of 36
// clusters of 4 the last waited for the first to end, which doubled the time.)
int shrink_splits(int64_t rows, int64_t k) {
    const int64_t tiles = row_tiles(rows), blocks = (k + 63) / 64;
    if (2 * tiles > kSms) return 1;
    for (int s = kMaxSplits; s > 1; --s)
        if (blocks / s >= 4 && tiles * s <= kSms && tiles <= clusters_at_once(s)) return s;
    return 1;
}

// Clusters of a row tile, each for a part of its adapters: as many as there can be
// adapters and as all run at once, since one cluster draws only so much of the
// adapters (us, one part / as many: 252 rows with 20 adapters of rank 48 62 / 38;
// 92 rows with 6 of rank 112 33 / 21; 714 rows with 1 to 5 of rank 32 a tile 30.7 /
// 31.3).  Only as many as passes over x saved 1 to 2 us less.
int shrink_parts(int64_t tiles, int splits, int64_t slots) {
    if (splits == 1) return 1;
    const int64_t most = clusters_at_once(splits) / tiles, useful = slots < kTileRows ? slots : kTileRows;
    return static_cast<int>(most < 1 ? 1 : most < useful ? most : useful);
}

template <int kUnit>
cudaError_t launch_expand(const ExpandMaps &maps, const nvfp4_lora_args &p, const ExpandPlan &plan,
                          int64_t at_once, int most_adapters, int *err, cudaStream_t stream) {
    const int64_t tiles = row_tiles(p.rows), units = tiles * ((p.n + kUnit - 1) / kUnit);
    const int64_t chunks = units / kUnitsPerCta;
    const int64_t grid = units < at_once ? units : chunks > at_once ? chunks : at_once;
    const bool weighed = tiles <= kWeighedTiles && units >= kWeighedUnits * grid && p.row_slot != nullptr;
    auto *kernel = weighed ? lora_expand_kernel<kUnit, true> : lora_expand_kernel<kUnit, false>;
    const cudaError_t e = allow_smem(kernel, plan.smem_bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kExpandThreads);
    cfg.dynamicSmemBytes = plan.smem_bytes;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, maps, p, plan, most_adapters, err);
}

// Room for every split's fp32 sums: splits times the row tiles are at most an SM
// each, whatever the device makes of the split.
size_t partial_bytes(int64_t rows, int64_t rank) {
    const int64_t tiles = row_tiles(rows), most = kMaxSplits < kSms / tiles ? kMaxSplits : kSms / tiles;
    return most <= 1 ? 0 : static_cast<size_t>(most * rows * rank) * sizeof(float);
}

size_t flag_bytes(int64_t rows) { return static_cast<size_t>((row_tiles(rows) + 3) / 4) * 16; }

}  // namespace

// The waits of these kernels and of the residual norm's, each by a warp of its own
// on a barrier of which one of two arrivals comes; all return after the limit.
__global__ void selftest_block_waits_kernel(uint64_t timeout_ns, int tag, int *err) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int flags[2];
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        bar_init(s32(&bar), 2);
        flags[0] = flags[1] = 0;
        bar_init_fence();
    }
    __syncthreads();
    if (threadIdx.x == 0) bar_arrive(s32(&bar));
    __syncwarp();
    const uint64_t t0 = timer_ns();
    bool completed = false;
    if (warp == 0) {
        if (threadIdx.x == 0) completed = bar_wait(s32(&bar), 0, Abort{&flags[0], err, timeout_ns}, tag);
    } else if (warp == 1) {
        completed = bar_wait_warp(s32(&bar), 0, Abort{&flags[1], err, timeout_ns}, tag);
    } else {
        if (threadIdx.x == 64) bar_drain(s32(&bar), 0, t0 + timeout_ns);
    }
    __syncthreads();
    // Given up, said so to the CTA, and not before the limit.
    if (completed || (threadIdx.x == 0 && (flags[0] == 0 || flags[1] == 0 || timer_ns() - t0 < timeout_ns)))
        err[1] = tag + 1;
}

cudaError_t launch_selftest_block_waits(uint64_t timeout_ns, int tag, cudaStream_t stream) {
    int *err = device_error_word();
    if (err == nullptr) return cudaErrorUnknown;
    selftest_block_waits_kernel<<<1, 96, 0, stream>>>(timeout_ns, tag, err);
    return cudaGetLastError();
}

size_t lora_tile_workspace_bytes(int64_t rows, int64_t rank) {
    const TLayout tl(static_cast<int>(rank));
    return partial_bytes(rows, rank) + static_cast<size_t>(rows) * static_cast<size_t>(tl.groups) * 128 +
           flag_bytes(rows);
}

cudaError_t launch_lora_tile(const nvfp4_lora_args &p, int most_adapters, const int **crowded_out,
                             cudaStream_t stream) {
    int *err = device_error_word();
    if (err == nullptr) return cudaErrorUnknown;
    const TLayout tl(static_cast<int>(p.rank));
    float *partial = static_cast<float *>(p.workspace);
    uint16_t *t = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(p.workspace) +
                                               partial_bytes(p.rows, p.rank));
    int *crowded = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(t) +
                                           static_cast<size_t>(p.rows) * tl.groups * 128);
    *crowded_out = crowded;
    const ExpandPlan plan = expand_plan(p.rank);
    ShrinkMaps sm;
    ExpandMaps em;
    std::memset(&sm, 0, sizeof(sm));
    std::memset(&em, 0, sizeof(em));
    if (!encode_map(&sm.x, p.x, p.k, p.rows, p.x_stride, kTileRows) ||
        !encode_map(&sm.a, p.a, p.k, p.slots * p.rank, p.k, static_cast<uint32_t>(p.rank)) ||
        !encode_map(&em.y, p.y, p.n, p.rows, p.y_stride, kTileRows) ||
        !encode_map(&em.b, p.b, p.rank, p.slots * p.n, p.rank, static_cast<uint32_t>(expand_unit(p.rank))) ||
        !encode_map(&em.out, p.out, p.n, p.rows, p.out_stride, 32) ||
        !encode_map(&em.t, t, tl.groups * 64, p.rows, tl.groups * 64, kTileRows))
        return cudaErrorInvalidValue;
    cudaError_t e = allow_smem(lora_shrink_kernel, kLargeRings + 1024);
    if (e != cudaSuccess) return e;
    const int splits = shrink_splits(p.rows, p.k);
    const int64_t tiles = row_tiles(p.rows);
    const int parts = shrink_parts(tiles, splits, p.slots);
    const uint32_t rings = tiles * splits <= kSms ? kLargeRings : kSmallRings;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = shrink_config(tiles * parts, splits, rings, &attr, stream);
    e = cudaLaunchKernelEx(&cfg, lora_shrink_kernel, sm, p, splits, parts, rings, most_adapters, crowded, partial,
                           t, err);
    if (e != cudaSuccess) return e;
    return expand_unit(p.rank) == 64 ? launch_expand<64>(em, p, plan, 2 * kSms, most_adapters, err, stream)
                                     : launch_expand<128>(em, p, plan, kSms, most_adapters, err, stream);
}

}  // namespace nvfp4
