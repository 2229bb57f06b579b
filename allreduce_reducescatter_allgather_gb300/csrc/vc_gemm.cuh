// The product kernel of the training-step operators: D = A B on the tcgen05
// tensor cores, 16-bit operands (bf16 or fp16), 32-bit accumulators, with the
// operator's own arithmetic in the epilogue.
//
// One persistent kernel: a block (or a pair of blocks that share one 256-row
// product) walks over the output tiles.  Its warps have roles:
//   warp 0     loads the tiles of A and B through TMA into a ring of shared
//              memory stages (64 deep along K, 128-byte swizzle);
//   warp 1     issues the matrix instructions, which accumulate in tensor
//              memory (two accumulators, so that the next tile's products
//              run while this tile's epilogue reads);
//   the others read the accumulators and run the epilogue.  Each warp owns 32 rows (a warp
//              may only read the tensor-memory lanes of its quarter) and one
//              half of the columns; a 32 x 32 chunk goes through shared
//              memory so that global accesses run along the rows.
// Every wait is bounded: a wait that runs out marks the block as dead, which
// ends all of its loops, and counts it in a device word that the host can read.
//
// Either operand may be stored with K contiguous (K-major) or with M or N
// contiguous (MN-major): the matrix instruction takes both, so no operand is
// ever transposed in memory.  Sizes need not be multiples of anything: TMA
// fills what lies outside with zeros and the epilogue masks its accesses.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace vc {
namespace gemm {

constexpr int kBlockK = 64;            // 64 16-bit values: one 128-byte swizzle row
constexpr int kRowsPerCta = 128;       // tensor-memory lanes
constexpr int kStageRow = 36;          // floats per row of an epilogue chunk (32 + 4: no bank
                                       // conflicts in either direction)
constexpr int kEpilogueWarps = 8;
constexpr int kGemmThreads = 32 * (2 + kEpilogueWarps);
constexpr long long kWaitCycles = 4000000000ll;  // about two seconds

struct Shape {
    int M, N, K;            // of one product
    int batch;
    int tiles_m, tiles_n;   // tiles of one product (tiles_m counts block-pair tiles in pair mode)
    int tiles;              // tiles of one product that are computed
    int kblocks;            // ceil(K / 64)
    int group;              // tile rows walked together, for reuse in L2
    int a_mn, b_mn;         // operand is MN-major
    unsigned idesc;         // instruction descriptor
    unsigned* timeouts;     // counts blocks whose waits ran out
};

// ------------------------------------------------------------------ PTX --

__device__ __forceinline__ unsigned smem_u32(const void* p) {
    return (unsigned)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}

// The address, in the cluster's shared window, of block `rank`'s copy of `addr`.
__device__ __forceinline__ unsigned map_rank(unsigned addr, unsigned rank) {
    unsigned r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void mbar_init(unsigned bar, unsigned count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_expect(unsigned bar, unsigned bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

// Arrives on a barrier of any block of the cluster (a map_rank address).
__device__ __forceinline__ void mbar_arrive_cluster(unsigned bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
                 : "memory");
}

__device__ __forceinline__ bool mbar_try(unsigned bar, unsigned parity) {
    unsigned ok;
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Waits for the barrier's phase; false when the block is dead or the wait
// has run out (and the block is dead from then on).
__device__ __forceinline__ bool mbar_wait(unsigned bar, unsigned parity, volatile int* dead) {
    if (mbar_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try(bar, parity)) {
        if (*dead) return false;
        if (clock64() - t0 > kWaitCycles) {
            *dead = 1;
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// One box into this block's shared memory; `bar` may lie in the pair's
// leading block.
template <int kPair>
__device__ __forceinline__ void tma_load(unsigned dst, const CUtensorMap* map, unsigned bar, int x,
                                         int y, int z) {
    if constexpr (kPair == 2) {
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
            ".cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
            "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
            : "memory");
    } else {
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
            "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
            : "memory");
    }
}

template <int kPair>
__device__ __forceinline__ void tmem_alloc(unsigned where, int cols) {
    if constexpr (kPair == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(where),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(where),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}

template <int kPair>
__device__ __forceinline__ void tmem_free(unsigned tmem, int cols) {
    if constexpr (kPair == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols)
                     : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols)
                     : "memory");
}

template <int kPair>
__device__ __forceinline__ void mma_f16(unsigned d, uint64_t a, uint64_t b, unsigned idesc,
                                        bool add) {
    if constexpr (kPair == 2)
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((unsigned)add)
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((unsigned)add)
            : "memory");
}

// Arrives on `bar` (in pair mode on both blocks' barriers) once every matrix
// instruction issued so far has completed.
template <int kPair>
__device__ __forceinline__ void mma_commit(unsigned bar) {
    if constexpr (kPair == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
            ".multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"((unsigned short)3)
            : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
            : "memory");
}

__device__ __forceinline__ void tcgen05_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tcgen05_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 32 columns of this warp's 32 lanes: v[j] is column j of the thread's lane.
__device__ __forceinline__ void tmem_load32(unsigned addr, float (&v)[32]) {
    unsigned r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
}

// Shared-memory descriptor of a 128-byte-swizzled operand tile.  K-major: rows
// of 128 bytes (64 values of K), groups of 8 rows 1024 bytes apart.  MN-major:
// rows of 64 values of M or N, one row per k; groups of 8 k 1024 bytes apart,
// the next 64 values of M or N a whole stage depth (64 k) further.
__device__ __forceinline__ uint64_t smem_desc(unsigned addr, bool mn_major) {
    const uint64_t lead = mn_major ? (kBlockK * 128) >> 4 : 1;
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (lead << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// Descriptor steps (16-byte units) from one k of 16 to the next.
__device__ __forceinline__ unsigned desc_step(bool mn_major) { return mn_major ? 2048 >> 4 : 32 >> 4; }

// ------------------------------------------------------- memory helpers --

// Up to four consecutive values as float; `vec`: the address is aligned to
// the four (and n is 4 wherever a vector is taken).
__device__ __forceinline__ float4 load4(const float* p, int n, bool vec) {
    if (vec && n == 4) return *reinterpret_cast<const float4*>(p);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    v.x = p[0];
    if (n > 1) v.y = p[1];
    if (n > 2) v.z = p[2];
    if (n > 3) v.w = p[3];
    return v;
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p, int n, bool vec) {
    if (vec && n == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                           __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
    }
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    v.x = __bfloat162float(p[0]);
    if (n > 1) v.y = __bfloat162float(p[1]);
    if (n > 2) v.z = __bfloat162float(p[2]);
    if (n > 3) v.w = __bfloat162float(p[3]);
    return v;
}
__device__ __forceinline__ float4 load4(const __half* p, int n, bool vec) {
    if (vec && n == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    v.x = __half2float(p[0]);
    if (n > 1) v.y = __half2float(p[1]);
    if (n > 2) v.z = __half2float(p[2]);
    if (n > 3) v.w = __half2float(p[3]);
    return v;
}
__device__ __forceinline__ void store4(float* p, float4 v, int n, bool vec) {
    if (vec && n == 4) {
        *reinterpret_cast<float4*>(p) = v;
        return;
    }
    p[0] = v.x;
    if (n > 1) p[1] = v.y;
    if (n > 2) p[2] = v.z;
    if (n > 3) p[3] = v.w;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v, int n, bool vec) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    if (vec && n == 4) {
        uint2 u;
        u.x = *reinterpret_cast<const unsigned*>(&a);
        u.y = *reinterpret_cast<const unsigned*>(&b);
        *reinterpret_cast<uint2*>(p) = u;
        return;
    }
    p[0] = a.x;
    if (n > 1) p[1] = a.y;
    if (n > 2) p[2] = b.x;
    if (n > 3) p[3] = b.y;
}
__device__ __forceinline__ void store4(__half* p, float4 v, int n, bool vec) {
    const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    if (vec && n == 4) {
        uint2 u;
        u.x = *reinterpret_cast<const unsigned*>(&a);
        u.y = *reinterpret_cast<const unsigned*>(&b);
        *reinterpret_cast<uint2*>(p) = u;
        return;
    }
    p[0] = a.x;
    if (n > 1) p[1] = a.y;
    if (n > 2) p[2] = b.x;
    if (n > 3) p[3] = b.y;
}

// A matrix that an epilogue reads or writes: float or bf16 by a flag.
struct View {
    void* data;
    long long ld, batch_stride;
    int f32;
    int vec;  // four values starting at a column that is a multiple of four are one aligned vector
};
__device__ __forceinline__ float4 view_load(const View& v, int b, long long row, int col, int n) {
    const long long at = (long long)b * v.batch_stride + row * v.ld + col;
    return v.f32 ? load4(static_cast<const float*>(v.data) + at, n, v.vec)
                 : load4(static_cast<const __nv_bfloat16*>(v.data) + at, n, v.vec);
}
__device__ __forceinline__ void view_store(const View& v, int b, long long row, int col, int n,
                                           float4 x) {
    const long long at = (long long)b * v.batch_stride + row * v.ld + col;
    if (v.f32)
        store4(static_cast<float*>(v.data) + at, x, n, v.vec);
    else
        store4(static_cast<__nv_bfloat16*>(v.data) + at, x, n, v.vec);
}

// --------------------------------------------------------------- kernel --

// Shared memory: stages (1024-byte aligned), epilogue chunks, barriers.
template <int kPair, int kBN>
struct Config {
    static constexpr int kBRows = kBN / kPair;  // rows of B (columns of D) that this block loads
    static constexpr int kABytes = kRowsPerCta * kBlockK * 2;
    static constexpr int kBBytes = kBRows * kBlockK * 2;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kChunkBytes = kEpilogueWarps * 32 * kStageRow * 4;
    static constexpr int kBarBytes = 256;
    static constexpr int kStages = (232448 - 1024 - kBarBytes - kChunkBytes) / kStageBytes > 8
                                       ? 8
                                       : (232448 - 1024 - kBarBytes - kChunkBytes) / kStageBytes;
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kChunkBytes + kBarBytes;
    static constexpr int kTmemCols = 2 * kBN;  // two accumulators; a power of two >= 32
    static_assert(kStages >= 3, "too few stages");
    static_assert((2 * kStages + 4) * 8 + 8 <= kBarBytes, "barriers");
};

// Tile t of a product: its tile row and tile column.  Symmetric products
// compute the tiles on and below the diagonal only, row by row; others walk
// down `group` tile rows before they move to the next tile column.
template <bool kSym>
__device__ __forceinline__ void tile_at(const Shape& s, int t, int& tm, int& tn) {
    if constexpr (kSym) {
        int r = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
        while ((r + 1) * (r + 2) / 2 <= t) ++r;
        while (r * (r + 1) / 2 > t) --r;
        tm = r;
        tn = t - r * (r + 1) / 2;
    } else {
        const int per = s.group * s.tiles_n;
        const int g = t / per, in = t - g * per;
        const int rows = min(s.group, s.tiles_m - g * s.group);
        tn = in / rows;
        tm = g * s.group + (in - tn * rows);
    }
}

// Epi: the operator's epilogue.
//   kSym            the product is symmetric
//   regs(p, s, b, row, col0, v, off): v[j] = D[row][col0 + j], one row per lane, all lanes
//                   call it; `off`: the tile lies off the diagonal (of a symmetric product)
//   kRows           whether the row pass below follows, with
//   Col cols(p, s, b, col, n)            what depends on the columns alone
//   Aux load(p, s, b, row, col, n)       what is read before anything is written
//   store(p, s, b, row, col, n, acc, aux, colv)
template <int kPair, int kBN, class Epi>
__global__ void __launch_bounds__(kGemmThreads, 1)
gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
            const __grid_constant__ Shape s, const __grid_constant__ typename Epi::Params ep) {
    using C = Config<kPair, kBN>;
    extern __shared__ unsigned char smem_raw[];
    const unsigned base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char* const gen = smem_raw + (base - smem_u32(smem_raw));
    float* const chunks = reinterpret_cast<float*>(gen + C::kStages * C::kStageBytes);
    const unsigned bars = base + C::kStages * C::kStageBytes + C::kChunkBytes;
    const unsigned full = bars, empty = full + 8 * C::kStages, tfull = empty + 8 * C::kStages,
                   tempty = tfull + 16;
    unsigned char* const tail = gen + (tempty + 16 - base);
    unsigned* const tmem_slot = reinterpret_cast<unsigned*>(tail);
    volatile int* const dead = reinterpret_cast<volatile int*>(tail + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned rank = kPair == 2 ? cluster_rank() : 0;
    const bool leader = rank == 0;
    const int first = blockIdx.x / kPair, step = gridDim.x / kPair;
    const int total = s.tiles * s.batch;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull + 8 * i, 1);
            mbar_init(tempty + 8 * i, kPair * kEpilogueWarps);
        }
        *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch(&map_a);
        tma_prefetch(&map_b);
    }
    if (warp == 1) tmem_alloc<kPair>(smem_u32(tmem_slot), C::kTmemCols);
    tcgen05_fence_before();
    if constexpr (kPair == 2)
        cluster_sync_all();
    else
        __syncthreads();
    tcgen05_fence_after();
    const unsigned tmem = *tmem_slot;
    // The next kernel on the stream may be set up from here on; this one
    // touches global memory only after the kernel before it has completed.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            unsigned phase = 0;
            bool alive = true;
            const int arows = kRowsPerCta * kPair;
            for (int t = first; t < total && alive; t += step) {
                const int b = t / s.tiles;
                int tm, tn;
                tile_at<Epi::kSym>(s, t - b * s.tiles, tm, tn);
                const int m0 = tm * arows + (int)rank * kRowsPerCta;
                const int n0 = tn * kBN + (int)rank * C::kBRows;
                for (int kb = 0; kb < s.kblocks; ++kb) {
                    if (!mbar_wait(empty + 8 * stage, phase ^ 1, dead)) {
                        alive = false;
                        break;
                    }
                    const unsigned sa = base + stage * C::kStageBytes, sb = sa + C::kABytes;
                    const unsigned bar = kPair == 2 ? map_rank(full + 8 * stage, 0) : full + 8 * stage;
                    if (leader) mbar_expect(full + 8 * stage, kPair * C::kStageBytes);
                    const int k0 = kb * kBlockK;
                    if (s.a_mn) {
#pragma unroll
                        for (int i = 0; i < kRowsPerCta / 64; ++i)
                            tma_load<kPair>(sa + i * kBlockK * 128, &map_a, bar, m0 + 64 * i, k0, b);
                    } else {
                        tma_load<kPair>(sa, &map_a, bar, k0, m0, b);
                    }
                    if (s.b_mn) {
#pragma unroll
                        for (int i = 0; i < C::kBRows / 64; ++i)
                            tma_load<kPair>(sb + i * kBlockK * 128, &map_b, bar, n0 + 64 * i, k0, b);
                    } else {
                        tma_load<kPair>(sb, &map_b, bar, k0, n0, b);
                    }
                    if (++stage == C::kStages) stage = 0, phase ^= 1;
                }
            }
            // No copy of this block's may be in flight when it ends: wait
            // until every stage has been consumed.
            for (int i = 0; i < C::kStages && alive; ++i) {
                alive = mbar_wait(empty + 8 * stage, phase ^ 1, dead);
                if (++stage == C::kStages) stage = 0, phase ^= 1;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            int stage = 0, it = 0;
            unsigned phase = 0;
            bool alive = true;
            const unsigned step_a = desc_step(s.a_mn), step_b = desc_step(s.b_mn);
            for (int t = first; t < total && alive; t += step, ++it) {
                const int acc = it & 1;
                if (!mbar_wait(tempty + 8 * acc, ((it >> 1) & 1) ^ 1, dead)) break;
                tcgen05_fence_after();
                const unsigned d = tmem + acc * kBN;
                for (int kb = 0; kb < s.kblocks; ++kb) {
                    if (!mbar_wait(full + 8 * stage, phase, dead)) {
                        alive = false;
                        break;
                    }
                    tcgen05_fence_after();
                    const unsigned sa = base + stage * C::kStageBytes;
                    uint64_t da = smem_desc(sa, s.a_mn), db = smem_desc(sa + C::kABytes, s.b_mn);
#pragma unroll
                    for (int k = 0; k < kBlockK / 16; ++k) {
                        mma_f16<kPair>(d, da, db, s.idesc, kb > 0 || k > 0);
                        da += step_a;
                        db += step_b;
                    }
                    mma_commit<kPair>(empty + 8 * stage);
                    if (++stage == C::kStages) stage = 0, phase ^= 1;
                }
                mma_commit<kPair>(tfull + 8 * acc);
            }
        }
        __syncwarp();
    } else {
        const int ew = warp - 2;
        const int quarter = warp & 3;       // the tensor-memory lanes this warp may read
        const int half = ew >> 2;           // and its half of the columns
        float* const chunk = chunks + ew * 32 * kStageRow;
        const unsigned tempty_lead = kPair == 2 ? map_rank(tempty, 0) : tempty;
        int it = 0;
        for (int t = first; t < total; t += step, ++it) {
            const int b = t / s.tiles;
            int tm, tn;
            tile_at<Epi::kSym>(s, t - b * s.tiles, tm, tn);
            const int acc = it & 1;
            const int row0 = tm * kRowsPerCta * kPair + (int)rank * kRowsPerCta + quarter * 32;
            const int col_first = tn * kBN + half * (kBN / 2);
            // (every lane waits, and all lanes of a warp get the same answer
            // before the warp-wide instructions below)
            const bool ok = mbar_wait(tfull + 8 * acc, (it >> 1) & 1, dead);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tcgen05_fence_after();
#pragma unroll 1
            for (int c = 0; c < kBN / 64; ++c) {
                const int col0 = col_first + 32 * c;
                float v[32];
                tmem_load32(tmem + ((unsigned)(quarter * 32) << 16) + acc * kBN + half * (kBN / 2) +
                                32 * c,
                            v);
                if (c == kBN / 64 - 1) {
                    tcgen05_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(tempty_lead + 8 * acc);
                }
                if (s.kblocks == 0) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0.0f;
                }
                if (row0 >= s.M || col0 >= s.N) continue;  // the same for the whole warp
                Epi::regs(ep, s, b, row0 + lane, col0, v, tm != tn);
                if constexpr (Epi::kRows) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        *reinterpret_cast<float4*>(chunk + lane * kStageRow + j) =
                            make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                    __syncwarp();
                    const int lr = lane >> 3, col = col0 + (lane & 7) * 4;
                    const int n = min(4, s.N - col);
                    if (n > 0) {
                        const typename Epi::Col cv = Epi::cols(ep, s, b, col, n);
#pragma unroll
                        for (int r = 0; r < 8; r += 4) {
                            typename Epi::Aux aux[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const int row = row0 + (r + u) * 4 + lr;
                                if (row < s.M) aux[u] = Epi::load(ep, s, b, row, col, n);
                            }
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const int row = row0 + (r + u) * 4 + lr;
                                const float4 a = *reinterpret_cast<const float4*>(
                                    chunk + ((r + u) * 4 + lr) * kStageRow + (lane & 7) * 4);
                                if (row < s.M) Epi::store(ep, s, b, row, col, n, a, aux[u], cv);
                            }
                        }
                    }
                    __syncwarp();
                }
            }
        }
    }
    tcgen05_fence_before();
    if constexpr (kPair == 2)
        cluster_sync_all();
    else
        __syncthreads();
    tcgen05_fence_after();
    if (*dead) {
        if (threadIdx.x == 0) atomicAdd(s.timeouts, 1u);
        // copies and products in flight end within microseconds
        const long long t0 = clock64();
        while (clock64() - t0 < 4000000) {
        }
    }
    if (warp == 1) tmem_free<kPair>(tmem, C::kTmemCols);
}

// ------------------------------------------------------------- host side --

// One operand of a product as the kernel loads it: `major` values contiguous
// (K, or M / N when mn_major), `outer` rows of them, ld apart.
struct Operand {
    const void* data;
    long long inner, outer, ld, batch_stride;
    bool bf16;
    bool mn_major;
};

// Encodes the tensor map for boxes of 64 x box_rows; false when the driver
// refuses it.
bool encode_operand(CUtensorMap* map, const Operand& o, int batch, int box_rows);

// Whether TMA can read it where it lies.
inline bool tma_ready(const void* data, long long ld, long long batch, long long batch_stride) {
    return (reinterpret_cast<uintptr_t>(data) & 15) == 0 && (ld * 2) % 16 == 0 &&
           (batch <= 1 || (batch_stride * 2) % 16 == 0);
}

int device_sms();
// The current device's count of waits that ran out; nullptr on error.
unsigned* timeout_counter();

inline unsigned instruction_desc(bool bf16, bool a_mn, bool b_mn, int m, int n) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) |
           ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((unsigned)(n >> 3) << 17) |
           ((unsigned)(m >> 4) << 24);
}

// Launches D = A B with the tile kPair * 128 x kBN.
template <int kPair, int kBN, class Epi>
cudaError_t launch_tile(const Operand& a, const Operand& b, int M, int N, int K, int batch,
                        const typename Epi::Params& ep, cudaStream_t st) {
    using C = Config<kPair, kBN>;
    constexpr int kBM = kRowsPerCta * kPair;
    static_assert(!Epi::kSym || kBM == kBN, "symmetric products use square tiles");
    Shape s = {};
    s.M = M;
    s.N = N;
    s.K = K;
    s.batch = batch;
    s.tiles_m = (M + kBM - 1) / kBM;
    s.tiles_n = (N + kBN - 1) / kBN;
    const long long tiles = Epi::kSym ? (long long)s.tiles_m * (s.tiles_m + 1) / 2
                                      : (long long)s.tiles_m * s.tiles_n;
    if (tiles * batch > 0x3FFFFFFF) return cudaErrorInvalidValue;
    s.tiles = (int)tiles;
    if (s.tiles * batch == 0) return cudaSuccess;
    s.kblocks = (K + kBlockK - 1) / kBlockK;
    s.group = 8;
    s.a_mn = a.mn_major;
    s.b_mn = b.mn_major;
    s.idesc = instruction_desc(a.bf16, a.mn_major, b.mn_major, kBM, kBN);
    CUtensorMap ma, mb;
    if (K > 0) {
        if (!encode_operand(&ma, a, batch, a.mn_major ? kBlockK : kRowsPerCta) ||
            !encode_operand(&mb, b, batch, b.mn_major ? kBlockK : C::kBRows))
            return cudaErrorInvalidValue;
    } else {  // nothing is loaded
        ma = CUtensorMap{};
        mb = CUtensorMap{};
    }
    const int sms = device_sms();
    s.timeouts = timeout_counter();
    if (sms < 1 || s.timeouts == nullptr) return cudaErrorInvalidConfiguration;
    auto* kernel = gemm_kernel<kPair, kBN, Epi>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::kSmem);
    if (e != cudaSuccess) return e;
    const int slots = sms / kPair;
    const int want = s.tiles * batch < slots ? s.tiles * batch : slots;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(want * kPair);
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kPair;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kernel, ma, mb, s, ep);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace gemm
}  // namespace vc
