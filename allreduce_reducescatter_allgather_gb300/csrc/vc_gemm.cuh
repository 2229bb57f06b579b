// The product kernels of the training-step operators: D = A B on the tcgen05
// tensor cores, 16-bit operands (bf16 or fp16), 32-bit accumulators, with the
// operator's own arithmetic in the epilogue.
//
// Warps have roles:
//   warp 0     loads the tiles of A and B through TMA into a ring of shared
//              memory stages (64 deep along K, 128-byte swizzle);
//   warp 1     issues the matrix instructions, which accumulate in tensor
//              memory;
//   the others read the accumulators and run the epilogue.  Each warp reads
//              32 rows (a warp may only read the tensor-memory lanes of its
//              quarter), 32 x 32 values at a time.
// Two kernels share this:
//   pair_kernel   for products with many tiles: persistent pairs of blocks,
//                 one 256 x 256 tile per pair (each block holds half of A's
//                 rows and half of B's, which halves the operands' traffic),
//                 two accumulators, so that the next tile's products run
//                 while this tile's epilogue reads;
//   split_kernel  for products with few tiles: 128-row tiles, each computed by
//                 a cluster of blocks that share out K and add their partial
//                 tiles through distributed shared memory, in rank order.
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

#include "vc_error.cuh"

namespace vc {
namespace gemm {

constexpr int kBlockK = 64;            // 64 16-bit values: one 128-byte swizzle row
constexpr int kRowsPerCta = 128;       // tensor-memory lanes
constexpr int kWarpStage = 2048;       // bytes of shared memory of an epilogue warp
constexpr int kGroup = 8;              // tile rows walked together, for reuse in L2
constexpr int kSmemPerBlock = 232448;  // 227 KB
constexpr int kSmemPerSm = 233472;     // 228 KB, of which each block takes 1 KB more than it asks for
constexpr long long kWaitCycles = 4000000000ll;  // about two seconds

struct Shape {
    int M, N, K;            // of one product
    int tiles_m, tiles_n;   // tiles of one product
    int tiles;              // tiles of one product that are computed
    int total;              // tiles of all products of the batch
    int kblocks;            // K blocks summed: per_plane, for each plane of A
    int per_plane;          // ceil(K / 64)
    int segment;            // K blocks summed in tensor memory at a time
    int a_mn, b_mn;         // operand is MN-major
    int planes_of_b;        // the operand that is a sum of planes is B, not A
    unsigned idesc;         // instruction descriptor
};

// ------------------------------------------------------------------ PTX --

__device__ __forceinline__ unsigned smem_u32(const void* p) {
    return (unsigned)__cvta_generic_to_shared(p);
}

// One lane of a converged warp, the same one each time.  (The instructions
// that one thread issues for the warp take their operands from uniform
// registers; under this predicate the compiler knows that there is only one.)
__device__ __forceinline__ bool elect_one() {
    unsigned ok;
    asm volatile(
        "{\n.reg .pred p;\n.reg .b32 r;\nelect.sync r|p, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok));
    return ok != 0;
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
__device__ __forceinline__ bool mbar_wait(unsigned bar, unsigned parity, volatile int* dead,
                                          long long limit = kWaitCycles) {
    if (mbar_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try(bar, parity)) {
        if (*dead) return false;
        if (clock64() - t0 > limit) {
            *dead = 1;
            return false;
        }
    }
    return true;
}

// The same for a whole converged warp: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(unsigned bar, unsigned parity, volatile int* dead,
                                          long long limit = kWaitCycles) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, dead, limit));
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

// 16 columns.
__device__ __forceinline__ void tmem_load16(unsigned addr, float (&v)[16]) {
    unsigned r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
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

// Two float operations in one instruction, each rounded to nearest.
__device__ __forceinline__ uint64_t pack2(float2 a) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)), "l"(pack2(c)));
    return unpack2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)));
    return unpack2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)));
    return unpack2(r);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

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
// A matrix that an epilogue reads or writes: float or bf16 by a flag.
struct View {
    void* data;
    long long ld, batch_stride;
    int f32;
    int vec;  // four values starting at a column that is a multiple of four are one aligned vector
    int vec16;  // rows are on 16 bytes
};
// Value by value; the stores out of line, to keep the common case's code short.
static __device__ __noinline__ void store_few(void* p, int f32, int n, float4 x) {
    if (f32)
        store4(static_cast<float*>(p), x, n, false);
    else
        store4(static_cast<__nv_bfloat16*>(p), x, n, false);
}
// n <= 4 values of a row.
__device__ __forceinline__ float4 view_load(const View& v, int b, long long row, int col, int n) {
    const char* p = static_cast<const char*>(v.data) +
                    (((long long)b * v.batch_stride + row * v.ld + col) << (v.f32 ? 2 : 1));
    if (!v.vec || n < 4)
        return v.f32 ? load4(reinterpret_cast<const float*>(p), n, false)
                     : load4(reinterpret_cast<const __nv_bfloat16*>(p), n, false);
    if (v.f32) return *reinterpret_cast<const float4*>(p);
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
}
__device__ __forceinline__ void view_store(const View& v, int b, long long row, int col, int n,
                                           float4 x) {
    char* p = static_cast<char*>(v.data) +
              (((long long)b * v.batch_stride + row * v.ld + col) << (v.f32 ? 2 : 1));
    if (!v.vec || n < 4)
        store_few(p, v.f32, n, x);
    else if (v.f32)
        store4(reinterpret_cast<float*>(p), x, 4, true);
    else
        store4(reinterpret_cast<__nv_bfloat16*>(p), x, 4, true);
}

// ------------------------------------------------------------- epilogues --

// Where a warp's 32 x 32 chunk of a product lies.
struct Place {
    int b, row0, col0;  // product of the batch, first row, first column
    int M, N;           // its extents
    int lane;
    bool off;              // the tile lies off the diagonal (of a symmetric product)
    unsigned char* stage;  // the warp's piece of shared memory, kWarpStage bytes
    __device__ __forceinline__ int row() const { return row0 + lane; }
    __device__ __forceinline__ bool whole() const { return col0 + 32 <= N; }
};

// A chunk of 16-bit values passes between its two forms through the warp's
// piece of shared memory: one row per lane, which the accumulators have, and
// 64 bytes of a row per four lanes, which global memory wants.  The 16-byte
// pieces are permuted within each 128 bytes so that neither side has bank
// conflicts.
struct Chunk16 {
    uint4 u[4];  // across: piece lane % 4 of row 8 i + lane / 4; own: piece i of row lane
};
__device__ __forceinline__ uint4* piece_of(unsigned char* stage, int row, int c) {
    return reinterpret_cast<uint4*>(stage + (row >> 1) * 128 + (row & 1) * 64 +
                                    ((c ^ ((row >> 1) & 3)) * 16));
}
__device__ __forceinline__ void across_to_own(const Place& q, Chunk16& x) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) *piece_of(q.stage, 8 * i + (q.lane >> 2), q.lane & 3) = x.u[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) x.u[i] = *piece_of(q.stage, q.lane, i);
}
__device__ __forceinline__ void own_to_across(const Place& q, Chunk16& x) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) *piece_of(q.stage, q.lane, i) = x.u[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) x.u[i] = *piece_of(q.stage, 8 * i + (q.lane >> 2), q.lane & 3);
}
// `corner`: the chunk's first value; ld and the 16-byte pieces in bytes.
__device__ __forceinline__ void load_across(const void* corner, long long ld_bytes, const Place& q,
                                            Chunk16& x) {
    const unsigned char* p = static_cast<const unsigned char*>(corner) +
                             (long long)(q.lane >> 2) * ld_bytes + (q.lane & 3) * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (q.row0 + 8 * i + (q.lane >> 2) < q.M)
            x.u[i] = *reinterpret_cast<const uint4*>(p + 8 * i * ld_bytes);
}
__device__ __forceinline__ void store_across(void* corner, long long ld_bytes, const Place& q,
                                             const Chunk16& x) {
    unsigned char* p = static_cast<unsigned char*>(corner) + (long long)(q.lane >> 2) * ld_bytes +
                       (q.lane & 3) * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (q.row0 + 8 * i + (q.lane >> 2) < q.M)
            *reinterpret_cast<uint4*>(p + 8 * i * ld_bytes) = x.u[i];
}

__device__ __forceinline__ unsigned word_of(const Chunk16& x, int i) {
    const uint4 u = x.u[i >> 2];
    return (i & 3) == 0 ? u.x : (i & 3) == 1 ? u.y : (i & 3) == 2 ? u.z : u.w;
}
// Values 2 i and 2 i + 1 of the lane's row.
__device__ __forceinline__ float2 pair_at(const Chunk16& x, int i, __nv_bfloat16) {
    const unsigned w = word_of(x, i);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 pair_at(const Chunk16& x, int i, __half) {
    const unsigned w = word_of(x, i);
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ unsigned packed(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const unsigned*>(&h);
}
__device__ __forceinline__ unsigned packed(float a, float b, __half) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const unsigned*>(&h);
}
template <class T>
__device__ __forceinline__ Chunk16 packed_row(const float (&v)[32], T) {
    Chunk16 x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x.u[i] = make_uint4(packed(v[8 * i], v[8 * i + 1], T()), packed(v[8 * i + 2], v[8 * i + 3], T()),
                            packed(v[8 * i + 4], v[8 * i + 5], T()),
                            packed(v[8 * i + 6], v[8 * i + 7], T()));
    return x;
}
template <class T>
__device__ __forceinline__ void store_chunk(T* corner, long long ld, const Place& q,
                                            const float (&v)[32]) {
    Chunk16 x = packed_row(v, T());
    own_to_across(q, x);
    store_across(corner, ld * (long long)sizeof(T), q, x);
}

// Whether the chunk can be accessed in 16-byte pieces.
__device__ __forceinline__ bool in_pieces(const View& v, const Place& q) {
    return v.vec16 && q.whole();
}
__device__ __forceinline__ long long corner_of(const View& v, const Place& q) {
    return (long long)q.b * v.batch_stride + (long long)q.row0 * v.ld + q.col0;
}

// Chunks that 16-byte pieces do not cover (odd row lengths, the last columns)
// take the same way through shared memory, but value by value on global
// memory's side: 32 16-bit values of a row, or 16 floats of two rows, per
// instruction.
template <class T>
__device__ __forceinline__ void load_values(const T* corner, long long ld, const Place& q, int cols,
                                            Chunk16& x) {
    constexpr int kAcross = 64 / sizeof(T), kRows = 32 / kAcross;
    const int c = q.lane % kAcross, r0 = q.lane / kAcross;
    const T* at = corner + r0 * ld + c;
    __syncwarp();
#pragma unroll 1
    for (int i0 = 0; i0 < 32 / kRows; i0 += 8) {
        T v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = (i0 + i) * kRows + r0;
            if (c < cols && q.row0 + r < q.M) v[i] = at[(long long)(i0 + i) * kRows * ld];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            reinterpret_cast<T*>(piece_of(q.stage, (i0 + i) * kRows + r0, c * (int)sizeof(T) / 16))
                [c % (16 / sizeof(T))] = v[i];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) x.u[i] = *piece_of(q.stage, q.lane, i);
}
template <class T>
__device__ __forceinline__ void store_values(T* corner, long long ld, const Place& q, int cols,
                                             const Chunk16& x) {
    constexpr int kAcross = 64 / sizeof(T), kRows = 32 / kAcross;
    const int c = q.lane % kAcross, r0 = q.lane / kAcross;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) *piece_of(q.stage, q.lane, i) = x.u[i];
    __syncwarp();
    T* at = corner + r0 * ld + c;
#pragma unroll 1
    for (int i0 = 0; i0 < 32 / kRows; i0 += 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = (i0 + i) * kRows + r0;
            const T v = reinterpret_cast<const T*>(
                piece_of(q.stage, r, c * (int)sizeof(T) / 16))[c % (16 / sizeof(T))];
            if (c < cols && q.row0 + r < q.M) at[(long long)(i0 + i) * kRows * ld] = v;
        }
    }
}

// The chunk of a matrix, one row per lane: v[j] = X[row0 + lane][col0 + j].
// All lanes call it.
__device__ __forceinline__ void get_rows(const View& x, const Place& q, float (&v)[32]) {
    Chunk16 c;
    if (x.f32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float* corner = static_cast<const float*>(x.data) + corner_of(x, q) + 16 * h;
            if (in_pieces(x, q)) {
                load_across(corner, x.ld * 4, q, c);
                across_to_own(q, c);
            } else {
                load_values(corner, x.ld, q, q.N - q.col0 - 16 * h, c);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) v[16 * h + i] = __uint_as_float(word_of(c, i));
        }
    } else {
        const __nv_bfloat16* corner = static_cast<const __nv_bfloat16*>(x.data) + corner_of(x, q);
        if (in_pieces(x, q)) {
            load_across(corner, x.ld * 2, q, c);
            across_to_own(q, c);
        } else {
            load_values(reinterpret_cast<const unsigned short*>(corner), x.ld, q, q.N - q.col0, c);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 f = pair_at(c, i, __nv_bfloat16());
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

__device__ __forceinline__ void put_rows(const View& x, const Place& q, const float (&v)[32]) {
    Chunk16 c;
    if (x.f32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                c.u[i] = make_uint4(
                    __float_as_uint(v[16 * h + 4 * i]), __float_as_uint(v[16 * h + 4 * i + 1]),
                    __float_as_uint(v[16 * h + 4 * i + 2]), __float_as_uint(v[16 * h + 4 * i + 3]));
            float* corner = static_cast<float*>(x.data) + corner_of(x, q) + 16 * h;
            if (in_pieces(x, q)) {
                own_to_across(q, c);
                store_across(corner, x.ld * 4, q, c);
            } else {
                store_values(corner, x.ld, q, q.N - q.col0 - 16 * h, c);
            }
        }
    } else {
        __nv_bfloat16* corner = static_cast<__nv_bfloat16*>(x.data) + corner_of(x, q);
        c = packed_row(v, __nv_bfloat16());
        if (in_pieces(x, q)) {
            own_to_across(q, c);
            store_across(corner, x.ld * 2, q, c);
        } else {
            store_values(reinterpret_cast<unsigned short*>(corner), x.ld, q, q.N - q.col0, c);
        }
    }
}

// Transposed: v[j] = X[col0 + j][row0 + lane], which a warp accesses along
// X's rows.  M and N are still the product's, so X has N rows.
__device__ __forceinline__ void get_columns(const View& x, const Place& q, float (&v)[32]) {
    const long long at = (long long)q.b * x.batch_stride + (long long)q.col0 * x.ld + q.row();
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        v[j] = 0.0f;
        if (q.row() < q.M && q.col0 + j < q.N)
            v[j] = x.f32 ? static_cast<const float*>(x.data)[at + j * x.ld]
                         : __bfloat162float(static_cast<const __nv_bfloat16*>(x.data)[at + j * x.ld]);
    }
}
__device__ __forceinline__ void put_columns(const View& x, const Place& q, const float (&v)[32]) {
    const long long at = (long long)q.b * x.batch_stride + (long long)q.col0 * x.ld + q.row();
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        if (q.row() < q.M && q.col0 + j < q.N) {
            if (x.f32)
                static_cast<float*>(x.data)[at + j * x.ld] = v[j];
            else
                static_cast<__nv_bfloat16*>(x.data)[at + j * x.ld] = __float2bfloat16(v[j]);
        }
    }
}

// Epi: the operator's epilogue.
//   kSym                  the product is symmetric: only the tiles on and
//                         below the diagonal are computed
//   odd(p)                whether a matrix it touches has rows off 16 bytes
//   Pre                   what the epilogue of a chunk reads, as loaded
//   prefetch(p, q, pre)   starts these loads; called before the chunk's products are read
//   apply(p, q, pre, v)   v[j] = D[row0 + lane][col0 + j]; all lanes call it
// and, for sums that are promoted to registers,
//   sums32(p)             whether the output is 32 bits wide
//   start(p, q, sum)      the value that the sum begins with
//   finish(p, q, sum)     stores it
template <class Epi>
__device__ __forceinline__ bool inside(const Place& q) {
    return q.row0 < q.M && q.col0 < q.N;  // the same for the whole warp
}

// ------------------------------------------------------- loads and products --

// Tile t of a product: its tile row and tile column.  Symmetric products
// compute the tiles that reach the diagonal or lie below it, row by row (a
// tile row holds kAcross tiles per tile height); others walk down kGroup tile
// rows before they move to the next tile column.
template <bool kSym, int kAcross>
__device__ __forceinline__ void tile_at(const Shape& s, int t, int& tm, int& tn) {
    if constexpr (kSym) {
        const int u = t / kAcross;
        int r = (int)((sqrtf(8.0f * (float)u + 1.0f) - 1.0f) * 0.5f);
        while ((long long)(r + 1) * (r + 2) / 2 <= u) ++r;
        while ((long long)r * (r + 1) / 2 > u) --r;
        tm = r;
        tn = t - (int)((long long)r * (r + 1) / 2) * kAcross;
    } else {
        const int per = kGroup * s.tiles_n;
        const int g = t / per, in = t - g * per;
        const int rows = min(kGroup, s.tiles_m - g * kGroup);
        tn = in / rows;
        tm = g * kGroup + (in - tn * rows);
    }
}

// A place in the ring of stages.
template <int kStages>
struct Ring {
    int stage = 0;
    unsigned phase = 0;
    __device__ __forceinline__ void next() {
        if (++stage == kStages) stage = 0, phase ^= 1;
    }
};

// One stage: 128 rows of A and kBRows of B, K block kb of product b.  (Where an
// operand is a sum of two planes, its blocks follow each other and the other's
// are read again.)
template <int kPair, int kBRows>
__device__ __forceinline__ void load_stage(unsigned sa, const CUtensorMap* map_a,
                                           const CUtensorMap* map_b, const Shape& s, unsigned bar,
                                           int m0, int n0, int kb, int b) {
    const int plane = kb >= s.per_plane;
    const int k0 = (kb - (plane ? s.per_plane : 0)) * kBlockK;
    const int za = b + (plane & (s.planes_of_b ^ 1)), zb = b + (plane & s.planes_of_b);
    const unsigned sb = sa + kRowsPerCta * kBlockK * 2;
    if (s.a_mn) {
#pragma unroll
        for (int i = 0; i < kRowsPerCta / 64; ++i)
            tma_load<kPair>(sa + i * kBlockK * 128, map_a, bar, m0 + 64 * i, k0, za);
    } else {
        tma_load<kPair>(sa, map_a, bar, k0, m0, za);
    }
    if (s.b_mn) {
#pragma unroll
        for (int i = 0; i < (kBRows + 63) / 64; ++i)
            tma_load<kPair>(sb + i * kBlockK * 128, map_b, bar, n0 + 64 * i, k0, zb);
    } else {
        tma_load<kPair>(sb, map_b, bar, k0, n0, zb);
    }
}

template <int kPair>
__device__ __forceinline__ void multiply_stage(unsigned d, unsigned sa, const Shape& s, bool add) {
    uint64_t da = smem_desc(sa, s.a_mn), db = smem_desc(sa + kRowsPerCta * kBlockK * 2, s.b_mn);
    const unsigned step_a = desc_step(s.a_mn), step_b = desc_step(s.b_mn);
#pragma unroll
    for (int k = 0; k < kBlockK / 16; ++k) {
        mma_f16<kPair>(d, da, db, s.idesc, add || k > 0);
        da += step_a;
        db += step_b;
    }
}

// A dead block waits until its copies and products in flight, which end
// within microseconds, can no longer touch its memory; and is counted.
__device__ __forceinline__ void bury(volatile int* dead, unsigned* timeouts) {
    if (*dead) {
        if (threadIdx.x == 0) atomicAdd(timeouts, 1u);
        const long long t0 = clock64();
        while (clock64() - t0 < 4000000) {
        }
    }
}

// ------------------------------------------------------------- pair kernel --

template <int kEpilogueWarps>
struct Pair {
    static constexpr int kBN = 256, kBM = 256;
    static constexpr int kWarps = kEpilogueWarps;  // 8, or 16 with half the registers
    static constexpr int kThreads = 32 * (2 + kWarps);
    static constexpr int kBRows = kBN / 2;  // rows of B (columns of D) that a block loads
    static constexpr int kStageBytes = (kRowsPerCta + kBRows) * kBlockK * 2;
    static constexpr int kChunkBytes = kWarps * kWarpStage;
    static constexpr int kBarBytes = 256;
    static constexpr int kStages = 6;
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kChunkBytes + kBarBytes;
    static constexpr int kTmemCols = 2 * kBN;  // two accumulators
    static_assert(kSmem <= kSmemPerBlock, "shared memory");
};

// Sums in registers want more warps, with fewer columns each (and fewer registers:
// the Newton-Schulz update's epilogue is slower with 16, 17.7 -> 19.9 us at 4096
// x 1024 x 1024).
template <bool kPromote>
struct PairFor : Pair<kPromote ? 16 : 8> {};

// One or two products in one launch (the second one's tiles may be 0), whose
// blocks then share the work of both: the first has the longer tiles.
template <class Epi>
struct PairWork {
    Shape s[2];
    typename Epi::Params ep[2];
    int extra;  // second product's tiles that a pair without a last tile of the first takes first
    unsigned* timeouts;
};

// The i-th tile of pair `slot`: false when there is none.  First the first
// product's tiles in turn; where these do not come out even, the pairs that
// are one short take `extra` tiles of the second product, about as long
// together; then the rest of it in turn.
template <class Epi>
__device__ __forceinline__ bool work_item(const PairWork<Epi>& w, int slot, int slots, int i, int& which,
                                          int& t) {
    const int n0 = w.s[0].total, n1 = w.s[1].total;
    const int c0 = slot < n0 ? (n0 - slot + slots - 1) / slots : 0;
    which = 0;
    t = slot + i * slots;
    if (i < c0) return true;
    if (n1 == 0) return false;
    which = 1;
    i -= c0;
    const int r = n0 % slots;
    if (r == 0) {
        t = slot + i * slots;
        return t < n1;
    }
    if (slot >= r) {
        if (i < w.extra) {
            t = i * (slots - r) + (slot - r);
            return t < n1;
        }
        i -= w.extra;
    }
    t = (slots - r) * w.extra + slot + i * slots;
    return t < n1;
}

// kPromote: sums in tensor memory are cut to `segment` K blocks, which the
// epilogue warps add in registers, rounding to nearest.  (The tensor cores
// cut accumulated sums off instead: measured 1e-6 relative, towards zero, for
// sums of 1024 products, and growing with their number.)
template <class Epi, int kCount, bool kPromote>
__global__ void __launch_bounds__(PairFor<kPromote>::kThreads, 1)
pair_kernel(const __grid_constant__ CUtensorMap map_a0, const __grid_constant__ CUtensorMap map_b0,
            const __grid_constant__ CUtensorMap map_a1, const __grid_constant__ CUtensorMap map_b1,
            const __grid_constant__ PairWork<Epi> w) {
    using C = PairFor<kPromote>;
    extern __shared__ unsigned char smem_raw[];
    const unsigned base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char* const gen = smem_raw + (base - smem_u32(smem_raw));
    unsigned char* const chunks = gen + C::kStages * C::kStageBytes;
    const unsigned full = base + C::kStages * C::kStageBytes + C::kChunkBytes;
    const unsigned empty = full + 8 * C::kStages, tfull = empty + 8 * C::kStages, tempty = tfull + 16;
    unsigned char* const tail = gen + (tempty + 16 - base);
    unsigned* const tmem_slot = reinterpret_cast<unsigned*>(tail);
    volatile int* const dead = reinterpret_cast<volatile int*>(tail + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned rank = cluster_rank();
    const bool leader = rank == 0;
    const int slot = blockIdx.x / 2, slots = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull + 8 * i, 1);
            mbar_init(tempty + 8 * i, 2 * C::kWarps);
        }
        *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch(&map_a0);
        tma_prefetch(&map_b0);
    }
    if (warp == 1) tmem_alloc<2>(smem_u32(tmem_slot), C::kTmemCols);
    tcgen05_fence_before();
    cluster_sync_all();
    tcgen05_fence_after();
    const unsigned tmem = *tmem_slot;
    // The next kernel on the stream may be set up from here on; this one
    // touches global memory only after the kernel before it has completed.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    int which, t;
    if (warp == 0) {
        Ring<C::kStages> ring;
        bool alive = true;
        for (int i = 0; alive && work_item(w, slot, slots, i, which, t); ++i) {
            const Shape s = w.s[kCount == 1 ? 0 : which];
            const CUtensorMap* ma = which ? &map_a1 : &map_a0;
            const CUtensorMap* mb = which ? &map_b1 : &map_b0;
            const int b = t / s.tiles;
            int tm, tn;
            tile_at<Epi::kSym, C::kBM / C::kBN>(s, t - b * s.tiles, tm, tn);
            const int m0 = tm * C::kBM + (int)rank * kRowsPerCta;
            const int n0 = tn * C::kBN + (int)rank * C::kBRows;
            for (int kb = 0; kb < s.kblocks; ++kb) {
                alive = warp_wait(empty + 8 * ring.stage, ring.phase ^ 1, dead);
                if (!alive) break;
                if (elect_one()) {
                    // both blocks' copies count on the leading block's barrier
                    if (leader) mbar_expect(full + 8 * ring.stage, 2 * C::kStageBytes);
                    load_stage<2, C::kBRows>(base + ring.stage * C::kStageBytes, ma, mb, s,
                                             map_rank(full + 8 * ring.stage, 0), m0, n0, kb, b);
                }
                __syncwarp();
                ring.next();
            }
        }
        // No copy of this block's may be in flight when it ends: wait until
        // every stage has been consumed.
        for (int i = 0; i < C::kStages && alive; ++i) {
            alive = warp_wait(empty + 8 * ring.stage, ring.phase ^ 1, dead);
            ring.next();
        }
    } else if (warp == 1) {
        if (leader) {
            Ring<C::kStages> ring;
            Ring<2> acc;
            bool alive = true;
            for (int i = 0; alive && work_item(w, slot, slots, i, which, t); ++i) {
                const Shape s = w.s[kCount == 1 ? 0 : which];
                int kb = 0;
                do {
                    const int stop = kPromote ? min(kb + s.segment, s.kblocks) : s.kblocks;
                    alive = warp_wait(tempty + 8 * acc.stage, acc.phase ^ 1, dead);
                    if (!alive) break;
                    tcgen05_fence_after();
                    for (bool add = false; kb < stop; ++kb, add = true) {
                        alive = warp_wait(full + 8 * ring.stage, ring.phase, dead);
                        if (!alive) break;
                        tcgen05_fence_after();
                        if (elect_one()) {
                            multiply_stage<2>(tmem + acc.stage * C::kBN,
                                              base + ring.stage * C::kStageBytes, s, add);
                            mma_commit<2>(empty + 8 * ring.stage);
                        }
                        __syncwarp();
                        ring.next();
                    }
                    if (elect_one()) mma_commit<2>(tfull + 8 * acc.stage);
                    __syncwarp();
                    acc.next();
                } while (alive && kb < s.kblocks);
            }
        }
    } else {
        const int ew = warp - 2;
        const int quarter = warp & 3;  // the tensor-memory lanes this warp may read
        constexpr int kChunks = C::kBN / 32 / (C::kWarps / 4);
        const int first_col = (ew >> 2) * kChunks * 32;  // its part of the columns
        const unsigned lanes = tmem + ((unsigned)(quarter * 32) << 16) + first_col;
        const unsigned tempty_lead = map_rank(tempty, 0);
        Ring<2> acc;
        bool alive = true;
        // (the parameters of each product are read at fixed places, which the
        // compiler turns into operands of the instructions)
        auto tile = [&](const Shape& s, const typename Epi::Params& ep) {
            const int b = t / s.tiles;
            int tm, tn;
            tile_at<Epi::kSym, C::kBM / C::kBN>(s, t - b * s.tiles, tm, tn);
            Place q;
            q.b = b;
            q.row0 = tm * C::kBM + (int)rank * kRowsPerCta + quarter * 32;
            q.col0 = tn * C::kBN + first_col;
            q.M = s.M;
            q.N = s.N;
            q.lane = lane;
            q.off = tm != tn;
            q.stage = chunks + ew * kWarpStage;
            bool summed = false;
            if constexpr (kPromote) {
              if (s.segment < s.kblocks) {
                summed = true;
                float sum[kChunks][32];
                Place at = q;
#pragma unroll
                for (int c = 0; c < kChunks; ++c, at.col0 += 32) Epi::start(ep, at, sum[c]);
                int kb = 0;
                do {
                    kb += s.segment;
                    alive = warp_wait(tfull + 8 * acc.stage, acc.phase, dead);
                    if (!alive) break;
                    tcgen05_fence_after();
#pragma unroll
                    for (int c = 0; c < 2 * kChunks; ++c) {
                        float v[16];
                        tmem_load16(lanes + acc.stage * C::kBN + 16 * c, v);
#pragma unroll
                        for (int j = 0; j < 16; ++j) sum[c / 2][(c & 1) * 16 + j] += v[j];
                    }
                    tcgen05_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(tempty_lead + 8 * acc.stage);
                    acc.next();
                } while (kb < s.kblocks);
                if (!alive) return;
#pragma unroll
                for (int c = 0; c < kChunks; ++c, q.col0 += 32) {
                    if (inside<Epi>(q)) Epi::finish(ep, q, sum[c]);
                }
              }
            }
            if (!summed) {
                typename Epi::Pre pre;
                if (inside<Epi>(q)) Epi::prefetch(ep, q, pre);
                alive = warp_wait(tfull + 8 * acc.stage, acc.phase, dead);
                if (!alive) return;
                tcgen05_fence_after();
#pragma unroll 1
                for (int c = 0; c < kChunks; ++c) {
                    float v[32];
                    tmem_load32(lanes + acc.stage * C::kBN + 32 * c, v);
                    if (c == kChunks - 1) {
                        tcgen05_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(tempty_lead + 8 * acc.stage);
                    }
                    if (s.kblocks == 0) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0.0f;
                    }
                    if (inside<Epi>(q)) Epi::apply(ep, q, pre, v);
                    q.col0 += 32;
                    if (c < kChunks - 1 && inside<Epi>(q)) Epi::prefetch(ep, q, pre);
                }
                acc.next();
            }
        };
        for (int i = 0; alive && work_item(w, slot, slots, i, which, t); ++i) {
            if (kCount == 1 || which == 0)
                tile(w.s[0], w.ep[0]);
            else
                tile(w.s[1], w.ep[1]);
        }
    }
    tcgen05_fence_before();
    cluster_sync_all();
    tcgen05_fence_after();
    bury(dead, w.timeouts);
    if (warp == 1) tmem_free<2>(tmem, C::kTmemCols);
}

// ------------------------------------------------------------ split kernel --

template <int kTileN>
struct Split {
    static constexpr int kBM = kRowsPerCta, kBN = kTileN;
    static constexpr int kStageBytes = (kRowsPerCta + kBN) * kBlockK * 2;
    static constexpr int kWarps = kBN == 128 ? 8 : 4;  // of the epilogue
    static constexpr int kThreads = 32 * (2 + kWarps);
    static constexpr int kUnits = kBN / 8;  // 32 x 32 chunks of the tile
    // Partial chunks that the cluster's blocks (1, 2, 4 or 8; with 128 columns
    // also 3) send to this one.
    static constexpr int kParts = kBN == 128 ? 18 : 8;
    static constexpr int kPartBytes = kParts * 4096;
    static constexpr int kChunkBytes = kWarps * kWarpStage;
    static constexpr int kBarBytes = 256;
    static constexpr int kMaxStages = 8;
    static constexpr int kFixed = kPartBytes + kChunkBytes + kBarBytes;
    static constexpr int kTmemCols = kBN;
    // Two blocks fit an SM with few stages, so that one's set-up, or the
    // next launch's, runs beside the other's work; with one block per SM,
    // more stages cover the latency of the memory.
    static constexpr int kBlocksPerSm = kBN == 128 ? 1 : 2;
    static constexpr int kFewStages = (kSmemPerSm / kBlocksPerSm - 1024 - kFixed) / kStageBytes;
    static constexpr int kManyStages =
        (kSmemPerBlock - kFixed) / kStageBytes < kMaxStages ? (kSmemPerBlock - kFixed) / kStageBytes : kMaxStages;
    static_assert(kFewStages >= 2, "shared memory");
    static_assert((2 * kMaxStages + 1) * 8 + 8 <= kBarBytes, "barriers");
};

// A cluster of blocks computes one 128 x kBN tile; block `rank` takes K blocks
// rank, rank + ranks, ... (neighbours in memory at about the same time).  The tile's 32 x 32 chunks are shared out over the
// blocks: each sends its partial chunks to their owners, who add them in rank
// order and run the epilogue.
//
// One or two products in a launch: clusters from `second` on work on the second.
template <class Epi, int kCount>
struct SplitWork {
    Shape s[kCount];
    typename Epi::Params ep[kCount];
    int second, ranks, stages;
    unsigned* timeouts;
};

template <int kBN, class Epi, int kCount>
__global__ void __launch_bounds__(Split<kBN>::kThreads, Split<kBN>::kBlocksPerSm)
split_kernel(const __grid_constant__ CUtensorMap map_a0, const __grid_constant__ CUtensorMap map_b0,
             const __grid_constant__ CUtensorMap map_a1, const __grid_constant__ CUtensorMap map_b1,
             const __grid_constant__ SplitWork<Epi, kCount> w) {
    using C = Split<kBN>;
    // (aligned by its declaration: rounding up would cost a stage of two blocks)
    extern __shared__ __align__(1024) unsigned char smem_aligned[];
    const unsigned base = smem_u32(smem_aligned);
    unsigned char* const gen = smem_aligned;
    float4* const part = reinterpret_cast<float4*>(gen + w.stages * C::kStageBytes);
    unsigned char* const chunks = gen + w.stages * C::kStageBytes + C::kPartBytes;
    const unsigned full = base + w.stages * C::kStageBytes + C::kPartBytes + C::kChunkBytes;
    const unsigned empty = full + 8 * C::kMaxStages, tfull = empty + 8 * C::kMaxStages;
    unsigned char* const tail = gen + (tfull + 8 - base);
    unsigned* const tmem_slot = reinterpret_cast<unsigned*>(tail);
    volatile int* const dead = reinterpret_cast<volatile int*>(tail + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank(), ranks = w.ranks, stages = w.stages;
    const int cluster = blockIdx.x / ranks;
    const int which = kCount == 2 && cluster >= w.second ? 1 : 0;
    const Shape s = w.s[which];
    const typename Epi::Params& ep = w.ep[which];
    const CUtensorMap* const map_a = which ? &map_a1 : &map_a0;
    const CUtensorMap* const map_b = which ? &map_b1 : &map_b0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        mbar_init(tfull, 1);
        *dead = (base & 1023) != 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch(map_a);
        tma_prefetch(map_b);
    }
    if (warp == 1) tmem_alloc<1>(smem_u32(tmem_slot), C::kTmemCols);
    tcgen05_fence_before();
    // (every block of the cluster has begun before another writes to it)
    if (ranks > 1)
        cluster_sync_all();
    else
        __syncthreads();
    tcgen05_fence_after();
    const unsigned tmem = *tmem_slot;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int tile = which ? cluster - w.second : cluster;
    const int b = tile / s.tiles;
    int tm, tn;
    tile_at<Epi::kSym, C::kBM / C::kBN>(s, tile - b * s.tiles, tm, tn);
    const int m0 = tm * C::kBM, n0 = tn * kBN;
    const int ew = warp - 2, quarter = warp & 3;
    constexpr int kUnits = C::kUnits;  // unit u has rows (u & 3), columns u >> 2
    constexpr int kShare = kBN / 32 / (C::kWarps / 4);  // chunk columns of a warp
    Place q;
    q.b = b;
    q.M = s.M;
    q.N = s.N;
    q.lane = lane;
    q.off = tn / (C::kBM / C::kBN) != tm;
    q.stage = chunks + ew * kWarpStage;
    typename Epi::Pre pre;
    // this warp's first unit: its own quarter where K is not split
    int unit = ranks == 1 ? quarter + 4 * kShare * (ew >> 2) : rank + ranks * ew;

    if (warp == 0) {
        int stage = 0;
        unsigned phase = 0;
        for (int kb = rank; kb < s.kblocks; kb += ranks) {
            if (!warp_wait(empty + 8 * stage, phase ^ 1, dead)) break;
            if (elect_one()) {
                mbar_expect(full + 8 * stage, C::kStageBytes);
                load_stage<1, kBN>(base + stage * C::kStageBytes, map_a, map_b, s,
                                   full + 8 * stage, m0, n0, kb, b);
            }
            __syncwarp();
            if (++stage == stages) stage = 0, phase ^= 1;
        }
    } else if (warp == 1) {
        int stage = 0;
        unsigned phase = 0;
        for (int kb = rank; kb < s.kblocks; kb += ranks) {
            if (!warp_wait(full + 8 * stage, phase, dead)) break;
            tcgen05_fence_after();
            if (elect_one()) {
                multiply_stage<1>(tmem, base + stage * C::kStageBytes, s, kb >= ranks);
                mma_commit<1>(empty + 8 * stage);
            }
            __syncwarp();
            if (++stage == stages) stage = 0, phase ^= 1;
        }
        if (elect_one()) mma_commit<1>(tfull);
        __syncwarp();
    } else {
        q.row0 = m0 + (unit & 3) * 32;
        q.col0 = n0 + (unit >> 2) * 32;
        if (unit < kUnits && inside<Epi>(q)) Epi::prefetch(ep, q, pre);
        const bool ok = warp_wait(tfull, 0, dead);
        tcgen05_fence_after();
        if (ok) {
            for (int h = 0; h < kShare; ++h) {
                const int c = (ew >> 2) * kShare + h;
                float v[32];
                tmem_load32(tmem + ((unsigned)(quarter * 32) << 16) + 32 * c, v);
                if (rank >= s.kblocks) {  // no K block: nothing was written
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0.0f;
                }
                if (ranks == 1) {
                    if (inside<Epi>(q)) Epi::apply(ep, q, pre, v);
                    q.col0 += 32;
                    if (h + 1 < kShare && inside<Epi>(q)) Epi::prefetch(ep, q, pre);
                } else {
                    // to slot [unit of the owner][from rank][8 x 32 lanes]
                    const int u = c * 4 + quarter, owner = u % ranks, k = u / ranks;
                    const unsigned at = map_rank(smem_u32(part + (k * ranks + rank) * 256 + lane), owner);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         at + j * 512),
                                     "f"(v[4 * j]), "f"(v[4 * j + 1]), "f"(v[4 * j + 2]),
                                     "f"(v[4 * j + 3])
                                     : "memory");
                }
            }
        }
    }
    tcgen05_fence_before();
    if (ranks > 1) {
        cluster_sync_all();
        if (ew >= 0) {
            for (int k = ew; unit < kUnits; unit += ranks * C::kWarps, k += C::kWarps) {
                q.row0 = m0 + (unit & 3) * 32;
                q.col0 = n0 + (unit >> 2) * 32;
                if (!inside<Epi>(q)) continue;
                if (k != ew) Epi::prefetch(ep, q, pre);
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = 0.0f;
                for (int r = 0; r < ranks; ++r) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 x = part[(k * ranks + r) * 256 + j * 32 + lane];
                        v[4 * j] += x.x;
                        v[4 * j + 1] += x.y;
                        v[4 * j + 2] += x.z;
                        v[4 * j + 3] += x.w;
                    }
                }
                Epi::apply(ep, q, pre, v);
            }
        }
        __syncthreads();
    } else {
        __syncthreads();
    }
    tcgen05_fence_after();
    bury(dead, w.timeouts);
    if (warp == 1) tmem_free<1>(tmem, C::kTmemCols);
}

// ------------------------------------------------------------- host side --

// One operand of a product as the kernel loads it: `inner` values contiguous
// (along K, or along M / N when mn_major), `outer` rows of them, ld apart.
struct Operand {
    const void* data;
    long long inner, outer, ld, batch_stride;
    bool bf16;
    bool mn_major;
};

// One product D[M, N] = A[M, K] B[K, N], or a batch of them; or, with planes =
// 2 and a batch of one, D = (A_0 + A_1) B, A's planes batch_stride apart (or, with
// planes_of_b, A (B_0 + B_1)).
struct Product {
    Operand a, b;
    int M, N, K, batch, planes;
    bool planes_of_b = false;
};
inline int k_blocks(const Product& p) { return (p.K + kBlockK - 1) / kBlockK * p.planes; }

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

__host__ __device__ inline unsigned instruction_desc(bool bf16, bool a_mn, bool b_mn, int m, int n) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) |
           ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((unsigned)(n >> 3) << 17) |
           ((unsigned)(m >> 4) << 24);
}

// (a symmetric product's last tile row may hold a tile beyond its columns,
// which computes nothing that is written)
inline long long tile_count(long long M, long long N, int bm, int bn, bool sym) {
    const long long tm = (M + bm - 1) / bm, tn = (N + bn - 1) / bn;
    return sym ? tm * (tm + 1) / 2 * (bm / bn) : tm * tn;
}

inline cudaError_t shape_of(const Product& p, int bm, int bn, bool sym, Shape* s) {
    *s = Shape{};
    s->M = p.M;
    s->N = p.N;
    s->K = p.K;
    s->tiles_m = (p.M + bm - 1) / bm;
    s->tiles_n = (p.N + bn - 1) / bn;
    const long long tiles = tile_count(p.M, p.N, bm, bn, sym);
    if (tiles * p.batch > 0x0FFFFFFF) return cudaErrorInvalidValue;
    s->tiles = (int)tiles;
    s->total = (int)(tiles * p.batch);
    s->per_plane = (p.K + kBlockK - 1) / kBlockK;
    s->kblocks = k_blocks(p);
    s->segment = s->kblocks > 0 ? s->kblocks : 1;
    s->a_mn = p.a.mn_major;
    s->b_mn = p.b.mn_major;
    s->planes_of_b = p.planes_of_b;
    s->idesc = instruction_desc(p.a.bf16, p.a.mn_major, p.b.mn_major, bm, bn);
    return cudaSuccess;
}

inline bool encode_product(const Product& p, int b_rows, CUtensorMap* ma, CUtensorMap* mb) {
    *ma = CUtensorMap{};
    *mb = CUtensorMap{};
    if (p.K == 0) return true;  // nothing is loaded
    const int pa = p.planes_of_b ? 1 : p.planes, pb = p.planes_of_b ? p.planes : 1;
    return encode_operand(ma, p.a, p.batch * pa, p.a.mn_major ? kBlockK : kRowsPerCta) &&
           encode_operand(mb, p.b, p.batch * pb, p.b.mn_major ? kBlockK : b_rows);
}

// Lets the kernel have all of an SM's shared memory that it does not have of its own, once
// per device.  (One limit for all of its launches: a limit of each launch's own size
// would refuse a larger one of another host thread.)
cudaError_t allow_smem(const void* kernel);

template <class Kernel, class... Args>
cudaError_t launch_cluster(Kernel* kernel, int blocks, int threads, int cluster, int smem,
                           cudaStream_t st, const Args&... args) {
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return reported(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// One or two products in one launch of the pair kernel.  segment: K
// blocks summed in tensor memory at a time for 32-bit outputs (kPromote).
template <class Epi, int kCount, bool kPromote>
cudaError_t launch_pair(const Product* p, const typename Epi::Params* ep, int segment,
                        cudaStream_t st) {
    PairWork<Epi> w = {};
    CUtensorMap m[4] = {};
    // the product with the longer tiles first
    const int first = kCount == 2 && k_blocks(p[kCount - 1]) > k_blocks(p[0]) ? 1 : 0;
    for (int i = 0; i < kCount; ++i) {
        const int from = i == 0 ? first : 1 - first;
        const cudaError_t e = shape_of(p[from], Pair<8>::kBM, Pair<8>::kBN, Epi::kSym, &w.s[i]);
        if (e != cudaSuccess) return e;
        if constexpr (kPromote) {
            if (Epi::sums32(ep[from])) w.s[i].segment = segment;
        }
        w.ep[i] = ep[from];
        if (!encode_product(p[from], Pair<8>::kBRows, &m[2 * i], &m[2 * i + 1]))
            return cudaErrorInvalidValue;
    }
    const int sms = device_sms();
    w.timeouts = timeout_counter();
    if (sms < 2 || w.timeouts == nullptr) return cudaErrorInvalidConfiguration;
    const int slots = sms / 2, total = w.s[0].total + w.s[1].total;
    if (total == 0) return cudaSuccess;
    const int pairs = total < slots ? total : slots;
    if (w.s[1].total > 0 && w.s[0].total % pairs != 0)
        w.extra = w.s[0].kblocks / (w.s[1].kblocks > 0 ? w.s[1].kblocks : 1);
    return launch_cluster(pair_kernel<Epi, kCount, kPromote>, pairs * 2, PairFor<kPromote>::kThreads,
                          2, PairFor<kPromote>::kSmem, st, m[0], m[1],
                          m[2], m[3], w);
}

template <int kBN, class Epi, int kCount>
cudaError_t launch_split(const Product* p, const typename Epi::Params* ep, int ranks,
                         cudaStream_t st) {
    using C = Split<kBN>;
    SplitWork<Epi, kCount> w = {};
    CUtensorMap m[4] = {};
    int clusters = 0;
    for (int i = 0; i < kCount; ++i) {
        const cudaError_t e = shape_of(p[i], C::kBM, C::kBN, Epi::kSym, &w.s[i]);
        if (e != cudaSuccess) return e;
        if (!encode_product(p[i], kBN, &m[2 * i], &m[2 * i + 1])) return cudaErrorInvalidValue;
        w.ep[i] = ep[i];
        if (i == 0) w.second = w.s[0].total;
        clusters += w.s[i].total;
    }
    if (clusters == 0) return cudaSuccess;
    if (clusters > 0x0FFFFFFF) return cudaErrorInvalidValue;
    const int blocks = clusters * ranks;
    w.ranks = ranks;
    w.stages = blocks <= device_sms() ? C::kManyStages : C::kFewStages;
    w.timeouts = timeout_counter();
    if (w.timeouts == nullptr) return cudaErrorInvalidConfiguration;
    return launch_cluster(split_kernel<kBN, Epi, kCount>, blocks, C::kThreads, ranks,
                          C::kFixed + w.stages * C::kStageBytes, st, m[0], m[1], m[2], m[3], w);
}

// How long a product takes, in microseconds, by a model of the kernels that was
// fitted to measurements of 1 to 512 tiles and K of 64 to 8192 on operands in
// L2, with plain stores: a fixed part, and for each wave of tiles the larger of
// its K blocks' time and its epilogue's, which is longer where a matrix's rows
// are off 16 bytes (`odd`).  It is within 20 % of most of those, but too low
// for the Newton-Schulz products, whose epilogues read and write more: of 4096 x
// 1024, the update 11.4 us by the model and 19.4 measured, X^T X 9.5 and 12.5,
// b A + c A^2 6.1 and 9.0; of 8 x 2048 x 8192 258 and 366, 149 and 176, 44 and
// 55.  It is there to choose a kernel, not to predict a time.
//   pair kernel, 256 x 256:   6.5 + waves of 76 x max(0.275 K blocks + 0.5, 3.2)
//   split kernel, 128 x 64:   1.5 + 2.3 waves of 304 + 0.2 (blocks per SM) K blocks
//   split kernel, 128 x 128:  1.5 + waves of 152 x (2.8 + 0.28 K blocks)
//                             (split: + 0.7 where K is)
// e.g. 2048 x 2048 x 2048: 17 us (pair), 25 us (128 x 64); 512 x 512 x 2048:
// 15.8 us and 6.1 us; 1024 x 1024 x 4096: 24 us and 14 us.
struct Plan {
    double us;
    int tile, ranks;  // 256: the pair kernel; 128, 64: the split kernel's columns
};

inline double pair_us(const Product* p, int count, bool sym, bool odd) {
    double tile_us = 0.0, longest = 0.0;
    long long total = 0;
    const int slots = device_sms() / 2;
    for (int i = 0; i < count; ++i) {
        const long long tiles = tile_count(p[i].M, p[i].N, Pair<8>::kBM, Pair<8>::kBN, sym) * p[i].batch;
        const double k = 0.275 * k_blocks(p[i]) + 0.5, epilogue = odd ? 9.0 : 3.2;
        const double each = k > epilogue ? k : epilogue;
        longest = each > longest ? each : longest;
        tile_us += each * (double)tiles;
        total += tiles;
    }
    const double fixed = odd ? 8.0 : 6.5;
    if (count == 1) return fixed + longest * (double)((total + slots - 1) / slots);
    const double even = tile_us / slots;
    return fixed + (even > longest ? even : longest);
}

// The split kernel's best tile and number of ranks for one product or two in a
// launch; limit[i] > 0: at most so many K blocks per rank of product i (1e9 us
// where 8 ranks do not reach that).
inline Plan plan_split(const Product* p, int count, bool sym, bool odd, const int* limit) {
    const int sms = device_sms();
    Plan best = {1e9, 64, 1};
    for (int tile = 64; tile <= 128; tile += 64) {
        for (int ranks = 1; ranks <= 8; ranks += ranks == 3 ? 1 : ranks > 3 ? 4 : 1) {
            if (ranks == 3 && tile == 64) continue;
            long long blocks = 0;
            double sum = 0.0;  // K blocks of all ranks
            int most = 0;      // of one
            bool fits = true;
            for (int i = 0; i < count; ++i) {
                const long long mine = tile_count(p[i].M, p[i].N, kRowsPerCta, tile, sym) * p[i].batch * ranks;
                const int kb = (k_blocks(p[i]) + ranks - 1) / ranks;
                fits = fits && (limit == nullptr || limit[i] == 0 || kb <= limit[i]);
                blocks += mine;
                sum += (double)mine * kb;
                most = kb > most ? kb : most;
            }
            if (!fits) continue;
            // blocks are shared out whole: up to two per SM the fullest one counts
            const double per_sm = blocks > 2 * sms ? (double)blocks / sms
                                                   : (double)((blocks + sms - 1) / sms);
            const double even = blocks > 0 ? sum / (double)blocks * per_sm : 0.0;
            const double kb = even > most ? even : most;
            const double epilogue = (odd ? 2.5 : 0.0) / ranks;
            double us = 1.5 + (ranks > 1 ? 0.7 : 0.0);
            if (tile == 64)
                us += (2.3 + epilogue) * (double)((blocks + 2 * sms - 1) / (2 * sms)) + 0.2 * kb;
            else
                us += (2.8 + epilogue) * (double)((blocks + sms - 1) / sms) + 0.28 * kb;
            if (us < best.us) best = {us, tile, ranks};
        }
    }
    return best;
}

template <class Epi, int kCount>
cudaError_t launch_planned(const Product* p, const typename Epi::Params* ep, const Plan& plan,
                           cudaStream_t st) {
    if (plan.tile == 128) return launch_split<128, Epi, kCount>(p, ep, plan.ranks, st);
    return launch_split<64, Epi, kCount>(p, ep, plan.ranks, st);
}

// Picks the kernel, the tile and the ranks.
template <class Epi>
cudaError_t launch(const Product& p, const typename Epi::Params& ep, cudaStream_t st) {
    const bool odd = Epi::odd(ep);
    const Plan split = plan_split(&p, 1, Epi::kSym, odd, nullptr);
    if (split.us < pair_us(&p, 1, Epi::kSym, odd)) return launch_planned<Epi, 1>(&p, &ep, split, st);
    return launch_pair<Epi, 1, false>(&p, &ep, 0, st);
}

// A product with few columns (up to 64): tiles 32 or 64 across.  It is bound by
// reading A once, so K is split until every SM has a block (with many stages in
// flight), but not further: 32 columns, 4096 rows and K = 4096 from memory take
// 10.1 us with 4 ranks (128 blocks of 6 stages) and 10.9 us with 8 (256 of 3),
// 17.8 us with 1.
inline Plan plan_skinny(const Product& p) {
    const long long tiles = (p.M + kRowsPerCta - 1) / kRowsPerCta;
    const int sms = device_sms();
    int ranks = 1;
    while (ranks < 8 && tiles * ranks * 2 <= sms && ranks * 2 <= k_blocks(p)) ranks *= 2;
    const double kb = (double)((k_blocks(p) + ranks - 1) / ranks);
    return {3.8 + (ranks > 1 ? 0.7 : 0.0) + 0.2 * kb * (double)((tiles * ranks + sms - 1) / sms),
            p.N <= 32 ? 32 : 64, ranks};
}

template <class Epi>
cudaError_t launch_skinny(const Product& p, const typename Epi::Params& ep, cudaStream_t st) {
    const Plan plan = plan_skinny(p);
    if (plan.tile == 32) return launch_split<32, Epi, 1>(&p, &ep, plan.ranks, st);
    return launch_split<64, Epi, 1>(&p, &ep, plan.ranks, st);
}

}  // namespace gemm
}  // namespace vc
