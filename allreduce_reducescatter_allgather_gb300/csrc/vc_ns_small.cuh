// Newton-Schulz for matrices whose smaller side is at most 128: the whole
// operator -- momentum, norm, every pass, the weight update -- in one kernel.
//
// X stays on the chip.  With r <= 128 rows (the smaller side; a tall matrix is
// read and written transposed), a block holds up to 256 of X's columns in
// shared memory, and a cluster of up to eight blocks up to 2048.  Per pass:
//   A      each block multiplies its columns, X X^T, 128 x 128; the blocks add
//          their parts through distributed shared memory (each owns some 32 x
//          32 chunks of A, adds them in rank order, and sends the finished
//          chunk, in fp16, to all);
//   A^2    every block computes the whole of it, 128 x 128 x 128;
//   B X    each block its own columns.
// X's tile of 64 columns is 128 rows of 128 bytes, swizzled, which serves as
// K-major operand of X X^T and as MN-major operand of B X alike.
//
// Measured (one matrix, back to back): 64 x 64 24 us, 128 x 256 39 us, 128 x 2048
// (eight blocks) 62 us.  A launch per product spends 4 to 6 us on each of fifteen
// products however small they are: 83 us at 128 x 256.  A pass at 128 x 256 is
// about 12,000 cycles, of which the three products and the barriers around them
// take half and the arithmetic on the chunks the other half; a pass over eight
// blocks adds about 7,000 for the exchange.
#pragma once

#include "vc_train_common.cuh"

namespace vc {
namespace train {

// Whether pass `step` reads X as two fp16 values.
__host__ __device__ inline bool keeps_lo(int step, int steps) { return step == 0 || step < steps - 2; }

// How a matrix enters the iteration.  Its X_0 has the norm n = norm / (norm + eps),
// which bounds its singular values.  Where eps outweighs the norm, X_0 would
// be too small for fp16; but then a pass is a multiplication by a as far as
// the products' accuracy goes: b n^2 + c n^4 is at most 2^-12 of a.  Such
// passes are left out and a goes into the scale, until n is above 2^-7 (where
// fp16 loses 4e-5) or one pass is left.  If that one is linear too, X goes
// through it in a unit of its own.
struct Start {
    float scale;  // the stored X_0 is the update times this; 0 for a zero matrix
    float unit;   // of X: 1, or a power of two
    int skip;     // passes left out
    int linear;   // passes left out or linear: skip, or all of them
};
__device__ __forceinline__ Start start_of(float squares, float eps, float size, int steps, float a,
                                          float b, float c) {
    const float norm = sqrtf(squares), divisor = norm + eps;
    if (norm == 0.0f) return {0.0f, 1.0f, 0, 0};
    Start s = {size / divisor, 1.0f, 0, 0};
    if (!(norm <= 0.0078125f * divisor)) return s;  // (NaN too)
    // (in 64 bits: n and the powers of a pass float32's range)
    double n = (double)norm / divisor, factor = 1.0;
    auto linear = [&] {
        const double q = n * n;
        return n <= 0.0078125 && q * (fabs(b) + q * fabs(c)) <= 0.000244140625 * fabs(a);
    };
    while (s.skip < steps - 1 && linear()) {
        ++s.skip;
        factor *= a;
        n *= fabs(a);
    }
    s.linear = s.skip;
    if (linear()) {
        s.linear = steps;
        // n, or 2^-120, rounded up to a power of two
        s.unit = __uint_as_float((__float_as_uint((float)fmax(n, 0x1p-120)) + 0x7FFFFFu) & 0x7F800000u);
    }
    s.scale = (float)((double)size / divisor * (factor / s.unit));
    return s;
}

struct SmallParams {
    gemm::View g, m, out;
    int has_momentum, nesterov, weights, tall;
    int r, c;       // smaller and larger side
    int width;      // columns of X per block, a multiple of 64
    int steps;
    float beta, eps;
    float ca, cb, cc;  // the polynomial
    float size;        // X is stored times this / its unit
    float keep, scale;  // out <- keep out + scale X, or scale X
    unsigned* timeouts;
};

struct Small {
    static constexpr int kThreads = 512, kWarps = kThreads / 32, kMaxWidth = 256, kMaxRanks = 8, kRows = 128;
    static constexpr int kAtom = 128 * 128;  // bytes of 64 columns
    static constexpr int kHi = 0, kLo = 4 * kAtom, kO = 8 * kAtom, kParts = 10 * kAtom;
    static constexpr int kVectors = 14 * kAtom;  // diagonals of A and B, norms, sums, unit
    static constexpr int kBar = kVectors + 1024 + 192;
    static constexpr int kSmem = 1024 + kBar + 64;
    static constexpr int kTmemCols = 512;  // 128 for A and A^2, up to 256 for B X
    static_assert(kSmem <= gemm::kSmemPerBlock, "shared memory");
};

// Piece k (8 values) of row i of a swizzled tile of 64 columns.
__device__ __forceinline__ uint4* small_piece(unsigned char* base, int i, int col) {
    return reinterpret_cast<uint4*>(base + (col >> 6) * Small::kAtom + i * 128 +
                                    ((((col & 63) >> 3) ^ (i & 7)) * 16));
}
__device__ __forceinline__ unsigned short* small_value(unsigned char* base, int i, int col) {
    return reinterpret_cast<unsigned short*>(small_piece(base, i, col)) + (col & 7);
}
__device__ __forceinline__ void load_pieces(unsigned char* base, int i, int col, gemm::Chunk16& x) {
#pragma unroll
    for (int k = 0; k < 4; ++k) x.u[k] = *small_piece(base, i, col + 8 * k);
}
__device__ __forceinline__ void store_pieces(unsigned char* base, int i, int col,
                                             const gemm::Chunk16& x) {
#pragma unroll
    for (int k = 0; k < 4; ++k) *small_piece(base, i, col + 8 * k) = x.u[k];
}

__device__ __forceinline__ uint64_t small_desc(unsigned addr, unsigned lead_bytes) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(lead_bytes >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ void store_remote(unsigned at, uint4 v) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ void store_remote(unsigned at, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

// hi + lo with hi = x rounded to fp16.
__device__ __forceinline__ void split_halves(const float (&x)[32], gemm::Chunk16& hi,
                                             gemm::Chunk16& lo) {
    hi = gemm::packed_row(x, __half());
    float rest[32];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float2 h = gemm::pair_at(hi, i, __half());
        rest[2 * i] = x[2 * i] - h.x;
        rest[2 * i + 1] = x[2 * i + 1] - h.y;
    }
    lo = gemm::packed_row(rest, __half());
}

// beta m + g, of the momentum; with the new momentum for m, the Nesterov update.
__device__ __forceinline__ float4 new_momentum(float beta, float4 g, float4 m) {
    return make_float4(fmaf(beta, m.x, g.x), fmaf(beta, m.y, g.y), fmaf(beta, m.z, g.z),
                       fmaf(beta, m.w, g.w));
}
// The value that a store into the matrix leaves there.
__device__ __forceinline__ float4 as_stored(const gemm::View& v, float4 x) {
    if (v.f32) return x;
    return make_float4(__bfloat162float(__float2bfloat16(x.x)), __bfloat162float(__float2bfloat16(x.y)),
                       __bfloat162float(__float2bfloat16(x.z)), __bfloat162float(__float2bfloat16(x.w)));
}

__global__ void __launch_bounds__(Small::kThreads, 1)
ns_small_kernel(const __grid_constant__ SmallParams p, int ranks) {
    using S = Small;
    extern __shared__ unsigned char smem_raw[];
    const unsigned base = (gemm::smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char* const gen = smem_raw + (base - gemm::smem_u32(smem_raw));
    unsigned char *const hi = gen + S::kHi, *const lo = gen + S::kLo, *const o = gen + S::kO;
    float4* const parts = reinterpret_cast<float4*>(gen + S::kParts);
    float* const d_a = reinterpret_cast<float*>(gen + S::kVectors);
    float *const d_b = d_a + 128, *const norms = d_a + 256, *const sums = d_a + 264;
    float* const unit = d_a + 280;
    const unsigned bar = base + S::kBar;
    unsigned* const tmem_slot = reinterpret_cast<unsigned*>(gen + S::kBar + 8);
    volatile int* const dead = reinterpret_cast<volatile int*>(gen + S::kBar + 12);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)gemm::cluster_rank(), b = blockIdx.x / ranks;
    // a warp reads the tensor-memory lanes of its quarter; four warps share its columns
    const int quarter = warp & 3, share = warp >> 2, row = quarter * 32 + lane;
    const int j0 = rank * p.width, across = max(0, min(p.width, p.c - j0));

    if (threadIdx.x == 0) {
        gemm::mbar_init(bar, 1);
        *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) gemm::tmem_alloc<1>(gemm::smem_u32(tmem_slot), S::kTmemCols);
    gemm::tcgen05_fence_before();
    gemm::cluster_sync_all();
    gemm::tcgen05_fence_after();
    const unsigned tmem = *tmem_slot;
    const unsigned lanes = tmem + ((unsigned)(quarter * 32) << 16);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- the update's values, as raw 32-bit floats in two 16-bit halves
    float sum = 0.0f;
    {
        // Groups of four values: `line` is a row of the stored matrix, `first` the
        // group's place in it.  A warp takes neighbouring groups of a line; of
        // a tall matrix, whose lines are X's columns, eight groups of four
        // lines, since its values go to 32 rows of X and all of one column
        // would meet in two of the memory's banks.  All loads of a batch come
        // before its first store, so that a batch waits once.
        const int vecs = p.tall ? 32 : p.width / 4;
        const int lines = p.tall ? p.width : S::kRows;
        const int lines_in = p.tall ? across : p.r, cols_in = p.tall ? p.r : across;
        const int row_at = p.tall ? j0 : 0, col_at = p.tall ? 0 : j0;
        const int dline = p.tall ? S::kWarps : S::kThreads / vecs;
        const int dvec = p.tall ? 0 : S::kThreads % vecs;
        int line0 = p.tall ? (warp >> 2) * 4 + (lane >> 3) : threadIdx.x / vecs;
        int vec0 = p.tall ? (warp & 3) * 8 + (lane & 7) : threadIdx.x % vecs;
        constexpr int kBatch = 8;
#pragma unroll 1
        while (line0 < lines) {
          float4 gs[kBatch], ms[kBatch];
          int ls[kBatch], fs[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            ls[k] = line0;
            fs[k] = vec0 * 4;
            line0 += dline;
            vec0 += dvec;
            if (vec0 >= vecs) vec0 -= vecs, ++line0;
            gs[k] = ms[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (ls[k] < lines_in && fs[k] < cols_in) {
                const int n = min(4, cols_in - fs[k]);
                gs[k] = gemm::view_load(p.g, b, row_at + ls[k], col_at + fs[k], n);
                if (p.has_momentum) ms[k] = gemm::view_load(p.m, b, row_at + ls[k], col_at + fs[k], n);
            }
          }
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int line = ls[k], first = fs[k];
            if (line >= lines) continue;
            float4 u = gs[k];
            if (p.has_momentum && line < lines_in && first < cols_in) {
                float4 m = new_momentum(p.beta, gs[k], ms[k]);
                gemm::view_store(p.m, b, row_at + line, col_at + first, min(4, cols_in - first), m);
                m = as_stored(p.m, m);
                u = p.nesterov ? new_momentum(p.beta, gs[k], m) : m;
            }
            sum += u.x * u.x + u.y * u.y + u.z * u.z + u.w * u.w;  // 0 outside
            const unsigned w[4] = {__float_as_uint(u.x), __float_as_uint(u.y), __float_as_uint(u.z),
                                   __float_as_uint(u.w)};
            if (p.tall) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    *small_value(hi, first + k, line) = (unsigned short)(w[k] >> 16);
                    *small_value(lo, first + k, line) = (unsigned short)w[k];
                }
            } else {
                *reinterpret_cast<uint2*>(small_value(hi, line, first)) =
                    make_uint2((w[0] >> 16) | (w[1] & 0xFFFF0000u), (w[2] >> 16) | (w[3] & 0xFFFF0000u));
                *reinterpret_cast<uint2*>(small_value(lo, line, first)) =
                    make_uint2((w[0] & 0xFFFFu) | (w[1] << 16), (w[2] & 0xFFFFu) | (w[3] << 16));
            }
          }
        }
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, k);
    if (lane == 0) sums[warp] = sum;
    __syncthreads();
    if (threadIdx.x < ranks) {
        float s = 0.0f;
        for (int w = 0; w < S::kWarps; ++w) s += sums[w];
        store_remote(gemm::map_rank(gemm::smem_u32(norms + rank), threadIdx.x), s);
    }
    gemm::cluster_sync_all();
    float square = 0.0f;
    for (int i = 0; i < ranks; ++i) square += norms[i];
    const Start start = start_of(square, p.eps, p.size, p.steps, p.ca, p.cb, p.cc);
    const float to_x = start.scale;

    // ---- X_0, in place
    const int chunks = p.width / 32;
    for (int c = share; c < chunks; c += 4) {
        gemm::Chunk16 h, l;
        load_pieces(hi, row, 32 * c, h);
        load_pieces(lo, row, 32 * c, l);
        float x[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const unsigned hw = gemm::word_of(h, i), lw = gemm::word_of(l, i);
            x[2 * i] = __uint_as_float((hw << 16) | (lw & 0xFFFFu)) * to_x;
            x[2 * i + 1] = __uint_as_float((hw & 0xFFFF0000u) | (lw >> 16)) * to_x;
        }
        split_halves(x, h, l);
        store_pieces(hi, row, 32 * c, h);
        store_pieces(lo, row, 32 * c, l);
    }

    const unsigned square_desc = gemm::instruction_desc(false, false, false, 128, 128);
    const unsigned update_desc = gemm::instruction_desc(false, false, true, 128, p.width);
    // (a linear pass takes A for 0)
    const float to_a = start.linear == p.steps ? 0.0f : 1.0f / (p.size * p.size);
    if (threadIdx.x == 0) *unit = start.unit;
    const int kuse = (p.r + 15) / 16;  // 16-deep steps over X's rows that are not padding
    unsigned phase = 0;
    // After the block's writes to shared memory: makes them visible to the
    // matrix instructions that `issue` starts, and waits for these.
    auto multiply = [&](auto issue) {
        fence_async();
        gemm::tcgen05_fence_before();
        __syncthreads();
        if (warp == 0) {
            gemm::tcgen05_fence_after();
            if (gemm::elect_one()) {
                fence_async();
                issue();
                gemm::mma_commit<1>(bar);
            }
            __syncwarp();
        }
        gemm::warp_wait(bar, phase, dead);
        phase ^= 1;
        gemm::tcgen05_fence_after();
    };

    for (int step = start.skip; step < p.steps; ++step) {
        // ---- A = X X^T
        multiply([&] {
            for (int k = 0; k < p.width / 16; ++k) {
                const uint64_t d = small_desc(base + S::kHi + (k >> 2) * S::kAtom + (k & 3) * 32, 16);
                gemm::mma_f16<1>(tmem, d, d, square_desc, k > 0);
            }
        });
        // chunks of A: the diagonal in 32 bits, the rest in fp16
        auto finish_chunk = [&](float (&v)[32], int i, int col0, gemm::Chunk16& out, float& diag) {
            diag = 0.0f;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                v[j] *= to_a;
                if (i == col0 + j) {
                    diag = v[j];
                    v[j] = 0.0f;
                }
            }
            out = gemm::packed_row(v, __half());
        };
        {
            const int cc = share;  // chunk column
            float v[32];
            gemm::tmem_load32(lanes + 32 * cc, v);
            if (ranks == 1) {
                gemm::Chunk16 out;
                float diag;
                finish_chunk(v, row, 32 * cc, out, diag);
                store_pieces(o, row, 32 * cc, out);
                if (cc == quarter) d_a[row] = diag;
            } else {
                const int u = cc * 4 + quarter, owner = u % ranks, k = u / ranks;
                const unsigned at = gemm::map_rank(
                    gemm::smem_u32(parts + (k * ranks + rank) * 256 + lane), owner);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    store_remote(at + j * 512,
                                 make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                            __float_as_uint(v[4 * j + 2]),
                                            __float_as_uint(v[4 * j + 3])));
            }
        }
        if (ranks > 1) {
            gemm::cluster_sync_all();
            for (int k = warp, u; (u = rank + ranks * k) < 16; k += S::kWarps) {
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = 0.0f;
                for (int from = 0; from < ranks; ++from) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 x = parts[(k * ranks + from) * 256 + j * 32 + lane];
                        v[4 * j] += x.x;
                        v[4 * j + 1] += x.y;
                        v[4 * j + 2] += x.z;
                        v[4 * j + 3] += x.w;
                    }
                }
                const int i = (u & 3) * 32 + lane, col0 = (u >> 2) * 32;
                gemm::Chunk16 out;
                float diag;
                finish_chunk(v, i, col0, out, diag);
                for (int to = 0; to < ranks; ++to) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        store_remote(gemm::map_rank(gemm::smem_u32(small_piece(o, i, col0 + 8 * q)), to),
                                     out.u[q]);
                    if ((u & 3) == (u >> 2))
                        store_remote(gemm::map_rank(gemm::smem_u32(d_a + i), to), diag);
                }
            }
            fence_async();
            gemm::cluster_sync_all();
        }

        // ---- B = b A + c A^2, over A's place
        multiply([&] {
            for (int k = 0; k < 8; ++k) {
                const uint64_t d = small_desc(base + S::kO + (k >> 2) * S::kAtom + (k & 3) * 32, 16);
                gemm::mma_f16<1>(tmem, d, d, square_desc, k > 0);
            }
        });
        {
            const float di = d_a[row];
            const int cc = share;
            float v[32];
            gemm::tmem_load32(lanes + 32 * cc, v);
            gemm::Chunk16 a;
            load_pieces(o, row, 32 * cc, a);
            if (cc == quarter) {
                float d = 0.0f;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (lane == j) {
                        d = v[j];
                        v[j] = 0.0f;
                    }
                }
                d_b[row] = p.cb * di + p.cc * (di * di + d);
            }
            const float k0 = fmaf(p.cc, di, p.cb);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 x = gemm::pair_at(a, i, __half());
                const float2 dj = *reinterpret_cast<const float2*>(d_a + 32 * cc + 2 * i);
                v[2 * i] = fmaf(fmaf(p.cc, dj.x, k0), x.x, p.cc * v[2 * i]);
                v[2 * i + 1] = fmaf(fmaf(p.cc, dj.y, k0), x.y, p.cc * v[2 * i + 1]);
            }
            store_pieces(o, row, 32 * cc, gemm::packed_row(v, __half()));
        }

        // ---- X <- (a + diag B) X + offdiag(B) X
        multiply([&] {
            for (int k = 0; k < kuse; ++k) {
                const uint64_t da = small_desc(base + S::kO + (k >> 2) * S::kAtom + (k & 3) * 32, 16);
                const uint64_t db = small_desc(base + S::kHi + k * 2048, S::kAtom);
                gemm::mma_f16<1>(tmem + 128, da, db, update_desc, k > 0);
            }
        });
        const float kx = p.ca + d_b[row];
        for (int c = share; c < chunks; c += 4) {
            float v[32];
            gemm::tmem_load32(lanes + 128 + 32 * c, v);
            gemm::Chunk16 h, l;
            load_pieces(hi, row, 32 * c, h);
            if (keeps_lo(step, p.steps)) {
                load_pieces(lo, row, 32 * c, l);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 r = gemm::pair_at(l, i, __half());
                    v[2 * i] = fmaf(kx, r.x, v[2 * i]);
                    v[2 * i + 1] = fmaf(kx, r.y, v[2 * i + 1]);
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 a = gemm::pair_at(h, i, __half());
                v[2 * i] = fmaf(kx, a.x, v[2 * i]);
                v[2 * i + 1] = fmaf(kx, a.y, v[2 * i + 1]);
            }
            if (step + 1 < p.steps) {
                if (keeps_lo(step + 1, p.steps)) {
                    split_halves(v, h, l);
                    store_pieces(lo, row, 32 * c, l);
                } else {
                    h = gemm::packed_row(v, __half());
                }
                store_pieces(hi, row, 32 * c, h);
            } else {
                // (the parts' buffer is free: no block sends to another any more)
                gemm::Place q;
                q.b = b;
                q.row0 = quarter * 32;
                q.col0 = j0 + 32 * c;
                q.M = p.r;
                q.N = p.c;
                q.lane = lane;
                q.off = false;
                q.stage = gen + S::kParts + warp * gemm::kWarpStage;
                if (q.row0 >= q.M || q.col0 >= q.N) continue;
                const float scale = p.scale * *unit;
                if (p.weights) {
                    float w[32];
                    if (p.tall)
                        gemm::get_columns(p.out, q, w);
                    else
                        gemm::get_rows(p.out, q, w);
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = fmaf(p.keep, w[j], scale * v[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] *= scale;
                }
                if (p.tall)
                    gemm::put_columns(p.out, q, v);
                else
                    gemm::put_rows(p.out, q, v);
            }
        }
    }
    gemm::tcgen05_fence_before();
    __syncthreads();
    gemm::tcgen05_fence_after();
    gemm::bury(dead, p.timeouts);
    if (warp == 1) gemm::tmem_free<1>(tmem, S::kTmemCols);
}

// Blocks of a cluster for a larger side of c: 0 where eight do not hold it.
inline int small_ranks(long long r, long long c) {
    if (r > Small::kRows) return 0;
    for (int ranks = 1; ranks <= Small::kMaxRanks; ranks *= 2)
        if (c <= (long long)ranks * Small::kMaxWidth) return ranks;
    return 0;
}

inline cudaError_t launch_small(SmallParams p, long long batch, int ranks, cudaStream_t st) {
    p.width = ((p.c + ranks - 1) / ranks + 63) / 64 * 64;
    p.timeouts = gemm::timeout_counter();
    if (p.timeouts == nullptr) return cudaErrorInvalidConfiguration;
    return gemm::launch_cluster(ns_small_kernel, (int)batch * ranks, Small::kThreads, ranks,
                                Small::kSmem, st, p, ranks);
}

}  // namespace train
}  // namespace vc
