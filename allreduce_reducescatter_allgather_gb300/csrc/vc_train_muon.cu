// Newton-Schulz orthogonalisation of matrices, and the Muon step around it.
//
// With r the smaller and c the larger side, one pass of the iteration is
//   A = X X^T        (r x r, symmetric: half of the tiles)
//   B = b A + c A^2  (r x r, symmetric)
//   X <- a X + B X   (r x c)
// on whichever side the smaller dimension is: a tall matrix uses X^T X and
// X B, which only changes which operands are K-major.
//
// Numbers.  The products' operands are fp16: their values are bounded (|X| at
// most about 1.2 in the spectral norm), so fp16's 11 significant bits are
// worth more than bf16's range.  Three measures keep the result near the exact
// iteration, beside 1.65e-3 of the norm for the bf16 rounding of the output:
// 4e-4 to 1e-3 off for matrices of full rank (bf16 operands: 2e-2 to 3e-2), 2.5e-3
// to 3.3e-3 for sums of few outer products (bf16: 0.1 to 1.9); 5e-3 was the worst
// (rank one of 96 rows, matrices of a few values).  What is left are the
// roundings of A and B, which coefficients of up to 4.8 raise in each pass:
//   - X is stored times a power of two near sqrt(c), so that its values are
//     about 1 at the end and normal fp16 numbers at the start (where eps
//     outweighs the norm: struct Start);
//   - the diagonals of A and B, which are far larger than the rest, are kept
//     apart in 32 bits; with A = D + O,
//       A^2 = D^2 + D O + O D + O^2,   B X = diag(B) X + offdiag(B) X;
//   - X itself is kept as a sum of two fp16 values, of which the a X and
//     diag(B) X terms use both and the products the larger one.  Without it,
//     directions with small singular values, which the iteration raises by
//     up to 500, would be raised from the rounding noise of the large ones.
//     In the last two passes, where what counts is near 1 and is raised no
//     more, the larger value does alone.
#include <algorithm>
#include <math.h>

#include "vc_ns_small.cuh"
#include "vc_train_common.cuh"

namespace vc {
namespace train {
namespace {

using gemm::Operand;
using gemm::Product;
using gemm::Shape;
using gemm::View;

// ---------------------------------------------------- momentum and scaling --

constexpr int kMaxParts = 1024;  // partial sums of squares per matrix

struct PrepareParams {
    View g, m;
    int has_momentum, nesterov;
    float beta;
    float* parts;  // [batch][gridDim.x]
    __half *hi, *lo;
    long long ld, batch_stride;  // of hi and lo
    float size, eps;             // X is stored times size
    int steps;
    float ca, cb, cc;
    Start* starts;               // of each matrix
    int rows, cols;
    int lanes;  // lanes that share a row, a power of two; 8 columns each at a time
};

// Eight consecutive values of a row: n of them are there.
struct Eight {
    float v[8];
};
__device__ __forceinline__ Eight load_eight(const View& x, int b, long long row, int col, int n) {
    Eight r;
    const long long at = (long long)b * x.batch_stride + row * x.ld + col;
    if (x.f32) {
        const float* p = static_cast<const float*>(x.data) + at;
        if (x.vec16 && n == 8) {
            const float4 lo = *reinterpret_cast<const float4*>(p);
            const float4 hi = *reinterpret_cast<const float4*>(p + 4);
            return {{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = j < n ? p[j] : 0.0f;
    } else {
        const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(x.data) + at;
        if (x.vec16 && n == 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                r.v[2 * j] = __uint_as_float(w[j] << 16);
                r.v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
            return r;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = j < n ? __bfloat162float(p[j]) : 0.0f;
    }
    return r;
}
// Stores them; r becomes what was stored.
__device__ __forceinline__ void store_eight(const View& x, int b, long long row, int col, int n,
                                            Eight& r) {
    const long long at = (long long)b * x.batch_stride + row * x.ld + col;
    if (x.f32) {
        float* p = static_cast<float*>(x.data) + at;
        if (x.vec16 && n == 8) {
            *reinterpret_cast<float4*>(p) = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
            *reinterpret_cast<float4*>(p + 4) = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) p[j] = r.v[j];
        }
    } else {
        __nv_bfloat16* p = static_cast<__nv_bfloat16*>(x.data) + at;
        unsigned w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = gemm::packed(r.v[2 * j], r.v[2 * j + 1], __nv_bfloat16());
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r.v[2 * j] = __uint_as_float(w[j] << 16);
            r.v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
        if (x.vec16 && n == 8) {
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) p[j] = __float2bfloat16(r.v[j]);
        }
    }
}

// beta m + g: the new momentum, or, with that for m, the Nesterov update.
__device__ __forceinline__ Eight axpy(float beta, const Eight& m, const Eight& g) {
    Eight r;
#pragma unroll
    for (int j = 0; j < 8; ++j) r.v[j] = fmaf(beta, m.v[j], g.v[j]);
    return r;
}

// A thread's groups of eight columns, one after the other: along the rows that
// its lanes take, `lanes` groups at a time.
struct Groups {
    int row, col, first_col, row_step, col_step;
    __device__ __forceinline__ explicit Groups(const PrepareParams& p) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = 32 / p.lanes;
        row = (blockIdx.x * 8 + warp) * per + lane / p.lanes;
        col = first_col = (lane % p.lanes) * 8;
        row_step = gridDim.x * 8 * per;
        col_step = p.lanes * 8;
    }
    __device__ __forceinline__ void next(const PrepareParams& p) {
        col += col_step;
        if (col >= p.cols) col = first_col, row += row_step;
    }
};

// Groups that a thread loads before it stores the first.
constexpr int kPrepareBatch = 2;

struct Loaded {
    Eight g, m;
    int row, col, n;  // n: values of the group, 0 beyond the matrix
};
__device__ __forceinline__ void load_batch(const PrepareParams& p, int b, Groups& at,
                                           Loaded (&x)[kPrepareBatch]) {
#pragma unroll
    for (int k = 0; k < kPrepareBatch; ++k) {
        x[k].row = at.row;
        x[k].col = at.col;
        x[k].n = at.row < p.rows ? max(0, min(8, p.cols - at.col)) : 0;
        if (x[k].n > 0) {
            x[k].g = load_eight(p.g, b, at.row, at.col, x[k].n);
            if (p.has_momentum) x[k].m = load_eight(p.m, b, at.row, at.col, x[k].n);
        }
        at.next(p);
    }
}

__device__ __forceinline__ float block_sum(float v, float* tmp) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += tmp[w];
    __syncthreads();
    return s;
}

// M <- beta M + G, and this block's part of the sum of the update's squares.
__global__ void __launch_bounds__(256) momentum_kernel(const __grid_constant__ PrepareParams p) {
    __shared__ float tmp[8];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.y;
    float sum = 0.0f;
    for (Groups at(p); at.row < p.rows;) {
        Loaded x[kPrepareBatch];
        load_batch(p, b, at, x);
#pragma unroll
        for (int k = 0; k < kPrepareBatch; ++k) {
            if (x[k].n == 0) continue;
            Eight u = x[k].g;
            if (p.has_momentum) {
                Eight m = axpy(p.beta, x[k].m, x[k].g);
                store_eight(p.m, b, x[k].row, x[k].col, x[k].n, m);
                u = p.nesterov ? axpy(p.beta, m, x[k].g) : m;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(u.v[j], u.v[j], sum);  // 0 beyond n
        }
    }
    sum = block_sum(sum, tmp);
    if (threadIdx.x == 0) p.parts[b * gridDim.x + blockIdx.x] = sum;
}

// X_0 = update size / (norm + eps), or what start_of makes of it, as two fp16
// values.  Every block adds up the partial sums, in the same order.
__global__ void __launch_bounds__(256) scale_kernel(const __grid_constant__ PrepareParams p) {
    __shared__ float tmp[8];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.y;
    float sum = 0.0f;
    for (unsigned i = threadIdx.x; i < gridDim.x; i += 256) sum += p.parts[b * gridDim.x + i];
    const Start start = start_of(block_sum(sum, tmp), p.eps, p.size, p.steps, p.ca, p.cb, p.cc);
    const float scale = start.scale;
    if (blockIdx.x == 0 && threadIdx.x == 0) p.starts[b] = start;
    for (Groups at(p); at.row < p.rows;) {
        Loaded x[kPrepareBatch];
        load_batch(p, b, at, x);
#pragma unroll
        for (int k = 0; k < kPrepareBatch; ++k) {
            if (x[k].n == 0) continue;
            const Eight u = !p.has_momentum ? x[k].g : p.nesterov ? axpy(p.beta, x[k].m, x[k].g) : x[k].m;
            unsigned hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = u.v[2 * j] * scale, c = u.v[2 * j + 1] * scale;
                hi[j] = gemm::packed(a, c, __half());
                const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi[j]));
                lo[j] = gemm::packed(a - h.x, c - h.y, __half());
            }
            // (rows of hi and lo are whole groups; what lies beyond n is read by nobody)
            const long long to = (long long)b * p.batch_stride + (long long)x[k].row * p.ld + x[k].col;
            *reinterpret_cast<uint4*>(p.hi + to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(p.lo + to) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
}

// ------------------------------------------------------------- epilogues --

using gemm::Place;

// Matrices in the workspace have rows of whole chunks (layout_of), so that
// chunks are accessed in 16-byte pieces whatever the matrix's size;
// what lies beyond the matrix is written with zeros and read by nobody.

// The mirrored chunk of a symmetric matrix, along its rows.
__device__ __forceinline__ void put_mirror(__half* o, long long ld, const Place& q,
                                           const float (&v)[32]) {
    if (!q.off || q.row() >= q.M) return;
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (q.col0 + j < q.N) o[(long long)(q.col0 + j) * ld + q.row()] = __float2half_rn(v[j]);
}

// The diagonal's value of this lane's row, if the chunk holds it (else 0); and
// sets it to zero in the chunk.
__device__ __forceinline__ float take_diagonal(const Place& q, float (&v)[32]) {
    float d = 0.0f;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        if (q.row() == q.col0 + j) {
            d = v[j];
            v[j] = 0.0f;
        }
    }
    return d;
}

// A = X X^T: the diagonal to 32 bits, the rest to fp16 on both sides.
struct EpiGram {
    static constexpr bool kSym = true;
    struct Params {
        __half* o;
        float* d;
        long long ld, batch_stride;
        float scale;
    };
    static bool odd(const Params&) { return false; }
    struct Pre {};
    __device__ static void prefetch(const Params&, const Place&, Pre&) {}
    __device__ static void apply(const Params& p, const Place& q, Pre&, float (&v)[32]) {
        __half* const o = p.o + (long long)q.b * p.batch_stride;
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= p.scale;
        if (q.row0 == q.col0) {
            const float d = take_diagonal(q, v);
            if (q.row() < q.M) p.d[(long long)q.b * q.M + q.row()] = d;
        }
        store_chunk(o + (long long)q.row0 * p.ld + q.col0, p.ld, q, v);
        put_mirror(o, p.ld, q, v);
    }
};

// B = b A + c A^2 from the product O O of A's off-diagonal part.
struct EpiPoly {
    static constexpr bool kSym = true;
    struct Params {
        const __half* o;
        const float* d;
        __half* ob;
        float* db;
        const Start* starts;
        long long ld, batch_stride;
        float ca, cb, cc;
        int step;
    };
    static bool odd(const Params&) { return false; }
    struct Pre {
        gemm::Chunk16 o;
        float row, col;  // A's diagonal at the lane's row and at its column
        int skip, linear;
    };
    __device__ static void prefetch(const Params& p, const Place& q, Pre& pre) {
        const float* const d = p.d + (long long)q.b * q.M;
        pre.col = q.col0 + q.lane < q.N ? d[q.col0 + q.lane] : 0.0f;
        pre.row = q.row() < q.M ? d[q.row()] : 0.0f;
        pre.skip = p.starts[q.b].skip;
        pre.linear = p.starts[q.b].linear;
        load_across(p.o + (long long)q.b * p.batch_stride + (long long)q.row0 * p.ld + q.col0, p.ld * 2,
                    q, pre.o);
    }
    __device__ static void apply(const Params& p, const Place& q, Pre& pre, float (&v)[32]) {
        __half* const ob = p.ob + (long long)q.b * p.batch_stride;
        // a pass that is left out: a + B = 1; a linear one: B = 0
        const bool none = p.step < pre.linear;
        const float cb = none ? 0.0f : p.cb, cc = none ? 0.0f : p.cc;
        if (q.row0 == q.col0) {
            const float d = take_diagonal(q, v);  // (O O)_ii
            if (q.row() < q.M)
                p.db[(long long)q.b * q.M + q.row()] =
                    p.step < pre.skip ? 1.0f - p.ca : cb * pre.row + cc * (pre.row * pre.row + d);
        }
        across_to_own(q, pre.o);
        const float k = fmaf(cc, pre.row, cb);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 a = pair_at(pre.o, i, __half());  // (0 on the diagonal)
            const float k0 = fmaf(cc, __shfl_sync(0xFFFFFFFFu, pre.col, 2 * i), k);
            const float k1 = fmaf(cc, __shfl_sync(0xFFFFFFFFu, pre.col, 2 * i + 1), k);
            v[2 * i] = fmaf(k0, a.x, cc * v[2 * i]);
            v[2 * i + 1] = fmaf(k1, a.y, cc * v[2 * i + 1]);
        }
        store_chunk(ob + (long long)q.row0 * p.ld + q.col0, p.ld, q, v);
        put_mirror(ob, p.ld, q, v);
    }
};

// X <- (a + diag B) X + offdiag(B) X, and on the last pass the operator's
// output instead of X.
struct UpdateParams {
    const __half* hi;
    __half* lo;
    __half* hi_out;
    const float* db;  // diagonal of B, [batch][r]
    long long ld, batch_stride;
    float a;
    int tall;  // B stands on the right: its diagonal goes with the columns
    int r;
    int read_lo, write_lo;
};
struct UpdatePre {
    gemm::Chunk16 hi, lo;
    float k;  // a + B's diagonal at the lane's row, or at its column (tall)
};
__device__ __forceinline__ void update_prefetch(const UpdateParams& p, const Place& q, UpdatePre& pre) {
    const int at = p.tall ? q.col0 + q.lane : q.row();
    pre.k = at < p.r ? p.a + p.db[(long long)q.b * p.r + at] : 0.0f;
    const long long x = (long long)q.b * p.batch_stride + (long long)q.row0 * p.ld + q.col0;
    load_across(p.hi + x, p.ld * 2, q, pre.hi);
    if (p.read_lo) load_across(p.lo + x, p.ld * 2, q, pre.lo);
}
__device__ __forceinline__ void update_apply(const UpdateParams& p, const Place& q, UpdatePre& pre,
                                             float (&v)[32]) {
    across_to_own(q, pre.hi);
    if (p.read_lo) across_to_own(q, pre.lo);
    auto add = [&](bool with_lo) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float2 x = pair_at(pre.hi, i, __half());
            if (with_lo) x = gemm::add2(x, pair_at(pre.lo, i, __half()));
            const float k0 = p.tall ? __shfl_sync(0xFFFFFFFFu, pre.k, 2 * i) : pre.k;
            const float k1 = p.tall ? __shfl_sync(0xFFFFFFFFu, pre.k, 2 * i + 1) : pre.k;
            v[2 * i] = fmaf(k0, x.x, v[2 * i]);
            v[2 * i + 1] = fmaf(k1, x.y, v[2 * i + 1]);
        }
    };
    p.read_lo ? add(true) : add(false);
}

struct EpiUpdate {
    static constexpr bool kSym = false;
    using Params = UpdateParams;
    static bool odd(const Params&) { return false; }
    using Pre = UpdatePre;
    __device__ static void prefetch(const Params& p, const Place& q, Pre& pre) {
        update_prefetch(p, q, pre);
    }
    __device__ static void apply(const Params& p, const Place& q, Pre& pre, float (&v)[32]) {
        update_apply(p, q, pre, v);
        const long long at = (long long)q.b * p.batch_stride + (long long)q.row0 * p.ld + q.col0;
        store_chunk(p.hi_out + at, p.ld, q, v);
        if (!p.write_lo) return;
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] -= __half2float(__float2half_rn(v[j]));
        store_chunk(p.lo + at, p.ld, q, v);
    }
};

struct EpiFinal {
    static constexpr bool kSym = false;
    struct Params {
        UpdateParams u;
        View out;     // the output, or the weights
        int weights;  // out <- keep out + scale y, else out <- scale y
        float keep, scale;
        const Start* starts;
    };
    static bool odd(const Params& p) { return !p.out.vec16; }
    struct Pre : UpdatePre {
        float unit;
    };
    __device__ static void prefetch(const Params& p, const Place& q, Pre& pre) {
        update_prefetch(p.u, q, pre);
        pre.unit = p.starts[q.b].unit;
    }
    __device__ static void apply(const Params& p, const Place& q, Pre& pre, float (&v)[32]) {
        update_apply(p.u, q, pre, v);
        const float scale = p.scale * pre.unit;
        if (p.weights) {
            float w[32];
            get_rows(p.out, q, w);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = fmaf(p.keep, w[j], scale * v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] *= scale;
        }
        put_rows(p.out, q, v);
    }
};

// -------------------------------------------------------------- host side --

struct Layout {
    long long r, c;        // smaller and larger side
    long long ldx, ldr;    // row lengths of X and of the r x r matrices
    long long xs, as;      // values from one matrix of the batch to the next
    int parts, lanes;
    size_t hi0, hi1, lo, a, b, da, db, sums, starts, bytes;
};

bool layout_of(long long batch, long long rows, long long cols, Layout* l) {
    if (batch < 0 || rows < 0 || cols < 0) return false;
    if (batch > (1 << 16) - 1 || rows > (1ll << 24) || cols > (1ll << 24)) return false;
    if (batch * rows > 0x3FFFFFFFll) return false;
    l->r = std::min(rows, cols);
    l->c = std::max(rows, cols);
    l->ldx = padded_ld(cols);  // whole chunks of the epilogues, too
    l->ldr = padded_ld(l->r);
    l->xs = rows * l->ldx;
    l->as = l->r * l->ldr;
    l->lanes = 1;
    while (l->lanes < 32 && l->lanes * 8 < cols) l->lanes *= 2;
    const long long per_block = 8 * (32 / l->lanes);  // rows
    // up to 8 blocks per SM over the batch
    const long long want = (rows + per_block - 1) / per_block;
    const long long fit = std::max(1ll, 152 * 8 / std::max(1ll, batch));
    l->parts = (int)std::max(1ll, std::min({want, fit, (long long)kMaxParts}));
    const size_t x = round256((size_t)batch * l->xs * 2), a = round256((size_t)batch * l->as * 2);
    const size_t d = round256((size_t)batch * l->r * 4);
    size_t at = 0;
    l->hi0 = at, at += x;
    l->hi1 = at, at += x;
    l->lo = at, at += x;
    l->a = at, at += a;
    l->b = at, at += a;
    l->da = at, at += d;
    l->db = at, at += d;
    l->sums = at, at += round256((size_t)batch * l->parts * 4);
    l->starts = at, at += round256((size_t)batch * sizeof(Start));
    l->bytes = at;
    return true;
}

bool valid_ns(const vc_newton_schulz_t* ns) {
    return ns != nullptr && ns->steps >= 1 && ns->steps <= 100 && isfinite(ns->a) &&
           isfinite(ns->b) && isfinite(ns->c) && isfinite(ns->eps) && ns->eps >= 0.0f;
}

// The whole iteration; ends in `fin` (out, weights, keep, scale set).
cudaError_t iterate(const Layout& l, long long batch, long long rows, long long cols,
                    PrepareParams p, const vc_newton_schulz_t& ns, EpiFinal::Params fin,
                    unsigned char* ws, cudaStream_t st) {
    const bool tall = rows > cols;
    int e2 = 0;  // X is stored times 2^e2, about sqrt(c)
    while (e2 < 12 && (1ll << (2 * e2)) < l.c) ++e2;
    const float size = (float)(1 << e2);
    if (const int ranks = small_ranks(l.r, l.c)) {
        SmallParams sp = {};
        sp.g = p.g;
        sp.m = p.m;
        sp.out = fin.out;
        sp.has_momentum = p.has_momentum;
        sp.nesterov = p.nesterov;
        sp.weights = fin.weights;
        sp.tall = tall;
        sp.r = (int)l.r;
        sp.c = (int)l.c;
        sp.steps = ns.steps;
        sp.beta = p.beta;
        sp.eps = ns.eps;
        sp.ca = ns.a;
        sp.cb = ns.b;
        sp.cc = ns.c;
        sp.size = size;
        sp.keep = fin.keep;
        sp.scale = fin.scale / size;
        return launch_small(sp, batch, ranks, st);
    }
    __half* x[2] = {reinterpret_cast<__half*>(ws + l.hi0), reinterpret_cast<__half*>(ws + l.hi1)};
    __half *const lo = reinterpret_cast<__half*>(ws + l.lo), *const oa = reinterpret_cast<__half*>(ws + l.a),
                  *const ob = reinterpret_cast<__half*>(ws + l.b);
    float *const da = reinterpret_cast<float*>(ws + l.da), *const db = reinterpret_cast<float*>(ws + l.db);
    p.parts = reinterpret_cast<float*>(ws + l.sums);
    p.hi = x[0];
    p.lo = lo;
    p.ld = l.ldx;
    p.batch_stride = l.xs;
    p.size = size;
    p.eps = ns.eps;
    p.steps = ns.steps;
    p.ca = ns.a;
    p.cb = ns.b;
    p.cc = ns.c;
    p.starts = reinterpret_cast<Start*>(ws + l.starts);
    p.rows = (int)rows;
    p.cols = (int)cols;
    p.lanes = l.lanes;
    const dim3 grid(l.parts, (unsigned)batch);
    cudaError_t e = launch_pdl(momentum_kernel, grid, dim3(256), st, p);
    if (e == cudaSuccess) e = launch_pdl(scale_kernel, grid, dim3(256), st, p);
    const int r = (int)l.r, c = (int)l.c, nb = (int)batch;
    for (int i = 0; i < ns.steps && e == cudaSuccess; ++i) {
        const Operand xk = {x[0], cols, rows, l.ldx, l.xs, false, false};
        Operand xm = xk;
        xm.mn_major = true;
        EpiGram::Params gp = {oa, da, l.ldr, l.as, 1.0f / (size * size)};
        const Operand& side = tall ? xm : xk;
        e = gemm::launch<EpiGram>(Product{side, side, r, r, c, nb, 1}, gp, st);
        if (e != cudaSuccess) break;
        const Operand ao = {oa, r, r, l.ldr, l.as, false, false};
        EpiPoly::Params pp = {oa, da, ob, db, p.starts, l.ldr, l.as, ns.a, ns.b, ns.c, i};
        e = gemm::launch<EpiPoly>(Product{ao, ao, r, r, r, nb, 1}, pp, st);
        if (e != cudaSuccess) break;
        const Operand bo = {ob, r, r, l.ldr, l.as, false, false};
        const UpdateParams u = {x[0], lo, x[1], db, l.ldx, l.xs, ns.a, tall, r, keeps_lo(i, ns.steps),
                                keeps_lo(i + 1, ns.steps)};
        const Operand &left = tall ? xk : bo, &right = tall ? bo : xm;
        if (i + 1 < ns.steps) {
            e = gemm::launch<EpiUpdate>(Product{left, right, (int)rows, (int)cols, r, nb, 1}, u, st);
        } else {
            fin.u = u;
            fin.scale /= size;
            fin.starts = p.starts;
            e = gemm::launch<EpiFinal>(Product{left, right, (int)rows, (int)cols, r, nb, 1}, fin, st);
        }
        std::swap(x[0], x[1]);
    }
    return e;
}

bool same_sizes(const vc_matrix_t* a, const vc_matrix_t* b) {
    return a->batch == b->batch && a->rows == b->rows && a->cols == b->cols;
}

bool workspace_ok(const void* ws, size_t have, size_t need) {
    return ws != nullptr && (reinterpret_cast<uintptr_t>(ws) & 255) == 0 && have >= need;
}

}  // namespace
}  // namespace train
}  // namespace vc

using namespace vc;
using namespace vc::train;

extern "C" {

size_t vc_orthogonalize_workspace(long long batch, long long rows, long long cols) {
    Layout l;
    if (!layout_of(batch, rows, cols, &l)) return 0;
    return batch == 0 || rows == 0 || cols == 0 ? 0 : l.bytes;
}

vc_status_t vc_orthogonalize(const vc_matrix_t* g, const vc_matrix_t* out,
                             const vc_newton_schulz_t* ns, void* workspace, size_t workspace_bytes,
                             vc_stream_t stream) {
    if (!valid_matrix(g) || !valid_matrix(out) || !same_sizes(g, out) ||
        out->dtype != VC_BFLOAT16 || !valid_ns(ns))
        return VC_ERR_INVALID_ARGUMENT;
    Layout l;
    if (!layout_of(g->batch, g->rows, g->cols, &l)) return VC_ERR_INVALID_ARGUMENT;
    if (g->batch == 0 || g->rows == 0 || g->cols == 0) return VC_SUCCESS;
    if (!workspace_ok(workspace, workspace_bytes, l.bytes)) return VC_ERR_INVALID_ARGUMENT;
    const Span ws = span_of(workspace, l.bytes);
    if ((overlap(span_of(g), span_of(out)) && !same_matrix(g, out)) || overlap(span_of(g), ws) ||
        overlap(span_of(out), ws))
        return VC_ERR_ALIAS;
    if (test_launch_failure()) return VC_ERR_CUDA;
    PrepareParams p = {};
    p.g = view_of(g);
    EpiFinal::Params fin = {};
    fin.out = view_of(out);
    fin.scale = 1.0f;
    const cudaError_t e = iterate(l, g->batch, g->rows, g->cols, p, *ns, fin,
                                  static_cast<unsigned char*>(workspace),
                                  static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? VC_SUCCESS : VC_ERR_CUDA;
}

vc_status_t vc_muon_step(const vc_matrix_t* weight, const vc_matrix_t* grad,
                         const vc_matrix_t* momentum, const vc_muon_t* args, void* workspace,
                         size_t workspace_bytes, vc_stream_t stream) {
    if (!valid_matrix(weight) || !valid_matrix(grad) || !valid_matrix(momentum) ||
        args == nullptr || !same_sizes(weight, grad) || !same_sizes(weight, momentum) ||
        !valid_ns(&args->ns) || !isfinite(args->lr) || !isfinite(args->beta) ||
        !isfinite(args->weight_decay) || !isfinite(args->scale))
        return VC_ERR_INVALID_ARGUMENT;
    Layout l;
    if (!layout_of(grad->batch, grad->rows, grad->cols, &l)) return VC_ERR_INVALID_ARGUMENT;
    if (grad->batch == 0 || grad->rows == 0 || grad->cols == 0) return VC_SUCCESS;
    if (!workspace_ok(workspace, workspace_bytes, l.bytes)) return VC_ERR_INVALID_ARGUMENT;
    const Span s[4] = {span_of(weight), span_of(grad), span_of(momentum), span_of(workspace, l.bytes)};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(s[i], s[j])) return VC_ERR_ALIAS;
    if (test_launch_failure()) return VC_ERR_CUDA;
    PrepareParams p = {};
    p.g = view_of(grad);
    p.m = view_of(momentum);
    p.has_momentum = 1;
    p.nesterov = args->nesterov != 0;
    p.beta = args->beta;
    EpiFinal::Params fin = {};
    fin.out = view_of(weight);
    fin.weights = 1;
    fin.keep = 1.0f - args->lr * args->weight_decay;
    fin.scale = -args->lr * args->scale;
    const cudaError_t e = iterate(l, grad->batch, grad->rows, grad->cols, p, args->ns, fin,
                                  static_cast<unsigned char*>(workspace),
                                  static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? VC_SUCCESS : VC_ERR_CUDA;
}

}  // extern "C"
