// vc_embedding_forward / vc_embedding_backward: rows of a table looked up by
// token, and the sum of the tokens' gradients by row.
//
// Forward: y_t = s W[id_t - first].  One 16-byte vector of a row a thread, four
// of them in flight; bound by the bytes of y and of the rows.
//
// Backward: dW_v (+)= s sum_{t: row(t) = v} dy_t in three launches, none of which
// adds to memory that another block may add to:
//
//   sort   one cluster of blocks sorts (row, token) by row, keeping the tokens of a
//          row in order: a radix sort of up to 9 bits a pass, whose ranks come from
//          the lanes of a warp that share a digit, whose counts go through
//          distributed shared memory.  It is bound by latency and needs few SMs; the
//          other blocks of the same launch meanwhile write zeros to the rows that no
//          token has (each marks the tokens of its own rows first).
//   sum    every warp takes a window of neighbours in the sorted order and 256
//          columns: as many rows of dy to each, whatever the ids are.  Rows whose
//          tokens all lie in the window are stored, the first and the last one,
//          where they go on beyond it, left as partial sums.
//   join   adds the partial sums of rows that span windows, in order.
#include <algorithm>

#include "vc_step_common.cuh"

namespace vc {
namespace step {
namespace {

__device__ __forceinline__ long long load_id(const void* ids, int wide, long long t) {
    return wide ? static_cast<const long long*>(ids)[t] : (long long)static_cast<const int*>(ids)[t];
}

// ------------------------------------------------------------------ forward --

struct LookupParams {
    const void* ids;
    int wide;  // 64-bit ids
    Rows weight, out;
    long long first, units;
    unsigned long long rows;
    int cols, per_row;  // units of a row
    float scale;
};

// kVec: a unit is eight columns on 16 bytes (fewer at a row's end), else one.
template <int kUnits, bool kVec>
__global__ void __launch_bounds__(256) lookup_kernel(const __grid_constant__ LookupParams p) {
    pdl_next();
    pdl_wait();
    const long long base = (long long)blockIdx.x * (256 * kUnits);
    const long long t0 = base / p.per_row;
    const unsigned c0 = (unsigned)(base - t0 * p.per_row);
    long long token[kUnits];
    unsigned long long row[kUnits];  // (below the table's start: far above its end)
    int col[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const unsigned at = u * 256 + threadIdx.x, c = c0 + at, t = c / (unsigned)p.per_row;
        token[u] = base + at < p.units ? t0 + t : -1;
        col[u] = (int)(c - t * p.per_row) * (kVec ? 8 : 1);
        row[u] = token[u] >= 0 ? (unsigned long long)load_id(p.ids, p.wide, token[u]) -
                                     (unsigned long long)p.first
                               : ~0ull;
    }
    Eight v[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const bool in = row[u] < p.rows;
        const long long at = (in ? (long long)row[u] : 0) * p.weight.ld + col[u];
        const float* f = static_cast<const float*>(p.weight.data) + at;
        const __nv_bfloat16* b = static_cast<const __nv_bfloat16*>(p.weight.data) + at;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[u].v[j] = 0.0f;
        if (!in) continue;
        if constexpr (kVec) {
            const int n = p.cols - col[u];
            if (n >= 8 && p.weight.f32) {
                const float4 a = reinterpret_cast<const float4*>(f)[0];
                const float4 c = reinterpret_cast<const float4*>(f)[1];
                v[u] = {{a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w}};
            } else if (n >= 8) {
                v[u] = widen(*reinterpret_cast<const uint4*>(b));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < n) v[u].v[j] = p.weight.f32 ? f[j] : __bfloat162float(b[j]);
            }
        } else {
            v[u].v[0] = p.weight.f32 ? *f : __bfloat162float(*b);
        }
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        if (token[u] < 0) continue;
        const bool in = row[u] < p.rows;
        const long long at = token[u] * p.out.ld + col[u];
        float* f = static_cast<float*>(p.out.data) + at;
        __nv_bfloat16* b = static_cast<__nv_bfloat16*>(p.out.data) + at;
        Eight r;
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = in ? v[u].v[j] * p.scale : 0.0f;
        if constexpr (kVec) {
            const int n = p.cols - col[u];
            if (n >= 8 && p.out.f32) {
                reinterpret_cast<float4*>(f)[0] = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
                reinterpret_cast<float4*>(f)[1] = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
            } else if (n >= 8) {
                *reinterpret_cast<uint4*>(b) = narrow(r);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < n) {
                        if (p.out.f32)
                            f[j] = r.v[j];
                        else
                            b[j] = __float2bfloat16(r.v[j]);
                    }
            }
        } else if (p.out.f32) {
            *f = r.v[0];
        } else {
            *b = __float2bfloat16(r.v[0]);
        }
    }
}

// --------------------------------------------------------- sorting by row --

constexpr int kCluster = 8;         // blocks that sort
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kItems = 8;           // of a thread at a time
constexpr int kChunk = kSortThreads * kItems;
constexpr int kDigitBits = 9, kBins = 1 << kDigitBits;
constexpr int kMarkRows = 16384;    // rows that a block marks at a time

struct SortParams {
    const void* ids;
    int wide;
    long long first, padding;  // padding < 0: none
    unsigned rows;             // also the key of tokens that are left out
    int tokens, passes, bits;  // bits of a pass
    uint2 *a, *b;              // (row, token); the last pass writes a
    // the rows that no token has are set to zero, by the blocks that do not sort
    char* out;
    long long row_bytes, pitch;
    int vec;                   // rows on 16 bytes
};

__device__ __forceinline__ unsigned key_of(const SortParams& p, int t) {
    const long long id = load_id(p.ids, p.wide, t);
    const unsigned long long row = (unsigned long long)id - (unsigned long long)p.first;
    const bool live = row < p.rows && (p.padding < 0 || id != p.padding);
    return live ? (unsigned)row : p.rows;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
}
__device__ __forceinline__ unsigned remote_load(const unsigned* at, int rank) {
    unsigned address, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(address) : "r"((unsigned)__cvta_generic_to_shared(at)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(address) : "memory");
    return v;
}

struct SortShared {
    unsigned short count[kSortWarps][kBins];  // of a warp, then of the warps before
    unsigned chunk[kBins], total[kBins], base[kBins], scan[32];
};

// Ranks the chunk's items among those of their warp with the same digit, and leaves
// the counts of the warps before each in count[][], the chunk's in chunk[].
__device__ void rank_chunk(SortShared& s, const uint2 (&item)[kItems], int begin, int end, int shift,
                           unsigned mask, int (&rank)[kItems]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kSortWarps * kBins / 2; i += kSortThreads)
        reinterpret_cast<unsigned*>(s.count)[i] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const bool live = begin + warp * (kItems * 32) + k * 32 + lane < end;
        const unsigned digit = live ? (item[k].x >> shift) & mask : kBins;
        const unsigned same = __match_any_sync(~0u, digit);
        const int before = live ? s.count[warp][digit] : 0;
        rank[k] = before + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (live && (same & ((1u << lane) - 1)) == 0)
            s.count[warp][digit] = (unsigned short)(before + __popc(same));
        __syncwarp();
    }
    __syncthreads();
    if (threadIdx.x <= mask) {
        unsigned sum = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const unsigned n = s.count[w][threadIdx.x];
            s.count[w][threadIdx.x] = (unsigned short)sum;
            sum += n;
        }
        s.chunk[threadIdx.x] = sum;
    }
    __syncthreads();
}

__device__ void sort_tokens(const SortParams& p, SortShared& s) {
    const int me = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int each = (p.tokens + kCluster - 1) / kCluster;
    const int lo = min((long long)p.tokens, (long long)me * each);
    const int hi = min((long long)p.tokens, (long long)(me + 1) * each);
    const bool once = each <= kChunk;
    const unsigned mask = (1u << p.bits) - 1;
    for (int pass = 0; pass < p.passes; ++pass) {
        // the last pass writes a
        const bool into_a = ((p.passes - 1 - pass) & 1) == 0;
        const uint2* from = into_a ? p.b : p.a;
        uint2* to = into_a ? p.a : p.b;
        const int shift = pass * p.bits;
        uint2 item[kItems];
        int rank[kItems];
        auto load = [&](int begin) {
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                const int i = begin + warp * (kItems * 32) + k * 32 + lane;
                if (i >= hi)
                    item[k] = make_uint2(0, 0);
                else
                    item[k] = pass == 0 ? make_uint2(key_of(p, i), i) : __ldcg(from + i);
            }
        };
        if (threadIdx.x <= mask) s.total[threadIdx.x] = 0;
        for (int begin = lo; begin < hi || (once && begin == lo); begin += kChunk) {
            load(begin);
            rank_chunk(s, item, begin, hi, shift, mask, rank);
            if (threadIdx.x <= mask) s.total[threadIdx.x] += s.chunk[threadIdx.x];
            if (once) break;
        }
        cluster_sync();
        // where each digit of this block starts: behind all smaller ones, and
        // behind those of the blocks before
        unsigned all = 0, before = 0;
        if (threadIdx.x <= mask) {
#pragma unroll
            for (int c = 0; c < kCluster; ++c) {
                const unsigned n = remote_load(&s.total[threadIdx.x], c);
                all += n;
                before += c < me ? n : 0;
            }
        }
        unsigned sum = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned n = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += n;
        }
        if (lane == 31) s.scan[warp] = sum;
        __syncthreads();
        unsigned smaller = 0;
        for (int w = 0; w < kBins / 32; ++w) smaller += w < warp ? s.scan[w] : 0;
        if (threadIdx.x <= mask) s.base[threadIdx.x] = smaller + sum - all + before;
        __syncthreads();
        for (int begin = lo; begin < hi; begin += kChunk) {
            if (!once) {
                load(begin);
                rank_chunk(s, item, begin, hi, shift, mask, rank);
            }
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                if (begin + warp * (kItems * 32) + k * 32 + lane >= hi) continue;
                const unsigned digit = (item[k].x >> shift) & mask;
                const unsigned at = s.base[digit] + s.count[warp][digit] + rank[k];
                if (at < (unsigned)p.tokens) __stcg(to + at, item[k]);  // (ids that change meanwhile)
            }
            if (!once) {
                __syncthreads();
                if (threadIdx.x <= mask) s.base[threadIdx.x] += s.chunk[threadIdx.x];
            }
        }
        // what was written is read by other blocks; totals are rewritten
        __threadfence();
        cluster_sync();
    }
}

// Zeros to those of this block's rows that no token has.
__device__ void fill_rows(const SortParams& p, unsigned* marks, int part, int parts) {
    const unsigned lo = (unsigned)((unsigned long long)p.rows * part / parts);
    const unsigned hi = (unsigned)((unsigned long long)p.rows * (part + 1) / parts);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (unsigned at = lo; at < hi; at += kMarkRows) {
        const unsigned n = min(hi - at, (unsigned)kMarkRows);
        for (int i = threadIdx.x; i < kMarkRows / 32; i += kSortThreads) marks[i] = 0;
        __syncthreads();
        for (int t0 = 0; t0 < p.tokens; t0 += kSortThreads * kItems) {
            unsigned key[kItems];
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                const int t = t0 + k * kSortThreads + threadIdx.x;
                key[k] = t < p.tokens ? key_of(p, t) : p.rows;
            }
#pragma unroll
            for (int k = 0; k < kItems; ++k)
                if (key[k] - at < n) atomicOr(&marks[(key[k] - at) >> 5], 1u << ((key[k] - at) & 31));
        }
        __syncthreads();
        for (unsigned i = warp; i < n; i += kSortWarps) {
            if (marks[i >> 5] >> (i & 31) & 1) continue;
            char* row = p.out + (long long)(at + i) * p.pitch;
            long long done = 0;
            if (p.vec) {
                done = p.row_bytes & ~15ll;
                for (long long c = lane * 16; c < done; c += 512)
                    *reinterpret_cast<uint4*>(row + c) = make_uint4(0, 0, 0, 0);
            }
            for (long long c = done + lane * 2; c < p.row_bytes; c += 64)
                *reinterpret_cast<unsigned short*>(row + c) = 0;
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kSortThreads, 1) __cluster_dims__(kCluster, 1, 1)
    sort_kernel(const __grid_constant__ SortParams p) {
    __shared__ SortShared s;
    pdl_next();
    pdl_wait();
    if (blockIdx.x < kCluster)
        sort_tokens(p, s);
    else
        fill_rows(p, reinterpret_cast<unsigned*>(&s), blockIdx.x - kCluster, gridDim.x - kCluster);
}
static_assert(sizeof(SortShared) >= kMarkRows / 8, "a block's marks fit");

// ------------------------------------------------------------ sums by row --

constexpr int kSlice = 256;  // columns of a warp
constexpr int kSumWarps = 4;

struct SumParams {
    const uint2* sorted;
    Rows dy, dw;
    float* parts;  // [window][2][padded columns]: the first and the last row's
    long long padded;
    unsigned rows;
    int tokens, windows, slices, cols, accumulate;
    float scale;
};

// Eight columns of a row: neighbours on 16 bytes, or every 32nd one.
template <bool kVec>
__device__ __forceinline__ Eight load_row(const Rows& x, long long row, int c0, int lane, int cols) {
    const long long at = row * x.ld + c0;
    const float* f = static_cast<const float*>(x.data) + at;
    const __nv_bfloat16* b = static_cast<const __nv_bfloat16*>(x.data) + at;
    Eight r;
    if constexpr (kVec) {
        const int c = lane * 8;
        if (c0 + c + 8 <= cols) {
            if (x.f32) {
                const float4 lo = *reinterpret_cast<const float4*>(f + c),
                             hi = *reinterpret_cast<const float4*>(f + c + 4);
                return {{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
            }
            return widen(*reinterpret_cast<const uint4*>(b + c));
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = kVec ? lane * 8 + j : j * 32 + lane;
        r.v[j] = c0 + c < cols ? (x.f32 ? f[c] : __bfloat162float(b[c])) : 0.0f;
    }
    return r;
}
template <bool kVec>
__device__ __forceinline__ void store_row(const Rows& x, long long row, int c0, int lane, int cols,
                                          const Eight& r) {
    const long long at = row * x.ld + c0;
    float* f = static_cast<float*>(x.data) + at;
    __nv_bfloat16* b = static_cast<__nv_bfloat16*>(x.data) + at;
    if constexpr (kVec) {
        const int c = lane * 8;
        if (c0 + c + 8 <= cols) {
            if (x.f32) {
                *reinterpret_cast<float4*>(f + c) = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
                *reinterpret_cast<float4*>(f + c + 4) = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
            } else {
                *reinterpret_cast<uint4*>(b + c) = narrow(r);
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = kVec ? lane * 8 + j : j * 32 + lane;
        if (c0 + c >= cols) continue;
        if (x.f32)
            f[c] = r.v[j];
        else
            b[c] = __float2bfloat16(r.v[j]);
    }
}

// dW row (+)= scale * sum
template <bool kVec>
__device__ __forceinline__ void finish_row(const SumParams& p, unsigned row, int c0, int lane,
                                           const Eight& sum) {
    Eight r;
    if (p.accumulate) {
        r = load_row<kVec>(p.dw, row, c0, lane, p.cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = fmaf(p.scale, sum.v[j], r.v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = p.scale * sum.v[j];
    }
    store_row<kVec>(p.dw, row, c0, lane, p.cols, r);
}

__device__ __forceinline__ float* part_at(const SumParams& p, int window, int last, int c0, int lane) {
    return p.parts + ((long long)window * 2 + last) * p.padded + c0 + lane * 8;
}

template <int kWindow, bool kVec>
__global__ void __launch_bounds__(kSumWarps * 32) sum_kernel(const __grid_constant__ SumParams p) {
    constexpr int kBatch = 8;  // rows in flight
    pdl_next();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * kSumWarps + (threadIdx.x >> 5);
    const int window = (int)(unit / p.slices), c0 = (int)(unit - (long long)window * p.slices) * kSlice;
    if (window >= p.windows) return;
    const int begin = window * kWindow;
    const uint2 none = make_uint2(p.rows, 0);
    uint2 mine[(kWindow + 31) / 32];
#pragma unroll
    for (int i = 0; i < (kWindow + 31) / 32; ++i) {
        const int t = begin + i * 32 + lane;
        mine[i] = i * 32 + lane < kWindow && t < p.tokens ? p.sorted[t] : none;
    }
    const unsigned before = begin > 0 ? p.sorted[begin - 1].x : p.rows;
    const unsigned after = p.tokens - begin > kWindow ? p.sorted[begin + kWindow].x : p.rows;
    Eight sum;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum.v[j] = 0.0f;
    unsigned row = __shfl_sync(~0u, mine[0].x, 0);
    bool first = true;
    auto flush = [&](bool end) {
        if (row >= p.rows) return;
        const bool from = first && row == before, on = end && row == after;
        if (from || on) {
            float4* to = reinterpret_cast<float4*>(part_at(p, window, from ? 0 : 1, c0, lane));
            to[0] = make_float4(sum.v[0], sum.v[1], sum.v[2], sum.v[3]);
            to[1] = make_float4(sum.v[4], sum.v[5], sum.v[6], sum.v[7]);
        } else {
            finish_row<kVec>(p, row, c0, lane, sum);
        }
    };
#pragma unroll 1
    for (int b = 0; b < kWindow; b += kBatch) {
        Eight v[kBatch];
        unsigned key[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const uint2 from = kWindow > 32 && b >= 32 ? mine[(kWindow + 31) / 32 - 1] : mine[0];
            key[i] = __shfl_sync(~0u, from.x, (b + i) & 31);
            const unsigned token = __shfl_sync(~0u, from.y, (b + i) & 31);
            if (key[i] < p.rows) v[i] = load_row<kVec>(p.dy, token, c0, lane, p.cols);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (key[i] != row) {
                flush(false);
                first = false;
                row = key[i];
#pragma unroll
                for (int j = 0; j < 8; ++j) sum.v[j] = 0.0f;
            }
            if (row < p.rows) {
#pragma unroll
                for (int j = 0; j < 8; ++j) sum.v[j] += v[i].v[j];
            }
        }
    }
    flush(true);
}

// A row that starts in one window and goes on into others: its last partial sum
// there and the first ones of the windows behind, by the warps of a block in
// turn.  Blocks look for such rows among their windows.
constexpr int kJoinWarps = 8, kJoinThreads = kJoinWarps * 32;

template <int kWindow, bool kVec>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ SumParams p) {
    __shared__ int found[kJoinThreads + 1];
    __shared__ int behind;
    __shared__ float4 shared[kJoinWarps][64];
    pdl_next();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = blockIdx.x * kSlice;
    const int lo = (int)((long long)p.windows * blockIdx.y / gridDim.y);
    const int hi = (int)((long long)p.windows * (blockIdx.y + 1) / gridDim.y);
    auto key = [&](int window, int i) { return p.sorted[(long long)window * kWindow + i].x; };
    for (int w0 = lo; w0 < hi; w0 += kJoinThreads) {
        const int w = w0 + threadIdx.x;
        bool starts = false;
        if (w < hi && w + 1 < p.windows) {
            const unsigned last = key(w, kWindow - 1);
            starts = last < p.rows && key(w + 1, 0) == last &&
                     !(key(w, 0) == last && w > 0 && p.sorted[(long long)w * kWindow - 1].x == last);
        }
        if (threadIdx.x == 0) found[kJoinThreads] = 0;
        __syncthreads();
        // (which slot a window gets changes nothing but the order of work)
        if (starts) found[atomicAdd(&found[kJoinThreads], 1)] = w;
        __syncthreads();
        const int n = found[kJoinThreads];
        for (int f = 0; f < n; ++f) {
            const int start = found[f];
            const unsigned row = key(start, kWindow - 1);
            // windows behind that go on with the row
            int ends = p.windows;
            for (int u0 = start + 1; u0 < p.windows; u0 += kJoinThreads) {
                __syncthreads();
                if (threadIdx.x == 0) behind = p.windows;
                __syncthreads();
                const int u = u0 + threadIdx.x;
                if (u < p.windows && key(u, 0) != row) atomicMin(&behind, u);
                __syncthreads();
                ends = behind;
                if (ends < p.windows) break;
            }
            Eight sum;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum.v[j] = 0.0f;
#pragma unroll 4
            for (int u = start + warp; u < ends; u += kJoinWarps) {
                const float4* from =
                    reinterpret_cast<const float4*>(part_at(p, u, u == start ? 1 : 0, c0, lane));
                const float4 a = from[0], b = from[1];
                sum.v[0] += a.x, sum.v[1] += a.y, sum.v[2] += a.z, sum.v[3] += a.w;
                sum.v[4] += b.x, sum.v[5] += b.y, sum.v[6] += b.z, sum.v[7] += b.w;
            }
            __syncthreads();
            shared[warp][lane * 2] = make_float4(sum.v[0], sum.v[1], sum.v[2], sum.v[3]);
            shared[warp][lane * 2 + 1] = make_float4(sum.v[4], sum.v[5], sum.v[6], sum.v[7]);
            __syncthreads();
            if (warp == 0) {
                for (int o = 1; o < kJoinWarps; ++o) {
                    const float4 a = shared[o][lane * 2], b = shared[o][lane * 2 + 1];
                    sum.v[0] += a.x, sum.v[1] += a.y, sum.v[2] += a.z, sum.v[3] += a.w;
                    sum.v[4] += b.x, sum.v[5] += b.y, sum.v[6] += b.z, sum.v[7] += b.w;
                }
                finish_row<kVec>(p, row, c0, lane, sum);
            }
        }
        __syncthreads();
    }
}

// Tokens of a window: as many as leave a warp window for each of 32 warps an SM.
int window_of(long long tokens, long long cols) {
    const long long slices = (cols + kSlice - 1) / kSlice;
    int w = 64;
    while (w > 8 && (tokens + w - 1) / w * slices < kSMs * 32) w /= 2;
    return w;
}

constexpr long long kMaxTokens = train::kMaxExtent;  // (sums with a block's share fit ints)

struct BackwardSpace {
    size_t pairs, parts;
    int window;
    long long windows, slices;
};
BackwardSpace space_of(long long tokens, long long cols) {
    BackwardSpace s = {};
    s.window = window_of(tokens, cols);
    s.windows = (tokens + s.window - 1) / s.window;
    s.slices = (cols + kSlice - 1) / kSlice;
    s.pairs = round256((size_t)tokens * sizeof(uint2));
    s.parts = (size_t)s.windows * 2 * s.slices * kSlice * 4;
    return s;
}

template <int kWindow, bool kVec>
cudaError_t launch_sums(const SumParams& p, cudaStream_t st) {
    const long long units = (long long)p.windows * p.slices;
    cudaError_t e = launch_pdl(sum_kernel<kWindow, kVec>, dim3((unsigned)((units + kSumWarps - 1) / kSumWarps)),
                               dim3(kSumWarps * 32), st, p);
    if (e != cudaSuccess || p.windows == 1) return e;
    const int across = std::max(1, std::min(p.windows, kSMs * 4 / std::min(p.slices, kSMs * 4)));
    return launch_pdl(join_kernel<kWindow, kVec>, dim3(p.slices, across), dim3(kJoinThreads), st, p);
}
template <bool kVec>
cudaError_t launch_sums(const SumParams& p, int window, cudaStream_t st) {
    switch (window) {
    case 8: return launch_sums<8, kVec>(p, st);
    case 16: return launch_sums<16, kVec>(p, st);
    case 32: return launch_sums<32, kVec>(p, st);
    default: return launch_sums<64, kVec>(p, st);
    }
}

int id_size(vc_dtype_t d) { return d == VC_INT32 ? 4 : d == VC_INT64 ? 8 : 0; }

// The ids, and the first row's id, whose sum with the rows must not wrap.
bool valid_ids(const void* ids, vc_dtype_t d, long long tokens, long long first) {
    const int size = id_size(d);
    return size != 0 && tokens >= 0 && tokens <= kMaxTokens && first >= 0 && first <= (1ll << 62) &&
           (tokens == 0 || (ids != nullptr && reinterpret_cast<uintptr_t>(ids) % size == 0));
}

}  // namespace
}  // namespace step
}  // namespace vc

using namespace vc;
using namespace vc::step;

extern "C" {

vc_status_t vc_embedding_forward(const void* ids, vc_dtype_t id_dtype, long long tokens,
                                 const vc_matrix_t* weight, long long first, float scale,
                                 const vc_matrix_t* out, vc_stream_t stream) {
    if (!valid_ids(ids, id_dtype, tokens, first) || !valid_matrix(weight) || weight->batch != 1 ||
        !plain_matrix(out, tokens, weight->cols))
        return VC_ERR_INVALID_ARGUMENT;
    if (overlap(span_of(out), span_of(weight)) ||
        overlap(span_of(out), span_of(tokens > 0 ? ids : nullptr, (size_t)tokens * id_size(id_dtype))))
        return VC_ERR_ALIAS;
    if (tokens == 0 || weight->cols == 0) return VC_SUCCESS;
    if (test_launch_failure()) return VC_ERR_CUDA;
    LookupParams p = {};
    p.ids = ids;
    p.wide = id_dtype == VC_INT64;
    p.weight = rows_of(weight);
    p.out = rows_of(out);
    p.first = first;
    p.rows = weight->rows;
    p.cols = (int)weight->cols;
    p.scale = scale;
    const bool vec = p.weight.vec && p.out.vec;
    p.per_row = vec ? (p.cols + 7) / 8 : p.cols;
    p.units = tokens * p.per_row;
    // four units a thread where that still gives every SM its share
    const bool many = p.units >= 4ll * 256 * kSMs * 4;
    const long long blocks = (p.units + (many ? 1024 : 256) - 1) / (many ? 1024 : 256);
    if (blocks > 0x7FFFFFFF) return VC_ERR_INVALID_ARGUMENT;
    auto* kernel = many ? (vec ? lookup_kernel<4, true> : lookup_kernel<4, false>)
                        : (vec ? lookup_kernel<1, true> : lookup_kernel<1, false>);
    const cudaError_t e = launch_pdl(kernel, dim3((unsigned)blocks), dim3(256),
                                     static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? VC_SUCCESS : VC_ERR_CUDA;
}

size_t vc_embedding_backward_workspace(long long tokens, long long rows, long long cols) {
    if (tokens < 0 || tokens > kMaxTokens || rows < 0 || rows > train::kMaxExtent || cols < 0 ||
        cols > train::kMaxExtent)
        return 0;
    if (tokens == 0 || rows == 0 || cols == 0) return 0;
    const BackwardSpace s = space_of(tokens, cols);
    return 2 * s.pairs + round256(s.parts);
}

vc_status_t vc_embedding_backward(const vc_matrix_t* dy, const void* ids, vc_dtype_t id_dtype,
                                  long long first, long long padding, float scale,
                                  const vc_matrix_t* dweight, int accumulate, void* workspace,
                                  size_t workspace_bytes, vc_stream_t stream) {
    if (!valid_matrix(dy) || dy->batch != 1 || !valid_matrix(dweight) || dweight->batch != 1 ||
        dy->cols != dweight->cols || !valid_ids(ids, id_dtype, dy->rows, first))
        return VC_ERR_INVALID_ARGUMENT;
    const long long tokens = dy->rows, V = dweight->rows, D = dweight->cols;
    const size_t need = vc_embedding_backward_workspace(tokens, V, D);
    if (!workspace_ok(workspace, workspace_bytes, need)) return VC_ERR_INVALID_ARGUMENT;
    const Span outs[2] = {span_of(dweight), span_of(workspace, need)};
    const Span ins[2] = {span_of(dy),
                         span_of(tokens > 0 ? ids : nullptr, (size_t)tokens * id_size(id_dtype))};
    for (const Span& o : outs)
        for (const Span& i : ins)
            if (overlap(o, i)) return VC_ERR_ALIAS;
    if (overlap(outs[0], outs[1])) return VC_ERR_ALIAS;
    if (V == 0 || D == 0 || (tokens == 0 && accumulate)) return VC_SUCCESS;
    const BackwardSpace sp = space_of(tokens, D);
    if (sp.windows * sp.slices > 0x7FFFFFFFll * kSumWarps || sp.slices > 0x7FFFFFFF)
        return VC_ERR_INVALID_ARGUMENT;
    if (test_launch_failure()) return VC_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned char* ws = static_cast<unsigned char*>(workspace);

    SortParams s = {};
    s.ids = ids;
    s.wide = id_dtype == VC_INT64;
    s.first = first;
    s.padding = padding;
    s.rows = (unsigned)V;
    s.tokens = (int)tokens;
    int bits = 1;
    while (V >> bits) ++bits;
    s.passes = (bits + kDigitBits - 1) / kDigitBits;
    s.bits = (bits + s.passes - 1) / s.passes;
    s.a = reinterpret_cast<uint2*>(ws);
    s.b = reinterpret_cast<uint2*>(ws + sp.pairs);
    const Rows dw = rows_of(dweight);
    const int es = elem_size(dweight->dtype);
    s.out = static_cast<char*>(dw.data);
    s.row_bytes = D * es;
    s.pitch = dw.ld * es;
    s.vec = dw.vec;
    // blocks for the zeros: those of the clusters that fit beside the sorting one
    const int fill = accumulate ? 0 : (int)std::min((long long)(kSMs / kCluster - 1), (V + 31) / 32) * kCluster;
    cudaError_t e = launch_pdl(sort_kernel, dim3(kCluster + fill), dim3(kSortThreads), st, s);
    if (e != cudaSuccess) return VC_ERR_CUDA;
    if (tokens == 0) return VC_SUCCESS;

    SumParams p = {};
    p.sorted = s.a;
    p.dy = rows_of(dy);
    p.dw = dw;
    p.parts = reinterpret_cast<float*>(ws + 2 * sp.pairs);
    p.padded = sp.slices * kSlice;
    p.rows = s.rows;
    p.tokens = s.tokens;
    p.windows = (int)sp.windows;
    p.slices = (int)sp.slices;
    p.cols = (int)D;
    p.accumulate = accumulate != 0;
    p.scale = scale;
    e = p.dy.vec && p.dw.vec ? launch_sums<true>(p, sp.window, st) : launch_sums<false>(p, sp.window, st);
    return e == cudaSuccess ? VC_SUCCESS : VC_ERR_CUDA;
}

}  // extern "C"
