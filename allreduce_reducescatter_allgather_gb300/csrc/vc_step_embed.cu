// vc_embedding_forward / vc_embedding_backward: rows of a table looked up by
// token, and the sum of the tokens' gradients by row.
//
// Forward: y_t = s W[id_t - first].  One 16-byte vector of a row a thread, four
// of them in flight; bound by the bytes of y and of the rows: 65536 x 4096 from a table
// of 131072 rows take 117 us (6.05 TB/s), 8 x 1024 take 4.0 us, the launch.
//
// Backward: dW_v (+)= s sum_{t: row(t) = v} dy_t in three launches, none of which
// adds to memory that another block may add to:
//
//   sort   one block (up to 4096 tokens) or one cluster of blocks sorts (row, token) by
//          row, keeping the tokens of a row in order: a radix sort of up to 9 bits a
//          pass, whose ranks come from the lanes of a warp that share a digit, and whose
//          counts go through distributed shared memory in a cluster.  It is bound by
//          latency and needs few SMs; the other blocks of the same launch meanwhile
//          mark the rows that tokens have, and write zeros to as many of the others
//          as they have time for.
//   sum    writes zeros to the rest of those, in blocks among the summing ones: writes
//          alone reach 4.0 TB/s, together with reads 6.8.  Every summing warp takes a
//          window of neighbours in the sorted order and 256 columns: as many rows of dy
//          to each, whatever the ids are.  Rows whose tokens all lie in the window are
//          stored, the first and the last one, where they go on beyond it, left as
//          partial sums.  Bound by the bytes of dy and dW.
//   join   adds the partial sums of rows that span windows, in order.
//
// 65536 x 4096 into 131072 rows take 271 us (5.8 TB/s), 16384 x 1024 into 32000 rows 32
// us, of which the sort is 13, and 1003 x 517 into 5003 rows 12 us: three launches that
// wait for one another.
#include <algorithm>
#include <type_traits>

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
    long long first, tokens;
    unsigned long long rows;
    int cols, shift;  // log2 of the threads that share a row
    float scale;
};

constexpr int kLookupThreads = 256, kLookupUnits = 4;  // units of a thread in flight

// A group of threads a token.  Rows on 16 bytes eight columns at a time, others one (12352
// x 1735 of those take 28 us, 29 % of the floor).  A kernel for each pair of types:
// with all in one 65536 x 4096 took 123 us, with these 117.
template <bool kVec, bool kFrom32, bool kTo32>
__global__ void __launch_bounds__(kLookupThreads) lookup_kernel(const __grid_constant__ LookupParams p) {
    using From = std::conditional_t<kFrom32, float, __nv_bfloat16>;
    using To = std::conditional_t<kTo32, float, __nv_bfloat16>;
    pdl_next();
    pdl_wait();
    const int width = 1 << p.shift, lane = threadIdx.x & (width - 1);
    const long long token = ((long long)blockIdx.x * kLookupThreads + threadIdx.x) >> p.shift;
    if (token >= p.tokens) return;
    const unsigned long long row =
        (unsigned long long)load_id(p.ids, p.wide, token) - (unsigned long long)p.first;
    const bool in = row < p.rows;  // (a row below the table's start is far above its end)
    const From* const from = static_cast<const From*>(p.weight.data) + (in ? (long long)row : 0) * p.weight.ld;
    To* const to = static_cast<To*>(p.out.data) + token * p.out.ld;
    int done = 0;  // columns
    if constexpr (kVec) {
        const int units = p.cols / 8;
        done = units * 8;
        for (int u0 = lane; u0 < units; u0 += kLookupUnits * width) {
            uint4 raw[kLookupUnits][kFrom32 ? 2 : 1];
#pragma unroll
            for (int u = 0; u < kLookupUnits; ++u)
                if (in && u0 + u * width < units) {
                    const uint4* at = reinterpret_cast<const uint4*>(from + (u0 + u * width) * 8);
                    raw[u][0] = at[0];
                    if constexpr (kFrom32) raw[u][1] = at[1];
                }
#pragma unroll
            for (int u = 0; u < kLookupUnits; ++u) {
                if (u0 + u * width >= units) continue;
                Eight r = zeros();
                if (in) {
                    if constexpr (kFrom32)
                        r = {{__uint_as_float(raw[u][0].x), __uint_as_float(raw[u][0].y), __uint_as_float(raw[u][0].z),
                              __uint_as_float(raw[u][0].w), __uint_as_float(raw[u][1].x), __uint_as_float(raw[u][1].y),
                              __uint_as_float(raw[u][1].z), __uint_as_float(raw[u][1].w)}};
                    else
                        r = widen(raw[u][0]);
                    r = mul(p.scale, r);
                }
                To* at = to + (u0 + u * width) * 8;
                if constexpr (kTo32) {
                    reinterpret_cast<float4*>(at)[0] = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
                    reinterpret_cast<float4*>(at)[1] = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
                } else {
                    *reinterpret_cast<uint4*>(at) = narrow(r);
                }
            }
        }
    }
    auto value = [&](int c) {
        if constexpr (kFrom32)
            return from[c];
        else
            return __bfloat162float(from[c]);
    };
    for (int c0 = done + lane; c0 < p.cols; c0 += kLookupUnits * width) {
        float v[kLookupUnits];
#pragma unroll
        for (int u = 0; u < kLookupUnits; ++u) v[u] = in && c0 + u * width < p.cols ? value(c0 + u * width) : 0.0f;
#pragma unroll
        for (int u = 0; u < kLookupUnits; ++u) {
            const int c = c0 + u * width;
            if (c >= p.cols) continue;
            const float r = in ? v[u] * p.scale : 0.0f;
            if constexpr (kTo32)
                to[c] = r;
            else
                to[c] = __float2bfloat16(r);
        }
    }
}

// --------------------------------------------------------- sorting by row --

constexpr int kCluster = 8;         // blocks that sort
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kItems = 8;           // of a thread at a time
constexpr int kChunk = kSortThreads * kItems;
// Tokens that one block sorts (256 columns, by one block and by the cluster: 256 tokens
// 11.3 and 13.0 us, 1024 12.0 and 13.4, 2048 13.2 and 13.9, 3000 16.4 and 15.9, 4096 17.2 and
// 15.4, 6000 21.0 and 16.8).
constexpr int kFewTokens = 4096;
constexpr int kFillClusters = 14;   // beside the one that sorts: 15 run at a time
constexpr int kDigitBits = 9, kBins = 1 << kDigitBits;
constexpr int kMarkRows = 16384;    // rows that a block marks at a time

// Rows to be set to zero.
struct ZeroRows {
    char* out;
    long long row_bytes, pitch;
};
__device__ __forceinline__ void zero_row(const ZeroRows& z, unsigned row, int lane) {
    char* const at = z.out + (long long)row * z.pitch;
    // 16 bytes at a time between the first and the last 16-byte boundary
    const long long head = min(z.row_bytes, (long long)(-reinterpret_cast<uintptr_t>(at) & 15));
    const long long done = head + ((z.row_bytes - head) & ~15ll);
    for (long long c = head + lane * 16; c < done; c += 512)
        __stcs(reinterpret_cast<uint4*>(at + c), make_uint4(0, 0, 0, 0));
    const int edge = lane * 2;  // (of less than 16 bytes each, in elements of two bytes)
    if (edge < head) *reinterpret_cast<unsigned short*>(at + edge) = 0;
    if (done + edge < z.row_bytes) *reinterpret_cast<unsigned short*>(at + done + edge) = 0;
}

struct SortParams {
    const void* ids;
    int wide;
    long long first, padding;  // padding < 0: none
    unsigned rows;             // also the key of tokens that are left out
    int tokens, passes, bits;  // bits of a pass
    uint2 *a, *b;              // (row, token); the last pass writes a
    // the rows that no token has: below `split` the blocks that do not sort set them to
    // zero, from there on they leave marks
    ZeroRows zero;
    unsigned split;
    unsigned* marks;           // a bit a row from split on: a token has it
    int fill, few;             // whether there is any of that; one block sorts
};

__device__ __forceinline__ unsigned key_of(const SortParams& p, int t) {
    const long long id = load_id(p.ids, p.wide, t);
    const unsigned long long row = (unsigned long long)id - (unsigned long long)p.first;
    const bool live = row < p.rows && (p.padding < 0 || id != p.padding);
    return live ? (unsigned)row : p.rows;
}

// Loops stay loops here: a launch runs each of them a few times only, and code that
// has not run yet comes slowly (16 items unrolled took 7 us to the first sum).
struct SortShared {
    uint2 pair[2][kChunk];
    unsigned short rank[kChunk];
    unsigned short count[kSortWarps][kBins];  // of a warp, then of the warps before
    unsigned chunk[kBins], total[kBins], base[kBins], scan[32];
};

// Ranks n items of the chunk, each of which has a place of 32 in a warp, among those of
// their warp with the same digit; leaves the counts of the warps before each in
// count[][], the chunk's in chunk[].
__device__ __noinline__ void rank_chunk(SortShared& s, const uint2* pairs, int items, int n, int shift,
                                        unsigned mask) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = lane; i <= (int)mask / 2; i += 32) reinterpret_cast<unsigned*>(s.count[warp])[i] = 0;
    __syncwarp();
#pragma unroll 1
    for (int k = 0; k < items; ++k) {
        const int i = (warp * items + k) * 32 + lane;
        const bool live = i < n;
        const unsigned digit = live ? (pairs[i].x >> shift) & mask : 0;
        // the lanes with this digit, bit by bit (the instruction that finds them at once
        // takes four times as long)
        unsigned same = __ballot_sync(~0u, live);
        for (unsigned bit = 1; bit <= mask; bit <<= 1) {
            const unsigned with = __ballot_sync(~0u, digit & bit);
            same &= digit & bit ? with : ~with;
        }
        const int before = s.count[warp][digit], ahead = __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (live) {
            s.rank[i] = (unsigned short)(before + ahead);
            if (ahead == 0) s.count[warp][digit] = (unsigned short)(before + __popc(same));
        }
        __syncwarp();
    }
    __syncthreads();
    if (threadIdx.x <= mask) {
        unsigned n[kSortWarps], sum = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) n[w] = s.count[w][threadIdx.x];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            s.count[w][threadIdx.x] = (unsigned short)sum;
            sum += n[w];
        }
        s.chunk[threadIdx.x] = sum;
    }
    __syncthreads();
}

// base[] <- the sum of `n` over the threads before, of the first mask + 1, plus `more`.
__device__ __noinline__ void place_bins(SortShared& s, unsigned n, unsigned more, unsigned mask) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned m = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += m;
    }
    if (lane == 31) s.scan[warp] = sum;
    __syncthreads();
    const unsigned smaller = __reduce_add_sync(~0u, lane < warp ? s.scan[lane] : 0);
    if (threadIdx.x <= mask) s.base[threadIdx.x] = smaller + sum - n + more;
    __syncthreads();
}

// One block sorts up to a chunk of tokens without leaving its shared memory.
__device__ void sort_few(const SortParams& p, SortShared& s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int items = (p.tokens + kSortThreads - 1) / kSortThreads;
    const unsigned mask = (1u << p.bits) - 1;
#pragma unroll 2
    for (int i = threadIdx.x; i < p.tokens; i += kSortThreads) s.pair[0][i] = make_uint2(key_of(p, i), i);
    __syncthreads();
#pragma unroll 1
    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * p.bits;
        const uint2* from = s.pair[pass & 1];
        uint2* to = s.pair[(pass & 1) ^ 1];
        rank_chunk(s, from, items, p.tokens, shift, mask);
        place_bins(s, threadIdx.x <= mask ? s.chunk[threadIdx.x] : 0, 0, mask);
#pragma unroll 2
        for (int k = 0; k < items; ++k) {
            const int i = (warp * items + k) * 32 + lane;
            if (i >= p.tokens) break;
            const uint2 pair = from[i];
            const unsigned digit = (pair.x >> shift) & mask;
            to[s.base[digit] + s.count[warp][digit] + s.rank[i]] = pair;
        }
        __syncthreads();
    }
#pragma unroll 2
    for (int i = threadIdx.x; i < p.tokens; i += kSortThreads) p.a[i] = s.pair[p.passes & 1][i];
}

// Where this block's digits start: behind all smaller ones of the cluster, and behind
// those of the blocks before.
__device__ __forceinline__ void place_cluster(SortShared& s, unsigned mask) {
    cluster_sync();
    unsigned all = 0, before = 0;
    if (threadIdx.x <= mask) {
#pragma unroll
        for (int c = 0; c < kCluster; ++c) {
            const unsigned n = remote_load(&s.total[threadIdx.x], c);
            all += n;
            before += c < (int)blockIdx.x ? n : 0;
        }
    }
    place_bins(s, all, before, mask);
}

// A cluster sorts up to a chunk for each block: the pairs go from block to block.
__device__ void sort_chunks(const SortParams& p, SortShared& s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int each = (p.tokens + kCluster - 1) / kCluster;
    const int lo = min(p.tokens, (int)blockIdx.x * each), n = min(each, p.tokens - lo);
    const int items = (each + kSortThreads - 1) / kSortThreads;
    const unsigned mask = (1u << p.bits) - 1;
#pragma unroll 2
    for (int i = threadIdx.x; i < n; i += kSortThreads) s.pair[0][i] = make_uint2(key_of(p, lo + i), lo + i);
    __syncthreads();
#pragma unroll 1
    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * p.bits;
        const uint2* from = s.pair[pass & 1];
        uint2* to = s.pair[(pass & 1) ^ 1];
        rank_chunk(s, from, items, n, shift, mask);
        if (threadIdx.x <= mask) s.total[threadIdx.x] = s.chunk[threadIdx.x];
        place_cluster(s, mask);
        const bool last = pass + 1 == p.passes;
#pragma unroll 2
        for (int k = 0; k < items; ++k) {
            const int i = (warp * items + k) * 32 + lane;
            if (i >= n) break;
            const uint2 pair = from[i];
            const unsigned digit = (pair.x >> shift) & mask;
            const unsigned at = s.base[digit] + s.count[warp][digit] + s.rank[i];
            if (last) {
                p.a[at] = pair;
            } else {
                const unsigned block = at / each;
                remote_store(to + (at - block * each), block, pair);
            }
        }
        // (also before a block ends whose totals others read)
        cluster_sync();
    }
}

// A cluster sorts any number, each block a run of neighbours, chunk by chunk, through
// the workspace.
__device__ void sort_tokens(const SortParams& p, SortShared& s) {
    const int me = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int each = (p.tokens + kCluster - 1) / kCluster;
    const int lo = min((long long)p.tokens, (long long)me * each);
    const int hi = min((long long)p.tokens, (long long)(me + 1) * each);
    const unsigned mask = (1u << p.bits) - 1;
#pragma unroll 1
    for (int pass = 0; pass < p.passes; ++pass) {
        // the last pass writes a
        const bool into_a = ((p.passes - 1 - pass) & 1) == 0;
        const uint2* from = into_a ? p.b : p.a;
        uint2* to = into_a ? p.a : p.b;
        const int shift = pass * p.bits;
        auto rank = [&](int begin) {
            const int n = min(kChunk, hi - begin);
            __syncthreads();  // (the last chunk is used up)
#pragma unroll 4
            for (int i = threadIdx.x; i < n; i += kSortThreads)
                s.pair[0][i] = pass == 0 ? make_uint2(key_of(p, begin + i), begin + i) : __ldcg(from + begin + i);
            __syncthreads();
            rank_chunk(s, s.pair[0], kItems, n, shift, mask);
        };
        if (threadIdx.x <= mask) s.total[threadIdx.x] = 0;
#pragma unroll 1
        for (int begin = lo; begin < hi; begin += kChunk) {
            rank(begin);
            if (threadIdx.x <= mask) s.total[threadIdx.x] += s.chunk[threadIdx.x];
        }
        place_cluster(s, mask);
#pragma unroll 1
        for (int begin = lo; begin < hi; begin += kChunk) {
            rank(begin);
#pragma unroll 2
            for (int k = 0; k < kItems; ++k) {
                const int i = (warp * kItems + k) * 32 + lane;
                if (begin + i >= hi) break;
                const uint2 pair = s.pair[0][i];
                const unsigned digit = (pair.x >> shift) & mask;
                const unsigned at = s.base[digit] + s.count[warp][digit] + s.rank[i];
                if (at < (unsigned)p.tokens) __stcg(to + at, pair);  // (ids that change meanwhile)
            }
            __syncthreads();
            if (threadIdx.x <= mask) s.base[threadIdx.x] += s.chunk[threadIdx.x];
        }
        // what was written is read by other blocks; totals are rewritten
        __threadfence();
        cluster_sync();
    }
}

// This block's share of the rows below split, which it sets to zero where no token has
// them, and of the others, which it marks.  One pass over the ids for both.
__device__ void clear_rows(const SortParams& p, unsigned* marks, int part, int parts) {
    const unsigned behind = p.rows - p.split, words = (behind + 31) / 32;
    unsigned a = (unsigned)((unsigned long long)p.split * part / parts);
    const unsigned a_end = (unsigned)((unsigned long long)p.split * (part + 1) / parts);
    unsigned b = (unsigned)((unsigned long long)words * part / parts) * 32;
    const unsigned b_end = min(behind, (unsigned)((unsigned long long)words * (part + 1) / parts) * 32);
    unsigned* const marks_b = marks + kMarkRows / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    while (a < a_end || b < b_end) {
        const unsigned na = min(a_end - a, (unsigned)kMarkRows), nb = b < b_end ? min(b_end - b, (unsigned)kMarkRows) : 0;
        for (int i = threadIdx.x; i < 2 * kMarkRows / 32; i += kSortThreads) marks[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int t = threadIdx.x; t < p.tokens; t += kSortThreads) {
            const unsigned key = key_of(p, t), i = key - a, j = key - p.split - b;
            if (i < na) atomicOr(&marks[i >> 5], 1u << (i & 31));
            if (j < nb) atomicOr(&marks_b[j >> 5], 1u << (j & 31));
        }
        __syncthreads();
        for (unsigned i = threadIdx.x; i < (nb + 31) / 32; i += kSortThreads) p.marks[b / 32 + i] = marks_b[i];
        for (unsigned i = warp; i < na; i += kSortWarps)
            if (!(marks[i >> 5] >> (i & 31) & 1)) zero_row(p.zero, a + i, lane);
        __syncthreads();
        a += na;
        b += nb;
    }
}

__global__ void __launch_bounds__(kSortThreads, 1)
    sort_kernel(const __grid_constant__ SortParams p) {
    extern __shared__ uint4 shared[];
    SortShared& s = *reinterpret_cast<SortShared*>(shared);
    pdl_next();
    pdl_wait();
    const int sorters = p.few ? 1 : kCluster;
    if (blockIdx.x >= sorters) {
        if (p.fill) clear_rows(p, reinterpret_cast<unsigned*>(shared), blockIdx.x - sorters, gridDim.x - sorters);
    } else if (p.few) {
        sort_few(p, s);
    } else if (p.tokens <= kCluster * kChunk) {
        sort_chunks(p, s);
    } else {
        sort_tokens(p, s);
    }
}
static_assert(sizeof(SortShared) >= 2 * kMarkRows / 8, "a block's marks fit");
static_assert(kFewTokens <= kChunk && sizeof(SortShared) + 1024 <= kSharedLimit, "what a block has");

// ------------------------------------------------------------ sums by row --

// Columns of a warp, a vector a lane.  (Two vectors a lane halve the warps that wait
// for one token after the other: 14.4 -> 19.6 us for 16384 x 1024.)
constexpr int kVectors = 1, kSlice = 256 * kVectors;
constexpr int kSumWarps = 4;

struct SumParams {
    const uint2* sorted;
    Rows dy, dw;
    float* parts;  // [window][2][padded columns]: the first and the last row's
    long long padded;
    unsigned rows;
    int tokens, windows, slices, cols, accumulate;
    float scale;
    // rows from split on whose mark is not set become zero
    ZeroRows zero;
    const unsigned* marks;
    unsigned split;
    int zero_rows;                       // of a block
    unsigned zero_blocks, sum_blocks;    // of the launch
};

__device__ __forceinline__ void zero_unmarked(const SumParams& p, unsigned block) {
    const unsigned first = block * p.zero_rows, behind = p.rows - p.split;
    const int lane = threadIdx.x & 31;
    for (unsigned i = first + threadIdx.x / 32; i < min(behind, first + p.zero_rows); i += kSumWarps)
        if (!(p.marks[i >> 5] >> (i & 31) & 1)) zero_row(p.zero, p.split + i, lane);
}

// dW row (+)= scale * sum, vector v.  What is added to 32-bit values is sent to memory,
// which adds it once, and nobody waits for the old ones.
template <bool kVec>
__device__ __forceinline__ void finish_row(const SumParams& p, unsigned row, int v, int lane, const Eight& sum) {
    Eight r = mul(p.scale, sum);
    if (p.accumulate && p.dw.f32) {
        float* to = static_cast<float*>(p.dw.data) + (long long)row * p.dw.ld;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = column<32>(kVec, v, lane, j);
            if (c < p.cols) asm volatile("red.global.add.f32 [%0], %1;" ::"l"(to + c), "f"(r.v[j]) : "memory");
        }
        return;
    }
    if (p.accumulate) r = add(r, load_any<32>(p.dw, row, kVec, v, lane, p.cols));
    store_any<32>(p.dw, p.dw.f32, row, kVec, v, lane, p.cols, r);
}

// The rows of a window as one warp takes them: on 16 bytes through shared memory, where
// each lane's own columns of the next rows are on their way (128 bytes a lane);
// others by fours through registers.  16384 x 4096 into 32768 rows: 65 us for 116 MB read
// and 205 written, from cold caches.
template <int kWindow, bool kVec, bool kF32>
__global__ void __launch_bounds__(kSumWarps * 32) sum_kernel(const __grid_constant__ SumParams p) {
    constexpr int kWords = kF32 ? 2 : 1, kAhead = 8 / kWords, kBatch = 4, kPairs = (kWindow + 31) / 32;
    __shared__ uint4 ring[kSumWarps][kVec ? kAhead : 1][kVec ? kVectors * kWords : 1][32];
    pdl_next();
    pdl_wait();
    // the zeroing blocks lie evenly among the others
    const unsigned zeroing = (unsigned)((unsigned long long)blockIdx.x * p.zero_blocks / gridDim.x);
    if ((unsigned)((unsigned long long)(blockIdx.x + 1) * p.zero_blocks / gridDim.x) != zeroing)
        return zero_unmarked(p, zeroing);
    const int lane = threadIdx.x & 31, warp = __shfl_sync(~0u, threadIdx.x / 32, 0);
    const long long unit = (long long)(blockIdx.x - zeroing) * kSumWarps + warp;
    const int window = (int)(unit / p.slices), slice = (int)(unit - (long long)window * p.slices);
    if (window >= p.windows) return;
    const int begin = window * kWindow;
    uint2 mine[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const int t = begin + i * 32 + lane;
        mine[i] = i * 32 + lane < kWindow && t < p.tokens ? p.sorted[t] : make_uint2(p.rows, 0);
    }
    const unsigned before = begin > 0 ? p.sorted[begin - 1].x : p.rows;
    const unsigned after = p.tokens - begin > kWindow ? p.sorted[begin + kWindow].x : p.rows;
    auto key_at = [&](int j) { return __shfl_sync(~0u, kPairs > 1 && j >= 32 ? mine[kPairs - 1].x : mine[0].x, j & 31); };
    auto token_at = [&](int j) { return __shfl_sync(~0u, kPairs > 1 && j >= 32 ? mine[kPairs - 1].y : mine[0].y, j & 31); };
    // how many tokens there are (those that are left out come last), and which ones
    // start a row
    int live = 0;
    unsigned starts[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        live += __popc(__ballot_sync(~0u, mine[i].x < p.rows));
        unsigned last = __shfl_up_sync(~0u, mine[i].x, 1);
        const unsigned other = __shfl_sync(~0u, mine[0].x, i == 0 ? 0 : 31);
        if (lane == 0) last = other;
        starts[i] = __ballot_sync(~0u, mine[i].x != last);
    }
    if (live == 0) return;
    Eight sum[kVectors];
#pragma unroll
    for (int i = 0; i < kVectors; ++i) sum[i] = zeros();
    unsigned row = key_at(0);
    bool first = true;
    const Rows parts = {p.parts, p.padded, 1, 1};
    auto flush = [&](bool end) {
        const bool from = first && row == before, on = end && row == after;
#pragma unroll
        for (int i = 0; i < kVectors; ++i) {
            const int v = slice * kVectors + i;
            if (from || on)
                store_any<32>(parts, true, (long long)window * 2 + (from ? 0 : 1), kVec, v, lane, p.cols, sum[i]);
            else
                finish_row<kVec>(p, row, v, lane, sum[i]);
        }
    };
    auto next = [&](int j) {
        if (!((kPairs > 1 && j >= 32 ? starts[kPairs - 1] : starts[0]) >> (j & 31) & 1)) return;
        flush(false);
        first = false;
        row = key_at(j);
#pragma unroll
        for (int i = 0; i < kVectors; ++i) sum[i] = zeros();
    };
    if constexpr (kVec) {
        const long long pitch = p.dy.ld * (kF32 ? 4 : 2);
        const char* base[kVectors];
        int bytes[kVectors], more[kVectors];
#pragma unroll
        for (int i = 0; i < kVectors; ++i) {
            const int c = ((slice * kVectors + i) * 32 + lane) * 8, left = p.cols - c;
            bytes[i] = max(0, min(16, left * (kF32 ? 4 : 2)));
            more[i] = max(0, min(16, left * 4 - 16));
            base[i] = static_cast<const char*>(p.dy.data) + (left > 0 ? (long long)c * (kF32 ? 4 : 2) : 0);
        }
        auto issue = [&](int j) {
            if (j < live) {
                const long long at = token_at(j) * pitch;
                uint4* to = &ring[warp][j % kAhead][0][lane];
#pragma unroll
                for (int i = 0; i < kVectors; ++i) {
                    copy16(to + i * kWords * 32, base[i] + at, bytes[i]);
                    if constexpr (kF32) copy16(to + (i * kWords + 1) * 32, base[i] + at + (more[i] ? 16 : 0), more[i]);
                }
            }
            copies_end();
        };
#pragma unroll 1
        for (int j = 0; j < kAhead; ++j) issue(j);
#pragma unroll 1
        for (int j = 0; j < live; ++j) {
            copies_wait<kAhead - 1>();
            next(j);
            const uint4(*at)[32] = ring[warp][j % kAhead];
#pragma unroll
            for (int i = 0; i < kVectors; ++i) {
                if constexpr (kF32) {
                    const uint4 lo = at[i * kWords][lane], hi = at[i * kWords + kWords - 1][lane];
                    sum[i] = add(sum[i], {{__uint_as_float(lo.x), __uint_as_float(lo.y), __uint_as_float(lo.z),
                                           __uint_as_float(lo.w), __uint_as_float(hi.x), __uint_as_float(hi.y),
                                           __uint_as_float(hi.z), __uint_as_float(hi.w)}});
                } else {
                    sum[i] = add(sum[i], widen(at[i][lane]));
                }
            }
            issue(j + kAhead);
        }
        copies_wait<0>();
    } else {
#pragma unroll 1
        for (int b = 0; b < live; b += kBatch) {
            Raw v[kBatch][kVectors];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const unsigned token = token_at(b + k);
                if (b + k < live)
#pragma unroll
                    for (int i = 0; i < kVectors; ++i)
                        v[k][i] = load_raw<32>(p.dy, kF32, token, kVec, slice * kVectors + i, lane, p.cols);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (b + k >= live) break;
                next(b + k);
#pragma unroll
                for (int i = 0; i < kVectors; ++i) sum[i] = add(sum[i], widen_raw(v[k][i], kF32, kVec));
            }
        }
    }
    flush(true);
}

// A row that starts in one window and goes on into others: its last partial sum
// there and the first ones of the windows behind, for 128 columns.  A warp looks after
// a window; where the row goes on for long, all warps of the block share its windows.
// (The windows of a block are neighbours, of which few have such a row; the columns of
// one window are different blocks'.)  7.7 us for 256 windows of 4096 columns.
// kJoinLong: the windows up to which a warp does it alone (the gradient of 16384 x 1024 whose
// rows have 4 windows each: 24.7 us by a warp, 27.6 by the block; 16: 25.2 and 25.7; 32: 26.7 and
// 25.2; 128: 39.4 and 31.3).
constexpr int kJoinWarps = 8, kJoinColumns = 128, kJoinLong = 16;

template <int kWindow, bool kVec>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ SumParams p) {
    __shared__ int spans[kJoinWarps];  // windows behind that a long row reaches, or 0
    __shared__ float4 part[kJoinWarps][32];
    pdl_next();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = __shfl_sync(~0u, threadIdx.x / 32, 0);
    const int first = blockIdx.x * kJoinWarps, c = blockIdx.y * kJoinColumns + lane * 4;
    auto key = [&](int window, int i) { return p.sorted[(long long)window * kWindow + i].x; };
    // the partial sums of the windows from `begin` on, every step-th one, eight in flight
    auto add_up = [&](int begin, int end, int step, float4 sum) {
        constexpr int kBatch = 8;
        const long long pitch = (long long)step * 2 * p.padded;
        const float* at = p.parts + (long long)begin * 2 * p.padded + c;
        for (int u = begin; u < end; u += kBatch * step, at += kBatch * pitch) {
            float4 v[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                v[k] = u + k * step < end ? *reinterpret_cast<const float4*>(at + k * pitch)
                                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) sum.x += v[k].x, sum.y += v[k].y, sum.z += v[k].z, sum.w += v[k].w;
        }
        return sum;
    };
    auto store = [&](unsigned row, float4 sum) {
        const float s[4] = {sum.x, sum.y, sum.z, sum.w};
        const long long to = (long long)row * p.dw.ld + c;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (c + j >= p.cols) break;
            if (p.dw.f32) {
                float* f = static_cast<float*>(p.dw.data) + to + j;
                *f = fmaf(p.scale, s[j], p.accumulate ? *f : 0.0f);
            } else {
                __nv_bfloat16* b = static_cast<__nv_bfloat16*>(p.dw.data) + to + j;
                *b = __float2bfloat16(fmaf(p.scale, s[j], p.accumulate ? __bfloat162float(*b) : 0.0f));
            }
        }
    };
    auto last_part = [&](int window) {
        return *reinterpret_cast<const float4*>(p.parts + ((long long)window * 2 + 1) * p.padded + c);
    };
    const int start = first + warp;
    int span = 0;
    if (start + 1 < p.windows) {
        const unsigned row = key(start, kWindow - 1), front = key(start, 0);
        const unsigned back = start > 0 ? key(start - 1, kWindow - 1) : p.rows;
        for (int u = start + 1 + lane;; u += 32) {
            const unsigned other = __ballot_sync(~0u, u >= p.windows || key(u, 0) != row);
            if (other != 0) {
                span += __ffs(other) - 1;
                break;
            }
            span += 32;
        }
        if (row >= p.rows || (front == row && back == row)) span = 0;
        if (span > 0 && span <= kJoinLong && c < p.cols)
            store(row, add_up(start + 1, start + 1 + span, 1, last_part(start)));
    }
    if (lane == 0) spans[warp] = span > kJoinLong ? span : 0;
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < kJoinWarps; ++w) {
        const int n = spans[w], from = first + w;
        if (n == 0) continue;
        const float4 none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c < p.padded)
            part[warp][lane] = add_up(from + 1 + warp, from + 1 + n, kJoinWarps, warp == 0 ? last_part(from) : none);
        __syncthreads();
        if (warp == 0 && c < p.cols) {
            float4 sum = part[0][lane];
#pragma unroll
            for (int o = 1; o < kJoinWarps; ++o) {
                const float4 v = part[o][lane];
                sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
            }
            store(key(from, kWindow - 1), sum);
        }
        __syncthreads();
    }
}

// Tokens of a window: as many as leave a window for each of 24 warps an SM, or 1024
// windows: more would lengthen the joins of frequent rows, whose windows are added
// one after the other.
int window_of(long long tokens, long long cols) {
    const long long slices = (cols + kSlice - 1) / kSlice;
    int w = 64;
    while (w > 8 && (tokens + w - 1) / w < 1024 && (tokens + w - 1) / w * slices < kSMs * 24) w /= 2;
    return w;
}

constexpr long long kMaxColumns = 1 << 22;
static_assert(kMaxColumns / kJoinColumns <= 65535, "a grid's second extent");
constexpr long long kMaxTokens = train::kMaxExtent;  // (sums with a block's share fit ints)

struct BackwardSpace {
    size_t pairs, parts, marks;
    int window;
    long long windows, slices;
};
BackwardSpace space_of(long long tokens, long long rows, long long cols) {
    BackwardSpace s = {};
    s.window = window_of(tokens, cols);
    s.windows = (tokens + s.window - 1) / s.window;
    s.slices = (cols + kSlice - 1) / kSlice;
    s.pairs = round256((size_t)tokens * sizeof(uint2));
    s.parts = round256((size_t)s.windows * 2 * s.slices * kSlice * 4);
    s.marks = round256((size_t)(rows + 31) / 32 * 4);
    return s;
}

template <int kWindow, bool kVec>
cudaError_t launch_sums(const SumParams& p, cudaStream_t st) {
    cudaError_t e = launch_pdl(p.dy.f32 ? sum_kernel<kWindow, kVec, true> : sum_kernel<kWindow, kVec, false>,
                               dim3(p.sum_blocks + p.zero_blocks), dim3(kSumWarps * 32), st, p);
    if (e != cudaSuccess || p.windows == 1) return e;
    return launch_pdl(join_kernel<kWindow, kVec>,
                      dim3((p.windows + kJoinWarps - 1) / kJoinWarps, (p.cols + kJoinColumns - 1) / kJoinColumns),
                      dim3(kJoinWarps * 32), st, p);
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
    p.tokens = tokens;
    const bool vec = p.weight.vec && p.out.vec;
    // a warp a row; half of one or less where that reaches over the row; up to a block
    // where there are few rows, down to one unit a thread
    const long long units = vec ? (p.cols + 7) / 8 : p.cols;
    p.shift = 0;
    while (p.shift < 8 && (1ll << p.shift) < units &&
           (p.shift < 5 || (tokens << p.shift) < (long long)kSMs * 1024))
        ++p.shift;
    const long long blocks = ((tokens << p.shift) + kLookupThreads - 1) / kLookupThreads;
    void (*kernel)(LookupParams);
    switch (vec * 4 + p.weight.f32 * 2 + p.out.f32) {
    case 0: kernel = lookup_kernel<false, false, false>; break;
    case 1: kernel = lookup_kernel<false, false, true>; break;
    case 2: kernel = lookup_kernel<false, true, false>; break;
    case 3: kernel = lookup_kernel<false, true, true>; break;
    case 4: kernel = lookup_kernel<true, false, false>; break;
    case 5: kernel = lookup_kernel<true, false, true>; break;
    case 6: kernel = lookup_kernel<true, true, false>; break;
    default: kernel = lookup_kernel<true, true, true>;
    }
    const cudaError_t e = launch_pdl(kernel, dim3((unsigned)blocks), dim3(kLookupThreads),
                                     static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? VC_SUCCESS : VC_ERR_CUDA;
}

size_t vc_embedding_backward_workspace(long long tokens, long long rows, long long cols) {
    if (tokens < 0 || tokens > kMaxTokens || rows < 0 || rows > train::kMaxExtent || cols < 0 ||
        cols > kMaxColumns)
        return 0;
    if (tokens == 0 || rows == 0 || cols == 0) return 0;
    const BackwardSpace s = space_of(tokens, rows, cols);
    return 2 * s.pairs + s.parts + s.marks;
}

vc_status_t vc_embedding_backward(const vc_matrix_t* dy, const void* ids, vc_dtype_t id_dtype,
                                  long long first, long long padding, float scale,
                                  const vc_matrix_t* dweight, int accumulate, void* workspace,
                                  size_t workspace_bytes, vc_stream_t stream) {
    if (!valid_matrix(dy) || dy->batch != 1 || !valid_matrix(dweight) || dweight->batch != 1 ||
        dy->cols != dweight->cols || !valid_ids(ids, id_dtype, dy->rows, first))
        return VC_ERR_INVALID_ARGUMENT;
    const long long tokens = dy->rows, V = dweight->rows, D = dweight->cols;
    if (D > kMaxColumns) return VC_ERR_INVALID_ARGUMENT;
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
    const BackwardSpace sp = space_of(tokens, V, D);
    const long long sum_blocks = (sp.windows * sp.slices + kSumWarps - 1) / kSumWarps;
    if (sum_blocks > 1ll << 30) return VC_ERR_INVALID_ARGUMENT;
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
    s.zero = {static_cast<char*>(dw.data), D * es, dw.ld * es};
    // what can be zeroed while the tokens are sorted (13 us for 16384 of them, 28 us for
    // 65536), at 4 TB/s
    const long long early = tokens == 0 ? V : ((16ll << 20) + 1400 * tokens) / (D * es);
    s.split = (unsigned)std::min(V, early);
    s.marks = reinterpret_cast<unsigned*>(ws + 2 * sp.pairs + sp.parts);
    // blocks for the zeros: those of the clusters that fit beside the sorting one
    s.few = tokens <= kFewTokens;
    s.fill = !accumulate;
    const int fill = accumulate ? 0 : (int)std::min((long long)kFillClusters, (V + 31) / 32) * kCluster;
    cudaError_t e = launch_pdl_shared(sort_kernel, dim3(kCluster + fill), dim3(kSortThreads), sizeof(SortShared), kCluster, st, s);
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
    p.sum_blocks = (unsigned)sum_blocks;
    if (!accumulate && s.split < s.rows) {
        // 64 KiB a block
        p.zero = s.zero;
        p.marks = s.marks;
        p.split = s.split;
        p.zero_rows = (int)std::max(4ll, std::min(32ll, (64ll << 10) / (D * es)));
        p.zero_blocks = (s.rows - s.split + p.zero_rows - 1) / p.zero_rows;
    }
    e = p.dy.vec && p.dw.vec ? launch_sums<true>(p, sp.window, st) : launch_sums<false>(p, sp.window, st);
    return e == cudaSuccess ? VC_SUCCESS : VC_ERR_CUDA;
}

}  // extern "C"
