// vc_clip_plan / vc_grad_norm / vc_clip_grad_norm: the norm of many gradients as
// one vector, and c = min(1, max_norm / (norm + eps)) times each of them.
//
// Two kernels, both over the plan's tiles of up to 16 KiB: the first sums squares
// (or takes the largest magnitude) and leaves one value a block, the second adds
// those in a fixed order, in every block by itself, and scales.  The bound is the
// gradients' bytes, which clipping reads twice where they are more than the second-
// level cache holds: 368 MB of bfloat16 in 145 tensors, clipped, take 173 us (the two
// reads and the write at 6.4 TB/s); 2.1 GB of float32 that need no clipping 319 us (6.7
// TB/s); 4 MB 7 us, most of it launches.  (Small sets in one launch of one cluster,
// whose blocks read each other's sums, took 10 us with 16 blocks and 6.2 with 8, where
// these two took 5.0.)
//
// Squares are added in 32 bits over a tile's 16 or 32 values of a thread, and from there
// on as pairs of 32-bit values that keep what the additions round off (48 bits; this
// GPU adds two 64-bit values a clock and SM: a block's 64-bit sum took 9 us).
// float32's range does not hold the squares of its own values: where a thread's sum
// over a tile leaves [2^-90, 2^90] it is computed again, in 64 bits, from the registers
// that still hold the values, and added apart.  (At a sum of 2^-90 or more, squares
// below 2^-126, which lose digits, do not count.)
#include <algorithm>
#include <math.h>

#include "vc_step_common.cuh"

namespace vc {
namespace step {
namespace {

constexpr int kClipThreads = 256;
constexpr int kTileBytes = VC_CLIP_TILE_MAX_BYTES;
constexpr int kVecs = kTileBytes / 16 / kClipThreads;  // 16-byte vectors of a thread
constexpr int kResident = 4;  // blocks of an SM
constexpr int kMaxBlocks = kSMs * kResident;
constexpr size_t kCacheBytes = 80u << 20;

int clip_blocks(int ntiles) { return std::max(1, std::min(ntiles, kMaxBlocks)); }

// kAllInPlace: all tiles of the plan are (so that nothing is to be done where c = 1).
enum { kTileF32 = 1, kAllInPlace = 2 };

// A tile's values as a thread holds them: up to kVecs vectors of 16 bytes from
// the first 16-byte boundary on, and at most one value before or behind them.
struct Held {
    uint4 v[kVecs];
    float edge;
};

struct Cut {
    int head, vecs, tail;  // values, vectors, values
};
__device__ __forceinline__ Cut cut_of(const vc_clip_tile_t& t) {
    const int es = t.flags & kTileF32 ? 4 : 2;
    const int off = (int)(reinterpret_cast<uintptr_t>(t.src) & 15);
    Cut c;
    c.head = min(t.count, off ? (16 - off) / es : 0);
    c.vecs = (t.count - c.head) / (16 / es);
    c.tail = t.count - c.head - c.vecs * (16 / es);
    return c;
}

// The index of the value before the vectors that thread i holds, or of the one
// behind them that thread 32 + i holds; -1: none.
__device__ __forceinline__ int edge_of(const vc_clip_tile_t& t, const Cut& c) {
    const int i = threadIdx.x;
    if (i < c.head) return i;
    if (i >= 32 && i - 32 < c.tail) return t.count - c.tail + i - 32;
    return -1;
}

__device__ __forceinline__ float load_value(const vc_clip_tile_t& t, int i) {
    if (t.flags & kTileF32) return static_cast<const float*>(t.src)[i];
    return __bfloat162float(static_cast<const __nv_bfloat16*>(t.src)[i]);
}

// kOnce: not read again.
template <bool kOnce>
__device__ __forceinline__ void load_tile(const vc_clip_tile_t& t, const Cut& c, Held& h) {
    const char* base = static_cast<const char*>(t.src) + c.head * (t.flags & kTileF32 ? 4 : 2);
    const uint4* p = reinterpret_cast<const uint4*>(base);
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        const int i = u * kClipThreads + threadIdx.x;
        h.v[u] = i < c.vecs ? load_word<kOnce>(p + i) : make_uint4(0, 0, 0, 0);
    }
    const int e = edge_of(t, c);
    h.edge = e >= 0 ? load_value(t, e) : 0.0f;
}

__device__ __forceinline__ float lo16(unsigned w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(unsigned w) { return __uint_as_float(w & 0xFFFF0000u); }

template <class F>
__device__ __forceinline__ void each_value(const Held& h, bool f32, F f) {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        const unsigned w[4] = {h.v[u].x, h.v[u].y, h.v[u].z, h.v[u].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (f32) {
                f(__uint_as_float(w[j]), j);
            } else {
                f(lo16(w[j]), j);
                f(hi16(w[j]), j);
            }
        }
    }
    f(h.edge, 0);
}

// A sum of squares: s + c, where |c| is at most half a step of s, and what is out of
// their range.  Of the largest magnitude: its bits in s.
struct __align__(16) Part {
    float s, c;
    double rest;
};
constexpr float kLeast = 0x1p-90f, kMost = 0x1p90f;

// s + c += x + d, for s and x of one sign.  What the addition of s and x rounds off joins c, and
// their sum is split again, so that c never grows to more than half a step of s (left to
// itself it becomes the whole error of a 32-bit sum: 1.3e-6 of the norm of 2 GB of equal values).
__device__ __forceinline__ void add_pair(float& s, float& c, float x, float d) {
    const float t = s + x, b = t - s;
    const float e = c + (((s - (t - b)) + (x - b)) + d);
    s = t + e;
    c = e - (s - t);
}

__device__ __forceinline__ void squares(const Held& h, bool f32, Part& p) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    each_value(h, f32, [&](float x, int j) { s[j] = fmaf(x, x, s[j]); });
    const float sum = (s[0] + s[1]) + (s[2] + s[3]);
    if (sum >= kLeast && sum <= kMost) return add_pair(p.s, p.c, sum, 0.0f);
    unsigned any = __float_as_uint(h.edge);
#pragma unroll
    for (int u = 0; u < kVecs; ++u) any |= h.v[u].x | h.v[u].y | h.v[u].z | h.v[u].w;
    if ((any & (f32 ? 0x7FFFFFFFu : 0x7FFF7FFFu)) == 0) return;
    double d = 0.0;
    each_value(h, f32, [&](float x, int) { d = ::fma((double)x, (double)x, d); });
    p.rest += d;
}

// The largest magnitude as float32 bits, which order like the values; a NaN's
// are above infinity's.
__device__ __forceinline__ unsigned largest(const Held& h, bool f32) {
    unsigned m = 0;
    each_value(h, f32, [&](float x, int) { m = max(m, __float_as_uint(x) & 0x7FFFFFFFu); });
    return m;
}

// The sum or maximum of the warp's parts, in every lane.
template <bool kMax>
__device__ __forceinline__ Part warp_total(Part p) {
    if constexpr (kMax) {
        p.s = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(p.s)));
    } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float s = __shfl_xor_sync(~0u, p.s, o), c = __shfl_xor_sync(~0u, p.c, o);
            // (in the same order in both lanes, for the same bits)
            const bool low = (threadIdx.x & o) == 0;
            float t = low ? p.s : s, d = low ? p.c : c;
            add_pair(t, d, low ? s : p.s, low ? c : p.c);
            p.s = t, p.c = d;
        }
        if (__any_sync(~0u, p.rest != 0.0)) p.rest = warp_sum(p.rest);  // (NaN: too)
    }
    return p;
}
// The block's, in every thread.
template <bool kMax>
__device__ Part block_total(Part p, Part* shared) {
    p = warp_total<kMax>(p);
    const int lane = threadIdx.x & 31, warps = blockDim.x / 32;
    if (lane == 0) shared[threadIdx.x >> 5] = p;
    __syncthreads();
    p = lane < warps ? shared[lane] : Part{0.0f, 0.0f, 0.0};
    p = warp_total<kMax>(p);
    __syncthreads();
    return p;
}

// Block b's tiles: a run of neighbours, so that the second kernel, which takes
// them backwards, meets first what the first one read last.
__device__ __forceinline__ int first_tile(int b, int blocks, int ntiles) {
    return (int)((long long)b * ntiles / blocks);
}

// One value a block: 268 MB of float32 in 48 us (5.6 TB/s from cold caches).  A tile is
// on its way while the one before it is summed, 64 bytes a thread.
template <bool kMax>
__global__ void __launch_bounds__(kClipThreads, kResident)
    norm_kernel(const vc_clip_tile_t* tiles, int ntiles, int again, Part* parts) {
    __shared__ Part shared[kClipThreads / 32];
    pdl_next();
    pdl_wait();
    const int end = first_tile(blockIdx.x + 1, gridDim.x, ntiles);
    const int keep = end - again;  // the tiles from here on are read again
    Part sum = {0.0f, 0.0f, 0.0};
    int i = first_tile(blockIdx.x, gridDim.x, ntiles);
    // a tile is on its way while the one before it is summed, and the place of the next
    vc_clip_tile_t next = {};
    Held coming;
    auto load = [&](int at) {
        if (at < keep)
            load_tile<true>(next, cut_of(next), coming);
        else
            load_tile<false>(next, cut_of(next), coming);
    };
    if (i < end) {
        next = tiles[i];
        load(i);
    }
    for (; i < end; ++i) {
        const bool f32 = next.flags & kTileF32;
        const Held h = coming;
        if (i + 1 < end) {
            next = tiles[i + 1];
            load(i + 1);
        }
        if constexpr (kMax)
            sum.s = __uint_as_float(max(__float_as_uint(sum.s), largest(h, f32)));
        else
            squares(h, f32, sum);
    }
    sum = block_total<kMax>(sum, shared);
    if (threadIdx.x == 0) parts[blockIdx.x] = sum;
}

template <bool kMax>
__device__ __forceinline__ float norm_of(const Part& p) {
    if (kMax) return p.s;
    if (p.rest == 0.0) return __fsqrt_rn(p.s);  // (c is below half a step)
    return (float)sqrt((double)p.s + (double)p.c + p.rest);
}
__device__ __forceinline__ float scale_of(float norm, float max_norm, float eps) {
    const float q = __fdiv_rn(max_norm, norm + eps);
    return q >= 1.0f ? 1.0f : q;  // (a NaN stays one)
}

// c x, rounded to the tile's type, where the plan says.
__device__ __forceinline__ void store_tile(const vc_clip_tile_t& t, const Cut& c, const Held& h,
                                           float scale) {
    const bool f32 = t.flags & kTileF32;
    const int es = f32 ? 4 : 2;
    char* base = static_cast<char*>(t.dst) + c.head * es;
    const bool vec = (reinterpret_cast<uintptr_t>(base) & 15) == 0;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        const int i = u * kClipThreads + threadIdx.x;
        if (i >= c.vecs) continue;
        const uint4 v = h.v[u];
        const unsigned w[4] = {v.x, v.y, v.z, v.w};
        unsigned o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = f32 ? __float_as_uint(scale * __uint_as_float(w[j]))
                       : narrow2(scale * lo16(w[j]), scale * hi16(w[j]));
        if (vec) {
            __stcs(reinterpret_cast<uint4*>(base) + i, make_uint4(o[0], o[1], o[2], o[3]));
        } else if (f32) {
#pragma unroll
            for (int j = 0; j < 4; ++j) reinterpret_cast<unsigned*>(base)[i * 4 + j] = o[j];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                reinterpret_cast<unsigned short*>(base)[i * 8 + 2 * j] = (unsigned short)o[j];
                reinterpret_cast<unsigned short*>(base)[i * 8 + 2 * j + 1] = (unsigned short)(o[j] >> 16);
            }
        }
    }
    const int e = edge_of(t, c);
    if (e >= 0) {
        if (f32)
            static_cast<float*>(t.dst)[e] = scale * h.edge;
        else
            static_cast<__nv_bfloat16*>(t.dst)[e] = __float2bfloat16(scale * h.edge);
    }
}

// The norm, and the scaled gradients: 268 MB of float32 in 84 us (5.8 TB/s, read and
// written, from cold caches).  Each block adds up all blocks' values by itself (at most
// 608, from the second-level cache), which saves a launch.
template <bool kMax, bool kClip>
__global__ void __launch_bounds__(kClipThreads, kResident) clip_kernel(const vc_clip_tile_t* tiles, int ntiles,
                                                            const Part* parts, int nparts,
                                                            float max_norm, float eps, float* norm) {
    __shared__ Part shared[kClipThreads / 32];
    pdl_next();
    pdl_wait();
    Part all = {0.0f, 0.0f, 0.0};
    for (int i = threadIdx.x; i < nparts; i += kClipThreads) {
        const Part p = parts[i];
        if constexpr (kMax) {
            all.s = __uint_as_float(max(__float_as_uint(all.s), __float_as_uint(p.s)));
        } else {
            add_pair(all.s, all.c, p.s, p.c);
            if (p.rest != 0.0) all.rest += p.rest;
        }
    }
    const float total = norm_of<kMax>(block_total<kMax>(all, shared));
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
    if constexpr (kClip) {
        const float scale = scale_of(total, max_norm, eps);
        const int begin = first_tile(blockIdx.x, gridDim.x, ntiles);
        int i = first_tile(blockIdx.x + 1, gridDim.x, ntiles) - 1;
        if (i < begin) return;
        vc_clip_tile_t next = tiles[i];
        if (scale == 1.0f && next.flags & kAllInPlace) return;
        Held coming;
        load_tile<true>(next, cut_of(next), coming);
        for (; i >= begin; --i) {
            const vc_clip_tile_t t = next;
            const Held h = coming;
            if (i > begin) {
                next = tiles[i - 1];
                load_tile<true>(next, cut_of(next), coming);
            }
            if (t.dst == nullptr || (scale == 1.0f && t.src == t.dst)) continue;
            store_tile(t, cut_of(t), h, scale);
        }
    }
}

template <bool kMax>
cudaError_t launch_clip(const vc_clip_tile_t* tiles, int ntiles, bool clip, float max_norm, float eps,
                        float* norm, Part* parts, cudaStream_t st) {
    const int blocks = clip_blocks(ntiles);
    // what the second-level cache can hold for the second kernel
    const int again = clip ? (int)(kCacheBytes / kTileBytes / blocks) : 0;
    const cudaError_t e = launch_pdl(norm_kernel<kMax>, dim3(blocks), dim3(kClipThreads), st, tiles,
                                     ntiles, again, parts);
    if (e != cudaSuccess) return e;
    if (clip)
        return launch_pdl(clip_kernel<kMax, true>, dim3(blocks), dim3(kClipThreads), st, tiles, ntiles,
                          (const Part*)parts, blocks, max_norm, eps, norm);
    return launch_pdl(clip_kernel<kMax, false>, dim3(1), dim3(kClipThreads), st, tiles, ntiles,
                      (const Part*)parts, blocks, max_norm, eps, norm);
}

vc_status_t run_clip(const vc_clip_tile_t* dev_tiles, int ntiles, vc_grad_norm_t kind, bool clip,
                     float max_norm, float eps, float* norm, void* workspace, size_t workspace_bytes,
                     vc_stream_t stream) {
    if (ntiles < 0 || (ntiles > 0 && dev_tiles == nullptr) ||
        reinterpret_cast<uintptr_t>(dev_tiles) % 16 != 0)
        return VC_ERR_INVALID_ARGUMENT;
    if (kind != VC_GRAD_NORM_L2 && kind != VC_GRAD_NORM_MAX) return VC_ERR_INVALID_ARGUMENT;
    if (norm == nullptr || reinterpret_cast<uintptr_t>(norm) % 4 != 0) return VC_ERR_INVALID_ARGUMENT;
    if (clip && (!(max_norm >= 0.0f) || !(eps >= 0.0f))) return VC_ERR_INVALID_ARGUMENT;
    const size_t need = vc_clip_workspace(ntiles);
    if (!workspace_ok(workspace, workspace_bytes, need)) return VC_ERR_INVALID_ARGUMENT;
    const Span table = span_of(dev_tiles, sizeof(vc_clip_tile_t) * (size_t)ntiles),
               out = span_of(norm, 4), ws = span_of(workspace, need);
    if (overlap(table, out) || overlap(table, ws) || overlap(out, ws)) return VC_ERR_ALIAS;
    if (test_launch_failure()) return VC_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    Part* parts = static_cast<Part*>(workspace);
    const cudaError_t e =
        kind == VC_GRAD_NORM_MAX
            ? launch_clip<true>(dev_tiles, ntiles, clip, max_norm, eps, norm, parts, st)
            : launch_clip<false>(dev_tiles, ntiles, clip, max_norm, eps, norm, parts, st);
    return e == cudaSuccess ? VC_SUCCESS : VC_ERR_CUDA;
}

// Whether outputs overlap each other, or an input other than their own.  Sorts
// the tiles in place by output, and back.
bool tiles_alias(vc_clip_tile_t* tiles, int n) {
    auto bytes = [](const vc_clip_tile_t& t) {
        return (uintptr_t)t.count * (t.flags & kTileF32 ? 4 : 2);
    };
    auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
    auto by_place = [&](const vc_clip_tile_t& a, const vc_clip_tile_t& b) { return at(a.dst) < at(b.dst); };
    const bool sorted = std::is_sorted(tiles, tiles + n, by_place);
    if (!sorted) std::sort(tiles, tiles + n, by_place);
    bool bad = false;
    for (int i = 0; i + 1 < n; ++i) bad = bad || at(tiles[i].dst) + bytes(tiles[i]) > at(tiles[i + 1].dst);
    for (int i = 0; i < n && !bad; ++i) {
        const uintptr_t lo = at(tiles[i].src), hi = lo + bytes(tiles[i]);
        // the first output that ends behind the input's start
        const vc_clip_tile_t* o = std::partition_point(
            tiles, tiles + n, [&](const vc_clip_tile_t& t) { return at(t.dst) + bytes(t) <= lo; });
        for (; o != tiles + n && at(o->dst) < hi && !bad; ++o)
            bad = !(o == tiles + i && at(o->dst) == lo);
    }
    if (!sorted)
        std::sort(tiles, tiles + n,
                  [](const vc_clip_tile_t& a, const vc_clip_tile_t& b) { return a.index < b.index; });
    return bad;
}

}  // namespace
}  // namespace step
}  // namespace vc

using namespace vc;
using namespace vc::step;

extern "C" {

vc_status_t vc_clip_plan(const void* const* grads, void* const* outs, const size_t* counts,
                         const vc_dtype_t* dtypes, int ntensors, vc_clip_tile_t* tiles,
                         int max_tiles, int* ntiles) {
    if (ntensors < 0 || ntiles == nullptr || max_tiles < 0) return VC_ERR_INVALID_ARGUMENT;
    if (ntensors > 0 && (grads == nullptr || counts == nullptr || dtypes == nullptr))
        return VC_ERR_INVALID_ARGUMENT;
    long long total = 0;
    for (int k = 0; k < ntensors; ++k) {
        if (!valid_dtype(dtypes[k])) return VC_ERR_INVALID_ARGUMENT;
        const int es = elem_size(dtypes[k]);
        const size_t per = kTileBytes / es;
        if (counts[k] > (1ull << 46)) return VC_ERR_INVALID_ARGUMENT;
        if (counts[k] > 0 &&
            (grads[k] == nullptr || reinterpret_cast<uintptr_t>(grads[k]) % es != 0 ||
             (outs != nullptr && (outs[k] == nullptr || reinterpret_cast<uintptr_t>(outs[k]) % es != 0))))
            return VC_ERR_INVALID_ARGUMENT;
        total += (long long)((counts[k] + per - 1) / per);
        if (total > 0x7FFFFFFF) return VC_ERR_INVALID_ARGUMENT;
    }
    *ntiles = (int)total;
    if (tiles == nullptr) return VC_SUCCESS;
    if (max_tiles < total) return VC_ERR_INVALID_ARGUMENT;
    int n = 0;
    for (int k = 0; k < ntensors; ++k) {
        const int es = elem_size(dtypes[k]);
        const size_t per = kTileBytes / es;
        for (size_t at = 0; at < counts[k]; at += per) {
            vc_clip_tile_t& t = tiles[n];
            t.src = static_cast<const char*>(grads[k]) + at * es;
            t.dst = outs == nullptr ? nullptr : static_cast<char*>(outs[k]) + at * es;
            t.count = (int)std::min(per, counts[k] - at);
            t.flags = dtypes[k] == VC_FLOAT32 ? kTileF32 : 0;
            t.index = n++;
        }
    }
    bool in_place = outs != nullptr;
    for (int i = 0; i < n && in_place; ++i) in_place = tiles[i].src == tiles[i].dst;
    for (int i = 0; i < n && in_place; ++i) tiles[i].flags |= kAllInPlace;
    return outs != nullptr && tiles_alias(tiles, n) ? VC_ERR_ALIAS : VC_SUCCESS;
}

size_t vc_clip_workspace(int ntiles) {
    return ntiles < 0 ? 0 : round256(sizeof(Part) * clip_blocks(ntiles));
}

vc_status_t vc_grad_norm(const vc_clip_tile_t* dev_tiles, int ntiles, vc_grad_norm_t kind,
                         float* norm, void* workspace, size_t workspace_bytes, vc_stream_t stream) {
    return run_clip(dev_tiles, ntiles, kind, false, 0.0f, 0.0f, norm, workspace, workspace_bytes,
                    stream);
}

vc_status_t vc_clip_grad_norm(const vc_clip_tile_t* dev_tiles, int ntiles, vc_grad_norm_t kind,
                              float max_norm, float eps, float* norm, void* workspace,
                              size_t workspace_bytes, vc_stream_t stream) {
    return run_clip(dev_tiles, ntiles, kind, true, max_norm, eps, norm, workspace, workspace_bytes,
                    stream);
}

}  // extern "C"
