// vc_block_norm_forward / vc_block_norm_backward: the norm behind a block, its
// gate, the residual and the norm before the next block in one pass over the rows.
// Here: what both directions share.
//
//   u = post(h),  r = a x + act(gate) u,  n = pre(r)
//
// Every matrix is read or written once; the bound is their bytes.  A team of
// threads (a warp for short rows, a whole block or a cluster of blocks for long ones)
// holds a row, eight columns a thread and vector, between the sums that the norms
// need: in registers, or in shared memory where it has come through that.  Rows that
// are longer than a cluster can hold (65536 values, 32768 in the gradient) are read
// again for every sum (from the caches), by kernels of their own.
//
// The gradient's column sums (weights, biases, a gate that rows share) stay in
// registers over the rows of a team, which are neighbours, and go to the
// workspace once; a second kernel adds those parts in order.  The statistics are
// computed again from r and h, which the gradient reads anyway.
#pragma once

#include <algorithm>
#include <initializer_list>

#include "vc_step_common.cuh"

namespace vc {
namespace step {

enum { kGateNone = 0, kGateShared = 1, kGateFull = 2, kGateGroups = 3 };

struct Affine {
    Rows weight, bias;
};

struct NormParams {
    // forward: h, x, gate -> r, n; backward: dr, dn, r, h, gate -> dx, dh, dgate
    Rows h, x, gate, r, n, dr, dn, dx, dh, dgate;
    Affine post, pre;
    long long rows, group;  // rows that share a gate row
    int cols, vec;
    int gate_mode, sigmoid, accumulate;
    int stream_gate;  // backward: a gate for every element comes as the other matrices do
    float scale, eps, inv_cols;
    // backward: parts[block][kind][padded], slots[team][2][padded]
    float *parts, *slots;
    long long padded;
    int kinds;  // bits of enum kSum
    int teams, blocks;
    int span;  // blocks of a cluster that share a row
    long long gates;  // rows of dgate, where there are no rows
    unsigned* timeouts;
    Affine dpost, dpre;
};
enum { kSumPre = 0, kSumPreBias = 1, kSumPost = 2, kSumPostBias = 3, kSumGate = 4, kSums = 5 };

// Eight neighbours of a row of any alignment, outside of the kernels' streams.
template <int kTeam>
__device__ __forceinline__ Eight load_near(const Rows& x, long long row, int v, int lane, int cols) {
    if (x.vec) return load_any<kTeam>(x, row, true, v, lane, cols);
    const int c = (v * kTeam + lane) * 8;
    const long long at = row * x.ld + c;
    Eight r;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        r.v[j] = c + j >= cols ? 0.0f
                 : x.f32       ? static_cast<const float*>(x.data)[at + j]
                               : __bfloat162float(static_cast<const __nv_bfloat16*>(x.data)[at + j]);
    return r;
}

// 16 bytes from byte `off` (even, below 16) of 32 on; 32 from byte `off` (a multiple of
// 4) of 48 on.
__device__ __forceinline__ uint4 cut16(uint4 lo, uint4 hi, unsigned off) {
    unsigned w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int j = 0; j < 6; ++j) w[j] = off & 8 ? w[j + 2] : w[j];
#pragma unroll
    for (int j = 0; j < 5; ++j) w[j] = off & 4 ? w[j + 1] : w[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], (off & 2) * 8);
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ Eight cut32(uint4 a, uint4 b, uint4 c, unsigned off) {
    unsigned w[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
#pragma unroll
    for (int j = 0; j < 10; ++j) w[j] = off & 8 ? w[j + 2] : w[j];
#pragma unroll
    for (int j = 0; j < 9; ++j) w[j] = off & 4 ? w[j + 1] : w[j];
    Eight r;
#pragma unroll
    for (int j = 0; j < 8; ++j) r.v[j] = __uint_as_float(w[j]);
    return r;
}

// Eight neighbours to a row of any alignment, by a whole warp.  Off 16 bytes, each lane
// stores the 16-byte words that its first values end, with the last ones of the lane
// before it; what no word of the warp covers goes value by value.  (Value by value all
// of it is eight accesses of 16 sectors each.)
template <int kTeam>
__device__ __forceinline__ void store_near(const Rows& x, bool f32, long long row, int v, int lane, int cols,
                                           const Eight& r) {
    const int es = f32 ? 4 : 2, c = (v * kTeam + lane) * 8, l = lane & 31;
    char* const to = static_cast<char*>(x.data) + (row * x.ld + c) * es;
    const unsigned off = (unsigned)reinterpret_cast<uintptr_t>(to) & 15;
    if (off == 0) return store_any<kTeam>(x, f32, row, true, v, lane, cols, r);
    const int first = 8 - (int)off / es;  // of the lane's values, in its own words
    const bool own = l > 0 && c + first <= cols, next = l < 31 && c + 8 + first <= cols;
    if (f32) {
        uint4 before, a, b;
        a = make_uint4(__float_as_uint(r.v[0]), __float_as_uint(r.v[1]), __float_as_uint(r.v[2]), __float_as_uint(r.v[3]));
        b = make_uint4(__float_as_uint(r.v[4]), __float_as_uint(r.v[5]), __float_as_uint(r.v[6]), __float_as_uint(r.v[7]));
        before.x = __shfl_up_sync(~0u, b.x, 1), before.y = __shfl_up_sync(~0u, b.y, 1);
        before.z = __shfl_up_sync(~0u, b.z, 1), before.w = __shfl_up_sync(~0u, b.w, 1);
        const Eight o = cut32(before, a, b, 16 - off);
        if (own) {
            float4* const at = reinterpret_cast<float4*>(to - off);
            at[0] = make_float4(o.v[0], o.v[1], o.v[2], o.v[3]);
            at[1] = make_float4(o.v[4], o.v[5], o.v[6], o.v[7]);
        }
    } else {
        const uint4 a = narrow(r);
        uint4 before;
        before.x = __shfl_up_sync(~0u, a.x, 1), before.y = __shfl_up_sync(~0u, a.y, 1);
        before.z = __shfl_up_sync(~0u, a.z, 1), before.w = __shfl_up_sync(~0u, a.w, 1);
        const uint4 o = cut16(before, a, 16 - off);
        if (own) *reinterpret_cast<uint4*>(to - off) = o;
    }
    if (own && next) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if ((j < first ? own : next) || c + j >= cols) continue;
        if (f32)
            reinterpret_cast<float*>(to)[j] = r.v[j];
        else
            reinterpret_cast<__nv_bfloat16*>(to)[j] = __float2bfloat16(r.v[j]);
    }
}

// The rows of up to five matrices as a team passes over them.  Rows on 16 bytes come
// through shared memory (kRing): each thread copies its own columns of the next row
// (asynchronously, so that they cost no registers on the way) while it works on this
// one, and no other thread reads them.  Others are held in registers, from where the
// last one has been used up, or where there are too few of those come through shared
// memory as well (kRing without kVec): the thread copies the 16-byte words that its
// columns lie in, two or three, and shifts them when it reads them.  The words' other
// bytes are read but not used.
constexpr int kStages = 2;

template <int kThreads, int kTeam, int kVecs, int kArrays, bool kVec, bool kRing>
struct Stream {
    uint4* ring;       // [stage][word][thread]
    int words, stage;  // of a row; the one that is read
    int at[kArrays];   // an array's first word
    bool f32[kArrays];
    int v0;            // the block's first vector
    // what there is of the thread's columns, in bytes of 16 or 32 bits a value, and where
    int bytes[kRing ? 3 : 1][kRing ? kVecs : 1], offset[kRing ? kVecs : 1];
    unsigned here, there;  // four bits an array: the row's byte in a 16-byte word
    Raw raw[kRing ? 1 : kArrays][kRing ? 1 : kVecs];

    __device__ __forceinline__ void begin(uint4* shared, int first, int lane, int cols) {
        ring = shared + threadIdx.x;
        words = stage = 0;
        here = there = 0;
        v0 = first;
        if constexpr (kRing)
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int c = ((v0 + i) * kTeam + lane) * 8, n = cols - c;
                bytes[0][i] = max(0, min(16, n * 2));
                bytes[1][i] = max(0, min(16, n * 4));
                bytes[2][i] = max(0, min(16, n * 4 - 16));
                offset[i] = n > 0 ? c : 0;  // (nothing is read where there is nothing)
            }
    }
    __device__ __forceinline__ void array(int a, bool present, bool wide) {
        at[a] = words;
        f32[a] = wide;
        if (present) words += kVecs * ((wide ? 2 : 1) + (kRing && !kVec));
    }
    __device__ __forceinline__ void load(int a, const Rows& x, long long row, int lane, int cols) {
        if constexpr (kRing && !kVec) {
            uint4* const to = ring + ((stage ^ 1) * words + at[a]) * kThreads;
            const char* const from = static_cast<const char*>(x.data) + row * x.ld * (f32[a] ? 4 : 2);
            // (eight columns are whole words: the same for all of the row)
            const unsigned off = (unsigned)reinterpret_cast<uintptr_t>(from) & 15;
            there = (there & ~(15u << 4 * a)) | off << 4 * a;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int n = f32[a] ? bytes[1][i] + bytes[2][i] : bytes[0][i], end = n > 0 ? n + (int)off : 0;
                const char* const first = from + offset[i] * (f32[a] ? 4 : 2) - off;
                auto word = [&](int w, int k) {
                    copy16(to + w * kThreads, first + (end > 16 * k ? 16 * k : 0), max(0, min(16, end - 16 * k)));
                };
                if (f32[a]) {
                    word(i * 3, 0);
                    word(i * 3 + 1, 1);
                    word(i * 3 + 2, 2);
                } else {
                    word(i * 2, 0);
                    word(i * 2 + 1, 1);
                }
            }
        } else if constexpr (kRing) {
            uint4* to = ring + ((stage ^ 1) * words + at[a]) * kThreads;
            if (f32[a]) {
                const float* from = static_cast<const float*>(x.data) + row * x.ld;
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    copy16(to + i * 2 * kThreads, from + offset[i], bytes[1][i]);
                    copy16(to + (i * 2 + 1) * kThreads, from + offset[i] + (bytes[2][i] ? 4 : 0), bytes[2][i]);
                }
            } else {
                const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(x.data) + row * x.ld;
#pragma unroll
                for (int i = 0; i < kVecs; ++i) copy16(to + i * kThreads, from + offset[i], bytes[0][i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) raw[a][i] = load_raw<kTeam>(x, f32[a], row, kVec, v0 + i, lane, cols);
        }
    }
    // What has been loaded is read from here on.
    __device__ __forceinline__ void turn() {
        stage ^= 1;
        if constexpr (kRing && !kVec) {
            const unsigned h = here;
            here = there;
            there = h;
        }
    }
    // kOther: from the stage that loads write to.
    template <bool kOther = false>
    __device__ __forceinline__ Eight get(int a, int i) const {
        if constexpr (kRing) {
            const uint4* from = ring + ((kOther ? stage ^ 1 : stage) * words + at[a]) * kThreads;
            if constexpr (!kVec) {
                const unsigned off = (kOther ? there : here) >> 4 * a & 15;
                if (!f32[a]) return widen(cut16(from[i * 2 * kThreads], from[(i * 2 + 1) * kThreads], off));
                from += i * 3 * kThreads;
                return cut32(from[0], from[kThreads], from[2 * kThreads], off);
            }
            if (!f32[a]) return widen(from[i * kThreads]);
            const uint4 lo = from[i * 2 * kThreads], hi = from[(i * 2 + 1) * kThreads];
            return {{__uint_as_float(lo.x), __uint_as_float(lo.y), __uint_as_float(lo.z), __uint_as_float(lo.w),
                     __uint_as_float(hi.x), __uint_as_float(hi.y), __uint_as_float(hi.z), __uint_as_float(hi.w)}};
        } else {
            return widen_raw(raw[a][i], f32[a], kVec);
        }
    }
};

// A vector of the row's length that is used in every row (a weight, a bias, the gate
// of the rows at hand): in shared memory, in 32 bits, each thread's own columns.
template <int kTeam, int kVecs, class Access>
struct Held {
    static constexpr int kBytes = kVecs * 2 * kTeam * 16;
    float4* at;  // [vector][half][lane]
    __device__ __forceinline__ void put(int i, const Eight& x) const {
        at[i * 2 * kTeam] = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
        at[(i * 2 + 1) * kTeam] = make_float4(x.v[4], x.v[5], x.v[6], x.v[7]);
    }
    __device__ __forceinline__ void hold(const Rows& x, int v0, int lane, int cols) const {
        if (x.data != nullptr)
#pragma unroll
            for (int i = 0; i < kVecs; ++i) put(i, Access{v0 + i, lane, cols}.load(x, 0));
    }
    __device__ __forceinline__ Eight get(int i) const {
        const float4 lo = at[i * 2 * kTeam], hi = at[(i * 2 + 1) * kTeam];
        return {{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
    }
};

// ---------------------------------------------------------------------- sums --

// Sums over a team of up to four values at a time.  A warp's lanes share the values
// out while they add (of four values each lane keeps two, then one), the warps of a
// block leave theirs in shared memory, the blocks of a cluster in that of every one.
// Calls take turns between two buffers there, so that one wait a call does.
//
// In a cluster the values bring their own signal: they are counted on a barrier of the
// block that they go to.  (The cluster's own barrier also waits for all that its blocks
// have stored to memory: 1.4 us a call.)  Its waits are bounded as those of the
// products' kernels are: a block whose wait runs out goes on without, and is counted.
constexpr int kMaxSpan = 8;  // blocks of a cluster that share a row

struct SpanShared {
    unsigned long long barrier[2];
    int dead;
};

template <int kTeam, bool kSpan>
struct TeamSums {
    static constexpr int kWarps = kTeam / 32, kAll = kWarps + (kSpan ? kMaxSpan : 0);
    float (*shared)[4];  // [2 * kAll][4]
    int turn, span;      // blocks that share a row
    SpanShared* signals;
    unsigned parity;
    // Of a cluster: before the first call, and after the last one.
    __device__ __forceinline__ void begin() {
        const unsigned bar = gemm::smem_u32(signals->barrier);
        if (threadIdx.x == 0) {
            signals->dead = 0;
            gemm::mbar_init(bar, 1);
            gemm::mbar_init(bar + 8, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        cluster_sync();
    }
    __device__ __forceinline__ void end(unsigned* timeouts) {
        if (threadIdx.x == 0 && *static_cast<volatile int*>(&signals->dead)) atomicAdd(timeouts, 1u);
        cluster_sync();  // (no block leaves while others still send to it)
    }
    template <int kN>
    __device__ __forceinline__ void operator()(float (&v)[kN]) {
        static_assert(kN <= 4, "a buffer has four columns");
        constexpr int kP = kN == 3 ? 4 : kN;
        const int lane = threadIdx.x & 31;
        float c;
        if constexpr (kP == 4) {
            const bool high = lane & 16, odd = lane & 8;
            const float v3 = kN == 4 ? v[kN - 1] : 0.0f;
            float a = high ? v[2] : v[0], b = high ? v3 : v[1];
            a += __shfl_xor_sync(~0u, high ? v[0] : v[2], 16);
            b += __shfl_xor_sync(~0u, high ? v[1] : v3, 16);
            c = (odd ? b : a) + __shfl_xor_sync(~0u, odd ? a : b, 8);
        } else if constexpr (kP == 2) {
            const bool high = lane & 16;
            c = (high ? v[1] : v[0]) + __shfl_xor_sync(~0u, high ? v[0] : v[1], 16);
        } else {
            c = v[0];
        }
#pragma unroll
        for (int o = 16 / kP; o > 0; o >>= 1) c += __shfl_xor_sync(~0u, c, o);
        if constexpr (kTeam == 32) {
#pragma unroll
            for (int i = 0; i < kN; ++i) v[i] = __shfl_sync(~0u, c, i * (32 / kP));
        } else {
            float(*buf)[4] = shared + turn * kAll;
            const int q = lane % kP, w = lane / kP;
            if (lane % (32 / kP) == 0) buf[threadIdx.x >> 5][lane / (32 / kP)] = c;
            __syncthreads();
            c = w < kWarps ? buf[w][q] : 0.0f;
#pragma unroll
            for (int more = 32 / kP; more < kWarps; more += 32 / kP)
                if (w + more < kWarps) c += buf[w + more][q];
#pragma unroll
            for (int o = 16; o >= kP; o >>= 1) c += __shfl_xor_sync(~0u, c, o);
            if constexpr (kSpan) {
                // one lane a value sends the block's to every block
                float(*all)[4] = buf + kWarps;
                const unsigned bar = gemm::smem_u32(&signals->barrier[turn]);
                if (threadIdx.x < kP)
                    for (int r = 0; r < span; ++r)
                        asm volatile(
                            "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                                remote_address(&all[blockIdx.x % span][q], r)),
                            "r"(__float_as_uint(c)), "r"(remote_address(&signals->barrier[turn], r))
                            : "memory");
                if (threadIdx.x == 0) gemm::mbar_expect(bar, span * kP * 4);
                gemm::warp_wait(bar, parity >> turn & 1, &signals->dead);
                parity ^= 1u << turn;
#pragma unroll
                for (int i = 0; i < kN; ++i) v[i] = 0.0f;
                for (int r = 0; r < span; ++r)
#pragma unroll
                    for (int i = 0; i < kN; ++i) v[i] += all[r][i];
            } else {
#pragma unroll
                for (int i = 0; i < kN; ++i) v[i] = __shfl_sync(~0u, c, i);
            }
            turn ^= 1;
        }
    }
};

__device__ __forceinline__ float gate_value(float g, bool sigmoid) {
    return sigmoid ? train::logistic(g) : g;
}
__device__ __forceinline__ float gate_slope(float g, bool sigmoid) {
    if (!sigmoid) return 1.0f;
    const float s = train::logistic(g);
    return s * train::logistic(-g);  // (1 - s would lose what is left of it near 1)
}
__device__ __forceinline__ Eight gate_value(const Eight& g, bool sigmoid) {
    if (!sigmoid) return g;
    Eight r;
#pragma unroll
    for (int j = 0; j < 8; ++j) r.v[j] = train::logistic(g.v[j]);
    return r;
}
__device__ __forceinline__ long long gate_row(const NormParams& p, long long row) {
    return p.gate_mode == kGateFull ? row : p.gate_mode == kGateGroups ? row / p.group : 0;
}

// v minus its mean in the columns that are there, zeros beyond them.
template <int kTeam>
__device__ __forceinline__ Eight centered(const Eight& v, float mean, bool vec, int i, int lane, int cols) {
    Eight r = add(-mean, v);
    if (vec ? (i * kTeam + lane) * 8 + 8 > cols : true)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (column<kTeam>(vec, i, lane, j) >= cols) r.v[j] = 0.0f;
    return r;
}

// Takes the row's mean off (LAYER) and returns 1 / sqrt(mean square + eps).
template <int kVecs, bool kLayer, int kTeam, bool kSpan>
__device__ __forceinline__ float center(const NormParams& p, Eight (&v)[kVecs], bool vec, int v0, int lane,
                                        TeamSums<kTeam, kSpan>& sums) {
    if constexpr (kLayer) {
        float2 part = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) total(part, v[i]);
        float s[1] = {sum_of(part)};
        sums(s);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = centered<kTeam>(v[i], s[0] * p.inv_cols, vec, v0 + i, lane, p.cols);
    }
    float2 part = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) dot(part, v[i], v[i]);
    float s[1] = {sum_of(part)};
    sums(s);
    return rsqrtf(fmaf(s[0], p.inv_cols, p.eps));
}

// Rows that are too long for a cluster's registers: a block a row, in steps of 8 *
// kLong columns, the inputs read again for every sum.
constexpr int kLong = 512;

template <bool kLayer, class F>
__device__ __forceinline__ void long_statistics(const NormParams& p, TeamSums<kLong, false>& sums, int steps, int lane,
                                                F load, float& mean, float& rstd) {
    mean = 0.0f;
    if constexpr (kLayer) {
        float s[1] = {0.0f};
        for (int i = 0; i < steps; ++i) {
            const Eight v = load(i);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += v.v[j];
        }
        sums(s);
        mean = s[0] * p.inv_cols;
    }
    float s[1] = {0.0f};
    for (int i = 0; i < steps; ++i) {
        const Eight v = load(i);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = v.v[j] - mean;
            if (!kLayer || column<kLong>(p.vec, i, lane, j) < p.cols) s[0] = fmaf(d, d, s[0]);
        }
    }
    sums(s);
    rstd = rsqrtf(fmaf(s[0], p.inv_cols, p.eps));
}

__device__ __forceinline__ Eight normalised(const NormParams& p, const Affine& a, Eight v, float mean, float rstd,
                                            int i, int lane) {
    const Eight w = load_any<kLong>(a.weight, 0, p.vec, i, lane, p.cols);
#pragma unroll
    for (int j = 0; j < 8; ++j) v.v[j] = (v.v[j] - mean) * rstd * w.v[j];
    if (a.bias.data != nullptr) {
        const Eight b = load_any<kLong>(a.bias, 0, p.vec, i, lane, p.cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) v.v[j] += b.v[j];
    }
    return v;
}

// ---------------------------------------------------------------- arguments --

// A row of `cols` columns by `team` threads of each of `span` blocks, with `vecs`
// vectors each; team 0: the kernels for the longest rows.
struct Shape {
    int team, vecs, span;
};

// Clusters of `span` blocks that run at a time on a GB300, with one or two blocks on an SM
// (what its occupancy query says: a cluster's SMs are of one group).
inline int clusters_of(int span, int per_sm) {
    constexpr int kOne[kMaxSpan + 1] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
    constexpr int kTwo[kMaxSpan + 1] = {0, 304, 152, 97, 74, 58, 46, 38, 36};
    return (per_sm > 1 ? kTwo : kOne)[span];
}

inline bool valid_affine(const vc_affine_t* a, bool needed) {
    if (a == nullptr || a->weight == nullptr) return !needed && (a == nullptr || a->bias == nullptr);
    const int es = elem_size(a->dtype);
    return es != 0 && reinterpret_cast<uintptr_t>(a->weight) % es == 0 &&
           reinterpret_cast<uintptr_t>(a->bias) % es == 0;
}
inline bool has_bias(const vc_affine_t* a) { return a != nullptr && a->bias != nullptr; }
inline Rows vector_of(void* data, vc_dtype_t dtype) {
    return {data, 0, dtype == VC_FLOAT32, reinterpret_cast<uintptr_t>(data) % 16 == 0};
}
inline Affine affine_of(const vc_affine_t* a) {
    if (a == nullptr || (a->weight == nullptr && a->bias == nullptr)) return {};
    return {vector_of(a->weight, a->dtype), vector_of(a->bias, a->dtype)};
}
inline bool valid_args(const vc_block_norm_t* a) {
    return a != nullptr && (a->norm == VC_NORM_RMS || a->norm == VC_NORM_LAYER) &&
           (a->gate_act == VC_GATE_NONE || a->gate_act == VC_GATE_SIGMOID) && a->eps >= 0.0f;
}
// [G, D] with G a divisor of the rows (any where there are none).
inline bool valid_gate(const vc_matrix_t* g, long long rows, long long cols) {
    return valid_matrix(g) && g->batch == 1 && g->cols == cols && g->rows > 0 && rows % g->rows == 0;
}
inline bool is_bf16(const vc_matrix_t* m) { return m->dtype == VC_BFLOAT16; }
inline int mode_of(const vc_matrix_t* g, long long rows) {
    return g == nullptr ? kGateNone : g->rows == 1 ? kGateShared : g->rows == rows ? kGateFull : kGateGroups;
}
inline Span span_of_vector(const void* p, vc_dtype_t dtype, long long cols) {
    return span_of(p, (size_t)cols * elem_size(dtype));
}

inline void common_params(NormParams* p, const vc_matrix_t* gate, const vc_affine_t* post, const vc_affine_t* pre,
                   const vc_block_norm_t* args, long long rows, long long cols) {
    p->gate = rows_of(gate);
    p->post = affine_of(post);
    p->pre = affine_of(pre);
    p->rows = rows;
    p->cols = (int)cols;
    p->gate_mode = mode_of(gate, rows);
    p->group = gate == nullptr ? 1 : rows / gate->rows;
    p->sigmoid = args->gate_act == VC_GATE_SIGMOID;
    p->scale = args->residual_scale;
    p->eps = args->eps;
    p->inv_cols = (float)(1.0 / (double)cols);
}
// Whether all that is there lies on 16 bytes.
inline bool all_vec(std::initializer_list<const Rows*> xs) {
    bool vec = true;
    for (const Rows* x : xs) vec = vec && (x->data == nullptr || x->vec);
    return vec;
}

}  // namespace step
}  // namespace vc
