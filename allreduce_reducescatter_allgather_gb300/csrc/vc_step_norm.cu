// vc_block_norm_forward / vc_block_norm_backward: the norm behind a block, its
// gate, the residual and the norm before the next block in one pass over the rows.
//
//   u = post(h),  r = a x + act(gate) u,  n = pre(r)
//
// Every matrix is read or written once; the bound is their bytes.  A team of
// threads (a warp for short rows, a whole block for long ones) holds a row in
// registers, eight columns a thread and vector, between the sums that the norms
// need.  Rows that are longer than a team can hold are read again for every sum
// (from the caches), by kernels of their own.
//
// The gradient's column sums (weights, biases, a gate that rows share) stay in
// registers over the rows of a team, which are neighbours, and go to the
// workspace once; a second kernel adds those parts in order.  The statistics are
// computed again from r and h, which the gradient reads anyway.
#include <algorithm>
#include <initializer_list>

#include "vc_step_common.cuh"

namespace vc {
namespace step {
namespace {

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
    float scale, eps, inv_cols;
    // backward: parts[block][kind][padded], slots[team][2][padded]
    float *parts, *slots;
    long long padded;
    int kinds;  // bits of enum kSum
    int teams, blocks;
    Affine dpost, dpre;
};
enum { kSumPre = 0, kSumPreBias = 1, kSumPost = 2, kSumPostBias = 3, kSumGate = 4, kSums = 5 };

// ------------------------------------------------------------------- columns --

// The columns of thread `lane` of a team in its v-th vector: eight neighbours on
// 16 bytes, or every kTeam-th one.
template <int kTeam>
__device__ __forceinline__ int column(bool vec, int v, int lane, int j) {
    return vec ? (v * kTeam + lane) * 8 + j : (v * 8 + j) * kTeam + lane;
}

template <int kTeam>
__device__ __forceinline__ Eight load_f32(const void* data, long long at, bool vec, int v, int lane, int cols) {
    const float* p = static_cast<const float*>(data) + at;
    const int c = (v * kTeam + lane) * 8;
    if (vec && c + 8 <= cols) {
        const float4 lo = *reinterpret_cast<const float4*>(p + c), hi = *reinterpret_cast<const float4*>(p + c + 4);
        return {{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
    }
    Eight r;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int k = column<kTeam>(vec, v, lane, j);
        r.v[j] = k < cols ? p[k] : 0.0f;
    }
    return r;
}
template <int kTeam>
__device__ __forceinline__ Eight load_bf16(const void* data, long long at, bool vec, int v, int lane, int cols) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(data) + at;
    const int c = (v * kTeam + lane) * 8;
    if (vec && c + 8 <= cols) return widen(*reinterpret_cast<const uint4*>(p + c));
    Eight r;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int k = column<kTeam>(vec, v, lane, j);
        r.v[j] = k < cols ? __bfloat162float(p[k]) : 0.0f;
    }
    return r;
}
template <int kTeam>
__device__ __forceinline__ Eight load_any(const Rows& x, long long row, bool vec, int v, int lane, int cols) {
    return x.f32 ? load_f32<kTeam>(x.data, row * x.ld, vec, v, lane, cols)
                 : load_bf16<kTeam>(x.data, row * x.ld, vec, v, lane, cols);
}
template <int kTeam, bool kF32>
__device__ __forceinline__ Eight load_as(const Rows& x, long long row, bool vec, int v, int lane, int cols) {
    return kF32 ? load_f32<kTeam>(x.data, row * x.ld, vec, v, lane, cols)
                : load_bf16<kTeam>(x.data, row * x.ld, vec, v, lane, cols);
}
template <int kTeam>
__device__ __forceinline__ void store_any(const Rows& x, bool f32, long long row, bool vec, int v, int lane,
                                          int cols, const Eight& r) {
    float* f = static_cast<float*>(x.data) + row * x.ld;
    __nv_bfloat16* b = static_cast<__nv_bfloat16*>(x.data) + row * x.ld;
    const int c = (v * kTeam + lane) * 8;
    if (vec && c + 8 <= cols) {
        if (f32) {
            *reinterpret_cast<float4*>(f + c) = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
            *reinterpret_cast<float4*>(f + c + 4) = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
        } else {
            *reinterpret_cast<uint4*>(b + c) = narrow(r);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int k = column<kTeam>(vec, v, lane, j);
        if (k >= cols) continue;
        if (f32)
            f[k] = r.v[j];
        else
            b[k] = __float2bfloat16(r.v[j]);
    }
}

// ---------------------------------------------------------------------- sums --

// Sums over a team; the team is a warp, or the whole block, whose calls then take
// turns between two buffers, so that one barrier a call does.
template <int kTeam>
struct TeamSums {
    static constexpr int kWarps = kTeam / 32;
    float (*shared)[kWarps];  // [2 * 4][kWarps]
    int turn;
    template <int kN>
    __device__ __forceinline__ void operator()(float (&v)[kN]) {
        static_assert(kN <= 4, "a buffer has four rows");
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = warp_sum(v[i]);
        if constexpr (kTeam > 32) {
            float(*buf)[kWarps] = shared + turn * 4;
            turn ^= 1;
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int i = 0; i < kN; ++i) buf[i][threadIdx.x >> 5] = v[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                float s = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s += buf[i][w];
                v[i] = s;
            }
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
__device__ __forceinline__ long long gate_row(const NormParams& p, long long row) {
    return p.gate_mode == kGateFull ? row : p.gate_mode == kGateGroups ? row / p.group : 0;
}

// ------------------------------------------------------------------- forward --

constexpr int kForwardThreads = 128;  // of a block of teams that are warps

// The mean and 1 / sqrt(variance + eps) of the row in v (RMS: 0 and that of the
// mean square).
template <int kTeam, int kVecs, bool kLayer>
__device__ __forceinline__ void statistics(const NormParams& p, const Eight (&v)[kVecs], int lane,
                                           TeamSums<kTeam>& sums, float& mean, float& rstd) {
    mean = 0.0f;
    if constexpr (kLayer) {
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += v[i].v[j];
        sums(s);
        mean = s[0] * p.inv_cols;
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = v[i].v[j] - mean;
            if (!kLayer || column<kTeam>(p.vec, i, lane, j) < p.cols) s[0] = fmaf(d, d, s[0]);
        }
    sums(s);
    rstd = rsqrtf(fmaf(s[0], p.inv_cols, p.eps));
}

template <int kTeam, int kVecs, bool kLayer, bool kStream32>
__global__ void __launch_bounds__(kTeam == 32 ? kForwardThreads : kTeam) forward_kernel(const __grid_constant__ NormParams p) {
    constexpr int kTeams = (kTeam == 32 ? kForwardThreads : kTeam) / kTeam;
    __shared__ float shared[kTeam > 32 ? 8 : 1][kTeam / 32];
    TeamSums<kTeam> sums = {shared, 0};
    const int lane = threadIdx.x % kTeam;
    pdl_next();
    pdl_wait();
    for (long long row = (long long)blockIdx.x * kTeams + threadIdx.x / kTeam; row < p.rows;
         row += (long long)gridDim.x * kTeams) {
        Eight u[kVecs], x[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) u[i] = load_bf16<kTeam>(p.h.data, row * p.h.ld, p.vec, i, lane, p.cols);
        if (p.x.data != nullptr)
#pragma unroll
            for (int i = 0; i < kVecs; ++i) x[i] = load_as<kTeam, kStream32>(p.x, row, p.vec, i, lane, p.cols);
        if (p.post.weight.data != nullptr) {
            float mean, rstd;
            statistics<kTeam, kVecs, kLayer>(p, u, lane, sums, mean, rstd);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const Eight w = load_any<kTeam>(p.post.weight, 0, p.vec, i, lane, p.cols);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[i].v[j] = (u[i].v[j] - mean) * rstd * w.v[j];
                if (p.post.bias.data != nullptr) {
                    const Eight b = load_any<kTeam>(p.post.bias, 0, p.vec, i, lane, p.cols);
#pragma unroll
                    for (int j = 0; j < 8; ++j) u[i].v[j] += b.v[j];
                }
            }
        }
        if (p.gate_mode != kGateNone) {
            const long long g = gate_row(p, row);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const Eight v = load_any<kTeam>(p.gate, g, p.vec, i, lane, p.cols);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[i].v[j] *= gate_value(v.v[j], p.sigmoid);
            }
        }
        if (p.x.data != nullptr)
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) u[i].v[j] = fmaf(p.scale, x[i].v[j], u[i].v[j]);
        if (p.r.data != nullptr)
#pragma unroll
            for (int i = 0; i < kVecs; ++i) store_any<kTeam>(p.r, kStream32, row, p.vec, i, lane, p.cols, u[i]);
        if (p.n.data == nullptr) continue;
        float mean, rstd;
        statistics<kTeam, kVecs, kLayer>(p, u, lane, sums, mean, rstd);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const Eight w = load_any<kTeam>(p.pre.weight, 0, p.vec, i, lane, p.cols);
#pragma unroll
            for (int j = 0; j < 8; ++j) u[i].v[j] = (u[i].v[j] - mean) * rstd * w.v[j];
            if (p.pre.bias.data != nullptr) {
                const Eight b = load_any<kTeam>(p.pre.bias, 0, p.vec, i, lane, p.cols);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[i].v[j] += b.v[j];
            }
            store_any<kTeam>(p.n, false, row, p.vec, i, lane, p.cols, u[i]);
        }
    }
}

// Rows that are too long for registers: a block a row, in steps of 8 * kLong
// columns, the inputs read again for every sum.
constexpr int kLong = 512;

template <bool kLayer, class F>
__device__ __forceinline__ void long_statistics(const NormParams& p, TeamSums<kLong>& sums, int steps, int lane,
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

template <bool kLayer, bool kStream32>
__global__ void __launch_bounds__(kLong) forward_long_kernel(const __grid_constant__ NormParams p) {
    __shared__ float shared[8][kLong / 32];
    TeamSums<kLong> sums = {shared, 0};
    const int lane = threadIdx.x, steps = (p.cols + 8 * kLong - 1) / (8 * kLong);
    pdl_next();
    pdl_wait();
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        auto load_h = [&](int i) { return load_bf16<kLong>(p.h.data, row * p.h.ld, p.vec, i, lane, p.cols); };
        float mean = 0.0f, rstd = 0.0f;
        if (p.post.weight.data != nullptr) long_statistics<kLayer>(p, sums, steps, lane, load_h, mean, rstd);
        const long long g = gate_row(p, row);
        auto load_r = [&](int i) {
            Eight u = load_h(i);
            if (p.post.weight.data != nullptr) u = normalised(p, p.post, u, mean, rstd, i, lane);
            if (p.gate_mode != kGateNone) {
                const Eight v = load_any<kLong>(p.gate, g, p.vec, i, lane, p.cols);
#pragma unroll
                for (int j = 0; j < 8; ++j) u.v[j] *= gate_value(v.v[j], p.sigmoid);
            }
            if (p.x.data != nullptr) {
                const Eight x = load_as<kLong, kStream32>(p.x, row, p.vec, i, lane, p.cols);
#pragma unroll
                for (int j = 0; j < 8; ++j) u.v[j] = fmaf(p.scale, x.v[j], u.v[j]);
            }
            return u;
        };
        float r_mean = 0.0f, r_rstd = 0.0f;
        if (p.n.data != nullptr) long_statistics<kLayer>(p, sums, steps, lane, load_r, r_mean, r_rstd);
        // (x and h may be r and n: each column is read before it is written)
        for (int i = 0; i < steps; ++i) {
            const Eight r = load_r(i);
            if (p.r.data != nullptr) store_any<kLong>(p.r, kStream32, row, p.vec, i, lane, p.cols, r);
            if (p.n.data != nullptr)
                store_any<kLong>(p.n, false, row, p.vec, i, lane, p.cols,
                                 normalised(p, p.pre, r, r_mean, r_rstd, i, lane));
        }
    }
}

// ------------------------------------------------------------------ backward --

// The rows of team t: a run of neighbours.
__device__ __forceinline__ long long first_row(const NormParams& p, long long t) { return t * p.rows / p.teams; }

// A team's sum of dr u over the rows of group g that it has: the whole of it goes to
// dgate, a part to one of the team's two slots: 0 where the group started before
// its rows, 1 where it goes on behind them.
template <int kTeam>
__device__ __forceinline__ void flush_gate(const NormParams& p, long long team, long long g, long long lo,
                                           long long hi, int v, int lane, Eight sum) {
    const bool before = g * p.group < lo, behind = (g + 1) * p.group > hi;
    if (before || behind) {
        const Rows slot = {p.slots, p.padded, 1, 1};
        store_any<kTeam>(slot, true, team * 2 + (before ? 0 : 1), p.vec, v, lane, p.cols, sum);
        return;
    }
    const Eight gate = load_any<kTeam>(p.gate, g, p.vec, v, lane, p.cols);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum.v[j] *= gate_slope(gate.v[j], p.sigmoid);
    if (p.accumulate) {
        const Eight old = load_any<kTeam>(p.dgate, g, p.vec, v, lane, p.cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum.v[j] += old.v[j];
    }
    store_any<kTeam>(p.dgate, p.dgate.f32, g, p.vec, v, lane, p.cols, sum);
}

// A gate of its own for every element.
template <int kTeam>
__device__ __forceinline__ void store_gate(const NormParams& p, long long row, int v, int lane, Eight d,
                                           const Eight& gate) {
#pragma unroll
    for (int j = 0; j < 8; ++j) d.v[j] *= gate_slope(gate.v[j], p.sigmoid);
    if (p.accumulate) {
        const Eight old = load_any<kTeam>(p.dgate, row, p.vec, v, lane, p.cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) d.v[j] += old.v[j];
    }
    store_any<kTeam>(p.dgate, p.dgate.f32, row, p.vec, v, lane, p.cols, d);
}

constexpr int kBackwardThreads = 256;  // of a block of teams that are warps

template <int kTeam, int kVecs, bool kLayer, bool kStream32>
__global__ void __launch_bounds__(kTeam == 32 ? kBackwardThreads : kTeam) backward_kernel(const __grid_constant__ NormParams p) {
    constexpr int kThreads = kTeam == 32 ? kBackwardThreads : kTeam, kTeams = kThreads / kTeam;
    // RMS norms have no biases
    constexpr int kKept = kLayer ? 5 : 3;
    constexpr int kPre = 0, kPost = 1, kGate = 2, kPreBias = 3, kPostBias = 4;
    __shared__ float shared[kTeam > 32 ? 8 : 1][kTeam / 32];
    __shared__ float joined[kTeams > 1 ? kTeams : 1][kTeams > 1 ? 8 * kTeam * kVecs : 1];
    TeamSums<kTeam> sums = {shared, 0};
    const int lane = threadIdx.x % kTeam;
    const long long team = (long long)blockIdx.x * kTeams + threadIdx.x / kTeam;
    const bool has_pre = p.dn.data != nullptr, has_post = p.post.weight.data != nullptr;
    const bool needs_h = p.h.data != nullptr;
    const bool sums_gate = p.dgate.data != nullptr && (p.gate_mode == kGateShared || p.gate_mode == kGateGroups);
    Eight kept[kKept][kVecs];
#pragma unroll
    for (int k = 0; k < kKept; ++k)
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) kept[k][i].v[j] = 0.0f;
    pdl_next();
    pdl_wait();
    const long long lo = first_row(p, team), hi = first_row(p, team + 1);
    long long group_end = p.gate_mode == kGateGroups ? (lo / p.group + 1) * p.group : 0;
    for (long long row = lo; row < hi; ++row) {
        Eight dr[kVecs], h[kVecs], gate[kVecs];
        if (p.dr.data != nullptr) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) dr[i] = load_as<kTeam, kStream32>(p.dr, row, p.vec, i, lane, p.cols);
        } else {
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) dr[i].v[j] = 0.0f;
        }
        if (needs_h)
#pragma unroll
            for (int i = 0; i < kVecs; ++i) h[i] = load_bf16<kTeam>(p.h.data, row * p.h.ld, p.vec, i, lane, p.cols);
        if (p.gate_mode != kGateNone) {
            const long long g = gate_row(p, row);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) gate[i] = load_any<kTeam>(p.gate, g, p.vec, i, lane, p.cols);
        }
        if (has_pre) {
            Eight r[kVecs], dn[kVecs];
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                r[i] = load_as<kTeam, kStream32>(p.r, row, p.vec, i, lane, p.cols);
                dn[i] = load_bf16<kTeam>(p.dn.data, row * p.dn.ld, p.vec, i, lane, p.cols);
            }
            if constexpr (kLayer) {
                float s[1] = {0.0f};
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[0] += r[i].v[j];
                sums(s);
                const float mean = s[0] * p.inv_cols;
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        r[i].v[j] = column<kTeam>(p.vec, i, lane, j) < p.cols ? r[i].v[j] - mean : 0.0f;
            }
            float s[3] = {0.0f, 0.0f, 0.0f};
            Eight w[kVecs];
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                w[i] = load_any<kTeam>(p.pre.weight, 0, p.vec, i, lane, p.cols);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    w[i].v[j] *= dn[i].v[j];
                    s[0] = fmaf(r[i].v[j], r[i].v[j], s[0]);
                    s[1] = fmaf(w[i].v[j], r[i].v[j], s[1]);
                    if constexpr (kLayer) s[2] += w[i].v[j];
                }
            }
            sums(s);
            const float rstd = rsqrtf(fmaf(s[0], p.inv_cols, p.eps));
            const float m2 = s[1] * p.inv_cols * rstd, m1 = s[2] * p.inv_cols;
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float hat = r[i].v[j] * rstd;
                    kept[kPre][i].v[j] = fmaf(dn[i].v[j], hat, kept[kPre][i].v[j]);
                    if constexpr (kLayer) kept[kPreBias][i].v[j] += dn[i].v[j];
                    dr[i].v[j] = fmaf(rstd, w[i].v[j] - m1 - hat * m2, dr[i].v[j]);
                }
        }
        if (p.dx.data != nullptr)
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                Eight d;
#pragma unroll
                for (int j = 0; j < 8; ++j) d.v[j] = p.scale * dr[i].v[j];
                store_any<kTeam>(p.dx, kStream32, row, p.vec, i, lane, p.cols, d);
            }
        float rstd = 0.0f;
        if (has_post) {
            float mean = 0.0f;
            statistics<kTeam, kVecs, kLayer>(p, h, lane, sums, mean, rstd);
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i].v[j] = (h[i].v[j] - mean) * rstd;  // the hats
        }
        // dgate, and du in dr's place
        if (p.gate_mode != kGateNone) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                if (p.dgate.data != nullptr) {
                    Eight d = h[i];
                    if (has_post) {
                        const Eight w = load_any<kTeam>(p.post.weight, 0, p.vec, i, lane, p.cols);
#pragma unroll
                        for (int j = 0; j < 8; ++j) d.v[j] *= w.v[j];
                        if (p.post.bias.data != nullptr) {
                            const Eight b = load_any<kTeam>(p.post.bias, 0, p.vec, i, lane, p.cols);
#pragma unroll
                            for (int j = 0; j < 8; ++j) d.v[j] += b.v[j];
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) d.v[j] *= dr[i].v[j];
                    if (sums_gate) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) kept[kGate][i].v[j] += d.v[j];
                    } else {
                        store_gate<kTeam>(p, row, i, lane, d, gate[i]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) dr[i].v[j] *= gate_value(gate[i].v[j], p.sigmoid);
            }
            if (p.gate_mode == kGateGroups && (row + 1 == group_end || row + 1 == hi)) {
                if (sums_gate)
#pragma unroll
                    for (int i = 0; i < kVecs; ++i) {
                        flush_gate<kTeam>(p, team, row / p.group, lo, hi, i, lane, kept[kGate][i]);
#pragma unroll
                        for (int j = 0; j < 8; ++j) kept[kGate][i].v[j] = 0.0f;
                    }
                group_end += p.group;
            }
        }
        if (has_post) {
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const Eight w = load_any<kTeam>(p.post.weight, 0, p.vec, i, lane, p.cols);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    kept[kPost][i].v[j] = fmaf(dr[i].v[j], h[i].v[j], kept[kPost][i].v[j]);
                    if constexpr (kLayer) kept[kPostBias][i].v[j] += dr[i].v[j];
                    dr[i].v[j] *= w.v[j];
                    s[0] = fmaf(dr[i].v[j], h[i].v[j], s[0]);
                    if constexpr (kLayer) s[1] += dr[i].v[j];
                }
            }
            if (p.dh.data != nullptr) {
                sums(s);
                const float m2 = s[0] * p.inv_cols, m1 = s[1] * p.inv_cols;
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) dr[i].v[j] = rstd * (dr[i].v[j] - m1 - h[i].v[j] * m2);
            }
        }
        if (p.dh.data != nullptr)
#pragma unroll
            for (int i = 0; i < kVecs; ++i) store_any<kTeam>(p.dh, false, row, p.vec, i, lane, p.cols, dr[i]);
    }
    // the column sums
    const Rows parts = {p.parts, p.padded, 1, 1};
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
        const int kind = k == kPre ? kSumPre : k == kPost ? kSumPost : k == kGate ? kSumGate
                         : k == kPreBias ? kSumPreBias : kSumPostBias;
        if (!(p.kinds >> kind & 1)) continue;
        const long long at = (long long)blockIdx.x * kSums + kind;
        if constexpr (kTeams == 1) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                store_any<kTeam>(parts, true, at, p.vec, i, lane, p.cols, kept[k][i]);
        } else {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    joined[threadIdx.x / kTeam][column<kTeam>(p.vec, i, lane, j)] = kept[k][i].v[j];
            __syncthreads();
            for (int c = threadIdx.x; c < p.cols; c += kThreads) {
                float s = 0.0f;
#pragma unroll
                for (int t = 0; t < kTeams; ++t) s += joined[t][c];
                p.parts[at * p.padded + c] = s;
            }
        }
    }
}

// The same for rows too long for registers: the column sums lie in the block's
// parts, where each thread adds to its own columns.
template <bool kLayer, bool kStream32>
__global__ void __launch_bounds__(kLong) backward_long_kernel(const __grid_constant__ NormParams p) {
    __shared__ float shared[8][kLong / 32];
    TeamSums<kLong> sums = {shared, 0};
    const int lane = threadIdx.x, steps = (p.cols + 8 * kLong - 1) / (8 * kLong);
    const bool has_pre = p.dn.data != nullptr, has_post = p.post.weight.data != nullptr;
    const bool sums_gate = p.dgate.data != nullptr && (p.gate_mode == kGateShared || p.gate_mode == kGateGroups);
    const long long team = blockIdx.x;
    pdl_next();
    pdl_wait();
    const long long lo = first_row(p, team), hi = first_row(p, team + 1);
    const Rows parts = {p.parts, p.padded, 1, 1};
    auto add = [&](int kind, bool fresh, int i, const Eight& d) {
        const long long at = team * kSums + kind;
        Eight s = d;
        if (!fresh) {
            const Eight old = load_f32<kLong>(parts.data, at * parts.ld, p.vec, i, lane, p.cols);
#pragma unroll
            for (int j = 0; j < 8; ++j) s.v[j] += old.v[j];
        }
        store_any<kLong>(parts, true, at, p.vec, i, lane, p.cols, s);
    };
    for (long long row = lo; row < hi; ++row) {
        auto load_h = [&](int i) { return load_bf16<kLong>(p.h.data, row * p.h.ld, p.vec, i, lane, p.cols); };
        auto load_r = [&](int i) { return load_as<kLong, kStream32>(p.r, row, p.vec, i, lane, p.cols); };
        auto load_dn = [&](int i) { return load_bf16<kLong>(p.dn.data, row * p.dn.ld, p.vec, i, lane, p.cols); };
        float mean = 0.0f, rstd = 0.0f, m1 = 0.0f, m2 = 0.0f;
        if (has_pre) {
            long_statistics<kLayer>(p, sums, steps, lane, load_r, mean, rstd);
            float s[2] = {0.0f, 0.0f};
            for (int i = 0; i < steps; ++i) {
                const Eight r = load_r(i), dn = load_dn(i), w = load_any<kLong>(p.pre.weight, 0, p.vec, i, lane, p.cols);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = w.v[j] * dn.v[j];
                    s[0] = fmaf(d, (r.v[j] - mean) * rstd, s[0]);
                    if constexpr (kLayer) s[1] += d;
                }
            }
            sums(s);
            m2 = s[0] * p.inv_cols;
            m1 = s[1] * p.inv_cols;
        }
        auto load_dr = [&](int i) {
            Eight dr = {{0, 0, 0, 0, 0, 0, 0, 0}};
            if (p.dr.data != nullptr) dr = load_as<kLong, kStream32>(p.dr, row, p.vec, i, lane, p.cols);
            if (has_pre) {
                const Eight r = load_r(i), dn = load_dn(i), w = load_any<kLong>(p.pre.weight, 0, p.vec, i, lane, p.cols);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    dr.v[j] = fmaf(rstd, w.v[j] * dn.v[j] - m1 - (r.v[j] - mean) * rstd * m2, dr.v[j]);
            }
            return dr;
        };
        const long long g = gate_row(p, row);
        auto load_gate = [&](int i) { return load_any<kLong>(p.gate, g, p.vec, i, lane, p.cols); };
        float h_mean = 0.0f, h_rstd = 0.0f, h_m1 = 0.0f, h_m2 = 0.0f;
        if (has_post) {
            long_statistics<kLayer>(p, sums, steps, lane, load_h, h_mean, h_rstd);
            float s[2] = {0.0f, 0.0f};
            for (int i = 0; i < steps; ++i) {
                Eight d = load_dr(i);
                const Eight h = load_h(i), w = load_any<kLong>(p.post.weight, 0, p.vec, i, lane, p.cols);
                if (p.gate_mode != kGateNone) {
                    const Eight v = load_gate(i);
#pragma unroll
                    for (int j = 0; j < 8; ++j) d.v[j] *= gate_value(v.v[j], p.sigmoid);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    d.v[j] *= w.v[j];
                    s[0] = fmaf(d.v[j], (h.v[j] - h_mean) * h_rstd, s[0]);
                    if constexpr (kLayer) s[1] += d.v[j];
                }
            }
            sums(s);
            h_m2 = s[0] * p.inv_cols;
            h_m1 = s[1] * p.inv_cols;
        }
        const bool first = row == lo, group_first = first || (p.gate_mode == kGateGroups && row % p.group == 0);
        const bool group_last = p.gate_mode == kGateGroups && ((row + 1) % p.group == 0 || row + 1 == hi);
        // (dr and dn may be dx and dh: each column is read before it is written)
        for (int i = 0; i < steps; ++i) {
            Eight d = load_dr(i);
            if (has_pre) {
                const Eight r = load_r(i), dn = load_dn(i);
                Eight t;
#pragma unroll
                for (int j = 0; j < 8; ++j) t.v[j] = dn.v[j] * (r.v[j] - mean) * rstd;
                if (p.kinds >> kSumPre & 1) add(kSumPre, first, i, t);
                if (p.kinds >> kSumPreBias & 1) add(kSumPreBias, first, i, dn);
            }
            if (p.dx.data != nullptr) {
                Eight t;
#pragma unroll
                for (int j = 0; j < 8; ++j) t.v[j] = p.scale * d.v[j];
                store_any<kLong>(p.dx, kStream32, row, p.vec, i, lane, p.cols, t);
            }
            Eight h;
            if (p.h.data != nullptr) h = load_h(i);
            if (p.gate_mode != kGateNone) {
                const Eight v = load_gate(i);
                if (p.dgate.data != nullptr) {
                    Eight t = has_post ? normalised(p, p.post, h, h_mean, h_rstd, i, lane) : h;
#pragma unroll
                    for (int j = 0; j < 8; ++j) t.v[j] *= d.v[j];
                    if (sums_gate) {
                        add(kSumGate, group_first, i, t);
                        if (group_last)
                            flush_gate<kLong>(p, team, g, lo, hi, i, lane,
                                              load_f32<kLong>(parts.data, (team * kSums + kSumGate) * parts.ld,
                                                              p.vec, i, lane, p.cols));
                    } else {
                        store_gate<kLong>(p, row, i, lane, t, v);
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) d.v[j] *= gate_value(v.v[j], p.sigmoid);
            }
            if (has_post) {
                const Eight w = load_any<kLong>(p.post.weight, 0, p.vec, i, lane, p.cols);
                Eight t;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    h.v[j] = (h.v[j] - h_mean) * h_rstd;
                    t.v[j] = d.v[j] * h.v[j];
                }
                if (p.kinds >> kSumPost & 1) add(kSumPost, first, i, t);
                if (p.kinds >> kSumPostBias & 1) add(kSumPostBias, first, i, d);
#pragma unroll
                for (int j = 0; j < 8; ++j) d.v[j] = h_rstd * (d.v[j] * w.v[j] - h_m1 - h.v[j] * h_m2);
            }
            if (p.dh.data != nullptr) store_any<kLong>(p.dh, false, row, p.vec, i, lane, p.cols, d);
        }
        __syncthreads();
    }
}

// The parts of 32 columns, by 32 warps in turn: blocks y < kSums the column sums,
// the others gate rows whose rows several teams have.
constexpr int kJoinRows = 16;

__global__ void __launch_bounds__(1024) finish_kernel(const __grid_constant__ NormParams p) {
    __shared__ float shared[32][33];
    pdl_next();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + lane;
    const bool live = c < p.cols;
    // the sum over the warps, in warp 0
    auto total = [&](float s) {
        __syncthreads();
        shared[warp][lane] = s;
        __syncthreads();
        float t = 0.0f;
        if (warp == 0)
            for (int w = 0; w < 32; ++w) t += shared[w][lane];
        return t;
    };
    auto put = [&](const Rows& x, long long row, float s) {
        if (warp != 0 || !live) return;
        const long long at = row * x.ld + c;
        if (x.f32) {
            float* f = static_cast<float*>(x.data) + at;
            *f = p.accumulate ? *f + s : s;
        } else {
            __nv_bfloat16* b = static_cast<__nv_bfloat16*>(x.data) + at;
            *b = __float2bfloat16(p.accumulate ? __bfloat162float(*b) + s : s);
        }
    };
    auto slope = [&](long long g) {
        if (!live) return 0.0f;
        const long long at = g * p.gate.ld + c;
        return gate_slope(p.gate.f32 ? static_cast<const float*>(p.gate.data)[at]
                                     : __bfloat162float(static_cast<const __nv_bfloat16*>(p.gate.data)[at]),
                          p.sigmoid);
    };
    const int kind = blockIdx.y;
    if (kind < kSums) {
        if (!(p.kinds >> kind & 1)) return;
        float s = 0.0f;
        if (live)
#pragma unroll 4
            for (int b = warp; b < p.blocks; b += 32) s += p.parts[((long long)b * kSums + kind) * p.padded + c];
        s = total(s);
        if (kind == kSumGate) s *= slope(0);
        put(kind == kSumPre ? p.dpre.weight : kind == kSumPreBias ? p.dpre.bias
            : kind == kSumPost ? p.dpost.weight : kind == kSumPostBias ? p.dpost.bias : p.dgate, 0, s);
        return;
    }
    for (long long t = kind - kSums; t < p.teams; t += kJoinRows) {
        // the group of the team's last row, where it starts there and goes on
        const long long lo = first_row(p, t), hi = first_row(p, t + 1), g = (hi - 1) / p.group;
        if (lo == hi || g * p.group < lo || (g + 1) * p.group <= hi) continue;
        const long long last = ((g + 1) * p.group * p.teams - 1) / p.rows;  // the team of its last row
        float s = 0.0f;
        if (live)
#pragma unroll 4
            for (long long w = t + warp; w <= last; w += 32)
                if (first_row(p, w) < first_row(p, w + 1))
                    s += p.slots[(w * 2 + (w == t ? 1 : 0)) * p.padded + c];
        s = total(s);
        put(p.dgate, g, s * slope(g));
    }
}

// ------------------------------------------------------------------- launches --

// What a row of `cols` columns is given.
struct Shape {
    int team, vecs;  // team 0: the kernels for long rows
};
Shape forward_shape(int cols) {
    if (cols <= 256) return {32, 1};
    if (cols <= 512) return {32, 2};
    if (cols <= 1024) return {128, 1};
    if (cols <= 2048) return {128, 2};
    if (cols <= 4096) return {256, 2};
    if (cols <= 8192) return {512, 2};
    return {0, 0};
}
Shape backward_shape(int cols) {
    if (cols <= 256) return {32, 1};
    if (cols <= 512) return {32, 2};
    if (cols <= 1024) return {128, 1};
    if (cols <= 2048) return {256, 1};
    if (cols <= 4096) return {512, 1};
    if (cols <= 8192) return {512, 2};
    return {0, 0};
}

template <bool kLayer, bool kStream32>
cudaError_t launch_forward(const NormParams& p, cudaStream_t st) {
    const Shape s = forward_shape(p.cols);
    const int threads = s.team == 0 ? kLong : std::max(kForwardThreads, s.team), per = s.team == 0 ? 1 : threads / s.team;
    const long long want = (p.rows + per - 1) / per;
    const dim3 grid((unsigned)std::min(want, (long long)kSMs * (2048 / threads)));
    void (*kernel)(NormParams);
    switch (s.team * 4 + s.vecs) {
    case 32 * 4 + 1: kernel = forward_kernel<32, 1, kLayer, kStream32>; break;
    case 32 * 4 + 2: kernel = forward_kernel<32, 2, kLayer, kStream32>; break;
    case 128 * 4 + 1: kernel = forward_kernel<128, 1, kLayer, kStream32>; break;
    case 128 * 4 + 2: kernel = forward_kernel<128, 2, kLayer, kStream32>; break;
    case 256 * 4 + 2: kernel = forward_kernel<256, 2, kLayer, kStream32>; break;
    case 512 * 4 + 2: kernel = forward_kernel<512, 2, kLayer, kStream32>; break;
    default: kernel = forward_long_kernel<kLayer, kStream32>;
    }
    return launch_pdl(kernel, grid, dim3(threads), st, p);
}

// Blocks and teams of the gradient.
struct Split {
    Shape shape;
    int blocks, teams, threads;
    long long padded;
};
Split split_of(long long rows, long long cols) {
    Split s = {};
    s.shape = backward_shape((int)std::min(cols, 1ll << 20));
    const int team = s.shape.team == 0 ? kLong : s.shape.team;
    s.threads = team == 32 ? kBackwardThreads : team;
    const int per = s.threads / team;
    // four rows a team at least, so that the parts stay few beside the rows
    const long long want = (rows + 4 * per - 1) / (4 * per);
    s.blocks = (int)std::max(1ll, std::min(want, (long long)kSMs * std::max(1, 1024 / s.threads)));
    s.teams = s.blocks * per;
    s.padded = (cols + 7) / 8 * 8;
    return s;
}

template <bool kLayer, bool kStream32>
cudaError_t launch_backward(const NormParams& p, const Split& s, cudaStream_t st) {
    void (*kernel)(NormParams);
    switch (s.shape.team * 4 + s.shape.vecs) {
    case 32 * 4 + 1: kernel = backward_kernel<32, 1, kLayer, kStream32>; break;
    case 32 * 4 + 2: kernel = backward_kernel<32, 2, kLayer, kStream32>; break;
    case 128 * 4 + 1: kernel = backward_kernel<128, 1, kLayer, kStream32>; break;
    case 256 * 4 + 1: kernel = backward_kernel<256, 1, kLayer, kStream32>; break;
    case 512 * 4 + 1: kernel = backward_kernel<512, 1, kLayer, kStream32>; break;
    case 512 * 4 + 2: kernel = backward_kernel<512, 2, kLayer, kStream32>; break;
    default: kernel = backward_long_kernel<kLayer, kStream32>;
    }
    cudaError_t e = launch_pdl(kernel, dim3(s.blocks), dim3(s.threads), st, p);
    const bool groups = p.dgate.data != nullptr && p.gate_mode == kGateGroups;
    if (e != cudaSuccess || (p.kinds == 0 && !groups)) return e;
    const dim3 grid((unsigned)((p.cols + 31) / 32), kSums + (groups ? std::min(kJoinRows, s.teams) : 0));
    return launch_pdl(finish_kernel, grid, dim3(1024), st, p);
}

bool valid_affine(const vc_affine_t* a, bool needed) {
    if (a == nullptr || a->weight == nullptr) return !needed && (a == nullptr || a->bias == nullptr);
    const int es = elem_size(a->dtype);
    return es != 0 && reinterpret_cast<uintptr_t>(a->weight) % es == 0 &&
           reinterpret_cast<uintptr_t>(a->bias) % es == 0;
}
Rows vector_of(void* data, vc_dtype_t dtype) {
    return {data, 0, dtype == VC_FLOAT32, reinterpret_cast<uintptr_t>(data) % 16 == 0};
}
Affine affine_of(const vc_affine_t* a) {
    if (a == nullptr || (a->weight == nullptr && a->bias == nullptr)) return {};
    return {vector_of(a->weight, a->dtype), vector_of(a->bias, a->dtype)};
}
bool valid_args(const vc_block_norm_t* a) {
    return a != nullptr && (a->norm == VC_NORM_RMS || a->norm == VC_NORM_LAYER) &&
           (a->gate_act == VC_GATE_NONE || a->gate_act == VC_GATE_SIGMOID) && a->eps >= 0.0f;
}
// [G, D] with G a divisor of the rows (any where there are none).
bool valid_gate(const vc_matrix_t* g, long long rows, long long cols) {
    return valid_matrix(g) && g->batch == 1 && g->cols == cols && g->rows > 0 && rows % g->rows == 0;
}
bool is_bf16(const vc_matrix_t* m) { return m->dtype == VC_BFLOAT16; }
int mode_of(const vc_matrix_t* g, long long rows) {
    return g == nullptr ? kGateNone : g->rows == 1 ? kGateShared : g->rows == rows ? kGateFull : kGateGroups;
}
Span span_of_vector(const void* p, vc_dtype_t dtype, long long cols) {
    return span_of(p, (size_t)cols * elem_size(dtype));
}

void common_params(NormParams* p, const vc_matrix_t* gate, const vc_affine_t* post, const vc_affine_t* pre,
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
bool all_vec(std::initializer_list<const Rows*> xs) {
    bool vec = true;
    for (const Rows* x : xs) vec = vec && (x->data == nullptr || x->vec);
    return vec;
}

}  // namespace
}  // namespace step
}  // namespace vc

using namespace vc;
using namespace vc::step;

extern "C" {

vc_status_t vc_block_norm_forward(const vc_matrix_t* h, const vc_matrix_t* x, const vc_matrix_t* gate,
                                  const vc_affine_t* post, const vc_affine_t* pre, const vc_block_norm_t* args,
                                  const vc_matrix_t* r, const vc_matrix_t* n, vc_stream_t stream) {
    if (!valid_matrix(h) || h->batch != 1 || !is_bf16(h) || !valid_args(args)) return VC_ERR_INVALID_ARGUMENT;
    const long long T = h->rows, D = h->cols;
    if ((x != nullptr && !plain_matrix(x, T, D)) || (r != nullptr && !plain_matrix(r, T, D)) ||
        (n != nullptr && (!plain_matrix(n, T, D) || !is_bf16(n))) || (gate != nullptr && !valid_gate(gate, T, D)))
        return VC_ERR_INVALID_ARGUMENT;
    if (x != nullptr && r != nullptr && x->dtype != r->dtype) return VC_ERR_INVALID_ARGUMENT;
    if (!valid_affine(post, false) || !valid_affine(pre, n != nullptr)) return VC_ERR_INVALID_ARGUMENT;
    const Span outs[2] = {span_of(r), span_of(n)};
    if (overlap(outs[0], outs[1])) return VC_ERR_ALIAS;
    const vc_affine_t none = {};
    const vc_affine_t &a = post != nullptr ? *post : none, &b = pre != nullptr ? *pre : none;
    const Span ins[7] = {span_of(h), span_of(x), span_of(gate), span_of_vector(a.weight, a.dtype, D),
                         span_of_vector(a.bias, a.dtype, D), span_of_vector(b.weight, b.dtype, D),
                         span_of_vector(b.bias, b.dtype, D)};
    for (int o = 0; o < 2; ++o)
        for (int i = 0; i < 7; ++i)
            if (overlap(outs[o], ins[i]) && !(o == 0 && i == 1 && same_matrix(r, x)) &&
                !(o == 1 && i == 0 && same_matrix(n, h)))
                return VC_ERR_ALIAS;
    if (T == 0 || D == 0 || (r == nullptr && n == nullptr)) return VC_SUCCESS;
    if (test_launch_failure()) return VC_ERR_CUDA;
    NormParams p = {};
    common_params(&p, gate, post, pre, args, T, D);
    p.h = rows_of(h);
    p.x = rows_of(x);
    p.r = rows_of(r);
    p.n = rows_of(n);
    p.vec = all_vec({&p.h, &p.x, &p.gate, &p.r, &p.n, &p.post.weight, &p.post.bias, &p.pre.weight, &p.pre.bias});
    const bool f32 = (x != nullptr && x->dtype == VC_FLOAT32) || (r != nullptr && r->dtype == VC_FLOAT32);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool layer = args->norm == VC_NORM_LAYER;
    const cudaError_t e = layer ? (f32 ? launch_forward<true, true>(p, st) : launch_forward<true, false>(p, st))
                                : (f32 ? launch_forward<false, true>(p, st) : launch_forward<false, false>(p, st));
    return e == cudaSuccess ? VC_SUCCESS : VC_ERR_CUDA;
}

size_t vc_block_norm_backward_workspace(long long rows, long long cols, long long gates) {
    if (rows <= 0 || rows > train::kMaxExtent || cols <= 0 || cols > train::kMaxExtent || gates < 0 ||
        gates > rows)
        return 0;
    const Split s = split_of(rows, cols);
    const size_t parts = (size_t)s.blocks * kSums * s.padded * 4;
    const size_t slots = gates > 1 && gates < rows ? (size_t)s.teams * 2 * s.padded * 4 : 0;
    return round256(parts) + round256(slots);
}

vc_status_t vc_block_norm_backward(const vc_block_norm_in_t* in, const vc_affine_t* post, const vc_affine_t* pre,
                                   const vc_block_norm_t* args, const vc_block_norm_out_t* out, int accumulate,
                                   void* workspace, size_t workspace_bytes, vc_stream_t stream) {
    if (in == nullptr || out == nullptr || !valid_args(args)) return VC_ERR_INVALID_ARGUMENT;
    const vc_matrix_t* shape = in->dr != nullptr ? in->dr : in->dn;
    if (!valid_matrix(shape) || shape->batch != 1) return VC_ERR_INVALID_ARGUMENT;
    const long long T = shape->rows, D = shape->cols;
    const bool has_pre = in->dn != nullptr, has_post = post != nullptr && post->weight != nullptr;
    const bool layer = args->norm == VC_NORM_LAYER;
    auto bad = [&](const vc_matrix_t* m, bool bf16) {
        return m != nullptr && (!plain_matrix(m, T, D) || (bf16 && !is_bf16(m)));
    };
    if (bad(in->dr, false) || bad(in->dn, true) || bad(in->r, false) || bad(in->h, true) || bad(out->dx, false) ||
        bad(out->dh, true))
        return VC_ERR_INVALID_ARGUMENT;
    if (has_pre && in->r == nullptr) return VC_ERR_INVALID_ARGUMENT;
    // one type for the residual stream
    const vc_matrix_t* stream_like = in->dr != nullptr ? in->dr : in->r;
    if ((has_pre && in->r->dtype != stream_like->dtype) ||
        (out->dx != nullptr && out->dx->dtype != stream_like->dtype))
        return VC_ERR_INVALID_ARGUMENT;
    if (in->gate != nullptr && !valid_gate(in->gate, T, D)) return VC_ERR_INVALID_ARGUMENT;
    if (out->dgate != nullptr && (in->gate == nullptr || !plain_matrix(out->dgate, in->gate->rows, D)))
        return VC_ERR_INVALID_ARGUMENT;
    if (!valid_affine(post, false) || !valid_affine(pre, has_pre)) return VC_ERR_INVALID_ARGUMENT;
    auto bad_sum = [&](const vc_affine_t& s, bool there) {
        if (s.weight == nullptr && s.bias == nullptr) return false;
        const int es = elem_size(s.dtype);
        return !there || es == 0 || reinterpret_cast<uintptr_t>(s.weight) % es != 0 ||
               reinterpret_cast<uintptr_t>(s.bias) % es != 0 || (s.bias != nullptr && !layer);
    };
    if (bad_sum(out->dpre, has_pre) || bad_sum(out->dpost, has_post)) return VC_ERR_INVALID_ARGUMENT;
    if ((post != nullptr && post->bias != nullptr && !layer) || (pre != nullptr && pre->bias != nullptr && !layer))
        return VC_ERR_INVALID_ARGUMENT;
    const bool post_work = has_post && (out->dh != nullptr || out->dgate != nullptr || out->dpost.weight != nullptr ||
                                        out->dpost.bias != nullptr);
    const bool needs_h = post_work || out->dgate != nullptr;
    if (needs_h && in->h == nullptr) return VC_ERR_INVALID_ARGUMENT;
    const long long gates = in->gate != nullptr ? in->gate->rows : 0;
    const size_t need = T > 0 ? vc_block_norm_backward_workspace(T, D, gates) : 0;
    if (!workspace_ok(workspace, workspace_bytes, need)) return VC_ERR_INVALID_ARGUMENT;
    const vc_affine_t none = {};
    const vc_affine_t &a = post != nullptr ? *post : none, &b = pre != nullptr ? *pre : none;
    const Span outs[8] = {span_of(out->dx), span_of(out->dh), span_of(out->dgate),
                          span_of_vector(out->dpost.weight, out->dpost.dtype, D),
                          span_of_vector(out->dpost.bias, out->dpost.dtype, D),
                          span_of_vector(out->dpre.weight, out->dpre.dtype, D),
                          span_of_vector(out->dpre.bias, out->dpre.dtype, D), span_of(workspace, need)};
    const Span ins[9] = {span_of(in->dr), span_of(in->dn), has_pre ? span_of(in->r) : Span{},
                         needs_h ? span_of(in->h) : Span{}, span_of(in->gate),
                         span_of_vector(a.weight, a.dtype, D), span_of_vector(a.bias, a.dtype, D),
                         span_of_vector(b.weight, b.dtype, D), span_of_vector(b.bias, b.dtype, D)};
    for (int o = 0; o < 8; ++o) {
        for (int i = 0; i < 9; ++i)
            if (overlap(outs[o], ins[i]) && !(o == 0 && i == 0 && same_matrix(out->dx, in->dr)) &&
                !(o == 1 && i == 1 && same_matrix(out->dh, in->dn)))
                return VC_ERR_ALIAS;
        for (int q = 0; q < o; ++q)
            if (overlap(outs[o], outs[q])) return VC_ERR_ALIAS;
    }
    if (D == 0) return VC_SUCCESS;
    NormParams p = {};
    p.dx = rows_of(out->dx);
    p.dh = rows_of(out->dh);
    p.dgate = rows_of(out->dgate);
    p.dpost = affine_of(&out->dpost);
    p.dpre = affine_of(&out->dpre);
    p.kinds = (p.dpre.weight.data != nullptr) << kSumPre | (p.dpre.bias.data != nullptr) << kSumPreBias |
              (p.dpost.weight.data != nullptr) << kSumPost | (p.dpost.bias.data != nullptr) << kSumPostBias |
              (p.dgate.data != nullptr && mode_of(in->gate, T) == kGateShared) << kSumGate;
    p.accumulate = accumulate != 0;
    if (p.dx.data == nullptr && p.dh.data == nullptr && p.dgate.data == nullptr && p.kinds == 0) return VC_SUCCESS;
    // (without rows, gate rows have none either, and the sums are zeros)
    if (T == 0 && (p.kinds == 0 || accumulate)) return VC_SUCCESS;
    if (test_launch_failure()) return VC_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    common_params(&p, in->gate, post, pre, args, T, D);
    if (T == 0) {
        const cudaError_t e = launch_pdl(finish_kernel, dim3((unsigned)((D + 31) / 32), kSums), dim3(1024), st, p);
        return e == cudaSuccess ? VC_SUCCESS : VC_ERR_CUDA;
    }
    p.dr = rows_of(in->dr);
    p.dn = rows_of(in->dn);
    if (has_pre) p.r = rows_of(in->r);
    if (needs_h) p.h = rows_of(in->h);
    if (!post_work) p.post = {};
    p.vec = all_vec({&p.h, &p.r, &p.gate, &p.dr, &p.dn, &p.dx, &p.dh, &p.dgate, &p.post.weight, &p.post.bias,
                     &p.pre.weight});
    const Split s = split_of(T, D);
    p.blocks = s.blocks;
    p.teams = s.teams;
    p.padded = s.padded;
    p.parts = static_cast<float*>(workspace);
    p.slots = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) +
                                       round256((size_t)s.blocks * kSums * s.padded * 4));
    const bool f32 = stream_like->dtype == VC_FLOAT32;
    const cudaError_t e = layer ? (f32 ? launch_backward<true, true>(p, s, st) : launch_backward<true, false>(p, s, st))
                                : (f32 ? launch_backward<false, true>(p, s, st)
                                       : launch_backward<false, false>(p, s, st));
    return e == cudaSuccess ? VC_SUCCESS : VC_ERR_CUDA;
}

}  // extern "C"
