// vc_block_norm_backward: from dr and dn to dx, dh, dgate and the column sums.
#include <type_traits>

#include "vc_step_norm.cuh"

namespace vc {
namespace step {
namespace {

// The rows of team t: a run of neighbours.
__device__ __forceinline__ long long first_row(const NormParams& p, long long t) {
    return t < p.teams ? t * p.rows / p.teams : p.rows;
}

// A team's sum of dr u over the rows of group g that it has: the whole of it goes to
// dgate, a part to one of the team's two slots: 0 where the group started before
// its rows, 1 where it goes on behind them.
template <class Access>
__device__ __forceinline__ void flush_gate(const NormParams& p, long long team, long long g, long long lo,
                                           long long hi, const Access& access, Eight sum) {
    const bool before = g * p.group < lo, behind = (g + 1) * p.group > hi;
    if (before || behind) return access.part({p.slots, p.padded, 1, 1}, team * 2 + (before ? 0 : 1), sum);
    const Eight gate = access.load(p.gate, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum.v[j] *= gate_slope(gate.v[j], p.sigmoid);
    if (p.accumulate) {
        const Eight old = access.load(p.dgate, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum.v[j] += old.v[j];
    }
    access.store(p.dgate, p.dgate.f32, g, sum);
}

// A gate of its own for every element.
template <class Access>
__device__ __forceinline__ void store_gate(const NormParams& p, long long row, const Access& access, Eight d,
                                           const Eight& gate) {
#pragma unroll
    for (int j = 0; j < 8; ++j) d.v[j] *= gate_slope(gate.v[j], p.sigmoid);
    if (p.accumulate) {
        const Eight old = access.load(p.dgate, row);
#pragma unroll
        for (int j = 0; j < 8; ++j) d.v[j] += old.v[j];
    }
    access.store(p.dgate, p.dgate.f32, row, d);
}

// How a thread reads and writes its columns of vector v: neighbours of rows of any
// alignment,
template <int kTeam>
struct Near {
    int v, lane, cols;
    __device__ __forceinline__ Eight load(const Rows& x, long long row) const {
        return load_near<kTeam>(x, row, v, lane, cols);
    }
    __device__ __forceinline__ void store(const Rows& x, bool f32, long long row, const Eight& r) const {
        store_near<kTeam>(x, f32, row, v, lane, cols, r);
    }
    __device__ __forceinline__ void part(const Rows& x, long long row, const Eight& r) const {
        store_any<kTeam>(x, true, row, true, v, lane, cols, r);
    }
};
// neighbours of rows on 16 bytes or else every kTeam-th one,
template <int kTeam, bool kVec>
struct Plain {
    int v, lane, cols;
    __device__ __forceinline__ Eight load(const Rows& x, long long row) const {
        return load_any<kTeam>(x, row, kVec, v, lane, cols);
    }
    __device__ __forceinline__ void store(const Rows& x, bool f32, long long row, const Eight& r) const {
        store_any<kTeam>(x, f32, row, kVec, v, lane, cols, r);
    }
    __device__ __forceinline__ void part(const Rows& x, long long row, const Eight& r) const {
        store_any<kTeam>(x, true, row, kVec, v, lane, cols, r);
    }
};
// and the same known at run time.
struct Long {
    bool vec;
    int v, lane, cols;
    __device__ __forceinline__ Eight load(const Rows& x, long long row) const {
        return load_any<kLong>(x, row, vec, v, lane, cols);
    }
    __device__ __forceinline__ void store(const Rows& x, bool f32, long long row, const Eight& r) const {
        store_any<kLong>(x, f32, row, vec, v, lane, cols, r);
    }
    __device__ __forceinline__ void part(const Rows& x, long long row, const Eight& r) const {
        store_any<kLong>(x, true, row, vec, v, lane, cols, r);
    }
};

constexpr int kBackwardThreads = 256;  // of a block of teams that are warps

// Blocks on an SM: 16 to 20 warps with 100 to 128 registers a thread, fewer where a layer
// norm's rows come through registers, or are 32 bits wide beside 96 registers (16384 x 2560,
// 16 gate rows: 282 us with two blocks of 320 threads, 230 with one; of 16 bits, one gate
// row: 180 and 197).
__host__ __device__ constexpr int resident_blocks(int team, bool layer, bool f32, bool vec) {
    const bool crowded = layer && (team == 320 ? f32 : !vec);
    return team == 32    ? 2
           : team == 64  ? (crowded ? 6 : 8)
           : team == 128 ? (crowded ? 3 : 4)
           : team == 192 ? 2
           : team == 256 ? 2
           : team == 320 ? (crowded ? 1 : 2)
                         : 1;
}

// Rows off 16 bytes: in registers, strided over the team, or by the larger teams shifted
// out of shared memory.  (The registers do not hold the next row beside the sums of a
// layer norm, and with spilled ones a row waits for the next one's loads: 9120 x 4095 took
// 213 us in registers, RMS, and 482, layer norm, 9120 x 4100 479 and 1487.  Shifted they
// take 176, 250, 354 and 545.  9120 x 1021 took 49 and 61 us in registers, 53 and 93
// shifted.)
__host__ __device__ constexpr bool shifted(int team, bool layer, bool vec) {
    return !vec && (team == 512 || (team == 256 && layer));
}

// One row after the other, the next one's inputs on their way meanwhile, the column sums
// in registers, which are what bounds how many warps an SM has: 16384 x 8192 (1.61 GB) take
// 276 us, 5.85 TB/s, with one block of 16 warps an SM.  A row's last sums and the next
// row's statistics are one exchange (two: 340 us).  h^ is computed again for dh: two
// vectors a thread have no registers to keep it.  kGates: a gate for every element or for
// groups of rows; two vectors a thread have a kernel without that, whose code leaves them
// no register spilled (with it 309 to 417 us, as the compiler chose which ones).
template <int kTeam, int kVecs, bool kLayer, bool kStream32, bool kVec, bool kSpan = false, bool kGates = true>
__global__ void __launch_bounds__(kTeam == 32 ? kBackwardThreads : kTeam, resident_blocks(kTeam, kLayer, kStream32, kVec))
    backward_kernel(const __grid_constant__ NormParams p) {
    constexpr int kThreads = kTeam == 32 ? kBackwardThreads : kTeam, kTeams = kThreads / kTeam;
    // RMS norms have no biases
    constexpr int kKept = kLayer ? 5 : 3;
    constexpr int kPre = 0, kPost = 1, kGate = 2, kPreBias = 3, kPostBias = 4;
    constexpr bool kShift = shifted(kTeam, kLayer, kVec), kRing = kVec || kShift;
    using Access = std::conditional_t<kShift, Near<kTeam>, Plain<kTeam, kVec>>;
    constexpr int kR = 0, kDn = 1, kH = 2, kDr = 3, kG = 4;
    using Sums = TeamSums<kTeam, kSpan>;
    __shared__ float shared[2 * Sums::kAll][4];
    __shared__ float joined[kTeams > 1 ? kTeams : 1][kTeams > 1 ? 8 * kTeam * kVecs : 1];
    extern __shared__ uint4 ring[];
    __shared__ SpanShared signals;
    Sums sums = {shared, 0, p.span, &signals, 0};
    const int v0 = kSpan ? blockIdx.x % p.span * kVecs : 0;  // the block's first vector
    const int lane = kTeams == 1 ? threadIdx.x : threadIdx.x % 32;
    const int part = kTeams == 1 ? 0 : __shfl_sync(~0u, threadIdx.x / 32, 0);  // the team in the block
    const long long block = kSpan ? blockIdx.x / p.span : blockIdx.x, team = block * kTeams + part;
    const bool has_pre = p.dn.data != nullptr, has_post = p.post.weight.data != nullptr;
    const bool has_h = p.h.data != nullptr, has_dr = p.dr.data != nullptr;
    const bool full_gate = kGates && p.gate_mode == kGateFull, stream_gate = full_gate && (!kShift || p.stream_gate);
    const bool sums_gate = p.dgate.data != nullptr && (p.gate_mode == kGateShared || p.gate_mode == kGateGroups);
    Eight kept[kKept][kVecs];
    // sum k += a b
    auto add_product = [&](int k, int i, const Eight& a, const Eight& b) { kept[k][i] = fma(a, b, kept[k][i]); };
    const Eight ones = {{1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f}};
#pragma unroll
    for (int k = 0; k < kKept; ++k)
#pragma unroll
        for (int i = 0; i < kVecs; ++i) kept[k][i] = zeros();

    Stream<kThreads, kTeam, kVecs, 5, kVec, kRing> in;
    in.begin(ring, v0, lane, p.cols);
    in.array(kR, has_pre, kStream32);
    in.array(kDn, has_pre, false);
    in.array(kH, has_h, false);
    in.array(kDr, has_dr, kStream32);
    in.array(kG, stream_gate, kVecs == 1 && p.gate.f32);  // (two vectors: not with one in 32 bits)
    using Vector = Held<kTeam, kVecs, Access>;
    float4* const held = reinterpret_cast<float4*>(ring + (kRing ? kStages * in.words * kThreads : 0)) + lane;
    const Vector pre = {held}, post = {held + Vector::kBytes / 16}, shift = {held + 2 * (Vector::kBytes / 16)},
                 held_gate = {held + ((kLayer ? 3 : 2) + part) * (Vector::kBytes / 16)};  // (a team's own)
    // what a row needs until its dr is there, and what it needs to the end
    auto load_early = [&](long long row) {
        if (has_pre) {
            in.load(kR, p.r, row, lane, p.cols);
            in.load(kDn, p.dn, row, lane, p.cols);
        }
        if (has_dr) in.load(kDr, p.dr, row, lane, p.cols);
        if (stream_gate) in.load(kG, p.gate, row, lane, p.cols);
    };
    auto load_late = [&](long long row) {
        if (has_h) in.load(kH, p.h, row, lane, p.cols);
    };
    auto load = [&](long long row) {
        load_early(row);
        load_late(row);
    };
    // A row's statistics, in two steps: the totals that a layer norm needs for its means,
    // and the products.
    struct Stats {
        float mean = 0.0f, h_mean = 0.0f, rstd = 0.0f, h_rstd = 0.0f, m1 = 0.0f, m2 = 0.0f;
    };
    auto centered_r = [&](const Stats& s, int i) {
        const Eight r = in.get(kR, i);
        return kLayer ? centered<kTeam>(r, s.mean, kRing, v0 + i, lane, p.cols) : r;
    };
    auto centered_h = [&](const Stats& s, const Eight& h, int i) {
        return kLayer && has_post ? centered<kTeam>(h, s.h_mean, kRing, v0 + i, lane, p.cols) : h;
    };
    auto add_totals = [&](float& r, float& h) {
        float2 a = make_float2(0.0f, 0.0f), b = a;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            if (has_pre) total(a, in.get(kR, i));
            if (has_post) total(b, in.get(kH, i));
        }
        r = sum_of(a), h = sum_of(b);
    };
    auto add_products = [&](const Stats& s, float& r, float& gr, float& h, float& g) {
        float2 a = make_float2(0.0f, 0.0f), b = a, c = a, d = a;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            if (has_pre) {
                const Eight r = centered_r(s, i);
                const Eight g = mul(pre.get(i), in.get(kDn, i));
                dot(a, r, r);
                dot(b, g, r);
                if constexpr (kLayer) total(c, g);
            }
            if (has_post) {
                const Eight h = centered_h(s, in.get(kH, i), i);
                dot(d, h, h);
            }
        }
        r = sum_of(a), gr = sum_of(b), h = sum_of(d), g = sum_of(c);
    };
    auto set_products = [&](Stats& s, float r, float gr, float h, float g) {
        s.rstd = rsqrtf(fmaf(r, p.inv_cols, p.eps));
        s.h_rstd = rsqrtf(fmaf(h, p.inv_cols, p.eps));
        s.m2 = gr * (p.inv_cols * s.rstd * s.rstd);
        s.m1 = g * p.inv_cols;
    };
    auto sum_products = [&](Stats& s) {
        float r, gr, h, g;
        add_products(s, r, gr, h, g);
        if constexpr (kLayer) {
            float v[4] = {r, gr, h, g};
            sums(v);
            set_products(s, v[0], v[1], v[2], v[3]);
        } else {
            float v[3] = {r, gr, h};
            sums(v);
            set_products(s, v[0], v[1], v[2], 0.0f);
        }
    };
    auto statistics = [&] {
        Stats s;
        if constexpr (kLayer) {
            float v[2];
            add_totals(v[0], v[1]);
            sums(v);
            s.mean = v[0] * p.inv_cols;
            s.h_mean = v[1] * p.inv_cols;
        }
        sum_products(s);
        return s;
    };
    if constexpr (kSpan) sums.begin();
    pdl_next();
    pdl_wait();
    const long long lo = first_row(p, team), hi = first_row(p, team + 1);
    long long group_end = p.gate_mode == kGateGroups ? (lo / p.group + 1) * p.group : 0;
    if (lo < hi) load(lo);
    if constexpr (kRing) {
        copies_end();
        in.turn();
        if (lo + 1 < hi) load(lo + 1);
        copies_end();
    }
    // (threads read what they have written themselves)
    pre.hold(p.pre.weight, v0, lane, p.cols);
    post.hold(p.post.weight, v0, lane, p.cols);
    if constexpr (kLayer) shift.hold(p.post.bias, v0, lane, p.cols);
    long long g = p.gate_mode == kGateGroups ? lo / p.group : 0;  // the rows' gate
    bool new_gate = p.gate_mode == kGateShared || p.gate_mode == kGateGroups;
    Stats now;  // the row's
    if constexpr (kRing) {
        copies_wait<1>();
        if (lo < hi) now = statistics();
    }
    for (long long row = lo; row < hi; ++row) {
        if (new_gate) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                held_gate.put(i, gate_value(Access{v0 + i, lane, p.cols}.load(p.gate, g), p.sigmoid));
            new_gate = false;
        }
        if constexpr (!kRing) now = statistics();
        Eight du[kVecs], kept_hat[kRing ? 1 : kVecs];
        float2 t1 = make_float2(0.0f, 0.0f), t2 = t1;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            Eight dr = has_dr ? in.get(kDr, i) : zeros();
            if (has_pre) {
                const Eight r = mul(now.rstd, centered_r(now, i)), dn = in.get(kDn, i);
                const Eight w = pre.get(i);
                add_product(kPre, i, dn, r);
                if constexpr (kLayer) add_product(kPreBias, i, dn, ones);
                dr = fma(-now.m2, r, dr);
                if constexpr (kLayer) dr = add(-now.m1 * now.rstd, dr);
                dr = fma(mul(now.rstd, w), dn, dr);
            }
            if (p.dx.data != nullptr)
                Access{v0 + i, lane, p.cols}.store(p.dx, kStream32, row, mul(p.scale, dr));
            Eight w, hat;
            if (has_h) hat = centered_h(now, in.get(kH, i), i);
            if (has_post) {
                w = post.get(i);
                hat = mul(now.h_rstd, hat);
            }
            if constexpr (!kRing) kept_hat[i] = hat;
            du[i] = dr;
            if (p.gate_mode != kGateNone) {
                Eight gate, value;
                if (full_gate) {
                    gate = stream_gate ? in.get(kG, i) : Access{v0 + i, lane, p.cols}.load(p.gate, row);
                    value = gate_value(gate, p.sigmoid);
                } else {
                    value = held_gate.get(i);
                }
                if (p.dgate.data != nullptr) {
                    Eight u = hat;
                    if (has_post) {
                        u = mul(u, w);
                        if (kLayer && p.post.bias.data != nullptr)
                            u = add(u, shift.get(i));
                    }
                    if (sums_gate)
                        add_product(kGate, i, u, dr);
                    else if constexpr (kGates)
                        store_gate(p, row, Access{v0 + i, lane, p.cols}, mul(u, dr), gate);
                }
                du[i] = mul(dr, value);
            }
            if (has_post) {
                add_product(kPost, i, du[i], hat);
                if constexpr (kLayer) add_product(kPostBias, i, du[i], ones);
                du[i] = mul(du[i], w);
                dot(t1, du[i], hat);
                if constexpr (kLayer) total(t2, du[i]);
            }
        }
        // (this row's inputs are used up)
        if constexpr (!kRing)
            if (row + 1 < hi) load(row + 1);
        if (kGates && p.gate_mode == kGateGroups && (row + 1 == group_end || row + 1 == hi)) {
            if (sums_gate)
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    flush_gate(p, team, g, lo, hi, Access{v0 + i, lane, p.cols}, kept[kGate][i]);
                    kept[kGate][i] = zeros();
                }
            group_end += p.group;
            ++g;
            new_gate = true;
        }
        // dh's sums, and the next row's: in one
        float s1 = sum_of(t1), s2 = sum_of(t2);
        Stats next;
        if constexpr (kRing) {
            in.turn();
            if (row + 2 < hi) load_early(row + 2);
            copies_end();
            copies_wait<1>();
            const bool more = row + 1 < hi;
            if constexpr (kLayer) {
                float v[4] = {s1, s2, 0.0f, 0.0f};
                if (more) add_totals(v[2], v[3]);
                sums(v);
                s1 = v[0], s2 = v[1];
                next.mean = v[2] * p.inv_cols;
                next.h_mean = v[3] * p.inv_cols;
            } else {
                float v[4] = {s1, 0.0f, 0.0f, 0.0f}, none;
                if (more) add_products(next, v[1], v[2], v[3], none);
                sums(v);
                s1 = v[0];
                set_products(next, v[1], v[2], v[3], 0.0f);
            }
        } else if (has_post && p.dh.data != nullptr) {
            if constexpr (kLayer) {
                float v[2] = {s1, s2};
                sums(v);
                s1 = v[0], s2 = v[1];
            } else {
                float v[1] = {s1};
                sums(v);
                s1 = v[0];
            }
        }
        if (p.dh.data != nullptr) {
            if (has_post) {
                const float h_m2 = s1 * (p.inv_cols * now.h_rstd), h_m1 = s2 * (p.inv_cols * now.h_rstd);
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    const Eight hat = kRing ? mul(now.h_rstd, centered_h(now, in.template get<true>(kH, i), i))
                                            : kept_hat[kRing ? 0 : i];
                    du[i] = fma(-h_m2, hat, mul(now.h_rstd, du[i]));
                    if constexpr (kLayer) du[i] = add(-h_m1, du[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < kVecs; ++i) Access{v0 + i, lane, p.cols}.store(p.dh, false, row, du[i]);
        }
        if constexpr (kRing) {
            if (row + 2 < hi) load_late(row + 2);
            copies_end();
            if constexpr (kLayer)
                if (row + 1 < hi) sum_products(next);
            now = next;
        }
    }
    if constexpr (kSpan) sums.end(p.timeouts);
    // the column sums
    const Rows parts = {p.parts, p.padded, 1, 1};
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
        const int kind = k == kPre ? kSumPre : k == kPost ? kSumPost : k == kGate ? kSumGate
                         : k == kPreBias ? kSumPreBias : kSumPostBias;
        if (!(p.kinds >> kind & 1)) continue;
        const long long at = block * kSums + kind;
        if constexpr (kTeams == 1) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                Access{v0 + i, lane, p.cols}.part(parts, at, kept[k][i]);
        } else {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    joined[part][column<kTeam>(kVec, i, lane, j)] = kept[k][i].v[j];
            }
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

// The longest rows, read again for every pass (from the second-level cache); the column
// sums lie in the block's parts, where each thread adds to its own columns.
template <bool kLayer, bool kStream32>
__global__ void __launch_bounds__(kLong) backward_long_kernel(const __grid_constant__ NormParams p) {
    __shared__ float shared[2 * kLong / 32][4];
    TeamSums<kLong, false> sums = {shared, 0, 1, nullptr, 0};
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
        auto load_r = [&](int i) { return load_as<kLong>(p.r, kStream32, row, p.vec, i, lane, p.cols); };
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
            if (p.dr.data != nullptr) dr = load_as<kLong>(p.dr, kStream32, row, p.vec, i, lane, p.cols);
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
                            flush_gate(p, team, g, lo, hi, Long{p.vec != 0, i, lane, p.cols},
                                       load_f32<kLong>(parts.data, (team * kSums + kSumGate) * parts.ld, p.vec, i,
                                                       lane, p.cols));
                    } else {
                        store_gate(p, row, Long{p.vec != 0, i, lane, p.cols}, t, v);
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

// A group of rows that several teams have, from the one that has its first row to the
// one that has its last.
struct Spanning {
    int first, last, group;
};
constexpr int kJoinTeams = 256;  // that are looked at together

// The spanning groups that start with the teams t0, t0 + step, ... of kJoinTeams; their
// number.
__device__ __forceinline__ int find_spanning(const NormParams& p, int t0, int step, Spanning* found) {
    int* const count = &found[kJoinTeams].first;
    if (threadIdx.x == 0) *count = 0;
    __syncthreads();
    const long long t = t0 + (long long)threadIdx.x * step;
    if (threadIdx.x < kJoinTeams && t < p.teams) {
        const long long lo = first_row(p, t), hi = first_row(p, t + 1), g = (hi - 1) / p.group;
        if (g * p.group >= lo && (g + 1) * p.group > hi) {
            // (which place a group gets changes nothing but the order of work)
            const long long last = ((g + 1) * p.group * p.teams - 1) / p.rows;
            found[atomicAdd(count, 1)] = {(int)t, (int)last, (int)g};
        }
    }
    __syncthreads();
    return *count;
}

// The parts of 32 columns, by 32 warps in turn: blocks y < kSums the column sums,
// the others gate rows whose rows several teams have.  11.6 us for three sums of 152
// parts of 8192 columns, from cold caches; latency.  Without rows the column sums are
// zeros, and the others write those to the gates' gradient.
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
    if (kind >= kSums && p.rows == 0) {
        // no gate has any row: sums of nothing
        for (long long g = (kind - kSums) * 32 + warp; live && g < p.gates; g += 32 * (gridDim.y - kSums)) {
            const long long at = g * p.dgate.ld + c;
            if (p.dgate.f32)
                static_cast<float*>(p.dgate.data)[at] = 0.0f;
            else
                static_cast<__nv_bfloat16*>(p.dgate.data)[at] = __float2bfloat16(0.0f);
        }
        return;
    }
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
    // few groups, of many teams each
    __shared__ Spanning found[kJoinTeams + 1];
    for (int t0 = kind - kSums; t0 < p.teams; t0 += kJoinRows * kJoinTeams) {
        const int n = find_spanning(p, t0, kJoinRows, found);
        for (int f = 0; f < n; ++f) {
            float s = 0.0f;
            if (live)
#pragma unroll 4
                for (int w = found[f].first + warp; w <= found[f].last; w += 32)
                    s += p.slots[((long long)w * 2 + (w == found[f].first ? 1 : 0)) * p.padded + c];
            s = total(s);
            put(p.dgate, found[f].group, s * slope(found[f].group));
        }
        __syncthreads();
    }
}

// Many groups, of about 16 teams each or fewer (18 at most): a thread a column.
__global__ void __launch_bounds__(kJoinTeams) gates_kernel(const __grid_constant__ NormParams p) {
    __shared__ Spanning found[kJoinTeams + 1];
    pdl_next();
    pdl_wait();
    const long long c = (long long)blockIdx.x * kJoinTeams + threadIdx.x;
    for (int t0 = blockIdx.y; t0 < p.teams; t0 += gridDim.y * kJoinTeams) {
        const int n = find_spanning(p, t0, gridDim.y, found);
        if (c < p.cols)
#pragma unroll 2
            for (int f = 0; f < n; ++f) {
                const Spanning s = found[f];
                float sum = p.slots[((long long)s.first * 2 + 1) * p.padded + c];
                for (int w = s.first + 1; w <= s.last; ++w) sum += p.slots[(long long)w * 2 * p.padded + c];
                const long long from = (long long)s.group * p.gate.ld + c, to = (long long)s.group * p.dgate.ld + c;
                sum *= gate_slope(p.gate.f32 ? static_cast<const float*>(p.gate.data)[from]
                                             : __bfloat162float(static_cast<const __nv_bfloat16*>(p.gate.data)[from]),
                                  p.sigmoid);
                if (p.dgate.f32) {
                    float* f32 = static_cast<float*>(p.dgate.data) + to;
                    *f32 = p.accumulate ? *f32 + sum : sum;
                } else {
                    __nv_bfloat16* b16 = static_cast<__nv_bfloat16*>(p.dgate.data) + to;
                    *b16 = __float2bfloat16(p.accumulate ? __bfloat162float(*b16) + sum : sum);
                }
            }
        __syncthreads();
    }
}

// vec: on 16 bytes (rows that are not leave 320 threads too few registers: 9120 x 2300
// 364 us, RMS).  in_two: rows of up to 8192 values by two vectors a thread.
Shape backward_shape(int cols, bool vec, bool in_two) {
    for (int team : {32, 64, 128, 192, 256})
        if (cols <= team * 8) return {team, 1, 1};
    if (cols <= 2560 && vec) return {320, 1, 1};
    if (cols <= 4096) return {512, 1, 1};
    if (cols <= 8192 && in_two) return {512, 2, 1};
    if (cols <= 4096 * kMaxSpan) return {512, 1, (cols + 4095) / 4096};
    return {0, 0, 1};
}

// Blocks and teams of the gradient.
struct Split {
    Shape shape;
    int blocks, teams, threads;
    long long padded;
};
Split split_of(long long rows, long long cols, bool in_two, bool layer, bool f32, bool vec) {
    Split s = {};
    s.shape = backward_shape((int)std::min(cols, 1ll << 20), vec, in_two);
    const int team = s.shape.team == 0 ? kLong : s.shape.team;
    s.threads = team == 32 ? kBackwardThreads : team;
    const int per = s.threads / team;
    // two rows a team at least, so that the parts stay few beside the rows
    const long long want = (rows + 2 * per - 1) / (2 * per);
    const long long most = s.shape.span > 1 ? clusters_of(s.shape.span, 1)
                                            : (long long)kSMs * resident_blocks(team, layer, f32, vec);
    s.blocks = (int)std::max(1ll, std::min(want, most));  // or clusters
    s.teams = (int)std::min(rows, (long long)s.blocks * per);  // (the others have no rows)
    s.padded = (cols + 7) / 8 * 8;
    return s;
}

template <bool kLayer, bool kStream32, bool kVec>
cudaError_t launch_backward(NormParams& p, const Split& s, cudaStream_t st) {
    const bool groups = p.dgate.data != nullptr && p.gate_mode == kGateGroups;
    const bool shift = shifted(s.shape.team, kLayer, kVec), ring = kVec || shift;
    // 16-byte words a thread has of a vector of a matrix
    auto words = [&](bool present, bool f32) -> size_t { return !present ? 0 : 1 + f32 + shift; };
    const size_t rows = words(p.dn.data != nullptr, kStream32) + words(p.dn.data != nullptr, false) +
                        words(p.h.data != nullptr, false) + words(p.dr.data != nullptr, kStream32);
    const size_t gate = words(p.gate_mode == kGateFull, p.gate.f32);
    // two rows' inputs; held weights and gates
    auto shared = [&](size_t words) {
        return (ring ? kStages * words * s.shape.vecs * s.threads * 16 : 0) +
               (size_t)((kLayer ? 3 : 2) * s.shape.team +
                        (p.gate_mode == kGateShared || p.gate_mode == kGateGroups ? s.threads : 0)) *
                   s.shape.vecs * 32;
    };
    // (shifted rows in 32 bits leave no place for a gate of as many values)
    p.stream_gate = shared(rows + gate) + 2048 <= kSharedLimit;
    size_t bytes = shared(rows + (p.stream_gate ? gate : 0));
    p.span = s.shape.span;
    if (p.span > 1 && (p.timeouts = gemm::timeout_counter()) == nullptr) return cudaErrorInvalidValue;
    void (*kernel)(NormParams) = nullptr;
    switch (s.shape.team * 4 + s.shape.vecs) {
    case 32 * 4 + 1: kernel = backward_kernel<32, 1, kLayer, kStream32, kVec>; break;
    case 64 * 4 + 1: kernel = backward_kernel<64, 1, kLayer, kStream32, kVec>; break;
    case 128 * 4 + 1: kernel = backward_kernel<128, 1, kLayer, kStream32, kVec>; break;
    case 192 * 4 + 1: kernel = backward_kernel<192, 1, kLayer, kStream32, kVec>; break;
    case 320 * 4 + 1: kernel = backward_kernel<320, 1, kLayer, kStream32, true>; break;
    case 256 * 4 + 1: kernel = backward_kernel<256, 1, kLayer, kStream32, kVec>; break;
    case 512 * 4 + 1:
        kernel = s.shape.span > 1 ? backward_kernel<512, 1, kLayer, kStream32, kVec, true>
                                  : backward_kernel<512, 1, kLayer, kStream32, kVec>;
        break;
    case 512 * 4 + 2:
        kernel = p.gate_mode == kGateNone || p.gate_mode == kGateShared
                     ? backward_kernel<512, 2, false, false, true, false, false>
                     : backward_kernel<512, 2, false, false, true>;
        break;
    default: kernel = backward_long_kernel<kLayer, kStream32>; bytes = 0;
    }
    cudaError_t e = launch_pdl_shared(kernel, dim3(s.blocks * s.shape.span), dim3(s.threads), bytes, s.shape.span, st, p);
    if (e != cudaSuccess || (p.kinds == 0 && !groups)) return e;
    const unsigned across = (unsigned)((p.cols + 31) / 32);
    // By a warp a team of a group or by a thread a column (the whole gradient of 9120 x 1024: 24
    // gates of 25 teams 36.7 and 38.3 us, 2 of 304 35.5 and 53.2, 38 of 16 73.3 and 55.1; of 9120 x
    // 4096: 8 of 19 115.8 and 107.5, 10 of 15 116.7 and 107.8).
    const long long per_group = s.teams / (p.rows / p.group);  // teams
    const bool few = groups && per_group > 16;
    if (p.kinds != 0 || few) {
        e = launch_pdl(finish_kernel, dim3(across, kSums + (few ? std::min(kJoinRows, s.teams) : 0)), dim3(1024), st, p);
        if (e != cudaSuccess) return e;
    }
    if (groups && !few)
        e = launch_pdl(gates_kernel, dim3((p.cols + kJoinTeams - 1) / kJoinTeams, std::min(64, s.teams)),
                       dim3(kJoinTeams), st, p);
    return e;
}
template <bool kLayer, bool kStream32>
cudaError_t launch_backward(NormParams& p, const Split& s, cudaStream_t st) {
    return p.vec ? launch_backward<kLayer, kStream32, true>(p, s, st)
                 : launch_backward<kLayer, kStream32, false>(p, s, st);
}

}  // namespace
}  // namespace step
}  // namespace vc

using namespace vc;
using namespace vc::step;

extern "C" {

size_t vc_block_norm_backward_workspace(long long rows, long long cols, long long gates) {
    if (rows <= 0 || rows > train::kMaxExtent || cols <= 0 || cols > train::kMaxExtent || gates < 0 ||
        gates > rows)
        return 0;
    // (of the ways that rows of such a length may take, the one that needs most)
    const Split a = split_of(rows, cols, false, false, false, true), s = split_of(rows, cols, true, false, false, true);
    const size_t parts = (size_t)std::max(a.blocks, s.blocks) * kSums * s.padded * 4;
    const size_t slots = gates > 1 && gates < rows ? (size_t)std::max(a.teams, s.teams) * 2 * s.padded * 4 : 0;
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
    if (!layer && (has_bias(post) || has_bias(pre))) return VC_ERR_INVALID_ARGUMENT;
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
    // (without rows all sums are zeros)
    if (T == 0 && accumulate) return VC_SUCCESS;
    if (T == 0) p.kinds &= ~(1 << kSumGate);  // (all gates are written alike)
    if (T == 0 && p.kinds == 0 && p.dgate.data == nullptr) return VC_SUCCESS;
    if (test_launch_failure()) return VC_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    common_params(&p, in->gate, post, pre, args, T, D);
    if (T == 0) {
        p.gates = p.dgate.data != nullptr ? gates : 0;
        const unsigned more = (unsigned)std::min((long long)kJoinRows, (p.gates + 31) / 32);
        const cudaError_t e = launch_pdl(finish_kernel, dim3((unsigned)((D + 31) / 32), kSums + more), dim3(1024), st, p);
        return e == cudaSuccess ? VC_SUCCESS : VC_ERR_CUDA;
    }
    p.dr = rows_of(in->dr);
    p.dn = rows_of(in->dn);
    if (has_pre) p.r = rows_of(in->r);
    if (needs_h) p.h = rows_of(in->h);
    if (!post_work) p.post = {};
    p.vec = all_vec({&p.h, &p.r, &p.gate, &p.dr, &p.dn, &p.dx, &p.dh, &p.dgate, &p.post.weight, &p.post.bias,
                     &p.pre.weight});
    // (RMS norms of 16-bit streams on 16 bytes have the registers; not with a gate in 32
    // bits for every element, whose rows would not find their place in shared memory)
    const bool in_two = p.vec && !layer && stream_like->dtype == VC_BFLOAT16 &&
                        !(p.gate_mode == kGateFull && p.gate.f32);
    const Split s = split_of(T, D, in_two, layer, stream_like->dtype == VC_FLOAT32, p.vec);
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
