// vc_block_norm_forward: u = post(h), r = a x + act(gate) u, n = pre(r).
#include "vc_step_norm.cuh"

namespace vc {
namespace step {
namespace {

constexpr int kForwardThreads = 128;  // of a block of teams that are warps
// Threads of an SM; half of them where rows come through registers.
constexpr int kResident = 1024;

// One row after the other, the next one's inputs on their way meanwhile.  Bound by
// bytes: 32768 x 4096 with a gate for every element (1.34 GB) take 212 us, 6.35 TB/s; one
// row of 4096 takes 5.0 us, 2.7 in a graph.  Weights are read again for every row, from
// the first-level cache.
template <int kTeam, int kVecs, bool kLayer, bool kStream32, bool kVec, bool kSpan = false>
__global__ void __launch_bounds__(kTeam == 32 ? kForwardThreads : kTeam, (kVec ? kResident : kResident / 2) / (kTeam == 32 ? kForwardThreads : kTeam))
    forward_kernel(const __grid_constant__ NormParams p) {
    constexpr int kThreads = kTeam == 32 ? kForwardThreads : kTeam, kTeams = kThreads / kTeam;
    constexpr int kH = 0, kX = 1, kGate = 2;
    using Sums = TeamSums<kTeam, kSpan>;
    __shared__ float shared[2 * Sums::kAll][4];
    extern __shared__ uint4 ring[];
    __shared__ SpanShared signals;
    Sums sums = {shared, 0, p.span, &signals, 0};
    const int v0 = kSpan ? blockIdx.x % p.span * kVecs : 0;  // the block's first vector
    const int lane = kTeams == 1 ? threadIdx.x : threadIdx.x % 32;
    const int part = kTeams == 1 ? 0 : __shfl_sync(~0u, threadIdx.x / 32, 0);  // the team in the block
    const bool has_x = p.x.data != nullptr, full_gate = p.gate_mode == kGateFull;
    Stream<kThreads, kTeam, kVecs, 3, kVec, kVec> in;
    in.begin(ring, v0, lane, p.cols);
    in.array(kH, true, false);
    in.array(kX, has_x, kStream32);
    in.array(kGate, full_gate, p.gate.f32);
    auto load = [&](long long row) {
        in.load(kH, p.h, row, lane, p.cols);
        if (has_x) in.load(kX, p.x, row, lane, p.cols);
        if (full_gate) in.load(kGate, p.gate, row, lane, p.cols);
    };
    auto affine = [&](const Affine& a, const Eight& v, int i, float rstd) {
        const Eight w = mul(rstd, load_any<kTeam>(a.weight, 0, kVec, v0 + i, lane, p.cols));
        if (kLayer && a.bias.data != nullptr) return fma(v, w, load_any<kTeam>(a.bias, 0, kVec, v0 + i, lane, p.cols));
        return mul(v, w);
    };
    if constexpr (kSpan) sums.begin();
    pdl_next();
    pdl_wait();
    const int span = kSpan ? p.span : 1;
    const long long step = (long long)(gridDim.x / span) * kTeams;
    long long row = (long long)(blockIdx.x / span) * kTeams + part;
    if (row < p.rows) load(row);
    for (; row < p.rows; row += step) {
        if constexpr (kVec) {
            copies_end();
            copies_wait<0>();
            in.stage ^= 1;
            if (row + step < p.rows) load(row + step);
        }
        Eight u[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) u[i] = in.get(kH, i);
        if (p.post.weight.data != nullptr) {
            const float rstd = center<kVecs, kLayer>(p, u, kVec, v0, lane, sums);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) u[i] = affine(p.post, u[i], i, rstd);
        }
        if (p.gate_mode != kGateNone) {
            const long long g = gate_row(p, row);
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                u[i] = mul(u[i], gate_value(full_gate ? in.get(kGate, i)
                                                      : load_any<kTeam>(p.gate, g, kVec, v0 + i, lane, p.cols),
                                            p.sigmoid));
        }
        if (has_x)
#pragma unroll
            for (int i = 0; i < kVecs; ++i) u[i] = fma(p.scale, in.get(kX, i), u[i]);
        if constexpr (!kVec)
            if (row + step < p.rows) load(row + step);
        if (p.r.data != nullptr)
#pragma unroll
            for (int i = 0; i < kVecs; ++i) store_any<kTeam>(p.r, kStream32, row, kVec, v0 + i, lane, p.cols, u[i]);
        if (p.n.data == nullptr) continue;
        const float rstd = center<kVecs, kLayer>(p, u, kVec, v0, lane, sums);
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            store_any<kTeam>(p.n, false, row, kVec, v0 + i, lane, p.cols, affine(p.pre, u[i], i, rstd));
    }
    if constexpr (kSpan) sums.end(p.timeouts);
}

// Longer rows: a block a row, the inputs read four times, all but the first time from the
// second-level cache.
template <bool kLayer, bool kStream32>
__global__ void __launch_bounds__(kLong) forward_long_kernel(const __grid_constant__ NormParams p) {
    __shared__ float shared[2 * kLong / 32][4];
    TeamSums<kLong, false> sums = {shared, 0, 1, nullptr, 0};
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
                const Eight x = load_as<kLong>(p.x, kStream32, row, p.vec, i, lane, p.cols);
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

// The smallest shape that holds the row: with the next one 9120 x 256, RMS, take 6.6 us for 4.7,
// x 512 14.5 for 6.2, x 1024 23.2 for 13.4, x 2048 46.6 for 26.1, x 4096 91.2 for 51.3, and layer
// norms as much more.
Shape forward_shape(int cols) {
    if (cols <= 256) return {32, 1, 1};
    if (cols <= 512) return {32, 2, 1};
    if (cols <= 1024) return {128, 1, 1};
    if (cols <= 2048) return {128, 2, 1};
    if (cols <= 4096) return {256, 2, 1};
    if (cols <= 8192 * kMaxSpan) return {512, 2, (cols + 8191) / 8192};
    return {0, 0, 1};
}
template <bool kLayer, bool kStream32, bool kVec>
cudaError_t launch_forward(NormParams& p, cudaStream_t st) {
    const Shape s = forward_shape(p.cols);
    const int threads = s.team == 0 ? kLong : std::max(kForwardThreads, s.team);
    const int per = s.team == 0 ? 1 : threads / s.team;
    // 16-byte words a thread has of a vector of the inputs of one row
    const size_t words = 1 + (p.x.data == nullptr ? 0 : kStream32 ? 2 : 1) +
                         (p.gate_mode != kGateFull ? 0 : p.gate.f32 ? 2 : 1);
    const size_t bytes = kVec ? kStages * words * s.vecs * threads * 16 : 0;
    p.span = s.span;
    if (s.span > 1 && (p.timeouts = gemm::timeout_counter()) == nullptr) return cudaErrorInvalidValue;
    void (*kernel)(NormParams) = nullptr;
    switch (s.team * 4 + s.vecs) {
    case 32 * 4 + 1: kernel = forward_kernel<32, 1, kLayer, kStream32, kVec>; break;
    case 32 * 4 + 2: kernel = forward_kernel<32, 2, kLayer, kStream32, kVec>; break;
    case 128 * 4 + 1: kernel = forward_kernel<128, 1, kLayer, kStream32, kVec>; break;
    case 128 * 4 + 2: kernel = forward_kernel<128, 2, kLayer, kStream32, kVec>; break;
    case 256 * 4 + 2: kernel = forward_kernel<256, 2, kLayer, kStream32, kVec>; break;
    case 512 * 4 + 2:
        kernel = s.span > 1 ? forward_kernel<512, 2, kLayer, kStream32, kVec, true>
                            : forward_kernel<512, 2, kLayer, kStream32, kVec>;
        break;
    default: kernel = forward_long_kernel<kLayer, kStream32>;
    }
    // as many blocks as an SM holds at a time
    const int blocks = std::max(1, (int)std::min((size_t)((kVec || s.team == 0 ? kResident : kResident / 2) / threads),
                                                 (kSharedLimit + 1024) / (bytes + 2048 + (s.span > 1 ? 4096 : 0))));
    const long long want = (p.rows + per - 1) / per;
    const long long most = s.span > 1 ? clusters_of(s.span, blocks) : (long long)kSMs * blocks;
    return launch_pdl_shared(kernel, dim3((unsigned)(std::min(want, most) * s.span)), dim3(threads), bytes, s.span, st, p);
}
template <bool kLayer, bool kStream32>
cudaError_t launch_forward(NormParams& p, cudaStream_t st) {
    return p.vec ? launch_forward<kLayer, kStream32, true>(p, st) : launch_forward<kLayer, kStream32, false>(p, st);
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
    if (args->norm != VC_NORM_LAYER && (has_bias(post) || has_bias(pre))) return VC_ERR_INVALID_ARGUMENT;
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

}  // extern "C"
