// The linear layer with bias, activation and residual in its epilogue, and
// its gradient.
#include <algorithm>
#include <type_traits>

#include "vc_train_common.cuh"

namespace vc {
namespace train {
namespace {

using gemm::Operand;
using gemm::Product;
using gemm::Shape;
using gemm::View;

// ------------------------------------------------------------- epilogues --

using gemm::Place;

// y = act(acc + bias) + residual; z = acc + bias kept on request.  kSwap: the
// product is the transposed one, W x^T, so that a chunk's rows are y's columns.
template <int kFamily, bool kSwap, bool kResidual>
struct EpiForward {
    static constexpr bool kSym = false;
    struct Params {
        const __nv_bfloat16* bias;
        View residual, y, preact;
        int has_preact, bias_vec;
        Act act;
    };
    static bool odd(const Params& p) {
        return !p.y.vec16 || (p.has_preact && !p.preact.vec16) || (kResidual && !p.residual.vec16);
    }
    struct WithResidual {
        gemm::Chunk16 residual;  // across the rows, or, off 16 bytes, one row per lane
    };
    struct Without {};
    struct Pre : std::conditional_t<kResidual && !kSwap, WithResidual, Without> {
        gemm::Chunk16 bias;  // of the chunk's columns, the same in every lane
        float one_bias;      // else: of the lane's column (kSwap: row)
    };
    __device__ static bool bias_in_pieces(const Params& p, const Place& q) {
        return !kSwap && p.bias_vec && q.whole();
    }
    __device__ static void prefetch(const Params& p, const Place& q, Pre& pre) {
        if (p.bias != nullptr) {
            if (bias_in_pieces(p, q)) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    pre.bias.u[i] = *reinterpret_cast<const uint4*>(p.bias + q.col0 + 8 * i);
            } else {
                const int at = kSwap ? q.row() : q.col0 + q.lane;
                pre.one_bias = at < (kSwap ? q.M : q.N) ? __bfloat162float(p.bias[at]) : 0.0f;
            }
        }
        if constexpr (kResidual && !kSwap) {
            if (in_pieces(p.residual, q))
                load_across(static_cast<const __nv_bfloat16*>(p.residual.data) +
                                corner_of(p.residual, q),
                            p.residual.ld * 2, q, pre.residual);
            else
                load_values(static_cast<const unsigned short*>(p.residual.data) +
                                corner_of(p.residual, q),
                            p.residual.ld, q, q.N - q.col0, pre.residual);
        }
    }
    __device__ static void apply(const Params& p, const Place& q, Pre& pre, float (&v)[32]) {
        if (p.bias != nullptr) {
            if (bias_in_pieces(p, q)) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 f = pair_at(pre.bias, i, __nv_bfloat16());
                    v[2 * i] += f.x;
                    v[2 * i + 1] += f.y;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] += kSwap ? pre.one_bias : __shfl_sync(0xFFFFFFFFu, pre.one_bias, j);
            }
        }
        if (p.has_preact) kSwap ? put_columns(p.preact, q, v) : put_rows(p.preact, q, v);
        if (!p.act.identity) {
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
                const float2 y = act_value<kFamily>(make_float2(v[j], v[j + 1]), p.act);
                v[j] = y.x;
                v[j + 1] = y.y;
            }
        }
        if constexpr (kResidual && !kSwap) {
            if (in_pieces(p.residual, q)) across_to_own(q, pre.residual);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 f = pair_at(pre.residual, i, __nv_bfloat16());
                v[2 * i] += f.x;
                v[2 * i + 1] += f.y;
            }
        } else if constexpr (kResidual) {
            float r[32];
            get_columns(p.residual, q, r);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += r[j];
        }
        kSwap ? put_columns(p.y, q, v) : put_rows(p.y, q, v);
    }
};

// out = acc, or out += acc.
template <bool kSwap>
struct EpiStore {
    static constexpr bool kSym = false;
    struct Params {
        View out;
        int add;
    };
    static bool odd(const Params& p) { return !p.out.vec16; }
    struct Pre {};
    __device__ static void prefetch(const Params&, const Place&, Pre&) {}
    __device__ static void apply(const Params& p, const Place& q, Pre&, float (&v)[32]) {
        if (p.add) {
            float old[32];
            kSwap ? get_columns(p.out, q, old) : get_rows(p.out, q, old);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += old[j];
        }
        finish(p, q, v);
    }
    static bool sums32(const Params& p) { return p.out.f32; }
    __device__ static void start(const Params& p, const Place& q, float (&v)[32]) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.0f;
        if (p.add && gemm::inside<EpiStore>(q)) get_rows(p.out, q, v);
    }
    __device__ static void finish(const Params& p, const Place& q, const float (&v)[32]) {
        kSwap ? put_columns(p.out, q, v) : put_rows(p.out, q, v);
    }
};

// Up to this many rows of x the product is computed transposed: 128 rows of
// the weight per tile and the rows of x across it, for a product that is
// bound by reading the weight.
constexpr int kSwapRows = 64;

// The operands and options of a call.
struct Forward {
    Operand x, w;
    int M, N, K;
    const void* bias;
    const vc_matrix_t *residual, *y, *preact;
    vc_act_t act;
};

template <int kFamily, bool kSwap, bool kResidual>
cudaError_t forward(const Forward& f, cudaStream_t st) {
    using Epi = EpiForward<kFamily, kSwap, kResidual>;
    typename Epi::Params ep = {};
    ep.bias = static_cast<const __nv_bfloat16*>(f.bias);
    ep.bias_vec = (reinterpret_cast<uintptr_t>(f.bias) & 15) == 0;
    ep.residual = view_of(f.residual);
    ep.y = view_of(f.y);
    ep.preact = view_of(f.preact);
    ep.has_preact = f.preact != nullptr;
    ep.act = act_params(f.act);
    if constexpr (kSwap)
        return gemm::launch_skinny<Epi>(Product{f.w, f.x, f.N, f.M, f.K, 1, 1}, ep, st);
    else
        return gemm::launch<Epi>(Product{f.x, f.w, f.M, f.N, f.K, 1, 1}, ep, st);
}

template <int kFamily>
cudaError_t forward(const Forward& f, cudaStream_t st) {
    if (f.M <= kSwapRows)
        return f.residual != nullptr ? forward<kFamily, true, true>(f, st)
                                     : forward<kFamily, true, false>(f, st);
    return f.residual != nullptr ? forward<kFamily, false, true>(f, st)
                                 : forward<kFamily, false, false>(f, st);
}

// ------------------------------------------------------------ copy, dz, db --

// bf16 matrices copied to rows of ld_out values (a multiple of 16), so that TMA
// can read them; one or two in a launch.  A thread makes 16 bytes of a row.
struct PackJob {
    const unsigned short* src;
    uint4* dst;
    long long ld;
    int rows, cols, pieces;  // pieces: of 8 values per row
};
// db (+)= the sum of partial sums, in a fixed order.
struct SumJob {
    const float* sums;  // [parts][cols], or NULL
    void* db;
    int parts, cols, f32, add;
};
__device__ __forceinline__ void store_db(const SumJob& j, int col, float v) {
    if (j.f32) {
        float* d = static_cast<float*>(j.db) + col;
        *d = j.add ? *d + v : v;
    } else {
        __nv_bfloat16* d = static_cast<__nv_bfloat16*>(j.db) + col;
        *d = __float2bfloat16(j.add ? __bfloat162float(*d) + v : v);
    }
}

// What has to be done before the products, in one launch: the blocks of row y
// of the grid take job y, those of the last row the column sums (a block 32
// columns at a time, its warps every eighth part).
struct Jobs {
    PackJob pack[2];
    int packs;
    SumJob sum;
};
__global__ void __launch_bounds__(256) jobs_kernel(const __grid_constant__ Jobs jobs) {
    __shared__ float part[8][32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if ((int)blockIdx.y < jobs.packs) {
        const PackJob j = jobs.pack[blockIdx.y];
        const long long total = (long long)j.rows * j.pieces;
        for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total;
             i += (long long)gridDim.x * 256) {
            const int row = (int)(i / j.pieces), col = (int)(i - (long long)row * j.pieces) * 8;
            const unsigned short* s = j.src + row * j.ld + col;
            unsigned v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = col + k < j.cols ? s[k] : 0u;
            j.dst[i] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16,
                                  v[6] | v[7] << 16);
        }
        return;
    }
    const SumJob& j = jobs.sum;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (long long first = (long long)blockIdx.x * 32; first < j.cols;
         first += (long long)gridDim.x * 32) {
        const long long col = first + lane;
        float v = 0.0f;
        if (col < j.cols) {
#pragma unroll 8
            for (int i = warp; i < j.parts; i += 8) v += j.sums[(long long)i * j.cols + col];
        }
        __syncthreads();
        part[warp][lane] = v;
        __syncthreads();
        if (warp != 0 || col >= j.cols) continue;
#pragma unroll
        for (int w = 1; w < 8; ++w) v += part[w][lane];
        store_db(j, (int)col, v);
    }
}

struct DzParams {
    View dy, preact;
    __nv_bfloat16* dz;       // NULL: not written
    __nv_bfloat16* dz_rest;  // NULL, or receives what rounding dz left
    long long ld_dz;
    float* sums;  // [gridDim.y][N], or NULL
    SumJob direct;  // with one row of blocks: where the sums go at once
    long long rows, cols;
    int vec16;
    Act act;
};

constexpr int kDzRows = 4;  // rows that a thread loads before it uses them

// dz = dy * act'(z) and the column sums of each block's rows.  A warp covers
// 256 columns (8 per lane); the block's eight warps take groups of rows in
// turn.
// kNoActivation: dz is dy, and with half the registers (of which it spills some,
// 96 bytes of stack) six blocks fit an SM instead of three: 16 us for the column
// sums of 16384 x 1024.
template <int kFamily>
__global__ void __launch_bounds__(256, kFamily == kNoActivation ? 6 : 3) dz_kernel(const __grid_constant__ DzParams p) {
    __shared__ float4 part[8][64];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long col = (long long)blockIdx.x * 256 + lane * 8;
    const int n = (int)min(8ll, p.cols - col);
    const bool vec = p.vec16 && n == 8;
    float sum[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
    const __nv_bfloat16* const dy = static_cast<const __nv_bfloat16*>(p.dy.data) + col;
    const __nv_bfloat16* const z = static_cast<const __nv_bfloat16*>(p.preact.data) + col;
    auto load8 = [&](const __nv_bfloat16* at) {
        if (vec) return *reinterpret_cast<const uint4*>(at);
        const unsigned short* s = reinterpret_cast<const unsigned short*>(at);
        unsigned v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? s[j] : 0u;
        return make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    };
    auto low = [](unsigned w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); };
    const long long step = (long long)gridDim.y * 8 * kDzRows;
    for (long long row0 = ((long long)blockIdx.y * 8 + warp) * kDzRows; n > 0 && row0 < p.rows;
         row0 += step) {
        uint4 a[kDzRows], b[kDzRows];
#pragma unroll
        for (int u = 0; u < kDzRows; ++u) {
            if (row0 + u >= p.rows) continue;
            a[u] = load8(dy + (row0 + u) * p.dy.ld);
            if constexpr (kFamily != kNoActivation) b[u] = load8(z + (row0 + u) * p.preact.ld);
        }
#pragma unroll
        for (int u = 0; u < kDzRows; ++u) {
            if (row0 + u >= p.rows) continue;
            const unsigned aw[4] = {a[u].x, a[u].y, a[u].z, a[u].w};
            unsigned hi[4], rest[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 v = low(aw[j]);
                if constexpr (kFamily != kNoActivation) {
                    const float2 k = act_slope<kFamily>(low(j == 0 ? b[u].x : j == 1 ? b[u].y : j == 2 ? b[u].z : b[u].w), p.act);
                    v = make_float2(2 * j < n ? v.x * k.x : 0.0f, 2 * j + 1 < n ? v.y * k.y : 0.0f);
                }
                sum[2 * j] += v.x;
                sum[2 * j + 1] += v.y;
                hi[j] = gemm::packed(v.x, v.y, __nv_bfloat16());
                const float2 h = low(hi[j]);
                // (nothing is left of an infinity, nor of what rounds to one)
                rest[j] = gemm::packed(isinf(h.x) ? 0.0f : v.x - h.x, isinf(h.y) ? 0.0f : v.y - h.y,
                                       __nv_bfloat16());
            }
            // (the buffers' rows are whole groups of 16 values)
            if (p.dz != nullptr)
                *reinterpret_cast<uint4*>(p.dz + (row0 + u) * p.ld_dz + col) =
                    make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if (p.dz_rest != nullptr)
                *reinterpret_cast<uint4*>(p.dz_rest + (row0 + u) * p.ld_dz + col) =
                    make_uint4(rest[0], rest[1], rest[2], rest[3]);
        }
    }
    if (p.sums == nullptr && p.direct.db == nullptr) return;
    part[warp][lane * 2] = make_float4(sum[0], sum[1], sum[2], sum[3]);
    part[warp][lane * 2 + 1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
    __syncthreads();
    const long long mine = (long long)blockIdx.x * 256 + threadIdx.x;
    if (mine < p.cols) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += reinterpret_cast<const float*>(part[w])[threadIdx.x];
        if (p.direct.db != nullptr)
            store_db(p.direct, (int)mine, t);
        else
            p.sums[(long long)blockIdx.y * p.cols + mine] = t;
    }
}

// Blocks along the rows: enough for the three blocks per SM that fit (six
// without an activation), each with a group of rows at least for every warp.
int dz_row_blocks(long long rows, long long cols, vc_act_t act) {
    const long long across = std::max(1ll, (cols + 255) / 256);
    const long long want = (152 * (act == VC_ACT_NONE ? 6 : 3) + across - 1) / across;
    return (int)std::max(1ll, std::min(want, (rows + 8 * kDzRows - 1) / (8 * kDzRows)));
}

// Batches of up to this many rows keep what rounding dz to bf16 leaves as a
// second plane of the operand: their products are bound by the weight's bytes,
// so that it costs nothing, and with few rows single roundings show.  Larger
// ones do without: a second plane would double the operations of products that
// are bound by them, for 32-bit gradients that are 1.7e-3 of their norm off
// then (16384 x 1024 x 4096, gelu: 198 us; without an activation 1e-6, 190 us).
constexpr int kRestRows = 64;

// K blocks (of 64) summed in tensor memory at a time for 32-bit gradients.  (The
// kernel that does so has 96 registers a thread for 64 sums and spills: 3.3 KB
// of stores in its code with two products, 1.5 KB with one.  16384 x 1024 x 4096
// without column sums: 93 us for dW, 78 where it is bf16.)
constexpr int kSegment = 16;

// ----------------------------------------------------------- the operands --

bool operand_ready(const vc_matrix_t* m) {
    return gemm::tma_ready(m->data, m->rows > 1 ? m->ld : 0, 1, 0);
}

size_t packed_bytes(const vc_matrix_t* m) {
    return operand_ready(m) ? 0 : round256((size_t)m->rows * padded_ld(m->cols) * 2);
}

// Where TMA reads the matrix: in place, or packed at *ws (advanced), for which
// a job is added.
void ready_operand(const vc_matrix_t* m, unsigned char** ws, Jobs* jobs, Operand* o) {
    if (operand_ready(m) || m->rows == 0 || m->cols == 0) {
        o->data = m->data;
        o->ld = m->rows > 1 ? m->ld : padded_ld(m->cols);
        return;
    }
    o->data = *ws;
    o->ld = padded_ld(m->cols);
    jobs->pack[jobs->packs++] = {static_cast<const unsigned short*>(m->data),
                                 reinterpret_cast<uint4*>(*ws),
                                 m->rows > 1 ? m->ld : 0,
                                 (int)m->rows,
                                 (int)m->cols,
                                 (int)(o->ld / 8)};
    *ws += packed_bytes(m);
}

cudaError_t launch_jobs(const Jobs& jobs, cudaStream_t st) {
    const int rows = jobs.packs + (jobs.sum.sums != nullptr ? 1 : 0);
    if (rows == 0) return cudaSuccess;
    long long most = jobs.sum.sums != nullptr ? (jobs.sum.cols + 31) / 32 : 1;
    for (int i = 0; i < jobs.packs; ++i)
        most = std::max(most, ((long long)jobs.pack[i].rows * jobs.pack[i].pieces + 255) / 256);
    const int blocks = (int)std::min(152 * 16ll, most);
    return launch_pdl(jobs_kernel, dim3(blocks, rows), dim3(256), st, jobs);
}

bool is_bf16(const vc_matrix_t* m) { return m->dtype == VC_BFLOAT16; }

bool plain_matrix(const vc_matrix_t* m, long long rows, long long cols) {
    return valid_matrix(m) && m->batch == 1 && m->rows == rows && m->cols == cols;
}

bool valid_act(vc_act_t act) { return act >= VC_ACT_NONE && act <= VC_ACT_SILU; }

bool workspace_ok(const void* ws, size_t have, size_t need) {
    return need == 0 || (ws != nullptr && (reinterpret_cast<uintptr_t>(ws) & 15) == 0 && have >= need);
}

int dz_planes(long long rows, vc_act_t act) {
    return act != VC_ACT_NONE && rows <= kRestRows ? 2 : 1;
}

size_t backward_workspace(const vc_matrix_t* dy, const vc_matrix_t* x, const vc_matrix_t* weight,
                          vc_act_t act, bool has_dbias) {
    size_t need = packed_bytes(x) + packed_bytes(weight);
    if (act != VC_ACT_NONE || !operand_ready(dy))
        need += dz_planes(dy->rows, act) * round256((size_t)dy->rows * padded_ld(dy->cols) * 2);
    if (has_dbias) need += round256((size_t)dz_row_blocks(dy->rows, dy->cols, act) * dy->cols * 4);
    return need;
}

}  // namespace
}  // namespace train
}  // namespace vc

using namespace vc;
using namespace vc::train;

extern "C" {

size_t vc_linear_forward_workspace(const vc_matrix_t* x, const vc_matrix_t* weight) {
    if (!valid_matrix(x) || !valid_matrix(weight)) return 0;
    return packed_bytes(x) + packed_bytes(weight);
}

vc_status_t vc_linear_forward(const vc_matrix_t* x, const vc_matrix_t* weight, const void* bias,
                              const vc_matrix_t* residual, const vc_matrix_t* y,
                              const vc_matrix_t* preact, vc_act_t act, void* workspace,
                              size_t workspace_bytes, vc_stream_t stream) {
    if (!valid_matrix(x) || !valid_matrix(weight) || !valid_act(act)) return VC_ERR_INVALID_ARGUMENT;
    const long long M = x->rows, K = x->cols, N = weight->rows;
    if (!plain_matrix(x, M, K) || !plain_matrix(weight, N, K) || !plain_matrix(y, M, N) ||
        (residual != nullptr && !plain_matrix(residual, M, N)) ||
        (preact != nullptr && !plain_matrix(preact, M, N)))
        return VC_ERR_INVALID_ARGUMENT;
    if (!is_bf16(x) || !is_bf16(weight) || !is_bf16(y) || (residual != nullptr && !is_bf16(residual)) ||
        (preact != nullptr && !is_bf16(preact)))
        return VC_ERR_INVALID_ARGUMENT;
    if ((reinterpret_cast<uintptr_t>(bias) & 1) != 0) return VC_ERR_INVALID_ARGUMENT;
    const size_t need = packed_bytes(x) + packed_bytes(weight);
    if (!workspace_ok(workspace, workspace_bytes, need)) return VC_ERR_INVALID_ARGUMENT;
    const Span outs[3] = {span_of(y), span_of(preact), span_of(workspace, need)};
    const Span ins[4] = {span_of(x), span_of(weight), span_of(bias, (size_t)N * 2), span_of(residual)};
    for (int o = 0; o < 3; ++o) {
        for (int i = 0; i < 4; ++i)
            if (overlap(outs[o], ins[i]) &&
                !(o == 0 && i == 3 && same_matrix(y, residual)))
                return VC_ERR_ALIAS;
        for (int q = 0; q < o; ++q)
            if (overlap(outs[o], outs[q])) return VC_ERR_ALIAS;
    }
    if (M == 0 || N == 0) return VC_SUCCESS;
    if (test_launch_failure()) return VC_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    Operand a = {nullptr, K, M, 0, 0, true, false}, b = {nullptr, K, N, 0, 0, true, false};
    Jobs jobs = {};
    ready_operand(x, &ws, &jobs, &a);
    ready_operand(weight, &ws, &jobs, &b);
    if (launch_jobs(jobs, st) != cudaSuccess) return VC_ERR_CUDA;
    const Forward f = {a, b, (int)M, (int)N, (int)K, bias, residual, y, preact, act};
    cudaError_t e;
    switch (act_family(act)) {
    case kFamilyErf: e = forward<kFamilyErf>(f, st); break;
    case kFamilyLogistic: e = forward<kFamilyLogistic>(f, st); break;
    default: e = forward<kFamilyPiecewise>(f, st);
    }
    return e == cudaSuccess ? VC_SUCCESS : VC_ERR_CUDA;
}

size_t vc_linear_backward_workspace(const vc_matrix_t* dy, const vc_matrix_t* x,
                                    const vc_matrix_t* weight, vc_act_t act, int has_dbias) {
    if (!valid_matrix(dy) || !valid_matrix(x) || !valid_matrix(weight)) return 0;
    return backward_workspace(dy, x, weight, act, has_dbias != 0);
}

vc_status_t vc_linear_backward(const vc_matrix_t* dy, const vc_matrix_t* x,
                               const vc_matrix_t* weight, const vc_matrix_t* preact, vc_act_t act,
                               const vc_matrix_t* dx, const vc_matrix_t* dweight, void* dbias,
                               vc_dtype_t dbias_dtype, int accumulate, void* workspace,
                               size_t workspace_bytes, vc_stream_t stream) {
    if (!valid_matrix(dy) || !valid_matrix(x) || !valid_matrix(weight) || !valid_act(act))
        return VC_ERR_INVALID_ARGUMENT;
    const long long M = x->rows, K = x->cols, N = weight->rows;
    const bool has_act = act != VC_ACT_NONE;
    if (!plain_matrix(x, M, K) || !plain_matrix(weight, N, K) || !plain_matrix(dy, M, N) ||
        (has_act && (preact == nullptr || !plain_matrix(preact, M, N) || !is_bf16(preact))) ||
        (dx != nullptr && (!plain_matrix(dx, M, K) || !is_bf16(dx))) ||
        (dweight != nullptr && !plain_matrix(dweight, N, K)))
        return VC_ERR_INVALID_ARGUMENT;
    if (!is_bf16(x) || !is_bf16(weight) || !is_bf16(dy)) return VC_ERR_INVALID_ARGUMENT;
    const int bias_size = elem_size(dbias_dtype);
    if (dbias != nullptr &&
        (bias_size == 0 || reinterpret_cast<uintptr_t>(dbias) % bias_size != 0))
        return VC_ERR_INVALID_ARGUMENT;
    const size_t need = backward_workspace(dy, x, weight, act, dbias != nullptr);
    if (!workspace_ok(workspace, workspace_bytes, need)) return VC_ERR_INVALID_ARGUMENT;
    const Span outs[4] = {span_of(dx), span_of(dweight), span_of(dbias, (size_t)N * bias_size),
                          span_of(workspace, need)};
    const Span ins[4] = {span_of(dy), span_of(x), span_of(weight),
                         has_act ? span_of(preact) : Span{}};
    for (int o = 0; o < 4; ++o) {
        for (int i = 0; i < 4; ++i)
            if (overlap(outs[o], ins[i])) return VC_ERR_ALIAS;
        for (int q = 0; q < o; ++q)
            if (overlap(outs[o], outs[q])) return VC_ERR_ALIAS;
    }
    if (dx == nullptr && dweight == nullptr && dbias == nullptr) return VC_SUCCESS;
    if (N == 0 && M * K == 0) return VC_SUCCESS;
    if (test_launch_failure()) return VC_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned char* ws = static_cast<unsigned char*>(workspace);

    const bool write_dz = has_act || !operand_ready(dy);
    const void* dz = dy->data;
    long long ld_dz = M > 1 ? dy->ld : padded_ld(N);
    const int planes = dz_planes(M, act);
    const long long plane = (long long)(round256((size_t)M * padded_ld(N) * 2) / 2);
    float* sums = nullptr;
    const int parts = dz_row_blocks(M, N, act);
    if (dbias != nullptr) {
        sums = reinterpret_cast<float*>(ws);
        ws += round256((size_t)parts * N * 4);
    }
    if (write_dz) {
        dz = ws;
        ld_dz = padded_ld(N);
        ws += planes * round256((size_t)M * ld_dz * 2);
    }
    Jobs jobs = {};
    cudaError_t e = cudaSuccess;
    if (N > 0 && (sums != nullptr || (write_dz && M > 0))) {
        DzParams p = {};
        p.dy = view_of(dy);
        p.preact = view_of(has_act ? preact : nullptr);
        p.dz = write_dz ? static_cast<__nv_bfloat16*>(const_cast<void*>(dz)) : nullptr;
        p.dz_rest = planes == 2 ? p.dz + plane : nullptr;
        p.ld_dz = ld_dz;
        p.vec16 = p.dy.vec16 && (!has_act || p.preact.vec16);
        if (dbias != nullptr) {
            const SumJob sum = {sums, dbias, parts, (int)N, dbias_dtype == VC_FLOAT32, accumulate != 0};
            if (parts == 1) {
                p.direct = sum;
            } else {
                p.sums = sums;
                jobs.sum = sum;
            }
        }
        p.rows = M;
        p.cols = N;
        p.act = act_params(act);
        auto* kernel = !has_act                              ? dz_kernel<kNoActivation>
                       : act_family(act) == kFamilyErf        ? dz_kernel<kFamilyErf>
                       : act_family(act) == kFamilyLogistic ? dz_kernel<kFamilyLogistic>
                                                            : dz_kernel<kFamilyPiecewise>;
        e = launch_pdl(kernel, dim3((unsigned)((N + 255) / 256), parts), dim3(256), st, p);
        if (e != cudaSuccess) return VC_ERR_CUDA;
    }
    Product p[2];
    EpiStore<false>::Params ep[2];
    int count = 0;
    if (dx != nullptr && M > 0 && K > 0) {
        const Operand a = {dz, N, M, ld_dz, plane, true, false};
        Operand b = {nullptr, K, N, 0, 0, true, true};
        ready_operand(weight, &ws, &jobs, &b);
        p[count] = {a, b, (int)M, (int)K, (int)N, 1, planes};
        ep[count++] = {view_of(dx), 0};
    }
    if (dweight != nullptr && N > 0 && K > 0) {
        const Operand a = {dz, N, M, ld_dz, plane, true, true};
        Operand b = {nullptr, K, M, 0, 0, true, true};
        ready_operand(x, &ws, &jobs, &b);
        p[count] = {a, b, (int)N, (int)K, (int)M, 1, planes};
        ep[count++] = {view_of(dweight), accumulate != 0};
    }
    if (launch_jobs(jobs, st) != cudaSuccess) return VC_ERR_CUDA;
    if (count > 0) {
        // 32-bit sums are not left to the tensor cores for longer than a segment
        const bool promote = dweight != nullptr && dweight->dtype == VC_FLOAT32;
        int limit[2] = {0, 0};
        bool odd = false;
        for (int i = 0; i < count; ++i) {
            if (ep[i].out.f32) limit[i] = kSegment;
            odd = odd || !ep[i].out.vec16;
        }
        auto by_pairs = [&](int first, int n) {
            if (n == 2)
                return promote ? gemm::launch_pair<EpiStore<false>, 2, true>(p, ep, kSegment, st)
                               : gemm::launch_pair<EpiStore<false>, 2, false>(p, ep, 0, st);
            return promote
                       ? gemm::launch_pair<EpiStore<false>, 1, true>(p + first, ep + first, kSegment, st)
                       : gemm::launch_pair<EpiStore<false>, 1, false>(p + first, ep + first, 0, st);
        };
        // the products from `first` on, in one launch of the better kernel
        auto together = [&](int first, double* us) {
            const int n = count - first;
            const gemm::Plan plan = gemm::plan_split(p + first, n, false, odd, limit + first);
            const double pairs = gemm::pair_us(p + first, n, false, odd);
            if (us != nullptr) {
                *us = std::min(plan.us, pairs);
                return cudaSuccess;
            }
            if (plan.us >= pairs) return by_pairs(first, n);
            return n == 2 ? gemm::launch_planned<EpiStore<false>, 2>(p + first, ep + first, plan, st)
                          : gemm::launch_planned<EpiStore<false>, 1>(p + first, ep + first, plan, st);
        };
        // dx of few rows by itself, computed transposed as the forward product
        // is, where the model says so: dx alone of 4 x 2113 x 7168 takes 13.1 us
        // instead of 18.3, both gradients of 8 x 16384 x 1024 28.1 instead of 74.6
        bool skinny = false;
        gemm::Product turned = {};
        if (p[0].M == (int)M && p[0].N == (int)K && dx != nullptr && M <= kSwapRows) {
            Operand w = p[0].b, z = p[0].a;
            turned = {w, z, (int)K, (int)M, (int)N, 1, planes, true};
            double us = 0.0, rest = 0.0;
            together(0, &us);
            if (count == 2) together(1, &rest);
            skinny = gemm::plan_skinny(turned).us + rest + 2.5 * (count - 1) < us;
        }
        if (skinny) {
            const EpiStore<true>::Params sp = {ep[0].out, 0};
            e = gemm::launch_skinny<EpiStore<true>>(turned, sp, st);
            if (e == cudaSuccess && count == 2) e = together(1, nullptr);
        } else {
            e = together(0, nullptr);
        }
        if (e != cudaSuccess) return VC_ERR_CUDA;
    }
    return VC_SUCCESS;
}

}  // extern "C"
