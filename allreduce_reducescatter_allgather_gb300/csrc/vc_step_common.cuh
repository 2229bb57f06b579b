// What the entry points of vc_step.h share: rows of matrices eight values at a
// time, sums over warps, and launches.
#pragma once

#include "vc_step.h"
#include "vc_train_common.cuh"

namespace vc {
namespace step {

using train::elem_size;
using train::overlap;
using train::round256;
using train::same_matrix;
using train::Span;
using train::span_of;
using train::test_launch_failure;
using train::valid_matrix;

constexpr int kSMs = 152;
constexpr size_t kSharedLimit = 227u << 10;  // of a block; an SM has 1 KiB a block more

inline bool plain_matrix(const vc_matrix_t* m, long long rows, long long cols) {
    return valid_matrix(m) && m->batch == 1 && m->rows == rows && m->cols == cols;
}
inline bool workspace_ok(const void* ws, size_t have, size_t need) {
    return need == 0 || (ws != nullptr && (reinterpret_cast<uintptr_t>(ws) & 255) == 0 && have >= need);
}
inline bool valid_dtype(vc_dtype_t d) { return d == VC_FLOAT32 || d == VC_BFLOAT16; }

// A matrix as kernels take it.  vec: groups of eight columns start on 16 bytes in
// every row.
struct Rows {
    void* data;
    long long ld;
    int f32, vec;
};
inline Rows rows_of(const vc_matrix_t* m) {
    Rows r = {};
    if (m == nullptr) return r;
    r.data = m->data;
    r.ld = m->rows > 1 ? m->ld : 0;
    r.f32 = m->dtype == VC_FLOAT32;
    r.vec = reinterpret_cast<uintptr_t>(m->data) % 16 == 0 && r.ld % (r.f32 ? 4 : 8) == 0;
    return r;
}

// Eight values, computed two at a time.
struct Eight {
    float v[8];
    __device__ __forceinline__ float2 two(int j) const { return make_float2(v[2 * j], v[2 * j + 1]); }
    __device__ __forceinline__ void set(int j, float2 x) { v[2 * j] = x.x, v[2 * j + 1] = x.y; }
};
__device__ __forceinline__ Eight zeros() { return {{0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}}; }
__device__ __forceinline__ Eight fma(const Eight& a, const Eight& b, const Eight& c) {
    Eight r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.set(j, gemm::fma2(a.two(j), b.two(j), c.two(j)));
    return r;
}
__device__ __forceinline__ Eight fma(float a, const Eight& b, const Eight& c) {
    Eight r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.set(j, gemm::fma2(gemm::both(a), b.two(j), c.two(j)));
    return r;
}
__device__ __forceinline__ Eight mul(const Eight& a, const Eight& b) {
    Eight r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.set(j, gemm::mul2(a.two(j), b.two(j)));
    return r;
}
__device__ __forceinline__ Eight mul(float a, const Eight& b) {
    Eight r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.set(j, gemm::mul2(gemm::both(a), b.two(j)));
    return r;
}
__device__ __forceinline__ Eight add(const Eight& a, const Eight& b) {
    Eight r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.set(j, gemm::add2(a.two(j), b.two(j)));
    return r;
}
__device__ __forceinline__ Eight add(float a, const Eight& b) {
    Eight r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.set(j, gemm::add2(gemm::both(a), b.two(j)));
    return r;
}
// s += a b, in two halves
__device__ __forceinline__ void dot(float2& s, const Eight& a, const Eight& b) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s = gemm::fma2(a.two(j), b.two(j), s);
}
__device__ __forceinline__ void total(float2& s, const Eight& a) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s = gemm::add2(s, a.two(j));
}
__device__ __forceinline__ float sum_of(float2 s) { return s.x + s.y; }

// 16 bytes, of which the first `bytes` come from `from` and the others are zeros.
__device__ __forceinline__ void copy16(uint4* to, const void* from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 ::"r"((unsigned)__cvta_generic_to_shared(to)), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until all but the last kLeft groups of this thread's copies are there.
template <int kLeft>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

__device__ __forceinline__ Eight widen(uint4 u) {
    Eight r;
    const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        r.v[2 * j] = __uint_as_float(w[j] << 16);
        r.v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
    return r;
}
__device__ __forceinline__ unsigned narrow2(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const unsigned*>(&p);
}
__device__ __forceinline__ uint4 narrow(const Eight& r) {
    return make_uint4(narrow2(r.v[0], r.v[1]), narrow2(r.v[2], r.v[3]), narrow2(r.v[4], r.v[5]),
                      narrow2(r.v[6], r.v[7]));
}

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
template <int kTeam>
__device__ __forceinline__ Eight load_as(const Rows& x, bool f32, long long row, bool vec, int v, int lane, int cols) {
    return f32 ? load_f32<kTeam>(x.data, row * x.ld, vec, v, lane, cols)
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

// Eight columns of a row as they lie in memory, so that a thread can hold the next
// row's while it computes with this one's: eight 32-bit words of float32, or of
// bfloat16 four words of two (on 16 bytes) or eight of one.
struct Raw {
    unsigned w[8];
};
// kOnce: what is read once leaves the caches to what is not.
template <bool kOnce, class T>
__device__ __forceinline__ T load_word(const T* p) {
    return kOnce ? __ldcs(p) : *p;
}
template <int kTeam>
__device__ __forceinline__ Raw load_raw(const Rows& x, bool f32, long long row, bool vec, int v, int lane, int cols) {
    const long long at = row * x.ld;
    const int c = (v * kTeam + lane) * 8;
    Raw r;
    if (vec && c + 8 <= cols) {
        if (f32) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(x.data) + at + c);
            const uint4 lo = load_word<true>(p), hi = load_word<true>(p + 1);
            r = {{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
        } else {
            const uint4 u = load_word<true>(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x.data) + at + c));
            r.w[0] = u.x, r.w[1] = u.y, r.w[2] = u.z, r.w[3] = u.w;
        }
        return r;
    }
    if (!f32 && vec)
#pragma unroll
        for (int j = 0; j < 4; ++j) r.w[j] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int k = column<kTeam>(vec, v, lane, j);
        if (f32) {
            r.w[j] = k < cols ? load_word<true>(static_cast<const unsigned*>(x.data) + at + k) : 0;
        } else {
            const unsigned u = k < cols ? load_word<true>(static_cast<const unsigned short*>(x.data) + at + k) : 0;
            if (vec)
                r.w[j / 2] |= u << (j % 2 * 16);
            else
                r.w[j] = u;
        }
    }
    return r;
}
__device__ __forceinline__ Eight widen_raw(const Raw& r, bool f32, bool vec) {
    Eight e;
    if (f32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) e.v[j] = __uint_as_float(r.w[j]);
    } else if (vec) {
        e = widen(make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) e.v[j] = __uint_as_float(r.w[j] << 16);
    }
    return e;
}

// ---------------------------------------------------------------------- warps --

// The sum of a whole warp, the same in every lane.
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_next() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------------- clusters --

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
}
// What lies at `at` in block `rank` of the cluster.
__device__ __forceinline__ unsigned remote_address(const void* at, unsigned rank) {
    unsigned address;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(address) : "r"((unsigned)__cvta_generic_to_shared(at)), "r"(rank));
    return address;
}
__device__ __forceinline__ unsigned remote_load(const unsigned* at, unsigned rank) {
    unsigned v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote_address(at, rank)) : "memory");
    return v;
}
__device__ __forceinline__ void remote_store(uint2* at, unsigned rank, uint2 v) {
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};"
                 ::"r"(remote_address(at, rank)), "r"(v.x), "r"(v.y) : "memory");
}

// launch_pdl with dynamic shared memory, and clusters of `span` blocks.
template <class... KArgs, class... Args>
cudaError_t launch_pdl_shared(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t bytes, int span, cudaStream_t st,
                              Args&&... args) {
    if (bytes > 24u << 10) {  // (with what the kernel has of its own, above 48 KiB)
        const cudaError_t e = gemm::allow_smem(reinterpret_cast<const void*>(kernel));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = span;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = span > 1 ? 2 : 1;
    return reported(cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...));
}

}  // namespace step
}  // namespace vc
