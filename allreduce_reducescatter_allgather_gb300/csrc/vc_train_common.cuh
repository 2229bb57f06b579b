// What the training-step entry points share: argument checks of matrices,
// activations, and the operand copies.
#pragma once

#include <stdint.h>
#include <stdlib.h>

#include "vc_device.cuh"
#include "vc_gemm.cuh"
#include "vc_train.h"

namespace vc {
namespace train {

inline int elem_size(vc_dtype_t dt) { return dt == VC_FLOAT32 ? 4 : dt == VC_BFLOAT16 ? 2 : 0; }

// The largest extent of one dimension: tile and TMA coordinates are ints.
constexpr long long kMaxExtent = 1ll << 30;

// A matrix argument: sizes, alignment, strides.  Empty matrices need no data.
inline bool valid_matrix(const vc_matrix_t* m) {
    if (m == nullptr) return false;
    const int es = elem_size(m->dtype);
    if (es == 0) return false;
    if (m->batch < 0 || m->rows < 0 || m->cols < 0) return false;
    if (m->batch > kMaxExtent || m->rows > kMaxExtent || m->cols > kMaxExtent) return false;
    if (m->batch == 0 || m->rows == 0 || m->cols == 0) return true;
    if (m->data == nullptr || reinterpret_cast<uintptr_t>(m->data) % es != 0) return false;
    if (m->rows > 1 && (m->ld < m->cols || m->ld > (1ll << 40))) return false;
    const long long ld = m->rows > 1 ? m->ld : m->cols;
    const __int128 one = (__int128)(m->rows - 1) * ld + m->cols;
    if (one > ((__int128)1 << 58)) return false;
    if (m->batch > 1 && ((__int128)m->batch_stride < one || m->batch_stride > (1ll << 58)))
        return false;
    return m->batch == 1 || (__int128)m->batch * m->batch_stride <= ((__int128)1 << 58);
}

struct Span {
    uintptr_t lo, hi;
};
inline Span span_of(const vc_matrix_t* m) {
    if (m == nullptr || m->batch == 0 || m->rows == 0 || m->cols == 0) return {0, 0};
    const long long ld = m->rows > 1 ? m->ld : m->cols;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(m->data);
    const long long last = (m->batch - 1) * (m->batch > 1 ? m->batch_stride : 0) +
                           (m->rows - 1) * ld + m->cols;
    return {lo, lo + (uintptr_t)last * elem_size(m->dtype)};
}
inline Span span_of(const void* p, size_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return p == nullptr ? Span{0, 0} : Span{lo, lo + bytes};
}
inline bool overlap(Span a, Span b) {
    return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi;
}
// Exactly the same elements (an output that may stand in an input's place).
inline bool same_matrix(const vc_matrix_t* a, const vc_matrix_t* b) {
    return a->data == b->data && a->dtype == b->dtype && (a->rows <= 1 || a->ld == b->ld) &&
           (a->batch <= 1 || a->batch_stride == b->batch_stride);
}

inline bool test_launch_failure() {
    const char* v = getenv("VC_TEST_FAIL_LAUNCH");
    return v != nullptr && v[0] != '\0' && v[0] != '0';
}

inline gemm::View view_of(const vc_matrix_t* m) {
    gemm::View v = {};
    if (m == nullptr) return v;
    v.data = m->data;
    v.ld = m->rows > 1 ? m->ld : 0;
    v.batch_stride = m->batch > 1 ? m->batch_stride : 0;
    v.f32 = m->dtype == VC_FLOAT32;
    const uintptr_t bytes = v.f32 ? 16 : 8;
    v.vec = reinterpret_cast<uintptr_t>(m->data) % bytes == 0 && v.ld % 4 == 0 &&
            v.batch_stride % 4 == 0;
    return v;
}

inline size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// Row length, in 16-bit values, of matrices laid out in the workspace.
inline long long padded_ld(long long cols) { return (cols + 7) / 8 * 8; }

// ------------------------------------------------------------ activations --

// __expf is good to a few units in the last place of float32 over the range
// where its result matters here; the results are rounded to bf16.
__device__ __forceinline__ float logistic(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

constexpr float kGeluK = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;

// max(z, 0), NaN kept.
__device__ __forceinline__ float positive(float z) { return z <= 0.0f ? 0.0f : z; }

__device__ __forceinline__ float act_value(float z, int act) {
    switch (act) {
    case VC_ACT_RELU: return positive(z);
    case VC_ACT_RELU2: return positive(z) * positive(z);
    case VC_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    // (1 + tanh u) / 2 is the logistic function of 2 u
    case VC_ACT_GELU_TANH: return z * logistic(kGeluK * (z + kGeluC * z * z * z));
    case VC_ACT_SILU: return z * logistic(z);
    default: return z;
    }
}

__device__ __forceinline__ float act_slope(float z, int act) {
    switch (act) {
    case VC_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case VC_ACT_RELU2: return 2.0f * positive(z);
    case VC_ACT_GELU:
        return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) +
               z * __expf(-0.5f * z * z) * 0.39894228040143268f;
    case VC_ACT_GELU_TANH: {
        const float s = logistic(kGeluK * (z + kGeluC * z * z * z));
        return s + z * s * (1.0f - s) * kGeluK * (1.0f + 3.0f * kGeluC * z * z);
    }
    case VC_ACT_SILU: {
        const float s = logistic(z);
        return s * (1.0f + z * (1.0f - s));
    }
    default: return 1.0f;
    }
}

}  // namespace train
}  // namespace vc
