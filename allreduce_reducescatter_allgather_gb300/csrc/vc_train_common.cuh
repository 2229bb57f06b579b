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

// The largest extent of one dimension: tile and TMA coordinates are ints.  Of
// all: no more than any memory holds, so that tiles can be counted in ints.
// And of a row's pitch: TMA's stay below 2^40 bytes.
constexpr long long kMaxExtent = 1ll << 30, kMaxElements = 1ll << 38, kMaxPitch = (1ll << 39) - 8;

// A matrix argument: sizes, alignment, strides.  Empty matrices need no data.
inline bool valid_matrix(const vc_matrix_t* m) {
    if (m == nullptr) return false;
    const int es = elem_size(m->dtype);
    if (es == 0) return false;
    if (m->batch < 0 || m->rows < 0 || m->cols < 0) return false;
    if (m->batch > kMaxExtent || m->rows > kMaxExtent || m->cols > kMaxExtent) return false;
    if (m->batch == 0 || m->rows == 0 || m->cols == 0) return true;
    if ((__int128)m->batch * m->rows * m->cols > kMaxElements) return false;
    if (m->data == nullptr || reinterpret_cast<uintptr_t>(m->data) % es != 0) return false;
    if (m->rows > 1 && (m->ld < m->cols || m->ld > kMaxPitch)) return false;
    const long long ld = m->rows > 1 ? m->ld : m->cols;
    const __int128 one = (__int128)(m->rows - 1) * ld + m->cols;
    if (one > ((__int128)1 << 58)) return false;
    if (m->batch > 1 && ((__int128)m->batch_stride < one || m->batch_stride > (1ll << 58)))
        return false;
    return m->batch == 1 || (__int128)m->batch * m->batch_stride <= ((__int128)1 << 58);
}

// The bytes of an argument: rows of `width`, all of them whole pitches after the
// first (pitch 0: one row).
struct Span {
    uintptr_t lo, hi, width, pitch;
};
inline Span span_of(const void* p, size_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return p == nullptr ? Span{} : Span{lo, lo + bytes, bytes, 0};
}
inline Span span_of(const vc_matrix_t* m) {
    if (m == nullptr || m->batch == 0 || m->rows == 0 || m->cols == 0) return {};
    const uintptr_t es = elem_size(m->dtype), lo = reinterpret_cast<uintptr_t>(m->data);
    // (sizes and strides were checked: nothing here passes 2^61)
    const uintptr_t row = m->rows > 1 ? m->ld * es : 0, next = m->batch > 1 ? m->batch_stride * es : 0;
    const uintptr_t width = m->cols * es;
    const uintptr_t matrix = (m->rows - 1) * row + width, all = (m->batch - 1) * next + matrix;
    if (row == 0) return {lo, lo + all, width, next};
    if (next % row == 0) return {lo, lo + all, width, row};
    // matrices that do not lie on one grid of rows: taken whole
    return {lo, lo + all, matrix, next};
}
// Slices of one wider tensor interleave without an overlap: with the same
// pitch, b's rows lie between a's where b's first byte falls, in a's pitch,
// behind a's row, and b's row ends before a's next one.
inline bool overlap(Span a, Span b) {
    if (!(a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi)) return false;
    const uintptr_t pitch = a.pitch != 0 ? a.pitch : b.pitch;
    if (pitch == 0 || (a.pitch != 0 && b.pitch != 0 && a.pitch != b.pitch)) return true;
    const uintptr_t after = b.lo >= a.lo ? (b.lo - a.lo) % pitch : (pitch - (a.lo - b.lo) % pitch) % pitch;
    return after < a.width || after + b.width > pitch;
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
    const long long per = v.f32 ? 4 : 8;
    v.vec16 = reinterpret_cast<uintptr_t>(m->data) % 16 == 0 && v.ld % per == 0 &&
              v.batch_stride % per == 0;
    return v;
}

inline size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// Row length, in 16-bit values, of operands laid out in the workspace: whole 128
// bytes, the width of a TMA box, whose rows then do not straddle lines.
inline long long padded_ld(long long cols) { return (cols + 63) / 64 * 64; }

// ------------------------------------------------------------ activations --

// exp2 and the reciprocal are the hardware's approximations, good to two units
// in the last place of float32; the results are rounded to bf16.
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float logistic(float z) { return rcp_fast(1.0f + exp2_fast(-kLog2e * z)); }

constexpr float kGeluK = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;

// max(z, 0), NaN kept.
__device__ __forceinline__ float positive(float z) { return z <= 0.0f ? 0.0f : z; }

// z cut to at least, or at most, a value; NaN kept.  At infinities and where
// squares of z overflow, the activations and their derivatives take their
// limits: they are evaluated where the limit is reached in float32.
__device__ __forceinline__ float2 at_least(float2 z, float a) {
    float2 r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r.x) : "f"(z.x), "f"(a));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r.y) : "f"(z.y), "f"(a));
    return r;
}
__device__ __forceinline__ float2 at_most(float2 z, float a) {
    float2 r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r.x) : "f"(z.x), "f"(a));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r.y) : "f"(z.y), "f"(a));
    return r;
}
constexpr float kLogisticFlat = 128.0f;  // exp(-128) is 0 beside 1, exp(128) infinite
constexpr float kBellFlat = 30.0f;       // exp(-30^2 / 2) is 0

// The activations in three families, so that a kernel holds the arithmetic of
// one and no element branches: piecewise (none, relu, relu2), logistic (silu
// and the tanh form of gelu, z / (1 + exp(-k z (1 + c z^2)))), and erf.
enum { kFamilyPiecewise = 0, kFamilyLogistic = 1, kFamilyErf = 2, kNoActivation = 3 };

inline int act_family(int act) {
    return act == VC_ACT_GELU ? kFamilyErf
           : act == VC_ACT_GELU_TANH || act == VC_ACT_SILU ? kFamilyLogistic : kFamilyPiecewise;
}

struct Act {
    float k, c;      // logistic
    int identity, square;  // piecewise: none, or max(z, 0) and its square
};
inline Act act_params(int act) {
    Act a = {};
    a.k = act == VC_ACT_GELU_TANH ? kGeluK : 1.0f;
    a.c = act == VC_ACT_GELU_TANH ? kGeluC : 0.0f;
    a.identity = act == VC_ACT_NONE;
    a.square = act == VC_ACT_RELU2;
    return a;
}

// erfc(x / sqrt(2)) / 2 = Phi(-x) for x >= 0, given e = exp(-x^2 / 2): the
// rational approximation 7.1.26 of Abramowitz and Stegun, "Handbook of
// Mathematical Functions", with their coefficients halved and p divided by
// sqrt(2); its error is below 7.5e-8.
constexpr float kTailP = 0.3275911f * 0.70710678118654752f;
constexpr float kTail0 = 0.5f * 0.254829592f, kTail1 = 0.5f * -0.284496736f,
                kTail2 = 0.5f * 1.421413741f, kTail3 = 0.5f * -1.453152027f,
                kTail4 = 0.5f * 1.061405429f;
__device__ __forceinline__ float2 normal_tail(float2 x, float2 e) {
    const float2 d = gemm::fma2(x, gemm::both(kTailP), gemm::both(1.0f));
    const float2 t = make_float2(rcp_fast(d.x), rcp_fast(d.y));
    float2 y = gemm::fma2(t, gemm::both(kTail4), gemm::both(kTail3));
    y = gemm::fma2(t, y, gemm::both(kTail2));
    y = gemm::fma2(t, y, gemm::both(kTail1));
    y = gemm::fma2(t, y, gemm::both(kTail0));
    return gemm::mul2(gemm::mul2(t, y), e);
}
// exp(-z^2 / 2)
__device__ __forceinline__ float2 bell(float2 z) {
    const float2 q = gemm::mul2(gemm::mul2(z, z), gemm::both(-0.5f * kLog2e));
    return make_float2(exp2_fast(q.x), exp2_fast(q.y));
}

// Two values at a time: the epilogues are bound by instructions where K is
// short, and paired arithmetic halves them.  Not called for the identity.
template <int kFamily>
__device__ __forceinline__ float2 act_value(float2 z, const Act& a) {
    if constexpr (kFamily == kFamilyPiecewise) {
        const float2 y = make_float2(positive(z.x), positive(z.y));
        return a.square ? gemm::mul2(y, y) : y;
    } else if constexpr (kFamily == kFamilyLogistic) {
        // u = -log2(e) k z (1 + c z^2)
        const float2 y = at_least(z, -kLogisticFlat), x = at_most(y, kLogisticFlat);
        const float2 q = gemm::fma2(gemm::mul2(x, x), gemm::both(a.c), gemm::both(1.0f));
        const float2 u = gemm::mul2(gemm::mul2(x, gemm::both(-kLog2e * a.k)), q);
        const float2 d = gemm::add2(make_float2(exp2_fast(u.x), exp2_fast(u.y)), gemm::both(1.0f));
        return gemm::mul2(y, make_float2(rcp_fast(d.x), rcp_fast(d.y)));
    } else {
        // max(z, 0) - |z| Phi(-|z|)
        const float2 x = make_float2(fminf(fabsf(z.x), kBellFlat), fminf(fabsf(z.y), kBellFlat));
        const float2 h = gemm::mul2(x, normal_tail(x, bell(z)));
        return make_float2(fmaxf(z.x, 0.0f) - h.x, fmaxf(z.y, 0.0f) - h.y);
    }
}

// act'(v); not called for the identity.
template <int kFamily>
__device__ __forceinline__ float2 act_slope(float2 v, const Act& a) {
    if constexpr (kFamily == kFamilyPiecewise) {
        return a.square ? make_float2(2.0f * positive(v.x), 2.0f * positive(v.y))
                        : make_float2(v.x > 0.0f ? 1.0f : 0.0f, v.y > 0.0f ? 1.0f : 0.0f);
    } else if constexpr (kFamily == kFamilyLogistic) {
        // with u = k z (1 + c z^2): s(u) + z s(u) (1 - s(u)) k (1 + 3 c z^2)
        const float2 z = at_most(at_least(v, -kLogisticFlat), kLogisticFlat);
        const float2 q = gemm::mul2(gemm::mul2(z, z), gemm::both(a.c));
        const float2 u = gemm::mul2(gemm::mul2(z, gemm::both(a.k)), gemm::add2(q, gemm::both(1.0f)));
        const float2 s = make_float2(logistic(u.x), logistic(u.y));
        const float2 rest = make_float2(1.0f - s.x, 1.0f - s.y);
        const float2 k = gemm::mul2(gemm::fma2(q, gemm::both(3.0f), gemm::both(1.0f)), gemm::both(a.k));
        return gemm::mul2(s, gemm::fma2(gemm::mul2(z, rest), k, gemm::both(1.0f)));
    } else {
        // Phi(z) + z phi(z)
        const float2 z = at_most(at_least(v, -kBellFlat), kBellFlat), e = bell(z);
        const float2 x = make_float2(fabsf(z.x), fabsf(z.y));
        const float2 h = normal_tail(x, e);
        const float2 phi = make_float2(z.x > 0.0f ? 1.0f - h.x : h.x, z.y > 0.0f ? 1.0f - h.y : h.y);
        return gemm::fma2(gemm::mul2(z, gemm::both(0.39894228040143268f)), e, phi);
    }
}

}  // namespace train
}  // namespace vc
