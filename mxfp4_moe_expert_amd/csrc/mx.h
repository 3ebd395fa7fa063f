// mx.h -- what the microscaled-activation kernels share (mx.hip, mxmm.hip):
// group scales and codes, element types, and the host-side checks.
#pragma once

#include <math.h>

#include "k3g_common.h"

namespace k3g {

typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef short short2_t __attribute__((ext_vector_type(2)));

constexpr int kMxMaxIn = 65536;

// The exponent e of a group whose largest magnitude has the fp32 bits mb (all
// finite): the smallest e >= -126 with max <= M 2^e, M = 6 = 1.5 * 2^2 or
// 448 = 1.75 * 2^8. With max = m * 2^E, m in [1, 2), that is E - 2 or E - 8,
// one more where m is above M's mantissa. The floor keeps 2^e a normal fp32
// number; a subnormal or zero max ends there too.
template <int FMT>
__device__ inline int mx_exponent(uint32_t mb) {
    const int E = int(mb >> 23) - 127;
    const uint32_t frac = mb & 0x7FFFFFu;
    const int e = FMT == K3G_MXFP4 ? E - 2 + (frac > 0x400000u ? 1 : 0) : E - 8 + (frac > 0x600000u ? 1 : 0);
    return e < -126 ? -126 : e;
}

constexpr uint32_t kMxNotFinite = 0x7F800000u;  // magnitude bits from here on: an infinity or a NaN

// Eight entries of a group -> their codes (MXFP4: one dword, entry 0 in the low
// nibble; MXFP8: two), by gfx950's scaled converts (v / 2^e to nearest, ties to
// the even code; |v| <= M 2^e, so nothing saturates).
template <int FMT>
__device__ inline void mx_codes8(const float *v, float scale, uint32_t *w) {
    if constexpr (FMT == K3G_MXFP4) {
        uint32_t d = 0;
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[0], v[1], scale, 0);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[2], v[3], scale, 1);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[4], v[5], scale, 2);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[6], v[7], scale, 3);
        w[0] = d;
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            short2_t d = {0, 0};
            d = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(d, v[4 * k], v[4 * k + 1], scale, false);
            d = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(d, v[4 * k + 2], v[4 * k + 3], scale, true);
            w[k] = __builtin_bit_cast(uint32_t, d);
        }
    }
}

__device__ inline float pow2(int e) { return __builtin_bit_cast(float, uint32_t(e + 127) << 23); }  // e in [-126, 127]

// ---- element types: eight consecutive entries to and from fp32 ---------------------
// The pointers are aligned to their entries only; gfx950 reads and writes
// 16 bytes at any such address, and the compiler picks the width.

template <int TYPE>
struct Elem;
template <>
struct Elem<K3G_F32> {
    typedef float T;
    static __device__ inline float load(T v) { return v; }
    static __device__ inline T store(float v) { return v; }
};
template <>
struct Elem<K3G_BF16> {
    typedef __bf16 T;
    static __device__ inline float load(T v) { return (float)v; }
    static __device__ inline T store(float v) { return (__bf16)v; }
};
template <>
struct Elem<K3G_F16> {
    typedef _Float16 T;
    static __device__ inline float load(T v) { return (float)v; }
    static __device__ inline T store(float v) { return (_Float16)v; }
};

template <int TYPE, int N>
__device__ inline void load_n(float *v, const typename Elem<TYPE>::T *p) {
    typename Elem<TYPE>::T t[N];
    __builtin_memcpy(t, p, sizeof t);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = Elem<TYPE>::load(t[i]);
}

template <int TYPE, int N>
__device__ inline void store_n(typename Elem<TYPE>::T *p, const float *v) {
    typename Elem<TYPE>::T t[N];
#pragma unroll
    for (int i = 0; i < N; ++i) t[i] = Elem<TYPE>::store(v[i]);
    __builtin_memcpy(p, t, sizeof t);
}

// ---- host checks --------------------------------------------------------------------

int device_ok();  // abi.hip

inline bool mx_aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline size_t type_size(int type) { return type == K3G_F32 ? 4 : 2; }
inline bool type_ok(int type) { return type == K3G_F32 || type == K3G_BF16 || type == K3G_F16; }

// The addresses a call touches: one range, or (pitch not 0) rows of `width` bytes,
// `pitch` apart, of which the last ends at hi. Two sets of rows of one pitch meet
// where rows do; next to anything else the gaps between rows count as used.
struct Span {
    uintptr_t lo, hi;
    size_t pitch = 0, width = 0;
};
inline Span span(const void *p, size_t bytes) { return {(uintptr_t)p, (uintptr_t)p + bytes}; }
inline Span rows_span(const void *p, int type, int64_t n, int64_t stride, int64_t width) {
    if (!p || n < 1) return span(p, 0);
    Span s = span(p, type_size(type) * (size_t)((n - 1) * stride + width));
    s.pitch = type_size(type) * (size_t)stride;
    s.width = type_size(type) * (size_t)width;
    return s;
}
inline bool meet(const Span &a, const Span &b) {
    if (a.lo >= b.hi || b.lo >= a.hi) return false;
    if (a.pitch == 0 || a.pitch != b.pitch) return true;
    // a row of b begins d behind one of a's, and the next of a's pitch - d behind that
    const size_t back = (a.lo - b.lo) % a.pitch, d = b.lo >= a.lo ? (b.lo - a.lo) % a.pitch : back ? a.pitch - back : 0;
    return d < a.width || a.pitch - d < b.width;
}

inline size_t mx_code_bytes(const k3g_mx &m) { return (size_t)m.rows * m.in / (m.format == K3G_MXFP4 ? 2 : 1); }
inline Span codes_span(const k3g_mx &m) { return span(m.codes, mx_code_bytes(m)); }
inline Span scales_span(const k3g_mx &m) { return span(m.scales, (size_t)m.rows * (m.in / kGroup)); }

inline int mx_ok(const k3g_mx *m) {
    if (!m || (m->format != K3G_MXFP4 && m->format != K3G_MXFP8) || m->rows < 0 || m->in <= 0 || m->in % kGroup)
        return K3G_EINVAL;
    if (m->in > kMxMaxIn) return K3G_EUNSUPPORTED;
    if (m->rows == 0) return K3G_OK;
    if (!m->codes || !m->scales) return K3G_EINVAL;
    return mx_aligned(m->codes, 16) ? K3G_OK : K3G_EALIGN;
}

// A dense operand [n][width], rows `stride` entries apart, aligned to its entries.
inline int dense_ok(const void *p, int type, int64_t stride, int64_t width) {
    if (!p || !type_ok(type) || stride < width || stride > ((int64_t)1 << 40)) return K3G_EINVAL;
    return mx_aligned(p, type_size(type)) ? K3G_OK : K3G_EALIGN;
}

#define K3G_TRY(expr)                  \
    do {                               \
        const int rc_ = (expr);        \
        if (rc_ != K3G_OK) return rc_; \
    } while (0)

}  // namespace k3g
