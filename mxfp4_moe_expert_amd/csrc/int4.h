// int4.h -- what the int4 product kernels share (int4.hip, int4_stream.h):
// operands, codes on their way to the matrix cores, activations as operands.
//
// A weight is (n - z) s, n a code of 0 .. 15, s and z of its row's group of 32,
// 64 or 128 columns. The matrix cores multiply the codes themselves, which are
// exact in bf16 and fp16, and s is applied to the group's sum in fp32, so no
// weight is ever rounded:
//   y[t][r] = sum_g s_rg (sum_{c in g} n_rc x_tc - z_rg sum_{c in g} x_tc).
// The sum of x is a product with ones; -z times it, rounded, is what the product with
// the codes starts from, one group (32 columns at least) at a time. The vector kernel forms
// both sums and subtracts. Either way the result is off by roundings of the two
// sums, a few 2^-24 of (n + z) |x|: a row whose codes equal their zero gives nearly 0. (The
// tiles subtract z from the codes, which is exact, and give 0.)
#pragma once

#include "mxmm.h"

namespace k3g {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

// One product, or the products of every expert of a stack of matrices.
struct I4Args {
    const uint8_t *w[2];     // packed codes (GLU: w1, w3)
    const void *s[2];        // scales
    const uint8_t *z[2];     // zeros, or null: 8
    const void *x;
    const int32_t *offsets, *perm;  // grouped: ragged groups, and the source rows (null: straight)
    void *y;
    int64_t xs, ys;          // entries between rows
    int T;                   // rows of y (grouped: of all experts)
    int x_rows;
    int rows, in, G;         // outputs; entries and groups of a row
    int E, top_k;
    int s_type, y_type;
    int x_vec;  // the rows of x lie at 16-byte addresses
};

// Eight codes (a dword, the low nibble first) as bf16 or fp16, in order. A code
// zero-extended to a byte is n 2^-9 read as e4m3 (up to 7 subnormal, 8 to 15
// the lowest binade: one step throughout), so gfx950's scaled convert makes two of
// them at a time: 9 instructions, against 16 by single converts from int4.
template <int XT>
__device__ inline uint4 codes8(uint32_t d) {
    const uint32_t lo = d & 0x0F0F0F0Fu, hi = (d >> 4) & 0x0F0F0F0Fu;
    const uint32_t a = __builtin_amdgcn_perm(hi, lo, 0x05010400u), b = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
    if constexpr (XT == K3G_F16)
        return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 512.0f, false)),
                          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 512.0f, true)),
                          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 512.0f, false)),
                          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 512.0f, true)));
    else
        return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.0f, false)),
                          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.0f, true)),
                          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.0f, false)),
                          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.0f, true)));
}

// Eight entries of a token as they lie in memory.
template <int XT>
struct Raw4 {
    uint4 v;
    __device__ inline void load(const void *p) { __builtin_memcpy(&v, p, 16); }
};
template <>
struct Raw4<K3G_F32> {
    float f[8];
    __device__ inline void load(const void *p) { __builtin_memcpy(f, p, 32); }
};

// And as operand A. fp32 goes in as three bf16 parts, each the leading 8 bits of what the
// ones before leave. Their sum is the entry as far down as bf16 goes, 2^-133: from 2^-110 on
// all 24 bits, of smaller ones all but what is below that step.
template <int XT>
struct Act4;
template <>
struct Act4<K3G_BF16> {
    uint4 v;
    __device__ inline void take(const Raw4<K3G_BF16> &x) { v = x.v; }
    __device__ inline float4_t mul(const uint4 &w, float4_t c) const {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, v), __builtin_bit_cast(bf16x8_t, w), c, 0,
                                                       0, 0);
    }
    static __device__ inline uint4 ones() { return make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u); }
};
template <>
struct Act4<K3G_F16> {
    uint4 v;
    __device__ inline void take(const Raw4<K3G_F16> &x) { v = x.v; }
    __device__ inline float4_t mul(const uint4 &w, float4_t c) const {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, v), __builtin_bit_cast(f16x8_t, w), c, 0, 0,
                                                      0);
    }
    static __device__ inline uint4 ones() { return make_uint4(0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u); }
};
template <>
struct Act4<K3G_F32> {
    uint4 part[3];
    __device__ inline void take(const Raw4<K3G_F32> &x) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = x.f[i];
        uint32_t d[3][4];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a = __builtin_bit_cast(uint32_t, f[2 * i]), b = __builtin_bit_cast(uint32_t, f[2 * i + 1]);
                d[k][i] = __builtin_amdgcn_perm(b, a, 0x07060302u);
                f[2 * i] -= __builtin_bit_cast(float, a & 0xFFFF0000u);
                f[2 * i + 1] -= __builtin_bit_cast(float, b & 0xFFFF0000u);
            }
            part[k] = make_uint4(d[k][0], d[k][1], d[k][2], d[k][3]);
        }
    }
    __device__ inline float4_t mul(const uint4 &w, float4_t c) const {
#pragma unroll
        for (int k = 0; k < 3; ++k)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, part[k]),
                                                        __builtin_bit_cast(bf16x8_t, w), c, 0, 0, 0);
        return c;
    }
    static __device__ inline uint4 ones() { return Act4<K3G_BF16>::ones(); }
};

// An entry of a scale tensor.
__device__ inline float scale_at(const void *s, int type, int64_t i) {
    return type == K3G_F32 ? ((const float *)s)[i] : type == K3G_BF16 ? (float)((const __bf16 *)s)[i] : (float)((const _Float16 *)s)[i];
}
// N consecutive ones, as fp32.
template <int N>
__device__ inline void scales_at(float *v, const void *s, int type, int64_t i) {
    if (type == K3G_F32)
        load_n<K3G_F32, N>(v, (const float *)s + i);
    else if (type == K3G_BF16)
        load_n<K3G_BF16, N>(v, (const __bf16 *)s + i);
    else
        load_n<K3G_F16, N>(v, (const _Float16 *)s + i);
}

typedef const __attribute__((address_space(1))) uint8_t *global_t;

// BYTES (2, 4, 8 or 16) from any address into whole registers.
template <int BYTES>
__device__ inline void load_raw(uint32_t *v, global_t p) {
    if constexpr (BYTES == 2) {
        typedef uint16_t U __attribute__((aligned(1)));
        v[0] = *(const __attribute__((address_space(1))) U *)p;
    } else if constexpr (BYTES == 4) {
        typedef uint32_t U __attribute__((aligned(1)));
        v[0] = *(const __attribute__((address_space(1))) U *)p;
    } else {
        typedef uint32_t U __attribute__((ext_vector_type(BYTES / 4), aligned(1)));
        const U u = *(const __attribute__((address_space(1))) U *)p;
#pragma unroll
        for (int i = 0; i < BYTES / 4; ++i) v[i] = u[i];
    }
}

// The scales and zeros of N (2, 4 or 8) consecutive groups as they lie in memory.
// Loading looks at nothing that it loads and does not branch: a conversion, or a copy
// where two paths meet, would wait for every load that is under way. (Sixteen-bit
// scales are loaded twice, and where there are no zeros the caller has other bytes
// stand in for them.)
template <int N>
struct Scales4 {
    uint32_t lo[N / 2], hi[N / 2];  // fp32: one after the other
    uint32_t zero[(N + 3) / 4];
    __device__ inline void load(global_t s, int type, global_t z) {
        load_raw<2 * N>(lo, s);
        load_raw<2 * N>(hi, s + (type == K3G_F32 ? 2 * N : 0));
        load_raw<N>(zero, z);
    }
    __device__ inline float scale(int i, int type) const {
        const uint32_t word = i < N / 2 ? lo[i] : hi[i - N / 2], half = lo[i / 2] >> (i % 2 * 16) & 0xFFFFu;
        const float f16 = (float)__builtin_bit_cast(_Float16, (uint16_t)half);
        return type == K3G_F16 ? f16 : __builtin_bit_cast(float, type == K3G_F32 ? word : half << 16);
    }
    __device__ inline uint32_t zero_at(int i) const { return zero[i / 4] >> (i % 4 * 8) & 0xFFu; }
};

__device__ inline void store_out(void *y, int type, int64_t i, float v) {
    if (type == K3G_F32)
        ((float *)y)[i] = v;
    else if (type == K3G_BF16)
        ((__bf16 *)y)[i] = (__bf16)v;
    else
        ((_Float16 *)y)[i] = (_Float16)v;
}

// N consecutive outputs, of which the first n are there.
template <int N, int TYPE>
__device__ inline void store_outs_as(void *y, int64_t i, int n, const float *v) {
    typename Elem<TYPE>::T *p = (typename Elem<TYPE>::T *)y + i;
    if (n >= N) {
        store_n<TYPE, N>(p, v);
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (k < n) p[k] = Elem<TYPE>::store(v[k]);
    }
}
template <int N>
__device__ inline void store_outs(void *y, int type, int64_t i, int n, const float *v) {
    if (type == K3G_F32)
        store_outs_as<N, K3G_F32>(y, i, n, v);
    else if (type == K3G_BF16)
        store_outs_as<N, K3G_BF16>(y, i, n, v);
    else
        store_outs_as<N, K3G_F16>(y, i, n, v);
}

// The source row of row p of y.
__device__ inline int source(const I4Args &a, int p) {
    if (!a.perm) return p;
    const int q = a.perm[p];
    return min((int)((unsigned)max(q, 0) / (unsigned)a.top_k), a.x_rows - 1);
}

// v[c] of lane row q <-> v[q] of lane row c (a lane row: 16 lanes).
__device__ inline void transpose4(uint32_t *v) {
    auto s = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
    auto t = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
    auto a = __builtin_amdgcn_permlane16_swap(s[0], t[0], false, false);
    auto b = __builtin_amdgcn_permlane16_swap(s[1], t[1], false, false);
    v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1];
}

// A product's items at most (workgroups find the groups' real ones): tiles of `tok` rows by `out` outputs.
inline int64_t int4_items(const I4Args &a, int mode, int out, int tok) {
    const int64_t tiles = mode == DENSE ? ((int64_t)a.T + tok - 1) / tok : (int64_t)a.T / tok + (a.E < a.T ? a.E : a.T);
    return ((int64_t)a.rows + out - 1) / out * tiles;
}

// A launch: workgroups, and wavefronts of each.
struct Int4Grid {
    int64_t workgroups;
    int waves;
};

// The vector kernel's: a workgroup takes the outputs of `turns` turns of its wavefronts of one row of y.
constexpr int kGvWaves = 8;     // wavefronts of a workgroup: wk along a row times those along the outputs
constexpr int kGvCols = 2048;   // columns of a wavefront's load
constexpr int kGvGroups = 512;  // workgroups that run at once: two a CU
constexpr int kGvTurns = 16;    // most turns of four weight rows of a wavefront: a lane keeps one result
struct GvGrid : Int4Grid {
    int loads, wk, turns;  // loads of a wavefront, wavefronts along a row
    int64_t blocks;        // workgroups along the outputs
};
inline GvGrid gemv_grid(const I4Args &a, int mode) {
    GvGrid g;
    const int all = (a.in + kGvCols - 1) / kGvCols, b = mode == GLU ? 2 : 4;
    g.loads = all > kGvWaves ? 2 : 1;
    g.wk = (all + g.loads - 1) / g.loads;
    const int wr = kGvWaves / g.wk;
    g.waves = wr * g.wk;
    const int64_t turns = ((int64_t)a.rows + wr * b - 1) / (wr * b);  // of a workgroup that did all of a row's outputs
    const int64_t each = (turns * a.T + kGvGroups - 1) / kGvGroups;
    g.turns = (int)(each < 1 ? 1 : each > kGvTurns ? kGvTurns : each);
    g.blocks = (turns + g.turns - 1) / g.turns;
    g.workgroups = g.blocks * a.T;
    return g;
}

// A product's launch: int4_gemv.hip, int4_stream_{f32,bf16,f16}.hip, int4_tile_{f32,bf16,f16}.hip
constexpr int kGvMaxIn = 32768;
int launch_int4_gemv(const I4Args &a, int mode, int x_type, int group, hipStream_t st);
int launch_int4_stream_f32(const I4Args &a, int mode, int group, int form, hipStream_t st);
int launch_int4_stream_bf16(const I4Args &a, int mode, int group, int form, hipStream_t st);
int launch_int4_stream_f16(const I4Args &a, int mode, int group, int form, hipStream_t st);
int launch_int4_tile_f32(const I4Args &a, int mode, int group, int form, hipStream_t st);
int launch_int4_tile_bf16(const I4Args &a, int mode, int group, int form, hipStream_t st);
int launch_int4_tile_f16(const I4Args &a, int mode, int group, int form, hipStream_t st);

}  // namespace k3g
