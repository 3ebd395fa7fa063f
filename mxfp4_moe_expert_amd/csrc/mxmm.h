// mxmm.h -- what the product kernels of microscaled activations share
// (mxmm.hip, mxmm_tile.hip): operands, the step of 128 entries, and the ways out.
#pragma once

#include "mx.h"

namespace k3g {

// One product, or the products of every expert of a bank.
struct MmArgs {
    const uint8_t *a_codes, *a_scales;  // activations
    const uint8_t *w[2], *ws[2];        // weights (GLU: w1, w3), their scales; of expert 0
    int64_t stride;                     // from one expert's tensors to the next
    const int32_t *offsets, *perm;      // grouped: ragged groups, and the source rows (null: straight)
    void *y;                            // dense output
    uint8_t *h_codes, *h_scales;        // GLU output
    int64_t ys;
    int T;        // rows of y (grouped: of all experts)
    int a_rows;   // rows of the activations
    int rows;     // outputs
    int in, G;    // entries, groups of a row
    int E, top_k;
    int y_type, y_vec;  // y_vec: eight outputs lie at 16-byte addresses, and rows are a multiple of 8
    int h_format;
    int odd;  // some row's scale bytes lie off 16-byte addresses, or its groups end inside sixteen
};

// One step of 128 entries. The matrix cores add products of unlike magnitude
// eight at a time in a window narrower than fp32's: one 2^14 below the largest
// is dropped. e2m1 times e2m1 never spans that (1/4 to 36: the eight sums are
// exact), e4m3 times e2m1 does (2^-10 to 2688), and a sum of quantised normals
// then carries an error of 4e-6 of itself. So an e4m3 operand goes in as two:
// the codes below 2 (exponent field under 8; 2^-10 to 11 with a weight) and the
// others (1 to 2688), each inside the window, so every product is exact again
// and the sum is an fp32 one (2e-8 measured). A code left out of a half keeps
// its sign: a signed zero.
template <int AF>
struct Act;  // operand B of a step
template <>
struct Act<K3G_MXFP4> {
    v8i_t v;
    __device__ inline Act(const uint4 &b) : v{(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0} {}
    template <int SW = 0, int SA = 0>  // the bytes of sw and sa that hold the block scales
    __device__ inline float4_t mul(const v8i_t &w, float4_t c, uint32_t sw, uint32_t sa) const {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, v, c, 4, 4, SW, (int)sw, SA, (int)sa);
    }
};
template <>
struct Act<K3G_MXFP8> {
    v8i_t lo, hi;
    __device__ inline Act(const uint4 &b0, const uint4 &b1) {
        const uint32_t d[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t m = d[i] & 0x40404040u;     // the exponent field's top bit
            const uint32_t mask = (m << 1) - (m >> 6);  // 0x7F in each byte that has it
            hi[i] = (int)(d[i] & (mask | 0x80808080u));
            lo[i] = (int)(d[i] & ~mask);
        }
    }
    template <int SW = 0, int SA = 0>
    __device__ inline float4_t mul(const v8i_t &w, float4_t c, uint32_t sw, uint32_t sa) const {
        c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, lo, c, 4, 0, SW, (int)sw, SA, (int)sa);
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, hi, c, 4, 0, SW, (int)sw, SA, (int)sa);
    }
};

__device__ inline uint4 keep4(const uint4 &v, bool keep) {
    const uint32_t k = keep ? ~0u : 0u;
    return make_uint4(v.x & k, v.y & k, v.z & k, v.w & k);
}

enum { DENSE = 0, GROUPED = 1, GLU = 2 };

// Weight rows go to the operand tiles in pairs: of 32 consecutive rows, lane
// r + 16q of the pair's tile k takes row 8 (r/4) + r%4 + 4k, so that a lane's
// four results of tile 0 and four of tile 1 are the eight consecutive rows
// 8q .. 8q+7, one wide store.
__device__ inline int pair_row(int r, int k) { return 8 * (r >> 2) + (r & 3) + 4 * k; }

// Eight consecutive outputs of one token, at element `at` of y; the first `n`
// exist (VEC: all or none).
template <int TYPE, bool VEC>
__device__ inline void store8(void *y, int64_t at, int n, const float4_t &lo, const float4_t &hi) {
    typedef typename Elem<TYPE>::T T;
    T *p = (T *)y + at;
    if (n <= 0) return;
    const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    if constexpr (VEC) {
        store_n<TYPE, 8>((T *)__builtin_assume_aligned(p, 16), v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = Elem<TYPE>::store(v[i]);
    }
}

// f(store) with store = store8 for y's type and alignment (uniform).
template <class F>
__device__ inline void with_store(const MmArgs &a, F f) {
#define K3G_STORE(TYPE, VEC) \
    f([&](int64_t at, int n, const float4_t &lo, const float4_t &hi) { store8<TYPE, VEC>(a.y, at, n, lo, hi); })
    if (a.y_vec) {
        if (a.y_type == K3G_F32)
            K3G_STORE(K3G_F32, true);
        else if (a.y_type == K3G_BF16)
            K3G_STORE(K3G_BF16, true);
        else
            K3G_STORE(K3G_F16, true);
    } else {
        if (a.y_type == K3G_F32)
            K3G_STORE(K3G_F32, false);
        else if (a.y_type == K3G_BF16)
            K3G_STORE(K3G_BF16, false);
        else
            K3G_STORE(K3G_F16, false);
    }
#undef K3G_STORE
}

// A 32-group of h of one token, spread over the four lanes r + 16q: lane q
// holds entries 8q .. 8q+3 (lo) and 8q+4 .. (hi). All lanes of the wavefront
// take part; `live` ones store.
template <int FMT>
__device__ inline void store_h(const MmArgs &a, int64_t token, int group, const float4_t &lo, const float4_t &hi,
                               bool live) {
    const int q = (threadIdx.x & (kWave - 1)) >> 4;
    float v[8];  // (a bit cast of a vector's element would read element 0 whatever the index)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = lo[i];
        v[4 + i] = hi[i];
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    const bool fine = m < kMxNotFinite;
    const int e = fine ? mx_exponent<FMT>(m) : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fine ? v[i] : 0.0f;
    uint32_t w[2];
    mx_codes8<FMT>(v, pow2(e), w);
    if (!live) return;
    const int64_t G = a.rows / kGroup, at = token * G + group;
    if constexpr (FMT == K3G_MXFP4)
        *(uint32_t *)(a.h_codes + at * 16 + 4 * q) = w[0];
    else
        *(uint2 *)(a.h_codes + at * 32 + 8 * q) = make_uint2(w[0], w[1]);
    if (q == 0) a.h_scales[at] = fine ? (uint8_t)(e + 127) : (uint8_t)255;
}

// The expert whose group holds row p, its first row and its end, clipped to
// the rows of y; false where there is none. Two reads: 64 lanes cut the table
// into 64 parts, then the part into its entries.
__device__ inline bool find_group(const MmArgs &a, int p, int &e, int &p0, int &p1) {
    const int lane = threadIdx.x & (kWave - 1);
    const int step = a.E / kWave + 1;  // 64 * step > E
    const int i = min(lane * step, a.E);
    const uint64_t m0 = __ballot(a.offsets[i] <= p);
    if (!m0) return false;
    const int base = min((63 - __builtin_clzll(m0)) * step, a.E);
    const int j = min(base + min(lane, step - 1), a.E);
    const uint64_t m1 = __ballot(a.offsets[j] <= p);
    if (!m1) return false;
    e = __builtin_amdgcn_readfirstlane(min(base + min(63 - __builtin_clzll(m1), step - 1), a.E));
    if (e >= a.E) return false;
    p0 = max(__builtin_amdgcn_readfirstlane(a.offsets[e]), 0);
    p1 = min(__builtin_amdgcn_readfirstlane(a.offsets[e + 1]), a.T);
    return p0 <= p && p < p1;
}

// The activations' row behind row p of y.
__device__ inline int source_row(const MmArgs &a, int p) {
    if (!a.perm) return p;
    const int s = a.perm[p] / a.top_k;
    return min(max(s, 0), a.a_rows - 1);
}

int launch_tile(const MmArgs &a, int mode, int af, hipStream_t st);  // mxmm_tile.hip

}  // namespace k3g
