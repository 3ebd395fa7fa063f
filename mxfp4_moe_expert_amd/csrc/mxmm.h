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

// Four consecutive outputs, where a tile has no partner.
__device__ inline void store4(const MmArgs &a, int64_t at, int n, const float4_t &v) {
    for (int i = 0; i < 4 && i < n; ++i) {
        const float x = i == 0 ? v[0] : i == 1 ? v[1] : i == 2 ? v[2] : v[3];
        if (a.y_type == K3G_F32)
            ((float *)a.y)[at + i] = x;
        else if (a.y_type == K3G_BF16)
            ((__bf16 *)a.y)[at + i] = (__bf16)x;
        else
            ((_Float16 *)a.y)[at + i] = (_Float16)x;
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

// The work of a launch, item by item: BN rows of y (of one expert) by OUT
// outputs. Workgroup b runs on XCD b % 8; each XCD takes a contiguous eighth of
// the items: an expert after another, and in it blocks of outputs by groups of
// four row tiles, so the workgroups of an XCD that run together read 4 row tiles
// and a quarter as many blocks of weights as there are of them.
//
// Grouped: the constructor (all threads of the workgroup) counts the experts'
// row tiles into `table` (LDS, E + 1 numbers of tiles before each expert, and 16
// more for the scan). Groups are clipped to the rows of y; what a table that does
// not ascend gives more than y has rows for is left out.
struct Item {
    int e, p, n_tok, m0;  // expert, first row of y, rows, first output
};
template <int MODE, int BN, int OUT, class Args = MmArgs>
struct Items {
    const Args &a;
    const int32_t *table;
    int n_rb, n_tiles, step, near = 0;  // near: an expert at or before the next item's
    int64_t item, last;

    __device__ inline Items(const Args &a_, int32_t *t, int threads) : a(a_), table(t) {
        n_rb = (a.rows + OUT - 1) / OUT;
        if constexpr (MODE == DENSE) {
            n_tiles = (a.T + BN - 1) / BN;
        } else {
            const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
            int32_t *part = t + a.E + 1;
            const int per = (a.E + threads - 1) / threads, e0 = threadIdx.x * per, e1 = min(e0 + per, a.E);
            auto tiles = [&](int e) {
                const int p0 = max(a.offsets[e], 0), p1 = min(a.offsets[e + 1], a.T);
                return p1 > p0 ? (p1 - p0 + BN - 1) / BN : 0;
            };
            int n = 0;
            for (int e = e0; e < e1; ++e) n += tiles(e);
            int x = n;
            for (int d = 1; d < kWave; d <<= 1) {
                const int y = __shfl_up(x, d);
                if (lane >= d) x += y;
            }
            if (lane == kWave - 1) part[wave] = x;
            __syncthreads();
            int before = x - n;
            for (int w = 0; w < wave; ++w) before += part[w];
            for (int e = e0; e < e1; ++e) {
                t[e] = before;
                before += tiles(e);
            }
            if (e0 < a.E && e1 == a.E) t[a.E] = before;
            __syncthreads();
            n_tiles = min(__builtin_amdgcn_readfirstlane(t[a.E]), a.T / BN + min(a.E, a.T));
        }
        const int64_t n_items = (int64_t)n_tiles * n_rb;
        const int xcd = blockIdx.x % 8;
        step = gridDim.x / 8;
        last = n_items * (xcd + 1) / 8;
        item = n_items * xcd / 8 + blockIdx.x / 8;
    }

    // The next item that has rows (in an ascending table all have); whole wavefronts call it.
    __device__ inline bool next(Item &o) {
        for (; item < last; item += step) {
            int t0 = 0, nt = n_tiles;
            o.e = 0;
            if constexpr (MODE != DENSE) {
                const int tile = (int)(item / n_rb), lane = threadIdx.x & (kWave - 1);
                // experts after `near` whose first tile is at most this one, 64 at a time
                for (;;) {
                    const int i = near + 1 + lane;
                    const int n = __popcll(__ballot(i < a.E && table[min(i, a.E)] <= tile));
                    near += n;
                    if (n < kWave) break;
                }
                near = __builtin_amdgcn_readfirstlane(near);
                o.e = near;
                t0 = __builtin_amdgcn_readfirstlane(table[near]);
                nt = __builtin_amdgcn_readfirstlane(table[near + 1]) - t0;
            }
            const int64_t in_expert = item - (int64_t)t0 * n_rb;
            const int group = (int)(in_expert / (4 * n_rb)), wide = min(4, nt - group * 4);
            if (wide < 1) continue;
            const int in_group = (int)(in_expert - (int64_t)group * 4 * n_rb);
            o.m0 = in_group / wide * OUT;  // (a table whose tiles pass 32 bits may make it negative)
            o.p = (group * 4 + in_group % wide) * BN;
            int end = a.T;
            if constexpr (MODE != DENSE) {
                o.p += max(__builtin_amdgcn_readfirstlane(a.offsets[o.e]), 0);
                end = min(__builtin_amdgcn_readfirstlane(a.offsets[o.e + 1]), a.T);
            }
            o.n_tok = min(BN, end - o.p);
            if (o.p < 0 || o.n_tok < 1 || o.m0 < 0 || o.m0 >= a.rows) continue;
            item += step;
            return true;
        }
        return false;
    }
};

// The kernel that a product runs on: outputs << 16 | tokens of its weight rows' tile.
constexpr int form(int rows, int tokens) { return rows << 16 | tokens; }

// mxmm_tile.hip: the tile of a product (0: dense, with too few of the smallest to fill the chip), and its launch
int tile_form(const MmArgs &a, int mode, int af);
int launch_tile(const MmArgs &a, int mode, int af, int tile, hipStream_t st);

}  // namespace k3g
