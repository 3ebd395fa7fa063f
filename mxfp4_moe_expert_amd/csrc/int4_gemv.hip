// int4_gemv.hip -- products of single rows with int4 weights, on the vector units:
// one token, or the rows of a few tokens' experts.
//
// y[r] = sum over the row's 32-column pieces of s (sum n x - z sum x): a lane holds
// 32 columns of x in fp32, and their sum, for each 2048 columns of its wavefront's
// share, and takes 16 bytes of codes of each weight row. A piece lies in one group, so
// s and z are one number a lane. gfx950's scaled convert turns two codes at a time
// into fp32 (see int4.h: a code is n 2^-9 in e4m3), 15 instructions for eight weights
// with their multiply-adds; the wavefront's sum over its lanes ends a weight row.
// A token's 16 experts of 3584 x 3072, groups of 32: gated up-products 41 us (5.1 TB/s), w2 25
// (4.2: 96 pieces a row leave a quarter of two wavefronts' lanes empty); one token 7168
// -> 3584 8 us, latency.
#include "int4.h"

namespace k3g {

struct GvArgs {
    I4Args a;
    int wk;      // wavefronts along a row
    int turns;   // of a wavefront, four weight rows each
    int blocks;  // workgroups along the outputs
    int shift;   // log2 of a group's columns, less 5
    int x_type;
};

// The expert of row p: the last whose group starts at or before it. -1 where p is in no group.
__device__ inline int expert_of(const I4Args &a, int p) {
    const int lane = threadIdx.x & (kWave - 1);
    int e = 0;
    for (int i = 0; i < a.E; i += 8 * kWave) {  // eight loads under way at once
        int ends[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) ends[k] = a.offsets[min(i + k * kWave + lane, a.E - 1) + 1];
#pragma unroll
        for (int k = 0; k < 8; ++k) e += __popcll(__ballot(i + k * kWave + lane < a.E && ends[k] <= p));
    }
    e = __builtin_amdgcn_readfirstlane(e);
    return e < a.E && a.offsets[e] <= p && p < a.offsets[e + 1] ? e : -1;
}

// One piece's dot product of codes and x.
__device__ inline float dot32(const uint4 &w, const float *x) {
    const uint32_t d[4] = {w.x, w.y, w.z, w.w};
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t lo = d[k] & 0x0F0F0F0Fu, hi = (d[k] >> 4) & 0x0F0F0F0Fu;
        const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 512.0f, false);
        const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 512.0f, true);
        const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 512.0f, false);
        const auto e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 512.0f, true);
        s0 = __builtin_fmaf(a[0], x[8 * k], s0);
        s1 = __builtin_fmaf(c[0], x[8 * k + 1], s1);
        s0 = __builtin_fmaf(a[1], x[8 * k + 2], s0);
        s1 = __builtin_fmaf(c[1], x[8 * k + 3], s1);
        s0 = __builtin_fmaf(b[0], x[8 * k + 4], s0);
        s1 = __builtin_fmaf(e[0], x[8 * k + 5], s1);
        s0 = __builtin_fmaf(b[1], x[8 * k + 6], s0);
        s1 = __builtin_fmaf(e[1], x[8 * k + 7], s1);
    }
    return s0 + s1;
}

// NW weights (2: the gated up-product), CH loads of 2048 columns a wavefront, S32: fp32 scales.
template <int NW, int CH, bool S32>
__global__ __launch_bounds__(kGvWaves * kWave) void int4_gemv_kernel(GvArgs g) {
    const I4Args &a = g.a;
    constexpr int B = 4 / NW;  // outputs of a turn: four weight rows
    extern __shared__ __align__(16) float xs[];  // x, four columns of every lane side by side; then the parts of a row
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wr = (blockDim.x / kWave) / g.wk, kpart = wave % g.wk, rpart = wave / g.wk;
    const int p = blockIdx.x / g.blocks, block = blockIdx.x % g.blocks;
    int e = 0;
    if (a.offsets) {
        e = expert_of(a, p);
        if (e < 0) return;  // (the whole workgroup)
    }
    const int r0 = (block * wr + rpart) * g.turns * B;  // the wavefront's first output
    const int c0 = kpart * CH * kGvCols + 32 * lane;
    const int pitch = a.in / 2;
    const int64_t row0 = (int64_t)e * a.rows;
    struct Rows {
        uint4 w[4][CH];
        uint32_t s[4][CH], z[4][CH];
    };
    // the codes, scales and zeros of outputs r .. r + B - 1 (past the last: of the last); past the row's end: of its last piece
    auto load = [&](Rows &o, int r) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = i / B;
            const int64_t row = row0 + min(r + i % B, a.rows - 1);
            const uint8_t *wp = a.w[k] + row * pitch;
            const int64_t sp = row * a.G;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const uint32_t col = (uint32_t)min(c0 + c * kGvCols, a.in - 32), grp = (col >> 5) >> g.shift;
                o.w[i][c] = load16(wp + col / 2);
                o.s[i][c] = S32 ? ((const uint32_t *)a.s[k] + sp)[grp] : ((const uint16_t *)a.s[k] + sp)[grp];
                o.z[i][c] = a.z[k] ? (a.z[k] + sp)[grp] : 8u;
            }
        }
    };
    Rows cur;
    load(cur, r0);
    {
        // x into LDS: piece c of lane l at ((c * 8 + k) * 64 + l) * 4, k counting its fours
        const int64_t at = (int64_t)(a.perm ? source(a, p) : p) * a.xs;
        const int n_lanes = blockDim.x;
        const int fours = g.wk * CH * kGvCols / 4;
        for (int i = tid; i < fours; i += n_lanes) {
            const int col = 4 * i;
            float v[4] = {};
            if (col < a.in) {
                if (g.x_type == K3G_F32)
                    load_n<K3G_F32, 4>(v, (const float *)a.x + at + col);
                else if (g.x_type == K3G_BF16)
                    load_n<K3G_BF16, 4>(v, (const __bf16 *)a.x + at + col);
                else
                    load_n<K3G_F16, 4>(v, (const _Float16 *)a.x + at + col);
            }
            const int piece = i / 8;  // of 32 columns
            *(float4 *)(xs + (((piece / kWave) * 8 + i % 8) * kWave + piece % kWave) * 4) = make_float4(v[0], v[1], v[2], v[3]);
        }
    }
    __syncthreads();
    float x[CH][32], sum[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        sum[c] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float4 v = *(const float4 *)(xs + (((kpart * CH + c) * 8 + k) * kWave + lane) * 4);
            x[c][4 * k] = v.x, x[c][4 * k + 1] = v.y, x[c][4 * k + 2] = v.z, x[c][4 * k + 3] = v.w;
            sum[c] += (v.x + v.y) + (v.z + v.w);
        }
    }
    float res = 0.f;  // lane 4 t + i: value i of turn t
    auto use = [&](const Rows &o, int turn) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[i] = 0.f;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const float s = S32                       ? __builtin_bit_cast(float, o.s[i][c])
                                : a.s_type == K3G_BF16 ? __builtin_bit_cast(float, o.s[i][c] << 16)
                                                          : (float)__builtin_bit_cast(_Float16, (uint16_t)o.s[i][c]);
                const float d = __builtin_fmaf(-(float)o.z[i][c], sum[c], dot32(o.w[i][c], x[c]));
                // a lane past the row's end has no columns: its scale may be anything
                if (c0 + c * kGvCols < a.in) y[i] = __builtin_fmaf(s, d, y[i]);
            }
        }
        const float v = wave_sum4(y, lane);
        if ((lane >> 2) == turn) res = v;
    };
    for (int t = 0; t < g.turns; t += 2) {
        Rows next;
        load(next, r0 + (t + 1) * B);
        use(cur, t);
        if (t + 2 < g.turns) load(cur, r0 + (t + 2) * B);
        if (t + 1 < g.turns) use(next, t + 1);
    }
    if (g.wk > 1) {
        __syncthreads();  // x has been read
        xs[wave * kWave + lane] = res;
        __syncthreads();
        if (kpart != 0) return;
        for (int u = 1; u < g.wk; ++u) res += xs[(wave + u) * kWave + lane];
    }
    const float other = dpp<0x4E>(res);  // GLU: the up-product beside its gate, two lanes on
    const int turn = lane >> 2, i = lane & 3, row = r0 + turn * B + i % B;
    if (turn < g.turns && i < B && row < a.rows)
        store_out(a.y, a.y_type, (int64_t)p * a.ys + row, NW == 2 ? situ(res, other) : res);
}

int launch_int4_gemv(const I4Args &a, int mode, int x_type, int group, hipStream_t st) {
    GvArgs g = {};
    g.a = a;
    g.x_type = x_type;
    g.shift = group == 32 ? 0 : group == 64 ? 1 : 2;
    const GvGrid q = gemv_grid(a, mode);
    const int ch = q.loads, waves = q.waves;
    g.wk = q.wk, g.turns = q.turns, g.blocks = (int)q.blocks;
    const size_t lds = sizeof(float) * (size_t)g.wk * ch * kGvCols;
    const bool s32 = a.s_type == K3G_F32;
    const unsigned grid = (unsigned)q.workgroups;
#define K3G_GV(NW, CH, S32)                                                                                            \
    do {                                                                                                               \
        const void *f = (const void *)int4_gemv_kernel<NW, CH, S32>;                                                   \
        if (lds > 65536 && hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess) \
            return K3G_EHIP;                                                                                           \
        int4_gemv_kernel<NW, CH, S32><<<grid, waves * kWave, lds, st>>>(g);                                            \
    } while (0)
    if (mode == GLU) {
        if (ch == 2)
            if (s32) K3G_GV(2, 2, true); else K3G_GV(2, 2, false);
        else
            if (s32) K3G_GV(2, 1, true); else K3G_GV(2, 1, false);
    } else {
        if (ch == 2)
            if (s32) K3G_GV(1, 2, true); else K3G_GV(1, 2, false);
        else
            if (s32) K3G_GV(1, 1, true); else K3G_GV(1, 1, false);
    }
#undef K3G_GV
    return hipGetLastError() == hipSuccess ? K3G_OK : K3G_EHIP;
}

}  // namespace k3g
