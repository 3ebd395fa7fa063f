// int4_stream.h -- int4 products whose weights are streamed once: a workgroup
// takes 16 NT rows of activations and 16 RT outputs (of one expert) and splits
// the row's length over its wavefronts, 512 or 256 columns at a time, whose
// codes and scales are all in flight before the first product. The wavefronts' sums meet in
// LDS and are added in wavefront order.
//
// Operand A is the activations (16 tokens), operand B the codes (16 outputs):
// lane l = r + 16 q holds columns 8q .. 8q+7 of token or output r of a block of 32
// columns, and of the result output r of tokens 4q .. 4q+3, so that a group's scale
// and zero are one number a lane. Four consecutive lanes load 64 contiguous bytes
// of a row; a permutation over the wavefront and a transposition of the four
// 16-lane rows bring the dword of (output r, columns 8q ..) of each of the four
// blocks into place.
//
// Where there is an item for each of 16 wavefronts a CU (4096), a wavefront takes one to
// itself, the row's length turn after turn, and they keep loads under way without a
// barrier between them: 1024 rows over 323 experts of 3584 x 3072, gated up-products 0.98 ms against
// 1.26 split, w2 0.49 against 0.88 (3.9 TB/s; a wavefront's loads and products take
// turns); 500 bf16 rows over 64 experts of 1024 x 3584 (6,080 items at most) 58 us against
// 82, fp32 109, 135; 24 fp32 rows over 16 of 2048 x 7168 (2,176) 136 us, split 100. Split, one bf16 token's worth of codes is latency: 7168 -> 3584, 2 tokens 9.5 us,
// 16 tokens 11.4; 32 tokens 14 us. 61 fp32 tokens 3584 -> 7168 24 us: the wavefronts wait
// for loads 44% of the time (two turns' codes, and x from L2), and the vector units, busy
// 53%, have a third of their work in splitting x into bf16 parts.
#pragma once

#include "int4.h"

namespace k3g {

constexpr int kI4Waves = 8;
constexpr int i4_stream_occupancy(int tiles) { return tiles > 2 ? 2 : 4; }  // wavefronts a SIMD
// Steps of 128 columns that are loaded together. Two tiles: what lets 128 registers do, so that a CU holds two
// workgroups. Groups of 32 by four steps, at two wavefronts a SIMD (fp32; bf16 at three), 256 experts of 3584 x 3584 by 1024
// rows 1137 us (bf16 622), so 809 (516), their gated up-products 2169 (1143), 1559 (969); fp32 groups of 64 at three 1062, 773;
// bf16 groups of 64 by two steps 445, by four 426.
constexpr int i4_stream_steps(int tiles, int group) { return tiles > 2 || (group == 32 && tiles > 1) ? 2 : 4; }

template <int XT, int GROUP, int MODE, int RT, int NT>
__global__ __launch_bounds__(kI4Waves * kWave, i4_stream_occupancy(RT * (MODE == GLU ? 2 : 1) * NT)) void int4_stream_kernel(I4Args a) {
    constexpr int NW = MODE == GLU ? 2 : 1, TILES = RT * NW;
    constexpr int STEPS = i4_stream_steps(TILES, GROUP);
    constexpr int SPAN = XT == K3G_F32 || GROUP == 32 ? 1 : 2;             // blocks of 32 columns between two additions
    constexpr int NG = 128 * STEPS / GROUP;                                // groups of a turn
    constexpr int X = XT == K3G_F32 ? 4 : 2;
    extern __shared__ __align__(16) uint8_t lds[];
    const int waves = blockDim.x / kWave;
    float4_t *part = (float4_t *)lds;  // [wave][tile][token tile][lane]
    int32_t *table = (int32_t *)(part + (size_t)waves * TILES * NT * kWave);
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane & 15, q = lane >> 4;   // as the operands have them
    const int lr = lane >> 2, lq = lane & 3;  // as the codes are loaded
    const int psrc = 4 * (4 * r + q);
    const int units = a.in / 32, pitch = a.in / 2;
    Items<MODE, 16 * NT, 16 * RT, I4Args> items(a, table, blockDim.x);
    Item it;
    while (items.next(it)) {
        const int64_t first = (int64_t)it.e * a.rows + it.m0;
        uint32_t at[TILES];  // bytes from the first row's codes
        int srow[TILES];
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
            at[t] = (uint32_t)(min(16 * (t % RT) + lr, a.rows - 1 - it.m0) * pitch);
            srow[t] = min(16 * (t % RT) + r, a.rows - 1 - it.m0) * a.G;
        }
        const uint8_t *xc[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j)
            xc[j] = (const uint8_t *)a.x + X * ((int64_t)source(a, it.p + min(16 * j + r, it.n_tok - 1)) * a.xs + 8 * q);
        float4_t acc[TILES][NT];
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[t][j] = float4_t{0.f, 0.f, 0.f, 0.f};
        const int nf = (it.n_tok + 15) / 16;
        for (int u0 = 4 * STEPS * wave; u0 < units; u0 += 4 * STEPS * waves) {
            uint4 w[STEPS][TILES];
            float s[TILES][NG];
            uint8_t z[TILES][NG];
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
#pragma unroll
                for (int t = 0; t < TILES; ++t)
                    w[i][t] = load16(a.w[t / RT] + first * pitch + (at[t] + 16u * (uint32_t)min(u0 + 4 * i + lq, units - 1)));
            // raw entries of a token tile's span; of the next one while this one is used
            Raw4<XT> x[2][NT][SPAN];
            auto load_x = [&](int k) {
#pragma unroll
                for (int n = 0; n < SPAN; ++n)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        x[k & 1][j][n].load(xc[j] + X * 32 * (int64_t)min(u0 + SPAN * k + n, units - 1));
            };
            load_x(0);
            const int g0 = u0 * 32 / GROUP;
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
                const void *sp = a.s[t / RT];
                const int64_t s0 = first * a.G + srow[t];
                const uint8_t *zp = a.z[t / RT];
#pragma unroll
                for (int g = 0; g < NG; ++g) z[t][g] = 8;
                if (g0 + NG <= a.G) {
                    scales_at<NG>(s[t], sp, a.s_type, s0 + g0);
                    if (zp) __builtin_memcpy(z[t], zp + s0 + g0, NG);
                } else {
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const int64_t i = s0 + min(g0 + g, a.G - 1);
                        s[t][g] = scale_at(sp, a.s_type, i);
                        if (zp) z[t][g] = zp[i];
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                if (u0 + 4 * i < units) {
                    uint32_t d[TILES][4];
#pragma unroll
                    for (int t = 0; t < TILES; ++t) {
                        const uint4 v = to_operand(w[i][t], psrc);
                        d[t][0] = v.x, d[t][1] = v.y, d[t][2] = v.z, d[t][3] = v.w;
                        transpose4(d[t]);
                    }
#pragma unroll
                    for (int b = 0; b < 4; b += SPAN) {
                        if (u0 + 4 * i + b < units) {
                            const int k = (4 * i + b) / SPAN, g = (4 * i + b) * 32 / GROUP;
                            if (k + 1 < 4 * STEPS / SPAN) load_x(k + 1);
                            uint4 codes[TILES][SPAN];
#pragma unroll
                            for (int t = 0; t < TILES; ++t)
#pragma unroll
                                for (int n = 0; n < SPAN; ++n) codes[t][n] = codes8<XT>(d[t][b + n]);
#pragma unroll
                            for (int j = 0; j < NT; ++j) {
                                if (NT == 1 || j < nf) {
                                    Act4<XT> v[SPAN];
                                    float4_t sum = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                                    for (int n = 0; n < SPAN; ++n) {
                                        v[n].take(x[k & 1][j][n]);
                                        sum = v[n].mul(Act4<XT>::ones(), sum);
                                    }
#pragma unroll
                                    for (int t = 0; t < TILES; ++t) {
                                        float4_t p = -(float)z[t][g] * sum;
#pragma unroll
                                        for (int n = 0; n < SPAN; ++n) p = v[n].mul(codes[t][n], p);
#pragma unroll
                                        for (int n = 0; n < 4; ++n) acc[t][j][n] = __builtin_fmaf(s[t][g], p[n], acc[t][j][n]);
                                    }
                                }
                            }
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int j = 0; j < NT; ++j) part[((wave * TILES + t) * NT + j) * kWave + lane] = acc[t][j];
        __syncthreads();
        for (int o = wave; o < RT * NT; o += waves) {  // a wavefront sums an output tile of a token tile
            const int t = o / NT, j = o % NT;
            float4_t v[NW];
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                v[k] = part[((k * RT + t) * NT + j) * kWave + lane];
                for (int u = 1; u < waves; ++u) v[k] += part[((u * TILES + k * RT + t) * NT + j) * kWave + lane];
            }
            const int row = it.m0 + 16 * t + r;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int tok = 16 * j + 4 * q + k;
                const float y = MODE == GLU ? situ(v[0][k], v[NW - 1][k]) : v[0][k];
                if (tok < it.n_tok && row < a.rows) store_out(a.y, a.y_type, (int64_t)(it.p + tok) * a.ys + row, y);
            }
        }
        __syncthreads();  // part is read before the next item writes it
    }
}

// The launch of a tile (weight rows << 16 | tokens).
inline Int4Grid stream_grid(const I4Args &a, int mode, int group, int f) {
    const int units = 4 * i4_stream_steps((f >> 16) / 16, group), turns = (a.in / 32 + units - 1) / units;
    const int64_t items = int4_items(a, mode, (f >> 16) / (mode == GLU ? 2 : 1), f & 0xFFFF);
    const bool alone = items >= 4096;
    const int64_t most = alone ? 4096 : 1024;
    return {items < most ? (items + 7) / 8 * 8 : most, alone ? 1 : turns < kI4Waves ? turns : kI4Waves};
}

template <int XT, int GROUP, int MODE, int RT, int NT>
int launch_int4_stream(const I4Args &a, hipStream_t st) {
    constexpr int TILES = RT * (MODE == GLU ? 2 : 1);
    const Int4Grid g = stream_grid(a, MODE, GROUP, form(16 * TILES, 16 * NT));
    const int waves = g.waves;
    size_t lds = (size_t)waves * TILES * NT * kWave * 16 + (MODE == DENSE ? 0 : 4 * ((size_t)a.E + 1 + 16));
    const void *f = (const void *)int4_stream_kernel<XT, GROUP, MODE, RT, NT>;
    if (lds > 65536 && hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess)
        return K3G_EHIP;
    int4_stream_kernel<XT, GROUP, MODE, RT, NT><<<(unsigned)g.workgroups, waves * kWave, lds, st>>>(a);
    return hipGetLastError() == hipSuccess ? K3G_OK : K3G_EHIP;
}

template <int XT, int GROUP, int MODE>
int launch_int4_stream_form(const I4Args &a, int f, hipStream_t st) {
    constexpr int NW = MODE == GLU ? 2 : 1;
    if constexpr (MODE == DENSE)
        if (f == form(16, 16)) return launch_int4_stream<XT, GROUP, MODE, 1, 1>(a, st);
    if (f == form(32, 16)) return launch_int4_stream<XT, GROUP, MODE, 2 / NW, 1>(a, st);
    if constexpr (MODE == DENSE && XT != K3G_F32)
        if (f == form(64, 64)) return launch_int4_stream<XT, GROUP, MODE, 4, 4>(a, st);
    return launch_int4_stream<XT, GROUP, MODE, 4 / NW, 2>(a, st);
}

template <int XT, int GROUP>
int launch_int4_stream_mode(const I4Args &a, int mode, int f, hipStream_t st) {
    return mode == DENSE     ? launch_int4_stream_form<XT, GROUP, DENSE>(a, f, st)
           : mode == GROUPED ? launch_int4_stream_form<XT, GROUP, GROUPED>(a, f, st)
                             : launch_int4_stream_form<XT, GROUP, GLU>(a, f, st);
}

template <int XT>
int launch_int4_stream_type(const I4Args &a, int mode, int group, int f, hipStream_t st) {
    return group == 32   ? launch_int4_stream_mode<XT, 32>(a, mode, f, st)
           : group == 64 ? launch_int4_stream_mode<XT, 64>(a, mode, f, st)
                         : launch_int4_stream_mode<XT, 128>(a, mode, f, st);
}

}  // namespace k3g
