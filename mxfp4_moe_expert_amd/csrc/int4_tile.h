// int4_tile.h -- int4 products of many tokens: a workgroup takes 16 NJ rows of
// activations and 64 outputs a wavefront (GLU: 32 of each weight), four
// wavefronts. The activations come through LDS in steps of 128 columns, two
// steps' places; each wavefront loads its own codes a step ahead and makes operands
// of them in registers, once for all of the tile's tokens.
//
// A step of 128 columns is 128 matrix and about 650 vector instructions a wavefront
// at groups of 64: 304 make operands of 8192 codes, 256 apply the groups' scales to
// the partial sums. 4096 tokens 7168 -> 6144 386 us, 0.93 PFLOP/s; 65536 rows over 536
// experts of 3584 x 3072 2.8 ms, their gated up-products 6.1. Matrix cores are busy
// 36% of that time and the vector units 46%: the two hardly overlap, since the operands of a half
// step are made before its first product and each two token tiles begin with a branch and a
// wait for their rows. Two workgroups a CU take each other's waits: one alone needs 0.7 of
// the time of two.
//
// bf16 and fp16 rows off 16-byte addresses come through registers, which the compiler keeps in
// scratch memory: a step waits for the next one's rows (4096 tokens 7168 -> 3584 447 us; fp32's
// tile for rows on such addresses 446, the one by DMA 256).
#pragma once

#include "int4.h"

namespace k3g {

// Eight codes less their zero as bf16 or fp16, in order: z4 is the zero in each byte.
// The subtraction is on whole bytes (of n + 128, so that none borrows from the
// next), the conversion one instruction an entry that reads a byte with its sign, and
// the fp32 result's upper half is the bf16. 19 instructions; against codes8 it spares
// the product with ones and the multiplication of every partial sum, which a
// tile of this many tokens would spend more on. Zeros up to 128: a larger one borrows.
template <int XT>
__device__ inline uint4 codes8(uint32_t d, uint32_t z4) {
    uint32_t lo = ((d & 0x0F0F0F0Fu) | 0x80808080u) - z4, hi = (((d >> 4) & 0x0F0F0F0Fu) | 0x80808080u) - z4;
    lo ^= 0x80808080u, hi ^= 0x80808080u;
    uint32_t v[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const float e = (float)(int)(int8_t)(lo >> (8 * b)), o = (float)(int)(int8_t)(hi >> (8 * b));
        if constexpr (XT == K3G_F16)
            v[b] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(e, o));
        else
            v[b] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, o), __builtin_bit_cast(uint32_t, e), 0x07060302u);
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}
// The same less a zero of any byte, subtracted in fp32: eight instructions more (down to -255, so exact in bf16 too).
// Taken for the turns of a wavefront that meet a zero of 128 or more; that branch costs the others 1 to 2% (4096 tokens
// 7168 -> 6144, groups of 64, 391 us without it, 397 with).
template <int XT>
__device__ inline uint4 codes8_any(uint32_t d, float z) {
    uint32_t v[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const float e = (float)(d >> (8 * b) & 0xFu) - z, o = (float)(d >> (8 * b + 4) & 0xFu) - z;
        if constexpr (XT == K3G_F16)
            v[b] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(e, o));
        else
            v[b] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, o), __builtin_bit_cast(uint32_t, e), 0x07060302u);
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// Global -> LDS without registers, 16 bytes a lane, each from its own address, to `lds` + 16 * lane.
__device__ inline void dma16_from(const void *p, uint32_t lds) {
    lds = __builtin_amdgcn_readfirstlane(lds);
    __asm__ volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(p), "s"(lds) : "m0", "memory");
}

template <int XT, int NJ>
constexpr int i4_step_bytes() { return (XT == K3G_F32 ? 3 : 1) * 16 * NJ * 256; }  // a step of the activations in LDS
template <int GROUP>
constexpr int i4_scale_bytes() { return 256 * (256 / GROUP) * 5; }  // 256 columns' scales and zeros of 256 weight rows

template <int XT, int GROUP, int MODE, int NJ, bool DMA>
__global__ __launch_bounds__(256, 2) void int4_tile_kernel(I4Args a) {
    constexpr int NW = MODE == GLU ? 2 : 1, TILES = 4, RT = TILES / NW, OUT = 4 * 16 * RT;
    constexpr int SPAN = GROUP < 64 ? 1 : 2;  // blocks of 32 columns between two additions to the accumulators
    constexpr int NG = 256 / GROUP;           // groups of a turn of two steps
    constexpr int PLANES = XT == K3G_F32 ? 3 : 1, TOK = 16 * NJ, STEP = i4_step_bytes<XT, NJ>();
    constexpr int X = XT == K3G_F32 ? 4 : 2, PARTS = TOK * 16 / 256;  // chunks of eight columns that a thread stages
    static_assert(!DMA || PLANES == 1, "fp32 rows are split on the way");
    extern __shared__ __align__(16) uint8_t lds[];
    uint8_t *stage = lds;  // [2][plane][token][16 chunks of 8 columns, chunk c at c ^ (token % 16)]
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    float *scales = (float *)(lds + 2 * STEP) + wave * NG * kWave;                      // [group][weight row] of the wavefront
    uint8_t *zeros = lds + 2 * STEP + 4 * NG * 256 + wave * NG * kWave;                 // the same
    const uint8_t **src = (const uint8_t **)(lds + 2 * STEP + i4_scale_bytes<GROUP>());  // the tokens' rows
    int32_t *table = (int32_t *)(src + TOK);
    const int r = lane & 15, q = lane >> 4, lr = lane >> 2, lq = lane & 3, psrc = 4 * (4 * r + q);
    const int units = a.in / 32, pitch = a.in / 2, S = (units + 3) / 4;
    Items<MODE, TOK, OUT, I4Args> items(a, table, 256);
    Item it;
    while (items.next(it)) {
        if (tid < TOK)
            src[tid] = (const uint8_t *)a.x + X * ((int64_t)source(a, it.p + min(tid, it.n_tok - 1)) * a.xs);
        // the wavefront's outputs from m on; its weight rows are 16 of tile 0, then of tile 1 ..
        const int m = it.m0 + wave * 16 * RT, left = a.rows - 1 - m;
        const int64_t first = (int64_t)it.e * a.rows + min(m, a.rows - 1);
        uint32_t at[TILES];
#pragma unroll
        for (int t = 0; t < TILES; ++t) at[t] = (uint32_t)(max(min(16 * (t % RT) + lr, left), 0) * pitch);
        const uint8_t *w0 = a.w[0] + first * pitch, *w1 = a.w[NW - 1] + first * pitch;
        const int own = lane / (16 * RT);  // the weight whose scales this lane brings, and its row's groups from the first row's
        const int own_at = max(min(lane % (16 * RT), left), 0) * a.G;
        const int nf = (it.n_tok + 15) / 16;
        float4_t acc[TILES][NJ];
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[t][j] = float4_t{0.f, 0.f, 0.f, 0.f};
        uint4 w[TILES];
        Raw4<XT> xr[DMA ? 1 : PARTS];
        Scales4<NG> s;
        int s_shift = 0;  // its first groups that belong to the turn before
        auto load_w = [&](int step) {
            const uint32_t c = 16u * (uint32_t)min(4 * step + lq, units - 1);
#pragma unroll
            for (int t = 0; t < TILES; ++t) w[t] = load16((t < RT ? w0 : w1) + (at[t] + c));
        };
        // The bases are made anew each time (the empty assembly hides them): kept, the lanes' addresses would not fit the
        // registers, and a reload from scratch memory waits for every load under way. (Up to 16 registers that are
        // spilled all the same are loaded again between items, not in the loop over steps.)
        auto load_s = [&](int turn) {
            const int g0 = turn * NG, from = max(min(g0, a.G - NG), 0), size = a.s_type == K3G_F32 ? 4 : 2;
            s_shift = g0 - from;
            global_t sb[NW], zb[NW];
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                sb[k] = (global_t)a.s[k] + size * (first * a.G + from);
                zb[k] = (a.z[k] ? (global_t)a.z[k] : (global_t)a.s[k]) + (first * a.G + from);
                __asm__ volatile("" : "+s"(sb[k]), "+s"(zb[k]));
            }
            s.load((own ? sb[NW - 1] : sb[0]) + size * own_at, a.s_type, (own ? zb[NW - 1] : zb[0]) + own_at);
        };
        const bool given = a.z[NW == 2 ? own : 0];
        bool far = false;  // a zero of the turn's groups is 128 or more
        auto put_s = [&]() {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < (NG + 3) / 4; ++i) top |= s.zero[i];
            far = __ballot(given && (top & 0x80808080u)) != 0;
#pragma unroll
            for (int g = 0; g < NG; ++g)
                if (g >= s_shift) {
                    scales[(g - s_shift) * kWave + lane] = s.scale(g, a.s_type);
                    zeros[(g - s_shift) * kWave + lane] = given ? (uint8_t)s.zero_at(g) : 8;
                }
        };
        const bool short_row = a.G < NG;  // its groups go to LDS here, one by one
        if (short_row) {
            const int64_t at0 = first * a.G + own_at;
            for (int g = 0; g < a.G; ++g) {
                const uint8_t z = given ? a.z[NW == 2 ? own : 0][at0 + g] : 8;
                scales[g * kWave + lane] = scale_at(a.s[NW == 2 ? own : 0], a.s_type, at0 + g);
                zeros[g * kWave + lane] = z;
                far = far || __ballot(z > 127) != 0;
            }
        }
        // chunk tid % 16 of every 16th row from tid / 16 on
        auto load_x = [&](int step) {
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
                const int tok = tid / 16 + 16 * i, c = (tid & 15) ^ (tok & 15);
                const uint8_t *p = src[tok] + X * 8 * (int64_t)min(16 * step + c, 4 * units - 1);
                if constexpr (DMA)
                    dma16_from(p, lds_addr(stage + (step & 1) * STEP + (4 * wave + 16 * i) * 256));
                else
                    xr[i].load(p);
            }
        };
        auto put_x = [&](int step) {
            if constexpr (!DMA) {
#pragma unroll
                for (int i = 0; i < PARTS; ++i) {
                    uint8_t *to = stage + (step & 1) * STEP + 16 * tid + 16 * 256 * i;
                    if constexpr (XT == K3G_F32) {
                        Act4<XT> v;
                        v.take(xr[i]);
#pragma unroll
                        for (int k = 0; k < 3; ++k) *(uint4 *)(to + k * TOK * 256) = v.part[k];
                    } else {
                        *(uint4 *)to = xr[i].v;
                    }
                }
            }
        };
        __syncthreads();  // src; and the stages are free
        if (!short_row) load_s(0);
        load_w(0);
        load_x(0);
        for (int step = 0; step < S; ++step) {
            put_x(step);
            // Everything that was asked for a step ago is there (a wait that the compiler knows of: else it would wait again,
            // for the loads that follow, where it first uses a register that it had reloaded before the loop).
            __builtin_amdgcn_s_waitcnt(0x0F70);
            __asm__ volatile("" : : : "memory");
            if (step % 2 == 0 && !short_row) put_s();
            // this step's codes in operand order, before the registers are loaded again
            uint32_t d[TILES][4];
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
                const uint4 v = to_operand(w[t], psrc);
                d[t][0] = v.x, d[t][1] = v.y, d[t][2] = v.z, d[t][3] = v.w;
                transpose4(d[t]);
            }
            __syncthreads();
            if (step + 1 < S) {
                load_x(step + 1);
                if (step % 2 == 0 && step + 2 < S) load_s(step / 2 + 1);
            }
            const uint8_t *x0 = stage + (step & 1) * STEP + r * 256;
#pragma unroll
            for (int b = 0; b < 4; b += SPAN) {
                if (4 * step + b < units) {
                    const int g = (128 * (step & 1) + 32 * b) / GROUP;
                    Act4<XT> x[2][SPAN];
                    auto read_x = [&](int j) {
#pragma unroll
                        for (int k = 0; k < SPAN; ++k) {
                            const uint8_t *xp = x0 + j * 16 * 256 + 16 * ((4 * (b + k) + q) ^ r);
                            if constexpr (XT == K3G_F32) {
#pragma unroll
                                for (int n = 0; n < 3; ++n) x[j & 1][k].part[n] = *(const uint4 *)(xp + n * TOK * 256);
                            } else {
                                x[j & 1][k].v = *(const uint4 *)xp;
                            }
                        }
                    };
                    uint4 codes[TILES][SPAN];
                    float sc[TILES];
                    uint32_t zero[TILES];
#pragma unroll
                    for (int t = 0; t < TILES; ++t) {
                        sc[t] = scales[g * kWave + 16 * t + r];
                        zero[t] = zeros[g * kWave + 16 * t + r];
                    }
                    if (__builtin_expect(far, 0)) {  // (around all tiles: a choice for each makes the call 10% longer)
#pragma unroll
                        for (int t = 0; t < TILES; ++t)
#pragma unroll
                            for (int k = 0; k < SPAN; ++k) codes[t][k] = codes8_any<XT>(d[t][b + k], (float)zero[t]);
                    } else {
#pragma unroll
                        for (int t = 0; t < TILES; ++t)
#pragma unroll
                            for (int k = 0; k < SPAN; ++k) codes[t][k] = codes8<XT>(d[t][b + k], zero[t] * 0x01010101u);
                    }
                    // two token tiles at a time: the products of the second run as the sums of the first are added
#pragma unroll
                    for (int j0 = 0; j0 < NJ; j0 += 2) {
                        if (j0 < nf) {
                            float4_t p[2][TILES];
#pragma unroll
                            for (int h = 0; h < 2; ++h) read_x(j0 + h);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
#pragma unroll
                                for (int t = 0; t < TILES; ++t)
                                    p[h][t] = x[h][0].mul(codes[t][0], float4_t{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                                for (int k = 1; k < SPAN; ++k)
#pragma unroll
                                    for (int t = 0; t < TILES; ++t) p[h][t] = x[h][k].mul(codes[t][k], p[h][t]);
                            }
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int t = 0; t < TILES; ++t)
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        acc[t][j0 + h][i] = __builtin_fmaf(sc[t], p[h][t][i], acc[t][j0 + h][i]);
                        }
                    }
                }
                if (b == 4 - 2 * SPAN && step + 1 < S) load_w(step + 1);
            }
        }
        // The way out: 16 tokens at a time through the wavefront's own part of the stages, so that four lanes write a
        // token's outputs side by side (4096 tokens of 512 -> 512: 27 us with two bytes a lane, so 19).
        __syncthreads();  // the stages have been read
        constexpr int PITCH = 16 * RT + 4;  // 4 more: the four lane rows write to different banks
        float *out = (float *)stage + wave * 16 * PITCH;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            if (j < nf) {
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        out[(4 * q + i) * PITCH + 16 * t + r] =
                            MODE == GLU ? situ(acc[t][j][i], acc[TILES - RT + t][j][i]) : acc[t][j][i];
                const int tok = 16 * j + lr, row = m + 4 * RT * lq;
                float v[4 * RT];
                wave_lds_order();
                __builtin_memcpy(v, out + lr * PITCH + 4 * RT * lq, sizeof v);
                wave_lds_order();  // the next 16 tokens' results go to the same place
                if (tok < it.n_tok) store_outs<4 * RT>(a.y, a.y_type, (int64_t)(it.p + tok) * a.ys + row, a.rows - row, v);
            }
        }
    }
}

// The launch of a tile (weight rows << 16 | tokens).
inline Int4Grid tile_grid(const I4Args &a, int mode, int f) {
    const int64_t items = int4_items(a, mode, (f >> 16) / (mode == GLU ? 2 : 1), f & 0xFFFF), most = 512;
    return {items < most ? (items + 7) / 8 * 8 : most, 4};
}

template <int XT, int GROUP, int MODE, int NJ, bool DMA>
int launch_int4_tile(const I4Args &a, hipStream_t st) {
    constexpr int TOK = 16 * NJ;
    const Int4Grid g = tile_grid(a, MODE, form(256, TOK));
    const size_t lds = 2 * (size_t)i4_step_bytes<XT, NJ>() + i4_scale_bytes<GROUP>() + 8 * TOK +
                       (MODE == DENSE ? 0 : 4 * ((size_t)a.E + 1 + 16));
    const void *f = (const void *)int4_tile_kernel<XT, GROUP, MODE, NJ, DMA>;
    if (lds > 65536 && hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess)
        return K3G_EHIP;
    int4_tile_kernel<XT, GROUP, MODE, NJ, DMA><<<(unsigned)g.workgroups, 256, lds, st>>>(a);
    return hipGetLastError() == hipSuccess ? K3G_OK : K3G_EHIP;
}

template <int XT, int GROUP, int MODE>
int launch_int4_tile_form(const I4Args &a, int f, hipStream_t st) {
    if constexpr (XT != K3G_F32)
        if (f == form(256, 128)) return launch_int4_tile<XT, GROUP, MODE, 8, true>(a, st);
    return launch_int4_tile<XT, GROUP, MODE, 4, false>(a, st);
}

template <int XT, int GROUP>
int launch_int4_tile_mode(const I4Args &a, int mode, int f, hipStream_t st) {
    return mode == DENSE     ? launch_int4_tile_form<XT, GROUP, DENSE>(a, f, st)
           : mode == GROUPED ? launch_int4_tile_form<XT, GROUP, GROUPED>(a, f, st)
                             : launch_int4_tile_form<XT, GROUP, GLU>(a, f, st);
}

template <int XT>
int launch_int4_tile_type(const I4Args &a, int mode, int group, int f, hipStream_t st) {
    return group == 32   ? launch_int4_tile_mode<XT, 32>(a, mode, f, st)
           : group == 64 ? launch_int4_tile_mode<XT, 64>(a, mode, f, st)
                         : launch_int4_tile_mode<XT, 128>(a, mode, f, st);
}

}  // namespace k3g
