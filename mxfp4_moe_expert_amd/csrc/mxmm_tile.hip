// mxmm_tile.hip -- the products of microscaled activations with MXFP4 weights
// for many tokens: tiles of BM weight rows x BN tokens, both operands staged
// through LDS in steps of 128 entries.
//
// A stage holds 64 bytes of each weight row and 64 (e2m1) or 128 (e4m3) of each
// token, written by LDS DMA: four (eight) consecutive lanes take one row's
// contiguous bytes, 16-byte chunk c of row i at place c ^ (i/2 % 4) (c ^ i % 8),
// so that the operand reads (16 bytes of 16 rows a quarter wavefront) meet no
// bank twice. The rows' scale bytes come as aligned dwords the same way. The
// wavefront that loaded a row turns its four bytes of a stage into operand order
// (one dword a lane for four operand tiles: the instruction picks the byte),
// and where one is 255 or past the row's end it zeroes the group's codes in LDS
// and makes the scale finite.
//
// Pipeline, one barrier a stage, in the middle of its products:
//   products of stage s, first half | wait for the own rows of s+1, prepare them
//   barrier: s+1 is whole, and everyone has read s
//   DMA of stage s+NB into s's place | operands of s+1 into registers
//   products of stage s, second half
// so the matrix cores have work across the barrier, and NB - 1 stages are in
// flight or about to be read.
#include "mxmm.h"

namespace k3g {

template <int AF, int MODE_, int WR_, int WC_, int FM_, int FN_, int NB_>
struct Tile {
    static constexpr int MODE = MODE_, WR = WR_, WC = WC_, FM = FM_, FN = FN_, NB = NB_;
    static constexpr int NW = WR * WC, THREADS = NW * kWave;
    static constexpr int BM = WR * FM * 16, BN = WC * FN * 16;
    static constexpr int OUT = MODE == GLU ? BM / 2 : BM;  // outputs of a tile
    static constexpr int AB = AF == K3G_MXFP4 ? 64 : 128;  // bytes of a token a stage
    static constexpr int MW = BM / NW, MA = BN / NW;       // rows that a wavefront loads
    static constexpr int DW = MW / 16, DA = MA * AB / 1024;  // DMA instructions of 1 KB
    static constexpr int SW = (MW + 63) / 64, SA = (MA + 63) / 64;  // scale DMA instructions (one dword a row)
    static_assert(MW % 16 == 0 && MA % 16 == 0 && MW <= 64 && MA <= 64, "rows per wavefront");
    static_assert((FM % 4 == 0 || 4 % FM == 0) && (FN % 4 == 0 || 4 % FN == 0), "scale dwords");
    static_assert(MODE != GLU || FM % 4 == 0, "a wavefront owns whole 32-groups of h");
    static constexpr int V1 = DW + DA + 2;  // loads in flight per stage, scales in aligned dwords
    static constexpr int V2 = V1 + 2;       // scales that straddle dwords: two a row
    // LDS: data and raw scales per stage, operand-order scales (two stages)
    static constexpr int DATA = BM * 64 + BN * AB, RAW = (BM + BN) * 8, STAGE = DATA + RAW;
    static constexpr int SCALES = (BM + BN) * 4;
    static constexpr int TABLE = NB * STAGE + 2 * SCALES;  // then the grouped form's table
    static constexpr int lds(int E) { return TABLE + (MODE == DENSE ? 0 : 4 * (E + 1) + 64); }
};

__device__ inline void stage_barrier() {
    __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
}

// global -> LDS without registers as dma4, each lane from an address of its own
__device__ inline void dma4_at(const void *p, uint32_t lds) {
    lds = __builtin_amdgcn_readfirstlane(lds);
    __asm__ volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dword %0, off" : : "v"(p), "s"(lds) : "m0");
}

// Waits until at most K stages' loads are in flight, of the `left` stages that
// follow the one waited for (fewer near the end of the row: all of them).
template <int V1, int V2, int K>
__device__ inline void wait_stages(bool two, int left) {
    if (left >= K) {
        if (two)
            wait_vm<K * V2 < 64 ? K * V2 : 63>();
        else
            wait_vm<K * V1>();
    } else {
        wait_vm<0>();
    }
}

// Operand tiles i0 .. i1-1 of the weights with every token tile. The loops are
// unrolled by template: the byte that an instruction takes from a scale dword
// is part of the instruction.
template <int... I>
struct Seq {};
template <int N, int... I>
struct MakeSeq : MakeSeq<N - 1, N - 1, I...> {};
template <int... I>
struct MakeSeq<0, I...> {
    typedef Seq<I...> type;
};

template <int AF, class C, int J, int I0, int... I>
__device__ inline void mul_column(const uint4 *w, const uint4 *t, const uint32_t *sw, uint32_t st,
                                  float4_t (*acc)[C::FN], Seq<I...>) {
    const Act<AF> b = [&] {
        if constexpr (AF == K3G_MXFP4)
            return Act<AF>(t[0]);
        else
            return Act<AF>(t[0], t[1]);
    }();
    ((acc[I0 + I][J] = b.template mul<(I0 + I) & 3, J & 3>(
          v8i_t{(int)w[I0 + I].x, (int)w[I0 + I].y, (int)w[I0 + I].z, (int)w[I0 + I].w, 0, 0, 0, 0}, acc[I0 + I][J],
          sw[(I0 + I) / 4], st)),
     ...);
}
template <int AF, class C, int I0, int N, int... J>
__device__ inline void mul_tiles(const uint4 *w, const uint4 (*t)[C::AB / 64], const uint32_t *sw, const uint32_t *st,
                                 float4_t (*acc)[C::FN], Seq<J...>) {
    (mul_column<AF, C, J, I0>(w, t[J], sw, st[J / 4], acc, typename MakeSeq<N>::type{}), ...);
}

template <int H>
struct Half {
    static constexpr int value = H;
};

template <int AF, class C>
__global__ __launch_bounds__(C::THREADS) void mx_tile_kernel(MmArgs a) {
    extern __shared__ __align__(1024) uint8_t lds[];
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane & 15, q = lane >> 4;
    const int wr = wave / C::WC, wc = wave % C::WC;
    const uint32_t lds0 = lds_addr(lds);
    const int n_rb = (a.rows + C::OUT - 1) / C::OUT;
    int32_t *table = (int32_t *)(lds + C::TABLE);  // grouped: first tile of each expert, [E] the number of tiles

    int n_tiles;
    if constexpr (C::MODE == DENSE) {
        n_tiles = (a.T + C::BN - 1) / C::BN;
    } else {
        // tiles before each expert: every thread counts those of `per` experts,
        // then a scan over the wavefront's lanes and over the wavefronts
        int32_t *part = table + a.E + 1;
        const int per = (a.E + C::THREADS - 1) / C::THREADS, e0 = threadIdx.x * per;
        int n = 0;
        for (int e = e0; e < min(e0 + per, a.E); ++e) {
            const int p0 = max(a.offsets[e], 0), p1 = min(a.offsets[e + 1], a.T);
            n += p1 > p0 ? (p1 - p0 + C::BN - 1) / C::BN : 0;
        }
        int x = n;
        for (int d = 1; d < kWave; d <<= 1) {
            const int y = __shfl_up(x, d);
            if (lane >= d) x += y;
        }
        if (lane == kWave - 1) part[wave] = x;
        __syncthreads();
        int before = x - n;
        for (int w = 0; w < wave; ++w) before += part[w];
        for (int e = e0; e < min(e0 + per, a.E); ++e) {
            table[e] = before;
            const int p0 = max(a.offsets[e], 0), p1 = min(a.offsets[e + 1], a.T);
            before += p1 > p0 ? (p1 - p0 + C::BN - 1) / C::BN : 0;
        }
        if (e0 < a.E && e0 + per >= a.E) table[a.E] = before;
        __syncthreads();
        // (ascending groups have no more tiles than this)
        n_tiles = min(__builtin_amdgcn_readfirstlane(table[a.E]), a.T / C::BN + min(a.E, a.T));
    }

    // Workgroup b runs on XCD b % 8; each XCD takes a contiguous eighth of the
    // items, row blocks of one token tile after one another, so that its L2
    // serves the tokens of a tile to all of them.
    const int64_t n_items = (int64_t)n_tiles * n_rb;
    const int xcd = blockIdx.x % 8, step = gridDim.x / 8;
    const int64_t last = n_items * (xcd + 1) / 8;
    for (int64_t item = n_items * xcd / 8 + blockIdx.x / 8; item < last; item += step) {
        const int tile = (int)(item / n_rb), m0 = (int)(item % n_rb) * C::OUT;
        int e = 0, p, end;
        if constexpr (C::MODE == DENSE) {
            p = tile * C::BN;
            end = a.T;
        } else {
            int lo = 0, hi = a.E;  // the last expert whose first tile is at most this one
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (table[mid] <= tile)
                    lo = mid;
                else
                    hi = mid;
            }
            e = __builtin_amdgcn_readfirstlane(lo);
            p = max(__builtin_amdgcn_readfirstlane(a.offsets[e]), 0) +
                (tile - __builtin_amdgcn_readfirstlane(table[e])) * C::BN;
            end = min(__builtin_amdgcn_readfirstlane(a.offsets[e + 1]), a.T);
            if (p < 0 || p >= end) continue;
        }
        const int n_tok = min(C::BN, end - p);

        // ---- what this wavefront loads: MW weight rows from row MW * wave, MA tokens from MA * wave
        const int w_pitch = a.in / 2, a_pitch = AF == K3G_MXFP4 ? a.in / 2 : a.in;
        // row i of the tile's weights: tensor and row past m0
        auto w_tensor = [&](int i) { return C::MODE == GLU ? (i / (C::FM * 8)) & 1 : 0; };
        auto w_row = [&](int i) {
            const int row = C::MODE == GLU ? i / (C::FM * 16) * (C::FM * 8) + i % (C::FM * 8) : i;
            return min(row, a.rows - 1 - m0);
        };
        const int cw = (lane & 3) ^ ((lane >> 3) & 3);  // the chunk this lane moves, of row lane / 4
        const int ca = AF == K3G_MXFP4 ? cw : (lane & 7) ^ (lane >> 3);  // ... of row lane / 8
        uint32_t vw[C::DW], va[C::DA];
        const uint8_t *bw[C::DW];
        const uint8_t *ba = a.perm ? a.a_codes : a.a_codes + (int64_t)p * a_pitch;
        const uint8_t *bsa = a.perm ? a.a_scales : a.a_scales + (int64_t)p * a.G;
        auto a_row = [&](int i) {  // row of the activations past ba
            const int t = min(i, n_tok - 1);
            return a.perm ? source_row(a, p + t) : t;
        };
#pragma unroll
        for (int d = 0; d < C::DW; ++d) {
            const int i = wave * C::MW + 16 * d;
            bw[d] = a.w[w_tensor(i)] + e * a.stride + (int64_t)m0 * w_pitch;
            vw[d] = (uint32_t)w_row(i + lane / 4) * w_pitch + 16 * cw;
        }
        constexpr int RA = 1024 / C::AB;  // tokens of one DMA instruction
#pragma unroll
        for (int d = 0; d < C::DA; ++d)
            va[d] = (uint32_t)a_row(wave * C::MA + RA * d + lane / (64 / RA)) * a_pitch + 16 * ca;
        // scales: this lane's weight row and token (lanes past the wavefront's rows idle)
        const int iw = wave * C::MW + min(lane, C::MW - 1), ia = wave * C::MA + min(lane, C::MA - 1);
        const uint8_t *bsw = a.ws[0] + e * a.stride + (int64_t)m0 * a.G;
        uint64_t w_off = (uint64_t)w_row(iw) * a.G;
        if (C::MODE == GLU && w_tensor(iw)) w_off += a.ws[1] - a.ws[0];
        // addresses cut to dwords; `two`: some row's four bytes straddle dwords
        const uint64_t aw = (uint64_t)bsw + w_off, aa = (uint64_t)bsa + (uint64_t)a_row(ia) * a.G;
        const int shw = (int)(aw & 3), sha = (int)(aa & 3);
        const bool two = a.two;
        const int S = (a.G + 3) / 4, Gt = a.G - 4 * (S - 1);  // stages, groups of the last

        auto issue = [&](int s) {
            const uint32_t buf = lds0 + (uint32_t)(s % C::NB) * C::STAGE;
            const bool tail = s == S - 1;
            // past the row's end the last whole chunk is read again (its place is zeroed later)
            const uint32_t backw = tail ? 16u * (uint32_t)max(cw - (Gt - 1), 0) : 0u;
            const uint32_t backa =
                tail ? 16u * (uint32_t)max(ca - (AF == K3G_MXFP4 ? Gt - 1 : 2 * Gt - 1), 0) : 0u;
#pragma unroll
            for (int d = 0; d < C::DW; ++d)
                dma16(bw[d] + 64 * (int64_t)s, vw[d] - backw, buf + (wave * C::MW + 16 * d) * 64);
#pragma unroll
            for (int d = 0; d < C::DA; ++d)
                dma16(ba + C::AB * (int64_t)s, va[d] - backa, buf + C::BM * 64 + wave * C::MA * C::AB + 1024 * d);
            const uint32_t raw = buf + C::DATA;
            const int need = tail ? Gt - 1 : 3;
            const uint64_t w4 = aw + 4 * (uint64_t)s, a4 = aa + 4 * (uint64_t)s;
            if (lane < C::MW) {
                dma4_at((const void *)(w4 & ~3ull), raw + wave * C::MW * 4);
                if (two) dma4_at((const void *)((w4 + need) & ~3ull), raw + (C::BM + wave * C::MW) * 4);
            }
            if (lane < C::MA) {
                dma4_at((const void *)(a4 & ~3ull), raw + (2 * C::BM + wave * C::MA) * 4);
                if (two) dma4_at((const void *)((a4 + need) & ~3ull), raw + (2 * C::BM + C::BN + wave * C::MA) * 4);
            }
        };

        // this wavefront's rows of stage s, landed: scales to operand order, groups that add nothing zeroed
        auto prepare = [&](int s) {
            uint8_t *buf = lds + (s % C::NB) * C::STAGE;
            uint8_t *sc = lds + C::NB * C::STAGE + (s & 1) * C::SCALES;
            const uint32_t *raw = (const uint32_t *)(buf + C::DATA);
            const int n = s == S - 1 ? Gt : 4;
            const uint32_t past = n == 4 ? 0u : ~0u << (8 * n);
            uint32_t dw = raw[iw], da = raw[2 * C::BM + ia];
            if (two) {
                dw = __builtin_amdgcn_alignbyte(raw[C::BM + iw], dw, shw);
                da = __builtin_amdgcn_alignbyte(raw[2 * C::BM + C::BN + ia], da, sha);
            }
            dw |= past;
            da |= past;
            // bytes equal to 255: the top bit of (b & 127) + 1, where b's own top bit is set
            const uint32_t fw = ((dw & 0x7F7F7F7Fu) + 0x01010101u) & dw & 0x80808080u;
            const uint32_t fa = ((da & 0x7F7F7F7Fu) + 0x01010101u) & da & 0x80808080u;
            // 255 -> 127: take the top bit away
            const uint32_t ow = dw ^ fw, oa = da ^ fa;
            if (lane < C::MW) {
                uint8_t *o = sc + (iw / 64) * 256 + (iw & 15) * 4 + ((iw >> 4) & 3);
#pragma unroll
                for (int k = 0; k < 4; ++k) o[64 * k] = (uint8_t)(ow >> (8 * k));
            }
            if (lane < C::MA) {
                uint8_t *o = sc + C::BM * 4 + (ia / 64) * 256 + (ia & 15) * 4 + ((ia >> 4) & 3);
#pragma unroll
                for (int k = 0; k < 4; ++k) o[64 * k] = (uint8_t)(oa >> (8 * k));
            }
            if (__builtin_expect(__ballot((fw | fa) != 0) != 0, 0)) {
                const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (lane < C::MW && ((fw >> (8 * k)) & 0x80u))
                        *(uint4 *)(buf + iw * 64 + 16 * (k ^ ((iw >> 1) & 3))) = zero;
                    if (lane < C::MA && ((fa >> (8 * k)) & 0x80u)) {
                        uint8_t *row = buf + C::BM * 64 + ia * C::AB;
                        if constexpr (AF == K3G_MXFP4) {
                            *(uint4 *)(row + 16 * (k ^ ((ia >> 1) & 3))) = zero;
                        } else {
                            *(uint4 *)(row + 16 * ((2 * k) ^ (ia & 7))) = zero;
                            *(uint4 *)(row + 16 * ((2 * k + 1) ^ (ia & 7))) = zero;
                        }
                    }
                }
            }
        };

        // operands of a stage
        struct Ops {
            uint4 w[C::FM];
            uint4 t[C::FN][C::AB / 64];
            uint32_t sw[(C::FM + 3) / 4], st[(C::FN + 3) / 4];
        };
        const int w_at = (wr * C::FM * 16 + r) * 64 + 16 * (q ^ ((r >> 1) & 3));
        const int a_at = C::BM * 64 + (wc * C::FN * 16 + r) * C::AB +
                         16 * (AF == K3G_MXFP4 ? q ^ ((r >> 1) & 3) : q ^ (r & 7));
        auto read = [&](Ops &o, int s) {
            const uint8_t *buf = lds + (s % C::NB) * C::STAGE;
            const uint8_t *sc = lds + C::NB * C::STAGE + (s & 1) * C::SCALES + q * 64 + r * 4;
#pragma unroll
            for (int k = 0; k < (C::FM + 3) / 4; ++k) {
                const int f = wr * C::FM + 4 * k;
                o.sw[k] = *(const uint32_t *)(sc + (f / 4) * 256) >> (8 * (f & 3));
            }
#pragma unroll
            for (int k = 0; k < (C::FN + 3) / 4; ++k) {
                const int f = wc * C::FN + 4 * k;
                o.st[k] = *(const uint32_t *)(sc + C::BM * 4 + (f / 4) * 256) >> (8 * (f & 3));
            }
#pragma unroll
            for (int f = 0; f < C::FN; ++f)
#pragma unroll
                for (int k = 0; k < C::AB / 64; ++k)
                    o.t[f][k] = *(const uint4 *)(buf + (a_at ^ (64 * k)) + f * 16 * C::AB);
#pragma unroll
            for (int f = 0; f < C::FM; ++f) o.w[f] = *(const uint4 *)(buf + w_at + f * 1024);
        };

        float4_t acc[C::FM][C::FN];
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j) acc[i][j] = float4_t{0.f, 0.f, 0.f, 0.f};
        auto multiply = [&](const Ops &o, auto half) {
            mul_tiles<AF, C, decltype(half)::value * (C::FM / 2), C::FM / 2>(o.w, o.t, o.sw, o.st, acc,
                                                                             typename MakeSeq<C::FN>::type{});
        };
        const int ahead = min(C::NB, S);
        for (int s = 0; s < ahead; ++s) issue(s);
        wait_stages<C::V1, C::V2, C::NB - 1>(two, S - 1);
        prepare(0);
        stage_barrier();
        Ops ops[2];
        read(ops[0], 0);
        auto stage = [&](int s, Ops &now, Ops &next) {
            if (s + 1 < S) {
                // in flight behind s+1: stages up to s + NB - 1
                wait_stages<C::V1, C::V2, C::NB - 2>(two, S - 2 - s);
                prepare(s + 1);
            }
            multiply(now, Half<0>{});
            if (s + 1 < S) {
                stage_barrier();
                if (s + C::NB < S) issue(s + C::NB);
                read(next, s + 1);
            }
            multiply(now, Half<1>{});
        };
        for (int s = 0; s < S; s += 2) {
            stage(s, ops[0], ops[1]);
            if (s + 1 < S) stage(s + 1, ops[1], ops[0]);
        }

        // ---- out
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
            const int t = (wc * C::FN + j) * 16 + r;
            const bool live = t < n_tok;
            if constexpr (C::MODE == GLU) {
#pragma unroll
                for (int i = 0; i < C::FM / 2; i += 2) {
                    const int row = m0 + wr * C::FM * 8 + 16 * i;
                    float4_t h[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            h[k][x] = situ(acc[i + k][j][x], acc[C::FM / 2 + i + k][j][x]);
                    const bool on = live && row < a.rows;
                    if (a.h_format == K3G_MXFP4)
                        store_h<K3G_MXFP4>(a, p + t, row / kGroup, h[0], h[1], on);
                    else
                        store_h<K3G_MXFP8>(a, p + t, row / kGroup, h[0], h[1], on);
                }
            } else if (live) {
#pragma unroll
                for (int i = 0; i < C::FM; ++i)
                    store4(a, p + t, m0 + (wr * C::FM + i) * 16 + 4 * q, acc[i][j]);
            }
        }
        __syncthreads();  // the next item's loads come after everyone's last reads
    }
}

template <int AF, class C>
int launch(const MmArgs &a, hipStream_t st) {
    const int bytes = C::lds(a.E);
    // the attribute is a property of the kernel on a device: set at every
    // launch (a host-side store), so that no state is kept here
    if (hipFuncSetAttribute((const void *)mx_tile_kernel<AF, C>, hipFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
        hipSuccess)
        return K3G_EHIP;
    const int64_t n_rb = (a.rows + C::OUT - 1) / C::OUT;
    const int64_t tiles = C::MODE == DENSE ? ((int64_t)a.T + C::BN - 1) / C::BN
                                           : a.T / C::BN + (a.E < a.T ? a.E : a.T);
    const int64_t most = 256 * (163840 / bytes);  // one round of workgroups
    const int64_t items = tiles * n_rb, grid = items < most ? (items + 7) / 8 * 8 : most;
    mx_tile_kernel<AF, C><<<(unsigned)grid, C::THREADS, bytes, st>>>(a);
    return hipGetLastError() == hipSuccess ? K3G_OK : K3G_EHIP;
}

template <int AF, int MODE>
int launch_mode(const MmArgs &a, hipStream_t st) {
    if (MODE == DENSE ? a.T <= 64 : a.T <= 16 * a.E) return launch<AF, Tile<AF, MODE, 4, 1, 4, 4, 3>>(a, st);
    if constexpr (AF == K3G_MXFP4 && MODE == DENSE) {
        if ((int64_t)a.T * a.rows >= 128 * 65536) return launch<AF, Tile<AF, MODE, 2, 2, 8, 8, 4>>(a, st);
    }
    return launch<AF, Tile<AF, MODE, 2, 2, 4, 4, AF == K3G_MXFP4 ? 3 : 2>>(a, st);
}

template <int AF>
int launch_af(const MmArgs &a, int mode, hipStream_t st) {
    return mode == DENSE     ? launch_mode<AF, DENSE>(a, st)
           : mode == GROUPED ? launch_mode<AF, GROUPED>(a, st)
                             : launch_mode<AF, GLU>(a, st);
}

int launch_tile(const MmArgs &a, int mode, int af, hipStream_t st) {
    return af == K3G_MXFP4 ? launch_af<K3G_MXFP4>(a, mode, st) : launch_af<K3G_MXFP8>(a, mode, st);
}

}  // namespace k3g
