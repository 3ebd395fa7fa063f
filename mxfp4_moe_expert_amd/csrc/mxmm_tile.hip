// mxmm_tile.hip -- the products of microscaled activations with MXFP4 weights
// for many tokens: tiles of BM weight rows x BN tokens, both operands staged
// through LDS in steps of 128 entries.
//
// A stage holds 64 bytes of each weight row and 64 (e2m1) or 128 (e4m3) of each
// token, written by LDS DMA: four (eight) consecutive lanes take one row's
// contiguous bytes, each 16-byte chunk at a place that depends on the row, so
// that the operand reads (16 bytes of 16 rows a quarter wavefront) meet no bank
// twice. Scales come for four stages at a time, 16 bytes a row: one lane a
// row, whatever the width of the request, so a request a stage would cost the
// address unit as much as the data. The wavefront that loaded a row turns its
// bytes into operand order (for each group of a step one dword, a byte for each
// of the four stages: the instruction picks the byte), and where one is 255 or
// past the row's end it makes the scale finite and, when the stage has landed,
// zeroes the group's codes in LDS.
//
// Pipeline, one barrier a stage, in the middle of its products:
//   products of stage s, first half | wait for the own rows of s+1, prepare them
//   barrier: s+1 is whole, and everyone has read s
//   DMA of stage s+NB into s's place | operands of s+1 into registers
//   products of stage s, second half
// so the matrix cores have work across the barrier, and NB - 1 stages are in
// flight or about to be read.
//
// Measured, MXFP4: 4096 tokens at 7168 -> 6144 (256 x 256) 117-130 us, 2.8-3.1
// PFLOP/s; 65536 grouped rows at 896 experts (256 x 128) 0.81-0.89 ms, 1.6-1.8 PFLOP/s,
// and their gated up-products 1.8-1.9 ms, of which the way out (SiTU, quantising) is
// 18%. MXFP8: 240-258 us, 1.4-1.5 ms and 3.0-3.25 ms, two matrix instructions an operand
// pair. The matrix cores are 30% busy and the L2 serves 118-121 G requests a second
// (64 bytes a row and stage, and 16 of scales), neither at its limit: loads alone take
// 90 of the dense product's 120 us (158 G a second), products alone 85, and they overlap
// in part only, all wavefronts in step at one barrier a stage. 1024 grouped MXFP8 rows
// that meet 230 experts (128 x 32): 255-291 us, 4.7-5.3 TB/s of HBM, which bounds those;
// the 16 experts of one token 48 us, 3.9 TB/s (one item a workgroup: start and end show).
#include "mxmm.h"

namespace k3g {

// WR x WC wavefronts of FM x FN operand tiles (16 x 16) each, NB stages in LDS.
// ODD: rows whose scale bytes start off 16-byte addresses or end inside four
// stages; they come as five aligned dwords and are shifted into place (at a
// tensor's ends, where a dword would reach outside it, byte by byte).
template <int AF, int MODE_, int WR_, int WC_, int FM_, int FN_, int NB_, bool ODD_>
struct Tile {
    static constexpr int MODE = MODE_, WR = WR_, WC = WC_, FM = FM_, FN = FN_, NB = NB_;
    static constexpr bool ODD = ODD_;
    static constexpr int NW = WR * WC, THREADS = NW * kWave;
    static constexpr int BM = WR * FM * 16, BN = WC * FN * 16;
    static constexpr int OUT = MODE == GLU ? BM / 2 : BM;  // outputs of a tile
    static constexpr int AB = AF == K3G_MXFP4 ? 64 : 128;  // bytes of a token a stage
    // Rows that a wavefront loads and prepares; with fewer than 16 tokens for each, several load the
    // same ones to the same place.
    static constexpr int MW = BM / NW, MA = BN / NW < 16 ? 16 : BN / NW;
    static constexpr int DW = MW / 16, DA = MA * AB / 1024;  // DMA instructions of 1 KB
    static_assert(MW % 16 == 0 && MA % 16 == 0 && MW + MA <= kWave, "a lane for each row of a wavefront");
    static_assert(FM % 4 == 0 && (FN == 1 || FN % 2 == 0), "halves; GLU: a wavefront owns whole 32-groups of h");
    static constexpr int V = DW + DA, X = ODD ? 5 : 1;  // loads of a stage, and of four stages' scales
    static_assert(NB >= 2 && NB <= 4, "the scales of four stages are prepared before the next four's are loaded");
    // LDS: data per stage, raw scales of four stages, scales in operand order
    static constexpr int STAGE = BM * 64 + BN * AB, RAW_W = kWave * (ODD ? 20 : 16), RAW = NW * RAW_W;
    static constexpr int SCALES = (BM + BN) * 16;
    static constexpr int RAW_AT = NB * STAGE, SCALES_AT = RAW_AT + RAW;
    static constexpr int PERM_AT = SCALES_AT + SCALES;  // grouped: the next tile's source rows, and the table
    static constexpr int TABLE = PERM_AT + (MODE == DENSE ? 0 : NW * kWave * 4);
    static constexpr int lds(int E) { return TABLE + (MODE == DENSE ? 0 : 4 * (E + 1) + 64); }
    static constexpr int WGS = 163840 / lds(900);  // workgroups on a CU
    static constexpr int WAVES = NW * WGS < 8 ? 1 : 2;  // wavefronts per SIMD that the registers allow for
    // loads in flight behind stage s+1 (s % 4 = ph): stages s+2 .. s+NB-1
    static constexpr int behind(int ph) {
        int n = (NB - 2) * V;
        for (int k = 2; k < NB; ++k)
            if ((ph + k) % 4 == 0) n += X;
        return n;
    }
};

// Where chunk c of weight row i lies: c ^ w_swz(i). The rows of an operand tile
// are four of every eight (pair_row), and any eight lanes' rows meet each of the
// eight 16-byte places of 128 bytes once.
__device__ inline int w_swz(int row) { return ((row >> 1) & 1) | ((row >> 2) & 2); }

__device__ inline void stage_barrier() {
    __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
}

// global -> LDS without registers as dma4, each lane from an address of its own
__device__ inline void dma4_at(const void *p, uint32_t lds) {
    lds = __builtin_amdgcn_readfirstlane(lds);
    __asm__ volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dword %0, off" : : "v"(p), "s"(lds) : "m0");
}

__device__ inline void dma16_at(const void *p, uint32_t lds) {
    lds = __builtin_amdgcn_readfirstlane(lds);
    __asm__ volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(p), "s"(lds) : "m0");
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

// (w: the half's tiles; sw, st: a byte of each stage in turn, PH the stage's.)
template <int AF, class C, int PH, int J, int I0, int... I>
__device__ inline void mul_column(const uint4 *w, const uint4 *t, const uint32_t *sw, uint32_t st,
                                  float4_t (*acc)[C::FN], Seq<I...>) {
    const Act<AF> b = [&] {
        if constexpr (AF == K3G_MXFP4)
            return Act<AF>(t[0]);
        else
            return Act<AF>(t[0], t[1]);
    }();
    ((acc[I0 + I][J] =
          b.template mul<PH, PH>(v8i_t{(int)w[I].x, (int)w[I].y, (int)w[I].z, (int)w[I].w, 0, 0, 0, 0},
                                 acc[I0 + I][J], sw[I0 + I], st)),
     ...);
}
// Token tiles J0 + J... with the weights' tiles I0 .. I0+NI-1 (w, t: those tiles);
// the wavefront has tokens in its first nf tiles only (uniform; a dense product's
// tiles are all full but the last, itself more than half where it is the only
// one, and there the branches cost 5%).
template <int AF, class C, int PH, int I0, int NI, int J0, int... J>
__device__ inline void mul_tiles(const uint4 *w, const uint4 (*t)[C::AB / 64], const uint32_t *sw, const uint32_t *st,
                                 float4_t (*acc)[C::FN], int nf, Seq<J...>) {
    ((C::MODE == DENSE || J0 + J < nf ? mul_column<AF, C, PH, J0 + J, I0>(w, t[J], sw, st[J0 + J], acc, typename MakeSeq<NI>::type{})
                  : void()),
     ...);
}

template <int H_, int Q_>
struct Part {
    static constexpr int H = H_, Q = Q_;
};
template <int PH_>
struct Phase {
    static constexpr int PH = PH_;
};

template <int AF, class C>
__global__ __launch_bounds__(C::THREADS, C::WAVES) void mx_tile_kernel(MmArgs a) {
    extern __shared__ __align__(1024) uint8_t lds[];
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wr = wave / C::WC, wc = wave % C::WC;
    const uint32_t lds0 = lds_addr(lds);
    Items<C::MODE, C::BN, C::OUT> items(a, (int32_t *)(lds + C::TABLE), C::THREADS);
    Item now, next;

    // ---- what this wavefront loads: MW weight rows from row MW * wave, MA tokens from MA * wave
    const int w_pitch = a.in / 2, a_pitch = AF == K3G_MXFP4 ? a.in / 2 : a.in;
    const int S = (a.G + 3) / 4, Gt = a.G - 4 * (S - 1);  // stages, groups of the last
    const bool is_w = lane < C::MW, has_row = lane < C::MW + C::MA;
    const int iw = wave * C::MW + min(lane, C::MW - 1), ia_own = min(max(lane - C::MW, 0), C::MA - 1);
    const int a0 = wave * C::MA % C::BN, ia = a0 + ia_own;
    const int cw = (lane & 3) ^ w_swz(lane >> 2);                     // the chunk this lane moves, of row lane / 4
    const int ca = AF == K3G_MXFP4 ? (lane & 3) ^ ((lane >> 3) & 3)  // ... of a token
                                   : (lane & 7) ^ (lane >> 3);
    auto w_tensor = [&](int i) { return C::MODE == GLU ? (i / (C::FM * 8)) & 1 : 0; };  // of row i of the tile
    // the addresses that the loads are issued from: those of the item being loaded
    uint32_t vw[C::DW], va[C::DA];
    const uint8_t *bw[C::DW], *ba;
    uint64_t s_addr;  // of the row whose scales this lane loads and prepares: a weight row, from lane MW on a token
    // ODD: its first dword begins before the tensor (bit 0), its last ends behind it (bit 1); whether some
    // lane's does (uniform); and then the two dwords, of the row's own bytes
    int ends = 0;
    bool edged = false;
    uint32_t edge[2];
    // the tile's entries of perm, fetched ahead (each wavefront its own tokens')
    int32_t *perm = (int32_t *)(lds + C::PERM_AT) + wave * kWave;
    auto fetch_perm = [&](const Item &o) {
        if (C::MODE != DENSE && a.perm && lane < C::MA)
            dma4_at(a.perm + o.p + min(a0 + lane, o.n_tok - 1), lds0 + C::PERM_AT + wave * kWave * 4);
    };
    auto address = [&](const Item &o) {
        auto w_row = [&](int i) {  // row past m0 of row i of the tile
            const int row = C::MODE == GLU ? i / (C::FM * 16) * (C::FM * 8) + i % (C::FM * 8) : i;
            return min(row, a.rows - 1 - o.m0);
        };
        const bool gather = C::MODE != DENSE && a.perm;
        auto a_row = [&](int own) {  // row past ba of this wavefront's token `own`
            if (!gather) return min(a0 + own, o.n_tok - 1);
            return min(max(perm[own] / a.top_k, 0), a.a_rows - 1);
        };
        ba = gather ? a.a_codes : a.a_codes + (int64_t)o.p * a_pitch;
#pragma unroll
        for (int d = 0; d < C::DW; ++d) {
            const int i = wave * C::MW + 16 * d;
            bw[d] = a.w[w_tensor(i)] + o.e * a.stride + (int64_t)o.m0 * w_pitch;
            vw[d] = (uint32_t)w_row(i + lane / 4) * w_pitch + 16 * cw;
        }
        constexpr int RA = 1024 / C::AB;  // tokens of one DMA instruction
#pragma unroll
        for (int d = 0; d < C::DA; ++d) va[d] = (uint32_t)a_row(RA * d + lane / (64 / RA)) * a_pitch + 16 * ca;
        s_addr = is_w ? (uint64_t)(a.ws[w_tensor(iw)] + o.e * a.stride) + (uint64_t)(o.m0 + w_row(iw)) * a.G
                      : (uint64_t)a.a_scales + ((uint64_t)(gather ? 0 : o.p) + (uint64_t)a_row(ia_own)) * a.G;
        if constexpr (C::ODD) {
            const int row = is_w ? o.m0 + w_row(iw) : (gather ? 0 : o.p) + a_row(ia_own);
            const int behind = (is_w ? a.rows : a.a_rows) - 1 - row;  // rows of the tensor
            ends = (row < 3 && row * a.G < (int)(s_addr & 3) ? 1 : 0) |
                   (behind < 3 && behind * a.G < 3 - (int)((s_addr + a.G - 1) & 3) ? 2 : 0);
            edged = __ballot(ends != 0) != 0;
            if (edged) {  // (loaded here: prepare_scales comes a round of loads later)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    edge[k] = 0;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const uint64_t last = s_addr + a.G - 1, at = ((k ? last : s_addr) & ~3ull) + b;
                        const uint32_t byte = *(const uint8_t *)(at < s_addr ? s_addr : at > last ? last : at);
                        edge[k] |= at < s_addr || at > last ? 0u : byte << (8 * b);
                    }
                }
            }
        }
    };
    auto issue = [&](int s, int buffer) {
        const uint32_t buf = lds0 + (uint32_t)buffer * C::STAGE;
        // past the row's end the last whole chunk is read again (its place is zeroed later)
        const bool tail = s == S - 1;
        const uint32_t backw = tail ? 16u * (uint32_t)max(cw - (Gt - 1), 0) : 0u;
        const uint32_t backa = tail ? 16u * (uint32_t)max(ca - (AF == K3G_MXFP4 ? Gt - 1 : 2 * Gt - 1), 0) : 0u;
#pragma unroll
        for (int d = 0; d < C::DW; ++d)
            dma16(bw[d] + 64 * (int64_t)s, vw[d] - backw, buf + (wave * C::MW + 16 * d) * 64);
#pragma unroll
        for (int d = 0; d < C::DA; ++d)
            dma16(ba + C::AB * (int64_t)s, va[d] - backa, buf + C::BM * 64 + a0 * C::AB + 1024 * d);
    };
    const uint32_t raw = lds0 + C::RAW_AT + wave * C::RAW_W;
    // ODD: the aligned dwords that hold the bytes of the stages 4u .. 4u + 3; past the row's last byte, the
    // one that holds it. One with bytes outside the tensor is not read: its place takes some codes
    // instead, and prepare_scales what `edge` has.
    auto scale_dword = [&](int u, int k) {
        const uint64_t end = (s_addr + a.G - 1) & ~3ull, w = ((s_addr + 16 * (uint64_t)u) & ~3ull) + 4 * k;
        return w < end ? w : end;
    };
    auto outside = [&](uint64_t w) {  // 1: before the tensor, 2: behind it, 0: neither
        return (ends & 1) && w < s_addr ? 1 : (ends & 2) && w + 4 > s_addr + a.G ? 2 : 0;
    };
    auto issue_scales = [&](int u) {  // of the stages 4u .. 4u + 3
        if (!has_row) return;         // (lane 0 always has one)
        if constexpr (!C::ODD) {
            dma16_at((const void *)(s_addr + 16 * (uint64_t)u), raw);
        } else if (!edged) {
#pragma unroll
            for (int k = 0; k < 5; ++k) dma4_at((const void *)scale_dword(u, k), raw + 256 * k);
        } else {
            for (int k = 0; k < 5; ++k) {
                const uint64_t w = scale_dword(u, k);
                dma4_at(outside(w) ? (const void *)a.a_codes : (const void *)w, raw + 256 * k);
            }
        }
    };

    // this wavefront's rows: the scales of the stages 4u .. to operand order, and a stage's
    // groups that add nothing (bits in `out`, a dword a stage) zeroed
    const int s_at = C::SCALES_AT + 16 * (is_w ? iw : C::BM + ia);
    const int d_at = is_w ? iw * 64 : C::BM * 64 + ia * C::AB;
    const int d_swz = is_w ? w_swz(iw) : AF == K3G_MXFP4 ? (ia >> 1) & 3 : ia & 7;
    uint32_t out[4];
    auto prepare_scales = [&](int u) {
        uint32_t d[4];
        if constexpr (!C::ODD) {
            const uint4 v = *(const uint4 *)(lds + C::RAW_AT + wave * C::RAW_W + 16 * lane);
            d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
        } else {
            uint32_t v[5];
#pragma unroll
            for (int k = 0; k < 5; ++k) v[k] = ((const uint32_t *)(lds + C::RAW_AT + wave * C::RAW_W))[64 * k + lane];
            if (edged) {
#pragma unroll
                for (int k = 0; k < 5; ++k) {
                    const int o = outside(scale_dword(u, k));
                    v[k] = o == 1 ? edge[0] : o == 2 ? edge[1] : v[k];
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                d[k] = __builtin_amdgcn_alignbyte(v[k + 1], v[k], (uint32_t)s_addr & 3u);
                const int left = a.G - 16 * u - 4 * k;  // groups from this stage on
                if (left < 4) d[k] |= left > 0 ? ~0u << (8 * left) : ~0u;
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // bytes equal to 255: b's top bit, where (b & 127) + 1 has it too; they become 127
            const uint32_t f = ((d[k] & 0x7F7F7F7Fu) + 0x01010101u) & d[k] & 0x80808080u;
            d[k] ^= f;
            out[k] = has_row ? f : 0u;
        }
        // [stage][group] bytes -> [group][stage]
        const uint32_t a0 = __builtin_amdgcn_perm(d[1], d[0], 0x05010400u), a1 = __builtin_amdgcn_perm(d[1], d[0], 0x07030602u);
        const uint32_t b0 = __builtin_amdgcn_perm(d[3], d[2], 0x05010400u), b1 = __builtin_amdgcn_perm(d[3], d[2], 0x07030602u);
        const uint4 o = make_uint4(__builtin_amdgcn_perm(b0, a0, 0x05040100u), __builtin_amdgcn_perm(b0, a0, 0x07060302u),
                                   __builtin_amdgcn_perm(b1, a1, 0x05040100u), __builtin_amdgcn_perm(b1, a1, 0x07060302u));
        if (has_row) *(uint4 *)(lds + s_at) = o;
    };
    auto zero_groups = [&](uint32_t f, int buffer) {
        while (__ballot(f != 0) != 0) {  // rarely entered; a group a round
            if (f) {
                const int k = __builtin_ctz(f) >> 3;
                uint8_t *row = lds + buffer * C::STAGE + d_at;
                const uint4 zero = make_uint4(0, 0, 0, 0);
                if (AF == K3G_MXFP4 || is_w) {
                    *(uint4 *)(row + 16 * (k ^ d_swz)) = zero;
                } else {
                    *(uint4 *)(row + 16 * ((2 * k) ^ d_swz)) = zero;
                    *(uint4 *)(row + 16 * ((2 * k + 1) ^ d_swz)) = zero;
                }
                f &= f - 1;
            }
        }
    };

    // Operands of a stage in two halves: by weight rows, the tokens' tiles whole and
    // in two sets (now, next), or by tokens with the weights' whole: an e4m3
    // tile is cut in two for the matrix cores, which is done once that way.
    constexpr bool BY_ROWS = AF == K3G_MXFP4 || C::FN == 1;
    constexpr int HM = BY_ROWS ? C::FM / 2 : C::FM, HN = BY_ROWS ? C::FN : C::FN / 2;
    uint4 wt[2][HM], tk[2][HN][C::AB / 64];
    uint32_t sw[C::FM], st[C::FN];
    const int r = lane & 15, q = lane >> 4;
    const int w_at0 = (wr * C::FM * 16 + pair_row(r, 0)) * 64 + 16 * (q ^ w_swz(pair_row(r, 0)));
    const int a_at = C::BM * 64 + (wc * 16 + r) * C::AB + 16 * (AF == K3G_MXFP4 ? q ^ ((r >> 1) & 3) : q ^ (r & 7));
    auto read_w = [&](uint4 *o, int buffer, int half) {
#pragma unroll
        for (int i = 0; i < HM; ++i)  // (tile 1 of a pair: 4 rows on, where the swizzle is the same)
            o[i] = *(const uint4 *)(lds + buffer * C::STAGE + w_at0 + (half * HM + i) / 2 * 2048 + (i & 1) * 256);
    };
    auto read_t = [&](uint4(*o)[C::AB / 64], int buffer, int half) {
#pragma unroll
        for (int f = 0; f < HN; ++f)
#pragma unroll
            for (int k = 0; k < C::AB / 64; ++k)
                o[f][k] =
                    *(const uint4 *)(lds + buffer * C::STAGE + (a_at ^ (64 * k)) + (half * HN + f) * C::WC * 16 * C::AB);
    };
    auto read_s = [&] {
        const uint8_t *sw_at = lds + C::SCALES_AT + 16 * (wr * C::FM * 16 + pair_row(r, 0)) + 4 * q;
        const uint8_t *st_at = lds + C::SCALES_AT + 16 * (C::BM + wc * 16 + r) + 4 * q;
#pragma unroll
        for (int i = 0; i < C::FM; ++i) sw[i] = *(const uint32_t *)(sw_at + i / 2 * 512 + (i & 1) * 64);
#pragma unroll
        for (int j = 0; j < C::FN; ++j) st[j] = *(const uint32_t *)(st_at + j * C::WC * 256);
    };

    float4_t acc[C::FM][C::FN];
    int nf = 0;  // this wavefront's token tiles with tokens: a tile's go round the wavefronts
    // a quarter of a stage's products: half H, part Q
    auto multiply = [&](auto phase, auto part) {
        constexpr int PH = decltype(phase)::PH, H = decltype(part)::H, Q = decltype(part)::Q;
        if constexpr (BY_ROWS) {
            constexpr int N0 = C::FN / 2, J0 = Q * N0, N = Q ? C::FN - N0 : N0;
            mul_tiles<AF, C, PH, H * HM, HM, J0>(wt[H], tk[PH & 1] + J0, sw, st, acc, nf, typename MakeSeq<N>::type{});
        } else {
            constexpr int N0 = (HN + 1) / 2, J0 = Q * N0, N = Q ? HN - N0 : N0;
            mul_tiles<AF, C, PH, 0, HM, H * HN + J0>(wt[PH & 1], tk[H] + J0, sw, st, acc, nf,
                                                     typename MakeSeq<N>::type{});
        }
        __builtin_amdgcn_sched_barrier(0);
    };

    // Rows of whole four stages run on from item to item: the last NB stages of
    // one issue the first of the next, which land behind its way out.
    const bool run_on = S % 4 == 0 && S >= C::NB;
    bool have = items.next(now), loaded = false;  // loaded: its first NB stages are in LDS, stage 0 prepared
    int at = 0;                                          // the buffer of the stage being multiplied
    while (have) {
        const bool more = items.next(next), on = run_on && more;
        if (!loaded) {
            fetch_perm(now);
            wait_vm<0>();
            address(now);
            issue_scales(0);
            for (int s = 0; s < C::NB && s < S; ++s) issue(s, s);
            if (S >= C::NB)
                wait_vm<(C::NB - 1) * C::V>();
            else
                wait_vm<0>();
            prepare_scales(0);
            zero_groups(out[0], 0);
            stage_barrier();
            at = 0;
        }
        if (on) fetch_perm(next);
        const int landed = loaded ? C::NB : 1;
        nf = ((now.n_tok + 15) / 16 - wc + C::WC - 1) / C::WC;
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j) acc[i][j] = float4_t{0.f, 0.f, 0.f, 0.f};
        read_s();
        read_w(wt[0], at, 0);
        read_t(tk[0], at, 0);
        // (At a row's end with nothing to follow, the wait, the preparation and the reads of a stage
        // that does not exist are harmless: old bytes of this workgroup's LDS that nothing uses.)
        auto stage = [&](int s, auto phase) {
            constexpr int PH = decltype(phase)::PH;
            const int after = at + 1 == C::NB ? 0 : at + 1;
            if constexpr (BY_ROWS)
                read_w(wt[1], at, 1);
            else
                read_t(tk[1], at, 1);
            if (s + C::NB > S && !on)
                wait_vm<0>();
            else if (s + 1 >= landed)
                wait_vm<C::behind(PH)>();
            __builtin_amdgcn_sched_barrier(0);
            multiply(phase, Part<0, 0>{});
            if constexpr (PH == 3) prepare_scales(s + 1 == S ? 0 : (s + 1) / 4);
            zero_groups(out[(PH + 1) % 4], after);
            multiply(phase, Part<0, 1>{});
            stage_barrier();
            multiply(phase, Part<1, 0>{});
            if (s + C::NB < S || on) {
                int to = s + C::NB;
                if (to >= S) {
                    if constexpr ((PH + C::NB) % 4 == 0) {
                        if (to == S) {
                            if (a.perm && S < 2 * C::NB) wait_vm<0>();  // perm was fetched too late to be behind a wait
                            address(next);
                        }
                    }
                    to -= S;
                }
                if constexpr ((PH + C::NB) % 4 == 0) issue_scales(to / 4);
                issue(to, at);
            }
            read_w(wt[BY_ROWS ? 0 : (PH + 1) & 1], after, 0);
            read_t(tk[BY_ROWS ? (PH + 1) & 1 : 0], after, 0);
            __builtin_amdgcn_sched_barrier(0);
            multiply(phase, Part<1, 1>{});
            if constexpr (PH == 3) read_s();
            at = after;
        };
        for (int s = 0;; s += 4) {
            stage(s, Phase<0>{});
            if (s + 1 >= S) break;
            stage(s + 1, Phase<1>{});
            if (s + 2 >= S) break;
            stage(s + 2, Phase<2>{});
            if (s + 3 >= S) break;
            stage(s + 3, Phase<3>{});
            if (s + 4 >= S) break;
        }

        // ---- out. The next item's first stages land before the stores go out: a wait for
        // loads behind stores would wait for the stores too.
        if (on) wait_vm<0>();
        int out_lane = lane;
        __asm__ volatile("" : "+v"(out_lane));
        const int ro = out_lane & 15, qo = out_lane >> 4;
        if constexpr (C::MODE == GLU) {
#pragma unroll
            for (int j = 0; j < C::FN; ++j) {
                if (j >= nf) break;
                const int t = (wc + C::WC * j) * 16 + ro;
                const bool live = t < now.n_tok;
#pragma unroll
                for (int i = 0; i < C::FM / 2; i += 2) {
                    const int row = now.m0 + wr * C::FM * 8 + 16 * i;
                    float4_t h[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            h[k][x] = situ(acc[i + k][j][x], acc[C::FM / 2 + i + k][j][x]);
                    const bool in = live && row < a.rows;
                    if (a.h_format == K3G_MXFP4)
                        store_h<K3G_MXFP4>(a, now.p + t, row / kGroup, h[0], h[1], in);
                    else
                        store_h<K3G_MXFP8>(a, now.p + t, row / kGroup, h[0], h[1], in);
                }
            }
        } else {
            const int row = now.m0 + wr * C::FM * 16 + 8 * qo, t0 = wc * 16 + ro;
            with_store(a, [&](auto store) {
                int64_t to = (int64_t)(now.p + t0) * a.ys + row;
#pragma unroll
                for (int j = 0; j < C::FN; ++j, to += C::WC * 16 * a.ys)
                    if (t0 + C::WC * 16 * j < now.n_tok) {
#pragma unroll
                        for (int i = 0; i < C::FM; i += 2)
                            store(to + 16 * i, a.rows - row - 16 * i, acc[i][j], acc[i + 1][j]);
                    }
            });
        }
        if (!on) __syncthreads();  // the next item's first loads come after everyone's last reads
        now = next;
        have = more;
        loaded = on;
    }
}

template <int AF, class C>
int launch(const MmArgs &a, hipStream_t st) {
    const int bytes = C::lds(a.E);
    // (a host-side store, a launch's price; no state is kept here)
    if (bytes > 65536 && hipFuncSetAttribute((const void *)mx_tile_kernel<AF, C>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes) != hipSuccess)
        return K3G_EHIP;
    const int64_t n_rb = (a.rows + C::OUT - 1) / C::OUT;
    const int64_t tiles = C::MODE == DENSE ? ((int64_t)a.T + C::BN - 1) / C::BN
                                           : a.T / C::BN + (a.E < a.T ? a.E : a.T);
    const int64_t most = 256 * (163840 / bytes);  // one round of workgroups
    const int64_t items = tiles * n_rb, grid = items < most ? (items + 7) / 8 * 8 : most;
    mx_tile_kernel<AF, C><<<(unsigned)grid, C::THREADS, bytes, st>>>(a);
    return hipGetLastError() == hipSuccess ? K3G_OK : K3G_EHIP;
}

// ---- which tile ------------------------------------------------------------------------
//
// Dense: the largest tile that still gives kFill items, about two thirds of the
// chip's 256 CUs (an item costs its row's length in stages whatever its size, so
// idle CUs cost more than the larger tile's better reuse gains). Measured in us
// at 7168 -> 3584 (MXFP4), items in brackets: 512 tokens 128 x 128 26 (112),
// 128 x 64 23 (224); 1024 tokens 256 x 128 38 (112), 128 x 128 28 (224), 128 x 64
// 31 (448); 2048 tokens 256 x 128 40 (224), 128 x 128 43 (448). An e4m3 tile of
// 128 x 128 has room for two stages on two workgroups only and loses to both its
// neighbours (1024 tokens: 66 against 53 and 79).
//
// And no tile that the tokens fill to half or less: with outputs to fill the chip
// whatever the tile, few tokens would multiply empty columns. 7168 -> 65536, MXFP4: 1 token 128 x 32 49-54, 256 x 256 77; 33 tokens
// 128 x 64 54, 128 x 32 76, 256 x 256 79; 65 tokens 256 x 128 58, 128 x 64 79; 129
// tokens 256 x 256 81, 256 x 128 91. MXFP8: 32 tokens 128 x 32 58, 128 x 64 69, 256 x
// 128 98; 33 tokens 128 x 64 71, 128 x 32 89; 65 tokens 256 x 128 100, 128 x 64 121.
constexpr int kFill = 160;

// Grouped: by the rows an expert has on average over the whole bank (what the
// host knows; a routing leaves some experts empty, so a group is larger). Measured at
// 896 experts in us (w2, 3072 -> 3584, and the GLU), on a flat routing and on a skewed
// one that meets 235-316 experts:
//   rows          128 x 32     128 x 64     256 x 128
//   1   MXFP4     617  1176    581  1172    616  1244
//       MXFP8     680  1361    678  1381    804  1728
//       skewed    268   524    264   517    272   557   (MXFP8 275 542, 274 550, 331 673)
//   4.6 skewed    357   688    337   643    336   654   (MXFP8 383 763, 374 745, 418 857)
//   8   MXFP4    1047  2033   1036  2012   1049  2072
//       MXFP8    1113  2186   1118  2232   1260  2686
//   9   skewed    472   903    412   794    402   818   (MXFP8 483 981, 434 889, 454 940)
//   16  MXFP4    1124  2201   1107  2170   1110  2157
//       MXFP8    1180  2372   1195  2394   1288  2739
//       skewed    605  1140    496   947    445   921   (MXFP8 659 1379, 566 1206, 567 1187)
//   24  MXFP4    1192  2353   1153  2279   1151  2238
//       MXFP8    1288  2585   1250  2546   1315  2791
//       skewed    815  1498    566  1089    498  1051   (MXFP8 906 1901, 730 1605, 682 1508)
// So up to 2 rows 32 tokens (MXFP8's few rows; MXFP4 loses 6% there at most), up to 16
// 64, and 128 beyond, where MXFP8 gains on a skewed routing what it loses on a flat one.
template <int AF, int MODE, bool ODD>
struct Tiles {
    typedef Tile<AF, MODE, 2, 4, 8, 4, 4, ODD> T256x256;  // e2m1; all 256 registers, and 6 spilled (17 for ODD)
    typedef Tile<AF, MODE, 4, 2, 4, 4, 4, ODD> T256x128;  // e2m1
    typedef Tile<AF, MODE, 2, 4, 8, 2, 3, ODD> E256x128;  // e4m3: a token tile is cut once for eight weight tiles
    typedef Tile<AF, MODE, 2, 2, 4, 4, 3, ODD> T128x128;  // e2m1
    typedef Tile<AF, MODE, 2, 2, 4, 2, AF == K3G_MXFP4 ? 4 : 3, ODD> T128x64;
    typedef Tile<AF, MODE, 2, 2, 4, 1, 4, ODD> T128x32;
};

int tile_form(const MmArgs &a, int mode, int af) {
    const bool fp4 = af == K3G_MXFP4;
    if (mode != DENSE) {
        if (a.T <= 2 * (int64_t)a.E) return form(128, 32);
        return a.T <= 16 * (int64_t)a.E ? form(128, 64) : form(256, 128);
    }
    auto fills = [&](int bm, int bn) {
        return (bn == 32 || a.T > bn / 2) && ((int64_t)a.rows + bm - 1) / bm * (((int64_t)a.T + bn - 1) / bn) >= kFill;
    };
    if (fp4 && fills(256, 256)) return form(256, 256);
    if (fills(256, 128)) return form(256, 128);
    if (fp4 && fills(128, 128)) return form(128, 128);
    if (fills(128, 64)) return form(128, 64);
    return fills(128, 32) ? form(128, 32) : 0;
}

template <int AF, int MODE, bool ODD>
int launch_mode(const MmArgs &a, int tile, hipStream_t st) {
    typedef Tiles<AF, MODE, ODD> Ts;
    if constexpr (AF == K3G_MXFP4 && MODE == DENSE) {
        if (tile == form(256, 256)) return launch<AF, typename Ts::T256x256>(a, st);
        if (tile == form(128, 128)) return launch<AF, typename Ts::T128x128>(a, st);
    }
    if (tile == form(128, 64)) return launch<AF, typename Ts::T128x64>(a, st);
    if (tile == form(128, 32)) return launch<AF, typename Ts::T128x32>(a, st);
    if constexpr (AF == K3G_MXFP4)
        return launch<AF, typename Ts::T256x128>(a, st);
    else
        return launch<AF, typename Ts::E256x128>(a, st);
}

template <int AF, bool ODD>
int launch_af(const MmArgs &a, int mode, int tile, hipStream_t st) {
    return mode == DENSE     ? launch_mode<AF, DENSE, ODD>(a, tile, st)
           : mode == GROUPED ? launch_mode<AF, GROUPED, ODD>(a, tile, st)
                             : launch_mode<AF, GLU, ODD>(a, tile, st);
}

int launch_tile(const MmArgs &a, int mode, int af, int tile, hipStream_t st) {
    if (a.odd)
        return af == K3G_MXFP4 ? launch_af<K3G_MXFP4, true>(a, mode, tile, st)
                               : launch_af<K3G_MXFP8, true>(a, mode, tile, st);
    return af == K3G_MXFP4 ? launch_af<K3G_MXFP4, false>(a, mode, tile, st)
                           : launch_af<K3G_MXFP8, false>(a, mode, tile, st);
}

}  // namespace k3g
