// mxmm.hip -- products of microscaled activations with MXFP4 weights on the
// block-scaled matrix cores: dense, grouped by expert over ragged groups, and
// the experts' gated up-products with h quantised on the way out.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes both operands as they are stored.
// Operand A is the weights (16 rows of the output), operand B the activations
// (16 tokens), so a lane's four results are four consecutive outputs of one
// token. Lane l = r + 16 q holds, of row or token r and a step of 128 entries:
//   e2m1: the 16 bytes of group q (entries 32q .. 32q+31);
//   e4m3: the 16 bytes of entries 16q .. and the 16 of entries 64 + 16q ..;
//   the block scale of group q (in either format).
// (The scale operands have to be vector registers that differ by lane: a scale
// that the compiler can prove uniform would sit in a scalar register.)
// A group whose byte is 255, or past the end of the row, has its codes zeroed
// and its scale made finite: it adds exactly nothing.
#include "mxmm.h"

namespace k3g {

// ---- few tokens: the weights streamed once -----------------------------------------
//
// A dense product of so few tokens that tiles of 128 rows would leave most CUs
// idle: a workgroup takes 16 NT tokens and 16 TILES outputs and splits the rows'
// length, each wavefront four steps of 128 entries at a time: their weights and
// scales (4 KB a tile) are all in flight before the first product, the tokens' codes
// two steps ahead of it. The wavefronts' sums
// meet in LDS and are added in wavefront order. Four consecutive lanes load 64
// contiguous bytes of a row (the L2 serves that several times faster than 16 rows
// in consecutive lanes) and a permutation brings them into operand order.
// One MXFP8 token at 7168 -> 3584: 7.8 us for 14 MB, 61 MXFP4 tokens at 3584 ->
// 7168: 8.3 us for 16 MB. Latency bounds both (a launch, two to three rounds of
// loads in a row, the sum over the wavefronts, a store); the bytes alone would
// take a third.
constexpr int kSteps = 4;       // steps a wavefront loads together
constexpr int stream_waves(int nt) { return nt == 1 ? 16 : 8; }  // most wavefronts of a workgroup

// Sixteen scale bytes of a row from group g on (255 past the row's end).
__device__ inline uint4 scales16(const uint8_t *row, int g, int G) {
    uint4 v = make_uint4(~0u, ~0u, ~0u, ~0u);
    if (g + 16 <= G) {
        __builtin_memcpy(&v, row + g, 16);
    } else {
        uint8_t b[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) b[k] = g + k < G ? row[min(g + k, G - 1)] : 255;
        __builtin_memcpy(&v, b, 16);
    }
    return v;
}
__device__ inline uint32_t dword(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

template <int AF, int NT, int TILES>
__global__ __launch_bounds__(stream_waves(NT) * kWave) void mx_stream_kernel(MmArgs a) {
    constexpr int AH = AF == K3G_MXFP4 ? 1 : 2;
    extern __shared__ __align__(16) uint8_t lds[];
    const int waves = blockDim.x / kWave;
    float4_t *part = (float4_t *)lds;  // [wave][tile][token tile][lane]
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane & 15, q = lane >> 4;     // as the operand has them
    const int lr = lane >> 2, lq = lane & 3;    // as they are loaded
    const int psrc = 4 * (4 * r + q);
    const int w_pitch = a.in / 2, a_pitch = AF == K3G_MXFP4 ? a.in / 2 : a.in;
    const int S = (a.G + 3) / 4;
    Items<DENSE, 16 * NT, 16 * TILES> items(a, nullptr, blockDim.x);
    Item it;
    while (items.next(it)) {
        const uint8_t *wc[TILES], *wsc[TILES], *ac[NT], *asc[NT];
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
            wc[t] = a.w[0] + (int64_t)min(it.m0 + (TILES == 2 ? pair_row(lr, t) : lr), a.rows - 1) * w_pitch;
            wsc[t] = a.ws[0] + (int64_t)min(it.m0 + (TILES == 2 ? pair_row(r, t) : r), a.rows - 1) * a.G;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            ac[j] = a.a_codes + (int64_t)(it.p + min(16 * j + lr, it.n_tok - 1)) * a_pitch;
            asc[j] = a.a_scales + (int64_t)(it.p + min(16 * j + r, it.n_tok - 1)) * a.G;
        }
        float4_t acc[TILES][NT];
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[t][j] = float4_t{0.f, 0.f, 0.f, 0.f};
        const int nf = (it.n_tok + 15) / 16;  // token tiles with tokens
        for (int s0 = kSteps * wave; s0 < S; s0 += kSteps * waves) {
            uint4 w[kSteps][TILES], sw[TILES];
#pragma unroll
            for (int t = 0; t < TILES; ++t) sw[t] = scales16(wsc[t], 4 * s0, a.G);
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
                for (int t = 0; t < TILES; ++t)
                    w[i][t] = load16(wc[t] + 16 * (int64_t)min(4 * (s0 + i) + lq, a.G - 1));
            uint4 sa[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) sa[j] = scales16(asc[j], 4 * s0, a.G);
            uint4 b[2][NT][AH];
            auto load_b = [&](int i) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int h = 0; h < AH; ++h) {
                        // e4m3: half h of a step's 128 bytes, in chunks of half a group
                        const int c = AH * 4 * (s0 + i) + 4 * h + lq;
                        b[i & 1][j][h] = load16(ac[j] + 16 * (int64_t)min(c, AH * a.G - 1));
                    }
            };
            load_b(0);
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                if (s0 + i >= S) break;
                if (i + 1 < kSteps) load_b(i + 1);
                v8i_t W[TILES];
                uint32_t ws[TILES];
#pragma unroll
                for (int t = 0; t < TILES; ++t) {
                    uint32_t s = (dword(sw[t], i) >> (8 * q)) & 255u;
                    const uint4 v = keep4(to_operand(w[i][t], psrc), s != 255u);
                    W[t] = v8i_t{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
                    ws[t] = s == 255u ? 127u : s;
                    __asm__ volatile("" : "+v"(ws[t]));
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    if (NT > 1 && j >= nf) break;
                    const uint32_t d = dword(sa[j], i);
                    uint32_t s = (d >> (8 * q)) & 255u;
                    const Act<AF> B = [&] {
                        if constexpr (AF == K3G_MXFP4)
                            return Act<AF>(keep4(to_operand(b[i & 1][j][0], psrc), s != 255u));
                        else  // this lane's bytes belong to the groups q/2 and 2 + q/2
                            return Act<AF>(
                                keep4(to_operand(b[i & 1][j][0], psrc), ((d >> (8 * (q >> 1))) & 255u) != 255u),
                                keep4(to_operand(b[i & 1][j][1], psrc), ((d >> (16 + 8 * (q >> 1))) & 255u) != 255u));
                    }();
                    s = s == 255u ? 127u : s;
                    __asm__ volatile("" : "+v"(s));
#pragma unroll
                    for (int t = 0; t < TILES; ++t) acc[t][j] = B.mul(W[t], acc[t][j], ws[t], s);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int j = 0; j < NT; ++j) part[((wave * TILES + t) * NT + j) * kWave + lane] = acc[t][j];
        __syncthreads();
        for (int j = wave; j < nf; j += waves) {  // a wavefront sums a token tile
            float4_t s[TILES];
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
                s[t] = part[(t * NT + j) * kWave + lane];
                for (int v = 1; v < waves; ++v) s[t] += part[((v * TILES + t) * NT + j) * kWave + lane];
            }
            const bool live = 16 * j + r < it.n_tok;
            const int64_t token = it.p + 16 * j + r;
            const int row = it.m0 + 4 * TILES * q;
            if constexpr (TILES == 2) {
                if (live) with_store(a, [&](auto store) { store(token * a.ys + row, a.rows - row, s[0], s[1]); });
            } else {
                if (live) store4(a, token * a.ys + row, a.rows - row, s[0]);
            }
        }
        __syncthreads();  // part is read before the next item writes it
    }
}

template <int AF, int NT, int TILES>
int launch_stream(const MmArgs &a, hipStream_t st) {
    const int chunks = ((a.G + 3) / 4 + kSteps - 1) / kSteps;
    const int waves = chunks < stream_waves(NT) ? chunks : stream_waves(NT);
    const int64_t items = ((int64_t)a.rows + 16 * TILES - 1) / (16 * TILES) * (((int64_t)a.T + 16 * NT - 1) / (16 * NT));
    const int64_t most = 1024, grid = items < most ? (items + 7) / 8 * 8 : most;
    mx_stream_kernel<AF, NT, TILES><<<(unsigned)grid, waves * kWave, waves * TILES * NT * kWave * 16, st>>>(a);
    return hipGetLastError() == hipSuccess ? K3G_OK : K3G_EHIP;
}

// Grouped products and dense ones with enough tiles of 128 x 32 run tiled (256
// tokens at 7168 -> 3584: 20 us, here 19; 160 at 3584 -> 7168: 13, here 18; 96 at
// 7168 -> 3584: 20, here 10). Streamed, up to 16 tokens take 16 outputs a
// workgroup while each of these has a CU of its own: in us, of 16 and 32 outputs, one
// MXFP4 token 7168 -> 4096 7.5 and 9.3, 7168 -> 4608 11.7 and 9.1, MXFP8 8.4 and 9.8, 13.8
// and 9.8; of 3584 inputs 6.1 and 6.5, 7.1 and 6.7, MXFP8 6.6 and 6.9, 7.7 and 7.2. Up to 32 tokens two
// token tiles a workgroup, more four: 3584 -> 7168 (MXFP4, of one, two and four) 16
// tokens 6.8, 6.9, -; 17 tokens 8.2, 7.3, -; 32 tokens 8.5, 7.5, 8.1; 33 tokens 11.3, 9.0,
// 8.4; 64 tokens 13.0, 9.6, 9.2. (Where outputs are too few for the CUs, more workgroups
// of fewer tokens are ahead: 7168 -> 3584, 17 tokens 8.9 and 10.3, 64 tokens of two and four
// 10.2 and 13.4.)
int product_form(const MmArgs &a, int mode, int af) {
    if (const int tile = tile_form(a, mode, af)) return tile;
    if (a.T <= 16) return a.rows <= 16 * 256 ? form(16, 16) : form(32, 16);
    return a.T <= 32 ? form(32, 32) : form(32, 64);
}

template <int AF>
int launch_product(const MmArgs &a, int mode, hipStream_t st) {
    switch (const int f = product_form(a, mode, AF)) {
        case form(16, 16): return launch_stream<AF, 1, 1>(a, st);
        case form(32, 16): return launch_stream<AF, 1, 2>(a, st);
        case form(32, 32): return launch_stream<AF, 2, 2>(a, st);
        case form(32, 64): return launch_stream<AF, 4, 2>(a, st);
        default: return launch_tile(a, mode, AF, f, st);
    }
}

int launch_any(const MmArgs &a, int mode, int af, hipStream_t st) {
    return af == K3G_MXFP4 ? launch_product<K3G_MXFP4>(a, mode, st) : launch_product<K3G_MXFP8>(a, mode, st);
}

// ---- host ----------------------------------------------------------------------------

namespace {

constexpr int kMaxExperts = 2048;
constexpr int kMaxRows = 1 << 30;  // tiles are counted in 32 bits

struct Tensor {
    int p, s, rows, in;
};
Tensor bank_tensor(const k3g_expert_bank &b, int t) {
    if (t == K3G_W2) return {W2P, W2S, b.latent, b.inter};
    return t == K3G_W1 ? Tensor{W1P, W1S, b.inter, b.latent} : Tensor{W3P, W3S, b.inter, b.latent};
}

int bank_ok(const k3g_expert_bank *b) {
    if (!b || b->latent <= 0 || b->inter <= 0 || b->latent % kGroup || b->inter % kGroup || b->n_experts < 1)
        return K3G_EINVAL;
    if (b->n_experts > kMaxExperts || b->latent > kMxMaxIn || b->inter > kMxMaxIn) return K3G_EUNSUPPORTED;
    return K3G_OK;
}

// The bank's named tensor as a kernel's operand, and the addresses it covers.
int use_tensor(MmArgs *a, int slot, const k3g_expert_bank &b, int t, Span *covers) {
    const Tensor d = bank_tensor(b, t);
    const uint8_t *w = b.base + b.off[d.p], *s = b.base + b.off[d.s];
    if (b.stride < 0) return K3G_EINVAL;
    if (!mx_aligned(w, 16) || b.stride % 16) return K3G_EALIGN;
    a->w[slot] = w;
    a->ws[slot] = s;
    const int64_t last = (b.n_experts - 1) * b.stride;
    covers[0] = {(uintptr_t)w, (uintptr_t)w + last + (size_t)d.rows * d.in / 2};
    covers[1] = {(uintptr_t)s, (uintptr_t)s + last + (size_t)d.rows * (d.in / kGroup)};
    return K3G_OK;
}

// What the two grouped calls check alike.
int groups_ok(const k3g_mx *a, const int32_t *offsets, const int32_t *perm, int n_rows) {
    if (!offsets) return K3G_EINVAL;
    if (n_rows > kMaxRows) return K3G_EUNSUPPORTED;
    if (!mx_aligned(offsets, 4) || (perm && !mx_aligned(perm, 4))) return K3G_EALIGN;
    if (!perm && a->rows < n_rows) return K3G_EINVAL;
    if (a->rows < 1) return K3G_EINVAL;
    if (perm && (int64_t)a->rows * a->in >= ((int64_t)1 << 31)) return K3G_EUNSUPPORTED;
    return K3G_OK;
}

int y_vec(const void *y, int type, int64_t stride, int rows) {
    return mx_aligned(y, 16) && stride * (int64_t)type_size(type) % 16 == 0 && rows % 8 == 0;
}

// Whether some row's scale bytes lie off 16-byte addresses, or end inside sixteen.
int odd_scales(const MmArgs &m) {
    const uintptr_t bits = (uintptr_t)m.a_scales | (uintptr_t)m.ws[0] | (uintptr_t)m.ws[1] | (uintptr_t)m.G;
    return (bits & 15) != 0;
}

}  // namespace
}  // namespace k3g

using namespace k3g;

extern "C" {

int k3g_mx_matmul(void *y, int y_type, int64_t y_stride, const k3g_mx *a, const k3g_mxfp4 *w, void *stream) {
    K3G_TRY(mx_ok(a));
    if (!w || w->rows < 1 || w->in != a->in || !type_ok(y_type) || y_stride < w->rows) return K3G_EINVAL;
    if (a->rows > kMaxRows || w->rows > kMaxRows) return K3G_EUNSUPPORTED;
    if (a->rows == 0) return K3G_OK;
    if (!w->packed || !w->scales) return K3G_EINVAL;
    if (!mx_aligned(w->packed, 16)) return K3G_EALIGN;
    K3G_TRY(dense_ok(y, y_type, y_stride, w->rows));
    const Span ys = rows_span(y, y_type, a->rows, y_stride, w->rows);
    if (meet(ys, codes_span(*a)) || meet(ys, scales_span(*a)) ||
        meet(ys, span(w->packed, (size_t)w->rows * w->in / 2)) ||
        meet(ys, span(w->scales, (size_t)w->rows * (w->in / kGroup))))
        return K3G_EINVAL;
    K3G_TRY(device_ok());
    MmArgs m = {};
    m.a_codes = a->codes, m.a_scales = a->scales, m.a_rows = a->rows;
    m.w[0] = w->packed, m.ws[0] = w->scales;
    m.y = y, m.ys = y_stride, m.y_type = y_type, m.y_vec = y_vec(y, y_type, y_stride, w->rows);
    m.T = a->rows, m.rows = w->rows, m.in = a->in, m.G = a->in / kGroup;
    m.odd = odd_scales(m);
    return launch_any(m, DENSE, a->format, (hipStream_t)stream);
}

int k3g_mx_grouped_matmul(void *y, int y_type, int64_t y_stride, const k3g_mx *a, const k3g_expert_bank *bank,
                          int tensor, const int32_t *offsets, const int32_t *perm, int top_k, int n_rows,
                          void *stream) {
    K3G_TRY(mx_ok(a));
    K3G_TRY(bank_ok(bank));
    if (tensor < K3G_W1 || tensor > K3G_W2 || n_rows < 0 || top_k < 1 || !type_ok(y_type)) return K3G_EINVAL;
    const Tensor d = bank_tensor(*bank, tensor);
    if (d.in != a->in || y_stride < d.rows) return K3G_EINVAL;
    if (n_rows == 0) return K3G_OK;
    if (!bank->base) return K3G_EINVAL;
    K3G_TRY(groups_ok(a, offsets, perm, n_rows));
    K3G_TRY(dense_ok(y, y_type, y_stride, d.rows));
    MmArgs m = {};
    Span w[2];
    K3G_TRY(use_tensor(&m, 0, *bank, tensor, w));
    const Span ys = rows_span(y, y_type, n_rows, y_stride, d.rows);
    if (meet(ys, codes_span(*a)) || meet(ys, scales_span(*a)) || meet(ys, w[0]) || meet(ys, w[1]) ||
        meet(ys, span(offsets, 4 * ((size_t)bank->n_experts + 1))) || (perm && meet(ys, span(perm, 4 * (size_t)n_rows))))
        return K3G_EINVAL;
    K3G_TRY(device_ok());
    m.a_codes = a->codes, m.a_scales = a->scales, m.a_rows = a->rows;
    m.stride = bank->stride, m.offsets = offsets, m.perm = perm, m.top_k = top_k, m.E = bank->n_experts;
    m.y = y, m.ys = y_stride, m.y_type = y_type, m.y_vec = y_vec(y, y_type, y_stride, d.rows);
    m.T = n_rows, m.rows = d.rows, m.in = d.in, m.G = d.in / kGroup;
    m.odd = odd_scales(m);
    return launch_any(m, GROUPED, a->format, (hipStream_t)stream);
}

int k3g_mx_grouped_glu(const k3g_mx *h, const k3g_mx *a, const k3g_expert_bank *bank, const int32_t *offsets,
                       const int32_t *perm, int top_k, int n_rows, void *stream) {
    K3G_TRY(mx_ok(h));
    K3G_TRY(mx_ok(a));
    K3G_TRY(bank_ok(bank));
    if (n_rows < 0 || top_k < 1 || a->in != bank->latent || h->in != bank->inter || h->rows < n_rows)
        return K3G_EINVAL;
    if (n_rows == 0) return K3G_OK;
    if (!bank->base) return K3G_EINVAL;
    K3G_TRY(groups_ok(a, offsets, perm, n_rows));
    MmArgs m = {};
    Span w[4];
    K3G_TRY(use_tensor(&m, 0, *bank, K3G_W1, w));
    K3G_TRY(use_tensor(&m, 1, *bank, K3G_W3, w + 2));
    const Span hs[2] = {codes_span(*h), scales_span(*h)};
    if (meet(hs[0], hs[1])) return K3G_EINVAL;
    for (const Span &s : hs) {
        if (meet(s, codes_span(*a)) || meet(s, scales_span(*a)) ||
            meet(s, span(offsets, 4 * ((size_t)bank->n_experts + 1))) || (perm && meet(s, span(perm, 4 * (size_t)n_rows))))
            return K3G_EINVAL;
        for (const Span &t : w)
            if (meet(s, t)) return K3G_EINVAL;
    }
    K3G_TRY(device_ok());
    m.a_codes = a->codes, m.a_scales = a->scales, m.a_rows = a->rows;
    m.stride = bank->stride, m.offsets = offsets, m.perm = perm, m.top_k = top_k, m.E = bank->n_experts;
    m.h_codes = h->codes, m.h_scales = h->scales, m.h_format = h->format;
    m.T = n_rows, m.rows = bank->inter, m.in = bank->latent, m.G = bank->latent / kGroup;
    m.odd = odd_scales(m);
    return launch_any(m, GLU, a->format, (hipStream_t)stream);
}

int k3g_probe_mx_form(int a_format, int kind, int n_rows, int rows, int n_experts) {
    if ((a_format != K3G_MXFP4 && a_format != K3G_MXFP8) || kind < DENSE || kind > GLU || n_rows < 1 || rows < 1 ||
        n_rows > kMaxRows || rows > kMaxRows || (kind != DENSE && (n_experts < 1 || n_experts > kMaxExperts)))
        return K3G_EINVAL;
    MmArgs m = {};
    m.T = n_rows, m.rows = rows, m.E = n_experts;
    return product_form(m, kind, a_format);
}

}  // extern "C"
