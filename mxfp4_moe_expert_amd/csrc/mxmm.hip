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
// A workgroup takes 16 tokens (of one expert) and 32 outputs (GLU: 32 rows of
// w1 and the same 32 of w3), its eight wavefronts every eighth step of 128
// entries each; the partial sums meet in LDS, added in wavefront order.
constexpr int kStreamWaves = 8;

template <int AF, int MODE>
__global__ __launch_bounds__(kStreamWaves * kWave) void mx_stream_kernel(MmArgs a) {
    constexpr int TILES = MODE == GLU ? 4 : 2;
    __shared__ float4_t part[kStreamWaves][TILES][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane & 15, q = lane >> 4;
    const int row0 = blockIdx.x * 32;
    const int64_t w_pitch = a.in / 2, a_pitch = AF == K3G_MXFP4 ? a.in / 2 : a.in;
    for (int64_t tile = blockIdx.y;; tile += gridDim.y) {
        int e = 0, p, end;
        if constexpr (MODE == DENSE) {
            if (tile * 16 >= a.T) return;
            p = (int)(tile * 16);
            end = a.T;
        } else {
            if (tile >= a.T) return;
            int p0;
            p = (int)tile;
            if (!find_group(a, p, e, p0, end) || (p - p0) % 16) continue;
        }
        const int n_tok = min(16, end - p);
        const int64_t src = MODE == DENSE ? p + min(r, n_tok - 1) : source_row(a, p + min(r, n_tok - 1));
        const uint8_t *ac = a.a_codes + src * a_pitch, *as = a.a_scales + src * a.G;
        const uint8_t *wc[TILES], *wsc[TILES];
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
            const int64_t row = min(row0 + pair_row(r, t & 1), a.rows - 1);
            wc[t] = a.w[t >> 1] + e * a.stride + row * w_pitch;
            wsc[t] = a.ws[t >> 1] + e * a.stride + row * a.G;
        }
        float4_t acc[TILES];
#pragma unroll
        for (int t = 0; t < TILES; ++t) acc[t] = float4_t{0.f, 0.f, 0.f, 0.f};
        for (int g0 = 4 * wave; g0 < a.G; g0 += 4 * kStreamWaves) {
            const int g = g0 + q;
            const int gc = min(g, a.G - 1);
            uint32_t sa = g < a.G ? as[gc] : 255u;
            const Act<AF> B = [&] {
                if constexpr (AF == K3G_MXFP4) {
                    return Act<AF>(keep4(load16(ac + 16 * gc), sa != 255u));
                } else {
                    // this lane's bytes belong to the groups q/2 and 2 + q/2
                    const int g1 = g0 + (q >> 1), g2 = g1 + 2, g1c = min(g1, a.G - 1), g2c = min(g2, a.G - 1);
                    return Act<AF>(keep4(load16(ac + 32 * g1c + 16 * (q & 1)), g1 < a.G && as[g1c] != 255u),
                                   keep4(load16(ac + 32 * g2c + 16 * (q & 1)), g2 < a.G && as[g2c] != 255u));
                }
            }();
            sa = sa == 255u ? 127u : sa;
            __asm__ volatile("" : "+v"(sa));
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
                uint32_t sw = g < a.G ? wsc[t][gc] : 255u;
                const uint4 w = keep4(load16(wc[t] + 16 * gc), sw != 255u);
                sw = sw == 255u ? 127u : sw;
                __asm__ volatile("" : "+v"(sw));
                acc[t] = B.mul(v8i_t{(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0}, acc[t], sw, sa);
            }
        }
#pragma unroll
        for (int t = 0; t < TILES; ++t) part[wave][t][lane] = acc[t];
        __syncthreads();
        auto sum = [&](int t) {
            float4_t s = part[0][t][lane];
#pragma unroll
            for (int w = 1; w < kStreamWaves; ++w) s += part[w][t][lane];
            return s;
        };
        if constexpr (MODE == GLU) {
            if (wave == 0) {
                float4_t h[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const float4_t g = sum(t), u = sum(2 + t);
#pragma unroll
                    for (int i = 0; i < 4; ++i) h[t][i] = situ(g[i], u[i]);
                }
                const bool live = r < n_tok;  // a.rows is a multiple of 32
                if (a.h_format == K3G_MXFP4)
                    store_h<K3G_MXFP4>(a, p + r, row0 / kGroup, h[0], h[1], live);
                else
                    store_h<K3G_MXFP8>(a, p + r, row0 / kGroup, h[0], h[1], live);
            }
        } else if (wave == 0) {
            const float4_t lo = sum(0), hi = sum(1);
            const int row = row0 + 8 * q;
            if (r < n_tok) with_store(a, [&](auto store) { store((p + r) * a.ys + row, a.rows - row, lo, hi); });
        }
        __syncthreads();  // part is read before the next tile writes it
    }
}

template <int MODE>
int launch_stream(const MmArgs &a, int af, hipStream_t st) {
    if (MODE == DENSE ? a.T > 32 : a.T > 4 * a.E) return launch_tile(a, MODE, af, st);
    const int64_t tiles = MODE == DENSE ? ((int64_t)a.T + 15) / 16 : a.T;
    const dim3 grid((a.rows + 31) / 32, (unsigned)(tiles < 65535 ? tiles : 65535));
    if (af == K3G_MXFP4)
        mx_stream_kernel<K3G_MXFP4, MODE><<<grid, kStreamWaves * kWave, 0, st>>>(a);
    else
        mx_stream_kernel<K3G_MXFP8, MODE><<<grid, kStreamWaves * kWave, 0, st>>>(a);
    return hipGetLastError() == hipSuccess ? K3G_OK : K3G_EHIP;
}

// ---- host ----------------------------------------------------------------------------

namespace {

constexpr int kMaxExperts = 2048;

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
    if (!mx_aligned(w, 16) || b.stride % 16) return K3G_EALIGN;
    a->w[slot] = w;
    a->ws[slot] = s;
    const int64_t last = (b.n_experts - 1) * b.stride;
    covers[0] = {(uintptr_t)w, (uintptr_t)w + last + (size_t)d.rows * d.in / 2};
    covers[1] = {(uintptr_t)s, (uintptr_t)s + last + (size_t)d.rows * (d.in / kGroup)};
    return K3G_OK;
}

// What the two grouped calls check alike.
int groups_ok(const k3g_mx *a, const int32_t *offsets, const int32_t *perm, int top_k, int n_rows) {
    if (!offsets) return K3G_EINVAL;
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
    return launch_stream<DENSE>(m, a->format, (hipStream_t)stream);
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
    K3G_TRY(groups_ok(a, offsets, perm, top_k, n_rows));
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
    return launch_stream<GROUPED>(m, a->format, (hipStream_t)stream);
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
    K3G_TRY(groups_ok(a, offsets, perm, top_k, n_rows));
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
    return launch_stream<GLU>(m, a->format, (hipStream_t)stream);
}

}  // extern "C"
