// int4.hip -- products with int4 weights: the calls, their checks, and which
// kernels they run on.
#include "int4_stream.h"
#include "int4_tile.h"

using namespace k3g;

namespace {

constexpr int kMaxExperts = 2048;
constexpr int kMaxRows = 1 << 30;  // tiles are counted in 32 bits

// The matrices as the kernels' operand `slot`, and the addresses they cover.
int use_int4(I4Args *a, int slot, const k3g_int4 *w, Span *covers) {
    if (!w || w->n_experts < 1 || w->rows < 1 || w->in < 1 || (w->group != 32 && w->group != 64 && w->group != 128) ||
        w->in % w->group || !type_ok(w->scale_type))
        return K3G_EINVAL;
    if (w->n_experts > kMaxExperts || w->rows > kMaxRows || w->in > kMxMaxIn) return K3G_EUNSUPPORTED;
    if (!w->packed || !w->scales) return K3G_EINVAL;
    if (!mx_aligned(w->packed, 16) || !mx_aligned(w->scales, type_size(w->scale_type))) return K3G_EALIGN;
    const size_t rows = (size_t)w->n_experts * w->rows, groups = rows * (w->in / w->group);
    covers[0] = span(w->packed, rows * (w->in / 2));
    covers[1] = span(w->scales, groups * type_size(w->scale_type));
    covers[2] = span(w->zeros, w->zeros ? groups : 0);
    a->w[slot] = w->packed, a->s[slot] = w->scales, a->z[slot] = w->zeros;
    a->rows = w->rows, a->in = w->in, a->G = w->in / w->group, a->E = w->n_experts, a->s_type = w->scale_type;
    return K3G_OK;
}

// The kernel of a product: weight rows << 16 | tokens of its tile; the vector kernel's is 8 << 16 | 1.
//
// Figures are us, of groups of 64 with zeros and fp32 in brackets where nothing else is said; "experts" are 256 of
// 3584 x 3584 whose rows are spread evenly, by their average rows. Every border was measured on all three groups.
//
// A single row runs on the vector units, and so do two of fp32, and rows of experts, a workgroup's row each, where
// few experts would have two (vector, streamed). One token 7168 -> 3584 9.9, 9.4 (9.9, 16; groups of 32 10.3,
// 11.1), two 12, 9.6 (12, 16), three 16, 9.7 (16.2, 16.6). Experts, 64 rows in all 106, 110 (106, 191), 128 182,
// 182 (182, 322), 192 266, 221, 256 337, 257 (337, 461); groups of 32 128 rows 186, 257, of 128 180, 173; one
// token's 16 of 3584 x 3072, gated, 40, 60. It reads a matrix once a row, so it loses where rows crowd: on a
// routing that prefers some experts (the 16 best of scores some of which are higher) 64 rows 103, 99, 128 180, 163
// (179, 280), 256 rows of 896 experts of 3584 x 3072 296, 251; 128 rows on 8 experts 143, 34, 256 on 8 (268, 73).
// More than 256 rows are streamed.
//
// Tiles of 256 outputs pay where rows are many and items enough to fill half of the chip (streamed, tiled; items
// of 128 tokens, fp32 64). 3584 -> 7168, 512 tokens (112 items) 91, 95, 1024 (224) 151, 95; 7168 -> 3584, 1024
// (112) 149, 180, 1536 (168) 213, 181; groups of 32 1536 tokens 240, 222, 2048 278, 222. fp32 512 tokens (112)
// 156, 218, 1024 (224) 262, 222. Rows off 16-byte addresses take fp32's tile and border: 1024 tokens 137, 170,
// 2048 222, 226, 4096 436, 447, so their tile, whose staged rows lie in scratch memory, does not pay yet. Experts:
// 16 rows 611, 654, 20 667, 661, 32 914, 696; fp32 32 rows 1524, 1456, 48 2071, 1720, 64 2499, 2438, 80 3118,
// 3232, 96 3653, 3214, 128 4673, 3991 (groups of 48 rows take one tile of 64, of 80 two: the border leaves 48 rows
// a sixth slower than they could be).
//
// Streamed, 64 outputs by 32 tokens, or 32 by 16 where half a tile would be empty or where those are at most two
// workgroups a CU, which run at once (32 x 16 first): 7168 -> 3584, 64 tokens (448 workgroups) 22, 27 (36, 40), 80
// (560) 30, 25 (50, 37); 3584 -> 7168, 32 (448) 14, 17 (21, 26), 33 (672) 17, 16 (26, 25); 4096 -> 1024, 128 (256)
// 8.7, 16 (13, 24); 3584 -> 14336, 16 (448) 15, 16 (22, 21), 17 23, 18 (36, 26). Experts: 12 rows 541, 585, 13
// 577, 588, 14 612, 596; fp32 6 rows 813, 753, 8 826, 780, groups of 128 8 rows 813, 850, 12 863, 913. Up to 16
// tokens of few outputs take 16 a workgroup (16 x 16, 32 x 16): 7168 -> 3584 12, 15 (19, 23); 3584 -> 7168 11.4,
// 9.9 (18, 14). Where 64 x 32 would be more than a workgroup a CU, bf16 and fp16 take 64 x 64 (64 x 32 first):
// 7168 -> 3584, 128 tokens (224) 27, 40, 192 (336) 48, 39, 512 93, 74; 3584 -> 7168, 64 tokens (224) 17, 26, 128
// (448) 30, 25.
int product_form(const I4Args &a, int mode, int x_type) {
    const bool f32 = x_type == K3G_F32;
    const bool spread = a.T <= 256 && (f32 ? a.T : 2 * a.T) <= a.E && (int64_t)a.rows * a.T <= kMaxRows;
    if (a.in <= kGvMaxIn && (a.T == 1 || (mode == DENSE ? f32 && a.T == 2 : spread))) {
        const GvGrid g = gemv_grid(a, mode);
        if (g.workgroups * g.waves * kWave < (int64_t)1 << 32) return form(8, 1);  // (a launch's limit)
    }
    const bool wide = !f32 && a.x_vec;
    const int64_t n = mode == DENSE ? a.T : ((int64_t)a.T + a.E - 1) / a.E, most = wide ? 128 : 64;
    const int64_t tiles = mode == DENSE ? (n + most - 1) / most : (n + most - 1) / most * (a.E < a.T ? a.E : a.T);
    const int64_t items = ((int64_t)a.rows + 255) / 256 * tiles * (mode == GLU ? 2 : 1);
    if (n > (wide ? 20 : 80) && items >= (wide ? 128 : 160)) return wide ? form(256, 128) : form(256, 64);
    if (mode == DENSE && a.T <= 16 && a.rows <= 16 * 256) return form(16, 16);
    const bool few = mode == DENSE ? n <= 16 || ((int64_t)a.rows + 31) / 32 * ((n + 15) / 16) <= 512 : n <= (f32 ? 8 : 12);
    if (few) return form(32, 16);
    return mode == DENSE && !f32 && (a.rows + 63) / 64 * ((n + 31) / 32) > 256 ? form(64, 64) : form(64, 32);
}

int launch(I4Args &a, int mode, int x_type, int group, void *stream) {
    hipStream_t st = (hipStream_t)stream;
    a.x_vec = mx_aligned(a.x, 16) && (a.xs * type_size(x_type) % 16 == 0 || a.x_rows == 1);
    const int f = product_form(a, mode, x_type);
    if (f == form(8, 1)) return launch_int4_gemv(a, mode, x_type, group, st);
    if (f >> 16 <= 64)
        return x_type == K3G_F32    ? launch_int4_stream_f32(a, mode, group, f, st)
               : x_type == K3G_BF16 ? launch_int4_stream_bf16(a, mode, group, f, st)
                                    : launch_int4_stream_f16(a, mode, group, f, st);
    return x_type == K3G_F32    ? launch_int4_tile_f32(a, mode, group, f, st)
           : x_type == K3G_BF16 ? launch_int4_tile_bf16(a, mode, group, f, st)
                                : launch_int4_tile_f16(a, mode, group, f, st);
}

// The grouped calls' checks of everything but the weights; n_w spans of those in `use`.
int groups(I4Args *a, void *y, int y_type, int64_t y_stride, const void *x, int x_type, int64_t x_stride, int x_rows,
           const int32_t *offsets, const int32_t *perm, int top_k, int n_rows, const Span *use, int n_w) {
    if (!offsets || x_rows < 1 || (!perm && x_rows < n_rows)) return K3G_EINVAL;
    if (!mx_aligned(offsets, 4) || !mx_aligned(perm, 4)) return K3G_EALIGN;
    K3G_TRY(dense_ok(y, y_type, y_stride, a->rows));
    K3G_TRY(dense_ok(x, x_type, x_stride, a->in));
    const Span out = rows_span(y, y_type, n_rows, y_stride, a->rows);
    for (int i = 0; i < n_w; ++i)
        if (meet(out, use[i])) return K3G_EINVAL;
    if (meet(out, rows_span(x, x_type, x_rows, x_stride, a->in)) || meet(out, span(offsets, 4 * ((size_t)a->E + 1))) ||
        (perm && meet(out, span(perm, 4 * (size_t)n_rows))))
        return K3G_EINVAL;
    K3G_TRY(device_ok());
    a->x = x, a->xs = x_stride, a->x_rows = x_rows, a->offsets = offsets, a->perm = perm, a->top_k = top_k;
    a->y = y, a->ys = y_stride, a->y_type = y_type, a->T = n_rows;
    return K3G_OK;
}

}  // namespace

extern "C" {

int k3g_int4_matmul(void *y, int y_type, int64_t y_stride, const void *x, int x_type, int64_t x_stride, int n_tokens,
                    const k3g_int4 *w, void *stream) {
    I4Args a = {};
    Span use[3];
    K3G_TRY(use_int4(&a, 0, w, use));
    if (w->n_experts != 1 || n_tokens < 0 || !type_ok(y_type) || !type_ok(x_type) || y_stride < w->rows || x_stride < w->in)
        return K3G_EINVAL;
    if (n_tokens > kMaxRows) return K3G_EUNSUPPORTED;
    if (n_tokens == 0) return K3G_OK;
    K3G_TRY(dense_ok(y, y_type, y_stride, w->rows));
    K3G_TRY(dense_ok(x, x_type, x_stride, w->in));
    const Span out = rows_span(y, y_type, n_tokens, y_stride, w->rows);
    for (const Span &s : use)
        if (meet(out, s)) return K3G_EINVAL;
    if (meet(out, rows_span(x, x_type, n_tokens, x_stride, w->in))) return K3G_EINVAL;
    K3G_TRY(device_ok());
    a.x = x, a.xs = x_stride, a.x_rows = n_tokens, a.y = y, a.ys = y_stride, a.y_type = y_type, a.T = n_tokens;
    return launch(a, DENSE, x_type, w->group, stream);
}

int k3g_int4_grouped_matmul(void *y, int y_type, int64_t y_stride, const void *x, int x_type, int64_t x_stride, int x_rows,
                            const k3g_int4 *w, const int32_t *offsets, const int32_t *perm, int top_k, int n_rows,
                            void *stream) {
    I4Args a = {};
    Span use[3];
    K3G_TRY(use_int4(&a, 0, w, use));
    if (n_rows < 0 || x_rows < 0 || top_k < 1 || !type_ok(y_type) || !type_ok(x_type) || y_stride < w->rows ||
        x_stride < w->in)
        return K3G_EINVAL;
    if (n_rows > kMaxRows || x_rows > kMaxRows) return K3G_EUNSUPPORTED;
    if (n_rows == 0) return K3G_OK;
    K3G_TRY(groups(&a, y, y_type, y_stride, x, x_type, x_stride, x_rows, offsets, perm, top_k, n_rows, use, 3));
    return launch(a, GROUPED, x_type, w->group, stream);
}

int k3g_int4_grouped_glu(void *h, int h_type, int64_t h_stride, const void *x, int x_type, int64_t x_stride, int x_rows,
                         const k3g_int4 *w1, const k3g_int4 *w3, const int32_t *offsets, const int32_t *perm, int top_k,
                         int n_rows, void *stream) {
    I4Args a = {};
    Span use[6];
    K3G_TRY(use_int4(&a, 0, w1, use));
    K3G_TRY(use_int4(&a, 1, w3, use + 3));
    if (w1->n_experts != w3->n_experts || w1->rows != w3->rows || w1->in != w3->in || w1->group != w3->group ||
        w1->scale_type != w3->scale_type || n_rows < 0 || x_rows < 0 || top_k < 1 || !type_ok(h_type) ||
        !type_ok(x_type) || h_stride < w1->rows || x_stride < w1->in)
        return K3G_EINVAL;
    if (n_rows > kMaxRows || x_rows > kMaxRows) return K3G_EUNSUPPORTED;
    if (n_rows == 0) return K3G_OK;
    K3G_TRY(groups(&a, h, h_type, h_stride, x, x_type, x_stride, x_rows, offsets, perm, top_k, n_rows, use, 6));
    return launch(a, GLU, x_type, w1->group, stream);
}

int k3g_probe_int4_form(int x_type, int aligned, int kind, int n_rows, int rows, int in, int n_experts) {
    if (!type_ok(x_type) || kind < DENSE || kind > GLU || n_rows < 1 || rows < 1 || in < 32 || in % 32 || in > kMxMaxIn ||
        n_rows > kMaxRows || rows > kMaxRows || (kind != DENSE && (n_experts < 1 || n_experts > kMaxExperts)))
        return K3G_EINVAL;
    I4Args a = {};
    a.T = n_rows, a.rows = rows, a.in = in, a.E = n_experts, a.x_vec = aligned != 0;
    return product_form(a, kind, x_type);
}

int k3g_probe_int4_launch(int x_type, int aligned, int kind, int n_rows, int rows, int in, int n_experts, int group) {
    const int f = k3g_probe_int4_form(x_type, aligned, kind, n_rows, rows, in, n_experts);
    if (f < 0) return f;
    if ((group != 32 && group != 64 && group != 128) || in % group) return K3G_EINVAL;
    I4Args a = {};
    a.T = n_rows, a.rows = rows, a.in = in, a.E = n_experts;
    const Int4Grid g = f == form(8, 1) ? gemv_grid(a, kind) : f >> 16 <= 64 ? stream_grid(a, kind, group, f) : tile_grid(a, kind, f);
    return (int)(g.workgroups << 4) | g.waves;
}

}  // extern "C"
