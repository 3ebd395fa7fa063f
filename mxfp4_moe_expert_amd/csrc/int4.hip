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
// A single row runs on the vector units, and so do two of fp32, and rows of experts, a workgroup's row each, where
// few experts would have two (us; vector, streamed): one bf16 token 7168 -> 3584 8.6, 9.4; two 9.7, 9.5, fp32 9.8, 16, three
// 15, 16. Of 256 experts of 3584 x 3584, groups of 32, 64 rows 91, 132, 128 rows 149, 215, 256 286, 307 (groups of 128 145, 173
// by 128, 213, 205 by 192); fp32 128 rows 150, 351, 256 279, 483. More than 256 rows are streamed: rows that crowd
// on one expert cost this kernel what rows of many do.
//
// Tiles of 256 outputs pay where rows are many and items enough to fill half of the chip (streamed, tiled): bf16 3584
// -> 7168, 512 tokens (112 items) 100, 100, 1024 tokens (224) 182, 102; 7168 -> 3584, 1024 tokens (112) 138, 185, 1536
// (168) 207, 184.
// fp32 (64 tokens a tile) 7168 -> 3584, 512 tokens (112) 144, 219, 1024 (224) 253, 222. Grouped, by the average rows of the
// bank's experts: 256 of 3584 x 3584, bf16, 16 rows 584, 623, 32 rows 873, 698; fp32 64 rows 635, 684, 128 rows 1133, 1025.
//
// Streamed, 64 outputs by 32 tokens, or 32 by 16 where half a tile would be empty or where those are at most two
// workgroups a CU, which run at once (32 x 16 first; bf16, fp32 in brackets): 7168 -> 3584, 64 tokens (448) 23, 31 (34, 40),
// 80 (560) 33, 28 (50, 37); 3584 -> 7168, 32 (448) 15, 20 (21, 26), 33 (672) 20, 18 (27, 25); 4096 -> 1024, 128 (256) 9.7, 17
// (14, 25); 3584 -> 14336, 16 (448) 15, 18 (21, 21), 17 23, 20 (36, 26). Grouped, 256 of 3584 x 3584, 9 rows 575, 650 (896,
// 799), 11 rows 591, 659, 14 rows 694, 696; fp32 8 rows 837, 890. Up to 16 tokens of few outputs take 16 a workgroup: 7168 ->
// 3584, 16 tokens 13, 16; 3584 -> 7168 12, 11. Where
// 64 x 32 would be more than a workgroup a CU, bf16 and fp16 take 64 x 64: 7168 -> 3584, 128 tokens (224) 25, 39, 192 47,
// 38, 512 91, 71; 3584 -> 7168, 64 tokens (224) 20, 29, 128 36, 29 (fp32 49, 55; 512 tokens 162, 206).
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
