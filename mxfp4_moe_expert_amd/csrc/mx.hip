// mx.hip -- microscaled activations: the quantiser to MXFP4 and MXFP8 rows,
// the way back, and the residual + RMS norm that writes them.
//
// A group of 32 entries with largest magnitude m gets the scale 2^e, e the
// smallest exponent with m <= M 2^e (M = 6 for e2m1, 448 for e4m3), and the
// codes RNE(v / 2^e). Powers of two make the division exact, so the rounding
// to a code is the only one. All three kernels are bound by HBM: each entry is
// read once and written once.
#include "mx.h"

namespace k3g {

// The largest of a quad of lanes' magnitude bits (unsigned: a NaN is above an
// infinity is above every finite magnitude, so nothing non-finite is lost).
__device__ inline uint32_t quad_max(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
    return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
}

// Four lanes hold a group, eight entries each (v); lane j of the quad writes
// its codes, lane 0 the scale byte.
template <int FMT>
__device__ inline void quantize_quad(const float *v, uint8_t *codes, uint8_t *scale, int j, bool live) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
    m = quad_max(m);
    const bool fine = m < kMxNotFinite;
    const int e = fine ? mx_exponent<FMT>(m) : 0;
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = fine ? v[i] : 0.0f;
    uint32_t w[2];
    mx_codes8<FMT>(u, pow2(e), w);
    if (!live) return;
    if constexpr (FMT == K3G_MXFP4)
        *(uint32_t *)(codes + 4 * j) = w[0];
    else
        *(uint2 *)(codes + 8 * j) = make_uint2(w[0], w[1]);
    if (j == 0) *scale = fine ? (uint8_t)(e + 127) : (uint8_t)255;
}

// 64 groups a workgroup, in row order over the whole matrix: a wavefront reads 1 or
// 2 KB in a row. 8191 fp32 rows of 3584 to MXFP8: 25 us, 6.0 TB/s; one row of 7168
// 2 us, the launch.
template <int TYPE, int FMT>
__global__ __launch_bounds__(256) void mx_quantize_kernel(uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                                                          const typename Elem<TYPE>::T *__restrict__ x,
                                                          int64_t stride, int64_t n_groups, int G) {
    const int64_t first = (int64_t)blockIdx.x * 64;
    const int64_t row0 = first / G;  // uniform
    const uint32_t g0 = (uint32_t)(first - row0 * G) + threadIdx.x / 4;
    const int64_t row = row0 + g0 / (uint32_t)G;
    const int g = (int)(g0 % (uint32_t)G), j = threadIdx.x & 3;
    const int64_t group = first + threadIdx.x / 4;
    const bool live = group < n_groups;
    float v[8] = {};
    if (live) load_n<TYPE, 8>(v, x + row * stride + g * kGroup + 8 * j);
    quantize_quad<FMT>(v, codes + group * (FMT == K3G_MXFP4 ? 16 : 32), scales + group, j, live);
}

// As the quantiser. The same rows, MXFP8 to bf16: 15 us, 5.9 TB/s.
template <int TYPE, int FMT>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(typename Elem<TYPE>::T *__restrict__ y, int64_t stride,
                                                            const uint8_t *__restrict__ codes,
                                                            const uint8_t *__restrict__ scales, int64_t n_groups,
                                                            int G) {
    const int64_t first = (int64_t)blockIdx.x * 64;
    const int64_t row0 = first / G;
    const uint32_t g0 = (uint32_t)(first - row0 * G) + threadIdx.x / 4;
    const int64_t row = row0 + g0 / (uint32_t)G;
    const int g = (int)(g0 % (uint32_t)G), j = threadIdx.x & 3;
    const int64_t group = first + threadIdx.x / 4;
    if (group >= n_groups) return;
    const uint32_t s = scales[group];
    float v[8];
    if constexpr (FMT == K3G_MXFP4) {
        const uint32_t w = *(const uint32_t *)(codes + group * 16 + 4 * j);
        const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
        const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
        const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
        const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
        v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1], v[4] = c[0], v[5] = c[1], v[6] = d[0], v[7] = d[1];
    } else {
        const uint2 w = *(const uint2 *)(codes + group * 32 + 8 * j);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t d = k ? w.y : w.x;
            const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(d, 1.0f, false);
            const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(d, 1.0f, true);
            v[4 * k] = a[0], v[4 * k + 1] = a[1], v[4 * k + 2] = b[0], v[4 * k + 3] = b[1];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = apply_scale(v[i], s);
    store_n<TYPE, 8>(y + row * stride + g * kGroup + 8 * j, v);
}

// v * (hi + lo) * g as a sum of two floats, to about 46 bits: `near` is the nearest
// float, `odd` the sum cut towards zero with the last bit set where anything was cut
// off. A second rounding of `odd` to fewer bits (a code, a bf16) is then the rounding
// of the product itself, never that of a tie that the first rounding made. (What the
// two products leave, p_lo, can pass an ulp of p: the two are added before the cut.)
struct Scaled {
    float near, odd;
};
__device__ inline Scaled scaled(float v, float hi, float lo, float g) {
#pragma clang fp contract(off)  // p is the rounded product wherever it stands
    const float s = g * hi, s_lo = __builtin_fmaf(g, lo, __builtin_fmaf(g, hi, -s));
    const float p = v * s, p_lo = __builtin_fmaf(v, s_lo, __builtin_fmaf(v, s, -p));
    // of an infinite or NaN p, p_lo is no number (0x1F8: finite)
    const float near = __builtin_amdgcn_classf(p_lo, 0x1F8) ? p + p_lo : p, rest = p_lo - (near - p);
    // what is left has near's sign: near with its last bit set; else one below near in magnitude
    const uint32_t u = __builtin_bit_cast(uint32_t, near), w = __builtin_bit_cast(uint32_t, rest);
    const uint32_t odd = (u + (uint32_t)((int32_t)(u ^ w) >> 31)) | 1u;
    // 0x198: a number other than zero
    return {near, __builtin_amdgcn_classf(rest, 0x198) ? __builtin_bit_cast(float, odd) : near};
}

// One workgroup a row, its entries in registers between the sum of squares and
// the scaling: thread c holds entries 8(c + k * threads) .. + 7, k < NC, so a
// quad of lanes holds a group and a wavefront 2 KB of fp32.
struct NormArgs {
    void *y, *sum;
    const void *x, *r;
    int64_t ys, ss, xs, rs;
    uint8_t *codes, *scales;
    const float *gamma;
    float eps;
    int in;
    double inv_in;  // 1 / in
    int64_t row0;   // the launch's first row
};

template <int TYPE, int FMT, int NC>  // FMT -1: no quantised output
__global__ __launch_bounds__(1024) void add_rmsnorm_kernel(NormArgs a) {
    typedef typename Elem<TYPE>::T T;
    __shared__ double part[16];
    const int64_t row = a.row0 + blockIdx.x;
    const int in = a.in, nt = blockDim.x;
    const T *x = (const T *)a.x + row * a.xs;
    const T *r = a.r ? (const T *)a.r + row * a.rs : nullptr;
    float v[NC][8];
    double ss = 0.;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = 8 * ((int)threadIdx.x + k * nt);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = 0.f;
        if (c < in) {
            load_n<TYPE, 8>(v[k], x + c);
            if (r) {
                float b[8];
                load_n<TYPE, 8>(b, r + c);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] += b[i];
            }
            if (a.sum) store_n<TYPE, 8>((T *)a.sum + row * a.ss + c, v[k]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fma((double)v[k][i], (double)v[k][i], ss);
    }
    // The sum of squares and the row's scale in 64 bits, and each n to about 46 (a product
    // of two pairs of floats): an n that fp32 had rounded might cross the border between two
    // codes. The row's bytes take longer.
    const double wave_ss = wave_sum_f64(ss);
    if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = wave_ss;
    __syncthreads();
    double tot = 0.;
    for (int w = 0; w < nt / kWave; ++w) tot += part[w];
    // 1/sqrt by the 64-bit instruction (2^-24) and one Newton step (2^-47); of a mean of zero
    // or infinity, where the step is a NaN, the instruction's answer. It may lie past fp32's
    // ends on either side, and so may its product with gamma: its power of two goes to the
    // entries, which it brings to about 1, and s, hi and lo keep all their bits.
    const double m = tot * a.inv_in + (double)a.eps, r0 = __builtin_amdgcn_rsq(m);
    const double e = __builtin_fma(-m * r0, r0, 1.0), inv = e == e ? __builtin_fma(0.5 * r0, e, r0) : r0;
    const int up = __builtin_amdgcn_frexp_exp(inv);  // inv in [2^(up-1), 2^up); of 0, infinity or NaN 0
    const double unit = __builtin_ldexp(inv, -up);
    const float inv_hi = (float)unit, inv_lo = (float)(unit - (double)inv_hi);
    const int G = in / kGroup;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = 8 * ((int)threadIdx.x + k * nt);
        const bool live = c < in;
        if (live) {
            float gm[8];
            load_n<K3G_F32, 8>(gm, a.gamma + c);
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const Scaled n = scaled(__builtin_ldexpf(v[k][i], up), inv_hi, inv_lo, gm[i]);
                v[k][i] = n.odd;
                y[i] = TYPE == K3G_F32 ? n.near : n.odd;
            }
            if (a.y) store_n<TYPE, 8>((T *)a.y + row * a.ys + c, y);
        }
        if constexpr (FMT >= 0)
            quantize_quad<FMT>(v[k], a.codes + (row * G + c / kGroup) * (FMT == K3G_MXFP4 ? 16 : 32),
                               a.scales + row * G + c / kGroup, threadIdx.x & 3, live);
    }
}

// Threads a row: with rows to fill the chip many times over, up to 512 (several
// workgroups on a CU hide each other's waits: 8192 bf16 rows of 7168 in 83-90 us, 4.6-5.0
// TB/s; 3% more with 896 threads a row, 8% with 256); with few rows, eight entries a thread.
template <int TYPE, int FMT>
int launch_norm(NormArgs a, int n_rows, hipStream_t st) {
    const int chunks = a.in / 8, wide = n_rows >= 1024 ? 512 : 1024;
    const int nc = chunks <= wide ? 1 : chunks <= 2 * wide ? 2 : chunks <= 4 * wide ? 4 : 8;
    const int nt = ((chunks + nc - 1) / nc + kWave - 1) / kWave * kWave;
    const int64_t most = ((int64_t)1 << 31) / nt;  // a launch's threads are counted in 32 bits
    for (a.row0 = 0; a.row0 < n_rows; a.row0 += most) {
        const unsigned rows = (unsigned)(n_rows - a.row0 < most ? n_rows - a.row0 : most);
        if (nc == 1)
            add_rmsnorm_kernel<TYPE, FMT, 1><<<rows, nt, 0, st>>>(a);
        else if (nc == 2)
            add_rmsnorm_kernel<TYPE, FMT, 2><<<rows, nt, 0, st>>>(a);
        else if (nc == 4)
            add_rmsnorm_kernel<TYPE, FMT, 4><<<rows, nt, 0, st>>>(a);
        else
            add_rmsnorm_kernel<TYPE, FMT, 8><<<rows, nt, 0, st>>>(a);
        if (hipGetLastError() != hipSuccess) return K3G_EHIP;
    }
    return K3G_OK;
}

template <int TYPE>
int norm_fmt(const NormArgs &a, int fmt, int n_rows, hipStream_t st) {
    if (fmt == K3G_MXFP4) return launch_norm<TYPE, K3G_MXFP4>(a, n_rows, st);
    if (fmt == K3G_MXFP8) return launch_norm<TYPE, K3G_MXFP8>(a, n_rows, st);
    return launch_norm<TYPE, -1>(a, n_rows, st);
}

// Four threads a group, and a launch's threads are counted in 32 bits.
int launch_ok(const k3g_mx &q) {
    return (int64_t)q.rows * (q.in / kGroup) > ((int64_t)1 << 30) - 64 ? K3G_EUNSUPPORTED : K3G_OK;
}

template <int FMT>
int launch_quantize(const k3g_mx &q, const void *x, int type, int64_t stride, hipStream_t st) {
    const int G = q.in / kGroup;
    const int64_t n = (int64_t)q.rows * G;
    const dim3 grid((unsigned)((n + 63) / 64));
    if (type == K3G_F32)
        mx_quantize_kernel<K3G_F32, FMT><<<grid, 256, 0, st>>>(q.codes, q.scales, (const float *)x, stride, n, G);
    else if (type == K3G_BF16)
        mx_quantize_kernel<K3G_BF16, FMT><<<grid, 256, 0, st>>>(q.codes, q.scales, (const __bf16 *)x, stride, n, G);
    else
        mx_quantize_kernel<K3G_F16, FMT><<<grid, 256, 0, st>>>(q.codes, q.scales, (const _Float16 *)x, stride, n, G);
    return hipGetLastError() == hipSuccess ? K3G_OK : K3G_EHIP;
}

template <int FMT>
int launch_dequantize(void *y, int type, int64_t stride, const k3g_mx &q, hipStream_t st) {
    const int G = q.in / kGroup;
    const int64_t n = (int64_t)q.rows * G;
    const dim3 grid((unsigned)((n + 63) / 64));
    if (type == K3G_F32)
        mx_dequantize_kernel<K3G_F32, FMT><<<grid, 256, 0, st>>>((float *)y, stride, q.codes, q.scales, n, G);
    else if (type == K3G_BF16)
        mx_dequantize_kernel<K3G_BF16, FMT><<<grid, 256, 0, st>>>((__bf16 *)y, stride, q.codes, q.scales, n, G);
    else
        mx_dequantize_kernel<K3G_F16, FMT><<<grid, 256, 0, st>>>((_Float16 *)y, stride, q.codes, q.scales, n, G);
    return hipGetLastError() == hipSuccess ? K3G_OK : K3G_EHIP;
}

}  // namespace k3g

using namespace k3g;

extern "C" {

int k3g_mx_quantize(const k3g_mx *q, const void *x, int x_type, int64_t x_stride, void *stream) {
    K3G_TRY(mx_ok(q));
    if (!type_ok(x_type) || x_stride < q->in) return K3G_EINVAL;
    if (q->rows == 0) return K3G_OK;
    K3G_TRY(launch_ok(*q));
    K3G_TRY(dense_ok(x, x_type, x_stride, q->in));
    const Span xs = rows_span(x, x_type, q->rows, x_stride, q->in);
    if (meet(xs, codes_span(*q)) || meet(xs, scales_span(*q)) || meet(codes_span(*q), scales_span(*q)))
        return K3G_EINVAL;
    K3G_TRY(device_ok());
    return q->format == K3G_MXFP4 ? launch_quantize<K3G_MXFP4>(*q, x, x_type, x_stride, (hipStream_t)stream)
                                  : launch_quantize<K3G_MXFP8>(*q, x, x_type, x_stride, (hipStream_t)stream);
}

int k3g_mx_dequantize(void *y, int y_type, int64_t y_stride, const k3g_mx *q, void *stream) {
    K3G_TRY(mx_ok(q));
    if (!type_ok(y_type) || y_stride < q->in) return K3G_EINVAL;
    if (q->rows == 0) return K3G_OK;
    K3G_TRY(launch_ok(*q));
    K3G_TRY(dense_ok(y, y_type, y_stride, q->in));
    const Span ys = rows_span(y, y_type, q->rows, y_stride, q->in);
    if (meet(ys, codes_span(*q)) || meet(ys, scales_span(*q))) return K3G_EINVAL;
    K3G_TRY(device_ok());
    return q->format == K3G_MXFP4 ? launch_dequantize<K3G_MXFP4>(y, y_type, y_stride, *q, (hipStream_t)stream)
                                  : launch_dequantize<K3G_MXFP8>(y, y_type, y_stride, *q, (hipStream_t)stream);
}

int k3g_add_rmsnorm(void *y, int64_t y_stride, void *sum, int64_t sum_stride, const k3g_mx *q, const void *x,
                    int64_t x_stride, const void *r, int64_t r_stride, int type, const float *gamma, float eps,
                    int n_rows, int in, void *stream) {
    if (n_rows < 0 || in <= 0 || in % kGroup || !type_ok(type) || !(eps >= 0.0f) || !isfinite(eps)) return K3G_EINVAL;
    if (in > kMxMaxIn) return K3G_EUNSUPPORTED;
    if (q) {
        K3G_TRY(mx_ok(q));
        if (q->rows != n_rows || q->in != in) return K3G_EINVAL;
    }
    if (n_rows == 0) return K3G_OK;
    if ((!y && !q) || !gamma) return K3G_EINVAL;
    if (!mx_aligned(gamma, 4)) return K3G_EALIGN;
    K3G_TRY(dense_ok(x, type, x_stride, in));
    if (r) K3G_TRY(dense_ok(r, type, r_stride, in));
    if (y) K3G_TRY(dense_ok(y, type, y_stride, in));
    if (sum) K3G_TRY(dense_ok(sum, type, sum_stride, in));
    // a thread reads its entries of x and r before it writes the same entries
    // of sum and y, so an output may be an input itself, and nothing else
    const Span ins[] = {rows_span(x, type, n_rows, x_stride, in), rows_span(r, type, n_rows, r_stride, in),
                        span(gamma, 4 * (size_t)in)};
    const Span ys = rows_span(y, type, n_rows, y_stride, in), ss = rows_span(sum, type, n_rows, sum_stride, in);
    const bool y_is_x = y == x && y_stride == x_stride, y_is_r = y && y == r && y_stride == r_stride;
    const bool s_is_x = sum == x && sum_stride == x_stride, s_is_r = sum && sum == r && sum_stride == r_stride;
    if ((meet(ys, ins[0]) && !y_is_x) || (meet(ys, ins[1]) && !y_is_r) || meet(ys, ins[2])) return K3G_EINVAL;
    if ((meet(ss, ins[0]) && !s_is_x) || (meet(ss, ins[1]) && !s_is_r) || meet(ss, ins[2])) return K3G_EINVAL;
    if (meet(ys, ss)) return K3G_EINVAL;
    if (q) {
        const Span cs = codes_span(*q), sc = scales_span(*q);
        if (meet(cs, sc) || meet(cs, ys) || meet(cs, ss) || meet(sc, ys) || meet(sc, ss)) return K3G_EINVAL;
        for (const Span &i : ins)
            if (meet(cs, i) || meet(sc, i)) return K3G_EINVAL;
    }
    K3G_TRY(device_ok());
    const NormArgs a = {y,        sum,      x,        r,          y_stride,  sum_stride, x_stride,
                        r_stride, q ? q->codes : nullptr, q ? q->scales : nullptr, gamma, eps, in,
                        1.0 / in, 0};
    const int fmt = q ? q->format : -1;
    hipStream_t st = (hipStream_t)stream;
    return type == K3G_F32    ? norm_fmt<K3G_F32>(a, fmt, n_rows, st)
           : type == K3G_BF16 ? norm_fmt<K3G_BF16>(a, fmt, n_rows, st)
                              : norm_fmt<K3G_F16>(a, fmt, n_rows, st);
}

}  // extern "C"
