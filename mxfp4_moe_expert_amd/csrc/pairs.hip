// pairs.hip -- a batch's routed pairs (token t, slot k) sorted by expert, rows
// gathered into that order and summed back, and the gradients of both.
//
// inv[t][k] is the sorted row of pair t*top_k+k, or -1. With w = 1 where no
// weights are given, and rows of a pair that has no sorted row left out:
//   gather            ys[inv[t][k]] = w[t][k] x[t]
//   combine           y[t] = sum_k w[t][k] ys[inv[t][k]]
// The two are each other's transpose, so a gradient is the other map and a dot
// product for the weights:
//   gather_backward   dx[t] = sum_k w[t][k] dys[inv[t][k]],  dw[t][k] = <x[t], dys[inv[t][k]]>
//   combine_backward  dys[inv[t][k]] = w[t][k] dy[t],        dw[t][k] = <dy[t], ys[inv[t][k]]>
// One kernel does all four, token by token: each sorted row belongs to one pair,
// so nothing is added by two workgroups and results do not depend on timing. HBM
// bounds it at a prompt's size: of 4096 x 16 rows of 3584 bf16, written 84 us (5.4 TB/s),
// summed into fp32 100 us (5.3), summed with the dot products 110 us (4.4), written with the
// dot products 194 us (5.2; 1 GB). Sorted rows are read and written once and are
// more than the caches hold, so they pass them by (written through them 145 us,
// read through them 109 and 114). A batch of 64 tokens takes 5 to 9 us: a launch, and loads
// that wait for each other.
#include "mx.h"

namespace k3g {

constexpr int kSortMaxExperts = 2048;
constexpr int kPairMaxTopK = 64;
constexpr int kSortAlone = 4096;     // pairs that one workgroup sorts in one launch
constexpr int kSortChunk = 2048;     // pairs that a workgroup of several ranks at a time
constexpr int kSortMaxChunks = 256;  // workgroups of a large sort

// ---- sort ------------------------------------------------------------------------
//
// A stable counting sort. A workgroup takes pairs in order, each wavefront a
// contiguous piece of them 64 at a time: the lanes that hold the same expert find
// each other by one ballot a bit of the id, a lane's rank is the number of such
// lanes below it plus what its wavefront has counted for the expert before (16
// bits in LDS, a row of counters a wavefront), and the counters' prefix over the
// wavefronts is added when all have counted. One workgroup does up to 4096 pairs
// in one launch; more are cut into chunks, whose histograms a first launch
// writes and whose starts each workgroup of the second sums up itself.
//
// Latency bounds it: the bytes of 131,056 pairs would take under 1 us. In us, 896
// experts: 1,024 pairs 5.0 (the kernel alone), 4,096 8.7 (by two launches 9.9), 131,056
// 13.3 (chunks of 1,024 14.8, of 4,096 14.3), 960,000 30.

// The chunks of P pairs, and the pairs of each (a multiple of kSortChunk).
int sort_chunks(int64_t P) {
    if (P <= kSortAlone) return 1;
    const int64_t n = (P + kSortChunk - 1) / kSortChunk;
    return n < kSortMaxChunks ? (int)n : kSortMaxChunks;
}
inline int64_t sort_chunk_pairs(int64_t P) {
    const int n = sort_chunks(P);
    return ((P + n - 1) / n + kSortChunk - 1) / kSortChunk * kSortChunk;
}

__global__ __launch_bounds__(1024) void sort_count_kernel(int32_t *__restrict__ counts, const int32_t *__restrict__ idx,
                                                          int P, int E, int per_chunk) {
    __shared__ int32_t n[kSortMaxExperts];
    for (int e = threadIdx.x; e < E; e += 1024) n[e] = 0;
    __syncthreads();
    const int64_t p0 = (int64_t)blockIdx.x * per_chunk, p1 = min(p0 + per_chunk, (int64_t)P);
    for (int64_t p = p0 + threadIdx.x; p < p1; p += 1024) {
        const int e = idx[p];
        if ((unsigned)e < (unsigned)E) atomicAdd(&n[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 1024) counts[(int64_t)blockIdx.x * E + e] = n[e];
}

// The sum of v over the threads below this one; *total the sum over all.
template <int NT>
__device__ inline int block_prefix(int v, int32_t *part, int *total) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    int x = v;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(x, d);
        if (lane >= d) x += o;
    }
    if (lane == kWave - 1) part[wave] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NT / kWave; ++w) {
        before += w < wave ? part[w] : 0;
        all += part[w];
    }
    *total = all;
    return before + x - v;
}

// NT threads, S * NT pairs at a time. counts null: one workgroup, all pairs (P <= S * NT).
template <int NT, int S>
__global__ __launch_bounds__(NT) void sort_kernel(int32_t *__restrict__ offsets, int32_t *__restrict__ perm,
                                                  int32_t *__restrict__ inv, const int32_t *__restrict__ idx,
                                                  const int32_t *__restrict__ counts, int P, int E, int per_chunk) {
    constexpr int W = NT / kWave;
    extern __shared__ __align__(16) int32_t lds[];
    int32_t *next = lds, *sum = next + E, *part = sum + E;  // an expert's next place, its pairs of this turn; scan scratch
    uint16_t *seen = (uint16_t *)(part + W);                 // [W][E]
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int64_t p0 = (int64_t)blockIdx.x * per_chunk, p1 = min(p0 + per_chunk, (int64_t)P);
    const int per = (E + NT - 1) / NT, e0 = min(tid * per, E), e1 = min(e0 + per, E);
    int kept = 0;  // pairs that have an expert
    // From totals in `sum`: the first place of each expert into next, and into offsets.
    auto place = [&](bool write) {
        int n = 0;
        for (int e = e0; e < e1; ++e) n += sum[e];
        int at = block_prefix<NT>(n, part, &kept);
        for (int e = e0; e < e1; ++e) {
            if (write) offsets[e] = at;
            next[e] = at;
            at += sum[e];
        }
        if (write && tid == 0) offsets[E] = kept;
    };
    if (counts) {  // an expert's pairs in all chunks, and in those before this one (two experts a thread at most)
        static_assert(NT < 1024 || kSortMaxExperts <= 2 * NT, "");
        int before[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int e = tid + k * NT;
            if (e >= E) continue;
            int all = 0;
#pragma unroll 16
            for (int c = 0; c < (int)gridDim.x; ++c) {
                const int n = counts[(int64_t)c * E + e];
                all += n;
                before[k] += c < (int)blockIdx.x ? n : 0;
            }
            sum[e] = all;
        }
        __syncthreads();
        place(blockIdx.x == 0);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (tid + k * NT < E) next[tid + k * NT] += before[k];
    }
    int bits = 1;
    while ((1 << bits) < E) ++bits;
    int64_t c0 = p0;
    do {
        __syncthreads();
        for (int i = tid; i < (W * E + 1) / 2; i += NT) ((uint32_t *)seen)[i] = 0u;
        __syncthreads();
        int id[S], rank[S];
        uint16_t *mine = seen + wave * E;
        const int64_t first = c0 + (int64_t)wave * (S * kWave) + lane;
#pragma unroll
        for (int s = 0; s < S; ++s) id[s] = first + s * kWave < p1 ? idx[first + s * kWave] : -1;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const bool valid = (unsigned)id[s] < (unsigned)E;
            uint64_t same = __ballot(valid);
            for (int b = 0; b < bits; ++b) {
                const bool one = (id[s] >> b) & 1;
                const uint64_t m = __ballot(one);
                same &= one ? m : ~m;
            }
            const uint64_t below = same & ((1ull << lane) - 1ull);
            const int n = valid ? mine[id[s]] : 0;
            rank[s] = n + __popcll(below);
            wave_lds_order();  // all lanes of an expert read its counter before the first of them counts on
            if (valid && below == 0) mine[id[s]] = (uint16_t)(n + __popcll(same));
            wave_lds_order();
        }
        __syncthreads();
        for (int e = tid; e < E; e += NT) {
            int n = 0;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const int c = seen[w * E + e];
                seen[w * E + e] = (uint16_t)n;
                n += c;
            }
            sum[e] = n;
        }
        __syncthreads();
        if (!counts) {
            place(true);
            __syncthreads();
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int64_t p = first + s * kWave;
            if (p < p1) {
                int at = -1;
                if ((unsigned)id[s] < (unsigned)E) {
                    at = next[id[s]] + mine[id[s]] + rank[s];
                    perm[at] = (int32_t)p;
                }
                inv[p] = at;
                if (p >= kept) perm[p] = -1;
            }
        }
        __syncthreads();
        for (int e = tid; e < E; e += NT) next[e] += sum[e];
        c0 += S * NT;
    } while (c0 < p1);
}

inline size_t sort_lds_bytes(int E, int waves) { return 4 * (size_t)(2 * E + waves) + 4 * (((size_t)waves * E + 1) / 2); }

template <int NT, int S>
int launch_sort(int32_t *offsets, int32_t *perm, int32_t *inv, const int32_t *idx, const int32_t *counts, int P, int E,
                int chunks, int per_chunk, hipStream_t st) {
    const size_t lds = sort_lds_bytes(E, NT / kWave);
    if (lds > 65536 && hipFuncSetAttribute((const void *)sort_kernel<NT, S>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)lds) != hipSuccess)
        return K3G_EHIP;
    sort_kernel<NT, S><<<chunks, NT, lds, st>>>(offsets, perm, inv, idx, counts, P, E, per_chunk);
    return hipGetLastError() == hipSuccess ? K3G_OK : K3G_EHIP;
}

// ---- rows ------------------------------------------------------------------------

struct PairArgs {
    const void *tok;  // rows of tokens read: x or dy
    void *tok_out;    // rows of tokens written: y or dx
    const void *row;  // sorted rows read: ys or dys
    void *row_out;    // sorted rows written: ys or dys
    int64_t tok_ld, tok_out_ld, row_ld, row_out_ld;
    const float *wts;
    float *dwts;
    const int32_t *inv;
    int T, K, R, n;
    int waves;  // of a workgroup
    int parts;  // workgroups a token's columns are spread over
    int slots;  // pairs of a token that a workgroup takes
};

constexpr int kPairCols = 8;  // columns of a thread

typedef uint32_t Bits __attribute__((ext_vector_type(4), aligned(2)));  // 16 bytes at any entry's address

// The columns of a row that are there: eight, or the first of them. ONCE: past the caches.
template <int TYPE, bool ONCE>
__device__ inline void load_cols(float *v, const void *base, int64_t at, int n) {
    typedef typename Elem<TYPE>::T T;
    const T *p = (const T *)base + at;
    if (n >= kPairCols) {
        if constexpr (ONCE) {
            constexpr int M = kPairCols * sizeof(T) / 16;
            Bits b[M];
            T t[kPairCols];
#pragma unroll
            for (int i = 0; i < M; ++i) b[i] = __builtin_nontemporal_load((const Bits *)p + i);
            __builtin_memcpy(t, b, sizeof t);
#pragma unroll
            for (int i = 0; i < kPairCols; ++i) v[i] = Elem<TYPE>::load(t[i]);
        } else {
            load_n<TYPE, kPairCols>(v, p);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPairCols; ++i) v[i] = i < n ? Elem<TYPE>::load(p[i]) : 0.0f;
    }
}
template <int TYPE, bool ONCE>
__device__ inline void store_cols(void *base, int64_t at, int n, const float *v) {
    typedef typename Elem<TYPE>::T T;
    T *p = (T *)base + at;
    if (n >= kPairCols) {
        if constexpr (ONCE) {
            constexpr int M = kPairCols * sizeof(T) / 16;
            Bits b[M];
            T t[kPairCols];
#pragma unroll
            for (int i = 0; i < kPairCols; ++i) t[i] = Elem<TYPE>::store(v[i]);
            __builtin_memcpy(b, t, sizeof t);
#pragma unroll
            for (int i = 0; i < M; ++i) __builtin_nontemporal_store(b[i], (Bits *)p + i);
        } else {
            store_n<TYPE, kPairCols>(p, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPairCols; ++i)
            if (i < n) p[i] = Elem<TYPE>::store(v[i]);
    }
}

// SCATTER: sorted rows are written from the token's row. SUM: the sorted rows are
// summed into the token's. DOT: their products with the token's row are summed.
// An item: a token, a part of its columns and (no SUM) some of its pairs; DOT
// takes all columns. Lane k holds the sorted row and the weight of pair k of the item;
// U sorted rows are loaded at a time.
template <int ROW, int TOK, bool SCATTER, bool SUM, bool DOT, int U, bool ONCE>
__global__ __launch_bounds__(U > 4 ? 512 : 1024) void pairs_kernel(PairArgs a) {
    __shared__ float part[DOT ? 16 * kPairMaxTopK : 1];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int turns = (a.K + a.slots - 1) / a.slots, width = a.waves * kWave * kPairCols;
    const int64_t items = (int64_t)a.T * turns * a.parts;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t t = item / (turns * a.parts);
        const int rest = (int)(item - t * (turns * a.parts)), turn = rest / a.parts;
        const int k0 = turn * a.slots, n_pairs = min(a.slots, a.K - k0);
        int mine = lane < n_pairs ? a.inv[t * a.K + k0 + lane] : -1;
        if ((unsigned)mine >= (unsigned)a.R) mine = -1;
        const float weight = mine < 0 ? 0.0f : a.wts ? a.wts[t * a.K + k0 + lane] : 1.0f;
        if (DOT) {
            part[wave * kPairMaxTopK + lane] = 0.0f;
            wave_lds_order();  // other lanes add to them
        }
        for (int c0 = (rest - turn * a.parts) * width; c0 < a.n; c0 += a.parts * width) {
            const int c = c0 + tid * kPairCols, n = a.n - c;
            float tok[kPairCols], sum[kPairCols] = {};
            if (SCATTER || DOT) load_cols<TOK, false>(tok, a.tok, n > 0 ? t * a.tok_ld + c : 0, n);
            for (int k = 0; k < n_pairs; k += U) {
                int p[U], common = -1, some = 0;
                float w[U], v[U][kPairCols];
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    p[j] = __builtin_amdgcn_readlane(mine, k + j);
                    w[j] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, weight), k + j));
                    common &= p[j];
                    some |= p[j];
                }
                if (common < 0) continue;  // none has a row
                if (SUM || DOT) {
#pragma unroll
                    for (int j = 0; j < U; ++j) load_cols<ROW, ONCE>(v[j], a.row, n > 0 ? max(p[j], 0) * a.row_ld + c : 0, n);
                    if (some < 0) {  // a pair without a row adds nothing, whatever the row read in its place holds
#pragma unroll
                        for (int j = 0; j < U; ++j)
#pragma unroll
                            for (int i = 0; i < kPairCols; ++i) v[j][i] = p[j] < 0 ? 0.0f : v[j][i];
                    }
                }
                if (SUM) {
#pragma unroll
                    for (int j = 0; j < U; ++j)
#pragma unroll
                        for (int i = 0; i < kPairCols; ++i) sum[i] = __builtin_fmaf(w[j], v[j][i], sum[i]);
                }
                if (DOT) {
#pragma unroll
                    for (int j = 0; j < U; j += 4) {
                        float d[4];
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            d[m] = 0.0f;
#pragma unroll
                            for (int i = 0; i < kPairCols; ++i) d[m] = __builtin_fmaf(tok[i], v[j + m][i], d[m]);
                        }
                        const float all4 = wave_sum4(d, lane);
                        if (lane < 4) part[wave * kPairMaxTopK + k + j + lane] += all4;  // (always by the same lane)
                    }
                }
                if (SCATTER) {
#pragma unroll
                    for (int j = 0; j < U; ++j) {
                        if (p[j] < 0) continue;
                        float u[kPairCols];
#pragma unroll
                        for (int i = 0; i < kPairCols; ++i) u[i] = w[j] * tok[i];
                        store_cols<ROW, ONCE>(a.row_out, n > 0 ? p[j] * a.row_out_ld + c : 0, n, u);
                    }
                }
            }
            if (SUM) store_cols<TOK, false>(a.tok_out, n > 0 ? t * a.tok_out_ld + c : 0, n, sum);
        }
        if (DOT) {
            __syncthreads();
            if (tid < n_pairs) {  // the first wavefront: lane k's pair is k
                float d = part[tid];
                for (int w = 1; w < a.waves; ++w) d += part[w * kPairMaxTopK + tid];
                // a pair without a row was multiplied as zeros, which next to a token's infinity or NaN is no zero
                a.dwts[t * a.K + k0 + tid] = mine < 0 ? 0.0f : d;
            }
            __syncthreads();
        }
    }
}

// Wavefronts below which items are made smaller: columns, or slots, in workgroups of their own (61 tokens: rows
// written 9.4 us, so 5.6; summed 8.0, 6.2; written with the dot products, 64 tokens of fp32, 16.5, 9.2).
constexpr int64_t kPairFew = 4096;

template <int ROW, int TOK, bool SCATTER, bool SUM, bool DOT>
int launch_pairs(PairArgs a, hipStream_t st) {
    const int row_waves = (a.n + kWave * kPairCols - 1) / (kWave * kPairCols);
    a.slots = a.K;
    if (DOT) {
        a.waves = row_waves < 16 ? row_waves : 16;
        a.parts = 1;
    } else {
        a.waves = row_waves < 8 ? row_waves : 8;
        a.parts = (row_waves + a.waves - 1) / a.waves;
    }
    const bool few = (int64_t)a.T * a.parts * a.waves < kPairFew;
    if (few) {
        if (!SUM) a.slots = a.K < 4 ? a.K : 4;
        if (!DOT) {
            a.parts = row_waves;
            a.waves = 1;
        }
    }
    const int64_t items = (int64_t)a.T * a.parts * ((a.K + a.slots - 1) / a.slots), most = 1 << 20;
    const unsigned grid = (unsigned)(items < most ? items : most), threads = a.waves * kWave;
    if (!few)
        pairs_kernel<ROW, TOK, SCATTER, SUM, DOT, 4, true><<<grid, threads, 0, st>>>(a);
    else  // (a sum alone: all of a token's rows at once)
        pairs_kernel<ROW, TOK, SCATTER, SUM, DOT, SUM && !DOT ? 16 : 4, false><<<grid, threads, 0, st>>>(a);
    return hipGetLastError() == hipSuccess ? K3G_OK : K3G_EHIP;
}

template <bool SCATTER, bool SUM, bool DOT>
int launch_pairs_types(const PairArgs &a, int row, int tok, hipStream_t st) {
#define K3G_PAIR(R, T) \
    if (row == R && tok == T) return launch_pairs<R, T, SCATTER, SUM, DOT>(a, st)
    K3G_PAIR(K3G_F32, K3G_F32);
    K3G_PAIR(K3G_F32, K3G_BF16);
    K3G_PAIR(K3G_F32, K3G_F16);
    K3G_PAIR(K3G_BF16, K3G_F32);
    K3G_PAIR(K3G_BF16, K3G_BF16);
    K3G_PAIR(K3G_BF16, K3G_F16);
    K3G_PAIR(K3G_F16, K3G_F32);
    K3G_PAIR(K3G_F16, K3G_BF16);
    K3G_PAIR(K3G_F16, K3G_F16);
#undef K3G_PAIR
    return K3G_EINVAL;
}

// ---- host ------------------------------------------------------------------------

namespace {

constexpr int64_t kMaxPairs = (int64_t)1 << 30;

int pairs_shape(int n_tokens, int top_k, int n_rows, int in) {
    if (n_tokens < 0 || top_k < 1 || n_rows < 0 || in < 1) return K3G_EINVAL;
    if (top_k > kPairMaxTopK || (int64_t)n_tokens * top_k > kMaxPairs || n_rows > kMaxPairs || in > kMxMaxIn)
        return K3G_EUNSUPPORTED;
    return K3G_OK;
}

// inv and, where given, the weights and their gradient: dense [T][K] arrays.
int pairs_maps(const int32_t *inv, const float *wts, const float *dwts) {
    if (!inv) return K3G_EINVAL;
    return mx_aligned(inv, 4) && mx_aligned(wts, 4) && mx_aligned(dwts, 4) ? K3G_OK : K3G_EALIGN;
}

// A matrix of a call: its rows' addresses, once it has been looked over (rows = 0: none, the pointer may be null).
int matrix(Span *s, const void *p, int type, int64_t stride, int64_t rows, int in) {
    *s = span(nullptr, 0);
    if (!type_ok(type) || stride < in) return K3G_EINVAL;
    if (rows == 0) return K3G_OK;
    K3G_TRY(dense_ok(p, type, stride, in));
    *s = rows_span(p, type, rows, stride, in);
    return K3G_OK;
}

template <size_t A, size_t B>
bool any_meet(const Span (&out)[A], const Span (&in)[B]) {
    for (size_t i = 0; i < A; ++i) {
        for (size_t j = i + 1; j < A; ++j)
            if (meet(out[i], out[j])) return true;
        for (const Span &s : in)
            if (meet(out[i], s)) return true;
    }
    return false;
}

Span array_span(const void *p, int64_t n) { return span(p, p ? 4 * (size_t)n : 0); }

}  // namespace
}  // namespace k3g

using namespace k3g;

extern "C" {

int k3g_moe_sort(int32_t *offsets, int32_t *perm, int32_t *inv, const int32_t *idx, int n_tokens, int top_k,
                 int n_experts, void *ws, size_t ws_bytes, void *stream) {
    if (n_tokens < 0 || top_k < 1 || n_experts < 1 || !offsets) return K3G_EINVAL;
    const int64_t P = (int64_t)n_tokens * top_k;
    if (n_experts > kSortMaxExperts || P > kMaxPairs) return K3G_EUNSUPPORTED;
    if (!mx_aligned(offsets, 4) || !mx_aligned(perm, 4) || !mx_aligned(inv, 4) || !mx_aligned(idx, 4)) return K3G_EALIGN;
    const k3g_shape shape = {n_tokens, top_k, n_experts, 0, 0, 0, 0, 0};
    const size_t need = k3g_workspace_bytes(K3G_OP_MOE_SORT, &shape);
    if (P > 0) {
        if (!perm || !inv || !idx || !ws) return K3G_EINVAL;
        if (!mx_aligned(ws, 256)) return K3G_EALIGN;
        if (ws_bytes < need) return K3G_ENOSPACE;
    }
    const Span out[4] = {array_span(offsets, n_experts + 1), array_span(perm, P), array_span(inv, P),
                         span(ws, P > 0 ? need : 0)};
    const Span in[1] = {array_span(idx, P)};
    if (any_meet(out, in)) return K3G_EINVAL;
    K3G_TRY(device_ok());
    hipStream_t st = (hipStream_t)stream;
    const int chunks = sort_chunks(P), E = n_experts;
    if (chunks == 1) {
        if (P <= 256) return launch_sort<256, 1>(offsets, perm, inv, idx, nullptr, (int)P, E, 1, 256, st);
        if (P <= 1024) return launch_sort<1024, 1>(offsets, perm, inv, idx, nullptr, (int)P, E, 1, 1024, st);
        return launch_sort<1024, 4>(offsets, perm, inv, idx, nullptr, (int)P, E, 1, kSortAlone, st);
    }
    k3g_ws_layout l;
    K3G_TRY(k3g_workspace_layout(&l, K3G_OP_MOE_SORT, &shape));
    int32_t *counts = (int32_t *)((uint8_t *)ws + l.counts);
    const int per = (int)sort_chunk_pairs(P);
    sort_count_kernel<<<chunks, 1024, 0, st>>>(counts, idx, (int)P, E, per);
    if (hipGetLastError() != hipSuccess) return K3G_EHIP;
    return launch_sort<1024, 2>(offsets, perm, inv, idx, counts, (int)P, E, chunks, per, st);
}

int k3g_moe_gather(void *ys, int ys_type, int64_t ys_stride, const void *x, int x_type, int64_t x_stride,
                   const float *wts, const int32_t *inv, int n_tokens, int top_k, int n_rows, int in, void *stream) {
    K3G_TRY(pairs_shape(n_tokens, top_k, n_rows, in));
    Span out[1], use[3];
    K3G_TRY(matrix(&out[0], ys, ys_type, ys_stride, n_rows, in));
    K3G_TRY(matrix(&use[0], x, x_type, x_stride, n_tokens, in));
    if (n_tokens == 0) return K3G_OK;
    K3G_TRY(pairs_maps(inv, wts, nullptr));
    use[1] = array_span(inv, (int64_t)n_tokens * top_k);
    use[2] = array_span(wts, (int64_t)n_tokens * top_k);
    if (any_meet(out, use)) return K3G_EINVAL;
    if (n_rows == 0) return K3G_OK;
    K3G_TRY(device_ok());
    PairArgs a = {};
    a.tok = x, a.tok_ld = x_stride, a.row_out = ys, a.row_out_ld = ys_stride;
    a.wts = wts, a.inv = inv, a.T = n_tokens, a.K = top_k, a.R = n_rows, a.n = in;
    return launch_pairs_types<true, false, false>(a, ys_type, x_type, (hipStream_t)stream);
}

int k3g_moe_combine(void *y, int y_type, int64_t y_stride, const void *ys, int ys_type, int64_t ys_stride,
                    const float *wts, const int32_t *inv, int n_tokens, int top_k, int n_rows, int in, void *stream) {
    return k3g_moe_gather_backward(y, nullptr, ys, ys_type, ys_stride, nullptr, y_type, 0, y_stride, wts, inv, n_tokens,
                                   top_k, n_rows, in, stream);
}

int k3g_moe_gather_backward(void *dx, float *dwts, const void *dys, int dys_type, int64_t dys_stride, const void *x,
                            int x_type, int64_t x_stride, int64_t dx_stride, const float *wts, const int32_t *inv,
                            int n_tokens, int top_k, int n_rows, int in, void *stream) {
    K3G_TRY(pairs_shape(n_tokens, top_k, n_rows, in));
    Span out[2], use[4];
    const int64_t P = (int64_t)n_tokens * top_k;
    if (n_tokens > 0 && ((!dx && !dwts) || (dwts && !x))) return K3G_EINVAL;
    K3G_TRY(matrix(&out[0], dx, x_type, dx || n_tokens == 0 ? dx_stride : in, dx ? n_tokens : 0, in));
    K3G_TRY(matrix(&use[0], dys, dys_type, dys_stride, n_rows, in));
    K3G_TRY(matrix(&use[1], x, x_type, dwts ? x_stride : in, dwts ? n_tokens : 0, in));
    if (n_tokens == 0) return K3G_OK;
    K3G_TRY(pairs_maps(inv, wts, dwts));
    out[1] = array_span(dwts, P);
    use[2] = array_span(inv, P);
    use[3] = array_span(wts, P);
    if (any_meet(out, use)) return K3G_EINVAL;
    K3G_TRY(device_ok());
    PairArgs a = {};
    a.tok = x, a.tok_ld = x_stride, a.tok_out = dx, a.tok_out_ld = dx_stride, a.row = dys, a.row_ld = dys_stride;
    a.wts = wts, a.dwts = dwts, a.inv = inv, a.T = n_tokens, a.K = top_k, a.R = n_rows, a.n = in;
    hipStream_t st = (hipStream_t)stream;
    if (!dwts) return launch_pairs_types<false, true, false>(a, dys_type, x_type, st);
    if (!dx) return launch_pairs_types<false, false, true>(a, dys_type, x_type, st);
    return launch_pairs_types<false, true, true>(a, dys_type, x_type, st);
}

int k3g_moe_combine_backward(void *dys, float *dwts, const void *dy, int dy_type, int64_t dy_stride, const void *ys,
                             int ys_type, int64_t ys_stride, int64_t dys_stride, const float *wts, const int32_t *inv,
                             int n_tokens, int top_k, int n_rows, int in, void *stream) {
    K3G_TRY(pairs_shape(n_tokens, top_k, n_rows, in));
    Span out[2], use[4];
    const int64_t P = (int64_t)n_tokens * top_k;
    if (n_tokens > 0 && n_rows > 0 && ((!dys && !dwts) || (dwts && !ys))) return K3G_EINVAL;
    K3G_TRY(matrix(&out[0], dys, ys_type, dys ? dys_stride : in, dys ? n_rows : 0, in));
    K3G_TRY(matrix(&use[0], dy, dy_type, dy_stride, n_tokens, in));
    K3G_TRY(matrix(&use[1], ys, ys_type, dwts ? ys_stride : in, dwts ? n_rows : 0, in));
    if (n_tokens == 0) return K3G_OK;
    K3G_TRY(pairs_maps(inv, wts, dwts));
    out[1] = array_span(dwts, P);
    use[2] = array_span(inv, P);
    use[3] = array_span(wts, P);
    if (dys && dys == ys && dys_stride == ys_stride) use[1] = span(nullptr, 0);  // each entry is read before it is written
    if (any_meet(out, use)) return K3G_EINVAL;
    K3G_TRY(device_ok());
    PairArgs a = {};
    a.tok = dy, a.tok_ld = dy_stride, a.row = ys, a.row_ld = ys_stride, a.row_out = dys, a.row_out_ld = dys_stride;
    a.wts = wts, a.dwts = dwts, a.inv = inv, a.T = n_tokens, a.K = top_k, a.R = n_rows, a.n = in;
    hipStream_t st = (hipStream_t)stream;
    if (!dwts) return n_rows == 0 ? K3G_OK : launch_pairs_types<true, false, false>(a, ys_type, dy_type, st);
    if (!dys) return launch_pairs_types<false, false, true>(a, ys_type, dy_type, st);
    return launch_pairs_types<true, false, true>(a, ys_type, dy_type, st);
}

}  // extern "C"
