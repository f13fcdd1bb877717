// token_sort.cu -- token rows sorted by expert and back, with the routing weights applied, and the
// gradients of both; the gradient of the routing weights to the router logits.
//
// The order is a stable counting sort of the N * top_k entries by expert: entry (t, s) of expert e
// lands at expStart[e] + the number of earlier entries of e.  Everything else is a function of the
// entries' rows (tokRow) alone, one token at a time:
//   sort     rows[tokRow[t,s]] = x[t]                    unsort   out[t] = sum_s w[t,s] rows[tokRow[t,s]]
//   d_x[t] = sum_s d_rows[tokRow[t,s]]                   d_rows[tokRow[t,s]] = w[t,s] d_out[t],
//                                                        d_w[t,s] = <d_out[t], rows[tokRow[t,s]]>
// so a token's row is read or written once and its top_k sorted rows once each: (1 + top_k) D values
// a token (1 + 2 top_k for the unsort's gradient), and a few operations a value: all are bound by HBM.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "elem.cuh"

namespace moe {

namespace {

constexpr int COUNT_THREADS = 256;
constexpr int ROW_WARPS = 8;  // warps per CTA of the row kernels, a token each

// ------------------------------------------------------------------ order --
// Entries of each expert in token range blockIdx.x: table[range][e].
__global__ void __launch_bounds__(COUNT_THREADS)
sort_count_kernel(const int32_t *__restrict__ idx, int n_entries, int per_range, int E, int *__restrict__ table,
                  unsigned *__restrict__ status) {
    extern __shared__ int hist[];
    for (int e = threadIdx.x; e < E; e += COUNT_THREADS) hist[e] = 0;
    __syncthreads();
    const int lo = blockIdx.x * per_range, hi = min(lo + per_range, n_entries);
    for (int i = lo + threadIdx.x; i < hi; i += COUNT_THREADS) {
        const int e = idx[i];
        if (e >= 0 && e < E)
            atomicAdd(&hist[e], 1);
        else if (e != -1)
            atomicOr(status, MOE_DEV_BAD_ROUTING);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += COUNT_THREADS) table[(size_t)blockIdx.x * E + e] = hist[e];
}

// Row of every entry of range blockIdx.x, the CSR arrays, and the rows themselves.
template <typename T, int V>
__global__ void __launch_bounds__(ROW_WARPS * 32)
sort_place_kernel(const T *__restrict__ x, int64_t x_stride, const int32_t *__restrict__ idx, int n_entries,
                  int per_range, int top_k, int E, int D, const int *__restrict__ table, int n_ranges,
                  int32_t *__restrict__ expStart, int32_t *__restrict__ expTokI, int32_t *__restrict__ expTokK,
                  int32_t *tokRow, T *__restrict__ rows) {
    extern __shared__ int sm[];
    int *base = sm;           // [E]: next row of each expert for this range
    int *total = sm + E;      // [E]: entries of each expert
    __shared__ int kept_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int NT = ROW_WARPS * 32;
    for (int e = tid; e < E; e += NT) {
        int before = 0, all = 0;
        for (int g = 0; g < n_ranges; ++g) {
            const int c = table[(size_t)g * E + e];
            before += g < (int)blockIdx.x ? c : 0;
            all += c;
        }
        base[e] = before;
        total[e] = all;
    }
    __syncthreads();
    const int lo = blockIdx.x * per_range, hi = min(lo + per_range, n_entries);
    if (warp == 0) {
        // exclusive scan of the totals: expert e's segment start
        int run = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < E ? total[e] : 0;
            int inc = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            if (e < E) {
                base[e] += run + inc - c;
                if (blockIdx.x == 0) expStart[e] = run + inc - c;
            }
            run += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) {
            kept_s = run;
            if (blockIdx.x == 0) expStart[E] = run;
        }
        __syncwarp();
        // rank of each entry among the earlier ones of its expert, 32 entries at a time
        for (int i0 = lo; i0 < hi; i0 += 32) {
            const int i = i0 + lane;
            int e = i < hi ? idx[i] : -1;
            if (e < 0 || e >= E) e = -1;
            const unsigned same = __match_any_sync(0xffffffffu, e);
            int r = -1;
            if (e >= 0) r = base[e] + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (e >= 0 && lane == __ffs(same) - 1) base[e] += __popc(same);
            __syncwarp();
            if (i < hi) {
                tokRow[i] = r;
                if (r >= 0) {
                    expTokI[r] = i / top_k;
                    expTokK[r] = i % top_k;
                }
            }
        }
    }
    __syncthreads();
    // CSR entries past the last row: every range clears its own positions among them
    for (int i = max(lo, kept_s) + tid; i < hi; i += NT) {
        expTokI[i] = -1;
        expTokK[i] = -1;
    }
    const int t0 = lo / top_k, t1 = hi / top_k;
    for (int t = t0 + warp; t < t1; t += ROW_WARPS) {
        const int32_t *p = tokRow + (int64_t)t * top_k;  // this block's own stores above
        const T *src = x + (int64_t)t * x_stride;
        for (int c = lane * V; c < D; c += 32 * V) {
            const Vec<T, V> v = *reinterpret_cast<const Vec<T, V> *>(src + c);
            for (int s = 0; s < top_k; ++s) {
                const int r = p[s];
                if (r >= 0) *reinterpret_cast<Vec<T, V> *>(rows + (int64_t)r * D + c) = v;
            }
        }
    }
}

// ----------------------------------------------------------------- unsort --
// Sorted row of an entry, or -1 (a row outside [0, n_rows) is flagged and dropped).
__device__ __forceinline__ int checked_row(int r, int64_t n_rows, unsigned *status) {
    if (r >= 0 && r < n_rows) return r;
    if (r != -1) atomicOr(status, MOE_DEV_BAD_CSR);
    return -1;
}

// out[t] = sum over the slots of w * row (w == NULL: of the row), in slot order; a warp per token.
template <typename T, int V>
__global__ void __launch_bounds__(ROW_WARPS * 32)
unsort_kernel(const T *__restrict__ rows, int64_t n_rows, const int32_t *__restrict__ tokRow,
              const float *__restrict__ w, int N, int top_k, int D, T *__restrict__ out, int64_t out_stride,
              unsigned *__restrict__ status) {
    const int lane = threadIdx.x & 31;
    for (int64_t t = (int64_t)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5); t < N; t += (int64_t)gridDim.x * ROW_WARPS) {
        int r = -1;
        float ws = 1.0f;
        if (lane < top_k) {
            r = checked_row(tokRow[t * top_k + lane], n_rows, status);
            if (w != nullptr) ws = w[t * top_k + lane];
        }
        for (int c0 = 0; c0 < D; c0 += 32 * V) {
            const int c = c0 + lane * V;
            float acc[V];
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = 0.0f;
            for (int s = 0; s < top_k; ++s) {
                const int rs = __shfl_sync(0xffffffffu, r, s);
                const float wv = __shfl_sync(0xffffffffu, ws, s);
                if (rs >= 0 && c < D) {
                    const Vec<T, V> v = *reinterpret_cast<const Vec<T, V> *>(rows + (int64_t)rs * D + c);
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] = __fmaf_rn(wv, elem_f32(v.v[i]), acc[i]);
                }
            }
            if (c < D) {
                Vec<T, V> o;
#pragma unroll
                for (int i = 0; i < V; ++i) o.v[i] = elem_of<T>(acc[i]);
                *reinterpret_cast<Vec<T, V> *>(out + t * out_stride + c) = o;
            }
        }
    }
}

// d_rows of every entry of a token and the dots d_w; a warp per token.
template <typename T, int V>
__global__ void __launch_bounds__(ROW_WARPS * 32)
unsort_grad_kernel(const T *__restrict__ d_out, int64_t d_out_stride, const T *__restrict__ rows, int64_t n_rows,
                   const int32_t *__restrict__ tokRow, const float *__restrict__ w, int N, int top_k, int D,
                   T *__restrict__ d_rows, float *__restrict__ d_w, unsigned *__restrict__ status) {
    const int lane = threadIdx.x & 31;
    for (int64_t t = (int64_t)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5); t < N; t += (int64_t)gridDim.x * ROW_WARPS) {
        const T *src = d_out + t * d_out_stride;
        for (int s = 0; s < top_k; ++s) {
            const int r = checked_row(tokRow[t * top_k + s], n_rows, status);
            float dot = 0.0f;
            if (r >= 0) {
                const float ws = w[t * top_k + s];
                for (int c = lane * V; c < D; c += 32 * V) {
                    const Vec<T, V> dv = *reinterpret_cast<const Vec<T, V> *>(src + c);
                    const Vec<T, V> rv = *reinterpret_cast<const Vec<T, V> *>(rows + (int64_t)r * D + c);
                    Vec<T, V> o;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float d = elem_f32(dv.v[i]);
                        dot = __fmaf_rn(d, elem_f32(rv.v[i]), dot);
                        o.v[i] = elem_of<T>(__fmul_rn(ws, d));
                    }
                    *reinterpret_cast<Vec<T, V> *>(d_rows + (int64_t)r * D + c) = o;
                }
            }
            dot = warp_sum(dot);
            if (lane == 0) d_w[t * top_k + s] = dot;
        }
    }
}

// -------------------------------------------------------------- topk grad --
// One warp per token: softmax (over all experts, or over the selected ones), then
// d_l[e] = p[e] * (v[e] - sum_j p[j] v[j]) with v[e] the sum of the weights' gradients at e.
// EPL experts per lane (EPL * 32 >= E).
template <int EPL>
__global__ void __launch_bounds__(ROW_WARPS * 32)
topk_grad_kernel(const float *__restrict__ logits, const int32_t *__restrict__ idx, const float *__restrict__ d_w,
                 int N, int E, int top_k, int norm, float *__restrict__ d_logits, unsigned *__restrict__ status) {
    const int lane = threadIdx.x & 31;
    for (int64_t t = (int64_t)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5); t < N; t += (int64_t)gridDim.x * ROW_WARPS) {
        int my_e = -1;
        float my_d = 0.0f;
        if (lane < top_k) {
            my_e = idx[t * top_k + lane];
            my_d = d_w[t * top_k + lane];
            if (my_e < 0 || my_e >= E) {
                if (my_e != -1) atomicOr(status, MOE_DEV_BAD_ROUTING);
                my_e = -1;
            }
        }
        float p[EPL], v[EPL];
        unsigned sel = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 32 * i;
            p[i] = e < E ? logits[t * E + e] : -INFINITY;
            v[i] = 0.0f;
        }
        for (int s = 0; s < top_k; ++s) {
            const int e = __shfl_sync(0xffffffffu, my_e, s);
            const float d = __shfl_sync(0xffffffffu, my_d, s);
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (e == lane + 32 * i) {
                    v[i] += d;
                    sel |= 1u << i;
                }
        }
        float m = -INFINITY;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (norm && !((sel >> i) & 1)) p[i] = -INFINITY;
            nan |= p[i] != p[i];
            m = fmaxf(m, p[i]);
        }
        m = warp_max(m);
        nan = __any_sync(0xffffffffu, nan);
        const bool none = m == -INFINITY && !nan;  // nothing to take a softmax of
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            p[i] = (lane + 32 * i < E && !(norm && !((sel >> i) & 1)) && !none) ? expf(p[i] - m) : 0.0f;
            z += p[i];
        }
        z = none ? 1.0f : warp_sum(z);
        float c = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            p[i] = __fdiv_rn(p[i], z);
            if ((sel >> i) & 1) c = __fmaf_rn(p[i], v[i], c);
        }
        c = warp_sum(c);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 32 * i;
            if (e >= E) continue;
            const bool in = !none && (!norm || ((sel >> i) & 1));
            d_logits[t * E + e] = in ? __fmul_rn(p[i], __fsub_rn(v[i], c)) : 0.0f;
        }
    }
}

// Elements per access: 16 bytes when every address is a multiple of that, else the element alone.
template <typename T>
bool wide(std::initializer_list<const void *> ptrs, std::initializer_list<int64_t> strides) {
    for (const void *p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
    for (int64_t st : strides)
        if (st * (int64_t)sizeof(T) % 16 != 0) return false;
    return true;
}

unsigned row_grid(int64_t N) {
    const int64_t cap = (int64_t)std::max(1, device_sm_count()) * 8;
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>((N + ROW_WARPS - 1) / ROW_WARPS, cap));
}

// Calls f with a null pointer of the element type.
template <typename F>
int by_dtype(int dtype, F f) {
    switch (dtype) {
        case MOE_DTYPE_F32: return f(static_cast<float *>(nullptr));
        case MOE_DTYPE_F16: return f(static_cast<__half *>(nullptr));
        default: return f(static_cast<__nv_bfloat16 *>(nullptr));
    }
}

}  // namespace

int sort_ranges(int N, int *tokens) {
    const int sms = 152;  // ranges of a fixed number, so that the workspace's size is the shape's alone
    const int per = (N + sms - 1) / sms;
    if (tokens) *tokens = per;
    return (N + per - 1) / per;
}

size_t sort_scratch_bytes(int N, int E) { return (size_t)sort_ranges(N, nullptr) * E * 4; }

int launch_sort_tokens(const void *x, int64_t x_stride, int dtype, const int32_t *idx, int N, int top_k, int E, int D,
                       int32_t *expStart, int32_t *expTokI, int32_t *expTokK, int32_t *tokRow, void *rows, void *ws,
                       cudaStream_t s) {
    int tokens = 0;
    const int ranges = sort_ranges(N, &tokens);
    const int n = N * top_k, per = tokens * top_k;
    int *table = ws_ptr<int>(ws, SORT_SCRATCH_OFFSET);
    unsigned *status = static_cast<unsigned *>(ws);
    sort_count_kernel<<<ranges, COUNT_THREADS, (size_t)E * 4, s>>>(idx, n, per, E, table, status);
    const size_t smem = (size_t)2 * E * 4;
    return by_dtype(dtype, [&](auto *tp) {
        using T = std::remove_pointer_t<decltype(tp)>;
        auto go = [&](auto kernel) {  // E <= 1024: at most 8 KB of shared memory
            kernel<<<ranges, ROW_WARPS * 32, smem, s>>>(static_cast<const T *>(x), x_stride, idx, n, per, top_k, E, D,
                                                        table, ranges, expStart, expTokI, expTokK, tokRow,
                                                        static_cast<T *>(rows));
            return launch_status();
        };
        constexpr int V = 16 / sizeof(T);
        if (wide<T>({x, rows}, {x_stride, D})) return go(sort_place_kernel<T, V>);
        return go(sort_place_kernel<T, 1>);
    });
}

int launch_unsort_tokens(const void *rows, int64_t n_rows, int dtype, const int32_t *tokRow, const float *w, int N,
                         int top_k, int D, void *out, int64_t out_stride, unsigned *status, cudaStream_t s) {
    return by_dtype(dtype, [&](auto *tp) {
        using T = std::remove_pointer_t<decltype(tp)>;
        auto go = [&](auto kernel) {
            kernel<<<row_grid(N), ROW_WARPS * 32, 0, s>>>(static_cast<const T *>(rows), n_rows, tokRow, w, N, top_k, D,
                                                          static_cast<T *>(out), out_stride, status);
            return launch_status();
        };
        constexpr int V = 16 / sizeof(T);
        return wide<T>({rows, out}, {D, out_stride}) ? go(unsort_kernel<T, V>) : go(unsort_kernel<T, 1>);
    });
}

int launch_unsort_tokens_grad(const void *d_out, int64_t d_out_stride, const void *rows, int64_t n_rows, int dtype,
                              const int32_t *tokRow, const float *w, int N, int top_k, int D, void *d_rows, float *d_w,
                              unsigned *status, cudaStream_t s) {
    return by_dtype(dtype, [&](auto *tp) {
        using T = std::remove_pointer_t<decltype(tp)>;
        auto go = [&](auto kernel) {
            kernel<<<row_grid(N), ROW_WARPS * 32, 0, s>>>(static_cast<const T *>(d_out), d_out_stride,
                                                          static_cast<const T *>(rows), n_rows, tokRow, w, N, top_k, D,
                                                          static_cast<T *>(d_rows), d_w, status);
            return launch_status();
        };
        constexpr int V = 16 / sizeof(T);
        return wide<T>({d_out, rows, d_rows}, {d_out_stride, D}) ? go(unsort_grad_kernel<T, V>)
                                                                 : go(unsort_grad_kernel<T, 1>);
    });
}

int launch_topk_grad(const float *logits, const int32_t *idx, const float *d_w, int N, int E, int top_k, int norm,
                     float *d_logits, unsigned *status, cudaStream_t s) {
    auto go = [&](auto kernel) {
        kernel<<<row_grid(N), ROW_WARPS * 32, 0, s>>>(logits, idx, d_w, N, E, top_k, norm, d_logits, status);
        return launch_status();
    };
    if (E <= 32) return go(topk_grad_kernel<1>);
    if (E <= 64) return go(topk_grad_kernel<2>);
    if (E <= 128) return go(topk_grad_kernel<4>);
    if (E <= 256) return go(topk_grad_kernel<8>);
    if (E <= 512) return go(topk_grad_kernel<16>);
    return go(topk_grad_kernel<32>);
}

}  // namespace moe
