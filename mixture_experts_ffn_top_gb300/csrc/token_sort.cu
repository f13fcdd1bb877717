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
constexpr int ROW_WARPS = 8;      // warps per CTA of the router gradient, a token each
constexpr int ROW_THREADS = 256;  // threads per CTA of the row kernels

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
            Pack<T, V> v;
            v.load(src + c);
            for (int s = 0; s < top_k; ++s) {
                const int r = p[s];
                if (r >= 0) v.store(rows + (int64_t)r * D + c);
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

// out[t] = sum over the slots of w * row (w == NULL: of the row), in slot order.  Threads 0 .. tpt - 1 of a
// token's group (tpt a power of two, ROW_THREADS / tpt tokens a CTA) own V consecutive columns each at a
// time; SLOTS rows are loaded before the first is used.  HBM-bound: 8192 x 2048 bf16, top 8, takes 47.8 us
// (302 MB: 6.3 TB/s, 93% of the copy rate), 4096 x 2048 fp32 46.8 us (95%).  The entries' rows and weights wait
// in shared memory: held in registers by every thread they cost 57 us (a third of the warps).
constexpr int SLOTS = 8;

template <typename T, int V>
__global__ void __launch_bounds__(ROW_THREADS, 4)
unsort_kernel(const T *__restrict__ rows, int64_t n_rows, const int32_t *__restrict__ tokRow,
              const float *__restrict__ w, int N, int top_k, int D, int tpt_log2, T *__restrict__ out,
              int64_t out_stride, unsigned *__restrict__ status) {
    extern __shared__ int2 entry[];  // [tokens of the CTA][top_k]: row (or -1), weight
    const int tpt = 1 << tpt_log2, per = ROW_THREADS >> tpt_log2;
    const int64_t t0 = (int64_t)blockIdx.x * per;
    const int tokens = (int)min((int64_t)per, N - t0);
    for (int i = threadIdx.x; i < tokens * top_k; i += ROW_THREADS)
        entry[i] = make_int2(checked_row(tokRow[t0 * top_k + i], n_rows, status),
                             __float_as_int(w != nullptr ? w[t0 * top_k + i] : 1.0f));
    __syncthreads();
    const int mine = threadIdx.x >> tpt_log2;
    if (mine >= tokens) return;
    const int2 *en = entry + mine * top_k;
    T *dst = out + (t0 + mine) * out_stride;
    for (int64_t c = ((int64_t)blockIdx.y * tpt + (threadIdx.x & (tpt - 1))) * V; c < D;
         c += (int64_t)gridDim.y * tpt * V) {
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
        for (int s0 = 0; s0 < top_k; s0 += SLOTS) {
            Pack<T, V> v[SLOTS];
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
                if (s0 + s < top_k && en[s0 + s].x >= 0) v[s].load_once(rows + (int64_t)en[s0 + s].x * D + c);
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
                if (s0 + s < top_k && en[s0 + s].x >= 0) {
                    const float ws = __int_as_float(en[s0 + s].y);
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] = __fmaf_rn(ws, v[s].get(i), acc[i]);
                }
        }
        Pack<T, V> o;
        o.set(acc);
        o.store(dst + c);
    }
}

// d_row = w * d_out and the dot d_w = <d_out, row> of one entry (t, s) at a time, by TPE threads: the rows are
// read and written once, d_out's row comes from the caches for all but its first entry.  The dot: each thread's
// columns in order, a butterfly over the warp, the warps in order.  2048 x 2048 bf16, top 8: 25.5 us (143 MB:
// 83% of the copy rate); a token's threads holding all its entries at once took 35.8 us (registers, and a
// reduction of eight dots through shared memory).
template <typename T, int V, int TPE>
__global__ void __launch_bounds__(ROW_THREADS)
unsort_grad_kernel(const T *__restrict__ d_out, int64_t d_out_stride, const T *__restrict__ rows, int64_t n_rows,
                   const int32_t *__restrict__ tokRow, const float *__restrict__ w, int n_entries, int top_k, int D,
                   T *__restrict__ d_rows, float *__restrict__ d_w, unsigned *__restrict__ status) {
    constexpr int UNROLL = 4;
    __shared__ float part[ROW_THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * (ROW_THREADS / TPE) + threadIdx.x / TPE;
    if (i >= n_entries) return;  // whole warps; whole CTAs where TPE is the CTA
    const int r = checked_row(tokRow[i], n_rows, status);
    float dot = 0.0f;
    if (r >= 0) {
        const float ws = w[i];
        const T *src = d_out + (i / top_k) * d_out_stride, *row = rows + (int64_t)r * D;
        T *dst = d_rows + (int64_t)r * D;
        for (int c0 = (threadIdx.x & (TPE - 1)) * V; c0 < D; c0 += UNROLL * TPE * V) {
            Pack<T, V> dv[UNROLL], rv[UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int c = c0 + u * TPE * V;
                if (c < D) {
                    rv[u].load_once(row + c);
                    dv[u].load(src + c);
                }
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int c = c0 + u * TPE * V;
                if (c < D) {
                    Pack<T, V> o;
                    float f[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        dot = __fmaf_rn(dv[u].get(j), rv[u].get(j), dot);
                        f[j] = __fmul_rn(ws, dv[u].get(j));
                    }
                    o.set(f);
                    o.store(dst + c);
                }
            }
        }
    }
    dot = warp_sum(dot);
    if (TPE == 32) {
        if (lane == 0) d_w[i] = dot;
    } else {
        if (lane == 0) part[warp] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
#pragma unroll
            for (int k = 1; k < TPE / 32; ++k) dot += part[k];
            d_w[i] = dot;
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

// Bytes per access: the largest of 16, 8, 4 and 2 that divides every address and row stride.
int access_bytes(std::initializer_list<const void *> ptrs, std::initializer_list<int64_t> stride_bytes) {
    uint64_t bits = 16;
    for (const void *p : ptrs) bits |= reinterpret_cast<uintptr_t>(p);
    for (int64_t st : stride_bytes) bits |= (uint64_t)st;
    return (int)(bits & -bits);
}

// Calls f with the elements per access as a constant.
template <typename T, typename F>
int by_width(int bytes, F f) {
    constexpr int E = sizeof(T);
    if (bytes >= 16) return f(std::integral_constant<int, 16 / E>());
    if (bytes >= 8) return f(std::integral_constant<int, 8 / E>());
    if (bytes >= 4) return f(std::integral_constant<int, 4 / E>());
    return f(std::integral_constant<int, 1>());
}

int log2_ceil(int64_t n, int most) {
    int l = 0;
    while (l < most && ((int64_t)1 << l) < n) ++l;
    return l;
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
        const int b = access_bytes({x, rows}, {x_stride * (int64_t)sizeof(T), D * (int64_t)sizeof(T)});
        return by_width<T>(b, [&](auto v) { return go(sort_place_kernel<T, decltype(v)::value>); });
    });
}

int launch_unsort_tokens(const void *rows, int64_t n_rows, int dtype, const int32_t *tokRow, const float *w, int N,
                         int top_k, int D, void *out, int64_t out_stride, unsigned *status, cudaStream_t s) {
    const int sms = std::max(1, device_sm_count());
    return by_dtype(dtype, [&](auto *tp) {
        using T = std::remove_pointer_t<decltype(tp)>;
        const int b = access_bytes({rows, out}, {D * (int64_t)sizeof(T), out_stride * (int64_t)sizeof(T)});
        return by_width<T>(b, [&](auto v) {
            constexpr int V = decltype(v)::value;
            const int64_t cols = (D + V - 1) / V;
            // One access a thread until every SM has 2048 of them, then two, or four where they are narrow: 8192 x
            // 2048 bf16 at 16 bytes measured 49.8 / 47.8 / 49.2 us with 1 / 2 / 4, 13620 x 373 fp16 at 2 bytes
            // 45.9 / 39.1 / 35.0 us.
            const int64_t most = sizeof(T) * V == 16 ? 2 : 4;
            int64_t reps = 1;
            while (reps < most && N * cols / (2 * reps) >= (int64_t)sms * 2048) reps *= 2;
            const int tl = std::max(log2_ceil((cols + reps - 1) / reps, 8), 3);
            const int per = ROW_THREADS >> tl;
            const int64_t cta_cols = ((int64_t)1 << tl) * reps;
            const dim3 grid((unsigned)((N + per - 1) / per), (unsigned)std::min<int64_t>((cols + cta_cols - 1) / cta_cols, 65535));
            unsort_kernel<T, V><<<grid, ROW_THREADS, (size_t)per * top_k * sizeof(int2), s>>>(static_cast<const T *>(rows), n_rows, tokRow, w, N, top_k,
                                                             D, tl, static_cast<T *>(out), out_stride, status);
            return launch_status();
        });
    });
}

int launch_unsort_tokens_grad(const void *d_out, int64_t d_out_stride, const void *rows, int64_t n_rows, int dtype,
                              const int32_t *tokRow, const float *w, int N, int top_k, int D, void *d_rows, float *d_w,
                              unsigned *status, cudaStream_t s) {
    const int sms = std::max(1, device_sm_count());
    return by_dtype(dtype, [&](auto *tp) {
        using T = std::remove_pointer_t<decltype(tp)>;
        const int b = access_bytes({d_out, rows, d_rows}, {d_out_stride * (int64_t)sizeof(T), D * (int64_t)sizeof(T)});
        return by_width<T>(b, [&](auto v) {
            constexpr int V = decltype(v)::value;
            const int64_t cols = (D + V - 1) / V;
            const int64_t n = (int64_t)N * top_k;
            auto go = [&](auto kernel, int per) {
                kernel<<<(unsigned)((n + per - 1) / per), ROW_THREADS, 0, s>>>(
                    static_cast<const T *>(d_out), d_out_stride, static_cast<const T *>(rows), n_rows, tokRow, w,
                    (int)n, top_k, D, static_cast<T *>(d_rows), d_w, status);
                return launch_status();
            };
            // a warp an entry, or a CTA where the entries are few and their rows long
            if (n < (int64_t)sms * 8 && cols > 64) return go(unsort_grad_kernel<T, V, ROW_THREADS>, 1);
            return go(unsort_grad_kernel<T, V, 32>, ROW_THREADS / 32);
        });
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
