// norm.cu -- layer norm of token rows, its gradients, and the gradients of RMSNorm:
//   y = gamma (x - m) r + beta,   m = mean(x), v = mean((x - m)^2), r = 1 / sqrt(v + eps)
//   with h = (x - m) r and g = gamma d_y, along each row:
//   d_x = r (g - mean(g) - h mean(g h)),   d_gamma = sum over rows of d_y h,   d_beta = sum over rows of d_y
//   (RMSNorm: m = 0, and no mean(g)).
//
// One pass over the data bounds it: a row stays in registers between the sums over it and its result, the next
// row's loads fly meanwhile, and each thread keeps the same columns for all its rows, so that the column sums d_gamma
// and d_beta grow in its registers and leave the CTA once.  The gradient forms m and r again from the row it holds
// anyway: nothing is saved by the forward pass.  The variance is summed from the deviations (a second sum over the
// registers), not from squares: rows far off centre lose nothing.
//
// A row takes the threads that leave each 16 elements at most, of a CTA's 512 at most; a CTA works on as many rows
// at once as it has room for.  Rows of more than 8192 elements are shared by a cluster of CTAs, whose sums meet in
// distributed shared memory.
#include <algorithm>

#include "elem.cuh"

namespace moe {

namespace {

constexpr int NORM_THREADS = 512;
constexpr int NORM_EPT = 16;                             // elements a thread holds of a row
constexpr int NORM_CTA_COLS = NORM_THREADS * NORM_EPT;   // columns of a CTA
constexpr int SUM_SLICES = 16;                           // warps over the partial sums of 32 columns

enum { NORM_FORWARD, NORM_GRAD, NORM_RMS_GRAD };

struct NormArgs {
    const void *x, *dy;
    int64_t x_stride, dy_stride, out_stride;
    const float *gamma, *beta;
    float eps;
    int N, D;
    void *out;               // y or d_x
    float *part;             // [clusters][2][D] column sums, or NULL: the only cluster writes them
    float *d_gamma, *d_beta;  // d_beta may be NULL
    int tpr_log2;            // threads a row
    int cluster;             // CTAs a row
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The float at `p` of this CTA's shared memory, in CTA `rank` of the cluster.
__device__ __forceinline__ void store_peer(float *p, uint32_t rank, float v) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(r), "f"(v) : "memory");
}

// Sums of NVAL values over the threads of a row, in a fixed order, the same in all of them.  `buf` alternates, so
// that one barrier a sum is enough.
struct RowSum {
    float (*slots)[NORM_THREADS / 32][4];  // [2][warp][value]
    float (*peers)[8][4];                  // [2][rank][value]
    int tpr, first_warp, bar, cluster;
    int buf = 0;

    template <int NVAL>
    __device__ __forceinline__ void operator()(float (&v)[NVAL]) {
#pragma unroll
        for (int i = 0; i < NVAL; ++i) v[i] = warp_sum(v[i]);
        if (tpr == 32) return;
        const int warp = threadIdx.x >> 5, warps = tpr >> 5;
        float (*s)[4] = slots[buf];
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < NVAL; ++i) s[warp][i] = v[i];
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(tpr) : "memory");
#pragma unroll
        for (int i = 0; i < NVAL; ++i) v[i] = s[first_warp][i];
        for (int w = 1; w < warps; ++w)
#pragma unroll
            for (int i = 0; i < NVAL; ++i) v[i] += s[first_warp + w][i];
        if (cluster > 1) {
            if (threadIdx.x < cluster)
#pragma unroll
                for (int i = 0; i < NVAL; ++i) store_peer(&peers[buf][cluster_rank()][i], threadIdx.x, v[i]);
            cluster_sync();
#pragma unroll
            for (int i = 0; i < NVAL; ++i) v[i] = peers[buf][0][i];
            for (int r = 1; r < cluster; ++r)
#pragma unroll
                for (int i = 0; i < NVAL; ++i) v[i] += peers[buf][r][i];
        }
        buf ^= 1;
    }
};

template <typename T, int V, int MODE>
__global__ void __launch_bounds__(NORM_THREADS, MODE == NORM_FORWARD ? 2 : 1) norm_kernel(const NormArgs a) {
    constexpr int NV = NORM_EPT / V;
    constexpr bool GRAD = MODE != NORM_FORWARD, RMS = MODE == NORM_RMS_GRAD;
    extern __shared__ float col_sums[];  // [2][columns of the CTA] (gradients)
    __shared__ float slots[2][NORM_THREADS / 32][4];
    __shared__ float peers[2][8][4];
    const int tpr = 1 << a.tpr_log2, group = threadIdx.x >> a.tpr_log2, l = threadIdx.x & (tpr - 1);
    const int groups = blockDim.x >> a.tpr_log2;
    const int rank = a.cluster > 1 ? (int)cluster_rank() : 0;
    const int64_t first = (int64_t)(blockIdx.x / a.cluster) * groups + group;
    const int64_t step = (int64_t)(gridDim.x / a.cluster) * groups;
    const int c0 = rank * NORM_CTA_COLS;
    const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy);
    T *out = static_cast<T *>(a.out);
    const int col0 = c0 + l * V;  // of the thread's first access; the others lie tpr * V apart
    auto col = [&](int i) { return col0 + i * tpr * V; };
    float gm[NORM_EPT], second[NORM_EPT];  // second: beta, or the sums of d_gamma
    float db[GRAD && !RMS ? NORM_EPT : 1];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const bool in = col(i) < a.D;
            gm[i * V + j] = in ? a.gamma[col(i) + j] : 0.0f;
            second[i * V + j] = !GRAD && in && a.beta != nullptr ? a.beta[col(i) + j] : 0.0f;
            if (GRAD && !RMS) db[i * V + j] = 0.0f;
        }
    RowSum sum{slots, peers, tpr, (group << a.tpr_log2) >> 5, 1 + group, a.cluster};
    const float fd = (float)a.D;
    if (a.cluster > 1) cluster_sync();  // every CTA of the cluster runs before one stores into another
    Pack<T, V> nx[NV], nd[GRAD ? NV : 1];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (col(i) < a.D) {
                nx[i].load(x + row * a.x_stride + col(i));
                if (GRAD) nd[i].load(dy + row * a.dy_stride + col(i));
            }
    };
    if (first < a.N) fetch(first);
    for (int64_t row = first; row < a.N; row += step) {
        Pack<T, V> px[NV], pd[GRAD ? NV : 1];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            px[i] = nx[i];
            if (GRAD) pd[i] = nd[i];
        }
        if (row + step < a.N) fetch(row + step);
        float m = 0.0f;
        if (!RMS) {
            float s[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (col(i) < a.D)
#pragma unroll
                    for (int j = 0; j < V; ++j) s[0] += px[i].get(j);
            sum(s);
            m = __fdiv_rn(s[0], fd);
        }
        // the squared deviations; and of g and g (x - m)
        float s[GRAD ? (RMS ? 2 : 3) : 1] = {};
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (col(i) < a.D)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float d = px[i].get(j) - m;
                    s[0] = fmaf(d, d, s[0]);
                    if constexpr (GRAD) {
                        const float g = pd[i].get(j) * gm[i * V + j];
                        s[1] = fmaf(g, d, s[1]);
                        if constexpr (!RMS) s[2] += g;
                    }
                }
        sum(s);
        const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(s[0], fd) + a.eps));
        float mg = 0.0f, mgh = 0.0f;
        if constexpr (GRAD) {
            mgh = __fdiv_rn(s[1] * r, fd);
            if constexpr (!RMS) mg = __fdiv_rn(s[2], fd);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (col(i) < a.D) {
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int n = i * V + j;
                    const float h = (px[i].get(j) - m) * r;
                    if constexpr (GRAD) {
                        const float d = pd[i].get(j);
                        second[n] = fmaf(d, h, second[n]);
                        if constexpr (!RMS) db[n] += d;
                        o[j] = r * (fmaf(d, gm[n], -mg) - h * mgh);
                    } else {
                        o[j] = fmaf(h, gm[n], second[n]);
                    }
                }
                Pack<T, V> p;
                p.set(o);
                p.store(out + row * a.out_stride + col(i));
            }
    }
    if constexpr (GRAD) {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        // the rows' groups one after the other; a group's columns are apart
        const int cols = min(a.D - c0, NORM_CTA_COLS);
        float *sg = col_sums, *sb = col_sums + cols;
        for (int g = 0; g < groups; ++g) {
            if (group == g)
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (col(i) < a.D)
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const int c = col(i) - c0 + j;
                            sg[c] = g ? sg[c] + second[i * V + j] : second[i * V + j];
                            if constexpr (!RMS) sb[c] = g ? sb[c] + db[i * V + j] : db[i * V + j];
                        }
            __syncthreads();
        }
        float *to = a.part ? a.part + (int64_t)(blockIdx.x / a.cluster) * 2 * a.D : a.d_gamma;
        float *to_b = a.part ? to + a.D : a.d_beta;
        for (int c = threadIdx.x; c < cols; c += blockDim.x) {
            to[c0 + c] = sg[c];
            if (!RMS && to_b != nullptr) to_b[c0 + c] = sb[c];
        }
    }
}

// The partial sums of 32 columns: each warp adds every SUM_SLICES-th of them, then the warps' sums in order.
__global__ void __launch_bounds__(SUM_SLICES * 32) norm_sum_kernel(const float *__restrict__ part, int n, int D,
                                                                  float *__restrict__ d_gamma, float *__restrict__ d_beta) {
    __shared__ float s[SUM_SLICES][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const float *p = part + (blockIdx.y ? D : 0) + c;
    float v = 0.0f;
    if (c < D)
#pragma unroll 4
        for (int i = slice; i < n; i += SUM_SLICES) v += p[(int64_t)i * 2 * D];
    s[slice][lane] = v;
    __syncthreads();
    if (slice == 0 && c < D) {
        for (int i = 1; i < SUM_SLICES; ++i) v += s[i][lane];
        (blockIdx.y ? d_beta : d_gamma)[c] = v;
    }
}

int norm_cluster(int D) {
    int c = 1;
    while (c * NORM_CTA_COLS < D) c *= 2;
    return c;
}

// Launches MODE for element type T; rows in 16-byte, 4-byte or single-element accesses, as pointers and strides allow.
template <typename T, int MODE>
int launch_norm_typed(NormArgs a, void *scratch, cudaStream_t s) {
    constexpr bool GRAD = MODE != NORM_FORWARD;
    const int sms = std::max(1, device_sm_count());
    uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.out);
    bits |= (uintptr_t)((a.x_stride | a.dy_stride | a.out_stride | a.D) * (int64_t)sizeof(T));
    a.cluster = norm_cluster(a.D);
    const int cols = std::min(a.D, NORM_CTA_COLS);
    int l2 = 5;
    while ((NORM_EPT << l2) < cols) ++l2;
    if (a.cluster > 1) l2 = 9;
    // A row a CTA while there are SMs to spare (few rows answer soonest spread out), else all that fit
    int groups = a.cluster > 1 ? 1 : NORM_THREADS >> l2;
    while (groups > 1 && (int64_t)a.N < (int64_t)sms * groups) groups /= 2;
    a.tpr_log2 = l2;
    const int64_t turns = ((int64_t)a.N + groups - 1) / groups;
    const int64_t most = std::max<int64_t>(1, (int64_t)sms * (NORM_THREADS / (groups << l2)) * (GRAD ? 1 : 2) / a.cluster);
    const int clusters = (int)std::min<int64_t>({turns, most, NORM_PARTS});
    a.part = GRAD && clusters > 1 ? static_cast<float *>(scratch) : nullptr;
    const size_t smem = GRAD ? (size_t)2 * cols * 4 : 0;
    auto go = [&](auto kernel, SmemOptIn *done) {
        if (GRAD)
            if (int rc = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), 2 * NORM_CTA_COLS * 4, done)) return rc;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)(clusters * a.cluster));
        cfg.blockDim = dim3((unsigned)(groups << l2));
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)a.cluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = a.cluster > 1 ? 1 : 0;
        return cuda_status(cudaLaunchKernelEx(&cfg, kernel, a));
    };
    static SmemOptIn done[3];
    int rc;
    if (bits % 16 == 0)
        rc = go(norm_kernel<T, 16 / sizeof(T), MODE>, &done[0]);
    else if (sizeof(T) == 2 && bits % 4 == 0)
        rc = go(norm_kernel<T, 4 / sizeof(T), MODE>, &done[1]);
    else
        rc = go(norm_kernel<T, 1, MODE>, &done[2]);
    if (rc || a.part == nullptr) return rc;
    return launch_early(norm_sum_kernel, dim3((unsigned)((a.D + 31) / 32), a.d_beta ? 2 : 1), dim3(SUM_SLICES * 32), 0, s,
                        a.part, clusters, a.D, a.d_gamma, a.d_beta);
}

template <int MODE>
int launch_norm_mode(const NormArgs &a, int dtype, void *scratch, cudaStream_t s) {
    switch (dtype) {
        case MOE_DTYPE_F32: return launch_norm_typed<float, MODE>(a, scratch, s);
        case MOE_DTYPE_F16: return launch_norm_typed<__half, MODE>(a, scratch, s);
        default: return launch_norm_typed<__nv_bfloat16, MODE>(a, scratch, s);
    }
}

}  // namespace

size_t norm_scratch_bytes(int N, int D) { return (size_t)std::min(N, NORM_PARTS) * 2 * D * 4; }

int launch_layernorm(const void *x, int64_t x_stride, int dtype, const float *gamma, const float *beta, float eps, int N,
                     int D, void *y, int64_t y_stride, cudaStream_t s) {
    NormArgs a{};
    a.x = x;
    a.x_stride = x_stride;
    a.gamma = gamma;
    a.beta = beta;
    a.eps = eps;
    a.N = N;
    a.D = D;
    a.out = y;
    a.out_stride = y_stride;
    return launch_norm_mode<NORM_FORWARD>(a, dtype, nullptr, s);
}

int launch_norm_grad(bool rms, const void *d_y, int64_t d_y_stride, const void *x, int64_t x_stride, int dtype,
                     const float *gamma, float eps, int N, int D, void *d_x, int64_t d_x_stride, float *d_gamma,
                     float *d_beta, void *ws, cudaStream_t s) {
    NormArgs a{};
    a.x = x;
    a.x_stride = x_stride;
    a.dy = d_y;
    a.dy_stride = d_y_stride;
    a.gamma = gamma;
    a.eps = eps;
    a.N = N;
    a.D = D;
    a.out = d_x;
    a.out_stride = d_x_stride;
    a.d_gamma = d_gamma;
    a.d_beta = d_beta;
    void *scratch = ws_ptr<char>(ws, 256);
    return rms ? launch_norm_mode<NORM_RMS_GRAD>(a, dtype, scratch, s) : launch_norm_mode<NORM_GRAD>(a, dtype, scratch, s);
}

}  // namespace moe
