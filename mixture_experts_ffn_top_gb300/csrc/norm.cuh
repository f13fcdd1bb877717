// norm.cuh -- layer norm of token rows, its gradients, and the gradients of RMSNorm (norm.cu, norm_grad.cu):
//   y = gamma (x - m) r + beta,   m = mean(x), v = mean((x - m)^2), r = 1 / sqrt(v + eps)
//   with h = (x - m) r and g = gamma d_y, along each row:
//   d_x = r (g - mean(g) - h mean(g h)),   d_gamma = sum over rows of d_y h,   d_beta = sum over rows of d_y
//   (RMSNorm: m = 0, and no mean(g)).
//
// One pass over the data bounds it, if the instructions keep up: at the copy rate an SM has some 350 cycles for a row
// of 2048 16-bit values (520 with its gradient), so the fixed cost of a row -- sums across threads, the root, addresses
// -- must be shared by few warps, and arithmetic goes by pairs (add, mul, fma.f32x2).  A row is read once and stays in
// registers (or a tile in shared memory) between the sums over it and its result, while the next rows fly.  A thread
// keeps the same columns for all its rows, so that the column sums d_gamma and d_beta grow in its registers and leave
// the CTA once; a second kernel adds the CTAs' sums in order.  The gradient forms m and r again from the row it holds
// anyway: nothing is saved by the forward pass.  The variance is summed from the deviations (a second sum over the
// registers), not from squares: rows far off centre lose nothing.  Rows too long for a CTA are shared by a cluster of
// CTAs, whose sums meet in distributed shared memory.
// bf16, 8192 x 2048, from a graph: forward 15.4 us, 4.4 TB/s of the reads and writes its results need (the 33 MB written
// stay in L2; floor 9.9 us); gradient 29.3 us, 3.4 TB/s (14.8 us).  An SM takes 54 of these rows; what is left above the
// floors is the first rows' latency, the last rows' tail, the second kernel, and instructions.
#pragma once

#include <algorithm>

#include "elem.cuh"
#include "pair.cuh"

namespace moe {

namespace {

constexpr int NORM_THREADS = 512;
constexpr int NORM_CTA_COLS = 16384;  // columns of a CTA at most: gamma and beta, or two column sums, in shared memory
constexpr size_t NORM_SMEM = 200 * 1024;
constexpr int SUM_SLICES = 32;  // warps over the partial sums of 32 columns

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
    int tpr_log2;            // threads a row (of a CTA)
    int cluster, cta_cols;   // CTAs a row and the columns of each
    int stages;              // rows of a group's ring (gradients)
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

__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
template <typename E>
__device__ __forceinline__ E both(float a);
template <>
__device__ __forceinline__ F2 both<F2>(float a) { return pair_of(a, a); }
template <>
__device__ __forceinline__ float both<float>(float a) { return a; }
__device__ __forceinline__ float total(F2 p) {
    const float2 v = values_of(p);
    return v.x + v.y;
}
__device__ __forceinline__ float total(float v) { return v; }

// Unit j of an access: its elements 2 j and 2 j + 1, or its only one.
template <typename E, typename T, int V>
__device__ __forceinline__ E unit(const Pack<T, V> &p, int j) {
    if constexpr (V == 1)
        return p.get(0);
    else
        return pair_of(p.get(2 * j), p.get(2 * j + 1));
}

// The fp32 values of vector `v` out of `nvec` of V, as store_vec lays them out: halves of 8 apart, so that lanes with
// neighbouring vectors read without bank conflicts.
template <int V, typename E>
__device__ __forceinline__ void load_vec(const float *s, int v, int nvec, E *f) {
    if constexpr (V >= 4) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(s + (j / 4 * nvec + v) * 4);
            f[j / 2] = pair_of(q.x, q.y), f[j / 2 + 1] = pair_of(q.z, q.w);
        }
    } else if constexpr (V == 2) {
        const float2 q = *reinterpret_cast<const float2 *>(s + v * 2);
        f[0] = pair_of(q.x, q.y);
    } else {
        f[0] = s[v];
    }
}
template <int V>
__device__ __forceinline__ int vec_place(int c, int nvec) {  // of column c
    return V == 8 ? ((c >> 2 & 1) * nvec + (c >> 3)) * 4 + (c & 3) : c;
}

template <int BYTES>
__device__ __forceinline__ void copy_async(void *to, const void *from) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(a), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(a), "l"(from), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows in registers: the forward norm of few rows (gamma and beta in registers) and of rows that are not aligned or
// longer than 16384 columns, gradients of rows too long for tiles (all SMEM: gamma and beta in shared memory).
// T, V: elements and how many of them an access has; NV accesses a thread.
template <typename T, int V, int NV, int MODE, bool SMEM>
__global__ void __launch_bounds__(NORM_THREADS, 1) norm_kernel(const NormArgs a) {
    constexpr bool GRAD = MODE != NORM_FORWARD, RMS = MODE == NORM_RMS_GRAD;
    constexpr int BYTES = V * sizeof(T);
    using E = std::conditional_t<V == 1, float, F2>;
    constexpr int P = V == 1 ? 1 : V / 2;  // units of E an access
    static_assert(SMEM || !GRAD);
    constexpr bool RING = GRAD && BYTES >= 4;  // 2-byte accesses have no asynchronous copy
    constexpr int VECS = GRAD ? 1 : 2;          // gamma, or gamma and beta, in shared memory
    extern __shared__ __align__(16) char smem[];
    __shared__ float slots[2][NORM_THREADS / 32][4];
    __shared__ float peers[2][8][4];
    const int tid = threadIdx.x, tpr = 1 << a.tpr_log2, group = tid >> a.tpr_log2, l = tid & (tpr - 1);
    const int groups = blockDim.x >> a.tpr_log2;
    const int rank = a.cluster > 1 ? (int)cluster_rank() : 0;
    const int first = (blockIdx.x / a.cluster) * groups + group, step = (gridDim.x / a.cluster) * groups;
    const int c0 = rank * a.cta_cols, cols = min(a.cta_cols, a.D - c0), nvec = cols / V;
    const int have = l < nvec ? (nvec - l + tpr - 1) >> a.tpr_log2 : 0;  // accesses of this thread
    auto in = [&](int i) { return i < have; };
    const int at = l * V, apart = tpr * V;  // column of its first access, and from each to the next
    const T *x = static_cast<const T *>(a.x) + c0 + at;
    const T *dy = static_cast<const T *>(a.dy) + c0 + at;
    T *out = static_cast<T *>(a.out) + c0 + at;
    float *gs = reinterpret_cast<float *>(smem), *bs = gs + cols;

    // gradients: a.stages rows ahead in shared memory, each thread's own pieces; else the next row in registers
    char *ring = smem + (size_t)cols * 4 + (size_t)tid * BYTES;
    const int piece = blockDim.x * BYTES;  // from one access to the next in the ring
    int fill = 0, slot = 0;
    auto push = [&](int row) {
        if (row < a.N) {
            char *to = ring + fill * 2 * NV * piece;
            const T *px = x + (int64_t)row * a.x_stride, *pd = dy + (int64_t)row * a.dy_stride;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in(i)) {
                    copy_async<RING ? BYTES : 16>(to + i * piece, px + i * apart);
                    copy_async<RING ? BYTES : 16>(to + (NV + i) * piece, pd + i * apart);
                }
        }
        copies_commit();
        if (++fill == a.stages) fill = 0;
    };
    Pack<T, V> nx[GRAD ? 1 : NV];
    auto fetch = [&](int row) {
        const T *px = x + (int64_t)row * a.x_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in(i)) nx[GRAD ? 0 : i].load(px + i * apart);
    };
    if constexpr (RING)
        for (int i = 0; i < a.stages - 1; ++i) push(first + i * step);
    else if (!GRAD && first < a.N)
        fetch(first);
    E gm[SMEM ? 1 : NV * P], bt[SMEM ? 1 : NV * P];
    if constexpr (SMEM) {
        for (int c = tid; c < cols; c += blockDim.x) {
            gs[vec_place<V>(c, nvec)] = a.gamma[c0 + c];
            if (VECS == 2) bs[vec_place<V>(c, nvec)] = a.beta != nullptr ? a.beta[c0 + c] : 0.0f;
        }
        __syncthreads();
    } else {
        auto read = [&](const float *p, int i, int j) {
            const float *q = p + c0 + at + i * apart + (V == 1 ? 0 : 2 * j);
            if constexpr (V == 1)
                return *q;
            else
                return pair_of(q[0], q[1]);
        };
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < P; ++j) {
                gm[i * P + j] = in(i) ? read(a.gamma, i, j) : both<E>(0.0f);
                bt[i * P + j] = in(i) && a.beta != nullptr ? read(a.beta, i, j) : both<E>(0.0f);
            }
    }
    E dg[GRAD ? NV * P : 1], db[GRAD && !RMS ? NV * P : 1];
#pragma unroll
    for (int n = 0; n < (GRAD ? NV * P : 1); ++n) {
        dg[n] = both<E>(0.0f);
        if constexpr (GRAD && !RMS) db[n] = both<E>(0.0f);
    }
    RowSum sum{slots, peers, tpr, (group << a.tpr_log2) >> 5, 1 + group, a.cluster};
    const float inv = 1.0f / (float)a.D;
    if (a.cluster > 1) cluster_sync();  // every CTA of the cluster runs before one stores into another

    for (int row = first; row < a.N; row += step) {
        Pack<T, V> px[NV], pd[GRAD ? NV : 1];
        if constexpr (RING) {
            push(row + (a.stages - 1) * step);
            if (a.stages == 3)
                copies_wait<2>();
            else
                copies_wait<1>();
            const char *from = ring + slot * 2 * NV * piece;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in(i)) {
                    px[i].load(reinterpret_cast<const T *>(from + i * piece));
                    pd[i].load(reinterpret_cast<const T *>(from + (NV + i) * piece));
                }
            if (++slot == a.stages) slot = 0;
        } else if constexpr (GRAD) {
            const T *qx = x + (int64_t)row * a.x_stride, *qd = dy + (int64_t)row * a.dy_stride;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in(i)) {
                    px[i].load(qx + i * apart);
                    pd[i].load(qd + i * apart);
                }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) px[i] = nx[i];
            if (row + step < a.N) fetch(row + step);
        }
        float m = 0.0f;
        if constexpr (!RMS) {
            E s0 = both<E>(0.0f), s1 = s0;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in(i))
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        E &t = (i * P + j) % 2 ? s1 : s0;
                        t = add(t, unit<E>(px[i], j));
                    }
            float s[1] = {total(add(s0, s1))};
            sum(s);
            m = s[0] * inv;
        }
        // the squared deviations; and of g and g (x - m)
        const E minus_m = both<E>(-m);
        E q2 = both<E>(0.0f), qgd = q2, qg = q2;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in(i)) {
                E gv[P];
                if constexpr (GRAD) load_vec<V>(gs, l + i * tpr, nvec, gv);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const E d = RMS ? unit<E>(px[i], j) : add(unit<E>(px[i], j), minus_m);
                    q2 = fma(d, d, q2);
                    if constexpr (GRAD) {
                        const E g = mul(unit<E>(pd[i], j), gv[j]);
                        qgd = fma(g, d, qgd);
                        if constexpr (!RMS) qg = add(qg, g);
                    }
                }
            }
        float s[GRAD ? (RMS ? 2 : 3) : 1];
        s[0] = total(q2);
        if constexpr (GRAD) {
            s[1] = total(qgd);
            if constexpr (!RMS) s[2] = total(qg);
        }
        sum(s);
        const float r = rsqrtf(fmaf(s[0], inv, a.eps));  // within two units in the last place
        const E rr = both<E>(r);
        E minus_mg = both<E>(0.0f), minus_mgh = minus_mg;
        if constexpr (GRAD) {
            minus_mgh = both<E>(-(s[1] * r * inv));
            if constexpr (!RMS) minus_mg = both<E>(-(s[2] * inv));
        }
        T *to = out + (int64_t)row * a.out_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in(i)) {
                E gv[P], bv[P];
                float o[V];
                if constexpr (SMEM) {
                    load_vec<V>(gs, l + i * tpr, nvec, gv);
                    if constexpr (!GRAD) load_vec<V>(bs, l + i * tpr, nvec, bv);
                } else {
#pragma unroll
                    for (int j = 0; j < P; ++j) gv[j] = gm[i * P + j], bv[j] = bt[i * P + j];
                }
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const E h = mul(RMS ? unit<E>(px[i], j) : add(unit<E>(px[i], j), minus_m), rr);
                    E y;
                    if constexpr (GRAD) {
                        const E d = unit<E>(pd[i], j);
                        dg[i * P + j] = fma(d, h, dg[i * P + j]);
                        if constexpr (!RMS) db[i * P + j] = add(db[i * P + j], d);
                        y = mul(rr, fma(h, minus_mgh, RMS ? mul(d, gv[j]) : fma(d, gv[j], minus_mg)));
                    } else {
                        y = fma(h, gv[j], bv[j]);
                    }
                    if constexpr (V == 1) {
                        o[0] = y;
                    } else {
                        const float2 v = values_of(y);
                        o[2 * j] = v.x, o[2 * j + 1] = v.y;
                    }
                }
                Pack<T, V> p;
                p.set(o);
                p.store(to + i * apart);
            }
    }
    if constexpr (GRAD) {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        if (RING) copies_wait<0>();
        __syncthreads();  // the shared memory serves the sums now
        float *sg = reinterpret_cast<float *>(smem), *sb = sg + cols;
        // (the whole CTA works on a row: shorter ones go by tiles)
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in(i))
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int c = vec_place<V>(at + i * apart + j, nvec);
                    auto one = [&](const E *e) {
                        if constexpr (V == 1) {
                            return e[i];
                        } else {
                            const float2 v = values_of(e[i * P + j / 2]);
                            return j % 2 ? v.y : v.x;
                        }
                    };
                    sg[c] = one(dg);
                    if constexpr (!RMS) sb[c] = one(db);
                }
        __syncthreads();
        float *to = a.part ? a.part + (int64_t)(blockIdx.x / a.cluster) * 2 * a.D : a.d_gamma;
        float *to_b = a.part ? to + a.D : a.d_beta;
        for (int c = tid; c < cols; c += blockDim.x) {
            to[c0 + c] = sg[vec_place<V>(c, nvec)];
            if (!RMS && to_b != nullptr) to_b[c0 + c] = sb[vec_place<V>(c, nvec)];
        }
    }
}

// --------------------------------------------- gradients of many rows ---
// A CTA takes tiles of rows into shared memory, three of them in flight or at work, and goes through each twice: a warp
// forms the statistics of a row (or of a part of it: up to 1024 columns, in registers), then every thread finishes
// its own columns of all the tile's rows, gamma and the column sums in its registers.  Either half needs little of
// what the other keeps, so that two CTAs of 256 threads share an SM and fill each other's waits.  A part's sums of
// deviations are about its own mean; parts are put together by
//   M2 = sum M2_p + n_p (m_p - m)^2,   sum g (x - m) = sum C_p + (m_p - m) G_p.
constexpr int TILE_ROWS = 32;        // of a tile at most
constexpr int TILE_PARTS = 8;        // of a row at most
constexpr int TILE_MAX_D = 8192;
constexpr int TILE_MAX_BYTES = 32768;  // of a row of x and of d_y
constexpr int TILE_STAGES = 3;
constexpr size_t TILE_SMEM = 216 * 1024;
constexpr int LANE_UNITS = 8;        // units of 4 columns a lane holds

struct TileArgs {
    NormArgs n;
    int rows, parts, part_units;  // rows of a tile, parts of a row and units of each
    int pitch;                    // bytes from one row to the next in shared memory
    int split_log2;               // threads on a row's units: 1 << split_log2
    int load_bytes;               // accesses of 16 or 4 bytes
    int chunks, step_rows, step_chunks;  // accesses a row; from one access of a thread to its next
    uintptr_t lo[2], hi[2];       // SHIFT: where x and d_y begin and end
};

// Unit u of a row; SHIFT: of `left` columns from it on, the row `at` (even, below 16) bytes behind its place: whole
// words are read and shifted by two bytes where need be, columns behind the end are zeros.
template <typename T, bool SHIFT>
__device__ __forceinline__ void load_unit(const char *row, int u, F2 &a, F2 &b, int at = 0, int left = 4) {
    Pack<T, 4> p;
    if constexpr (SHIFT) {
        const uint2 *q = reinterpret_cast<const uint2 *>(row + (at & 8)) + u;
        const uint2 l = q[0], h = q[1];
        const bool word = at & 4;
        const uint32_t w0 = word ? l.y : l.x, w1 = word ? h.x : l.y, w2 = word ? h.y : h.x, how = at & 2 ? 0x5432 : 0x3210;
        p.w[0] = __byte_perm(w0, w1, how);
        p.w[1] = __byte_perm(w1, w2, how);
        if (left < 4) {
            p.w[0] &= left < 2 ? 0xffffu : 0xffffffffu;
            p.w[1] &= left < 3 ? 0u : 0xffffu;
        }
    } else {
        p.load(reinterpret_cast<const T *>(row) + u * 4);
    }
    a = pair_of(p.get(0), p.get(1));
    b = pair_of(p.get(2), p.get(3));
}
__device__ __forceinline__ void load_pairs(const float4 *p, F2 &a, F2 &b) {
    const float4 v = *p;
    a = pair_of(v.x, v.y);
    b = pair_of(v.z, v.w);
}

// NU: units a thread finishes.  FULL: every lane has all its units, and every thread (no conditions inside).  SHIFT
// (16-bit rows an odd number of elements apart, or at odd places): a row comes in whole 16-byte pieces, as far from one
// in shared memory as in global memory, what they hold beside it ignored (pieces that pass the ends of x or d_y come by
// elements), is shifted into place as it is read, and its results leave as pairs that neighbouring lanes complete. 
// 8192 x 2047 bf16 51 us, by elements 148 (rows on 4 bytes, copied and stored 4 bytes at a time, need no shifting).
template <typename T, bool RMS, int NU, int THREADS, bool FULL, bool SHIFT>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) norm_tile_kernel(const TileArgs t) {
    const NormArgs &a = t.n;
    extern __shared__ __align__(16) char smem[];
    __shared__ float4 parts_s[TILE_ROWS * TILE_PARTS];
    __shared__ float4 stat_s[TILE_ROWS][2];  // (-m, -m, r, r), (-mean g twice, -mean gh twice)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int threads = THREADS, warps = THREADS / 32;
    const int D = a.D, units = (D + 3) / 4, R = t.rows, tiles = (a.N + R - 1) / R;
    const int array = R * t.pitch, stage = 2 * array;
    float *gs = reinterpret_cast<float *>(smem + TILE_STAGES * stage);  // gamma, for the statistics
    const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy);

    const int load_r = tid / t.chunks, load_c = tid - load_r * t.chunks;
    auto piece = [&](const T *row, int c, char *dst, int which) {
        const uintptr_t from = (reinterpret_cast<uintptr_t>(row) & ~(uintptr_t)15) + c * 16, end = reinterpret_cast<uintptr_t>(row + D);
        if (from >= end) return;
        if (from >= t.lo[which] && from + 16 <= t.hi[which]) {
            copy_async<16>(dst, reinterpret_cast<const void *>(from));
        } else {
            for (int i = 0; i < 16; i += 2)
                if (from + i >= reinterpret_cast<uintptr_t>(row) && from + i < end)
                    *reinterpret_cast<uint16_t *>(dst + i) = *reinterpret_cast<const uint16_t *>(from + i);
        }
    };
    // how far (in bytes) a row lies behind a multiple of 16
    const unsigned x_at = reinterpret_cast<uintptr_t>(x) & 15, x_by = (unsigned)(a.x_stride * 2) & 15;
    const unsigned d_at = reinterpret_cast<uintptr_t>(dy) & 15, d_by = (unsigned)(a.dy_stride * 2) & 15;
    auto load = [&](int tile, int slot) {
        if (tile < tiles) {
            const int r0 = tile * R, n = min(R, a.N - r0);
            char *to = smem + slot * stage;
            for (int r = load_r, c = load_c; r < n;) {
                const T *row_x = x + (int64_t)(r0 + r) * a.x_stride, *row_d = dy + (int64_t)(r0 + r) * a.dy_stride;
                char *dst = to + r * t.pitch + c * t.load_bytes;
                if constexpr (SHIFT) {
                    piece(row_x, c, dst, 0);
                    piece(row_d, c, dst + array, 1);
                } else {
                    const char *px = reinterpret_cast<const char *>(row_x) + c * t.load_bytes;
                    const char *pd = reinterpret_cast<const char *>(row_d) + c * t.load_bytes;
                    if (t.load_bytes == 16) {
                        copy_async<16>(dst, px);
                        copy_async<16>(dst + array, pd);
                    } else {
                        copy_async<4>(dst, px);
                        copy_async<4>(dst + array, pd);
                    }
                }
                r += t.step_rows;
                c += t.step_chunks;
                if (c >= t.chunks) c -= t.chunks, ++r;
            }
        }
        copies_commit();
    };
    if (!SHIFT && D % 4 != 0)  // the columns behind a row's end count as zeros
        for (int i = tid; i < TILE_STAGES * 2 * R; i += threads)
            for (int c = D; c < units * 4; ++c) reinterpret_cast<T *>(smem + i * t.pitch)[c] = elem_of<T>(0.0f);
    const int step = gridDim.x;
    load(blockIdx.x, 0);
    load(blockIdx.x + step, 1);

    // the thread's columns and its share of the rows
    const int split = 1 << t.split_log2, u0 = tid & (split - 1), share = tid >> t.split_log2, shares = threads >> t.split_log2;
    F2 gm[2 * NU], dg[2 * NU], db[RMS ? 1 : 2 * NU];
#pragma unroll
    for (int j = 0; j < NU; ++j) {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = (u0 + j * split) * 4 + i;
            f[i] = c < D ? a.gamma[c] : 0.0f;
        }
        gm[2 * j] = pair_of(f[0], f[1]);
        gm[2 * j + 1] = pair_of(f[2], f[3]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            dg[2 * j + i] = pair_of(0.0f, 0.0f);
            if constexpr (!RMS) db[2 * j + i] = pair_of(0.0f, 0.0f);
        }
    }
    for (int c = tid; c < units * 4; c += threads) gs[c] = c < D ? a.gamma[c] : 0.0f;
    const float inv = 1.0f / (float)D;
    const bool pairs = split >= 32;  // a warp's lanes are neighbours of one row
    const uint32_t mask = pairs ? 0xffffffffu : ((1u << split) - 1) << (lane & ~(split - 1));  // the lanes of its row
    int slot = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += step) {
        copies_wait<1>();
        __syncthreads();  // this tile is there, and the one before it has been used
        load(tile + 2 * step, slot == 0 ? TILE_STAGES - 1 : slot - 1);
        const char *xs = smem + slot * stage, *ds = xs + array;
        const int n = min(R, a.N - tile * R);
        // ---- statistics
        for (int job = warp; job < n * t.parts; job += warps) {
            const int row = t.parts == 1 ? job : job / t.parts, part = job - row * t.parts;
            const int first = part * t.part_units, mine = min(t.part_units, units - first);  // units
            const char *xr = xs + row * t.pitch, *dr = ds + row * t.pitch;
            const int xa = (x_at + (tile * R + row) * x_by) & 15, da = (d_at + (tile * R + row) * d_by) & 15;
            F2 v[LANE_UNITS][2], s0 = pair_of(0.0f, 0.0f), s1 = s0;
#pragma unroll
            for (int i = 0; i < LANE_UNITS; ++i)
                if (FULL || lane + 32 * i < mine) {
                    load_unit<T, SHIFT>(xr, first + lane + 32 * i, v[i][0], v[i][1], xa, D - (first + lane + 32 * i) * 4);
                    if constexpr (!RMS) s0 = add(s0, v[i][0]), s1 = add(s1, v[i][1]);
                }
            float m = 0.0f;
            if constexpr (!RMS) m = __fdividef(warp_sum(total(add(s0, s1))), (float)min(mine * 4, D - first * 4));
            const F2 minus_m = both<F2>(-m);
            F2 q0 = pair_of(0.0f, 0.0f), q1 = q0, c0 = q0, c1 = q0, g0 = q0, g1 = q0;
#pragma unroll
            for (int i = 0; i < LANE_UNITS; ++i)
                if (FULL || lane + 32 * i < mine) {
                    const int u = first + lane + 32 * i;
                    F2 d0 = RMS ? v[i][0] : add(v[i][0], minus_m), d1 = RMS ? v[i][1] : add(v[i][1], minus_m);
                    if (!FULL && !RMS && u * 4 + 4 > D) {  // not the columns behind the end
                        float2 e = values_of(d0), f = values_of(d1);
                        e.y = u * 4 + 1 < D ? e.y : 0.0f;
                        f.x = u * 4 + 2 < D ? f.x : 0.0f;
                        d0 = pair_of(e.x, e.y);
                        d1 = pair_of(f.x, 0.0f);
                    }
                    F2 y0, y1, w0, w1;
                    load_unit<T, SHIFT>(dr, u, y0, y1, da, D - u * 4);
                    load_pairs(reinterpret_cast<const float4 *>(gs) + u, w0, w1);
                    y0 = mul(y0, w0), y1 = mul(y1, w1);
                    q0 = fma(d0, d0, q0), q1 = fma(d1, d1, q1);
                    c0 = fma(y0, d0, c0), c1 = fma(y1, d1, c1);
                    if constexpr (!RMS) g0 = add(g0, y0), g1 = add(g1, y1);
                }
            float4 p;
            p.x = m;
            p.y = warp_sum(total(add(q0, q1)));
            p.z = warp_sum(total(add(c0, c1)));
            p.w = RMS ? 0.0f : warp_sum(total(add(g0, g1)));
            if (lane == 0) parts_s[job] = p;
        }
        __syncthreads();
        if (tid < n) {
            float4 p = parts_s[tid * t.parts];
            if (t.parts > 1) {
                auto count = [&](int i) { return (float)(min((i + 1) * t.part_units * 4, D) - i * t.part_units * 4); };
                float m = 0.0f, q = 0.0f, c = 0.0f, g = 0.0f;
                if constexpr (!RMS)
                    for (int i = 0; i < t.parts; ++i) m = fmaf(parts_s[tid * t.parts + i].x, count(i) * inv, m);
                for (int i = 0; i < t.parts; ++i) {
                    const float4 e = parts_s[tid * t.parts + i];
                    const float d = RMS ? 0.0f : e.x - m;
                    q += fmaf(count(i) * d, d, e.y);
                    c += fmaf(d, e.w, e.z);
                    g += e.w;
                }
                p = make_float4(m, q, c, g);
            }
            const float r = rsqrtf(fmaf(p.y, inv, a.eps));  // within two units in the last place
            const float mg = p.w * inv, mgh = p.z * r * inv;
            stat_s[tid][0] = make_float4(-p.x, -p.x, r, r);
            stat_s[tid][1] = make_float4(-mg, -mg, -mgh, -mgh);
        }
        __syncthreads();
        // ---- the results
        T *out = static_cast<T *>(a.out) + (int64_t)tile * R * a.out_stride;
#pragma unroll 2
        for (int row = share; row < n; row += shares) {
            F2 minus_m, rr, minus_mg, minus_mgh;
            load_pairs(&stat_s[row][0], minus_m, rr);
            load_pairs(&stat_s[row][1], minus_mg, minus_mgh);
            T *to = out + (int64_t)row * a.out_stride;
            const int xa = (x_at + (tile * R + row) * x_by) & 15, da = (d_at + (tile * R + row) * d_by) & 15;
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                const int u = u0 + j * split;
                if (SHIFT ? __all_sync(mask, u >= units) : !FULL && u >= units) break;
                const int at = SHIFT ? min(u, units - 1) : u;
                F2 v[2], d[2];
                load_unit<T, SHIFT>(xs + row * t.pitch, at, v[0], v[1], xa);
                load_unit<T, SHIFT>(ds + row * t.pitch, at, d[0], d[1], da);  // (what stands behind the end is not stored)
                float o[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int e = 2 * j + i;
                    const F2 h = mul(RMS ? v[i] : add(v[i], minus_m), rr);
                    dg[e] = fma(d[i], h, dg[e]);
                    if constexpr (!RMS) db[e] = add(db[e], d[i]);
                    const float2 f = values_of(mul(rr, fma(h, minus_mgh, RMS ? mul(d[i], gm[e]) : fma(d[i], gm[e], minus_mg))));
                    o[2 * i] = f.x, o[2 * i + 1] = f.y;
                }
                Pack<T, 4> p;
                p.set(o);
                if constexpr (SHIFT) {
                    const uint32_t next = __shfl_down_sync(mask, p.w[0], 1);
                    // half a word off: the lane before stores the first result, this one the next lane's with its last
                    const bool off = reinterpret_cast<uintptr_t>(to) & 2, joined = off && pairs && lane > 0;
                    if (u * 4 + 4 <= D && (!off || pairs)) {
                        T *q = to + u * 4;
                        if (off) {
                            if (!joined) q[0] = elem_of<T>(o[0]);
                            *reinterpret_cast<uint32_t *>(q + 1) = __byte_perm(p.w[0], p.w[1], 0x5432);
                            if (lane < 31 && u + 1 < units)
                                *reinterpret_cast<uint32_t *>(q + 3) = __byte_perm(p.w[1], next, 0x5432);
                            else
                                q[3] = elem_of<T>(o[3]);
                        } else {
                            reinterpret_cast<uint32_t *>(q)[0] = p.w[0];
                            reinterpret_cast<uint32_t *>(q)[1] = p.w[1];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (u * 4 + i < D && !(i == 0 && joined)) to[u * 4 + i] = elem_of<T>(o[i]);
                    }
                } else if (FULL || t.load_bytes == 16) {
                    p.store(to + u * 4);
                } else {  // 4 bytes at a time
                    constexpr int W = 4 / sizeof(T);
#pragma unroll
                    for (int i = 0; i < 4 / W; ++i)
                        if (u * 4 + i * W < D) reinterpret_cast<uint32_t *>(to + u * 4)[i] = p.w[i];
                }
            }
        }
        if (++slot == TILE_STAGES) slot = 0;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    copies_wait<0>();
    __syncthreads();  // the shared memory serves the sums now
    float4 *sg = reinterpret_cast<float4 *>(smem), *sb = sg + units;
    for (int g = 0; g < shares; ++g) {  // the rows' shares one after the other
        if (share == g)
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                const int u = u0 + j * split;
                if (u >= units) break;
                auto put = [&](float4 &s, F2 lo, F2 hi) {
                    const float2 l = values_of(lo), h = values_of(hi);
                    s = g ? make_float4(s.x + l.x, s.y + l.y, s.z + h.x, s.w + h.y) : make_float4(l.x, l.y, h.x, h.y);
                };
                put(sg[u], dg[2 * j], dg[2 * j + 1]);
                if constexpr (!RMS) put(sb[u], db[2 * j], db[2 * j + 1]);
            }
        __syncthreads();
    }
    float *to = a.part ? a.part + (int64_t)blockIdx.x * 2 * D : a.d_gamma;
    float *to_b = a.part ? to + D : a.d_beta;
    for (int c = tid; c < D; c += threads) {
        to[c] = reinterpret_cast<const float *>(sg)[c];
        if (!RMS && to_b != nullptr) to_b[c] = reinterpret_cast<const float *>(sb)[c];
    }
}

// ------------------------------------------------ forward, many rows ---
// A row's values stay in registers as fp32 pairs, NP of 8 (or 4) elements a thread, converted once; the next row's
// flies packed.  FULL: every thread has all its accesses.
template <typename T, int NP, bool FULL>
__global__ void __launch_bounds__(NORM_THREADS, 1) norm_rows_kernel(const NormArgs a) {
    constexpr int V = 16 / sizeof(T), P = V / 2;
    extern __shared__ __align__(16) char smem[];
    __shared__ float slots[2][NORM_THREADS / 32][4];
    const int tid = threadIdx.x, tpr = 1 << a.tpr_log2, group = tid >> a.tpr_log2, l = tid & (tpr - 1);
    const int groups = blockDim.x >> a.tpr_log2, nvec = a.D / V;
    const int first = blockIdx.x * groups + group, step = gridDim.x * groups;
    const int have = l < nvec ? (nvec - l + tpr - 1) >> a.tpr_log2 : 0;
    auto in = [&](int i) { return FULL || i < have; };
    const T *x = static_cast<const T *>(a.x) + l * V;
    T *out = static_cast<T *>(a.out) + l * V;
    const int apart = tpr * V;
    Pack<T, V> next[NP];
    auto fetch = [&](int row) {
        const T *p = x + (int64_t)row * a.x_stride;
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (in(i)) next[i].load(p + i * apart);
    };
    if (first < a.N) fetch(first);
    float *gs = reinterpret_cast<float *>(smem), *bs = gs + a.D;
    for (int c = tid; c < a.D; c += blockDim.x) {
        gs[vec_place<V>(c, nvec)] = a.gamma[c];
        bs[vec_place<V>(c, nvec)] = a.beta != nullptr ? a.beta[c] : 0.0f;
    }
    __syncthreads();
    RowSum sum{slots, nullptr, tpr, (group << a.tpr_log2) >> 5, 1 + group, 1};
    const float inv = 1.0f / (float)a.D;
    for (int row = first; row < a.N; row += step) {
        F2 v[NP][P], s0 = pair_of(0.0f, 0.0f), s1 = s0;
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (in(i))
#pragma unroll
                for (int j = 0; j < P; j += 2) {
                    v[i][j] = unit<F2>(next[i], j);
                    v[i][j + 1] = unit<F2>(next[i], j + 1);
                    s0 = add(s0, v[i][j]);
                    s1 = add(s1, v[i][j + 1]);
                }
        if (row + step < a.N) fetch(row + step);
        float s[1] = {total(add(s0, s1))};
        sum(s);
        const F2 minus_m = both<F2>(-s[0] * inv);
        F2 q0 = pair_of(0.0f, 0.0f), q1 = q0;
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (in(i))
#pragma unroll
                for (int j = 0; j < P; j += 2) {
                    v[i][j] = add(v[i][j], minus_m);
                    v[i][j + 1] = add(v[i][j + 1], minus_m);
                    q0 = fma(v[i][j], v[i][j], q0);
                    q1 = fma(v[i][j + 1], v[i][j + 1], q1);
                }
        s[0] = total(add(q0, q1));
        sum(s);
        const F2 rr = both<F2>(rsqrtf(fmaf(s[0], inv, a.eps)));  // within two units in the last place
        T *to = out + (int64_t)row * a.out_stride;
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (in(i)) {
                F2 gv[P], bv[P];
                load_vec<V>(gs, l + i * tpr, nvec, gv);
                load_vec<V>(bs, l + i * tpr, nvec, bv);
                float o[V];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const float2 f = values_of(fma(mul(v[i][j], rr), gv[j], bv[j]));
                    o[2 * j] = f.x, o[2 * j + 1] = f.y;
                }
                Pack<T, V> p;
                p.set(o);
                p.store(to + i * apart);
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
#pragma unroll 10
        for (int i = slice; i < n; i += SUM_SLICES) v += p[(int64_t)i * 2 * D];
    s[slice][lane] = v;
    __syncthreads();
    if (slice == 0 && c < D) {
        for (int i = 1; i < SUM_SLICES; ++i) v += s[i][lane];
        (blockIdx.y ? d_beta : d_gamma)[c] = v;
    }
}

template <typename T, int MODE>
int launch_norm_sum(const NormArgs &a, int clusters, cudaStream_t s) {
    return launch_early(norm_sum_kernel, dim3((unsigned)((a.D + 31) / 32), a.d_beta ? 2 : 1), dim3(SUM_SLICES * 32), 0, s,
                        a.part, clusters, a.D, a.d_gamma, a.d_beta);
}

template <typename T, int MODE>
int launch_norm_tiles(const NormArgs &n, int load_bytes, void *scratch, cudaStream_t s) {
    constexpr bool RMS = MODE == NORM_RMS_GRAD;
    const int sms = std::max(1, device_sm_count());
    TileArgs t{};
    t.n = n;
    t.load_bytes = load_bytes;
    const int units = (n.D + 3) / 4;
    const bool shift = load_bytes == 2;
    t.chunks = shift ? (n.D * 2 + 14 + 15) / 16 : n.D * (int)sizeof(T) / load_bytes;
    t.pitch = (units * 4 * (int)sizeof(T) + 15) / 16 * 16;
    if (shift) {
        t.load_bytes = 16;
        t.pitch = std::max((units * 8 + 16 + 15) / 16 * 16, t.chunks * 16);
        t.lo[0] = reinterpret_cast<uintptr_t>(n.x), t.hi[0] = t.lo[0] + ((n.N - 1) * n.x_stride + n.D) * 2;
        t.lo[1] = reinterpret_cast<uintptr_t>(n.dy), t.hi[1] = t.lo[1] + ((n.N - 1) * n.dy_stride + n.D) * 2;
    }
    // two CTAs of 256 threads an SM with rows up to 2048 columns, else one of 512
    const int threads = units <= 512 ? 256 : 512, nu = units <= 256 ? 1 : units <= 1024 ? 2 : 4;
    const int room = (threads == 512 ? 160 : 97) * 1024 / TILE_STAGES;
    t.rows = 1;
    while (2 * t.rows <= TILE_ROWS && 4 * t.rows * t.pitch <= room) t.rows *= 2;
    t.parts = 1;
    while (t.parts * 32 * LANE_UNITS < units) t.parts *= 2;
    t.part_units = (units + t.parts - 1) / t.parts;
    t.split_log2 = 0;
    while ((1 << t.split_log2) < std::min(units, threads)) ++t.split_log2;
    t.step_rows = threads / t.chunks;
    t.step_chunks = threads % t.chunks;
    const bool full = load_bytes == 16 && n.D % 4 == 0 && units == nu << t.split_log2 && t.part_units == 32 * LANE_UNITS &&
                      units % t.part_units == 0;
    const int64_t tiles = ((int64_t)n.N + t.rows - 1) / t.rows;
    const int grid = (int)std::min<int64_t>({tiles, (int64_t)sms * (512 / threads), NORM_PARTS});
    t.n.part = grid > 1 ? static_cast<float *>(scratch) : nullptr;
    const size_t smem = std::max((size_t)TILE_STAGES * 2 * t.rows * t.pitch + units * 16, (size_t)units * 32);
    auto go = [&](auto kernel, SmemOptIn *done) {
        if (int rc = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), TILE_SMEM, done)) return rc;
        kernel<<<grid, threads, smem, s>>>(t);
        return launch_status();
    };
    auto by_full = [&](auto nc, auto tc) {
        constexpr int NU = decltype(nc)::value, THREADS = decltype(tc)::value;
        static SmemOptIn done[3];
        if constexpr (sizeof(T) == 2)
            if (shift) return go(norm_tile_kernel<T, RMS, NU, THREADS, false, true>, &done[2]);
        return full ? go(norm_tile_kernel<T, RMS, NU, THREADS, true, false>, &done[0])
                    : go(norm_tile_kernel<T, RMS, NU, THREADS, false, false>, &done[1]);
    };
    using std::integral_constant;
    const int rc = nu == 1          ? by_full(integral_constant<int, 1>(), integral_constant<int, 256>())
                   : threads == 256 ? by_full(integral_constant<int, 2>(), integral_constant<int, 256>())
                   : nu == 2        ? by_full(integral_constant<int, 2>(), integral_constant<int, 512>())
                                    : by_full(integral_constant<int, 4>(), integral_constant<int, 512>());
    return rc || t.n.part == nullptr ? rc : launch_norm_sum<T, MODE>(t.n, grid, s);
}

template <typename T>
int launch_norm_rows(NormArgs a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const int sms = std::max(1, device_sm_count());
    const int nvec = a.D / V;
    int np = 8;  // accesses a thread: eight (32 in flight a warp), fewer for short rows
    while (np > 2 && np * 32 > nvec) np /= 2;
    a.tpr_log2 = 5;
    while ((np << a.tpr_log2) < nvec) ++a.tpr_log2;
    const int groups = NORM_THREADS >> a.tpr_log2;
    const unsigned grid = (unsigned)std::min<int64_t>(((int64_t)a.N + groups - 1) / groups, sms);
    const bool full = nvec == np << a.tpr_log2;
    auto go = [&](auto kernel, SmemOptIn *done) {
        if (int rc = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), NORM_SMEM, done)) return rc;
        kernel<<<grid, NORM_THREADS, (size_t)a.D * 8, s>>>(a);
        return launch_status();
    };
    static SmemOptIn done[6];
    if (full)
        return np == 8   ? go(norm_rows_kernel<T, 8, true>, &done[0])
               : np == 4 ? go(norm_rows_kernel<T, 4, true>, &done[1])
                         : go(norm_rows_kernel<T, 2, true>, &done[2]);
    return np == 8   ? go(norm_rows_kernel<T, 8, false>, &done[3])
           : np == 4 ? go(norm_rows_kernel<T, 4, false>, &done[4])
                     : go(norm_rows_kernel<T, 2, false>, &done[5]);
}

// Launches MODE for element type T with accesses of V elements; NL accesses a thread, of few rows (forward) NS.
template <typename T, int V, int NL, int NS, int MODE>
int launch_norm_width(NormArgs a, void *scratch, cudaStream_t s) {
    constexpr bool GRAD = MODE != NORM_FORWARD;
    const int sms = std::max(1, device_sm_count());
    auto threads_log2 = [&](int per) {  // for a row of a.D, per elements a thread
        int l2 = 5;
        while ((per << l2) < a.D && l2 < 9) ++l2;
        return l2;
    };
    // Forward, few rows answer soonest spread over many threads.  bf16, us from a graph, so and as many rows:
    //   columns      512          1024         2048         4096         8192
    //   152 rows   2.4  2.5     2.8  3.4     3.2  4.9     3.9  6.2     5.5  7.7
    //   304        2.6  2.6     3.1  3.4     3.7  5.1     5.2  6.2     6.6  7.8
    //   456        2.7  2.6     3.7  3.4     5.0  5.1     6.3  6.3     8.2  8.4
    //   608        2.7  2.7     3.7  3.6     5.1  5.0     6.3  6.2     9.4  9.1
    //   1216       3.4  2.6     5.1  3.4     6.3  5.2     8.9  7.7    14.7 13.3
    // (Gradients gain nothing.)
    const bool small = !GRAD && ((int64_t)NS * V << threads_log2(NS * V)) >= a.D && a.N <= 4 * sms;
    if constexpr (GRAD) {
        if (a.D * 2 * (int)sizeof(T) <= TILE_MAX_BYTES && a.D <= TILE_MAX_D)
            return launch_norm_tiles<T, MODE>(a, V * (int)sizeof(T), scratch, s);
    } else if constexpr (V * sizeof(T) == 16) {
        if (!small && a.D <= std::min(NORM_THREADS * 8 * V, NORM_CTA_COLS)) return launch_norm_rows<T>(a, s);
    }
    const int per = (small ? NS : NL) * V;
    a.tpr_log2 = threads_log2(per);
    a.cta_cols = std::min(per << a.tpr_log2, NORM_CTA_COLS);
    a.cluster = 1;
    while (a.cluster * a.cta_cols < a.D) a.cluster *= 2;
    int groups = a.cluster > 1 ? 1 : NORM_THREADS >> a.tpr_log2;
    while (groups > 1 && (int64_t)a.N < (int64_t)sms * groups) groups /= 2;
    const int threads = groups << a.tpr_log2;
    const int cols = std::min(a.D, a.cta_cols);
    size_t smem = 0;
    int per_sm = NORM_THREADS / threads;
    if (GRAD) {
        const size_t row = (size_t)2 * NL * threads * V * sizeof(T), sums = (size_t)2 * cols * 4;
        a.stages = cols * 4 + 3 * row > NORM_SMEM ? 2 : 3;
        smem = std::max(sums, cols * 4 + a.stages * row);
        per_sm = std::min<int>(per_sm, (int)(NORM_SMEM / std::max<size_t>(smem, 1)));
    } else if (!small) {
        smem = (size_t)2 * cols * 4;
        per_sm = std::min<int>(per_sm, (int)(NORM_SMEM / smem));
    }
    per_sm = std::max(1, per_sm);
    const int64_t turns = ((int64_t)a.N + groups - 1) / groups;
    const int64_t most = std::max<int64_t>(1, (int64_t)sms * per_sm / a.cluster);
    const int clusters = (int)std::min<int64_t>({turns, most, GRAD ? NORM_PARTS : most});
    a.part = GRAD && clusters > 1 ? static_cast<float *>(scratch) : nullptr;
    auto go = [&](auto kernel, SmemOptIn *done) {
        if (int rc = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), NORM_SMEM, done)) return rc;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)(clusters * a.cluster));
        cfg.blockDim = dim3((unsigned)threads);
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
    static SmemOptIn done[2];
    if constexpr (!GRAD)
        if (small) return go(norm_kernel<T, V, NS, MODE, false>, &done[0]);
    const int rc = go(norm_kernel<T, V, NL, MODE, true>, &done[1]);
    return rc || a.part == nullptr ? rc : launch_norm_sum<T, MODE>(a, clusters, s);
}

// Rows in 16-byte, 4-byte or single-element accesses, as pointers and strides allow.
template <typename T, int MODE>
int launch_norm_typed(const NormArgs &a, void *scratch, cudaStream_t s) {
    constexpr bool GRAD = MODE != NORM_FORWARD;
    uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.out);
    bits |= (uintptr_t)((a.x_stride | a.dy_stride | a.out_stride | a.D) * (int64_t)sizeof(T));
    constexpr int W = 16 / sizeof(T);
    if (bits % 16 == 0) return launch_norm_width<T, W, GRAD ? 4 : 8, 2, MODE>(a, scratch, s);
    if constexpr (sizeof(T) == 2)
        if (bits % 4 == 0) return launch_norm_width<T, 2, 16, 4, MODE>(a, scratch, s);
    return launch_norm_width<T, 1, GRAD && sizeof(T) == 4 ? 16 : 32, 8, MODE>(a, scratch, s);
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

}  // namespace moe
