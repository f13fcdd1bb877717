// w4_matvec.cu -- products of a few rows with 4-bit weights and group scales, one matrix or one per
// expert over rows in CSR order:
//   y[j][r] = sum_g s[r,g] * sum_{k in group g} (q[r,k] - z[r,g]) * x[j,k]
// and, for a handle of gate and up, y = SiLU(gate) * up.
//
// Decode reads every touched weight once (K/2 bytes a row and a scale per group), so the bytes bound it;
// the unpacking must keep up with them.  A warp forms 16 weight rows x 8 activation columns with
// mma.sync m16n8k16: the codes become exact fp16 (or bf16) integers q - z in three instructions per
// pair (the code's bits under the exponent of 1024 or 128, less 1024 + z), the products are exact and
// summed in fp32 by the tensor cores, and one fp32 multiply-add per group applies the scale to the
// accumulator.  (tcgen05.mma would want the unpacked weights back in shared memory: twice the traffic
// of the packed stream, for columns that are not there.)
//
// Layout (w4_repack_kernel, once per weights): tiles of 16 rows (gate/up: 8 gate, then the same 8 up)
// by chunks of 128 columns, 1 KB of codes each, in the order the lanes hold them: lane (g, t) =
// (lane / 4, lane % 4) has row g's 16 bytes at 16 * lane and row g + 8's at 512 + 16 * lane, word b of
// them holding columns 32 b + 8 t .. + 7 of the chunk, pair j of those 8 in bits 4j and 16 + 4j.
// Scales and zero points follow the same tiles: [g][row g, row g + 8][groups of the chunk].
#include <algorithm>
#include <new>

#include "elem.cuh"

namespace moe {

namespace {

constexpr int W4_WARPS = 8;
constexpr int W4_CHUNK = 128;                  // columns of a chunk
constexpr int W4_XPAD = 32;                    // staged rows lie 64 bytes past a multiple of 128: no bank conflicts
constexpr size_t W4_SMEM_SM = 227 * 1024;      // shared memory of an SM's CTAs, less 1 KB each

// One thread per 32-bit word of codes and one per scale.
__global__ void w4_repack_kernel(const uint8_t *__restrict__ q, const uint16_t *__restrict__ sc,
                                 const uint8_t *__restrict__ zp, const uint8_t *__restrict__ uq,
                                 const uint16_t *__restrict__ usc, const uint8_t *__restrict__ uzp, int E, int R,
                                 int K, int group, int ntiles, int nchunk, uint32_t *__restrict__ codes,
                                 uint16_t *__restrict__ scales, uint8_t *__restrict__ zeros) {
    const bool pair = uq != nullptr;
    const int nb = W4_CHUNK / group, ng = K / group;
    const int64_t chunks = (int64_t)E * ntiles * nchunk;
    const int64_t words = chunks * 256, total = words + chunks * 16 * nb;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const bool code = i < words;
        const int64_t u = code ? i : i - words;
        const int in = (int)(code ? u % 256 : u % (16 * nb));
        const int64_t ch = code ? u / 256 : u / (16 * nb);
        const int c = (int)(ch % nchunk);
        const int64_t et = ch / nchunk;
        const int tile = (int)(et % ntiles);
        const int64_t e = et / ntiles;
        int half, g, k0;
        if (code) {
            half = in >> 7;
            const int lane = (in >> 2) & 31;
            g = lane >> 2;
            k0 = c * W4_CHUNK + (in & 3) * 32 + (lane & 3) * 8;
        } else {
            g = in / (2 * nb);
            half = (in / nb) & 1;
            k0 = c * W4_CHUNK + (in % nb) * group;
        }
        const int row = pair ? tile * 8 + g : tile * 16 + half * 8 + g;
        const bool up = pair && half;
        const bool there = row < R && k0 < K;
        if (code) {
            uint32_t w = 0;
            if (there) {
                const uint8_t *src = (up ? uq : q) + ((e * R + row) * (int64_t)K + k0) / 2;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w |= (uint32_t)(src[j] & 15) << (4 * j) | (uint32_t)(src[j] >> 4) << (16 + 4 * j);
            }
            codes[i] = w;
        } else {
            const int64_t at = (e * R + row) * (int64_t)ng + k0 / group;
            scales[u] = there ? (up ? usc : sc)[at] : (uint16_t)0;
            if (zeros) zeros[u] = there ? (uint8_t)((up ? uzp : zp)[at] & 15) : (uint8_t)0;
        }
    }
}

__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t m, uint32_t o) { return (a & m) | o; }

// D += A B, 16 x 8 x 16, fp32 accumulators.
template <bool BF>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if (BF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 8 codes of a word, less the zero point z, as four pairs (columns 2j, 2j + 1 of its 8).
template <bool BF>
__device__ __forceinline__ void unpack(uint32_t w, uint32_t z, uint32_t (&p)[4]) {
    const uint32_t zz = z * 0x00010001u;
    if (BF) {  // 128 + q: the code in the low mantissa bits of 128; both it and the difference are exact
        const uint32_t off = 0x43004300u + zz;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t v = and_or(w >> (4 * j), 0x000f000fu, 0x43004300u);
            const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v),
                                             *reinterpret_cast<const __nv_bfloat162 *>(&off));
            p[j] = *reinterpret_cast<const uint32_t *>(&d);
        }
    } else {  // 1024 + q, or 1024 + 16 q in the next four bits (a sixteenth of that is 64 + q): exact as well
        const uint32_t off = 0x64006400u + zz, off16 = 0xd400d400u + 16 * zz, s16 = 0x2c002c00u;  // -(64 + z), 1/16
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t v = and_or(w >> (j >= 2 ? 8 : 0), (j & 1) ? 0x00f000f0u : 0x000f000fu, 0x64006400u);
            const __half2 h = *reinterpret_cast<const __half2 *>(&v);
            const __half2 d = (j & 1) ? __hfma2(h, *reinterpret_cast<const __half2 *>(&s16),
                                                *reinterpret_cast<const __half2 *>(&off16))
                                      : __hsub2(h, *reinterpret_cast<const __half2 *>(&off));
            p[j] = *reinterpret_cast<const uint32_t *>(&d);
        }
    }
}

__device__ __forceinline__ float scale_f32(uint32_t b, bool bf) {
    return bf ? __uint_as_float(b << 16) : __half2float(__ushort_as_half((unsigned short)b));
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

struct W4Args {
    const char *codes;   // [E][ntiles][nchunk][1024]
    const char *scales;  // [E][ntiles][nchunk][32 * nb] bytes
    const char *zeros;   // [E][ntiles][nchunk][16 * nb] bytes, or NULL
    int scale_bf, pair, E, R, K, nchunk, ntiles;
    const void *x;
    int64_t x_stride;
    int dtype;
    const int32_t *expStart;
    int n_rows, pass_rows;  // rows of an expert taken at a time
    int wk;                 // warps that share a tile's chunks; the CTA's other warps take the next tiles
    int nt_max;             // column tiles of 8 that pass_rows rows fill
    void *y;
    int64_t y_stride;
    unsigned *status;
};

// Activation rows j0 .. j0 + rows - 1 into shared memory, 16 bits a value, zero past K.  fp32 rows become
// three rows of bf16: the value's upper bits, then what is left of it, twice (8 + 8 + 8 bits: exact; an
// infinity or NaN stays in the first).  Eight values a thread where the rows allow 16-byte loads.
__device__ void stage_x(const W4Args &a, int j0, int rows, uint16_t *xs, int KP, bool wide) {
    const int n8 = a.nchunk * (W4_CHUNK / 8);
    for (int i = threadIdx.x; i < rows * n8; i += W4_WARPS * 32) {
        const int j = i / n8, k = (i - j * n8) * 8;
        const int64_t at = (int64_t)(j0 + j) * a.x_stride + k;
        if (a.dtype == MOE_DTYPE_F32) {
            float v[8];
            const float *src = static_cast<const float *>(a.x) + at;
            if (wide && k + 8 <= a.K) {
                *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(src);
                *reinterpret_cast<float4 *>(v + 4) = *reinterpret_cast<const float4 *>(src + 4);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = k + q < a.K ? src[q] : 0.0f;
            }
            uint32_t part[3][4] = {};
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const bool fin = fabsf(v[q]) < INFINITY;
#pragma unroll
                for (int h = 0; h < 3; ++h) {
                    const uint32_t hi = __float_as_uint(v[q]) & 0xffff0000u;
                    part[h][q >> 1] |= ((hi >> 16) | (v[q] != v[q] ? 0x40u : 0u)) << (16 * (q & 1));
                    v[q] = fin ? v[q] - __uint_as_float(hi) : 0.0f;
                }
            }
#pragma unroll
            for (int h = 0; h < 3; ++h)
                *reinterpret_cast<uint4 *>(xs + (size_t)(3 * j + h) * KP + k) =
                    make_uint4(part[h][0], part[h][1], part[h][2], part[h][3]);
        } else {
            uint4 v;
            const uint16_t *src = static_cast<const uint16_t *>(a.x) + at;
            if (wide && k + 8 <= a.K) {
                v = *reinterpret_cast<const uint4 *>(src);
            } else {
                uint32_t u[4] = {};
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (k + q < a.K) u[q >> 1] |= (uint32_t)src[q] << (16 * (q & 1));
                v = make_uint4(u[0], u[1], u[2], u[3]);
            }
            *reinterpret_cast<uint4 *>(xs + (size_t)j * KP + k) = v;
        }
    }
}

__device__ __forceinline__ void store_y(const W4Args &a, int64_t at, float v) {
    if (a.dtype == MOE_DTYPE_F32)
        static_cast<float *>(a.y)[at] = v;
    else if (a.dtype == MOE_DTYPE_F16)
        static_cast<__half *>(a.y)[at] = __float2half_rn(v);
    else
        static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(v);
}

// One chunk (16 rows x 128 columns of weights) against NT tiles of 8 activation columns.  stage: the chunk in
// shared memory (codes, scales, zero points); xs: the staged rows at the chunk's first column; col[n]: the
// lane's column of tile n (columns past the last are copies of it: their sums are not used).
template <int G, bool BF, int NT>
__device__ __forceinline__ void chunk_mma(const char *stage, bool zp, bool sbf, const uint16_t *const (&col)[4], int k0,
                                          int lane, float (&sum)[4][4]) {
    constexpr int NB = W4_CHUNK / G;
    const int g = lane >> 2;
    const uint4 wl = *reinterpret_cast<const uint4 *>(stage + lane * 16);
    const uint4 wh = *reinterpret_cast<const uint4 *>(stage + 512 + lane * 16);
    const uint32_t lo[4] = {wl.x, wl.y, wl.z, wl.w}, hi[4] = {wh.x, wh.y, wh.z, wh.w};
    // this row's and row + 8's scales (16 bits) and zero points (8 bits), NB each
    uint32_t sc[NB], zr[(NB + 1) / 2];
    const char *sp = stage + 1024 + g * 4 * NB, *z8 = stage + 1024 + 32 * NB + g * 2 * NB;
    if (NB == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(sp);
        sc[0] = v.x, sc[1 % NB] = v.y, sc[2 % NB] = v.z, sc[3 % NB] = v.w;
    } else if (NB == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(sp);
        sc[0] = v.x, sc[1 % NB] = v.y;
    } else {
        sc[0] = *reinterpret_cast<const uint32_t *>(sp);
    }
#pragma unroll
    for (int i = 0; i < (NB + 1) / 2; ++i) zr[i] = 0x08080808u;
    if (zp) {
        if (NB == 4) {
            const uint2 v = *reinterpret_cast<const uint2 *>(z8);
            zr[0] = v.x, zr[((NB + 1) / 2) - 1] = v.y;
        } else if (NB == 2) {
            zr[0] = *reinterpret_cast<const uint32_t *>(z8);
        } else {
            zr[0] = *reinterpret_cast<const uint16_t *>(z8);
        }
    }
    auto scale = [&](int i) { return scale_f32((sc[i >> 1] >> (16 * (i & 1))) & 0xffffu, sbf); };
    auto zero = [&](int i) { return (zr[i >> 2] >> (8 * (i & 3))) & 0xffu; };
    float acc[NT][4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int gi = b * 32 / G;
        if (b * 32 % G == 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
        }
        uint32_t p[4], r[4];
        unpack<BF>(lo[b], zero(gi), p);
        unpack<BF>(hi[b], zero(NB + gi), r);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 xv = *reinterpret_cast<const uint4 *>(col[n] + k0 + b * 32);
            mma16816<BF>(acc[n], p[0], r[0], p[1], r[1], xv.x, xv.y);
            mma16816<BF>(acc[n], p[2], r[2], p[3], r[3], xv.z, xv.w);
        }
        if ((b + 1) * 32 % G == 0) {
            const float s0 = scale(gi), s1 = scale(NB + gi);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                sum[n][0] = __fmaf_rn(s0, acc[n][0], sum[n][0]);
                sum[n][1] = __fmaf_rn(s0, acc[n][1], sum[n][1]);
                sum[n][2] = __fmaf_rn(s1, acc[n][2], sum[n][2]);
                sum[n][3] = __fmaf_rn(s1, acc[n][3], sum[n][3]);
            }
        }
    }
}

// A persistent CTA takes a contiguous run of the work items (expert with rows, pass over at most pass_rows of
// them, group of W4_WARPS / wk tiles).  wk warps share a tile, each every wk-th chunk of it; their sums meet in
// shared memory in warp order.  Every warp streams its chunks through a ring of S slots of its own, filled by
// cp.async ahead of the items: the stream does not stop at the end of a tile or an expert.
template <int G, bool BF, int S>
__global__ void __launch_bounds__(W4_WARPS * 32, 2) w4_kernel(const W4Args a) {
    constexpr int NB = W4_CHUNK / G;
    constexpr int STAGE = 1024 + 48 * NB;
    extern __shared__ __align__(16) char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int KP = a.nchunk * W4_CHUNK + W4_XPAD;
    const int cpr = a.dtype == MOE_DTYPE_F32 ? 3 : 1;
    const int wt = warp / a.wk, wk = warp - wt * a.wk, per = W4_WARPS / a.wk;
    char *ring = smem + warp * S * STAGE;
    // the sums: two buffers, [warps][nt_max * 8 columns][20 (16 rows, padded against bank conflicts)]
    const int red_warp = a.nt_max * 8 * 20;
    float *red = reinterpret_cast<float *>(smem + W4_WARPS * S * STAGE);
    uint16_t *xs = reinterpret_cast<uint16_t *>(red + 2 * W4_WARPS * red_warp);
    int *first = reinterpret_cast<int *>(xs + (size_t)a.pass_rows * cpr * KP);  // [E + 1]: each expert's first pass
    __shared__ int wsum[W4_WARPS];

    int units = (a.n_rows + a.pass_rows - 1) / a.pass_rows;
    if (a.expStart != nullptr) {
        // passes of each expert, exclusive scan (four experts a thread); every offset is checked
        bool bad = false;
        int cnt[4], mine = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = tid * 4 + i;
            cnt[i] = 0;
            if (e < a.E) {
                const int p = a.expStart[e], q = a.expStart[e + 1];
                if (p < 0 || q < p || q > a.n_rows || (e == 0 && p != 0))
                    bad = true;
                else
                    cnt[i] = (q - p + a.pass_rows - 1) / a.pass_rows;
            }
            mine += cnt[i];
        }
        if (__syncthreads_or(bad)) {
            if (tid == 0) atomicOr(a.status, MOE_DEV_BAD_CSR);
            return;
        }
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        int run = inc - mine;
        units = 0;
#pragma unroll
        for (int w = 0; w < W4_WARPS; ++w) {
            if (w < warp) run += wsum[w];
            units += wsum[w];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (tid * 4 + i <= a.E) first[tid * 4 + i] = run;
            run += cnt[i];
        }
        if (a.E == 4 * W4_WARPS * 32 && tid == 0) first[a.E] = units;
        __syncthreads();
    }
    auto expert_of = [&](int u) {  // the expert with first[e] <= u < first[e + 1]
        if (a.expStart == nullptr) return 0;
        int lo = 0, hi = a.E;
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (first[m] <= u)
                lo = m;
            else
                hi = m;
        }
        return lo;
    };
    const int groups = (a.ntiles + per - 1) / per;
    const int64_t items = (int64_t)units * groups;
    const int64_t i0 = items * blockIdx.x / gridDim.x, i1 = items * (blockIdx.x + 1) / gridDim.x;
    if (i0 >= i1) return;

    // the fetching position: item fi (unit fu, group fg) of expert fe, chunk fc
    int64_t fi = i0;
    int fu = (int)(i0 / groups), fg = (int)(i0 - (int64_t)fu * groups), fe = expert_of(fu), fc = wk;
    auto settle = [&]() {  // to the next item with a chunk for this warp
        while (fi < i1 && (fc >= a.nchunk || fg * per + wt >= a.ntiles)) {
            fc = wk;
            ++fi;
            if (++fg == groups) {
                fg = 0;
                ++fu;
                if (a.expStart != nullptr && fi < i1) fe = expert_of(fu);
            }
            if (wk >= a.nchunk) fi = i1;
        }
    };
    settle();
    auto fetch = [&](int slot) {
        if (fi < i1) {
            const int64_t ch = ((int64_t)fe * a.ntiles + fg * per + wt) * a.nchunk + fc;
            char *dst = ring + slot * STAGE;
            const char *src = a.codes + ch * 1024 + lane * 16;
            cp_async16(dst + lane * 16, src);
            cp_async16(dst + 512 + lane * 16, src + 512);
            if (lane < 2 * NB) cp_async16(dst + 1024 + lane * 16, a.scales + ch * (32 * NB) + lane * 16);
            if (a.zeros != nullptr && lane >= 16 && lane < 16 + NB)
                cp_async16(dst + 1024 + 32 * NB + (lane - 16) * 16, a.zeros + ch * (16 * NB) + (lane - 16) * 16);
            fc += a.wk;
            settle();
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i);

    const bool wide = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.x_stride * (cpr == 3 ? 4 : 2) % 16 == 0;
    const bool zp = a.zeros != nullptr, sbf = a.scale_bf;
    int slot = 0, cur = -1, j0 = 0, rows = 0, nt = 0, buf = 0;
    const uint16_t *col[4] = {xs, xs, xs, xs};
    int u = (int)(i0 / groups), tg = (int)(i0 - (int64_t)u * groups);
    for (int64_t item = i0; item < i1; ++item) {
        if (u != cur) {
            cur = u;
            const int e = expert_of(u);
            const int lo = a.expStart ? a.expStart[e] : 0, hi = a.expStart ? a.expStart[e + 1] : a.n_rows;
            j0 = lo + (u - (a.expStart ? first[e] : 0)) * a.pass_rows;
            rows = min(a.pass_rows, hi - j0);
            const int cols = rows * cpr;
            nt = (cols + 7) >> 3;
#pragma unroll
            for (int n = 0; n < 4; ++n) col[n] = xs + (size_t)min(n * 8 + g, cols - 1) * KP + t * 8;
            __syncthreads();
            stage_x(a, j0, rows, xs, KP, wide);
            __syncthreads();
        }
        const int tile = tg * per + wt;
        float sum[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[n][i] = 0.0f;
        if (tile < a.ntiles) {
            for (int c = wk; c < a.nchunk; c += a.wk) {
                cp_async_wait<S - 2>();
                __syncwarp();
                fetch(slot == 0 ? S - 1 : slot - 1);  // the slot that every lane has read before this point
                const char *stage = ring + slot * STAGE;
                const int k0 = c * W4_CHUNK;
                if (nt == 1)
                    chunk_mma<G, BF, 1>(stage, zp, sbf, col, k0, lane, sum);
                else if (nt == 2)
                    chunk_mma<G, BF, 2>(stage, zp, sbf, col, k0, lane, sum);
                else if (nt == 3)
                    chunk_mma<G, BF, 3>(stage, zp, sbf, col, k0, lane, sum);
                else
                    chunk_mma<G, BF, 4>(stage, zp, sbf, col, k0, lane, sum);
                slot = slot == S - 1 ? 0 : slot + 1;
            }
        }
        float *mine = red + (buf * W4_WARPS + warp) * red_warp;
#pragma unroll
        for (int n = 0; n < 4; ++n)
            if (n < nt) {
                float *dst = mine + (n * 8 + 2 * t) * 20 + g;
                dst[0] = sum[n][0];
                dst[20] = sum[n][1];
                dst[8] = sum[n][2];
                dst[28] = sum[n][3];
            }
        if (a.wk == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + wt), "r"(a.wk * 32) : "memory");
        if (tile < a.ntiles) {
            const float *all = red + (buf * W4_WARPS + wt * a.wk) * red_warp;
            const int trows = a.pair ? 8 : 16;
            for (int i = wk * 32 + lane; i < trows * rows; i += a.wk * 32) {
                const int j = i / trows, rr = i - j * trows, r = tile * trows + rr;
                if (r >= a.R) continue;
                float v = 0.0f, up = 0.0f;
                for (int part = 0; part < cpr; ++part)
                    for (int w = 0; w < a.wk; ++w) {
                        const float *p = all + w * red_warp + (j * cpr + part) * 20 + rr;
                        v += p[0];
                        if (a.pair) up += p[8];
                    }
                if (a.pair) v = __fdiv_rn(v, 1.0f + expf(-v)) * up;
                store_y(a, (int64_t)(j0 + j) * a.y_stride + r, v);
            }
        }
        buf ^= 1;
        if (++tg == groups) {
            tg = 0;
            ++u;
        }
    }
    cp_async_wait<0>();
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

int w4_repack(moe_w4_weights_s *w, const uint8_t *q, const void *scales, const uint8_t *zeros, const uint8_t *up_q,
              const void *up_scales, const uint8_t *up_zeros, cudaStream_t s) {
    const int trows = w->pair ? 8 : 16;
    w->ntiles = (w->R + trows - 1) / trows;
    w->nchunk = (w->K + W4_CHUNK - 1) / W4_CHUNK;
    const size_t chunks = (size_t)w->E * w->ntiles * w->nchunk;
    const size_t per = (size_t)16 * (W4_CHUNK / w->group);
    const size_t code_bytes = align256(chunks * 1024), scale_bytes = align256(chunks * per * 2);
    const size_t zero_bytes = zeros ? align256(chunks * per) : 0;
    char *arena = nullptr;
    if (cudaMalloc(&arena, code_bytes + scale_bytes + zero_bytes) != cudaSuccess) {
        (void)cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    w->bytes = code_bytes + scale_bytes + zero_bytes;
    w->codes = arena;
    w->scales = arena + code_bytes;
    w->zeros = zeros ? arena + code_bytes + scale_bytes : nullptr;
    const unsigned blocks = (unsigned)std::max(1, device_sm_count()) * 16;
    w4_repack_kernel<<<blocks, 256, 0, s>>>(q, static_cast<const uint16_t *>(scales), zeros, up_q,
                                            static_cast<const uint16_t *>(up_scales), up_zeros, w->E, w->R, w->K,
                                            w->group, w->ntiles, w->nchunk, reinterpret_cast<uint32_t *>(w->codes),
                                            reinterpret_cast<uint16_t *>(w->scales),
                                            reinterpret_cast<uint8_t *>(w->zeros));
    int rc = launch_status();
    if (!rc) rc = cuda_status(cudaStreamSynchronize(s));
    return rc;
}

int launch_w4_matvec(const moe_w4_weights_s *w, const void *x, int64_t x_stride, int dtype, const int32_t *expStart,
                     int n_rows, void *y, int64_t y_stride, unsigned *status, cudaStream_t s) {
    W4Args a{};
    a.codes = w->codes;
    a.scales = w->scales;
    a.zeros = w->zeros;
    a.scale_bf = w->scale_dtype == MOE_DTYPE_BF16;
    a.pair = w->pair;
    a.E = w->E;
    a.R = w->R;
    a.K = w->K;
    a.nchunk = w->nchunk;
    a.ntiles = w->ntiles;
    a.x = x;
    a.x_stride = x_stride;
    a.dtype = dtype;
    a.expStart = expStart;
    a.n_rows = n_rows;
    a.y = y;
    a.y_stride = y_stride;
    a.status = status;
    const int sms = std::max(1, device_sm_count());
    const int cpr = dtype == MOE_DTYPE_F32 ? 3 : 1;
    const size_t row_bytes = (size_t)(a.nchunk * W4_CHUNK + W4_XPAD) * 2 * cpr;
    const size_t stage = 1024 + 48 * (W4_CHUNK / w->group);
    auto smem_for = [&](int rows, int depth) {
        const size_t nt = (rows * cpr + 7) / 8;
        return W4_WARPS * depth * stage + 2 * W4_WARPS * nt * 8 * 20 * 4 + row_bytes * rows + (size_t)(w->E + 1) * 4;
    };
    // most rows a pass with `ctas` CTAs of an SM and a ring of `depth`
    auto fit = [&](int ctas, int depth) {
        int rows = 32 / cpr;
        while (rows > 0 && smem_for(rows, depth) > W4_SMEM_SM / ctas - 1024) --rows;
        return rows;
    };
    // Rows wanted a pass: all of a single matrix; of many experts four times the mean, their segments being
    // uneven (a longer segment takes a pass more).
    const int want = std::min({32 / cpr, n_rows, w->E == 1 ? n_rows : std::max(8 / cpr, 4 * ((n_rows + w->E - 1) / w->E))});
    int ctas = 2, depth = 4, rows = std::min(want, fit(2, 4));
    if (rows < want) {  // one CTA an SM where that saves passes
        const int one = std::min(want, fit(1, 8));
        if (rows == 0 || (n_rows + one - 1) / one < (n_rows + rows - 1) / rows) ctas = 1, depth = 8, rows = one;
    }
    if (rows == 0) depth = 2, rows = std::min(want, fit(1, 2));
    if (rows == 0) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (w->E == 1) rows = (n_rows + (n_rows + rows - 1) / rows - 1) / ((n_rows + rows - 1) / rows);
    a.pass_rows = rows;
    a.nt_max = (rows * cpr + 7) / 8;
    // Warps a tile: at least two chunks each, or one where the weights have too few tiles for the GPU's warps.
    // The weights' shape alone decides, so that a row's sums do not depend on the rows beside it.
    const int64_t tiles = (int64_t)a.ntiles * a.E;
    int wk = 1;
    while (wk < W4_WARPS && (a.nchunk >= 4 * wk || (a.nchunk >= 2 * wk && tiles * wk < (int64_t)sms * 2 * W4_WARPS))) wk *= 2;
    a.wk = wk;
    const int per = W4_WARPS / wk;
    const int64_t most = (int64_t)((a.ntiles + per - 1) / per) *
                         (w->E == 1 ? (n_rows + rows - 1) / rows : (int64_t)n_rows);
    const unsigned grid = (unsigned)std::min<int64_t>(most, (int64_t)sms * ctas);
    const size_t smem = smem_for(rows, depth);
    const bool bf = dtype != MOE_DTYPE_F16;
    auto go = [&](auto kernel, SmemOptIn *done) {
        int rc = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), smem, done);
        if (rc) return rc;
        kernel<<<grid, W4_WARPS * 32, smem, s>>>(a);
        return launch_status();
    };
    auto by_g = [&](auto gc) {
        constexpr int G = decltype(gc)::value;
        static SmemOptIn d[6];
        if (depth == 2) return bf ? go(w4_kernel<G, true, 2>, &d[0]) : go(w4_kernel<G, false, 2>, &d[1]);
        if (depth == 4) return bf ? go(w4_kernel<G, true, 4>, &d[2]) : go(w4_kernel<G, false, 4>, &d[3]);
        return bf ? go(w4_kernel<G, true, 8>, &d[4]) : go(w4_kernel<G, false, 8>, &d[5]);
    };
    switch (w->group) {
        case 32: return by_g(std::integral_constant<int, 32>());
        case 64: return by_g(std::integral_constant<int, 64>());
        default: return by_g(std::integral_constant<int, 128>());
    }
}

}  // namespace moe
