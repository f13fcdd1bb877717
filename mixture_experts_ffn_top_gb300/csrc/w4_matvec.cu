// w4_matvec.cu -- products of a few rows with 4-bit weights and group scales, one matrix or one per
// expert over rows in CSR order:
//   y[j][r] = sum_g s[r,g] * sum_{k in group g} (q[r,k] - z[r,g]) * x[j,k]
// and, for a handle of gate and up, y = SiLU(gate) * up.
//
// Decode reads every touched weight once (K/2 bytes a row and a scale per group), so the bytes bound it;
// the unpacking must keep up with them: at the copy rate an SM has some 45 cycles for 2048 weights.  A warp
// forms 16 weight rows x 8 activation columns with mma.sync m16n8k16: the codes become exact fp16 integers
// q - z in a little over two instructions a pair (the code's bits under the exponent of 1024, less 1024 + z),
// the products are exact and summed in fp32 by the tensor cores, and one fp32 multiply-add per group applies
// the scale to the accumulator.  (tcgen05.mma would want the unpacked weights back in shared memory: four
// times the packed stream's traffic, for columns that are not there.)
//
// The activations enter as fp16.  fp16 rows as they are; bf16 and fp32 rows times a power of two that brings
// the row's largest magnitude to 2^14 .. 2^15, taken back out of the sums: a bf16 value keeps all its bits
// down to 2^-29 of the row's largest (below that an error of 2^-40 of it), an fp32 value is the sum of two
// columns, its upper 11 bits and 2^11 times the rest, which loses at most 2^-22 of itself (or 2^-50 of the
// row's largest): of the order of the sums' own fp32 roundings, with two columns where an exact split takes three.
//
// Layout (w4_repack_kernel, once per weights): tiles of 16 rows (gate/up: 8 gate, then the same 8 up) by
// chunks of 128 columns, a record each: 1 KB of codes in the order the lanes hold them -- lane (g, t) =
// (lane / 4, lane % 4) has row g's 16 bytes at 16 * lane and row g + 8's at 512 + 16 * lane, word b of them
// holding columns 32 b + 8 t .. + 7 of the chunk, pair j of those 8 in bits 4j and 16 + 4j -- then the scales
// (16 bits) and the zero points (8 bits, if any) as [g][row g, row g + 8][groups of the chunk].
#include <algorithm>
#include <new>

#include "elem.cuh"

namespace moe {

namespace {

constexpr int W4_WARPS = 16;                   // at most; a CTA has 8 or 16
constexpr int W4_CHUNK = 128;                  // columns of a chunk
constexpr int W4_XPAD = 32;                    // staged rows lie 64 bytes past a multiple of 128: no bank conflicts
constexpr size_t W4_SMEM_SM = 227 * 1024;      // shared memory of an SM's CTAs, less 1 KB each

__host__ __device__ constexpr int w4_record(int group, bool zeros) { return 1024 + (zeros ? 48 : 32) * (W4_CHUNK / group); }

// One thread per 32-bit word of codes and one per scale.
__global__ void w4_repack_kernel(const uint8_t *__restrict__ q, const uint16_t *__restrict__ sc,
                                 const uint8_t *__restrict__ zp, const uint8_t *__restrict__ uq,
                                 const uint16_t *__restrict__ usc, const uint8_t *__restrict__ uzp, int E, int R,
                                 int K, int group, int ntiles, int nchunk, char *__restrict__ out) {
    const bool pair = uq != nullptr;
    const int nb = W4_CHUNK / group, ng = K / group, record = w4_record(group, zp != nullptr);
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
        char *dst = out + ch * record;
        if (code) {
            uint32_t w = 0;
            if (there) {
                const uint8_t *src = (up ? uq : q) + ((e * R + row) * (int64_t)K + k0) / 2;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w |= (uint32_t)(src[j] & 15) << (4 * j) | (uint32_t)(src[j] >> 4) << (16 + 4 * j);
            }
            reinterpret_cast<uint32_t *>(dst)[in] = w;
        } else {
            const int64_t at = (e * R + row) * (int64_t)ng + k0 / group;
            reinterpret_cast<uint16_t *>(dst + 1024)[in] = there ? (up ? usc : sc)[at] : (uint16_t)0;
            if (zp) reinterpret_cast<uint8_t *>(dst + 1024 + 32 * nb)[in] = there ? (up ? uzp : zp)[at] & 15 : 0;
        }
    }
}

// D = A B + C, 16 x 8 x 16, fp16 operands, fp32 accumulators; FRESH: C = 0.
template <bool FRESH>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if (FRESH)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 8 codes of a word, less the zero point, as four pairs (columns 2j, 2j + 1 of its 8): 1024 + q, or
// 1024 + 16 q in the next four bits (a sixteenth of that is 64 + q); all of it exact.  off = 1024 + z and
// off16 = -(64 + z), twice each.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t m, uint32_t o) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(m), "r"(o));
    return d;
}
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ void unpack(uint32_t w, uint32_t off, uint32_t off16, uint32_t (&p)[4]) {
    const uint32_t m0 = 0x000f000fu, m1 = 0x00f000f0u, magic = 0x64006400u, s16 = 0x2c002c00u;  // s16: 1/16
    const uint32_t h = w >> 8;
    p[0] = sub2(and_or(w, m0, magic), off);
    p[1] = fma2(and_or(w, m1, magic), s16, off16);
    p[2] = sub2(and_or(h, m0, magic), off);
    p[3] = fma2(and_or(h, m1, magic), s16, off16);
}

__device__ __forceinline__ uint32_t smem32(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const char *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

struct W4Args {
    const char *records;  // [E][ntiles][nchunk]
    int pair, E, R, K, nchunk, ntiles;
    const void *x;
    int64_t x_stride;
    int dtype;
    const int32_t *expStart;
    int n_rows, pass_rows;  // rows of an expert taken at a time
    int wk;                 // warps that share a tile's chunks; the CTA's other warps take the next tiles
    int nt_max;             // column tiles of 8 that pass_rows rows fill
    int bufs;               // buffers for the sums
    void *y;
    int64_t y_stride;
    unsigned *status;
};

// Eight values of row x from column k on (zero past K), as fp32.
template <typename T>
__device__ __forceinline__ void load8(const T *src, int k, int K, bool wide, float (&v)[8]) {
    if (wide && k + 8 <= K) {
#pragma unroll
        for (int h = 0; h < 8; h += 16 / sizeof(T)) {
            Pack<T, 16 / sizeof(T)> p;
            p.load(src + k + h);
#pragma unroll
            for (int q = 0; q < 16 / (int)sizeof(T); ++q) v[h + q] = p.get(q);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            Pack<T, 1> p;
            v[q] = 0.0f;
            if (k + q < K) {
                p.load(src + k + q);
                v[q] = p.get(0);
            }
        }
    }
}

__device__ __forceinline__ float exp2_int(int e) {  // 2^e, e in [-149, 127]
    return __uint_as_float(e >= -126 ? (uint32_t)(e + 127) << 23 : 1u << (e + 149));
}

__device__ __forceinline__ uint32_t half_pair(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Activation rows j0 .. j0 + rows - 1 into shared memory as fp16, zero past K, in one column (fp16, bf16) or
// two (fp32); back[column] is the power of two that its sums are to be multiplied by.  top: a word per row.
template <typename T>
__device__ void stage_rows(const W4Args &a, int j0, int rows, uint16_t *xs, int KP, float *back, unsigned *top) {
    const T *x = static_cast<const T *>(a.x) + (int64_t)j0 * a.x_stride;
    const bool wide = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.x_stride * (int64_t)sizeof(T) % 16 == 0;
    const int n8 = a.nchunk * (W4_CHUNK / 8);
    if (!std::is_same_v<T, __half>) {  // largest finite magnitude of each row (as bits, which order alike)
        for (int j = threadIdx.x; j < rows; j += blockDim.x) top[j] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < rows * n8; i += blockDim.x) {
            const int j = i / n8, k = (i - j * n8) * 8;
            float v[8];
            load8(x + (int64_t)j * a.x_stride, k, a.K, wide, v);
            unsigned m = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const unsigned b = __float_as_uint(v[q]) & 0x7fffffffu;
                m = max(m, b < 0x7f800000u ? b : 0u);
            }
            if (m) atomicMax(&top[j], m);
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < rows * n8; i += blockDim.x) {
        const int j = i / n8, k = (i - j * n8) * 8;
        if (std::is_same_v<T, __half>) {
            const uint16_t *src = reinterpret_cast<const uint16_t *>(x) + (int64_t)j * a.x_stride;
            uint4 v;
            if (wide && k + 8 <= a.K) {
                v = *reinterpret_cast<const uint4 *>(src + k);
            } else {
                uint32_t u[4] = {};
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (k + q < a.K) u[q >> 1] |= (uint32_t)src[k + q] << (16 * (q & 1));
                v = make_uint4(u[0], u[1], u[2], u[3]);
            }
            *reinterpret_cast<uint4 *>(xs + (size_t)j * KP + k) = v;
            if (k == 0) back[j] = 1.0f;
            continue;
        }
        // 2^-ex times the row lies below 2^15; ex >= -126 keeps that factor a normal number
        const int ex = top[j] ? max((int)(top[j] >> 23) - 127 - 14, -126) : 0;
        const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
        float v[8];
        load8(x + (int64_t)j * a.x_stride, k, a.K, wide, v);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = __fmul_rn(v[q], down);
        constexpr int PARTS = std::is_same_v<T, float> ? 2 : 1;
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
            uint32_t u[4];
#pragma unroll
            for (int q = 0; q < 8; q += 2) u[q >> 1] = half_pair(v[q], v[q + 1]);
            *reinterpret_cast<uint4 *>(xs + (size_t)(PARTS * j + part) * KP + k) = make_uint4(u[0], u[1], u[2], u[3]);
            if (part + 1 < PARTS)
#pragma unroll
                for (int q = 0; q < 8; ++q) {  // what is left, 2^11 times; an infinity or NaN stays in the first
                    const float hi = __half2float(__ushort_as_half((unsigned short)(u[q >> 1] >> (16 * (q & 1)))));
                    v[q] = fabsf(v[q]) < INFINITY ? (v[q] - hi) * 2048.0f : 0.0f;
                }
        }
        if (k == 0) {
            back[PARTS * j] = exp2_int(ex);
            if (PARTS == 2) back[PARTS * j + 1] = exp2_int(ex - 11);
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

// One record (16 rows x 128 columns of weights) against NT tiles of 8 activation columns.  Offsets into smem:
// rec, the record plus 16 * lane; scp and zpp, the lane's scales and zero points; x[n] + k0, the lane's column of
// tile n at the record's first column (columns past the last are copies of it: their sums are not used).
template <typename V>
__device__ __forceinline__ V lds(const char *smem, uint32_t at) { return *reinterpret_cast<const V *>(smem + at); }

template <int G, bool ZP, bool SBF, int NT, int NTM>
__device__ __forceinline__ void chunk_mma(const char *smem, uint32_t rec, uint32_t scp, uint32_t zpp,
                                          const uint32_t (&x)[NTM], uint32_t k0, float (&sum)[NTM][4]) {
    constexpr int NB = W4_CHUNK / G;
    const uint4 wl = lds<uint4>(smem, rec), wh = lds<uint4>(smem, rec + 512);
    const uint32_t lo[4] = {wl.x, wl.y, wl.z, wl.w}, hi[4] = {wh.x, wh.y, wh.z, wh.w};
    // this row's and row + 8's scales (16 bits) and zero points (8 bits), NB each
    uint32_t sw[NB];
    if constexpr (NB == 4) {
        const uint4 v = lds<uint4>(smem, scp);
        sw[0] = v.x, sw[1] = v.y, sw[2] = v.z, sw[3] = v.w;
    } else if constexpr (NB == 2) {
        const uint2 v = lds<uint2>(smem, scp);
        sw[0] = v.x, sw[1] = v.y;
    } else {
        sw[0] = lds<uint32_t>(smem, scp);
    }
    float sc[2 * NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        if (SBF) {
            sc[2 * i] = __uint_as_float(sw[i] << 16), sc[2 * i + 1] = __uint_as_float(sw[i] & 0xffff0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&sw[i]));
            sc[2 * i] = f.x, sc[2 * i + 1] = f.y;
        }
    }
    uint32_t zr[(NB + 1) / 2] = {};
    if constexpr (ZP) {
        if constexpr (NB == 4) {
            const uint2 v = lds<uint2>(smem, zpp);
            zr[0] = v.x, zr[1] = v.y;
        } else if constexpr (NB == 2) {
            zr[0] = lds<uint32_t>(smem, zpp);
        } else {
            zr[0] = lds<uint16_t>(smem, zpp);
        }
    }
    auto zero = [&](int i) { return ZP ? ((zr[i >> 2] >> (8 * (i & 3))) & 0xffu) * 0x00010001u : 0x00080008u; };
    float acc[NT][4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int gi = b * 32 / G;
        const uint32_t z0 = zero(gi), z1 = zero(NB + gi);
        uint32_t p[4], r[4];
        unpack(lo[b], 0x64006400u + z0, 0xd400d400u + 16 * z0, p);
        unpack(hi[b], 0x64006400u + z1, 0xd400d400u + 16 * z1, r);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 xv = lds<uint4>(smem, x[n] + k0 + b * 64);
            if (b * 32 % G == 0)
                mma16816<true>(acc[n], p[0], r[0], p[1], r[1], xv.x, xv.y);
            else
                mma16816<false>(acc[n], p[0], r[0], p[1], r[1], xv.x, xv.y);
            mma16816<false>(acc[n], p[2], r[2], p[3], r[3], xv.z, xv.w);
        }
        if ((b + 1) * 32 % G == 0) {
            const float s0 = sc[gi], s1 = sc[NB + gi];
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

// A persistent CTA of 8 or 16 warps takes a contiguous run of the work items: the tiles of each unit, a unit
// being an expert and a pass over at most pass_rows of its rows.  wk warps share a tile, each every wk-th pair of
// its chunks; their sums meet in shared memory in warp order (wk == 1: the lanes hold whole sums).  Every warp
// streams its pairs of records through a ring of S slots of its own, filled by cp.async ahead of the tiles: the
// stream does not stop at the end of a tile or a unit.  NTM: column tiles of 8 that the accumulators hold.
template <int G, bool ZP, bool SBF, int NTM, int S>
__global__ void __launch_bounds__(W4_WARPS * 32, 1) w4_kernel(const W4Args a) {
    constexpr int NB = W4_CHUNK / G, REC = w4_record(G, ZP), MORE = (REC - 1024) / 16, SLOT = 2 * REC;
    extern __shared__ __align__(16) char smem[];
    __shared__ int wsum[W4_WARPS];
    __shared__ float back[NTM * 8];
    __shared__ unsigned top[NTM * 8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int warps = blockDim.x >> 5;
    const int KP = a.nchunk * W4_CHUNK + W4_XPAD;
    const int cpr = a.dtype == MOE_DTYPE_F32 ? 2 : 1;
    const int wt = warp / a.wk, wk = warp - wt * a.wk, per = warps / a.wk;
    const uint32_t ring = warp * S * SLOT;  // offsets into smem, as below
    // the sums: `bufs` buffers, [warps][nt_max * 8 columns][20 (16 rows, padded against bank conflicts)]
    const int red_warp = a.nt_max * 8 * 20;
    float *red = reinterpret_cast<float *>(smem + warps * S * SLOT);
    uint16_t *xs = reinterpret_cast<uint16_t *>(red + a.bufs * warps * red_warp);
    int *first = reinterpret_cast<int *>(xs + (size_t)a.pass_rows * cpr * KP);  // [E + 1]: each expert's first pass

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
        for (int w = 0; w < warps; ++w) {
            if (w < warp) run += wsum[w];
            units += wsum[w];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (tid * 4 + i < a.E) first[tid * 4 + i] = run;
            run += cnt[i];
        }
        if (tid == 0) first[a.E] = units;
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
    const int64_t items = (int64_t)units * a.ntiles;
    const int64_t i0 = items * blockIdx.x / gridDim.x, i1 = items * (blockIdx.x + 1) / gridDim.x;
    if (i0 >= i1) return;
    // tiles of this CTA, and its first
    int todo = (int)min(i1 - i0, (int64_t)0x7fffffff);
    const int u0 = (int)(i0 / a.ntiles), t0 = (int)(i0 - (int64_t)u0 * a.ntiles);

    // The CTA takes `per` tiles of a unit at a time.  The fetching position runs ahead of the computing one:
    // ftile of unit fu (fleft tiles to come), the pair at fsrc, fnum more of this warp's tile, the last of them
    // a single record where `odd`.
    const int pairs = (a.nchunk + 1) / 2;
    const int per_tile = wk < pairs ? (pairs - wk + a.wk - 1) / a.wk : 0;  // this warp's pairs of a tile
    const bool odd = (a.nchunk & 1) && (pairs - 1) % a.wk == wk;
    int fu = u0, ftile = t0, fleft = per_tile > 0 ? todo : 0, fnum = 0, fe = expert_of(u0);
    const char *fsrc = a.records;
    const int64_t fstep = (int64_t)a.wk * SLOT;
    auto next_tile = [&]() {  // the next of the CTA's tiles that is this warp's
        while (fleft > 0) {
            const int n = min(per, min(a.ntiles - ftile, fleft)), tile = ftile + wt, e = fe;
            fleft -= n;
            ftile += n;
            if (ftile == a.ntiles) {
                ftile = 0;
                ++fu;
                if (a.expStart != nullptr && fleft > 0) fe = expert_of(fu);
            }
            if (wt < n) {
                fsrc = a.records + (((int64_t)e * a.ntiles + tile) * a.nchunk + 2 * wk) * REC + lane * 16;
                fnum = per_tile;
                return;
            }
        }
    };
    const uint32_t smem0 = smem32(smem);
    auto fetch = [&](uint32_t to) {
        if (fnum == 0) next_tile();
        if (fnum > 0) {
            const uint32_t dst = smem0 + to;
            cp_async16(dst, fsrc);
            cp_async16(dst + 512, fsrc + 512);
            if (lane < MORE) cp_async16(dst + 1024, fsrc + 1024);
            if (!(odd && fnum == 1)) {
                cp_async16(dst + REC, fsrc + REC);
                cp_async16(dst + REC + 512, fsrc + REC + 512);
                if (lane < MORE) cp_async16(dst + REC + 1024, fsrc + REC + 1024);
            }
            fsrc += fstep;
            --fnum;
        }
        cp_async_commit();
    };
    const uint32_t ring0 = ring + lane * 16, ring1 = ring0 + (S - 1) * SLOT;  // the first and the last slot
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(ring0 + i * SLOT);

    int cur = -1, j0 = 0, rows = 0, nt = 0, buf = 0;
    uint32_t slot = ring0, free_slot = ring1, at[NTM];  // the slot to read, and the one read before it
    // the lane's scales and zero points, from its 16 bytes of codes
    const int sc_off = 1024 + g * 4 * NB - lane * 16, zp_off = 1024 + 32 * NB + g * 2 * NB - lane * 16;
    const uint32_t x0 = (uint32_t)(reinterpret_cast<char *>(xs) - smem);
    const int sh = a.pair ? 3 : 4;  // a tile's rows: 8 or 16
    int u = u0, tile0 = t0;
    while (todo > 0) {
        if (u != cur) {
            cur = u;
            const int e = expert_of(u);
            const int lo = a.expStart ? a.expStart[e] : 0, hi = a.expStart ? a.expStart[e + 1] : a.n_rows;
            j0 = lo + (u - (a.expStart ? first[e] : 0)) * a.pass_rows;
            rows = min(a.pass_rows, hi - j0);
            const int cols = rows * cpr;
            nt = (cols + 7) >> 3;
#pragma unroll
            for (int n = 0; n < NTM; ++n)
                at[n] = x0 + (min(n * 8 + g, cols - 1) * KP + t * 8 + wk * 2 * W4_CHUNK) * 2;
            __syncthreads();
            if (a.dtype == MOE_DTYPE_F32)
                stage_rows<float>(a, j0, rows, xs, KP, back, top);
            else if (a.dtype == MOE_DTYPE_F16)
                stage_rows<__half>(a, j0, rows, xs, KP, back, top);
            else
                stage_rows<__nv_bfloat16>(a, j0, rows, xs, KP, back, top);
            __syncthreads();
        }
        const int now = min(per, min(a.ntiles - tile0, todo)), tile = tile0 + wt;
        float sum[NTM][4];
#pragma unroll
        for (int n = 0; n < NTM; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[n][i] = 0.0f;
        if (wt < now) {
            uint32_t k0 = 0;
            for (int c = 0; c < per_tile; ++c) {
                cp_async_wait<S - 2>();
                __syncwarp();
                fetch(free_slot);  // every lane has read it before this point
                const bool both = !(odd && c == per_tile - 1);
                if (NTM == 1 || nt == 1) {
                    chunk_mma<G, ZP, SBF, 1, NTM>(smem, slot, slot + sc_off, slot + zp_off, at, k0, sum);
                    if (both)
                        chunk_mma<G, ZP, SBF, 1, NTM>(smem, slot + REC, slot + REC + sc_off, slot + REC + zp_off, at,
                                                      k0 + 2 * W4_CHUNK, sum);
                } else {
#pragma unroll 1
                    for (int h = 0; h < 1 + both; ++h) {
                        const uint32_t rec = slot + h * REC, k = k0 + h * 2 * W4_CHUNK;
                        if (nt == 2)
                            chunk_mma<G, ZP, SBF, NTM < 2 ? 1 : 2, NTM>(smem, rec, rec + sc_off, rec + zp_off, at, k, sum);
                        else if (nt == 3)
                            chunk_mma<G, ZP, SBF, NTM < 3 ? 1 : 3, NTM>(smem, rec, rec + sc_off, rec + zp_off, at, k, sum);
                        else
                            chunk_mma<G, ZP, SBF, NTM, NTM>(smem, rec, rec + sc_off, rec + zp_off, at, k, sum);
                    }
                }
                k0 += a.wk * W4_CHUNK * 4;
                free_slot = slot;
                slot = slot == ring1 ? ring0 : slot + SLOT;
            }
        }
        if (a.wk == 1) {
            // the lane's sums are whole: rows g and g + 8 of the tile (gate and up) times columns 2t and 2t + 1 (of
            // an fp32 row both its parts)
            if (wt < now) {
                const int r = (tile << sh) + g;
#pragma unroll
                for (int n = 0; n < NTM; ++n) {
                    if (n >= nt) break;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int c = n * 8 + 2 * t + h, j = cpr == 2 ? c >> 1 : c;
                        if ((cpr == 2 && h) || j >= rows) continue;
                        float v0 = __fmul_rn(sum[n][h], back[c]), v1 = __fmul_rn(sum[n][2 + h], back[c]);
                        if (cpr == 2) {
                            v0 = __fmaf_rn(sum[n][1], back[c + 1], v0);
                            v1 = __fmaf_rn(sum[n][3], back[c + 1], v1);
                        }
                        const int64_t to = (int64_t)(j0 + j) * a.y_stride;
                        if (a.pair) {
                            if (r < a.R) store_y(a, to + r, __fdiv_rn(v0, 1.0f + expf(-v0)) * v1);
                        } else {
                            if (r < a.R) store_y(a, to + r, v0);
                            if (r + 8 < a.R) store_y(a, to + r + 8, v1);
                        }
                    }
                }
            }
        } else {
            float *mine = red + (buf * warps + warp) * red_warp;
            const float *all = red + (buf * warps + wt * a.wk) * red_warp;
#pragma unroll
            for (int n = 0; n < NTM; ++n)
                if (n < nt) {
                    float *dst = mine + (n * 8 + 2 * t) * 20 + g;
                    dst[0] = sum[n][0];
                    dst[20] = sum[n][1];
                    dst[8] = sum[n][2];
                    dst[28] = sum[n][3];
                }
            asm volatile("bar.sync %0, %1;" ::"r"(1 + wt), "r"(a.wk * 32) : "memory");
            if (wt < now) {
                for (int i = wk * 32 + lane; i < rows << sh; i += a.wk * 32) {
                    const int j = i >> sh, rr = i & ((1 << sh) - 1), r = (tile << sh) + rr;
                    if (r >= a.R) continue;
                    float v = 0.0f, up = 0.0f;
                    for (int part = 0; part < cpr; ++part) {
                        const float *p = all + (j * cpr + part) * 20 + rr;
                        float s0 = p[0], s1 = a.pair ? p[8] : 0.0f;
#pragma unroll
                        for (int w = 1; w < 8; ++w)
                            if (w < a.wk) {
                                s0 += p[w * red_warp];
                                if (a.pair) s1 += p[w * red_warp + 8];
                            }
                        v = __fmaf_rn(s0, back[j * cpr + part], v);
                        up = __fmaf_rn(s1, back[j * cpr + part], up);
                    }
                    if (a.pair) v = __fdiv_rn(v, 1.0f + expf(-v)) * up;
                    store_y(a, (int64_t)(j0 + j) * a.y_stride + r, v);
                }
            }
            if (a.bufs == 2)
                buf ^= 1;  // the next sums go elsewhere, those after them behind the next barrier
            else
                asm volatile("bar.sync %0, %1;" ::"r"(1 + wt), "r"(a.wk * 32) : "memory");
        }
        todo -= now;
        tile0 += now;
        if (tile0 == a.ntiles) {
            tile0 = 0;
            ++u;
        }
    }
    cp_async_wait<0>();
}

}  // namespace

int w4_repack(moe_w4_weights_s *w, const uint8_t *q, const void *scales, const uint8_t *zeros, const uint8_t *up_q,
              const void *up_scales, const uint8_t *up_zeros, cudaStream_t s) {
    const int trows = w->pair ? 8 : 16;
    w->ntiles = (w->R + trows - 1) / trows;
    w->nchunk = (w->K + W4_CHUNK - 1) / W4_CHUNK;
    const size_t bytes = (size_t)w->E * w->ntiles * w->nchunk * w4_record(w->group, zeros != nullptr);
    if (cudaMalloc(&w->records, bytes) != cudaSuccess) {
        (void)cudaGetLastError();
        w->records = nullptr;
        return MOE_ERR_CUDA;
    }
    w->bytes = bytes;
    w->zeros = zeros != nullptr;
    const unsigned blocks = (unsigned)std::max(1, device_sm_count()) * 16;
    w4_repack_kernel<<<blocks, 256, 0, s>>>(q, static_cast<const uint16_t *>(scales), zeros, up_q,
                                            static_cast<const uint16_t *>(up_scales), up_zeros, w->E, w->R, w->K,
                                            w->group, w->ntiles, w->nchunk, w->records);
    int rc = launch_status();
    if (!rc) rc = cuda_status(cudaStreamSynchronize(s));
    return rc;
}

int launch_w4_matvec(const moe_w4_weights_s *w, const void *x, int64_t x_stride, int dtype, const int32_t *expStart,
                     int n_rows, void *y, int64_t y_stride, unsigned *status, cudaStream_t s) {
    W4Args a{};
    a.records = w->records;
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
    const int cpr = dtype == MOE_DTYPE_F32 ? 2 : 1;
    const size_t row_bytes = (size_t)(a.nchunk * W4_CHUNK + W4_XPAD) * 2 * cpr;
    const size_t record = w4_record(w->group, w->zeros);
    // Warps a tile: the fewest that leave the GPU's 16 warps an SM six tiles each in turn (a tile that is shared
    // costs a barrier and a reduction, long turns a longer tail), but no more than have a pair of chunks each.
    // The weights' shape alone decides, so that a row's sums do not depend on the rows beside it.
    const int64_t tiles = (int64_t)a.ntiles * a.E;
    const int pairs = (a.nchunk + 1) / 2;
    int wk = 1;
    while (wk < 8 && wk < pairs && tiles * wk < (int64_t)sms * 16 * 6) wk *= 2;
    a.wk = wk;
    auto smem_for = [&](int rows, int warps, int depth, int bufs) {
        const size_t nt = (rows * cpr + 7) / 8;
        return (size_t)warps * depth * 2 * record + (wk > 1 ? (size_t)bufs * warps * nt * 8 * 20 * 4 : 0) +
               row_bytes * rows + (size_t)(w->E + 1) * 4;
    };
    // most rows a pass of a CTA of so many warps (16 warps an SM) with a ring of `depth`
    auto fit = [&](int warps, int depth, int bufs) {
        int rows = 32 / cpr;
        while (rows > 0 && smem_for(rows, warps, depth, bufs) > W4_SMEM_SM / (16 / warps) - 1536) --rows;
        return rows;
    };
    // Rows wanted a pass: all of a single matrix; of many experts four times the mean, their segments being
    // uneven (a longer segment takes a pass more).
    const int want = std::min({32 / cpr, n_rows, w->E == 1 ? n_rows : std::max(8 / cpr, 4 * ((n_rows + w->E - 1) / w->E))});
    // two CTAs of 8 warps an SM where their rows fit; one of 16, the rows staged once, where they are long
    struct Shape {
        int warps, depth, bufs;
    };
    Shape shape{8, 3, 2};
    int rows = std::min(want, fit(8, 3, 2));
    for (const Shape &o : {Shape{16, 3, 2}, Shape{16, 3, 1}, Shape{16, 2, 1}, Shape{8, 2, 1}}) {
        if (rows == want) break;
        const int more = std::min(want, o.warps == 8 ? (smem_for(1, 8, 2, 1) <= W4_SMEM_SM - 1536 ? 1 : 0) : fit(o.warps, o.depth, o.bufs));
        if (more > 0 && (rows == 0 || (n_rows + more - 1) / more < (n_rows + rows - 1) / rows)) shape = o, rows = more;
    }
    if (rows == 0) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (w->E == 1) rows = (n_rows + (n_rows + rows - 1) / rows - 1) / ((n_rows + rows - 1) / rows);
    a.pass_rows = rows;
    a.nt_max = (rows * cpr + 7) / 8;
    a.bufs = wk > 1 ? shape.bufs : 0;
    const int depth = shape.depth, per = shape.warps / wk;
    const int64_t most = (int64_t)((a.ntiles + per - 1) / per) *
                         (w->E == 1 ? (n_rows + rows - 1) / rows : (int64_t)n_rows);
    const unsigned grid = (unsigned)std::min<int64_t>(most, (int64_t)sms * (16 / shape.warps));
    const size_t smem = smem_for(rows, shape.warps, shape.depth, shape.bufs);
    auto go = [&](auto kernel, SmemOptIn *done) {
        int rc = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), smem, done);
        if (rc) return rc;
        kernel<<<grid, shape.warps * 32, smem, s>>>(a);
        return launch_status();
    };
    auto by_types = [&](auto gc, auto zc, auto bc) {
        constexpr int G = decltype(gc)::value;
        constexpr bool ZP = decltype(zc)::value, SBF = decltype(bc)::value;
        static SmemOptIn d[4];
        if (a.nt_max > 1)
            return depth == 3 ? go(w4_kernel<G, ZP, SBF, 4, 3>, &d[0]) : go(w4_kernel<G, ZP, SBF, 4, 2>, &d[1]);
        return depth == 3 ? go(w4_kernel<G, ZP, SBF, 1, 3>, &d[2]) : go(w4_kernel<G, ZP, SBF, 1, 2>, &d[3]);
    };
    auto by_zeros = [&](auto gc, auto bc) {
        return w->zeros ? by_types(gc, std::true_type(), bc) : by_types(gc, std::false_type(), bc);
    };
    auto by_group = [&](auto gc) {
        return w->scale_dtype == MOE_DTYPE_BF16 ? by_zeros(gc, std::true_type()) : by_zeros(gc, std::false_type());
    };
    switch (w->group) {
        case 32: return by_group(std::integral_constant<int, 32>());
        case 64: return by_group(std::integral_constant<int, 64>());
        default: return by_group(std::integral_constant<int, 128>());
    }
}

}  // namespace moe
