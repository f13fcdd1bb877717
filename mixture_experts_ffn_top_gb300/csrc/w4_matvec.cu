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
// the row's largest magnitude to 2^14 .. 2^15, taken back out of the sums.  fp16's values end in multiples of
// 2^-24: the 8 bits of a bf16 value from 2^-17 on are kept, so all down to 2^-31 of the row's largest, and a
// smaller value moves by half a multiple at most, 2^-25, which is 2^-39 of a largest of 2^14.  An fp32 value is
// the sum of two columns, its upper 11 bits and 2^11 times the rest, which loses at most 2^-22 of itself (or
// 2^-25 / 2^11, 2^-50 of the row's largest): of the order of the sums' own fp32 roundings, with two columns
// where an exact split takes three.
//
// A group's sum of such a row is a multiple of 2^-24 below 128 * 15 * 2^15 < 2^26, whatever the row's own
// magnitude, and meets the scale as it is: sums over K <= 2^15 columns stay below 2^34 times the largest scale,
// and no product rounds among fp32's smallest numbers by more than 2^-150.  So fp16 scales, and bf16 ones of
// 2^-100 up to 2^90, leave nothing else to lose.  Weights with a bf16 scale beyond those (`wide`, found when they
// are laid out) take the power of two out of each group's sum before its scale, one multiplication more: the sums
// have the magnitude of the definition's and leave fp32's range only where those do.
//
// Layout (w4_repack_kernel, once per weights): tiles of 16 rows (gate/up: 8 gate, then the same 8 up) by
// chunks of 128 columns, a record each: 1 KB of codes in the order the lanes hold them -- lane (g, t) =
// (lane / 4, lane % 4) has row g's 16 bytes at 16 * lane and row g + 8's at 512 + 16 * lane, word b of them
// holding columns 32 b + 8 t .. + 7 of the chunk, pair j of those 8 in bits 4j and 16 + 4j -- then the scales
// (16 bits) and the zero points (if any, twice in 8 bits) as [g][row g, row g + 8][groups of the chunk].
#include <algorithm>
#include <new>

#include "elem.cuh"

namespace moe {

namespace {

constexpr int W4_WARPS = 16;                   // at most; a CTA has 8 or 16
constexpr int W4_TURNS = 6;                    // tiles of all experts for each warp (see launch_w4_matvec)
constexpr int W4_CHUNK = 128;                  // columns of a chunk
constexpr int W4_XPAD = 64;                    // bytes past a multiple of 128 that staged rows lie apart: no bank conflicts
constexpr size_t W4_SMEM_SM = 227 * 1024;      // shared memory of an SM's CTAs, less 1 KB each

__host__ __device__ constexpr int w4_record(int group, bool zeros) { return 1024 + (zeros ? 48 : 32) * (W4_CHUNK / group); }

// One thread per 32-bit word of codes and one per scale.  wide (bf16 scales): set where a finite one is not 0 and
// lies outside 2^-100 .. 2^90.
__global__ void w4_repack_kernel(const uint8_t *__restrict__ q, const uint16_t *__restrict__ sc,
                                 const uint8_t *__restrict__ zp, const uint8_t *__restrict__ uq,
                                 const uint16_t *__restrict__ usc, const uint8_t *__restrict__ uzp, int E, int R,
                                 int K, int group, int ntiles, int nchunk, char *__restrict__ out,
                                 unsigned *__restrict__ wide) {
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
            const uint16_t v = there ? (up ? usc : sc)[at] : (uint16_t)0;
            const int ex = (v >> 7) & 255;  // of a bf16 scale
            if (wide != nullptr && (v & 0x7fff) != 0 && ex != 255 && (ex < 127 - 100 || ex >= 127 + 90)) *wide = 1;
            reinterpret_cast<uint16_t *>(dst + 1024)[in] = v;
            if (zp) reinterpret_cast<uint8_t *>(dst + 1024 + 32 * nb)[in] = there ? (uint8_t)(((up ? uzp : zp)[at] & 15) * 17) : (uint8_t)0;
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

// The 8 codes of a word, less the zero point, as four pairs (columns 2j, 2j + 1 of its 8), by the conversion of
// small integers that Kim, Henry, Fahim and Awadalla published ("Who Says Elephants Can't Run: Bringing Large Scale
// MoE Models into Cloud Scale Production", 2022): a code under the exponent of 1024 is the fp16 number 1024 + q, or
// 1024 + 16 q from the next four bits (a sixteenth of that is 64 + q); all of it exact.  off = 1024 + z and
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
__device__ __forceinline__ void wait_all_but(int n) {  // the n (0 .. 2) groups begun last
    if (n == 2)
        cp_async_wait<2>();
    else if (n == 1)
        cp_async_wait<1>();
    else
        cp_async_wait<0>();
}

struct W4Args {
    const char *records;  // [E][ntiles][nchunk]
    int scale_bf, pair, E, R, K, nchunk, ntiles;
    const void *x;
    int64_t x_stride;
    int dtype;
    const int32_t *expStart;
    int n_rows, pass_rows;  // rows of an expert taken at a time
    int stage_rows;         // rows that shared memory holds
    int slots;              // of a warp's ring: 2 or 3 pairs of records
    int wk, wk_log2;        // warps that share a tile's chunks; the CTA's other warps take the next tiles
    int copy_log2, turn_log2;  // threads that share a row: as it is copied, as it is turned
    uint64_t ntiles_inv, pass_inv, grid_inv;  // for div_by
    int nt_max;             // column tiles of 8 that pass_rows rows fill
    int bufs;               // buffers for the sums
    void *y;
    int64_t y_stride;
    unsigned *status;
};

// n / d by the inverse M = ceil(2^64 / d) (0 for d = 1): M d - 2^64 < d, so n M / 2^64 lies less than
// n / 2^64 <= 1 / d above n / d for n, d < 2^32, and rounds down to the same.
inline uint64_t inverse(uint32_t d) { return d == 1 ? 0 : ~(uint64_t)0 / d + 1; }
__device__ __forceinline__ unsigned div_by(unsigned n, uint64_t inv) {
    return inv != 0 ? (unsigned)__umul64hi(n, inv) : n;
}

__device__ __forceinline__ float exp2_int(int e) {  // 2^e, e in [-149, 127]
    return __uint_as_float(e >= -126 ? (uint32_t)(e + 127) << 23 : 1u << (e + 149));
}

__device__ __forceinline__ uint32_t half_pair(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Activation rows in shared memory: 8 values lie together as 16 bytes of fp16, or for fp32 rows as 16 bytes of
// the first parts and 16 of the second, so that the caller's values are copied in as they are and turned in
// place.  copy_rows starts the copies of rows j0 .. j0 + rows - 1 (zero past K); after they have arrived and a
// barrier turn_rows makes the fp16 values; back[column] is the power of two that a column's sums are to be
// multiplied by.  top: a word per row.
__device__ __forceinline__ void copy_rows(const W4Args &a, int j0, int rows, char *xs, int row_bytes) {
    const int eb = a.dtype == MOE_DTYPE_F32 ? 4 : 2, nt = blockDim.x;
    const int64_t stride = a.x_stride * eb;
    const char *x = static_cast<const char *>(a.x) + j0 * stride;
    const int end = a.nchunk * W4_CHUNK * eb, kb = a.K * eb;  // bytes of a row, and of its values
    const bool wide = (reinterpret_cast<uintptr_t>(a.x) | (uint64_t)stride) % 16 == 0;
    const int tpr = 1 << a.copy_log2, jstep = nt >> a.copy_log2;
    for (int j = threadIdx.x >> a.copy_log2; j < rows; j += jstep) {
        const char *src = x + j * stride;
        char *dst = xs + j * row_bytes;
        for (int at = (threadIdx.x & (tpr - 1)) * 16; at < end; at += tpr * 16) {
            if (at >= kb) {
                *reinterpret_cast<uint4 *>(dst + at) = make_uint4(0, 0, 0, 0);
            } else if (wide) {
                cp_async16(smem32(dst + at), src + at);
            } else {
#pragma unroll 1
                for (int q = 0; q < 16; q += eb)
                    if (eb == 4)
                        *reinterpret_cast<uint32_t *>(dst + at + q) = *reinterpret_cast<const uint32_t *>(src + at + q);
                    else
                        *reinterpret_cast<uint16_t *>(dst + at + q) = *reinterpret_cast<const uint16_t *>(src + at + q);
            }
        }
    }
}

template <typename T>  // float or bf16 (fp16 rows stay as they are)
__device__ __forceinline__ void turn_rows(const W4Args &a, int rows, char *xs, int row_bytes, float *back, unsigned *top) {
    constexpr int PARTS = std::is_same_v<T, float> ? 2 : 1, V = 16 / sizeof(T);
    const int n8 = a.nchunk * (W4_CHUNK / 8), nt = blockDim.x;
    const int tpr = 1 << a.turn_log2, jstep = nt >> a.turn_log2, r0 = threadIdx.x >> a.turn_log2, i0 = threadIdx.x & (tpr - 1);
    for (int j = threadIdx.x; j < rows; j += nt) top[j] = 0;
    __syncthreads();
    for (int j = r0; j < rows; j += jstep) {  // the largest magnitude of each row, as bits
        unsigned m = 0;
        for (int i = i0; i < n8; i += tpr) {
            const char *src = xs + j * row_bytes + i * 8 * sizeof(T);
            if constexpr (PARTS == 1) {
                const uint4 p = *reinterpret_cast<const uint4 *>(src);
                const unsigned mask = 0x7fff7fffu;
                const unsigned q = __vmaxu2(__vmaxu2(p.x & mask, p.y & mask), __vmaxu2(p.z & mask, p.w & mask));
                m = max(m, max(q << 16, q & 0xffff0000u));
            } else {
#pragma unroll
                for (int h = 0; h < 8; h += V) {
                    const uint4 p = *reinterpret_cast<const uint4 *>(src + h * 4);
                    m = max(m, max(max(p.x & 0x7fffffffu, p.y & 0x7fffffffu), max(p.z & 0x7fffffffu, p.w & 0x7fffffffu)));
                }
            }
        }
        if (tpr >= 32) m = __reduce_max_sync(0xffffffffu, m);  // the warp is in one row: one atomic instead of 32
        if (m && (tpr < 32 || (threadIdx.x & 31) == 0)) atomicMax(&top[j], m);
    }
    __syncthreads();
    for (int j = r0; j < rows; j += jstep) {
        for (int i = i0; i < n8; i += tpr) {
            char *at = xs + j * row_bytes + i * 8 * sizeof(T);
            // 2^-ex times the row lies below 2^15; ex >= -126 keeps that factor a normal number.  With an infinity or
            // NaN in it no sum of the row is finite, whatever becomes of the others.
            const unsigned m = min(top[j], 0x7f7fffffu);
            const int ex = m ? max((int)(m >> 23) - 127 - 14, -126) : 0;
            const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
            float v[8];
#pragma unroll
            for (int h = 0; h < 8; h += V) {
                Pack<T, V> p;
                p.load(reinterpret_cast<const T *>(at) + h);
#pragma unroll
                for (int q = 0; q < V; ++q) v[h + q] = __fmul_rn(p.get(q), down);
            }
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
                uint32_t u[4];
#pragma unroll
                for (int q = 0; q < 8; q += 2) u[q >> 1] = half_pair(v[q], v[q + 1]);
                *reinterpret_cast<uint4 *>(at + part * 16) = make_uint4(u[0], u[1], u[2], u[3]);
                if (part + 1 < PARTS)
#pragma unroll
                    for (int q = 0; q < 8; ++q) {  // what is left, 2^11 times; an infinity or NaN stays in the first
                        const float hi = __half2float(__ushort_as_half((unsigned short)(u[q >> 1] >> (16 * (q & 1)))));
                        v[q] = fabsf(v[q]) < INFINITY ? (v[q] - hi) * 2048.0f : 0.0f;
                    }
            }
            if (i == 0) {
                back[PARTS * j] = exp2_int(ex);
                if (PARTS == 2) back[PARTS * j + 1] = exp2_int(ex - 11);
            }
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
// tile n at the record's first column, kb bytes further for each 32 (columns past the last are copies of it: their
// sums are not used).  WIDE: f[n], what the sums of the lane's two columns of tile n are multiplied by.
template <typename V>
__device__ __forceinline__ V lds(const char *smem, uint32_t at) { return *reinterpret_cast<const V *>(smem + at); }

template <int G, bool ZP, bool F32, bool WIDE, int NT, int NTM>
__device__ __forceinline__ void chunk_mma(const char *smem, uint32_t rec, uint32_t scp, uint32_t zpp, bool sbf,
                                          const uint32_t (&x)[NTM], uint32_t k0, const float (&f)[WIDE ? NTM : 1][2],
                                          float (&sum)[NTM][4]) {
    constexpr int NB = W4_CHUNK / G, KB = F32 ? 128 : 64;
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
        if (sbf) {
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
    // 1024 + z and -(64 + z) of the i-th zero point, twice each: its low four bits under 0x64.., its high ones
    // under 0xd4..
    auto off = [&](int i) {
        return ZP ? __byte_perm(zr[i >> 2] & 0x0f0f0f0fu, 0x64, 0x4040u + 0x0101u * (i & 3)) : 0x64086408u;
    };
    auto off16 = [&](int i) {
        return ZP ? __byte_perm(zr[i >> 2] & 0xf0f0f0f0u, 0xd4, 0x4040u + 0x0101u * (i & 3)) : 0xd480d480u;
    };
    float acc[NT][4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int gi = b * 32 / G;
        uint32_t p[4], r[4];
        unpack(lo[b], off(gi), off16(gi), p);
        unpack(hi[b], off(NB + gi), off16(NB + gi), r);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 xv = lds<uint4>(smem, x[n] + k0 + b * KB);
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
                if (WIDE)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][i] = __fmul_rn(acc[n][i], f[WIDE ? n : 0][i & 1]);
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
// Measured: 131072 x 4096 fp16, groups of 128, for eight rows 53.1 us (279 MB, 5.3 TB/s: 78% of the copy rate; 277 MB
// more take 40 us more, the copy rate; 3 us pass before the weights flow); gate and up of 64 experts (1024 x 2048,
// groups of 32) for 64 rows of eight tokens 24.8 us (59%); 128 experts of 2048 x 768 with zero points for 256 fp32
// rows 30.0 us (49%); one token through 2048 x 2048 3.7 us.  Without the products the same streams take 46.5, 20.4
// and 21.4 us: 137 (with zero points 165) instructions a record and their dependences, on 16 warps an SM at 60% of
// the issue slots, are what is left to hide.  24 warps of 70 - 80 registers: 76.7, 28.2 and 31.1 us.  A bulk copy a
// pair, counted on a barrier of its slot, in the place of the cp.async: 56.0, 25.6 and 30.9 us.
template <int G, bool ZP, bool F32, int NTM, bool WIDE>
__global__ void __launch_bounds__(W4_WARPS * 32, 1) w4_kernel(const W4Args a) {
    constexpr int NB = W4_CHUNK / G, REC = w4_record(G, ZP), MORE = (REC - 1024) / 16, SLOT = 2 * REC;
    constexpr int cpr = F32 ? 2 : 1;  // columns per row
    constexpr uint32_t KB = 64 * cpr;  // bytes of 32 values of a staged row
    extern __shared__ __align__(16) char smem[];
    __shared__ int wsum[W4_WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int warps = blockDim.x >> 5;
    const int row_bytes = a.nchunk * W4_CHUNK * 2 * cpr + W4_XPAD;  // of a staged row
    const int S = a.slots;
    const int wt = warp >> a.wk_log2, wk = warp & (a.wk - 1), per = warps >> a.wk_log2;
    const uint32_t ring = warp * S * SLOT;  // offsets into smem, as below
    float4 *red = reinterpret_cast<float4 *>(smem + warps * S * SLOT);  // the sums: [bufs][warps][nt_max][lanes]
    char *xs = reinterpret_cast<char *>(red + a.bufs * warps * a.nt_max * 32);
    int *first = reinterpret_cast<int *>(xs + a.stage_rows * row_bytes);  // [E + 1]: each expert's first pass
    float *back = reinterpret_cast<float *>(first + a.E + 1);             // [stage_rows][cpr]
    unsigned *top = reinterpret_cast<unsigned *>(back + a.stage_rows * cpr);  // [stage_rows]

    int units = (int)div_by((unsigned)(a.n_rows + a.pass_rows - 1), a.pass_inv);
    if (a.expStart != nullptr) {
        // passes of each expert, exclusive scan; every offset is checked
        const int each = (int)((a.E + blockDim.x - 1) >> (31 - __clz(blockDim.x))), e0 = tid * each;  // a thread's experts
        bool bad = false;
        auto passes = [&](int e) {
            if (e >= a.E) return 0;
            const int p = a.expStart[e], q = a.expStart[e + 1];
            if (p < 0 || q < p || q > a.n_rows || (e == 0 && p != 0)) {
                bad = true;
                return 0;
            }
            return (int)div_by((unsigned)(q - p + a.pass_rows - 1), a.pass_inv);
        };
        int mine = 0;
#pragma unroll 1
        for (int i = 0; i < each; ++i) mine += passes(e0 + i);
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) wsum[warp] = inc;
        if (__syncthreads_or(bad)) {
            if (tid == 0) atomicOr(a.status, MOE_DEV_BAD_CSR);
            return;
        }
        int run = inc - mine;
        units = 0;
#pragma unroll
        for (int w = 0; w < W4_WARPS; ++w) {
            const int n = w < warps ? wsum[w] : 0;
            run += w < warp ? n : 0;
            units += n;
        }
#pragma unroll 1
        for (int i = 0; i < each && e0 + i < a.E; ++i) {
            first[e0 + i] = run;
            run += each == 1 ? mine : passes(e0 + i);
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
    // tiles of this CTA (the host keeps their number below 2^31), and its first
    const unsigned items = (unsigned)units * (unsigned)a.ntiles, share = div_by(items, a.grid_inv), more = items - share * gridDim.x;
    const unsigned i0 = blockIdx.x * share + min(blockIdx.x, more);
    int todo = (int)(share + (blockIdx.x < more));
    if (todo == 0) return;
    const int u0 = (int)div_by(i0, a.ntiles_inv), t0 = (int)(i0 - (unsigned)u0 * a.ntiles);
    const int last_unit = (int)div_by(i0 + todo - 1, a.ntiles_inv);

    // The CTA takes `per` tiles of a unit at a time.  The fetching position runs ahead of the computing one:
    // ftile of unit fu (fleft tiles to come), the pair at fsrc, fnum more of this warp's tile, the last of them
    // a single record where `odd`.
    const int pairs = (a.nchunk + 1) / 2;
    const int per_tile = wk < pairs ? (pairs - wk + a.wk - 1) >> a.wk_log2 : 0;  // this warp's pairs of a tile
    const bool odd = (a.nchunk & 1) && ((pairs - 1) & (a.wk - 1)) == wk;
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
    // rows of a unit: the first, and how many
    auto unit_rows = [&](int v, int e, int *begin) {
        const int lo = a.expStart ? a.expStart[e] : 0, hi = a.expStart ? a.expStart[e + 1] : a.n_rows;
        *begin = lo + (v - (a.expStart ? first[e] : 0)) * a.pass_rows;
        return min(hi - *begin, a.pass_rows);
    };
    // The rows of the first unit are asked for before any weights; those of each next one while a unit is at
    // work, into the part of the staging room that it leaves, so that the warps need not stop for them.
    int j0, rows = unit_rows(u0, fe, &j0), x_at = 0;
    int next_rows = 0, next_j0 = 0, next_at = -1;  // the next unit's (next_at < 0: not asked for)
    int since = 0;                                 // groups of copies begun after its rows'
    copy_rows(a, j0, rows, xs, row_bytes);
    cp_async_commit();
    const uint32_t ring0 = ring + lane * 16, ring1 = ring0 + (S - 1) * SLOT;  // the first and the last slot
    for (int i = 0; i < S - 1; ++i) fetch(ring0 + i * SLOT);
    if (!F32 && a.dtype == MOE_DTYPE_F16)
        for (int i = tid; i < a.stage_rows; i += blockDim.x) back[i] = 1.0f;

    int cur = -1, nt = 0, buf = 0;
    uint32_t slot = ring0, free_slot = ring1, at[NTM];  // the slot to read, and the one read before it
    // WIDE: a column's power of two, as far as 2^100, goes into its groups' sums (below 2^26), the rest over it into
    // the whole sums (rows with a value of 2^115 or more: their sums lie up to 2^13 below the definition's)
    float f[WIDE ? NTM : 1][2];
    auto inside = [&](int c) { return fminf(back[x_at * cpr + c], 0x1p100f); };
    auto outside = [&](int c) { return WIDE ? __fdiv_rn(back[x_at * cpr + c], inside(c)) : back[x_at * cpr + c]; };
    // the lane's scales and zero points, from its 16 bytes of codes
    const int sc_off = 1024 + g * 4 * NB - lane * 16, zp_off = 1024 + 32 * NB + g * 2 * NB - lane * 16;
    const uint32_t x0 = (uint32_t)(xs - smem);
    const int sh = a.pair ? 3 : 4;  // a tile's rows: 8 or 16
    const bool sbf = a.scale_bf;
    int u = u0, tile0 = t0;
    while (todo > 0) {
        if (u != cur) {
            if (cur < 0) {  // all but the weights asked for since
                wait_all_but(S - 1);
                __syncthreads();
            } else if (next_at >= 0) {
                if (since < 2)
                    cp_async_wait<0>();
                else
                    cp_async_wait<2>();
                __syncthreads();
                j0 = next_j0, rows = next_rows, x_at = next_at;
            } else {
                rows = unit_rows(u, expert_of(u), &j0), x_at = 0;
                __syncthreads();
                copy_rows(a, j0, rows, xs, row_bytes);
                cp_async_commit();
                cp_async_wait<0>();
                __syncthreads();
            }
            cur = u;
            if (F32) {
                turn_rows<float>(a, rows, xs + x_at * row_bytes, row_bytes, back + x_at * cpr, top + x_at);
                __syncthreads();
            } else if (a.dtype == MOE_DTYPE_BF16) {
                turn_rows<__nv_bfloat16>(a, rows, xs + x_at * row_bytes, row_bytes, back + x_at * cpr, top + x_at);
                __syncthreads();
            }
            next_at = -1;
            if (u < last_unit) {
                next_rows = unit_rows(u + 1, expert_of(u + 1), &next_j0);
                if (x_at + rows + next_rows <= a.stage_rows)
                    next_at = x_at + rows;
                else if (next_rows <= x_at)
                    next_at = 0;
                if (next_at >= 0) {
                    copy_rows(a, next_j0, next_rows, xs + next_at * row_bytes, row_bytes);
                    cp_async_commit();
                    since = 0;
                }
            }
            const int cols = rows * cpr;
            nt = (cols + 7) >> 3;
#pragma unroll
            for (int n = 0; n < NTM; ++n) {
                const int c = min(n * 8 + g, cols - 1);
                at[n] = x0 + (F32 ? (x_at + (c >> 1)) * row_bytes + (c & 1) * 16 : (x_at + c) * row_bytes) + t * 16 * cpr +
                        wk * 8 * KB;
                if (WIDE)
#pragma unroll
                    for (int h = 0; h < 2; ++h) f[WIDE ? n : 0][h] = inside(min(n * 8 + 2 * t + h, cols - 1));
            }
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
                wait_all_but(S - 2);
                __syncwarp();
                fetch(free_slot);  // every lane has read it before this point
                ++since;
                const bool both = !(odd && c == per_tile - 1);
                if (NTM == 1 || nt == 1) {
                    chunk_mma<G, ZP, F32, WIDE, 1, NTM>(smem, slot, slot + sc_off, slot + zp_off, sbf, at, k0, f, sum);
                    if (both)
                        chunk_mma<G, ZP, F32, WIDE, 1, NTM>(smem, slot + REC, slot + REC + sc_off, slot + REC + zp_off, sbf, at,
                                                      k0 + 4 * KB, f, sum);
                } else {
#pragma unroll 1
                    for (int h = 0; h < 1 + both; ++h) {
                        const uint32_t rec = slot + h * REC, kh = k0 + h * 4 * KB;
                        if (NTM == 2 || nt == 2)
                            chunk_mma<G, ZP, F32, WIDE, NTM < 2 ? 1 : 2, NTM>(smem, rec, rec + sc_off, rec + zp_off, sbf, at, kh, f, sum);
                        else if (nt == 3)
                            chunk_mma<G, ZP, F32, WIDE, NTM < 3 ? 1 : 3, NTM>(smem, rec, rec + sc_off, rec + zp_off, sbf, at, kh, f, sum);
                        else
                            chunk_mma<G, ZP, F32, WIDE, NTM, NTM>(smem, rec, rec + sc_off, rec + zp_off, sbf, at, kh, f, sum);
                    }
                }
                k0 += a.wk * 8 * KB;
                free_slot = slot;
                slot = slot == ring1 ? ring0 : slot + SLOT;
            }
        }
        if (a.wk > 1) {
            // the sharing warps' sums, lane by lane: column tile n is finished by warp n % wk, which adds the
            // others' in warp order
            float4 *all = red + (buf * warps + wt * a.wk) * a.nt_max * 32 + lane;
#pragma unroll
            for (int n = 0; n < NTM; ++n)
                if (n < nt) all[(wk * a.nt_max + n) * 32] = make_float4(sum[n][0], sum[n][1], sum[n][2], sum[n][3]);
            asm volatile("bar.sync %0, %1;" ::"r"(1 + wt), "r"(a.wk * 32) : "memory");
#pragma unroll
            for (int n = 0; n < NTM; ++n)
                if (n < nt && (n & (a.wk - 1)) == wk) {
                    float4 v = all[n * 32];
#pragma unroll
                    for (int w = 1; w < 8; ++w)
                        if (w < a.wk) {
                            const float4 o = all[(w * a.nt_max + n) * 32];
                            v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
                        }
                    sum[n][0] = v.x, sum[n][1] = v.y, sum[n][2] = v.z, sum[n][3] = v.w;
                }
            if (a.bufs == 2)
                buf ^= 1;  // the next sums go elsewhere, those after them behind the next barrier
            else
                asm volatile("bar.sync %0, %1;" ::"r"(1 + wt), "r"(a.wk * 32) : "memory");
        }
        // the lane's sums: rows g and g + 8 of the tile (gate and up) times columns 2t and 2t + 1 (of an fp32 row
        // both its parts)
        if (wt < now) {
            const int r = (tile << sh) + g;
#pragma unroll
            for (int n = 0; n < NTM; ++n) {
                if (n >= nt) break;
                if ((n & (a.wk - 1)) != wk) continue;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = n * 8 + 2 * t + h, j = cpr == 2 ? c >> 1 : c;
                    if ((cpr == 2 && h) || j >= rows) continue;
                    float v0 = __fmul_rn(sum[n][h], outside(c)), v1 = __fmul_rn(sum[n][2 + h], outside(c));
                    if (cpr == 2) {
                        v0 = __fmaf_rn(sum[n][1], outside(c + 1), v0);
                        v1 = __fmaf_rn(sum[n][3], outside(c + 1), v1);
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
        todo -= now;
        tile0 += now;
        if (tile0 == a.ntiles) {
            tile0 = 0;
            ++u;
        }
    }
    cp_async_wait<0>();
}

int log2_of(int n) {  // rounded up
    int l = 0;
    while (1 << l < n) ++l;
    return l;
}

}  // namespace

int w4_repack(moe_w4_weights_s *w, const uint8_t *q, const void *scales, const uint8_t *zeros, const uint8_t *up_q,
              const void *up_scales, const uint8_t *up_zeros, cudaStream_t s) {
    const int trows = w->pair ? 8 : 16;
    w->ntiles = (w->R + trows - 1) / trows;
    w->nchunk = (w->K + W4_CHUNK - 1) / W4_CHUNK;
    const size_t records = (size_t)w->E * w->ntiles * w->nchunk * w4_record(w->group, zeros != nullptr);
    const size_t bytes = records + 16;  // and the word that tells of far scales
    if (cudaMalloc(&w->records, bytes) != cudaSuccess) {
        (void)cudaGetLastError();
        w->records = nullptr;
        return MOE_ERR_CUDA;
    }
    w->bytes = bytes;
    w->zeros = zeros != nullptr;
    unsigned *wide = reinterpret_cast<unsigned *>(w->records + records);
    int rc = cuda_status(cudaMemsetAsync(wide, 0, sizeof(unsigned), s));
    if (rc) return rc;
    const unsigned blocks = (unsigned)std::max(1, device_sm_count()) * 16;
    w4_repack_kernel<<<blocks, 256, 0, s>>>(q, static_cast<const uint16_t *>(scales), zeros, up_q,
                                            static_cast<const uint16_t *>(up_scales), up_zeros, w->E, w->R, w->K,
                                            w->group, w->ntiles, w->nchunk, w->records,
                                            w->scale_dtype == MOE_DTYPE_BF16 ? wide : nullptr);
    unsigned found = 0;
    rc = launch_status();
    if (!rc) rc = cuda_status(cudaMemcpyAsync(&found, wide, sizeof(found), cudaMemcpyDeviceToHost, s));
    if (!rc) rc = cuda_status(cudaStreamSynchronize(s));
    w->wide = found != 0;
    return rc;
}

int launch_w4_matvec(const moe_w4_weights_s *w, const void *x, int64_t x_stride, int dtype, const int32_t *expStart,
                     int n_rows, void *y, int64_t y_stride, unsigned *status, cudaStream_t s) {
    W4Args a{};
    a.records = w->records;
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
    const int cpr = dtype == MOE_DTYPE_F32 ? 2 : 1;
    const size_t row_bytes = (size_t)a.nchunk * W4_CHUNK * 2 * cpr + W4_XPAD;
    const size_t record = w4_record(w->group, w->zeros);
    // Warps a tile: the fewest that leave each of the GPU's 16 warps an SM a tile of a single matrix (28672 x 4096 17.0
    // us with four, 19.4 with eight; a shared tile costs a barrier and a reduction), and of many experts six, as few of
    // them may have rows (128 gates and ups of 768 x 2048, eight rows: 8.3 us with two, 10.3 with one; for the 64 rows
    // of 64 experts 24.8 with two, 28 with four) -- but no more than have two pairs of chunks each unless warps would
    // have no tile at all (35 experts of 5592 x 768 15.3 us with one, 17.4 with two).
    // The weights' shape alone decides, so that a row's sums do not depend on the rows beside it.
    const int64_t tiles = (int64_t)a.ntiles * a.E;
    const int pairs = (a.nchunk + 1) / 2;
    int wk = 1;
    while (wk < 8 && wk < pairs && tiles * wk < (int64_t)sms * 16 * (a.E == 1 || pairs < 4 * wk ? 1 : W4_TURNS)) wk *= 2;
    a.wk = wk;
    a.wk_log2 = log2_of(wk);
    a.ntiles_inv = inverse(a.ntiles);
    struct Shape {
        int warps, ctas, slots, bufs;  // CTAs an SM
    };
    const size_t per_row = row_bytes + 4 * cpr + 4;
    auto smem_for = [&](int rows, const Shape &o) {  // of a CTA
        const size_t nt = (rows * cpr + 7) / 8;
        return (size_t)o.warps * o.slots * 2 * record + (wk > 1 ? (size_t)o.bufs * o.warps * nt * 512 : 0) +
               per_row * rows + (size_t)(w->E + 1) * 4;
    };
    auto fit = [&](const Shape &o) {  // most rows a pass
        int rows = 32 / cpr;
        while (rows > 0 && smem_for(rows, o) > W4_SMEM_SM / o.ctas - 1536) --rows;
        return rows;
    };
    // Rows wanted a pass: all of a single matrix; of many experts twice the mean, their segments being uneven (a
    // longer segment takes a pass more), and a column tile at least.
    const int want = std::min({32 / cpr, n_rows, w->E == 1 ? n_rows : std::max(8 / cpr, 2 * ((n_rows + w->E - 1) / w->E))});
    // Two CTAs of 8 warps an SM where their rows fit; one of 16, the rows staged once, where they are long and that
    // saves passes; one of 8 for the longest.
    Shape shape{8, 2, 3, 2};
    int rows = std::min(want, fit(shape));
    for (const Shape &o : {Shape{16, 1, 3, 2}, Shape{16, 1, 2, 1}, Shape{8, 1, 3, 1}}) {
        const int more = std::min(want, fit(o));
        if (more > 0 && (rows == 0 || (n_rows + more - 1) / more < (n_rows + rows - 1) / rows)) shape = o, rows = more;
    }
    if (rows == 0) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (w->E == 1) {
        const int one = 8 / cpr;  // a column tile
        // few tiles: a CTA for each of them and each column tile of rows, as long as all run at once (the weights
        // come from L2 again, but no CTA stages all rows)
        if (rows > one && (int64_t)a.ntiles * ((n_rows + one - 1) / one) <= (int64_t)sms * shape.ctas) rows = one;
        rows = (n_rows + (n_rows + rows - 1) / rows - 1) / ((n_rows + rows - 1) / rows);
    }
    a.pass_rows = rows;
    a.nt_max = (rows * cpr + 7) / 8;
    a.bufs = wk > 1 ? shape.bufs : 0;
    if ((int64_t)a.ntiles * (w->E == 1 ? (n_rows + rows - 1) / rows : n_rows / rows + std::min(n_rows, w->E)) >= 0x7fffffff)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    const int per = shape.warps / wk;
    const int64_t most = (int64_t)((a.ntiles + per - 1) / per) *
                         (w->E == 1 ? (n_rows + rows - 1) / rows : (int64_t)n_rows);
    const unsigned grid = (unsigned)std::min<int64_t>(most, (int64_t)sms * shape.ctas);
    // room for the rows of the next experts beside those at work
    const size_t used = smem_for(rows, shape), room = W4_SMEM_SM / shape.ctas - 1536;
    const int64_t units = w->E == 1 ? (n_rows + rows - 1) / rows : n_rows;
    a.stage_rows = (int)std::min<int64_t>({(int64_t)n_rows, units * rows, rows + (int64_t)((room - used) / per_row)});
    a.slots = shape.slots;
    a.pass_inv = inverse(rows);
    a.grid_inv = inverse(grid);
    // a power of two of threads a row, so many that each has a piece of it where the CTA has as many
    const int nt = shape.warps * 32;
    a.turn_log2 = log2_of(std::min(nt, a.nchunk * (W4_CHUNK / 8)));
    a.copy_log2 = log2_of(std::min(nt, a.nchunk * (W4_CHUNK / 8) * cpr));
    const size_t smem = used + per_row * (a.stage_rows - rows);
    auto go = [&](auto kernel, SmemOptIn *done) {
        // one limit for every call, so that calls at once from two threads set the same
        int rc = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), W4_SMEM_SM - 1024, done);
        if (rc) return rc;
        kernel<<<grid, shape.warps * 32, smem, s>>>(a);
        return launch_status();
    };
    auto by_types = [&](auto gc, auto zc, auto fc) {
        constexpr int G = decltype(gc)::value;
        constexpr bool ZP = decltype(zc)::value, F32 = decltype(fc)::value;
        static SmemOptIn d[4];
        // scales of any magnitude: one form for any number of columns (fp16 rows have no power of two to take out)
        if (w->wide && dtype != MOE_DTYPE_F16) return go(w4_kernel<G, ZP, F32, 4, true>, &d[3]);
        if (a.nt_max == 1) return go(w4_kernel<G, ZP, F32, 1, false>, &d[0]);
        return a.nt_max == 2 ? go(w4_kernel<G, ZP, F32, 2, false>, &d[1]) : go(w4_kernel<G, ZP, F32, 4, false>, &d[2]);
    };
    auto by_zeros = [&](auto gc, auto fc) {
        return w->zeros ? by_types(gc, std::true_type(), fc) : by_types(gc, std::false_type(), fc);
    };
    auto by_group = [&](auto gc) {
        return dtype == MOE_DTYPE_F32 ? by_zeros(gc, std::true_type()) : by_zeros(gc, std::false_type());
    };
    switch (w->group) {
        case 32: return by_group(std::integral_constant<int, 32>());
        case 64: return by_group(std::integral_constant<int, 64>());
        default: return by_group(std::integral_constant<int, 128>());
    }
}

}  // namespace moe
