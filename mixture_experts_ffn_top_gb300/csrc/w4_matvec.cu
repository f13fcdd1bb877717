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
constexpr size_t W4_SMEM_X = 200 * 1024;       // shared memory for the staged activation rows

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
__device__ __forceinline__ void unpack(uint32_t w, int z, uint32_t (&p)[4]) {
    if (BF) {  // 128 + q: the code in the low mantissa bits of 128; both it and the difference are exact
        const __nv_bfloat162 off = __float2bfloat162_rn((float)(128 + z));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t v = and_or(w >> (4 * j), 0x000f000fu, 0x43004300u);
            const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), off);
            p[j] = *reinterpret_cast<const uint32_t *>(&d);
        }
    } else {  // 1024 + q, or 1024 + 16 q in the next four bits (a sixteenth of that is 64 + q): exact as well
        const __half2 off = __float2half2_rn((float)(1024 + z)), off16 = __float2half2_rn((float)(-64 - z));
        const __half2 s16 = __float2half2_rn(0.0625f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t v = and_or(w >> (j >= 2 ? 8 : 0), (j & 1) ? 0x00f000f0u : 0x000f000fu, 0x64006400u);
            const __half2 h = *reinterpret_cast<const __half2 *>(&v);
            const __half2 d = (j & 1) ? __hfma2(h, s16, off16) : __hsub2(h, off);
            p[j] = *reinterpret_cast<const uint32_t *>(&d);
        }
    }
}

__device__ __forceinline__ float scale_f32(uint16_t b, bool bf) {
    return bf ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
}

struct W4Args {
    const uint4 *codes;      // [E][ntiles][nchunk][64]
    const uint16_t *scales;  // [E][ntiles][nchunk][16 * nb]
    const uint8_t *zeros;    // as scales, or NULL
    int scale_bf, pair, E, R, K, nchunk, ntiles;
    const void *x;
    int64_t x_stride;
    int dtype;
    const int32_t *expStart;
    int n_rows, pass_rows;  // rows of an expert taken at a time
    void *y;
    int64_t y_stride;
    unsigned *status;
};

// Activation rows j0 .. j0 + rows - 1 into shared memory, 16 bits a value, zero past K.  fp32 rows become
// three rows of bf16: the value's upper bits, then what is left of it, twice (8 + 8 + 8 bits: exact).
__device__ __forceinline__ void stage_x(const W4Args &a, int j0, int rows, uint16_t *xs, int KP) {
    const int Kc = a.nchunk * W4_CHUNK;
    for (int i = threadIdx.x; i < rows * Kc; i += blockDim.x) {
        const int j = i / Kc, k = i - j * Kc;
        if (a.dtype == MOE_DTYPE_F32) {
            float v = k < a.K ? static_cast<const float *>(a.x)[(int64_t)(j0 + j) * a.x_stride + k] : 0.0f;
            uint16_t *dst = xs + (size_t)3 * j * KP + k;
            const bool fin = fabsf(v) < INFINITY;
#pragma unroll
            for (int part = 0; part < 3; ++part) {
                const uint32_t hi = __float_as_uint(v) & 0xffff0000u;
                dst[(size_t)part * KP] = (uint16_t)(hi >> 16) | (v != v ? 0x40 : 0);
                v = fin ? v - __uint_as_float(hi) : 0.0f;
            }
        } else {
            xs[(size_t)j * KP + k] =
                k < a.K ? static_cast<const uint16_t *>(a.x)[(int64_t)(j0 + j) * a.x_stride + k] : (uint16_t)0;
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

// A CTA per (tile of 16 weight rows, expert): its warps take the chunks of K in turn, their sums meet in
// shared memory in warp order.  NT: column tiles of 8.
template <int G, int NT, bool BF>
__global__ void __launch_bounds__(W4_WARPS * 32) w4_kernel(const W4Args a) {
    constexpr int NB = W4_CHUNK / G;
    extern __shared__ __align__(16) unsigned char smem[];
    float *red = reinterpret_cast<float *>(smem);  // [warps][16][NT * 8]
    uint16_t *xs = reinterpret_cast<uint16_t *>(smem + W4_WARPS * 16 * NT * 8 * 4);
    const int KP = a.nchunk * W4_CHUNK + W4_XPAD;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int tile = blockIdx.x, e = blockIdx.y;
    int lo = 0, hi = a.n_rows;
    if (a.expStart != nullptr) {
        bool bad = false;
        for (int i = threadIdx.x; i < a.E; i += W4_WARPS * 32) {
            const int p = a.expStart[i], q = a.expStart[i + 1];
            bad |= p < 0 || q < p || q > a.n_rows || (i == 0 && p != 0);
        }
        if (__syncthreads_or(bad)) {
            if (threadIdx.x == 0) atomicOr(a.status, MOE_DEV_BAD_CSR);
            return;
        }
        lo = a.expStart[e];
        hi = a.expStart[e + 1];
    }
    const int cpr = a.dtype == MOE_DTYPE_F32 ? 3 : 1;
    const int64_t ch0 = ((int64_t)e * a.ntiles + tile) * a.nchunk;
    for (int j0 = lo; j0 < hi; j0 += a.pass_rows) {
        const int rows = min(a.pass_rows, hi - j0), cols = rows * cpr;
        __syncthreads();
        stage_x(a, j0, rows, xs, KP);
        __syncthreads();
        float sum[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[n][i] = 0.0f;
        for (int c = warp; c < a.nchunk; c += W4_WARPS) {
            const uint4 *src = a.codes + (ch0 + c) * 64 + lane;
            const uint4 wl = __ldcs(src), wh = __ldcs(src + 32);
            const uint32_t lo_w[4] = {wl.x, wl.y, wl.z, wl.w}, hi_w[4] = {wh.x, wh.y, wh.z, wh.w};
            const int64_t sb = (ch0 + c) * (16 * NB) + g * 2 * NB;
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
                const int z0 = a.zeros ? a.zeros[sb + gi] : 8, z1 = a.zeros ? a.zeros[sb + NB + gi] : 8;
                uint32_t p[4], r[4];
                unpack<BF>(lo_w[b], z0, p);
                unpack<BF>(hi_w[b], z1, r);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int col = n * 8 + g;
                    uint4 xv = make_uint4(0, 0, 0, 0);
                    if (col < cols)
                        xv = *reinterpret_cast<const uint4 *>(xs + (size_t)col * KP + c * W4_CHUNK + b * 32 + t * 8);
                    mma16816<BF>(acc[n], p[0], r[0], p[1], r[1], xv.x, xv.y);
                    mma16816<BF>(acc[n], p[2], r[2], p[3], r[3], xv.z, xv.w);
                }
                if ((b + 1) * 32 % G == 0) {
                    const float s0 = scale_f32(a.scales[sb + gi], a.scale_bf);
                    const float s1 = scale_f32(a.scales[sb + NB + gi], a.scale_bf);
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
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float *dst = red + (warp * 16 + g) * NT * 8 + n * 8 + 2 * t;
            dst[0] = sum[n][0];
            dst[1] = sum[n][1];
            dst[8 * NT * 8] = sum[n][2];
            dst[8 * NT * 8 + 1] = sum[n][3];
        }
        __syncthreads();
        const int trows = a.pair ? 8 : 16;
        for (int i = threadIdx.x; i < trows * rows; i += W4_WARPS * 32) {
            const int j = i / trows, rr = i % trows, r = tile * trows + rr;
            if (r >= a.R) continue;
            float v[2] = {0.0f, 0.0f};
            for (int h = 0; h <= a.pair; ++h)
                for (int part = 0; part < cpr; ++part)
                    for (int w = 0; w < W4_WARPS; ++w)
                        v[h] += red[(w * 16 + rr + 8 * h) * NT * 8 + j * cpr + part];
            if (a.pair) v[0] = __fdiv_rn(v[0], 1.0f + expf(-v[0])) * v[1];
            store_y(a, (int64_t)(j0 + j) * a.y_stride + r, v[0]);
        }
    }
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
    a.codes = reinterpret_cast<const uint4 *>(w->codes);
    a.scales = reinterpret_cast<const uint16_t *>(w->scales);
    a.zeros = reinterpret_cast<const uint8_t *>(w->zeros);
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
    const int cpr = dtype == MOE_DTYPE_F32 ? 3 : 1;
    const size_t row_bytes = (size_t)(a.nchunk * W4_CHUNK + W4_XPAD) * 2 * cpr;
    // rows a pass: 32 columns of accumulators, what shared memory holds (one row always fits: K <= 32768)
    a.pass_rows = std::min({32 / cpr, (int)(W4_SMEM_X / row_bytes), n_rows});
    const int nt = (a.pass_rows * cpr + 7) / 8;
    const bool bf = dtype != MOE_DTYPE_F16;
    auto go = [&](auto kernel, int NT, SmemOptIn *done) {
        const size_t smem = (size_t)W4_WARPS * 16 * NT * 8 * 4 + row_bytes * a.pass_rows;
        int rc = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), smem, done);
        if (rc) return rc;
        kernel<<<dim3(a.ntiles, a.E), W4_WARPS * 32, smem, s>>>(a);
        return launch_status();
    };
    auto by_g = [&](auto gc) {
        constexpr int G = decltype(gc)::value;
        static SmemOptIn d[6];
        if (nt <= 1) return bf ? go(w4_kernel<G, 1, true>, 1, &d[0]) : go(w4_kernel<G, 1, false>, 1, &d[1]);
        if (nt <= 2) return bf ? go(w4_kernel<G, 2, true>, 2, &d[2]) : go(w4_kernel<G, 2, false>, 2, &d[3]);
        return bf ? go(w4_kernel<G, 4, true>, 4, &d[4]) : go(w4_kernel<G, 4, false>, 4, &d[5]);
    };
    switch (w->group) {
        case 32: return by_g(std::integral_constant<int, 32>());
        case 64: return by_g(std::integral_constant<int, 64>());
        default: return by_g(std::integral_constant<int, 128>());
    }
}

}  // namespace moe
