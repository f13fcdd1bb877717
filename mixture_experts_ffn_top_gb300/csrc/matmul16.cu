// matmul16.cu -- products of 16-bit rows with 16-bit matrices, one matrix or one per expert over rows in CSR order,
// with bias, activation (or gate and up) and residual in the epilogue:
//   y[j] = act(W[e] x[j] + b[e]) (* (U[e] x[j] + c[e])) (+ residual[j])
//
// Two kernels.  Up to 32 rows (serving): every weight is read for a few rows, so its bytes bound the product;
// few16_kernel streams them as stream16.cuh says.  More rows (prompts, training): rows16_kernel forms tiles of 128
// rows x 256 weight rows (gate and up: 128 of each, side by side) on the tensor cores.
//
// rows16_kernel is persistent, a CTA an SM, its warps in roles: a producer that brings both operands in by TMA
// (128-byte swizzle, 64 columns a stage, four stages), an issuer of tcgen05.mma (M 128, N 256, K 16; accumulators in
// tensor memory, two tiles of 256 columns so that the next tile's products run under this one's epilogue), and eight
// epilogue warps (a lane holds a row's 32 columns; bias from shared memory; the 16-bit results cross shared memory so
// that rows leave in whole sectors).  Segments start at any row: a tile reads past its segment's end and stores
// nothing of what it finds there.
#include <algorithm>

#include "act.cuh"
#include "stream16.cuh"

namespace moe {

namespace {

// ------------------------------------------------------------ few rows ---
namespace few {

using namespace s16;

struct Args {
    Matmul16Call c;
    unsigned *status;
    int kc, pitch, stages, x_pitch;
    int tile;       // weight rows (gate and up: pairs) of a unit
    int tiles;      // units a matrix
    int x_at, red_at;
};

template <typename T, int NTM>
__global__ void __launch_bounds__(THREADS, 1) few16_kernel(const Args a) {
    extern __shared__ __align__(1024) char smem[];
    __shared__ __align__(8) unsigned long long bars[GROUPS * 2 * MAX_STAGES + 1];
    __shared__ int abort_flag, listed_s, expert_s[MAX_ROWS], first_s[MAX_ROWS + 1];
    const Matmul16Call &c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool pair = c.w_up != nullptr;
    const T *x = static_cast<const T *>(c.x);
    const uint32_t bar = tc::smem_u32(bars), xbar = bar + GROUPS * 2 * MAX_STAGES * 8;
    if (tid == 0) {
        abort_flag = 0;
        tc::mbar_init(xbar, 1);
        init_rings(bar, a.stages);
    }
    // the experts that have rows
    if (warp == 0) {
        if (c.expStart == nullptr) {
            if (lane == 0) listed_s = 1, expert_s[0] = 0, first_s[0] = 0, first_s[1] = c.n_rows;
        } else {
            int n = 0;
            bool bad = false;
            for (int e0 = 0; e0 < c.E; e0 += 32) {
                const int e = e0 + lane;
                int s = 0, s1 = 0;
                if (e < c.E) {
                    s = c.expStart[e];
                    s1 = c.expStart[e + 1];
                    bad |= s < 0 || s1 < s || s1 > c.n_rows || (e == 0 && s != 0);
                }
                bad = __any_sync(0xffffffffu, bad);
                if (bad) break;
                const unsigned there = __ballot_sync(0xffffffffu, s1 > s);
                if (s1 > s) {
                    const int p = n + __popc(there & ((1u << lane) - 1));
                    expert_s[p] = e;  // at most as many as rows
                    first_s[p] = s;
                    first_s[p + 1] = s1;  // or the next one's, the same
                }
                n += __popc(there);
                __syncwarp();
            }
            if (lane == 0) {
                listed_s = bad ? 0 : n;
                if (bad && blockIdx.x == 0) atomicOr(a.status, MOE_DEV_BAD_CSR);
            }
        }
    }
    __syncthreads();
    const int64_t units = (int64_t)listed_s * a.tiles;
    const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
    if (u0 == u1) return;
    const int group = warp < CONSUMERS ? warp / GROUP_WARPS : warp - CONSUMERS;
    Ring ring(smem, bar, group, a.stages, a.pitch, &abort_flag, a.status);
    const int rows_x = first_s[listed_s];

    if (warp >= CONSUMERS) {
        int issued = 0;
        bool ok = true;
        if (a.x_pitch && group == 0) {
            if (lane == 0) tc::mbar_expect_tx(xbar, (uint32_t)(rows_x * c.K * 2));
            __syncwarp();
            if (lane < rows_x) tc::bulk_load(tc::smem_u32(smem + a.x_at) + lane * a.x_pitch, x + lane * c.x_stride, c.K * 2, xbar);
        }
        for (int64_t u = u0 + group; u < u1 && ok; u += GROUPS) {
            const int i = (int)(u / a.tiles), r = (int)(u - (int64_t)i * a.tiles) * a.tile, n = min(a.tile, c.R - r);
            const int l = pair ? lane & 7 : lane;
            const T *m = static_cast<const T *>(pair && (lane & 8) ? c.w_up : c.w);
            const T *src = m + ((int64_t)expert_s[i] * c.R + r + min(l, n - 1)) * c.K;
            for (int k0 = 0; k0 < c.K && ok; k0 += a.kc) {
                ok = ring.produce(lane, lane < 16 && l < n, pair ? 2 * n : n, src + k0, (uint32_t)min(a.kc, c.K - k0) * 2);
                issued += ok;
            }
        }
        if (lane == 0 && *reinterpret_cast<volatile int *>(&abort_flag)) {
            drain(ring.bar, a.stages, issued);
            if (a.x_pitch && group == 0) drain(xbar, 1, 1);
        }
        return;
    }

    if (a.x_pitch) tc::mbar_wait(xbar, 0, &abort_flag, a.status, WAIT_NS);
    const T *xb = a.x_pitch ? reinterpret_cast<const T *>(smem + a.x_at) : x;
    const int64_t xs = a.x_pitch ? a.x_pitch / 2 : c.x_stride;
    auto info = [&](int64_t u) {
        const int i = (int)(u / a.tiles);
        return make_int2(first_s[i], first_s[i + 1] - first_s[i]);
    };
    auto at = [&](int row) { return xb + row * xs; };
    auto done = [&](int64_t u, const int2 &in, const float4 *s, int nt, int thread) {
        if (*reinterpret_cast<volatile int *>(&abort_flag)) return;
        const int i = (int)(u / a.tiles), r = (int)(u - (int64_t)i * a.tiles) * a.tile, here = min(a.tile, c.R - r);
        const int64_t e = expert_s[i];
        const int rl = pair ? 3 : 4;  // a unit's rows: 8 or 16
        for (int j = thread; j < nt << (rl + 3); j += GROUP_WARPS * 32) {
            const int row = j & ((1 << rl) - 1), col = (j >> rl) & 7, tile = j >> (rl + 3), l = (row & 7) * 4 + (col >> 1);
            if (row >= here || tile * 8 + col >= in.y) continue;
            float v[1] = {sum_of(s, nt, tile, l, (row >> 3) * 2 + (col & 1))};
            if (c.bias != nullptr) v[0] += c.bias[e * c.R + r + row];
            activate(v, c.act);
            if (pair) {
                float up = sum_of(s, nt, tile, l, 2 + (col & 1));
                if (c.bias_up != nullptr) up += c.bias_up[e * c.R + r + row];
                v[0] *= up;
            }
            const int64_t to = in.x + tile * 8 + col;
            if (c.residual != nullptr) {
                Pack<T, 1> p;
                p.load(static_cast<const T *>(c.residual) + to * c.residual_stride + r + row);
                v[0] += p.get(0);
            }
            static_cast<T *>(c.y)[to * c.y_stride + r + row] = elem_of<T>(v[0]);
        }
    };
    stream_units<T, NTM>(ring, u0, u1, c.K, a.kc, reinterpret_cast<float4 *>(smem + a.red_at), warp, lane, info, at, done);
}

int launch(const Matmul16Call &c, unsigned *status, cudaStream_t s) {
    Args a{};
    a.c = c;
    a.status = status;
    const int sms = std::max(1, device_sm_count());
    const int ntm = c.n_rows <= 8 ? 1 : c.n_rows <= 16 ? 2 : 4;
    const bool pair = c.w_up != nullptr;
    // Units of 16 weight rows (8 pairs), fewer where that leaves SMs without one.
    const int64_t most_rows = (int64_t)std::min(c.E, c.n_rows) * c.R;
    a.tile = (int)std::min<int64_t>(pair ? 8 : 16, (most_rows + sms - 1) / sms);
    a.tiles = (c.R + a.tile - 1) / a.tile;
    a.kc = std::min(KC, (c.K + 31) / 32 * 32);
    a.pitch = pitch_of(a.kc);
    const size_t ring = (size_t)GROUPS * 16 * a.pitch, red = (size_t)CONSUMERS * ntm * 512, most = SMEM_LIMIT - 4096;
    a.stages = (int)std::min<size_t>(MAX_STAGES, (most - red) / ring);
    // the rows are staged where that costs a stage of each ring at most
    const size_t xb = (size_t)c.n_rows * pitch_of(c.K);
    const bool staged = a.stages > 2 && (a.stages - 1) * ring + red + xb <= most;
    if (staged && a.stages * ring + red + xb > most) --a.stages;
    a.x_pitch = staged ? pitch_of(c.K) : 0;
    a.x_at = (int)(a.stages * ring);
    a.red_at = a.x_at + (int)(staged ? xb : 0);
    const size_t smem = a.red_at + red;
    const int64_t units = (int64_t)std::min(c.E, c.n_rows) * a.tiles;
    const unsigned grid = (unsigned)std::min<int64_t>(units, sms);
    auto go = [&](auto kernel, SmemOptIn *done) {
        if (int rc = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), most, done)) return rc;
        kernel<<<grid, THREADS, smem, s>>>(a);
        return launch_status();
    };
    auto by_tiles = [&](auto *tp) {
        using T = std::remove_pointer_t<decltype(tp)>;
        static SmemOptIn done[3];
        if (ntm == 1) return go(few16_kernel<T, 1>, &done[0]);
        return ntm == 2 ? go(few16_kernel<T, 2>, &done[1]) : go(few16_kernel<T, 4>, &done[2]);
    };
    return c.dtype == MOE_DTYPE_F16 ? by_tiles(static_cast<__half *>(nullptr)) : by_tiles(static_cast<__nv_bfloat16 *>(nullptr));
}

}  // namespace few

// ----------------------------------------------------------- many rows ---
namespace rows {

using namespace tc;

constexpr int TM = 128, TK = 64, STAGES = 4;
constexpr int EPI_WARPS = 8, EPI0 = 4;  // the epilogue's first warp: warp & 3 is its quarter of the lanes
constexpr int THREADS = (EPI0 + EPI_WARPS) * 32;
constexpr int PATCH = 32 * 64;  // bytes a warp's 32 rows x 32 results take in shared memory
constexpr unsigned long long WAIT_NS = 2000000000ull;

struct Args {
    Matmul16Call c;
    unsigned *status;
    int wtiles;  // weight tiles a matrix
    int vec_y, vec_res;  // 16-byte accesses fit y, the residual
};

template <int TN>
__host__ __device__ constexpr int stage_bytes() { return (TM + TN) * TK * 2; }
template <int TN>
__host__ __device__ constexpr size_t smem_bytes() {
    return 1024 + (size_t)STAGES * stage_bytes<TN>() + EPI_WARPS * PATCH + 2 * 2 * TN * 4 + (MAX_E + 1) * 8;
}

struct Item {
    int e, row0, nrows, wt;
};

// TN: weight rows of a tile (gate and up together).
template <typename T, int TN, bool PAIR>
__global__ void __launch_bounds__(THREADS, 1)
rows16_kernel(const Args a, const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
              const __grid_constant__ CUtensorMap map_up) {
    constexpr int COLS = PAIR ? TN / 2 : TN;  // results of a tile's row
    extern __shared__ char smem_raw[];
    char *smem = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    char *patches = smem + STAGES * stage_bytes<TN>();
    float *bias_s = reinterpret_cast<float *>(patches + EPI_WARPS * PATCH);  // [2][2][TN]: bias, bias_up of a tile
    int *start_s = reinterpret_cast<int *>(bias_s + 2 * 2 * TN);             // [E + 1] offsets
    int *item_s = start_s + MAX_E + 1;                                       // [E + 1] first row tile of an expert
    __shared__ __align__(8) unsigned long long bars[2 * STAGES + 4];
    __shared__ uint32_t tmem_s;
    __shared__ int abort_flag, bad_s, scan_s[THREADS / 32];
    const Matmul16Call &c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t full = smem_u32(bars), empty = full + STAGES * 8, tfull = empty + STAGES * 8, tempty = tfull + 16;
    if (tid == 0) {
        abort_flag = bad_s = 0;
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full + i * 8, 1);
            mbar_init(empty + i * 8, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull + i * 8, 1);
            mbar_init(tempty + i * 8, EPI_WARPS);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&map_x);
        prefetch_map(&map_w);
        if (PAIR) prefetch_map(&map_up);
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_s)), "r"(2 * TN)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    __syncthreads();
    // ---- row tiles of every expert
    int nE = c.expStart == nullptr ? 1 : c.E;
    if (c.expStart == nullptr) {
        if (tid == 0) {
            start_s[0] = 0, start_s[1] = c.n_rows;
            item_s[0] = 0, item_s[1] = (c.n_rows + TM - 1) / TM;
        }
    } else {
        int base = 0;
        for (int e0 = 0; e0 < nE; e0 += THREADS) {
            const int e = e0 + tid;
            int t = 0;
            if (e < nE) {
                const int s = c.expStart[e], s1 = c.expStart[e + 1];
                if (s < 0 || s1 < s || s1 > c.n_rows || (e == 0 && s != 0)) bad_s = 1;
                start_s[e] = s;
                if (e == nE - 1) start_s[nE] = s1;
                t = (max(s1 - s, 0) + TM - 1) / TM;
            }
            int in = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, in, o);
                if (lane >= o) in += v;
            }
            if (lane == 31) scan_s[warp] = in;
            __syncthreads();
            int before = base;
            for (int w = 0; w < warp; ++w) before += scan_s[w];
            for (int w = 0; w < THREADS / 32; ++w) base += scan_s[w];
            if (e < nE) item_s[e] = before + in - t;
            __syncthreads();
        }
        if (tid == 0) item_s[nE] = base;
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_s;
    const bool bad = bad_s != 0;
    if (bad && blockIdx.x == 0 && tid == 0) atomicOr(a.status, MOE_DEV_BAD_CSR);
    const int64_t items = bad ? 0 : (int64_t)item_s[nE] * a.wtiles;
    const int steps = (c.K + TK - 1) / TK;
    // item: expert by expert, weight tile by weight tile, the row tiles of one beside each other (they share its weights)
    auto item_at = [&](int64_t it) {
        int lo = 0, hi = nE;  // the expert with item_s[e] * wtiles <= it < item_s[e + 1] * wtiles
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if ((int64_t)item_s[mid] * a.wtiles <= it)
                lo = mid;
            else
                hi = mid;
        }
        const int tiles = item_s[lo + 1] - item_s[lo], in = (int)(it - (int64_t)item_s[lo] * a.wtiles);
        Item x;
        x.e = lo;
        x.wt = in / tiles;
        x.row0 = start_s[lo] + (in - x.wt * tiles) * TM;
        x.nrows = min(TM, start_s[lo + 1] - x.row0);
        return x;
    };

    if (warp == 0) {
        if (lane == 0) {
            int slot = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int64_t it = blockIdx.x; it < items && ok; it += gridDim.x) {
                const Item x = item_at(it);
                const int wrow = x.e * c.R + x.wt * COLS;
                for (int k = 0; k < steps; ++k) {
                    ok = mbar_wait(empty + slot * 8, phase ^ 1, &abort_flag, a.status, WAIT_NS);
                    if (!ok) break;
                    const uint32_t at = smem_u32(smem) + slot * stage_bytes<TN>(), b = full + slot * 8;
                    mbar_expect_tx(b, stage_bytes<TN>());
                    tma_load_2d(at, &map_x, k * TK, x.row0, b);
                    tma_load_2d(at + TM * TK * 2, &map_w, k * TK, wrow, b);
                    if (PAIR) tma_load_2d(at + (TM + COLS) * TK * 2, &map_up, k * TK, wrow, b);
                    ++issued;
                    if (++slot == STAGES) slot = 0, phase ^= 1;
                }
            }
            if (!ok) s16::drain(full, STAGES, issued);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = (1u << 4) | (std::is_same_v<T, __half> ? 0u : (1u << 7) | (1u << 10)) |
                                       ((uint32_t)(TN >> 3) << 17) | ((uint32_t)(TM >> 4) << 24);
            int slot = 0, buf = 0;
            uint32_t phase = 0, tphase = 0;
            bool ok = true, any = false;
            for (int64_t it = blockIdx.x; it < items && ok; it += gridDim.x) {
                ok = mbar_wait(tempty + buf * 8, tphase ^ 1, &abort_flag, a.status, WAIT_NS);
                if (!ok) break;
                tc_fence_after();
                for (int k = 0; k < steps; ++k) {
                    ok = mbar_wait(full + slot * 8, phase, &abort_flag, a.status, WAIT_NS);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t at = smem_u32(smem) + slot * stage_bytes<TN>();
#pragma unroll
                    for (int j = 0; j < TK / 16; ++j)
                        mma_f16(tmem + buf * TN, smem_desc_sw128(at + j * 32), smem_desc_sw128(at + TM * TK * 2 + j * 32), idesc,
                                k > 0 || j > 0);
                    mma_commit(empty + slot * 8);
                    any = true;
                    if (++slot == STAGES) slot = 0, phase ^= 1;
                }
                if (!ok) break;
                mma_commit(tfull + buf * 8);
                if (++buf == 2) buf = 0, tphase ^= 1;
            }
            if (!ok && any) {
                // products still in flight: the last stage's commit tells when they are done (its barrier's phase)
                const int last = (slot + STAGES - 1) % STAGES;
                const uint32_t p = slot == 0 ? phase ^ 1 : phase;
                const uint64_t t0 = globaltimer();
                while (!mbar_try(empty + last * 8, p) && globaltimer() - t0 < WAIT_NS) {}
            }
        }
    } else if (warp >= EPI0) {
        const int ew = warp - EPI0, quarter = warp & 3, half = ew >> 2, et = tid - EPI0 * 32;
        char *patch = patches + ew * PATCH;
        int buf = 0;
        uint32_t tphase = 0;
        T *y = static_cast<T *>(c.y);
        const T *res = static_cast<const T *>(c.residual);
        for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
            const Item x = item_at(it);
            const int col0 = x.wt * COLS;
            float *bs = bias_s + buf * 2 * TN;
            if (c.bias != nullptr || c.bias_up != nullptr) {
                for (int i = et; i < COLS; i += EPI_WARPS * 32) {
                    const bool in = col0 + i < c.R;
                    const int64_t at = (int64_t)x.e * c.R + col0 + i;
                    bs[i] = in && c.bias != nullptr ? c.bias[at] : 0.0f;
                    if (PAIR) bs[TN + i] = in && c.bias_up != nullptr ? c.bias_up[at] : 0.0f;
                }
                asm volatile("bar.sync 2, %0;" ::"n"(EPI_WARPS * 32) : "memory");
            }
            const bool ok = __all_sync(0xffffffffu, mbar_wait(tfull + buf * 8, tphase, &abort_flag, a.status, WAIT_NS));
            if (ok) {
                tc_fence_after();
                const int row = quarter * 32 + lane;  // of the tile
                const bool warp_rows = quarter * 32 < x.nrows;
                const int64_t yrow = (int64_t)(x.row0 + quarter * 32);
#pragma unroll 1
                for (int c0 = half * (COLS / 2); c0 < (half + 1) * (COLS / 2); c0 += 32) {
                    if (!warp_rows || col0 + c0 >= c.R) break;
                    uint32_t r[32], ru[32];
                    tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + buf * TN + c0, r);
                    if (PAIR) tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + buf * TN + COLS + c0, ru);
                    tmem_wait_ld();
                    tmem_reg_fence32(r);
                    if (PAIR) tmem_reg_fence32(ru);
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
                    if (c.bias != nullptr)
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] += bs[c0 + i];
                    activate(v, c.act);
                    if (PAIR) {
                        if (c.bias_up != nullptr)
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] *= __uint_as_float(ru[i]) + bs[TN + c0 + i];
                        else
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] *= __uint_as_float(ru[i]);
                    }
                    if (res != nullptr && row < x.nrows) {
                        const T *from = res + (int64_t)(x.row0 + row) * c.residual_stride + col0 + c0;
                        if (a.vec_res && col0 + c0 + 32 <= c.R) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                Pack<T, 8> p;
                                p.load(from + i * 8);
#pragma unroll
                                for (int j = 0; j < 8; ++j) v[i * 8 + j] += p.get(j);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (col0 + c0 + i < c.R) {
                                    Pack<T, 1> p;
                                    p.load(from + i);
                                    v[i] += p.get(0);
                                }
                        }
                    }
                    // a row's 64 bytes in four pieces, their places turned by the row so that no two lanes of an access
                    // share a bank more often than they must
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        Pack<T, 8> p;
                        const float o[8] = {v[i * 8], v[i * 8 + 1], v[i * 8 + 2], v[i * 8 + 3], v[i * 8 + 4], v[i * 8 + 5], v[i * 8 + 6], v[i * 8 + 7]};
                        p.set(o);
                        *reinterpret_cast<uint4 *>(patch + lane * 64 + ((i ^ (lane >> 1)) & 3) * 16) = p.a;
                    }
                    __syncwarp();
                    if (a.vec_y && col0 + c0 + 32 <= c.R) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int rr = i * 8 + (lane >> 2), q = lane & 3;
                            const uint4 o = *reinterpret_cast<const uint4 *>(patch + rr * 64 + ((q ^ (rr >> 1)) & 3) * 16);
                            if (quarter * 32 + rr < x.nrows)
                                *reinterpret_cast<uint4 *>(y + (yrow + rr) * c.y_stride + col0 + c0 + q * 8) = o;
                        }
                    } else if (col0 + c0 + lane < c.R) {
                        for (int rr = 0; rr < 32 && quarter * 32 + rr < x.nrows; ++rr)
                            y[(yrow + rr) * c.y_stride + col0 + c0 + lane] = *reinterpret_cast<const T *>(
                                patch + rr * 64 + (((lane >> 3) ^ (rr >> 1)) & 3) * 16 + (lane & 7) * 2);
                    }
                }
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty + buf * 8);
            if (++buf == 2) buf = 0, tphase ^= 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * TN) : "memory");
}

int launch(const Matmul16Call &c, unsigned *status, cudaStream_t s) {
    const int sms = std::max(1, device_sm_count());
    const bool pair = c.w_up != nullptr, f16 = c.dtype == MOE_DTYPE_F16;
    Args a{};
    a.c = c;
    a.status = status;
    auto bits = [](const void *p, int64_t stride) { return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)(stride * 2)) % 16 == 0; };
    a.vec_y = bits(c.y, c.y_stride);
    a.vec_res = c.residual != nullptr && bits(c.residual, c.residual_stride);
    auto go = [&](auto kernel, int tn, size_t smem, SmemOptIn *done) {
        const int cols = pair ? tn / 2 : tn;
        a.wtiles = (c.R + cols - 1) / cols;
        CUtensorMap mx, mw, mu;
        if (!encode_16bit_sw128_2d(&mx, c.x, f16, c.n_rows, c.K, c.x_stride, TM) ||
            !encode_16bit_sw128_2d(&mw, c.w, f16, (uint64_t)c.E * c.R, c.K, c.K, cols) ||
            !encode_16bit_sw128_2d(&mu, pair ? c.w_up : c.w, f16, (uint64_t)c.E * c.R, c.K, c.K, cols))
            return (int)MOE_ERR_CUDA;
        if (int rc = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), smem, done)) return rc;
        const int64_t most = ((int64_t)(c.n_rows + TM - 1) / TM + (c.expStart ? c.E : 0)) * a.wtiles;
        kernel<<<(unsigned)std::min<int64_t>(most, sms), THREADS, smem, s>>>(a, mx, mw, mu);
        return launch_status();
    };
    auto by_type = [&](auto *tp) {
        using T = std::remove_pointer_t<decltype(tp)>;
        static SmemOptIn done[2];
        if (pair) return go(rows16_kernel<T, 256, true>, 256, smem_bytes<256>(), &done[0]);
        return go(rows16_kernel<T, 256, false>, 256, smem_bytes<256>(), &done[1]);
    };
    return f16 ? by_type(static_cast<__half *>(nullptr)) : by_type(static_cast<__nv_bfloat16 *>(nullptr));
}

}  // namespace rows

}  // namespace

int launch_matmul16(const Matmul16Call &c, unsigned *status, cudaStream_t s) {
    // 32 rows are four column tiles of the few-row kernel's instructions; beyond them it would read the weights again
    return c.n_rows <= s16::MAX_ROWS ? few::launch(c, status, s) : rows::launch(c, status, s);
}

}  // namespace moe
