// matmul16.cu -- products of 16-bit rows with 16-bit matrices, one matrix or one per expert over rows in CSR order,
// with bias, activation (or gate and up) and residual in the epilogue:
//   y[j] = act(W[e] x[j] + b[e]) (* (U[e] x[j] + c[e])) (+ residual[j])
//
// Two kernels.  Few rows (serving, see few::serves): every weight is read for a few rows, so its bytes bound the
// product; few16_kernel streams them as stream16.cuh says (8 x 32768 x 4096: 45 us, 6.0 TB/s, 89% of a copy).  More
// rows (prompts, training): rows16_kernel forms tiles of 256 weight rows (gate and up: 128 of each) on the tensor
// cores.
//
// rows16_kernel is persistent; two CTAs of a cluster work as a pair: the weights are the 256 rows of their products
// (tcgen05.mma cta_group::2, 128 rows a CTA), up to 256 token rows the columns, in steps of 16, so that ragged segments
// cost what they hold.  Warps in roles: in each CTA a producer that brings its 128 weight rows and its half of the
// token rows in by TMA (128-byte swizzle, 64 columns a stage, six stages), in the first an issuer of the products
// (accumulators in tensor memory, two tiles of 256 columns so that the next tile's products run under this one's
// epilogue), in each twelve epilogue warps (a lane holds a weight row's results for 32 tokens; where 16-byte accesses
// fit they cross shared memory so that rows leave in whole sectors).  Sharing the token rows between the CTAs is what
// lets shared memory keep up: alone, a CTA's products would read 96 bytes a cycle while its copies write 94.  Segments
// start at any row: a tile reads past its segment's end and stores nothing of what it finds there.
// bf16, 8192 x 8192 x 2048: 147 us, 1.87 PFLOP/s (with bias and GELU 154), the tensor pipe active in 90% of the cycles;
// gate and up of 64 experts of 1024 x 2048 over 16384 rows 118 us, 5.4 TB/s and 55% of the pipe: a wave of tiles asks
// for its weights all at once, and half of the experts have a few rows more than a tile holds.
#include <algorithm>
#include <atomic>

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
    const int units = listed_s * a.tiles;
    if ((int)blockIdx.x >= units) return;
    const int group = warp < CONSUMERS ? warp / GROUP_WARPS : warp - CONSUMERS;
    Ring ring(smem, bar, group, a.stages, a.pitch, &abort_flag, a.status);
    const int rows_x = first_s[listed_s];

    if (warp >= CONSUMERS) {
        const Layout lay(c.K);
        int issued = 0;
        bool ok = true;
        if (a.x_pitch && group == 0) {
            if (lane == 0) tc::mbar_expect_tx(xbar, (uint32_t)(rows_x * c.K * 2));
            __syncwarp();
            if (lane < rows_x) tc::bulk_load(tc::smem_u32(smem + a.x_at) + lane * a.x_pitch, x + lane * c.x_stride, c.K * 2, xbar);
        }
        for (int u = first_unit(group); u < units && ok; u += unit_stride()) {
            const int i = u / a.tiles, r = (u - i * a.tiles) * a.tile, n = min(a.tile, c.R - r);
            const int64_t row = (int64_t)expert_s[i] * c.R + r;
            const T *w = static_cast<const T *>(c.w) + row * c.K, *second = pair ? static_cast<const T *>(c.w_up) + row * c.K : w + (int64_t)8 * c.K;
            const int n0 = min(n, 8), n1 = pair ? n : n - n0;
            for (int k0 = 0; k0 < c.K && ok; k0 += a.kc) {
                ok = ring.produce(lane, lay, c.K, min(a.kc, c.K - k0), w + k0, n0, second + k0, n1);
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
    auto info = [&](int u) {
        const int i = u / a.tiles;
        return make_int2(first_s[i], first_s[i + 1] - first_s[i]);
    };
    auto at = [&](int row) { return xb + row * xs; };
    auto done = [&](int u, const int2 &in, const float4 *s, int nt, int thread) {
        if (*reinterpret_cast<volatile int *>(&abort_flag)) return;
        const int i = u / a.tiles, r = (u - i * a.tiles) * a.tile, here = min(a.tile, c.R - r);
        const int64_t e = expert_s[i];
        const int rl = pair ? 3 : 4;  // a unit's rows: 8 or 16
        for (int j = thread; j < nt << (rl + 3); j += GROUP_WARPS * 32) {
            const int row = j & ((1 << rl) - 1), col = (j >> rl) & 7, tile = j >> (rl + 3), l = lane_of_row(row & 7) * 4 + (col >> 1);
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
    stream_units<T, NTM>(ring, units, c.K, a.kc, reinterpret_cast<float4 *>(smem + a.red_at), warp, lane, info, at, done);
}

// Whether the rows of `c` can lie in shared memory beside the rings, and the stages of these.
bool stage_rows(const Matmul16Call &c, int pitch, size_t red, int *stages) {
    const size_t ring = (size_t)GROUPS * 16 * pitch, most = SMEM_LIMIT - 4096, xb = (size_t)c.n_rows * pitch_of(c.K);
    *stages = (int)std::min<size_t>(MAX_STAGES, (most - red) / ring);
    // where that costs a stage of each ring at most
    const bool staged = *stages > 2 && (*stages - 1) * ring + red + xb <= most;
    if (staged && *stages * ring + red + xb > most) --*stages;
    return staged;
}
int tiles_of(int n_rows) { return n_rows <= 8 ? 1 : n_rows <= 16 ? 2 : 4; }
size_t red_bytes(int n_rows) { return (size_t)CONSUMERS * tiles_of(n_rows) * 512; }
int columns(int K) { return std::min(KC, (K + 31) / 32 * 32); }

// Weight rows (gate and up: pairs) of a unit: 16 (8), fewer where that leaves SMs without one.
int tile_of(const Matmul16Call &c) {
    const int sms = std::max(1, device_sm_count());
    const int64_t most_rows = (int64_t)std::min(c.E, c.n_rows) * c.R;
    return (int)std::min<int64_t>(c.w_up != nullptr ? 8 : 16, (most_rows + sms - 1) / sms);
}

// The rows this kernel serves: 32 are four column tiles of its instructions, and beyond them it would read the weights
// again.  Up to 8 an expert on average are one column tile: always.  More cost it what each unit of weights takes to
// multiply with all of them (and to fetch them from L2, unless they lie in shared memory); tiles take a time of their own
// that grows with K only.  In us from a graph, here and on tiles:
//   one matrix        n = 12          16           24           32
//   1000 x 4096      8.0 17.0     8.4 17.0    12.5 17.2    15.6 17.3    (143 units)
//   2048 x 2048 *    5.9 10.9     6.1 10.9     8.4 11.0    10.2 11.0    (147; * in shared memory: 12 and 16 rows)
//   2048 x 16384    24.9 51.6    25.0 51.7    41.8 51.6    54.8 51.7    (147)
//   4096 x 4096     12.1 17.1    12.5 17.1    16.3 17.0    19.7 17.2    (256)
//   8192 x 2048 *   10.2 11.6    10.5 11.6    16.6 11.8    19.9 11.7    (512)
//   8192 x 8192     31.4 29.5    33.3 29.5    48.5 29.5    60.2 29.8    (512)
//   16384 x 2048 *  16.1 15.5    16.2 15.5    27.9 15.6    33.2 15.7    (1024)
//   by offsets, 8192 x 8192: 1 matrix 16 rows 33.9 34.7, 32 rows 60.7 34.9; 2 matrices 16 rows 46.9 50.5, 32 rows
//   60.9 50.5; 3, 32 rows 84.7 81.5; 4, 32 rows 86.5 91.8; 1000 x 4096: 2, 32 rows 10.9 18.7; 3, 32 rows 11.3 19.0
// (Where most of the rows are one expert's, which only the device knows, it is as with one matrix.)
bool serves(const Matmul16Call &c) {
    if (c.n_rows > MAX_ROWS) return false;
    if (c.n_rows <= 8 * c.E) return true;
    const int tile = tile_of(c);
    const int64_t units = (c.R + tile - 1) / tile;
    int stages;
    return units * c.n_rows <= (stage_rows(c, pitch_of(columns(c.K)), red_bytes(c.n_rows), &stages) ? 8192 : 5600);
}

int launch(const Matmul16Call &c, unsigned *status, cudaStream_t s) {
    Args a{};
    a.c = c;
    a.status = status;
    const int sms = std::max(1, device_sm_count());
    const int ntm = tiles_of(c.n_rows);
    a.tile = tile_of(c);
    a.tiles = (c.R + a.tile - 1) / a.tile;
    a.kc = columns(c.K);
    a.pitch = pitch_of(a.kc);
    const size_t red = red_bytes(c.n_rows), most = SMEM_LIMIT - 4096;
    const bool staged = stage_rows(c, a.pitch, red, &a.stages);
    a.x_pitch = staged ? pitch_of(c.K) : 0;
    a.x_at = (int)((size_t)a.stages * GROUPS * 16 * a.pitch);
    a.red_at = a.x_at + (staged ? c.n_rows * a.x_pitch : 0);
    const size_t smem = a.red_at + red;
    const int64_t units = (int64_t)std::min(c.E, c.n_rows) * a.tiles;
    if (units > 0x40000000) return MOE_ERR_UNSUPPORTED_SHAPE;
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

constexpr int TK = 64;         // columns of a stage: 128 bytes, the swizzle's width
constexpr int HALF = 128;      // weight rows of a CTA, and token rows it brings at most
constexpr int TILE = 2 * HALF; // of the pair
constexpr int MAX_STAGES = 10;
constexpr int STAGE_A = HALF * TK * 2;              // bytes of a stage's weight rows
constexpr size_t RING = 6 * 2 * (size_t)STAGE_A;    // six stages with all token rows, more with fewer
constexpr int SPAN = 2;        // stages that one wait of the issuer covers
constexpr int RASTER = 8;       // row tiles side by side
constexpr int EPI_WARPS = 12, EPI0 = 4;  // the epilogue's first warp: warp & 3 is its quarter of the lanes
constexpr int EPI_SETS = EPI_WARPS / 4; // of four warps, on 32 token rows in turn
constexpr int THREADS = (EPI0 + EPI_WARPS) * 32;
constexpr int PATCH = 32 * 64;          // bytes of 32 rows x 32 16-bit results
constexpr int SWAP = 32 * 32 * 4;       // bytes of 32 x 32 fp32 values of up on their way to the gate's warp
constexpr unsigned long long WAIT_NS = 2000000000ull;

template <bool PAIR>
struct Shape {
    static constexpr int COLS = PAIR ? HALF : TILE;  // result columns of the pair's tile
    // a patch a warp; gate and up: one for both warps of a pair, where up's values pass first
    static constexpr int PATCHES = (PAIR ? EPI_WARPS / 2 * SWAP : EPI_WARPS * PATCH);
    static constexpr size_t SMEM = 1024 + RING + PATCHES + (MAX_E + 1) * 8;
};

struct Args {
    Matmul16Call c;
    unsigned *status;
    int wtiles;  // weight tiles a matrix
    int width;   // token rows of a tile at most
    int vec_y;   // 16-byte accesses fit y
    int stages, stage;  // of the ring: how many (a multiple of SPAN), bytes of each
};
struct Maps {
    CUtensorMap w, up;
    CUtensorMap x[4];  // boxes of 16, 32, 64 and 128 rows
};

struct Item {
    int e, row0, nrows, wt;
    int n;  // columns of the product: nrows rounded up to 16
};

__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t at_cta(uint32_t addr, uint32_t rank) {  // the same place in CTA `rank`
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void pair_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Into this CTA's shared memory, counted on a barrier of either CTA of the pair.
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// One lane of a converged warp.  The issuer's warp walks its loops as a whole and lets one lane issue: what it computes
// is then known to be the same in all lanes and lies in the uniform registers that the instruction wants.
__device__ __forceinline__ bool elected() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, int accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void pair_commit(uint32_t bar) {  // arrives in both CTAs
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"((uint16_t)3)
                 : "memory");
}
// (Release at the CTA's scope: what it hands back is tensor memory, read behind tcgen05's own fence; a wider release
// would wait for the results' stores.)
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
template <typename T, bool PAIR>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
rows16_kernel(const Args a, const __grid_constant__ Maps maps) {
    using S = Shape<PAIR>;
    extern __shared__ char smem_raw[];
    char *smem = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int STAGES = a.stages, STAGE = a.stage;
    char *patches = smem + RING;
    int *start_s = reinterpret_cast<int *>(patches + S::PATCHES);  // [E + 1] offsets
    int *item_s = start_s + MAX_E + 1;                             // [E + 1] first row tile
    __shared__ __align__(8) unsigned long long bars[2 * MAX_STAGES + 4];
    __shared__ uint32_t tmem_s;
    __shared__ int abort_flag, bad_s, scan_s[THREADS / 32];
    const Matmul16Call &c = a.c;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, rank = (int)cta_rank();
    const uint32_t full = smem_u32(bars), empty = full + MAX_STAGES * 8, tfull = empty + MAX_STAGES * 8, tempty = tfull + 16;
    if (tid == 0) {
        abort_flag = bad_s = 0;
        for (int i = 0; i < STAGES; ++i) mbar_init(empty + i * 8, 1);
        for (int i = 0; i < STAGES / SPAN; ++i) mbar_init(full + i * 8, SPAN);
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull + i * 8, 1);
            mbar_init(tempty + i * 8, 2 * EPI_WARPS);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&maps.w);
        if (PAIR) prefetch_map(&maps.up);
        prefetch_map(&maps.x[3]);
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_s)), "r"(2 * TILE)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    __syncthreads();
    // ---- row tiles of every expert
    const int nE = c.expStart == nullptr ? 1 : c.E;
    if (c.expStart == nullptr) {
        if (tid == 0) {
            start_s[0] = 0, start_s[1] = c.n_rows;
            item_s[0] = 0, item_s[1] = (c.n_rows + a.width - 1) / a.width;
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
                t = (max(s1 - s, 0) + a.width - 1) / a.width;
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
    tc_fence_before();
    __syncthreads();
    pair_sync();  // both CTAs' barriers are initialised
    tc_fence_after();
    const uint32_t tmem = tmem_s;
    const bool bad = bad_s != 0;
    if (bad && blockIdx.x == 0 && tid == 0) atomicOr(a.status, MOE_DEV_BAD_CSR);
    const int64_t items = bad ? 0 : (int64_t)item_s[nE] * a.wtiles;
    // a wait in the thread that issues products costs it some 300 cycles of issue time, more than half of a stage's
    // products: it waits once for SPAN stages (an odd one out is followed by one without copies), which are released
    // one by one
    const int spans = (c.K + SPAN * TK - 1) / (SPAN * TK);
    const int64_t first = blockIdx.x / 2, stride = gridDim.x / 2;
    // item: expert by expert, RASTER row tiles at a time, weight tile by weight tile, the row tiles of one beside each
    // other (the pairs at work share weights and rows about evenly).
    // An expert's rows are dealt evenly to its row tiles: the product's width follows them in steps of 16.
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
        const int rows = start_s[lo + 1] - start_s[lo], per = ((rows + tiles - 1) / tiles + 15) / 16 * 16;
        const int g = in / (RASTER * a.wtiles), of = in - g * RASTER * a.wtiles, wide = min(RASTER, tiles - g * RASTER);
        Item x;
        x.e = lo;
        x.wt = of / wide;
        const int t = g * RASTER + of - x.wt * wide;
        x.row0 = start_s[lo] + t * per;
        x.nrows = max(0, min(per, rows - t * per));
        x.n = max(16, (x.nrows + 15) / 16 * 16);
        return x;
    };

    if (warp == 0) {
        const uint32_t base = smem_u32(smem), lead_full = at_cta(full, 0);
        int slot = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        auto wait_empty = [&]() {
            ok = __all_sync(0xffffffffu, mbar_wait(empty + slot * 8, phase ^ 1, &abort_flag, a.status, WAIT_NS));
            return ok;
        };
        for (int64_t it = first; it < items && ok; it += stride) {
            const Item x = item_at(it);
            const int mine = x.n / 2, box = mine <= 16 ? 0 : mine <= 32 ? 1 : mine <= 64 ? 2 : 3;
            const uint32_t bytes = STAGE_A + (16u << box) * TK * 2;
            const int wrow = x.e * c.R + x.wt * S::COLS + rank * (S::COLS / 2), xrow = x.row0 + rank * mine;
            for (int k = 0; k < spans * SPAN; ++k) {
                if (!wait_empty()) break;
                const uint32_t at = base + slot * STAGE, b = lead_full + slot / SPAN * 8;
                if (elected()) {
                    if (k * TK < c.K) {
                        if (rank == 0) mbar_expect_tx(full + slot / SPAN * 8, 2 * bytes);
                        pair_load_2d(at, &maps.w, k * TK, wrow, b);
                        if (PAIR) pair_load_2d(at + STAGE_A / 2, &maps.up, k * TK, wrow, b);
                        pair_load_2d(at + STAGE_A, &maps.x[box], k * TK, xrow, b);
                    } else if (rank == 0) {
                        mbar_arrive(full + slot / SPAN * 8);
                    }
                }
                __syncwarp();
                ++issued;
                if (++slot == STAGES) slot = 0, phase ^= 1;
            }
        }
        // the arrivals still on their way to this CTA's barriers
        for (int i = 0; i < STAGES && ok && wait_empty(); ++i)
            if (++slot == STAGES) slot = 0, phase ^= 1;
        if (!ok && rank == 0 && lane == 0) s16::drain(full, STAGES / SPAN, (issued + SPAN - 1) / SPAN);  // of both CTAs; the other waits for this one at the end
    } else if (warp == 1) {
        if (rank == 0) {
            constexpr uint32_t idesc = (1u << 4) | (std::is_same_v<T, __half> ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)(TILE >> 4) << 24);
            const uint32_t base = smem_u32(smem);
            int slot = 0, buf = 0;
            uint32_t phase = 0, tphase = 0;
            bool ok = true, any = false;
            for (int64_t it = first; it < items && ok; it += stride) {
                const uint32_t desc = idesc | ((uint32_t)(item_at(it).n >> 3) << 17);
                ok = __all_sync(0xffffffffu, mbar_wait(tempty + buf * 8, tphase ^ 1, &abort_flag, a.status, WAIT_NS));
                if (!ok) break;
                tc_fence_after();
                for (int k = 0; k < spans; ++k) {
                    ok = __all_sync(0xffffffffu, mbar_wait(full + slot / SPAN * 8, phase, &abort_flag, a.status, WAIT_NS));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t da = smem_desc_sw128(base + slot * STAGE), db = smem_desc_sw128(base + slot * STAGE + STAGE_A);
                    const uint32_t d = tmem + buf * TILE;
                    if (elected()) {
#pragma unroll
                        for (int q = 0; q < SPAN; ++q) {
                            if (q == 0 || (k * SPAN + q) * TK < c.K)
#pragma unroll
                                for (int j = 0; j < TK / 16; ++j)  // (addresses in a descriptor count 16 bytes)
                                    pair_mma(d, da + (uint32_t)(q * (STAGE / 16) + j * 2), db + (uint32_t)(q * (STAGE / 16) + j * 2), desc,
                                             k > 0 || q > 0 || j > 0);
                            pair_commit(empty + (slot + q) * 8);
                        }
                        if (k == spans - 1) pair_commit(tfull + buf * 8);
                    }
                    __syncwarp();
                    any = true;
                    if ((slot += SPAN) == STAGES) slot = 0, phase ^= 1;
                }
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
        // A lane has a weight row, its registers 32 token rows.  Gate and up: a CTA's first 64 lanes are gate rows, the
        // others the same up rows, whose warp hands its values to the gate's.
        const int ew = warp - EPI0, quarter = warp & 3, set = ew >> 2, side = PAIR ? quarter >> 1 : 0;
        const int pw = PAIR ? set * 2 + (quarter & 1) : ew;  // the warp's patch, and its pair of warps
        char *patch = patches + pw * (PAIR ? SWAP : PATCH);
        float *swap = reinterpret_cast<float *>(patch);
        int buf = 0;
        uint32_t tphase = 0;
        T *y = static_cast<T *>(c.y);
        const T *res = static_cast<const T *>(c.residual);
        const uint32_t lead_tempty = at_cta(tempty, 0);
        const float *bias = side ? c.bias_up : c.bias;
        for (int64_t it = first; it < items; it += stride) {
            const Item x = item_at(it);
            // the warp's 32 result columns
            const int col0 = x.wt * S::COLS + rank * (S::COLS / 2) + (PAIR ? quarter & 1 : quarter) * 32;
            const bool in = col0 + lane < c.R;
            const float b = bias != nullptr && in ? bias[(int64_t)x.e * c.R + col0 + lane] : 0.0f;
            const bool ok = __all_sync(0xffffffffu, mbar_wait(tfull + buf * 8, tphase, &abort_flag, a.status, WAIT_NS));
            tc_fence_after();
#pragma unroll 1
            for (int c0 = set * 32; c0 < x.nrows; c0 += EPI_SETS * 32) {
                if (col0 >= c.R) break;  // the same for both warps of a pair
                const int rows = min(32, x.nrows - c0);
                const int64_t row = x.row0 + c0;
                const bool add = res != nullptr && ok && !side;
                T rv[32];  // the residual, on its way while the results are formed (or, with two of these, while one waits)
                auto ask = [&]() {
                    if (!add) return;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (in && i < rows) rv[i] = res[(row + i) * c.residual_stride + col0 + lane];
                };
                if (!PAIR) ask();
                uint32_t r[32];
                float v[32];
                if (ok) {
                    tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + buf * TILE + c0, r);
                    tmem_wait_ld();
                    tmem_reg_fence32(r);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = ok ? __uint_as_float(r[i]) + b : 0.0f;
                if (PAIR) {
                    if (side) {
                        asm volatile("bar.sync %0, 64;" ::"r"(3 + 2 * pw) : "memory");  // the values before have been read
#pragma unroll
                        for (int i = 0; i < 32; ++i) swap[i * 32 + lane] = v[i];
                        asm volatile("bar.sync %0, 64;" ::"r"(4 + 2 * pw) : "memory");
                        continue;
                    }
                    activate(v, c.act);
                    ask();
                    asm volatile("bar.sync %0, 64;" ::"r"(3 + 2 * pw) : "memory");
                    asm volatile("bar.sync %0, 64;" ::"r"(4 + 2 * pw) : "memory");
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] *= swap[i * 32 + lane];
                } else {
                    activate(v, c.act);
                }
                if (add) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (in && i < rows) v[i] += (float)rv[i];
                }
                if (!ok) continue;
                if (a.vec_y && col0 + 32 <= c.R) {
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 32; ++i) *reinterpret_cast<T *>(patch + i * 64 + lane * 2) = elem_of<T>(v[i]);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int rr = i * 8 + (lane >> 2), q = lane & 3;
                        const uint4 o = *reinterpret_cast<const uint4 *>(patch + rr * 64 + q * 16);
                        if (rr < rows) *reinterpret_cast<uint4 *>(y + (row + rr) * c.y_stride + col0 + q * 8) = o;
                    }
                } else if (in) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (i < rows) y[(row + i) * c.y_stride + col0 + lane] = elem_of<T>(v[i]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_at(lead_tempty + buf * 8);
            if (++buf == 2) buf = 0, tphase ^= 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    pair_sync();  // neither CTA's barriers, shared or tensor memory are used by the other any more
    tc_fence_after();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * TILE) : "memory");
}

int launch(const Matmul16Call &c, unsigned *status, cudaStream_t s) {
    const bool f16 = c.dtype == MOE_DTYPE_F16;
    Args a{};
    a.c = c;
    a.status = status;
    a.vec_y = (reinterpret_cast<uintptr_t>(c.y) | (uintptr_t)(c.y_stride * 2)) % 16 == 0;
    auto go = [&](auto kernel, auto pc, SmemOptIn *done, std::atomic<int> *most_pairs) {
        using S = Shape<decltype(pc)::value>;
        a.wtiles = (c.R + S::COLS - 1) / S::COLS;
        const int wbox = c.w_up != nullptr ? HALF / 2 : HALF;
        Maps maps;
        bool ok = encode_16bit_sw128_2d(&maps.w, c.w, f16, (uint64_t)c.E * c.R, c.K, c.K, wbox) &&
                  encode_16bit_sw128_2d(&maps.up, c.w_up != nullptr ? c.w_up : c.w, f16, (uint64_t)c.E * c.R, c.K, c.K, wbox);
        for (int i = 0; i < 4; ++i) ok = ok && encode_16bit_sw128_2d(&maps.x[i], c.x, f16, c.n_rows, c.K, c.x_stride, 16 << i);
        if (!ok) return (int)MOE_ERR_CUDA;
        if (int rc = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), S::SMEM, done)) return rc;
        // every pair that runs at once (not all SMs need find a partner)
        const int dev = current_device();
        if (dev < 0) return (int)MOE_ERR_CUDA;
        int pairs = most_pairs[dev].load(std::memory_order_relaxed);
        if (pairs == 0) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(2);
            cfg.blockDim = dim3(THREADS);
            cfg.dynamicSmemBytes = S::SMEM;
            if (cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg) != cudaSuccess || pairs < 1) return (int)MOE_ERR_CUDA;
            most_pairs[dev].store(pairs, std::memory_order_relaxed);
        }
        // one matrix and few tiles: narrower ones, so that more SMs have one.  In us from a graph, tiles 64, 128 and 256
        // wide: 256 x 2048 x 2048 11.4 12.3 16.1, 1024 x 2048 x 2048 18.2 13.3 16.9, 2048 x 2048 x 2048 31.2 19.9 17.8,
        // 256 x 8192 x 2048 18.4 14.2 17.6, 300 x 1000 x 4096 17.6 19.0 20.3
        a.width = TILE;
        while (c.expStart == nullptr && a.width > 64 && (int64_t)((c.n_rows + a.width / 2 - 1) / (a.width / 2)) * a.wtiles <= pairs) a.width /= 2;
        // token rows of a CTA's half tile, as its box brings them
        const int half = c.expStart != nullptr ? HALF : std::min((std::min(a.width, c.n_rows) + 15) / 16 * 8, HALF);
        int box = 16;
        while (box < half) box *= 2;
        a.stage = STAGE_A + box * TK * 2;
        a.stages = std::min<int>(MAX_STAGES, (int)(RING / a.stage)) / SPAN * SPAN;
        const int64_t most = ((int64_t)(c.n_rows + a.width - 1) / a.width + (c.expStart ? std::min(c.E, c.n_rows) : 0)) * a.wtiles;
        kernel<<<(unsigned)(2 * std::min<int64_t>(most, pairs)), THREADS, S::SMEM, s>>>(a, maps);
        return launch_status();
    };
    auto by_type = [&](auto *tp) {
        using T = std::remove_pointer_t<decltype(tp)>;
        static SmemOptIn done[2];
        static std::atomic<int> pairs[2][MAX_DEVICES];
        if (c.w_up != nullptr) return go(rows16_kernel<T, true>, std::true_type(), &done[0], pairs[0]);
        return go(rows16_kernel<T, false>, std::false_type(), &done[1], pairs[1]);
    };
    return f16 ? by_type(static_cast<__half *>(nullptr)) : by_type(static_cast<__nv_bfloat16 *>(nullptr));
}

}  // namespace rows

}  // namespace

int launch_matmul16(const Matmul16Call &c, unsigned *status, cudaStream_t s) {
    return few::serves(c) ? few::launch(c, status, s) : rows::launch(c, status, s);
}

}  // namespace moe
