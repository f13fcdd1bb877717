// stream16.cuh -- 16-bit weight rows streamed through a shared-memory ring into products with a few activation rows,
// for the few-row products and the whole layer of decode batches.
//
// Such products read every weight once, so the bytes bound them.  A CTA's two groups of eight warps have a ring and a
// producer warp each, which asks for tiles of up to 16 weight rows x KC columns by bulk copies as far ahead as the ring
// reaches (some 200 KB an SM in both, more than the memory system needs in flight).  The group's warps share a tile's
// columns and multiply with mma.sync m16n8k16, weights as the 16 rows, up to 8 activation rows as the columns,
// accumulators in registers in fp32.  (tcgen05.mma would hold 128 rows against columns that are not there, and its
// operands' layout would cost the copies their freedom: a tenth of the tensor pipe's time is all that these products
// take.) Two groups: what a stage costs a warp beside its products (the wait, the addresses) is paid by half of the
// warps, and a group's latency passes while the other works.
//
// A dot product does not care for the order of its columns, as long as both operands share it: lane (g, t) takes the 8
// consecutive columns 8 t .. 8 t + 7 of a 32-wide chunk, one 16-byte access of weight row g, of row g + 8 and of
// activation row g, and feeds them to two instructions.  Rows lie 64 bytes past a multiple of 128 apart: no bank
// conflicts (see Layout for the weights').
#pragma once

#include "elem.cuh"
#include "tc_glue.cuh"

namespace moe {
namespace s16 {

constexpr int CONSUMERS = 16;                      // warps, in
constexpr int GROUPS = 2;                          // groups, each with a ring and a producer warp of its own
constexpr int GROUP_WARPS = CONSUMERS / GROUPS;
constexpr int THREADS = (CONSUMERS + GROUPS) * 32; // the producers are the last warps
constexpr int MAX_STAGES = 8;                      // of a ring
constexpr int MAX_ROWS = 32;                       // activation rows: four tiles of columns
constexpr size_t SMEM_LIMIT = 227 * 1024;
constexpr unsigned long long WAIT_NS = 1000000000ull;  // 1 s: a healthy wait takes microseconds

// Row pitch in bytes of `cols` 16-bit columns.
__host__ __device__ constexpr int pitch_of(int cols) { return (cols * 2 + 127) / 128 * 128 + 64; }

// How up to 16 weight rows lie in a stage.  The copy engine takes some 45 ns a copy whatever its size, as much as 2 KB
// take at the memory's rate.  Rows of up to half of that come four to a copy (they follow one another in memory): a
// layer of 5 tokens with experts of 512 columns takes 58 us, row by row 62.  Longer rows come a copy each, in pieces of
// KC columns: four at a time, a layer of 32 tokens with experts of 768 columns took 213 us against 207 (a slot is held
// until the last row of four has landed).  Row s lies at (s & 3) rows and (s >> 2) fours, and lane g reads rows
// (g >> 1) + 4 (g & 1) and 8 more: the two rows of an access phase belong to fours an odd multiple of 64 bytes apart,
// so that no two lanes meet in a bank.
constexpr int KC = 1024;    // columns of a stage at most
constexpr int FOURS = 512;  // columns of rows that come four at a time
struct Layout {
    int row, four;  // bytes
    bool whole;
    __device__ __forceinline__ explicit Layout(int K) {
        whole = K <= FOURS;
        row = whole ? K * 2 : (min(K, KC) + 31) / 32 * 64 + 16;
        four = 4 * row;
        if (four % 128 == 0) four += 64;  // (16 rows stay below 16 pitch_of(K))
    }
    __device__ __forceinline__ int lane_at(int g) const { return (g & 1) * four + (g >> 1) * row; }
};
// The lane that reads row r (0 .. 7).
__device__ __forceinline__ int lane_of_row(int r) { return (r & 3) * 2 + (r >> 2); }

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (std::is_same_v<T, __half>)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <typename T>
__device__ __forceinline__ void mma_chunk(float (&d)[4], const uint4 &lo, const uint4 &hi, const uint4 &b) {
    mma<T>(d, lo.x, hi.x, lo.y, hi.y, b.x, b.y);
    mma<T>(d, lo.z, hi.z, lo.w, hi.w, b.z, b.w);
}

// Named barriers: 1 of all consumers, 2 on of a group.
__device__ __forceinline__ void group_sync(int group) {
    asm volatile("bar.sync %0, %1;" ::"r"(2 + group), "n"(GROUP_WARPS * 32) : "memory");
}
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(CONSUMERS * 32) : "memory"); }

// A group's ring: stages of 16 rows `pitch` bytes apart; full barriers (the copies' bytes) and empty ones (a warp
// each).  The group sees every phase of its barriers in order, which their parity alone would not survive otherwise:
// copies land out of order, so a ring that two groups shared in turns could show one of them a slot's phase before
// last.  Every wait is bounded: when one runs out, the CTA's abort flag is raised and all further waits return at once,
// so that every thread still walks its loops and barriers to their end (and writes no result).
struct Ring {
    char *base;
    uint32_t bar;   // full barriers, then empty ones
    int stages, pitch;
    int *abort_flag;
    unsigned *status;
    int slot = 0;
    uint32_t phase = 0;

    // `mem`: the rings behind one another, `bars`: their barriers
    __device__ __forceinline__ Ring(char *mem, uint32_t bars, int group, int stages, int pitch, int *abort_flag, unsigned *status)
        : base(mem + (size_t)group * stages * 16 * pitch), bar(bars + group * stages * 16), stages(stages), pitch(pitch),
          abort_flag(abort_flag), status(status) {}

    __device__ __forceinline__ char *stage() const { return base + (size_t)slot * 16 * pitch; }
    __device__ __forceinline__ void next() {
        if (++slot == stages) slot = 0, phase ^= 1;
    }
    __device__ __forceinline__ bool wait_full() const {
        return tc::mbar_wait(bar + slot * 8, phase, abort_flag, status, WAIT_NS);
    }
    __device__ __forceinline__ bool wait_empty() const {
        return tc::mbar_wait(bar + (stages + slot) * 8, phase ^ 1, abort_flag, status, WAIT_NS);
    }
    __device__ __forceinline__ void release(int lane) const {  // one arrival a warp
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar + (stages + slot) * 8);
    }
    // Producer warp: `cols` columns of 16 rows or fewer, n0 from src0 on and, as rows 8 on, n1 from src1 on (rows K
    // columns long).  False after a timeout.
    template <typename T>
    __device__ __forceinline__ bool produce(int lane, const Layout &y, int K, int cols, const T *src0, int n0, const T *src1, int n1) {
        const bool ok = __all_sync(0xffffffffu, wait_empty());
        if (!ok) return false;
        const uint32_t full = bar + slot * 8;
        if (lane == 0) tc::mbar_expect_tx(full, (uint32_t)((n0 + n1) * cols * 2));
        __syncwarp();
        const int s = y.whole ? lane * 4 : lane, r = s & 7;  // first row of the lane's copy
        const int left = (s < 8 ? n0 : s < 16 ? n1 : 0) - r, rows = y.whole ? min(4, left) : min(1, left);
        if (rows > 0)
            tc::bulk_load(tc::smem_u32(stage()) + (s >> 2) * y.four + (s & 3) * y.row, (s < 8 ? src0 : src1) + (int64_t)r * K,
                          (uint32_t)(rows * cols * 2), full);
        next();
        return true;
    }
};

// After a timeout: the copies that `issued` phases of `stages` full barriers have in flight land (or a limit passes)
// before the CTA ends.
__device__ __forceinline__ void drain(uint32_t full, int stages, int issued) {
    const uint64_t t0 = tc::globaltimer();
    for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
        while (!tc::mbar_try(full + (i % stages) * 8, (i / stages) & 1) && tc::globaltimer() - t0 < WAIT_NS) {}
}

// The rings' barriers in shared memory at `bars`; call with one thread, then synchronise the CTA.
__device__ __forceinline__ void init_rings(uint32_t bars, int stages) {
    for (int r = 0; r < GROUPS; ++r)
        for (int i = 0; i < stages; ++i) {
            tc::mbar_init(bars + (r * 2 * stages + i) * 8, 1);
            tc::mbar_init(bars + ((r * 2 + 1) * stages + i) * 8, GROUP_WARPS);
        }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

constexpr int CHUNKS = KC / (GROUP_WARPS * 32);      // 32-wide chunks a warp takes of a stage

// The units of a group: what is at work at a time lies side by side in memory, and every CTA gets its share of each
// expert's, so that experts that cost more cost all of them the same.
__device__ __forceinline__ int first_unit(int group) { return blockIdx.x + group * gridDim.x; }
__device__ __forceinline__ int unit_stride() { return GROUPS * gridDim.x; }

// The sums of a group's warps meet in shared memory, red [GROUP_WARPS][nt][32] float4 in the accumulators' order.
template <int NTM>
__device__ __forceinline__ void share_sums(float4 *red, int nt, const float (&acc)[NTM][4], int warp, int lane) {
#pragma unroll
    for (int n = 0; n < NTM; ++n)
        if (n < nt) red[(warp * nt + n) * 32 + lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
}
// Component `i` (0..3) of lane `l` in tile n, added over `WARPS` warps in order.
template <int WARPS = GROUP_WARPS>
__device__ __forceinline__ float sum_of(const float4 *red, int nt, int n, int l, int i) {
    const float *p = reinterpret_cast<const float *>(red + n * 32 + l) + i;
    float v = p[0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) v += p[w * nt * 128];
    return v;
}

// A group's share of the units (tiles of weight rows, as its producer deals them) times the activation rows that each
// of them meets, K columns, kc a stage.
//   info(u)    {first, n}: the unit's activation rows, n <= 8 NTM of them from place `first` on
//   at(i)      address of the activation row in place i
//   done(u, info, sums, nt, thread)  by all threads of a group: its warps' sums of the unit's nt tiles of 8 rows (see sum_of)
// The activations of a stage are asked for before the wait for its weights.  red: GROUP_WARPS * NTM * 32 float4 a
// group.
template <typename T, int NTM, typename Info, typename At, typename Done>
__device__ __forceinline__ void stream_units(Ring &ring, int units, int K, int kc, float4 *red, int warp,
                                             int lane, Info info, At at, Done done) {
    const int g = lane >> 2, t = lane & 3, group = warp / GROUP_WARPS, gw = warp % GROUP_WARPS;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const Layout lay(K);
    float4 *sums = red + group * GROUP_WARPS * NTM * 32;
    for (int u = first_unit(group); u < units; u += unit_stride()) {
        const int2 in = info(u);
        const int nt = (in.y + 7) / 8;
        const T *x[NTM];
#pragma unroll
        for (int n = 0; n < NTM; ++n) x[n] = static_cast<const T *>(at(in.x + min(n * 8 + g, in.y - 1))) + t * 8;
        float acc[NTM][4] = {};
        for (int k0 = 0; k0 < K; k0 += kc) {
            const int cols = min(kc, K - k0);
            uint4 b[NTM == 1 ? 1 : 2][CHUNKS];
            auto fetch = [&](int n) {
#pragma unroll
                for (int q = 0; q < CHUNKS; ++q) {
                    const int c = (q * GROUP_WARPS + gw) * 32;
                    b[n % 2][q] = zero;
                    if (c + t * 8 < cols) b[n % 2][q] = *reinterpret_cast<const uint4 *>(x[n] + k0 + c);
                }
            };
            fetch(0);
            ring.wait_full();
            const char *w = ring.stage() + lay.lane_at(g) + t * 16;
#pragma unroll
            for (int n = 0; n < NTM; ++n)
                if (n == 0 || n < nt) {
                    if (n + 1 < NTM && n + 1 < nt) fetch(n + 1);  // while this tile is at work
#pragma unroll
                    for (int q = 0; q < CHUNKS; ++q) {
                        const int c = (q * GROUP_WARPS + gw) * 32;
                        if (c >= cols) break;
                        uint4 lo = zero, hi = zero;
                        if (c + t * 8 < cols) {
                            lo = *reinterpret_cast<const uint4 *>(w + c * 2);
                            hi = *reinterpret_cast<const uint4 *>(w + 2 * lay.four + c * 2);
                        }
                        mma_chunk<T>(acc[n], lo, hi, b[n % 2][q]);
                    }
                }
            ring.release(lane);
            ring.next();
        }
        group_sync(group);  // the sums before these have been read
        share_sums<NTM>(sums, nt, acc, gw, lane);
        group_sync(group);
        done(u, in, sums, nt, gw * 32 + lane);
    }
}

}  // namespace s16
}  // namespace moe
