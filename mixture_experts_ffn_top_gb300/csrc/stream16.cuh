// stream16.cuh -- 16-bit weight rows streamed through a shared-memory ring into products with a few activation rows,
// for the few-row products and the whole layer of decode batches.
//
// Such products read every weight once, so the bytes bound them.  One warp of a CTA asks for tiles of up to 16 weight
// rows x KC columns by bulk copies, as far ahead as the ring reaches (some 200 KB an SM, more than the memory system
// needs in flight); eight warps share each tile's columns and multiply with mma.sync m16n8k16, weights as the 16
// rows, up to 8 activation rows as the columns, accumulators in registers in fp32.  (tcgen05.mma would hold 128 rows
// against columns that are not there, and its operands' layout would cost the copies their freedom.)
//
// A dot product does not care for the order of its columns, as long as both operands share it: lane (g, t) takes the 8
// consecutive columns 8 t .. 8 t + 7 of a 32-wide chunk, one 16-byte access of weight row g, of row g + 8 and of
// activation row g, and feeds them to two instructions.  Rows lie 64 bytes past a multiple of 128 apart: no bank
// conflicts.
#pragma once

#include "elem.cuh"
#include "tc_glue.cuh"

namespace moe {
namespace s16 {

constexpr int CONSUMERS = 8;                       // warps
constexpr int THREADS = (CONSUMERS + 1) * 32;      // and the producer, the last warp
constexpr int MAX_STAGES = 16;
constexpr int MAX_ROWS = 32;                       // activation rows: four tiles of columns
constexpr size_t SMEM_LIMIT = 227 * 1024;
constexpr unsigned long long WAIT_NS = 1000000000ull;  // 1 s: a healthy wait takes microseconds

// Row pitch in bytes of `cols` 16-bit columns.
__host__ __device__ constexpr int pitch_of(int cols) { return (cols * 2 + 127) / 128 * 128 + 64; }

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

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(CONSUMERS * 32) : "memory"); }

// The ring: stages of 16 rows `pitch` bytes apart; full barriers (the copies' bytes) and empty ones (a warp each).
// Every wait is bounded: when one runs out, the CTA's abort flag is raised and all further waits return at once, so
// that every thread still walks its loops and barriers to their end (and writes no result).
struct Ring {
    char *base;
    uint32_t bar;   // full barriers, then empty ones
    int stages, pitch, slot = 0;
    uint32_t phase = 0;
    int *abort_flag;
    unsigned *status;

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
    // Producer warp: the `rows` lanes with `mine` copy `bytes` from their src into the rows of their numbers.  False
    // after a timeout.
    __device__ __forceinline__ bool produce(int lane, bool mine, int rows, const void *src, uint32_t bytes) {
        const bool ok = __all_sync(0xffffffffu, wait_empty());
        if (!ok) return false;
        const uint32_t full = bar + slot * 8;
        if (lane == 0) tc::mbar_expect_tx(full, bytes * rows);
        __syncwarp();
        if (mine) tc::bulk_load(tc::smem_u32(stage()) + lane * pitch, src, bytes, full);
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

// Two barriers a stage in shared memory at `bar`; call with one thread, then synchronise the CTA.
__device__ __forceinline__ void init_ring(uint32_t bar, int stages) {
    for (int i = 0; i < stages; ++i) {
        tc::mbar_init(bar + i * 8, 1);
        tc::mbar_init(bar + (stages + i) * 8, CONSUMERS);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// Adds the products of the ring's stage, `cols` columns of it from column k0 on, to acc: NT tiles of 8 activation
// rows, x[n] the lane's row of tile n (columns 8 t on).
template <typename T, int NT, int NTM>
__device__ __forceinline__ void stage_products(const Ring &r, int cols, int k0, const T *const (&x)[NTM],
                                               float (&acc)[NTM][4], int warp, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const char *w = r.stage() + g * r.pitch + t * 16;
#pragma unroll 4
    for (int c = warp * 32; c < cols; c += CONSUMERS * 32) {
        const bool in = c + t * 8 < cols;
        uint4 lo = make_uint4(0, 0, 0, 0), hi = lo, b[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) b[n] = lo;
        if (in) {
            lo = *reinterpret_cast<const uint4 *>(w + c * 2);
            hi = *reinterpret_cast<const uint4 *>(w + 8 * r.pitch + c * 2);
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = *reinterpret_cast<const uint4 *>(x[n] + k0 + c);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_chunk<T>(acc[n], lo, hi, b[n]);
    }
}
// The same for a number of tiles known at run time.
template <typename T, int NTM>
__device__ __forceinline__ void stage_products_nt(const Ring &r, int cols, int k0, int nt, const T *const (&x)[NTM],
                                                  float (&acc)[NTM][4], int warp, int lane) {
    if (NTM == 1 || nt == 1) return stage_products<T, 1, NTM>(r, cols, k0, x, acc, warp, lane);
    if (NTM == 2 || nt == 2) return stage_products<T, NTM < 2 ? 1 : 2, NTM>(r, cols, k0, x, acc, warp, lane);
    stage_products<T, NTM, NTM>(r, cols, k0, x, acc, warp, lane);
}

// The warps' sums of a tile meet in shared memory, red [CONSUMERS][nt][32] float4 in the accumulators' order.
template <int NTM>
__device__ __forceinline__ void share_sums(float4 *red, int nt, const float (&acc)[NTM][4], int warp, int lane) {
#pragma unroll
    for (int n = 0; n < NTM; ++n)
        if (n < nt) red[(warp * nt + n) * 32 + lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
}
// Component `i` (0..3) of lane `l` in tile n, added over the warps in order.
__device__ __forceinline__ float sum_of(const float4 *red, int nt, int n, int l, int i) {
    const float *p = reinterpret_cast<const float *>(red + n * 32 + l) + i;
    float v = p[0];
#pragma unroll
    for (int w = 1; w < CONSUMERS; ++w) v += p[w * nt * 128];
    return v;
}

}  // namespace s16
}  // namespace moe
