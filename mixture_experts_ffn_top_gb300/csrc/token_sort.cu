// token_sort.cu -- token rows sorted by expert and back, with the routing weights applied, and the
// gradients of both; the gradient of the routing weights to the router logits.
//
// The order is a stable counting sort of the N * top_k entries by expert: entry (t, s) of expert e
// lands at expStart[e] + the number of earlier entries of e.  Everything else is a function of the
// entries' rows (tokRow) alone, one token at a time:
//   sort     rows[tokRow[t,s]] = x[t]                    unsort   out[t] = sum_s w[t,s] rows[tokRow[t,s]]
//   d_x[t] = sum_s d_rows[tokRow[t,s]]                   d_rows[tokRow[t,s]] = w[t,s] d_out[t],
//                                                        d_w[t,s] = <d_out[t], rows[tokRow[t,s]]>
// so a token's row is read or written once and its top_k sorted rows once each: (1 + top_k) D values
// a token (1 + 2 top_k for the unsort's gradient), and a few operations a value: all are bound by HBM.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "elem.cuh"
#include "tc_glue.cuh"

namespace moe {

namespace {

constexpr int COUNT_THREADS = 512;
constexpr int ROW_WARPS = 8;      // warps per CTA of the router gradient, a token each
constexpr int ROW_THREADS = 256;  // threads per CTA of the row kernels

// ------------------------------------------------------------------ order --
// The tokens are split into ranges, one per CTA.  A range's first rows follow from the entries of each expert
// before it and in all: counted by every CTA itself where the entries are few (SORT_ONE_PASS), else taken from
// the table that sort_count_kernel leaves (summed over the ranges before by sort_scan_kernel where E is large).
constexpr int SORT_THREADS = 512;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_RANGES = 152;          // at most: a CTA per SM
constexpr int SORT_ONE_PASS = 4096;       // entries that every CTA counts by itself: 7.1 us, by the table 8.1
constexpr int SORT_SCAN_E = 256;          // experts from which the table is summed by a kernel of its own: 2048
                                          // tokens over 1024 experts 19 us, summed by every CTA 55
constexpr int SORT_RING = 12 * 1024;      // shared memory of a warp's rows in flight
constexpr int SORT_SMEM = 216 * 1024;      // a CTA's shared memory at most, beside its static 9 KB
constexpr int SORT_SLOTS = 4;             // at most this many of them
constexpr int SORT_POS = 2048;            // entries of a range whose rows wait in shared memory
constexpr unsigned long long SORT_WAIT_NS = 2000000000ull;

// f(i, idx[i]) for the entries lo .. hi - 1, four loads of a thread in flight.
template <int THREADS, typename F>
__device__ __forceinline__ void for_entries(const int32_t *__restrict__ idx, int lo, int hi, F f) {
    for (int i0 = lo + threadIdx.x; i0 < hi; i0 += 4 * THREADS) {
        int e[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) e[q] = i0 + q * THREADS < hi ? idx[i0 + q * THREADS] : -1;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (i0 + q * THREADS < hi) f(i0 + q * THREADS, e[q]);
    }
}

// Entries of each expert in token range blockIdx.x: table[range][e].
__global__ void __launch_bounds__(COUNT_THREADS)
sort_count_kernel(const int32_t *__restrict__ idx, int n_entries, int per_range, int E, int *__restrict__ table,
                  unsigned *__restrict__ status) {
    // the row kernel may be scheduled now (it waits for this grid before it reads the table)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ int hist[];
    for (int e = threadIdx.x; e < E; e += COUNT_THREADS) hist[e] = 0;
    __syncthreads();
    const int lo = blockIdx.x * per_range, hi = min(lo + per_range, n_entries);
    for_entries<COUNT_THREADS>(idx, lo, hi, [&](int, int e) {
        if (e >= 0 && e < E)
            atomicAdd(&hist[e], 1);
        else if (e != -1)
            atomicOr(status, MOE_DEV_BAD_ROUTING);
    });
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += COUNT_THREADS) table[(size_t)blockIdx.x * E + e] = hist[e];
}

// The table's columns summed exclusively over the ranges, in place; row n_ranges receives the totals.  A warp
// an expert: neighbouring lanes take neighbouring ranges.
__global__ void __launch_bounds__(COUNT_THREADS) sort_scan_kernel(int *table, int n_ranges, int E) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, e = blockIdx.x * (COUNT_THREADS / 32) + (threadIdx.x >> 5);
    if (e >= E) return;
    constexpr int STEPS = (SORT_RANGES + 31) / 32;
    int c[STEPS], run = 0;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) c[i] = i * 32 + lane < n_ranges ? table[(size_t)(i * 32 + lane) * E + e] : 0;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        int inc = c[i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (i * 32 + lane < n_ranges) table[(size_t)(i * 32 + lane) * E + e] = run + inc - c[i];
        run += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) table[(size_t)n_ranges * E + e] = run;
}

__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// How a range's counts are known.
enum SortCounts { COUNT_HERE, COUNT_TABLE, COUNT_SCANNED };

// Row of every entry of token range blockIdx.x and the CSR arrays.  BULK: the rows as well, in pieces through
// shared memory by bulk copies, one load and top_k stores each, the first loads issued before the order is
// known; a warp has `slots` pieces of at most `piece` bytes in flight.  The stores' bytes bound it past some
// 4 us for the order: 2048 x 2048 bf16, top 8 of 64, 17.0 us (76 MB: 66% of the copy rate), 16384 tokens
// 106.5 us (84%; rows that lie apart cost the writes some of it, a plain scatter of such rows with the order
// given takes 104 us).  Rows read by the sorted order instead measured 125 - 155 us there (x eight times
// from L2).  wait_ns: limit of a wait for a load; starve (failure-detection check, 0 normally): bytes that every
// load waits for beyond its own.
template <bool BULK, SortCounts COUNTS>
__global__ void __launch_bounds__(SORT_THREADS)
sort_rows_kernel(const char *__restrict__ x, int64_t x_stride, const int32_t *__restrict__ idx, int n_entries,
                 int tokens, int top_k, int E, int row_bytes, const int *table, int32_t *__restrict__ expStart,
                 int32_t *__restrict__ expTokI, int32_t *__restrict__ expTokK, int32_t *tokRow,
                 char *__restrict__ rows, int piece, int slots, int ring, unsigned long long wait_ns, int starve,
                 unsigned *__restrict__ status) {
    // the copying kernel, if there is one, may be scheduled now
    if (!BULK) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(128) char smem[];
    __shared__ int wsum[SORT_WARPS];
    __shared__ int kept_s, abort_s, pos_s[SORT_POS];
    __shared__ __align__(8) uint64_t bars[SORT_WARPS * SORT_SLOTS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int *before = reinterpret_cast<int *>(smem + (BULK ? SORT_WARPS * ring : 0));  // [E]
    int *rest = before + E;                                                       // [E]
    int *seen = rest + E;  // [warps][E]: entries of each expert in a warp's share of the range, then their first row
    const int N = n_entries / top_k, t0 = blockIdx.x * tokens, t1 = min(t0 + tokens, N);
    const int lo = t0 * top_k, hi = t1 * top_k;
    const int pieces = BULK ? (row_bytes + piece - 1) / piece : 1;
    // this warp's units: token t0 + (u / pieces) * SORT_WARPS + warp, piece u % pieces
    const int units = BULK ? (t1 - t0 > warp ? (t1 - t0 - warp + SORT_WARPS - 1) / SORT_WARPS : 0) * pieces : 0;
    auto unit_bytes = [&](int u) { return min(piece, row_bytes - (u % pieces) * piece); };
    auto load_unit = [&](int u) {
        const uint32_t bar = tc::smem_u32(&bars[warp * SORT_SLOTS + u % slots]);
        const int64_t t = t0 + (u / pieces) * SORT_WARPS + warp;
        const int bytes = unit_bytes(u);
        tc::mbar_expect_tx(bar, bytes + starve);
        tc::bulk_load(tc::smem_u32(smem + warp * ring + (u % slots) * piece),
                      x + t * x_stride + (int64_t)(u % pieces) * piece, bytes, bar);
    };
    if (BULK) {
        if (lane == 0) {
            for (int i = 0; i < slots; ++i) tc::mbar_init(tc::smem_u32(&bars[warp * SORT_SLOTS + i]), 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            for (int u = 0; u < min(units, slots); ++u) load_unit(u);
        }
        __syncwarp();
    }
    // a warp's share of the range: a multiple of 32 entries
    const int share = ((hi - lo + SORT_WARPS - 1) / SORT_WARPS + 31) / 32 * 32, shares = (hi - lo + share - 1) / share;
    const int my_lo = min(lo + warp * share, hi), my_hi = min(my_lo + share, hi);
    int *mine = seen + warp * E;
    // the entries' ranks, then rows: in shared memory, or where a range has too many in tokRow itself
    int *pos = hi - lo <= SORT_POS ? pos_s : tokRow + lo;
    if (tid == 0) abort_s = 0;
    for (int e = tid; e < (2 + shares) * E; e += SORT_THREADS) before[e] = 0;
    __syncthreads();
    // rank of each entry among the earlier ones of its expert in this warp's share, 32 at a time
    for (int i0 = my_lo; i0 < my_hi; i0 += 32) {
        const int i = i0 + lane;
        int e = i < my_hi ? idx[i] : -1;
        if (e < 0 || e >= E) e = -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        int r = -1;
        if (e >= 0) r = mine[e] + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
        if (i < my_hi) pos[i - lo] = r;
    }
    if (COUNTS == COUNT_HERE) {
        for_entries<SORT_THREADS>(idx, 0, n_entries, [&](int i, int e) {
            if (e >= 0 && e < E)
                atomicAdd(i < lo ? &before[e] : &rest[e], 1);
            else if (e != -1 && i >= lo && i < hi)
                atomicOr(status, MOE_DEV_BAD_ROUTING);
        });
    } else {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (COUNTS == COUNT_SCANNED) {
            for (int e = tid; e < E; e += SORT_THREADS) {
                const int a = table[(size_t)blockIdx.x * E + e];
                before[e] = a;
                rest[e] = table[(size_t)gridDim.x * E + e] - a;
            }
        } else {
            // a thread sums every `ways`-th range's count of its expert, 16 loads in flight
            const int ways = max(1, SORT_THREADS / E), n = gridDim.x;
            for (int j = tid; j < ways * E; j += SORT_THREADS) {
                const int e = j % E;
                int a = 0, b = 0;
                for (int g0 = j / E; g0 < n; g0 += 16 * ways) {
                    int c[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q) c[q] = g0 + q * ways < n ? table[(size_t)(g0 + q * ways) * E + e] : 0;
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        if (g0 + q * ways < (int)blockIdx.x)
                            a += c[q];
                        else
                            b += c[q];
                }
                atomicAdd(&before[e], a);
                atomicAdd(&rest[e], b);
            }
        }
    }
    __syncthreads();
    // exclusive scan of the totals (two experts a thread): each expert's first row, then each share's
    {
        const int e = 2 * tid;
        const int b0 = e < E ? before[e] : 0, b1 = e + 1 < E ? before[e + 1] : 0;
        const int c0 = e < E ? b0 + rest[e] : 0, c1 = e + 1 < E ? b1 + rest[e + 1] : 0;
        int inc = c0 + c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        int run = inc - c0 - c1, all = 0;
#pragma unroll
        for (int w = 0; w < SORT_WARPS; ++w) {
            if (w < warp) run += wsum[w];
            all += wsum[w];
        }
        if (blockIdx.x == 0) {
            if (e < E) expStart[e] = run;
            if (e + 1 < E) expStart[e + 1] = run + c0;
            if (tid == 0) expStart[E] = all;
        }
        if (tid == 0) kept_s = all;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (e + h >= E) break;
            int at = h ? run + c0 + b1 : run + b0;
            for (int w = 0; w < shares; ++w) {
                const int c = seen[w * E + e + h];
                seen[w * E + e + h] = at;
                at += c;
            }
        }
        __syncthreads();
    }
    for (int i = my_lo + lane; i < my_hi; i += 32) {
        int r = pos[i - lo];
        if (r >= 0) {
            r += mine[idx[i]];
            expTokI[r] = i / top_k;
            expTokK[r] = i % top_k;
        }
        tokRow[i] = r;
        pos[i - lo] = r;
    }
    // CSR entries past the last row: every range clears its own positions among them
    for (int i = max(lo, kept_s) + tid; i < hi; i += SORT_THREADS) {
        expTokI[i] = -1;
        expTokK[i] = -1;
    }
    if (BULK) {
        __syncthreads();
        int u = 0;
        for (; u < units; ++u) {
            const int slot = u % slots;
            const uint32_t bar = tc::smem_u32(&bars[warp * SORT_SLOTS + slot]);
            const int t = (u / pieces) * SORT_WARPS + warp;
            const int r = lane < top_k ? pos[t * top_k + lane] : -1;
            const bool here = tc::mbar_wait(bar, (u / slots) & 1, &abort_s, status, wait_ns);
            if (!__all_sync(0xffffffffu, here)) break;  // a copy that never came: flagged, its rows are left
            if (r >= 0)
                bulk_store(rows + (int64_t)r * row_bytes + (int64_t)(u % pieces) * piece,
                           tc::smem_u32(smem + warp * ring + slot * piece), unit_bytes(u));
            bulk_commit();
            if (u > 0 && u - 1 + slots < units) {  // the unit before has been read: its slot takes another
                bulk_wait_read<1>();
                __syncwarp();
                if (lane == 0) load_unit(u - 1 + slots);
            }
        }
        // after a timeout: the loads still in flight, with a limit again
        for (int p = u; p < min(units, u + slots - (u > 0)); ++p) {
            const uint64_t since = tc::globaltimer();
            while (!tc::mbar_try(tc::smem_u32(&bars[warp * SORT_SLOTS + p % slots]), (p / slots) & 1) &&
                   tc::globaltimer() - since < wait_ns) {
            }
        }
        bulk_wait_read<0>();
    }
}

// rows[tokRow[t,s]] = x[t] in accesses of B bytes, for rows that bulk copies cannot take (a length, stride or
// address that 16 bytes do not divide): threads as in unsort_kernel.  4096 x 1001 bf16, top 8: 30 us.
template <int B>
__global__ void __launch_bounds__(ROW_THREADS)
sort_copy_kernel(const char *__restrict__ x, int64_t x_stride, const int32_t *tokRow, int N, int top_k, int row_bytes,
                 int tpt_log2, char *__restrict__ rows) {
    using A = std::conditional_t<B == 8, uint2, std::conditional_t<B == 4, uint32_t, uint16_t>>;
    extern __shared__ int row_s[];  // [tokens of the CTA][top_k]
    const int tpt = 1 << tpt_log2, per = ROW_THREADS >> tpt_log2;
    const int64_t t0 = (int64_t)blockIdx.x * per;
    const int n = (int)min((int64_t)per, N - t0);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = threadIdx.x; i < n * top_k; i += ROW_THREADS) row_s[i] = tokRow[t0 * top_k + i];
    __syncthreads();
    const int mine = threadIdx.x >> tpt_log2;
    if (mine >= n) return;
    const char *src = x + (t0 + mine) * x_stride;
    constexpr int UNROLL = 4;
    const int64_t step = (int64_t)gridDim.y * tpt * B;
    for (int64_t c0 = ((int64_t)blockIdx.y * tpt + (threadIdx.x & (tpt - 1))) * B; c0 < row_bytes; c0 += UNROLL * step) {
        A v[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
            if (c0 + u * step < row_bytes) v[u] = *reinterpret_cast<const A *>(src + c0 + u * step);
        for (int s = 0; s < top_k; ++s) {
            const int r = row_s[mine * top_k + s];
            if (r < 0) continue;
            char *dst = rows + (int64_t)r * row_bytes + c0;
#pragma unroll
            for (int u = 0; u < UNROLL; ++u)
                if (c0 + u * step < row_bytes) *reinterpret_cast<A *>(dst + u * step) = v[u];
        }
    }
}

// ----------------------------------------------------------------- unsort --
// Sorted row of an entry, or -1 (a row outside [0, n_rows) is flagged and dropped).
__device__ __forceinline__ int checked_row(int r, int64_t n_rows, unsigned *status) {
    if (r >= 0 && r < n_rows) return r;
    if (r != -1) atomicOr(status, MOE_DEV_BAD_CSR);
    return -1;
}

// out[t] = sum over the slots of w * row (w == NULL: of the row), in slot order.  Threads 0 .. tpt - 1 of a
// token's group (tpt a power of two, ROW_THREADS / tpt tokens a CTA) own V consecutive columns each at a
// time; SLOTS rows are loaded before the first is used.  HBM-bound: 8192 x 2048 bf16, top 8, takes 47.8 us
// (302 MB: 6.3 TB/s, 93% of the copy rate), 4096 x 2048 fp32 46.8 us (95%).  The entries' rows and weights wait
// in shared memory: held in registers by every thread they cost 57 us (a third of the warps).
constexpr int SLOTS = 8;

template <typename T, int V>
__global__ void __launch_bounds__(ROW_THREADS, 4)
unsort_kernel(const T *__restrict__ rows, int64_t n_rows, const int32_t *__restrict__ tokRow,
              const float *__restrict__ w, int N, int top_k, int D, int tpt_log2, T *__restrict__ out,
              int64_t out_stride, unsigned *__restrict__ status) {
    extern __shared__ int2 entry[];  // [tokens of the CTA][top_k]: row (or -1), weight
    const int tpt = 1 << tpt_log2, per = ROW_THREADS >> tpt_log2;
    const int64_t t0 = (int64_t)blockIdx.x * per;
    const int tokens = (int)min((int64_t)per, N - t0);
    for (int i = threadIdx.x; i < tokens * top_k; i += ROW_THREADS)
        entry[i] = make_int2(checked_row(tokRow[t0 * top_k + i], n_rows, status),
                             __float_as_int(w != nullptr ? w[t0 * top_k + i] : 1.0f));
    __syncthreads();
    const int mine = threadIdx.x >> tpt_log2;
    if (mine >= tokens) return;
    const int2 *en = entry + mine * top_k;
    T *dst = out + (t0 + mine) * out_stride;
    for (int64_t c = ((int64_t)blockIdx.y * tpt + (threadIdx.x & (tpt - 1))) * V; c < D;
         c += (int64_t)gridDim.y * tpt * V) {
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
        for (int s0 = 0; s0 < top_k; s0 += SLOTS) {
            Pack<T, V> v[SLOTS];
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
                if (s0 + s < top_k && en[s0 + s].x >= 0) v[s].load_once(rows + (int64_t)en[s0 + s].x * D + c);
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
                if (s0 + s < top_k && en[s0 + s].x >= 0) {
                    const float ws = __int_as_float(en[s0 + s].y);
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] = __fmaf_rn(ws, v[s].get(i), acc[i]);
                }
        }
        Pack<T, V> o;
        o.set(acc);
        o.store(dst + c);
    }
}

// d_row = w * d_out and the dot d_w = <d_out, row> of one entry (t, s) at a time, by TPE threads: the rows are
// read and written once (read to be evicted first: d_out's row comes from the caches for all but its first entry),
// UNROLL accesses of each in flight.  The dot: each thread's columns in order, a butterfly over the warp, the warps
// in order.  HBM-bound: 2048 x 2048 bf16, top 8: 25.3 us (143 MB: 83% of the copy rate).  Streaming stores take 23.2,
// but leave less of d_rows in L2 for its reader: with the sort's gradient behind it 37.2 us against 35.1.  A token's
// threads holding all its entries at once took 35.8 us (registers, and a reduction of eight dots through shared
// memory).
template <typename T, int V, int TPE, int UNROLL>
__global__ void __launch_bounds__(ROW_THREADS)
unsort_grad_kernel(const T *__restrict__ d_out, int64_t d_out_stride, const T *__restrict__ rows, int64_t n_rows,
                   const int32_t *__restrict__ tokRow, const float *__restrict__ w, int n_entries, int top_k, int D,
                   T *__restrict__ d_rows, float *__restrict__ d_w, unsigned *__restrict__ status) {
    __shared__ float part[ROW_THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, me = threadIdx.x & (TPE - 1);
    const int64_t i = (int64_t)blockIdx.x * (ROW_THREADS / TPE) + threadIdx.x / TPE;
    const int r = i < n_entries ? checked_row(tokRow[i], n_rows, status) : -1;
    float dot = 0.0f;
    if (r >= 0) {
        const float ws = w[i];
        const T *src = d_out + (i / top_k) * d_out_stride, *row = rows + (int64_t)r * D;
        T *dst = d_rows + (int64_t)r * D;
        for (int c0 = me * V; c0 < D; c0 += UNROLL * TPE * V) {
            Pack<T, V> dv[UNROLL], rv[UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int c = c0 + u * TPE * V;
                if (c < D) {
                    rv[u].load_once(row + c);
                    dv[u].load(src + c);
                }
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int c = c0 + u * TPE * V;
                if (c < D) {
                    Pack<T, V> o;
                    float f[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        dot = __fmaf_rn(dv[u].get(j), rv[u].get(j), dot);
                        f[j] = __fmul_rn(ws, dv[u].get(j));
                    }
                    o.set(f);
                    o.store(dst + c);
                }
            }
        }
    }
#pragma unroll
    for (int o = (TPE < 32 ? TPE : 32) / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (TPE <= 32) {
        if (me == 0 && i < n_entries) d_w[i] = dot;
    } else {
        if (lane == 0) part[warp] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
#pragma unroll
            for (int k = 1; k < TPE / 32; ++k) dot += part[k];
            d_w[i] = dot;
        }
    }
}

// -------------------------------------------------------------- topk grad --
// TPT threads a token, the s-th on slot s: with p the softmax (over all experts, or over the selected ones) and
// c = sum_s p[idx_s] d_w_s,  d_l[e] = p[e] (v[e] - c), v[e] the sum of d_w over the slots of e: -p[e] c at every
// expert that no slot names (0 with norm, where the other logits are not even read), then the slots' own values
// over it.  VEC: four experts an access (E % 4 == 0, aligned).  EPL experts per thread (EPL * TPT >= E).
// Latency and launch bound at a router's sizes (2048 x 64 2.6 us); with many tokens the slots' rounds and the
// butterflies, the same for a warp's 32 / TPT tokens as for one, are what the instructions go to.  16384 x 256
// normalised 5.5 us (the logits and gradients of all experts once are 5.1 us of the copy rate; only the gradients and
// the slots' logits move), with 26% of the issue slots busy; over all experts 53%.
template <int EPL, bool VEC, int TPT>
__global__ void __launch_bounds__(ROW_WARPS * 32)
topk_grad_kernel(const float *__restrict__ logits, const int32_t *__restrict__ idx, const float *__restrict__ d_w,
                 int N, int E, int top_k, int norm, float *d_logits, unsigned *__restrict__ status) {
    constexpr int PER = 32 / TPT;
    const int lane = threadIdx.x & 31, me = lane & (TPT - 1);
    const unsigned mine = (TPT == 32 ? 0xffffffffu : (1u << (TPT & 31)) - 1u) << (lane & ~(TPT - 1));
    // the thread's i-th expert
    auto expert = [&](int i) { return VEC ? 4 * TPT * (i / 4) + 4 * me + i % 4 : TPT * i + me; };
    auto sum = [&](float v) {
#pragma unroll
        for (int o = TPT / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    for (int64_t t0 = ((int64_t)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5)) * PER; t0 < N;
         t0 += (int64_t)gridDim.x * ROW_WARPS * PER) {
        const int64_t t = t0 + lane / TPT;
        const int experts = t < N ? E : 0;  // the last warp's threads without a token go along with the others
        const float *lt = logits + t * E;
        float *dt = d_logits + t * E;
        int e = -1;
        float d = 0.0f, ls = -INFINITY;
        if (me < top_k && experts > 0) {
            e = idx[t * top_k + me];
            d = d_w[t * top_k + me];
            if (e < 0 || e >= E) {
                if (e != -1) atomicOr(status, MOE_DEV_BAD_ROUTING);
                e = -1;
                d = 0.0f;
            }
        }
        float p[EPL];
        if (!norm) {
#pragma unroll
            for (int i = 0; i < EPL; i += VEC ? 4 : 1) {
                if (VEC) {
                    float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                    if (expert(i) < experts) v = *reinterpret_cast<const float4 *>(lt + expert(i));
                    p[i] = v.x, p[(i + 1) % EPL] = v.y, p[(i + 2) % EPL] = v.z, p[(i + 3) % EPL] = v.w;
                } else {
                    p[i] = expert(i) < experts ? lt[expert(i)] : -INFINITY;
                }
            }
        }
        if (e >= 0) ls = lt[e];
        // the slots' sums of gradients by expert, and which slot is the first of its expert
        float v = 0.0f;
        bool first = e >= 0;
        for (int s = 0; s < top_k; ++s) {
            const int es = __shfl_sync(0xffffffffu, e, s, TPT);
            const float ds = __shfl_sync(0xffffffffu, d, s, TPT);
            if (es == e) {
                v += ds;
                first &= s >= me;
            }
        }
        float m = -INFINITY, z = 0.0f;
        bool nan = false;
        if (norm) {
            m = ls;
            nan = ls != ls;
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                m = fmaxf(m, p[i]);
                nan |= p[i] != p[i];
            }
        }
#pragma unroll
        for (int o = TPT / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        nan = (__ballot_sync(0xffffffffu, nan) & mine) != 0;
        const bool none = m == -INFINITY && !nan;  // nothing to take a softmax of
        float ps = e >= 0 && !none ? expf(ls - m) : 0.0f;
        if (norm) {
            z = first ? ps : 0.0f;
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                p[i] = expert(i) < E && !none ? expf(p[i] - m) : 0.0f;
                z += p[i];
            }
        }
        z = sum(z);  // by all of the warp, whose tokens may differ in `none`
        if (none) z = 1.0f;
        ps = __fdiv_rn(ps, z);
        const float c = sum(e >= 0 ? __fmul_rn(ps, d) : 0.0f);
        const float rest = __fdiv_rn(-c, z);  // of an expert without a slot, per exponential
#pragma unroll
        for (int i = 0; i < EPL; i += VEC ? 4 : 1) {
            if (expert(i) >= experts) continue;
            float o[4];
#pragma unroll
            for (int q = 0; q < (VEC ? 4 : 1); ++q) o[q] = norm || none ? 0.0f : __fmul_rn(p[(i + q) % EPL], rest);
            if (VEC)
                *reinterpret_cast<float4 *>(dt + expert(i)) = make_float4(o[0], o[1], o[2], o[3]);
            else
                dt[expert(i)] = o[0];
        }
        __syncwarp();  // the slots' values go over the others
        if (e >= 0) dt[e] = none ? 0.0f : __fmul_rn(ps, __fsub_rn(v, c));
    }
}

// Bytes per access: the largest of 16, 8, 4 and 2 that divides every address and row stride.
int access_bytes(std::initializer_list<const void *> ptrs, std::initializer_list<int64_t> stride_bytes) {
    uint64_t bits = 16;
    for (const void *p : ptrs) bits |= reinterpret_cast<uintptr_t>(p);
    for (int64_t st : stride_bytes) bits |= (uint64_t)st;
    return (int)(bits & -bits);
}

// Calls f with the elements per access as a constant.
template <typename T, typename F>
int by_width(int bytes, F f) {
    constexpr int E = sizeof(T);
    if (bytes >= 16) return f(std::integral_constant<int, 16 / E>());
    if (bytes >= 8) return f(std::integral_constant<int, 8 / E>());
    if (bytes >= 4) return f(std::integral_constant<int, 4 / E>());
    return f(std::integral_constant<int, 1>());
}

int log2_ceil(int64_t n, int most) {
    int l = 0;
    while (l < most && ((int64_t)1 << l) < n) ++l;
    return l;
}

// Calls f with a null pointer of the element type.
template <typename F>
int by_dtype(int dtype, F f) {
    switch (dtype) {
        case MOE_DTYPE_F32: return f(static_cast<float *>(nullptr));
        case MOE_DTYPE_F16: return f(static_cast<__half *>(nullptr));
        default: return f(static_cast<__nv_bfloat16 *>(nullptr));
    }
}

}  // namespace

int sort_ranges(int N, int *tokens) {
    // a number that does not depend on the device, so that the workspace's size is the shape's alone
    const int per = (N + SORT_RANGES - 1) / SORT_RANGES;
    if (tokens) *tokens = per;
    return (N + per - 1) / per;
}

// the ranges' counts and the totals
size_t sort_scratch_bytes(int N, int E) { return (size_t)(sort_ranges(N, nullptr) + 1) * E * 4; }

int launch_sort_tokens(const void *x, int64_t x_stride, int dtype, const int32_t *idx, int N, int top_k, int E, int D,
                       int32_t *expStart, int32_t *expTokI, int32_t *expTokK, int32_t *tokRow, void *rows, void *ws,
                       cudaStream_t s, unsigned long long starved_ns) {
    int tokens = 0;
    const int ranges = sort_ranges(N, &tokens);
    const int n = N * top_k;
    int *table = ws_ptr<int>(ws, SORT_SCRATCH_OFFSET);
    unsigned *status = static_cast<unsigned *>(ws);
    const int eb = (int)dtype_bytes(dtype), row_bytes = D * eb;
    const int64_t xb = x_stride * eb;
    const int width = access_bytes({x, rows}, {xb, row_bytes});
    const bool bulk = width == 16;
    if (starved_ns && !bulk) return MOE_ERR_UNSUPPORTED_SHAPE;  // no waits to check
    const unsigned long long wait_ns = starved_ns ? starved_ns : SORT_WAIT_NS;
    const int starve = starved_ns ? 16 : 0;
    // shared memory: the experts' counts, and the rest (at most SORT_RING a warp) for pieces of rows, as few as
    // the ring holds at two a warp, of equal size
    const int shares = std::min(SORT_WARPS, (tokens * top_k + 31) / 32);
    const int counts = (2 + shares) * E * 4;
    const int ring = std::min(SORT_RING, (SORT_SMEM - counts) / SORT_WARPS / 256 * 256);
    const int np = (row_bytes + ring / 2 - 1) / (ring / 2);
    const int piece = ((row_bytes + np - 1) / np + 15) / 16 * 16;
    const int slots = std::min(SORT_SLOTS, ring / piece);
    const size_t smem = (size_t)counts + (bulk ? SORT_WARPS * ring : 0);
    const int how = n <= SORT_ONE_PASS ? COUNT_HERE : E < SORT_SCAN_E ? COUNT_TABLE : COUNT_SCANNED;
    if (how != COUNT_HERE) {
        sort_count_kernel<<<ranges, COUNT_THREADS, (size_t)E * 4, s>>>(idx, n, tokens * top_k, E, table, status);
        int rc = launch_status();
        if (!rc && how == COUNT_SCANNED)
            rc = launch_early(sort_scan_kernel, dim3((E + COUNT_THREADS / 32 - 1) / (COUNT_THREADS / 32)),
                              dim3(COUNT_THREADS), 0, s, table, ranges, E);
        if (rc) return rc;
    }
    const char *xc = static_cast<const char *>(x);
    char *out = static_cast<char *>(rows);
    auto go = [&](auto kernel, SmemOptIn *done) {
        // one limit for every call, so that calls at once from two threads set the same
        int rc = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), SORT_SMEM, done);
        if (rc) return rc;
        if (how != COUNT_HERE)
            return launch_early(kernel, dim3(ranges), dim3(SORT_THREADS), smem, s, xc, xb, idx, n, tokens, top_k, E,
                                row_bytes, table, expStart, expTokI, expTokK, tokRow, out, piece, slots, ring, wait_ns,
                                starve, status);
        kernel<<<ranges, SORT_THREADS, smem, s>>>(xc, xb, idx, n, tokens, top_k, E, row_bytes, table, expStart, expTokI,
                                                  expTokK, tokRow, out, piece, slots, ring, wait_ns, starve, status);
        return launch_status();
    };
    auto by_counts = [&](auto bc) {
        constexpr bool B = decltype(bc)::value;
        static SmemOptIn d[3];
        if (how == COUNT_HERE) return go(sort_rows_kernel<B, COUNT_HERE>, &d[0]);
        if (how == COUNT_TABLE) return go(sort_rows_kernel<B, COUNT_TABLE>, &d[1]);
        return go(sort_rows_kernel<B, COUNT_SCANNED>, &d[2]);
    };
    if (bulk) return by_counts(std::true_type());
    const int rc = by_counts(std::false_type());
    if (rc) return rc;
    auto copy = [&](auto bc) {
        constexpr int B = decltype(bc)::value;
        const int64_t cols = row_bytes / B;
        const int tl = std::max(log2_ceil((cols + 3) / 4, 8), 3), per = ROW_THREADS >> tl;
        const int64_t cta_cols = (int64_t)4 << tl;
        const dim3 grid((unsigned)((N + per - 1) / per), (unsigned)std::min<int64_t>((cols + cta_cols - 1) / cta_cols, 65535));
        return launch_early(sort_copy_kernel<B>, grid, dim3(ROW_THREADS), (size_t)per * top_k * 4, s, xc, xb, tokRow, N,
                            top_k, row_bytes, tl, out);
    };
    switch (width) {
        case 8: return copy(std::integral_constant<int, 8>());
        case 4: return copy(std::integral_constant<int, 4>());
        default: return copy(std::integral_constant<int, 2>());
    }
}

int launch_unsort_tokens(const void *rows, int64_t n_rows, int dtype, const int32_t *tokRow, const float *w, int N,
                         int top_k, int D, void *out, int64_t out_stride, unsigned *status, cudaStream_t s) {
    const int sms = std::max(1, device_sm_count());
    return by_dtype(dtype, [&](auto *tp) {
        using T = std::remove_pointer_t<decltype(tp)>;
        const int b = access_bytes({rows, out}, {D * (int64_t)sizeof(T), out_stride * (int64_t)sizeof(T)});
        return by_width<T>(b, [&](auto v) {
            constexpr int V = decltype(v)::value;
            const int64_t cols = (D + V - 1) / V;
            // One access a thread until every SM has 2048 of them, then two, or four where they are narrow: 8192 x
            // 2048 bf16 at 16 bytes measured 49.8 / 47.8 / 49.2 us with 1 / 2 / 4, 13620 x 373 fp16 at 2 bytes
            // 45.9 / 39.1 / 35.0 us.
            const int64_t most = sizeof(T) * V == 16 ? 2 : 4;
            int64_t reps = 1;
            while (reps < most && N * cols / (2 * reps) >= (int64_t)sms * 2048) reps *= 2;
            const int tl = std::max(log2_ceil((cols + reps - 1) / reps, 8), 3);
            const int per = ROW_THREADS >> tl;
            const int64_t cta_cols = ((int64_t)1 << tl) * reps;
            const dim3 grid((unsigned)((N + per - 1) / per), (unsigned)std::min<int64_t>((cols + cta_cols - 1) / cta_cols, 65535));
            unsort_kernel<T, V><<<grid, ROW_THREADS, (size_t)per * top_k * sizeof(int2), s>>>(static_cast<const T *>(rows), n_rows, tokRow, w, N, top_k,
                                                             D, tl, static_cast<T *>(out), out_stride, status);
            return launch_status();
        });
    });
}

int launch_unsort_tokens_grad(const void *d_out, int64_t d_out_stride, const void *rows, int64_t n_rows, int dtype,
                              const int32_t *tokRow, const float *w, int N, int top_k, int D, void *d_rows, float *d_w,
                              unsigned *status, cudaStream_t s) {
    const int sms = std::max(1, device_sm_count());
    return by_dtype(dtype, [&](auto *tp) {
        using T = std::remove_pointer_t<decltype(tp)>;
        const int b = access_bytes({d_out, rows, d_rows}, {d_out_stride * (int64_t)sizeof(T), D * (int64_t)sizeof(T)});
        return by_width<T>(b, [&](auto v) {
            constexpr int V = decltype(v)::value;
            const int64_t cols = (D + V - 1) / V;
            const int64_t n = (int64_t)N * top_k;
            auto go = [&](auto kernel, int per) {
                kernel<<<(unsigned)((n + per - 1) / per), ROW_THREADS, 0, s>>>(
                    static_cast<const T *>(d_out), d_out_stride, static_cast<const T *>(rows), n_rows, tokRow, w,
                    (int)n, top_k, D, static_cast<T *>(d_rows), d_w, status);
                return launch_status();
            };
            // Eight threads an entry where its row is short, a CTA where the entries are few and their rows long, else
            // a warp.  Narrow accesses: more of them in flight (2048 x 1001 bf16 19.6 us with eight, 21.9 with four).
            constexpr int U = sizeof(T) * V == 16 ? 4 : 8;
            if (cols <= 32) return go(unsort_grad_kernel<T, V, 8, 4>, ROW_THREADS / 8);
            if (n < (int64_t)sms * 8 && cols > 64) return go(unsort_grad_kernel<T, V, ROW_THREADS, U>, 1);
            return go(unsort_grad_kernel<T, V, 32, U>, ROW_THREADS / 32);
        });
    });
}

int launch_topk_grad(const float *logits, const int32_t *idx, const float *d_w, int N, int E, int top_k, int norm,
                     float *d_logits, unsigned *status, cudaStream_t s) {
    auto go = [&](auto kernel, int tpt) {
        const int64_t per = ROW_WARPS * 32 / tpt, cap = (int64_t)std::max(1, device_sm_count()) * 8;
        kernel<<<(unsigned)std::max<int64_t>(1, std::min<int64_t>((N + per - 1) / per, cap)), ROW_WARPS * 32, 0, s>>>(
            logits, idx, d_w, N, E, top_k, norm, d_logits, status);
        return launch_status();
    };
    // Few threads a token share the issue slots best, more answer a small batch sooner (8, 16 and 32 threads:
    // 16384 x 64 3.9, 5.0 and 8.5 us, 16384 x 256 normalised 5.5, 6.9 and 8.1; 2048 x 128 3.2, 2.9 and 2.8).
    const bool many = N >= std::max(1, device_sm_count()) * 32;
    auto by_shape = [&](auto vec) {
        constexpr bool V = decltype(vec)::value;
        if (many && top_k <= 8 && E <= 256) {
            if (E <= 64) return go(topk_grad_kernel<8, V, 8>, 8);
            if (E <= 128) return go(topk_grad_kernel<16, V, 8>, 8);
            return go(topk_grad_kernel<32, V, 8>, 8);
        }
        if (top_k <= 16 && E <= 256) {
            if (E <= 64) return go(topk_grad_kernel<4, V, 16>, 16);
            if (E <= 128) return go(topk_grad_kernel<8, V, 16>, 16);
            return go(topk_grad_kernel<16, V, 16>, 16);
        }
        if (E <= 128) return go(topk_grad_kernel<4, V, 32>, 32);
        if (E <= 256) return go(topk_grad_kernel<8, V, 32>, 32);
        if (E <= 512) return go(topk_grad_kernel<16, V, 32>, 32);
        return go(topk_grad_kernel<32, V, 32>, 32);
    };
    if (E % 4 == 0 && access_bytes({logits, d_logits}, {}) == 16) return by_shape(std::true_type());
    return by_shape(std::false_type());
}

}  // namespace moe
