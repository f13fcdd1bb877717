// decode16.cu -- the whole routed-experts layer of a decode batch (at most 32 tokens) with 16-bit weights in one
// kernel:
//   l = routerW x;  (e_s, w_s) = softmax and top-k of l;
//   out = sum_s w_s W_d[e_s] (SiLU(W_g[e_s] x) * (W_u[e_s] x))  [ + sigmoid(g . x) shared(x) ]  [ + residual ]
//
// The bytes of the experts that any token chose bound it (3 F D 2 bytes each, read once); what a chain of kernels
// adds are its launches, and at each of them memory that idles until the next one's loads arrive.  Here one CTA an SM
// runs through, with two grid barriers:
//   1. router: an expert's row at a time over the CTA's threads; barrier; every CTA routes all tokens for itself
//      (top-k of a few tokens costs less than a third barrier) and lists the touched experts;
//   2. gate and up: tiles of 8 gate and the same 8 up rows, the tiles of all touched experts dealt evenly;
//      h = w_s SiLU(gate) up, in fp32, to the workspace; barrier;
//   3. down: each CTA owns some output rows and walks all touched experts over them.  The routing weight is in h, so
//      one accumulator takes the products of every expert and no partial rows are combined afterwards: sums go
//      expert by expert (ascending; the shared one last), their order fixed.
// The ring (stream16.cuh) runs on through the second barrier: the first down tiles fly while it completes.
//
// h enters the tensor cores as two 16-bit columns, its rounded value and the rest: 16 significant bits in bf16, at
// least 22 in fp16, where a token's h is first scaled by the power of two that brings its largest to 2^14 .. 2^15
// (a fp16 h itself could overflow or vanish).
#include <algorithm>

#include "stream16.cuh"
#include "topk_token.cuh"

namespace moe {

namespace {

using namespace s16;

constexpr int KC = 1024;                     // columns of a stage at most
constexpr int H_CHUNKS = KC / (CONSUMERS * 32);  // 32-wide chunks a warp takes of a stage
constexpr size_t X_SMEM = 48 * 1024;         // activations are staged in shared memory up to this size

struct DecodeArgs {
    const void *x;
    int64_t x_stride;
    const float *routerW, *shexp_gate;
    const void *gate, *up, *down, *sh_gate, *sh_up, *sh_down;
    const void *residual;
    int64_t residual_stride, out_stride;
    void *out;
    int N, D, E, F, Fs, top_k, norm;
    float *logits;    // [N][E + 1]
    unsigned *amax;   // [32] largest |h| of a token (fp16)
    float *h;         // [entries][hs]
    int hs;
    unsigned *status, *bar_count, *bar_gen;
    unsigned long long barrier_ns;
    int extra_arrivals;  // failure-detection check: arrivals the first barrier waits for beyond the grid (0 normally)
    int kc, pitch, stages, x_pitch;  // x_pitch 0: the activations stay in global memory
    int x_at, red_at, list_at;       // places in shared memory
};

// Small arrays of a CTA, behind one another from `p` on.
struct Lists {
    unsigned *mask;  // [E] tokens that chose an expert
    int *pos;        // [E] its place in the list
    int *expert;     // [touched + 1] the touched experts, then E: the shared one
    int *first;      // [touched + 1] their first entry
    int *tok;        // [entries] token
    float *w;        // [entries] weight
    int *idx;        // [N][k] the routing
    float *topw;     // [N][k]
    __device__ Lists(char *p, int E, int N, int k, bool) {
        const int touched = min(E, N * k) + 1, entries = N * k + N;
        mask = reinterpret_cast<unsigned *>(p);
        pos = reinterpret_cast<int *>(mask + E);
        expert = pos + E;
        first = expert + touched;
        tok = first + touched;
        w = reinterpret_cast<float *>(tok + entries);
        idx = reinterpret_cast<int *>(w + entries);
        topw = reinterpret_cast<float *>(idx + N * k);
    }
};
size_t list_bytes(int E, int N, int k) {
    return ((size_t)2 * E + 2 * (std::min(E, N * k) + 1) + 2 * (N * k + N) + 2 * N * k) * 4;
}

// Grid barrier (a cooperative launch) of the first `threads` threads of every CTA, which share named barrier 1: an
// arrival counter and a generation word, both zero between calls.  False when the limit ran out.
__device__ bool grid_barrier(unsigned *count, unsigned *gen, unsigned arrivals, unsigned *status,
                             unsigned long long limit_ns, int *ok_s) {
    consumer_sync();
    if (threadIdx.x == 0) {
        *ok_s = 1;
        const unsigned g0 = *reinterpret_cast<volatile unsigned *>(gen);
        __threadfence();
        if (atomicAdd(count, 1u) == arrivals - 1) {
            *reinterpret_cast<volatile unsigned *>(count) = 0;
            __threadfence();
            atomicAdd(gen, 1u);
        } else {
            const unsigned long long t0 = tc::globaltimer();
            while (*reinterpret_cast<volatile unsigned *>(gen) == g0)
                if (tc::globaltimer() - t0 > limit_ns) {
                    atomicOr(status, MOE_DEV_TIMEOUT);
                    *ok_s = 0;
                    break;
                }
        }
        __threadfence();
    }
    consumer_sync();
    return *ok_s != 0;
}

// 8 values times `scale` as 16-bit values and the 16-bit values of what those leave (nothing of an infinity).
template <typename T>
__device__ __forceinline__ void split8(const float4 &a, const float4 &b, float scale, uint4 &hi, uint4 &lo) {
    const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) v[j] = std::is_same_v<T, __half> ? f[2 * i + j] * scale : f[2 * i + j];
        Pack<T, 2> p, q;
        p.set(v);
        float r[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            r[j] = v[j] - p.get(j);
            r[j] = fabsf(r[j]) <= fabsf(v[j]) ? r[j] : 0.0f;
        }
        q.set(r);
        h[i] = p.w[0];
        l[i] = q.w[0];
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// The power of two that brings a token's largest |h| (its bits) to 2^14 .. 2^15; 1 where there is none.
__device__ __forceinline__ float h_scale(unsigned amax, bool inverse) {
    const int e = (int)(amax >> 23);
    if (e == 0 || e >= 255) return 1.0f;
    const int p = min(14 + 127 - e, 126);
    return __uint_as_float((unsigned)(127 + (inverse ? -p : p)) << 23);
}

template <typename T, int NTM>
__global__ void __launch_bounds__(THREADS, 1) decode16_kernel(const DecodeArgs a) {
    extern __shared__ __align__(1024) char smem[];
    __shared__ __align__(8) unsigned long long bars[2 * MAX_STAGES + 1];
    __shared__ int abort_flag, ok_s, touched_s;
    __shared__ unsigned amax_s[MAX_ROWS];
    __shared__ float scale_s[MAX_ROWS], gate_s[MAX_ROWS];
    __shared__ float part[CONSUMERS][8];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int N = a.N, D = a.D, E = a.E, k = a.top_k, G = gridDim.x, bid = blockIdx.x;
    const bool consumer = warp < CONSUMERS;
    const T *x = static_cast<const T *>(a.x);
    Lists ls(smem + a.list_at, E, N, k, true);
    const uint32_t bar = tc::smem_u32(bars), xbar = bar + 2 * MAX_STAGES * 8;
    if (tid == 0) {
        abort_flag = 0;
        tc::mbar_init(xbar, 1);
        init_ring(bar, a.stages);
    }
    if (bid == 0 && tid < MAX_ROWS) a.amax[tid] = 0;
    if (tid < MAX_ROWS) amax_s[tid] = 0;
    for (int e = tid; e < E; e += THREADS) ls.mask[e] = 0;
    __syncthreads();

    // ---- router: an expert's row (or the shared gate's) at a time
    if (consumer) {
        const int rows = E + (a.shexp_gate != nullptr);
        for (int e = bid; e < rows; e += G) {
            const float *w = e < E ? a.routerW + (int64_t)e * D : a.shexp_gate;
            for (int t0 = 0; t0 < N; t0 += 8) {
                float acc[8] = {};
                for (int c = tid * 8; c < D; c += CONSUMERS * 256) {
                    const float4 w0 = *reinterpret_cast<const float4 *>(w + c), w1 = *reinterpret_cast<const float4 *>(w + c + 4);
                    const float wf[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (t0 + j < N) {
                            Pack<T, 8> p;
                            p.load(x + (t0 + j) * a.x_stride + c);
#pragma unroll
                            for (int i = 0; i < 8; ++i) acc[j] = fmaf(wf[i], p.get(i), acc[j]);
                        }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (t0 + j < N) acc[j] = warp_sum(acc[j]);
                if (lane == 0)
#pragma unroll
                    for (int j = 0; j < 8; ++j) part[warp][j] = acc[j];
                consumer_sync();
                if (tid < 8 && t0 + tid < N) {
                    float v = part[0][tid];
                    for (int i = 1; i < CONSUMERS; ++i) v += part[i][tid];
                    a.logits[(t0 + tid) * (E + 1) + e] = v;
                }
                consumer_sync();
            }
        }
        grid_barrier(a.bar_count, a.bar_gen, G + a.extra_arrivals, a.status, a.barrier_ns, &ok_s);
    } else if (a.x_pitch) {
        // the producer has no weights to ask for yet: it brings the activations in
        if (lane == 0) tc::mbar_expect_tx(xbar, (uint32_t)(N * D * 2));
        __syncwarp();
        if (lane < N) tc::bulk_load(tc::smem_u32(smem + a.x_at) + lane * a.x_pitch, x + lane * a.x_stride, D * 2, xbar);
        tc::mbar_wait(xbar, 0, &abort_flag, a.status, WAIT_NS);
    }
    __syncthreads();
    if (!ok_s) return;  // the barrier's limit ran out

    // ---- every CTA routes all tokens
    for (int t = warp; t < N; t += CONSUMERS + 1) {
        bool bad = false, some = false;
        auto logit = [&](int e) {  // a NaN or an infinity leaves the choice among the others and makes the weights NaN
            const float v = __ldcg(a.logits + t * (E + 1) + e);
            if (fabsf(v) <= 3e38f) {
                some = true;
                return v;
            }
            bad |= !(v < 0.0f);
            return v > 0.0f ? 3e38f : -3e38f;
        };
        auto sg = [&]() { return __ldcg(a.logits + t * (E + 1) + E); };
        float *scale = a.shexp_gate != nullptr ? gate_s : nullptr;
        if (E <= 64)
            route_token<2>(logit, sg, E, k, a.norm, t, lane, ls.idx, ls.topw, scale, nullptr);
        else if (E <= 256)
            route_token<8>(logit, sg, E, k, a.norm, t, lane, ls.idx, ls.topw, scale, nullptr);
        else
            route_token<32>(logit, sg, E, k, a.norm, t, lane, ls.idx, ls.topw, scale, nullptr);
        __syncwarp();
        if ((__any_sync(0xffffffffu, bad) || !__any_sync(0xffffffffu, some)) && lane < k) ls.topw[t * k + lane] = __uint_as_float(0x7fffffffu);
        if (lane == 0 && a.shexp_gate == nullptr) gate_s[t] = 1.0f;
    }
    __syncthreads();
    for (int i = tid; i < N * k; i += THREADS) atomicOr(&ls.mask[ls.idx[i]], 1u << (i / k));
    __syncthreads();
    if (warp == 0) {
        int n = 0, at = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const unsigned m = e0 + lane < E ? ls.mask[e0 + lane] : 0;
            const unsigned there = __ballot_sync(0xffffffffu, m != 0);
            int c = __popc(m), before = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o) before += v;
            }
            if (m != 0) {
                const int p = n + __popc(there & ((1u << lane) - 1));
                ls.expert[p] = e0 + lane;
                ls.first[p] = at + before - c;
                ls.pos[e0 + lane] = p;
            }
            n += __popc(there);
            at += __shfl_sync(0xffffffffu, before, 31);
        }
        if (lane == 0) {
            ls.expert[n] = E;
            ls.first[n] = N * k;
            touched_s = n;
        }
    }
    __syncthreads();
    for (int i = tid; i < N * k; i += THREADS) {
        const int t = i / k, e = ls.idx[i];
        const int at = ls.first[ls.pos[e]] + __popc(ls.mask[e] & ((1u << t) - 1));
        ls.tok[at] = t;
        ls.w[at] = ls.topw[i];
    }
    for (int t = tid; t < N; t += THREADS) {
        ls.tok[N * k + t] = t;
        ls.w[N * k + t] = gate_s[t];
    }
    __syncthreads();

    // ---- the CTA's share
    const int touched = touched_s, listed = touched + (a.Fs > 0);
    const unsigned all = N == 32 ? 0xffffffffu : (1u << N) - 1;
    const int upe = a.F / 8;                            // tiles of 8 pairs an expert
    const int64_t units = (int64_t)touched * upe + a.Fs / 8;
    const int u0 = (int)(units * bid / G), u1 = (int)(units * (bid + 1) / G);
    const int row0 = (int)((int64_t)D * bid / G), row1 = (int)((int64_t)D * (bid + 1) / G);
    const int row_tiles = (row1 - row0 + 15) / 16;
    Ring ring{smem, bar, a.stages, a.pitch, 0, 0, &abort_flag, a.status};

    if (!consumer) {
        int issued = 0;
        bool ok = true;
        for (int u = u0; u < u1 && ok; ++u) {
            const int i = min(u / upe, touched), e = ls.expert[i], r = (u - i * upe) * 8 + (lane & 7);
            const T *m = static_cast<const T *>(e == E ? (lane & 8 ? a.sh_up : a.sh_gate) : (lane & 8 ? a.up : a.gate));
            const T *src = m + ((int64_t)(e == E ? 0 : e) * a.F + r) * D;
            for (int k0 = 0; k0 < D && ok; k0 += a.kc) {
                ok = ring.produce(lane, lane < 16, 16, src + k0, (uint32_t)min(a.kc, D - k0) * 2);
                issued += ok;
            }
        }
        for (int rt = 0; rt < row_tiles && ok; ++rt) {
            const int r0 = row0 + (row1 - row0) * rt / row_tiles, r1 = row0 + (row1 - row0) * (rt + 1) / row_tiles;
            for (int i = 0; i < listed && ok; ++i) {
                const int e = ls.expert[i], K = e == E ? a.Fs : a.F;
                const T *src = static_cast<const T *>(e == E ? a.sh_down : a.down) +
                               ((int64_t)(e == E ? 0 : e) * D + r0 + min(lane, r1 - r0 - 1)) * K;
                for (int k0 = 0; k0 < K && ok; k0 += a.kc) {
                    ok = ring.produce(lane, lane < r1 - r0, r1 - r0, src + k0, (uint32_t)min(a.kc, K - k0) * 2);
                    issued += ok;
                }
            }
        }
        if (lane == 0 && *reinterpret_cast<volatile int *>(&abort_flag)) drain(bar, a.stages, issued);
        return;
    }

    // ---- gate and up
    if (a.x_pitch) tc::mbar_wait(xbar, 0, &abort_flag, a.status, WAIT_NS);
    const T *xb = a.x_pitch ? reinterpret_cast<const T *>(smem + a.x_at) : x;
    const int64_t xs = a.x_pitch ? a.x_pitch / 2 : a.x_stride;
    float4 *red = reinterpret_cast<float4 *>(smem + a.red_at);
    int buf = 0;
    auto sums = [&]() { return red + buf * CONSUMERS * NTM * 32; };
    for (int u = u0; u < u1; ++u) {
        const int i = min(u / upe, touched), r = (u - i * upe) * 8, first = ls.first[i];
        const int n = i == touched ? N : __popc(ls.mask[ls.expert[i]]), nt = (n + 7) / 8;
        const T *xp[NTM];
#pragma unroll
        for (int j = 0; j < NTM; ++j) xp[j] = xb + ls.tok[first + min(j * 8 + g, n - 1)] * xs + t4 * 8;
        float acc[NTM][4] = {};
        for (int k0 = 0; k0 < D; k0 += a.kc) {
            ring.wait_full();
            stage_products_nt<T, NTM>(ring, min(a.kc, D - k0), k0, nt, xp, acc, warp, lane);
            ring.release(lane);
            ring.next();
        }
        share_sums<NTM>(sums(), nt, acc, warp, lane);
        consumer_sync();
        for (int j = tid; j < nt * 64; j += CONSUMERS * 32) {
            const int tile = j >> 6, l = (j & 63) >> 1, odd = j & 1, c = tile * 8 + 2 * (l & 3) + odd;
            if (c >= n) continue;
            const float gate = sum_of(sums(), nt, tile, l, odd), up = sum_of(sums(), nt, tile, l, 2 + odd);
            const float h = __fdiv_rn(gate, 1.0f + expf(-gate)) * up * ls.w[first + c];
            a.h[(int64_t)(first + c) * a.hs + r + (l >> 2)] = h;
            if (std::is_same_v<T, __half>) atomicMax(&amax_s[ls.tok[first + c]], __float_as_uint(h) & 0x7fffffffu);
        }
        buf ^= 1;  // the next sums go elsewhere, those after them behind the next barrier
    }
    if (std::is_same_v<T, __half>) {
        consumer_sync();
        if (tid < N) atomicMax(a.amax + tid, amax_s[tid]);
    }
    if (!grid_barrier(a.bar_count, a.bar_gen, G, a.status, a.barrier_ns, &ok_s)) *reinterpret_cast<volatile int *>(&abort_flag) = 1;
    if (std::is_same_v<T, __half>) {
        if (tid < N) scale_s[tid] = h_scale(__ldcg(a.amax + tid), false);
        consumer_sync();
    }

    // ---- down
    const int nt = (N + 7) / 8;
    for (int rt = 0; rt < row_tiles; ++rt) {
        const int r0 = row0 + (row1 - row0) * rt / row_tiles, r1 = row0 + (row1 - row0) * (rt + 1) / row_tiles;
        float acc[NTM][4] = {};
        for (int i = 0; i < listed; ++i) {
            const int e = ls.expert[i], K = e == E ? a.Fs : a.F;
            const unsigned mask = e == E ? all : ls.mask[e];
            const float *hp[NTM];
            float scale[NTM];
            bool on[NTM];
#pragma unroll
            for (int j = 0; j < NTM; ++j) {
                const int t = j * 8 + g;
                on[j] = (mask >> t) & 1;
                hp[j] = a.h + (int64_t)(ls.first[i] + __popc(mask & ((1u << t) - 1))) * a.hs + t4 * 8;
                scale[j] = std::is_same_v<T, __half> && on[j] ? scale_s[t] : 1.0f;
            }
            for (int k0 = 0; k0 < K; k0 += a.kc) {
                const int cols = min(a.kc, K - k0);
                const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                float4 f[NTM == 1 ? H_CHUNKS : 1][2];
                if (NTM == 1)  // asked for before the wait
#pragma unroll
                    for (int q = 0; q < H_CHUNKS; ++q) {
                        const int c = (q * CONSUMERS + warp) * 32;
                        f[NTM == 1 ? q : 0][0] = f[NTM == 1 ? q : 0][1] = zero;
                        if (on[0] && c + t4 * 8 < cols) {
                            f[NTM == 1 ? q : 0][0] = __ldcg(reinterpret_cast<const float4 *>(hp[0] + k0 + c));
                            f[NTM == 1 ? q : 0][1] = __ldcg(reinterpret_cast<const float4 *>(hp[0] + k0 + c + 4));
                        }
                    }
                ring.wait_full();
                const char *w = ring.stage() + g * ring.pitch + t4 * 16;
#pragma unroll
                for (int q = 0; q < H_CHUNKS; ++q) {
                    const int c = (q * CONSUMERS + warp) * 32;
                    if (c >= cols) break;
                    const bool in = c + t4 * 8 < cols;
                    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
                    if (in) {
                        lo = *reinterpret_cast<const uint4 *>(w + c * 2);
                        hi = *reinterpret_cast<const uint4 *>(w + 8 * ring.pitch + c * 2);
                    }
#pragma unroll
                    for (int j = 0; j < NTM; ++j) {
                        if (NTM > 1 && !((mask >> (j * 8)) & 0xffu)) continue;
                        float4 f0 = zero, f1 = zero;
                        if (NTM == 1) {
                            f0 = f[NTM == 1 ? q : 0][0];
                            f1 = f[NTM == 1 ? q : 0][1];
                        } else if (on[j] && in) {
                            f0 = __ldcg(reinterpret_cast<const float4 *>(hp[j] + k0 + c));
                            f1 = __ldcg(reinterpret_cast<const float4 *>(hp[j] + k0 + c + 4));
                        }
                        uint4 bh, bl;
                        split8<T>(f0, f1, scale[j], bh, bl);
                        mma_chunk<T>(acc[j], lo, hi, bh);
                        mma_chunk<T>(acc[j], lo, hi, bl);
                    }
                }
                ring.release(lane);
                ring.next();
            }
        }
        share_sums<NTM>(sums(), nt, acc, warp, lane);
        consumer_sync();
        if (!*reinterpret_cast<volatile int *>(&abort_flag))
            for (int j = tid; j < nt * 128; j += CONSUMERS * 32) {
                const int row = j & 15, tile = j >> 7, c = (j >> 4) & 7, t = tile * 8 + c;
                if (r0 + row >= r1 || t >= N) continue;
                float v = sum_of(sums(), nt, tile, (row & 7) * 4 + (c >> 1), (row >> 3) * 2 + (c & 1));
                if (std::is_same_v<T, __half>) v *= h_scale(__ldcg(a.amax + t), true);
                if (a.residual != nullptr) {
                    Pack<T, 1> p;
                    p.load(static_cast<const T *>(a.residual) + t * a.residual_stride + r0 + row);
                    v += p.get(0);
                }
                static_cast<T *>(a.out)[t * a.out_stride + r0 + row] = elem_of<T>(v);
            }
        buf ^= 1;
    }
}

struct DecodeWs {
    size_t logits, amax, h, total;
    int hs;
};
DecodeWs decode_ws(int N, int E, int F, int top_k, int Fs) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    DecodeWs w;
    w.hs = std::max(F, Fs);
    w.logits = 256;
    w.amax = w.logits + up((size_t)N * (E + 1) * 4);
    w.h = w.amax + 256;
    w.total = w.h + up((size_t)(N * top_k + (Fs ? N : 0)) * w.hs * 4);
    return w;
}

}  // namespace

size_t decode16_ws_bytes(int N, int E, int F, int top_k, int Fs) { return decode_ws(N, E, F, top_k, Fs).total; }

int launch_decode16(const Decode16Call &c, void *ws, cudaStream_t s, unsigned long long barrier_ns, int extra_arrivals) {
    const DecodeWs L = decode_ws(c.N, c.E, c.F, c.top_k, c.Fs);
    DecodeArgs a{};
    a.x = c.x;
    a.x_stride = c.x_stride;
    a.routerW = c.routerW;
    a.shexp_gate = c.shexp_gate;
    a.gate = c.gate;
    a.up = c.up;
    a.down = c.down;
    a.sh_gate = c.sh_gate;
    a.sh_up = c.sh_up;
    a.sh_down = c.sh_down;
    a.residual = c.residual;
    a.residual_stride = c.residual_stride;
    a.out = c.out;
    a.out_stride = c.out_stride;
    a.N = c.N;
    a.D = c.D;
    a.E = c.E;
    a.F = c.F;
    a.Fs = c.Fs;
    a.top_k = c.top_k;
    a.norm = c.norm;
    a.logits = ws_ptr<float>(ws, L.logits);
    a.amax = ws_ptr<unsigned>(ws, L.amax);
    a.h = ws_ptr<float>(ws, L.h);
    a.hs = L.hs;
    a.status = ws_ptr<unsigned>(ws, 0);
    a.bar_count = ws_ptr<unsigned>(ws, BUCKET_BARRIER_OFFSET);
    a.bar_gen = ws_ptr<unsigned>(ws, BUCKET_BARRIER_OFFSET + 64);
    a.barrier_ns = barrier_ns ? barrier_ns : WAIT_NS;
    a.extra_arrivals = extra_arrivals;
    const int ntm = c.N <= 8 ? 1 : c.N <= 16 ? 2 : 4;
    a.kc = std::min(KC, (std::max({c.D, c.F, c.Fs}) + 31) / 32 * 32);
    a.pitch = pitch_of(a.kc);
    const size_t xb = (size_t)c.N * pitch_of(c.D);
    a.x_pitch = xb <= X_SMEM ? pitch_of(c.D) : 0;
    const size_t red = (size_t)2 * CONSUMERS * ntm * 512, lists = list_bytes(c.E, c.N, c.top_k);
    const size_t fixed = (a.x_pitch ? xb : 0) + red + lists, most = SMEM_LIMIT - 4096;
    a.stages = (int)std::min<size_t>(MAX_STAGES, (most - fixed) / ((size_t)16 * a.pitch));
    if (a.stages < 2) return MOE_ERR_UNSUPPORTED_SHAPE;
    a.x_at = (int)((size_t)a.stages * 16 * a.pitch);
    a.red_at = a.x_at + (int)(a.x_pitch ? xb : 0);
    a.list_at = a.red_at + (int)red;
    const size_t smem = a.list_at + lists;
    const int grid = std::max(1, device_sm_count());
    auto go = [&](auto kernel, SmemOptIn *done) {
        if (int rc = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), most, done)) return rc;
        void *args[] = {(void *)&a};
        return cuda_status(cudaLaunchCooperativeKernel(reinterpret_cast<const void *>(kernel), dim3(grid), dim3(THREADS), args, smem, s));
    };
    auto by_tiles = [&](auto *tp) {
        using T = std::remove_pointer_t<decltype(tp)>;
        static SmemOptIn done[3];
        if (ntm == 1) return go(decode16_kernel<T, 1>, &done[0]);
        return ntm == 2 ? go(decode16_kernel<T, 2>, &done[1]) : go(decode16_kernel<T, 4>, &done[2]);
    };
    return c.dtype == MOE_DTYPE_F16 ? by_tiles(static_cast<__half *>(nullptr)) : by_tiles(static_cast<__nv_bfloat16 *>(nullptr));
}

}  // namespace moe
