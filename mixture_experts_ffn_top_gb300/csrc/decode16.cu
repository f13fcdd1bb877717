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
//   2. gate and up: tiles of 8 gate and the same 8 up rows, the tiles of all touched experts dealt in turn;
//      h = w_s SiLU(gate) up, in fp32, to the workspace; barrier;
//   3. down: each CTA owns some output rows and walks all touched experts over them.  The routing weight is in h, so
//      one accumulator takes the products of every expert and no partial rows are combined afterwards.  Which of the two
//      groups of warps takes a stage hangs on expert and columns alone, and each walks its experts ascending, so that a
//      token's sum has the same order whatever the other tokens chose (see Part).
// The rings (stream16.cuh) run on through the second barrier: the first down tiles fly while it completes.
// bf16, 64 experts of 1024 x 2048, top 8: one token 31.8 us (floor 14.9), eight tokens 94.8 us (43 experts touched, 84%
// of the copy rate).  Of eight tokens' time 9 us pass until the first weights (router, barrier, routing, lists), gate and
// up take 61, the second barrier 4 to 7, down 27: what is left above the bytes are the 9 us in which no weights fly and
// the barrier's wait for the slowest CTA.  32 tokens over 128 experts of 768: at uniform choice (111 touched) 196 us, 79%;
// where some are ahead (26 touched) 104 us, 34%: 43 us of them are down, where every CTA reads all of h from L2 (120 MB
// beside 80 MB of weights) and a popular expert's 32 entries take eight tiles of instructions for one stage of weights.
//
// h enters the tensor cores as two 16-bit columns, its rounded value and the rest: 16 significant bits in bf16.  In fp16 a
// token's h is first scaled by the power of two that brings its largest to 2^14 .. 2^15 (a fp16 h itself could overflow or
// vanish): off by at most 2^-22 of itself, or by 2^-39 of the token's largest where that is more, 17 binades below it.
#include <algorithm>

#include "stream16.cuh"

namespace moe {

namespace {

using namespace s16;

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
    void *h;          // [entries][hs]: fp32 (fp16 weights), or per 8 values 8 rounded and 8 rests (bf16)
    int hs;
    unsigned *status;
    unsigned long long *arrived;
    unsigned long long barrier_ns;
    int extra_arrivals;  // failure-detection check: arrivals the first barrier waits for beyond the grid (0 normally)
    int kc, pitch, stages, x_pitch;  // x_pitch 0: the activations stay in global memory
    int odd_pieces;                  // an expert's down rows are an odd number of stages
    int x_at, red_at, list_at;       // places in shared memory
};

// Small arrays of a CTA, behind one another from `p` on.
struct Lists {
    unsigned *mask;  // [E] tokens that chose an expert
    int *expert;     // [touched + 1] the touched experts, of several tokens' the even ones first, then E: the shared one
    int *first;      // [touched + 1] their first entry
    int *tok;        // [entries] token
    float *w;        // [entries] weight
    int *idx;        // [N][k] the routing
    float *topw;     // [N][k]
    short *at;       // [touched + 1][8] the entry of each of up to 8 tokens, or -1
    int *pos;        // [E] an expert's first entry (more than 8 tokens)
    __device__ Lists(char *p, int E, int N, int k) {
        const int touched = min(E, N * k) + 1, entries = N * k + N;
        mask = reinterpret_cast<unsigned *>(p);
        expert = reinterpret_cast<int *>(mask + E);
        first = expert + touched;
        tok = first + touched;
        w = reinterpret_cast<float *>(tok + entries);
        idx = reinterpret_cast<int *>(w + entries);
        topw = reinterpret_cast<float *>(idx + N * k);
        at = reinterpret_cast<short *>(topw + N * k);
        pos = reinterpret_cast<int *>(topw + N * k);
    }
};
size_t list_bytes(int E, int N, int k) {
    const size_t touched = std::min(E, N * k) + 1;
    return (E + 2 * touched + 2 * (N * k + N) + 2 * N * k) * 4 + (N <= 8 ? touched * 16 : (size_t)E * 4);
}

// Grid barrier of the consumer warps (a cooperative launch).  Arrivals are counted through, never reset: a call makes
// two for each CTA, so the count is a multiple of that before every call.  False when the limit ran out, here or in
// another CTA: the count is of no use then (some CTAs leave without their second arrival), so its top bit is set, which
// lets every waiting CTA go at once and has later calls refused until the workspace is initialised anew.
constexpr unsigned long long GIVEN_UP = 1ull << 63;
__device__ bool grid_barrier(unsigned long long *arrived, unsigned long long target, unsigned *status,
                             unsigned long long limit_ns, int *ok_s) {
    consumer_sync();
    if (threadIdx.x == 0) {
        unsigned long long n;  // releases what the CTA's threads wrote before their barrier above
        asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], 1;" : "=l"(n) : "l"(arrived) : "memory");
        ++n;
        if (n < target) {
            const unsigned long long t0 = tc::globaltimer();
            for (unsigned it = 1;; ++it) {
                asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(n) : "l"(arrived) : "memory");
                if (n >= target) break;  // or given up
                if ((it & 31) == 0 && tc::globaltimer() - t0 > limit_ns) {
                    atomicOr(status, MOE_DEV_TIMEOUT);
                    atomicOr(arrived, GIVEN_UP);
                    n = GIVEN_UP;
                    break;
                }
            }
        }
        *ok_s = n < GIVEN_UP;
    }
    consumer_sync();
    return *ok_s != 0;
}

// A float's place in the order of floats (no NaN; both zeros alike), and back.
__device__ __forceinline__ unsigned order_of(float v) {
    const unsigned u = __float_as_uint(v + 0.0f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned o) { return __uint_as_float((o >> 31) ? o & 0x7fffffffu : ~o); }

// One token by one warp: softmax over all E logits, top-k by logit (ties to the lower expert), the selected
// probabilities (over their sum where norm).  idx, w [k] and the experts' masks in shared memory.  A NaN or infinite
// logit leaves the choice among the others and makes the weights NaN.
template <int EPL>
__device__ __forceinline__ void route(const float *logits, int E, int k, int norm, int t, int lane, int *idx, float *w,
                                      unsigned *mask) {
    unsigned key[EPL];
    float l[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = lane + 32 * i < E ? __ldcg(logits + lane + 32 * i) : 0.0f;
    bool bad = false, some = false;
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        key[i] = 0;
        if (lane + 32 * i < E) {
            const bool fine = fabsf(l[i]) <= 3e38f;
            some |= fine;
            bad |= !fine && !(l[i] < 0.0f);
            if (!fine) l[i] = l[i] > 0.0f ? 3e38f : -3e38f;
            key[i] = order_of(l[i]);
        }
        top = max(top, key[i]);
    }
    const float m = value_of(__reduce_max_sync(0xffffffffu, top));
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) z += lane + 32 * i < E ? expf(l[i] - m) : 0.0f;
    z = warp_sum(z);
    bad = __any_sync(0xffffffffu, bad) || !__any_sync(0xffffffffu, some);
    float sum = 0.0f, mine = 0.0f;
    for (int s = 0; s < k; ++s) {
        unsigned best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i] > best) best = key[i], at = i;
        const unsigned got = __reduce_max_sync(0xffffffffu, best);
        const unsigned e = __reduce_min_sync(0xffffffffu, best == got ? (unsigned)(lane + 32 * at) : 0xffffffffu);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if ((unsigned)(lane + 32 * i) == e) key[i] = 0;
        const float p = __fdiv_rn(expf(value_of(got) - m), z);
        sum += p;
        if (lane == s) mine = p;
        if (lane == 0) {
            idx[s] = (int)e;
            atomicOr(mask + e, 1u << t);
        }
    }
    if (lane < k) w[lane] = bad ? __uint_as_float(0x7fffffffu) : norm ? __fdiv_rn(mine, sum) : mine;
}

// What a group of warps takes of the down part, in stages of kc columns of a listed expert's rows.  Of experts of one
// stage the first group takes the even ones, the second the odd ones, which are listed behind them; of longer ones each
// takes every second stage.  The shared expert comes last, to the second group if it is one stage.  So which warps add up
// a stage hangs on its expert and columns alone.  Dealt to the groups in turn, as they come, a token's products would meet
// in another order with each batch; but the groups would have as many stages, which even and odd experts share evenly but
// for chance.  Six batches each, so and in turn: eight tokens of 64 experts 92.2 us and 90.4, five of 256 59.0 and 58.3,
// 32 of 128 at skewed choice 97.6 and 97.2, at uniform choice 196 both.  (One token has no others: each group takes half
// of its experts.)
struct Part {
    struct Stage {
        int i, k0;  // place in the list of experts, first column
    };
    int group, touched, even, F, Fs, kc;
    bool flip;  // experts of an odd number of stages: the odd ones' first goes to the second group
    int past;   // the group's routed experts are before this place
    int end;    // behind the place of its last stage
    __device__ __forceinline__ Part(int group, int touched, int even, int F, int Fs, int kc, bool flip)
        : group(group), touched(touched), even(min(even, touched)), F(F), Fs(Fs), kc(kc), flip(flip) {
        past = F <= kc && group == 0 ? this->even : touched;
        end = touched + (Fs > (group == 0 ? kc : 0));
    }
    __device__ __forceinline__ void settle(Stage &s) const {  // at the beginning of place i
        if (s.i >= past) s.i = max(s.i, touched);
        const int K = s.i >= touched ? Fs : F;
        s.k0 = K <= kc ? 0 : (group ^ (flip && s.i >= even && s.i < touched)) * kc;
    }
    __device__ __forceinline__ Stage begin() const {
        Stage s{F <= kc && group == 1 ? even : 0, 0};
        settle(s);
        return s;
    }
    __device__ __forceinline__ void next(Stage &s) const {
        if ((s.k0 += 2 * kc) < (s.i >= touched ? Fs : F)) return;
        ++s.i;
        settle(s);
    }
};
static_assert(GROUPS == 2);

// 8 values times `scale` as 16-bit values, and as 16-bit values what those leave.
template <typename T>
__device__ __forceinline__ void split8(const uint4 &a, const uint4 &b, float scale, uint4 &hi, uint4 &lo) {
    const uint32_t f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float v[2] = {__uint_as_float(f[2 * i]) * scale, __uint_as_float(f[2 * i + 1]) * scale};
        Pack<T, 2> p, q;
        p.set(v);
        const float r[2] = {v[0] - p.get(0), v[1] - p.get(1)};
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

// NTM: tiles of 8 tokens, rounded up to 1, 2 or 4.
template <typename T, int NTM>
__global__ void __launch_bounds__(THREADS, 1) decode16_kernel(const DecodeArgs a) {
    constexpr bool F16 = std::is_same_v<T, __half>, PACKED = NTM > 1;  // (see the down part)
    extern __shared__ __align__(1024) char smem[];
    __shared__ __align__(8) unsigned long long bars[GROUPS * 2 * MAX_STAGES + 1];
    __shared__ int abort_flag, ok_s, touched_s, even_s;
    __shared__ unsigned amax_s[MAX_ROWS];
    __shared__ float scale_s[MAX_ROWS], gate_s[MAX_ROWS];
    __shared__ float part[2][CONSUMERS][16];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int N = a.N, D = a.D, E = a.E, k = a.top_k, G = gridDim.x, bid = blockIdx.x;
    const bool consumer = warp < CONSUMERS;
    const int row0 = (int)((unsigned)D * bid / (unsigned)G), row1 = (int)((unsigned)D * (bid + 1) / (unsigned)G);
    const int row_tiles = (row1 - row0 + 15) / 16;
    const T *x = static_cast<const T *>(a.x);
    Lists ls(smem + a.list_at, E, N, k);
    const uint32_t bar = tc::smem_u32(bars), xbar = bar + GROUPS * 2 * MAX_STAGES * 8;
    unsigned long long arrivals = 0;  // of the calls before this one
    if (tid == 0) {
        abort_flag = 0;
        ok_s = 1;
        tc::mbar_init(xbar, 1);
        init_rings(bar, a.stages);
        arrivals = *reinterpret_cast<volatile unsigned long long *>(a.arrived);
        if (arrivals >= GIVEN_UP) {
            atomicOr(a.status, MOE_DEV_TIMEOUT);
            ok_s = 0;
        }
        arrivals -= arrivals % (2u * (unsigned)G);
    }
    if (bid == 0 && tid < MAX_ROWS) a.amax[tid] = 0;
    if (tid < MAX_ROWS) amax_s[tid] = 0;
    for (int e = tid; e < E; e += THREADS) ls.mask[e] = 0;
    __syncthreads();
    if (!ok_s) return;  // an earlier call gave up

    // ---- router: an expert's row (or the shared gate's) and 8 tokens at a time, 16 where 8 would take more rounds;
    // two rows where a CTA has two, so that both share the tokens' loads (one token 40 to 36 us).  Few rows: a CTA
    // takes some of the tokens instead of all (32 tokens, 32 rows of 4096 and as many experts of 512: 115 to 109 us).
    if (consumer) {
        const int rows = E + (a.shexp_gate != nullptr);
        auto router = [&](auto rc, auto tc_) {
            constexpr int ROWS = decltype(rc)::value, TOKENS = decltype(tc_)::value, V = ROWS * TOKENS;
            int buf = 0;
            const int token_groups = ROWS == 1 ? (N + TOKENS - 1) / TOKENS : 1;
            for (int u = bid; u < rows * token_groups; u += ROWS * G) {
                const int e = ROWS == 1 ? u % rows : u, first = u / rows * TOKENS, last = ROWS == 1 ? first + 1 : N;
                const float *w[ROWS];
#pragma unroll
                for (int i = 0; i < ROWS; ++i) {
                    const int ei = min(e + i * G, rows - 1);
                    w[i] = ei < E ? a.routerW + (int64_t)ei * D : a.shexp_gate;
                }
                for (int t0 = first; t0 < last; t0 += TOKENS) {
                    float acc[V] = {};
                    for (int c = tid * 4; c < D; c += CONSUMERS * 128) {
                        float4 u[ROWS];
                        Pack<T, 4> p[TOKENS];
#pragma unroll
                        for (int i = 0; i < ROWS; ++i) u[i] = *reinterpret_cast<const float4 *>(w[i] + c);
#pragma unroll
                        for (int j = 0; j < TOKENS; ++j) p[j].load(x + min(t0 + j, N - 1) * a.x_stride + c);
#pragma unroll
                        for (int j = 0; j < TOKENS; ++j)
#pragma unroll
                            for (int i = 0; i < ROWS; ++i) {
                                float &v = acc[i * TOKENS + j];
                                v = fmaf(u[i].w, p[j].get(3), fmaf(u[i].z, p[j].get(2), fmaf(u[i].y, p[j].get(1), fmaf(u[i].x, p[j].get(0), v))));
                            }
                    }
                    // V sums over the warp: at each step a lane keeps half of its values and sends the other half
#pragma unroll
                    for (int o = 16, n = V / 2; n > 0; o >>= 1, n >>= 1)
#pragma unroll
                        for (int j = 0; j < n; ++j) {
                            const bool up = lane & o;
                            const float send = up ? acc[j] : acc[j + n], keep = up ? acc[j + n] : acc[j];
                            acc[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                        }
#pragma unroll
                    for (int o = 16 / V; o > 0; o >>= 1) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
                    if (lane % (32 / V) == 0) part[buf][warp][lane / (32 / V)] = acc[0];
                    consumer_sync();
                    const int t = t0 + tid % TOKENS, row = e + tid / TOKENS * G;
                    if (tid < V && t < N && row < rows) {
                        float v = part[buf][0][tid];
#pragma unroll
                        for (int i = 1; i < CONSUMERS; ++i) v += part[buf][i][tid];
                        a.logits[t * (E + 1) + row] = v;
                    }
                    buf ^= 1;
                }
            }
        };
        using std::integral_constant;
        if (rows > G)
            router(integral_constant<int, 2>(), integral_constant<int, 8>());
        else if (NTM == 1 || rows * ((N + 7) / 8) <= G)
            router(integral_constant<int, 1>(), integral_constant<int, 8>());
        else
            router(integral_constant<int, 1>(), integral_constant<int, 16>());
        grid_barrier(a.arrived, arrivals + G + a.extra_arrivals, a.status, a.barrier_ns, &ok_s);
    } else if (a.x_pitch && warp == CONSUMERS) {
        // there are no weights to ask for yet: a producer brings the activations in
        if (lane == 0) tc::mbar_expect_tx(xbar, (uint32_t)(N * D * 2));
        __syncwarp();
        if (lane < N) tc::bulk_load(tc::smem_u32(smem + a.x_at) + lane * a.x_pitch, x + lane * a.x_stride, D * 2, xbar);
        tc::mbar_wait(xbar, 0, &abort_flag, a.status, WAIT_NS);
    }
    __syncthreads();
    if (!ok_s) return;  // the barrier's limit ran out

    // ---- every CTA routes all tokens
    for (int t = warp; t < N; t += CONSUMERS + GROUPS) {
        const float *l = a.logits + t * (E + 1);
        if (E <= 64)
            route<2>(l, E, k, a.norm, t, lane, ls.idx + t * k, ls.topw + t * k, ls.mask);
        else if (E <= 128)
            route<4>(l, E, k, a.norm, t, lane, ls.idx + t * k, ls.topw + t * k, ls.mask);
        else if (E <= 256)
            route<8>(l, E, k, a.norm, t, lane, ls.idx + t * k, ls.topw + t * k, ls.mask);
        else
            route<32>(l, E, k, a.norm, t, lane, ls.idx + t * k, ls.topw + t * k, ls.mask);
        if (lane == 0) gate_s[t] = a.shexp_gate != nullptr ? __fdiv_rn(1.0f, 1.0f + expf(-__ldcg(l + E))) : 1.0f;
    }
    __syncthreads();
    // ---- the touched experts and their entries, by expert (the even ones first), then token.  A thread lists its expert;
    // how many there are before it every warp counts for itself.
    const int groups = (E + 31) / 32;
    const unsigned evens = N == 1 ? 0xffffffffu : 0x55555555u;  // the lanes of the experts that come first
    const bool even = evens >> lane & 1;
    const int shift = even ? 0 : 16;
    for (int gr = warp; gr < groups; gr += CONSUMERS + GROUPS) {
        // entries of either part in 16 bits (at most 32 x 32)
        unsigned before = 0, all = 0;
        int listed_before = 0;
        for (int other = 0; other < groups; ++other) {
            const int e = other * 32 + lane;
            const unsigned m = e < E ? ls.mask[e] : 0, there = __ballot_sync(0xffffffffu, m != 0);
            const unsigned sum = __reduce_add_sync(0xffffffffu, (unsigned)__popc(m) << shift);
            if (other < gr) before += sum;
            all += sum;
            listed_before += __popc(there & (other < gr ? (even ? evens : 0xffffffffu) : even ? 0u : evens));
        }
        const int e = gr * 32 + lane;
        unsigned m = e < E ? ls.mask[e] : 0;
        const unsigned alike = (even ? evens : ~evens) & ((1u << lane) - 1);  // the lanes before this one in its part
        const int n = listed_before + __popc(__ballot_sync(0xffffffffu, m != 0) & alike), c = __popc(m);
        unsigned in = (unsigned)c << shift;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned v = __shfl_up_sync(0xffffffffu, in, o);
            if (lane >= o) in += v;
        }
        in += before;
        if (m != 0) {
            int at = (int)(in >> shift & 0xffff) - c + (even ? 0 : (int)(all & 0xffff));
            ls.expert[n] = e;
            ls.first[n] = at;
            if (PACKED) {
                ls.pos[e] = at;
            } else {
                for (int t = 0; t < 8; ++t) ls.at[n * 8 + t] = -1;
                for (; m != 0; m &= m - 1, ++at) {
                    const int t = __ffs(m) - 1;
                    int s = 0;
                    while (ls.idx[t * k + s] != e) ++s;  // an expert in a token's mask is among its choices
                    ls.tok[at] = t;
                    ls.w[at] = ls.topw[t * k + s];
                    ls.at[n * 8 + t] = (short)at;
                }
            }
        }
    }
    if (warp == CONSUMERS + GROUPS - 1) {  // the shared expert, behind them
        int listed_before = 0, first_part = 0;
        for (int gr = 0; gr < groups; ++gr) {
            const int e = gr * 32 + lane;
            const unsigned there = __ballot_sync(0xffffffffu, e < E && ls.mask[e] != 0);
            listed_before += __popc(there);
            first_part += __popc(there & evens);
        }
        if (lane == 0) {
            ls.expert[listed_before] = E;
            ls.first[listed_before] = N * k;
            touched_s = listed_before;
            even_s = first_part;
        }
        if (lane < N) {
            ls.tok[N * k + lane] = lane;
            ls.w[N * k + lane] = gate_s[lane];
        }
        if (!PACKED && lane < 8) ls.at[listed_before * 8 + lane] = lane < N ? (short)(N * k + lane) : (short)-1;
    }
    __syncthreads();
    if (PACKED) {
        for (int i = tid; i < N * k; i += THREADS) {
            const int t = i / k, e = ls.idx[i], at = ls.pos[e] + __popc(ls.mask[e] & ((1u << t) - 1));
            ls.tok[at] = t;
            ls.w[at] = ls.topw[i];
        }
        __syncthreads();
    }

    // ---- the CTA's share
    const int touched = touched_s, listed = touched + (a.Fs > 0);
    const int upe = a.F / 8;  // tiles of 8 pairs an expert
    const int units = touched * upe + a.Fs / 8;
    const int group = consumer ? warp / GROUP_WARPS : warp - CONSUMERS;
    Ring ring(smem, bar, group, a.stages, a.pitch, &abort_flag, a.status);
    auto part_of_down = [&]() { return Part(group, touched, N == 1 ? (listed + 1) / 2 : even_s, a.F, a.Fs, a.kc, a.odd_pieces); };

    if (!consumer) {  // the group's producer
        const Layout lay(D);
        int issued = 0;
        bool ok = true;
        for (int u = first_unit(group); u < units && ok; u += unit_stride()) {
            const int i = min(u / upe, touched), e = ls.expert[i], r = (u - i * upe) * 8;
            const int64_t from = ((int64_t)(e == E ? 0 : e) * a.F + r) * D;
            const T *gate = static_cast<const T *>(e == E ? a.sh_gate : a.gate) + from;
            const T *up = static_cast<const T *>(e == E ? a.sh_up : a.up) + from;
            for (int k0 = 0; k0 < D && ok; k0 += a.kc) {
                ok = ring.produce(lane, lay, D, min(a.kc, D - k0), gate + k0, 8, up + k0, 8);
                issued += ok;
            }
        }
        const Part share = part_of_down();
        for (int rt = 0; rt < row_tiles && ok; ++rt) {
            const int r0 = row0 + (row1 - row0) * rt / row_tiles, r1 = row0 + (row1 - row0) * (rt + 1) / row_tiles;
            for (Part::Stage at = share.begin(); at.i < share.end && ok; share.next(at)) {
                const int e = ls.expert[at.i], K = e == E ? a.Fs : a.F, n = r1 - r0;
                const T *src = static_cast<const T *>(e == E ? a.sh_down : a.down) + ((int64_t)(e == E ? 0 : e) * D + r0) * K + at.k0;
                ok = ring.produce(lane, Layout(K), K, min(a.kc, K - at.k0), src, min(n, 8), src + (int64_t)8 * K, n - min(n, 8));
                issued += ok;
            }
        }
        if (lane == 0 && *reinterpret_cast<volatile int *>(&abort_flag)) drain(ring.bar, a.stages, issued);
        return;
    }

    // ---- gate and up
    if (a.x_pitch) tc::mbar_wait(xbar, 0, &abort_flag, a.status, WAIT_NS);
    const T *xb = a.x_pitch ? reinterpret_cast<const T *>(smem + a.x_at) : x;
    const int64_t xs = a.x_pitch ? a.x_pitch / 2 : a.x_stride;
    float4 *red = reinterpret_cast<float4 *>(smem + a.red_at);
    auto info = [&](int u) {
        const int i = min(u / upe, touched);
        return make_int2(ls.first[i], i == touched ? N : ls.first[i + 1] - ls.first[i]);
    };
    auto at = [&](int entry) { return xb + ls.tok[entry] * xs; };
    auto done = [&](int u, const int2 &in, const float4 *s, int nt, int thread) {
        const int r = (u - min(u / upe, touched) * upe) * 8;
        // a pair of threads a value: one adds up gate, the other up
        for (int j = thread; j < nt * 128; j += GROUP_WARPS * 32) {
            const int is_up = j & 1, row = (j >> 1) & 7, c = j >> 4, l = lane_of_row(row) * 4 + ((c & 7) >> 1);
            const float v = sum_of(s, nt, c >> 3, l, 2 * is_up + (c & 1));
            const float up = __shfl_xor_sync(0xffffffffu, v, 1);
            if (c >= in.y || is_up) continue;
            const float h = __fdiv_rn(v, 1.0f + expf(-v)) * up * ls.w[in.x + c];
            const int64_t to = (int64_t)(in.x + c) * a.hs + r;
            if (F16) {
                static_cast<float *>(a.h)[to + row] = h;
                atomicMax(&amax_s[ls.tok[in.x + c]], __float_as_uint(h) & 0x7fffffffu);
            } else {
                const T hi = elem_of<T>(h);
                T *p = static_cast<T *>(a.h) + to * 2 + row;
                p[0] = hi;
                p[8] = elem_of<T>(h - (float)hi);
            }
        }
    };
    stream_units<T, NTM>(ring, units, D, a.kc, red, warp, lane, info, at, done);
    if (F16) {
        consumer_sync();
        if (tid < N) atomicMax(a.amax + tid, amax_s[tid]);
    }
    if (!grid_barrier(a.arrived, arrivals + 2 * G, a.status, a.barrier_ns, &ok_s)) *reinterpret_cast<volatile int *>(&abort_flag) = 1;
    if (F16) {
        if (tid < N) scale_s[tid] = h_scale(__ldcg(a.amax + tid), false);
        consumer_sync();
    }

    // ---- down.  Up to 8 tokens: a token's column is its own throughout, rounded h and rests one after the other, the
    // accumulators run on over the experts.  More (PACKED): the columns are up to 4 of an expert's entries, rounded,
    // and the same entries' rests, and the sums are added to the warp's rows x tokens in shared memory (most experts
    // have a handful: one tile instead of eight that are all but empty).
    const int gw = warp % GROUP_WARPS, own_pitch = N + 1;
    float *own = reinterpret_cast<float *>(red) + warp * 16 * own_pitch;  // PACKED: [16][own_pitch] of the warp
    const uint4 zero = make_uint4(0, 0, 0, 0);
    auto length = [&](int i) { return i == touched ? a.Fs : a.F; };
    auto count = [&](int i) { return i == touched ? N : ls.first[i + 1] - ls.first[i]; };
    // the lane's h of a tile: 8 values of its column's entry (-1: none), CHUNKS times: fp32, or rounded and rests (a
    // packed tile's lane needs one of them)
    constexpr bool BOTH = F16 || !PACKED;
    struct Block {
        uint4 a[CHUNKS], b[BOTH ? CHUNKS : 1];
        float scale;
    };
    auto load = [&](int entry, int k0, int cols, Block &f) {
        if (F16) f.scale = entry >= 0 ? scale_s[ls.tok[entry]] : 1.0f;
        const char *h = static_cast<const char *>(a.h) + ((int64_t)entry * a.hs + k0 + t4 * 8) * 4 + (BOTH ? 0 : (g >> 2) * 16);
#pragma unroll
        for (int q = 0; q < CHUNKS; ++q) {
            const int c = (q * GROUP_WARPS + gw) * 32;
            const bool in = entry >= 0 && c + t4 * 8 < cols;
            f.a[q] = in ? __ldcg(reinterpret_cast<const uint4 *>(h + c * 4)) : zero;
            if constexpr (BOTH) f.b[q] = in ? __ldcg(reinterpret_cast<const uint4 *>(h + c * 4 + 16)) : zero;
        }
    };
    auto products = [&](const Layout &lay, int cols, const Block &f, float (&acc)[4], float (&rest_acc)[4]) {
        const char *w = ring.stage() + lay.lane_at(g) + t4 * 16;
#pragma unroll
        for (int q = 0; q < CHUNKS; ++q) {
            const int c = (q * GROUP_WARPS + gw) * 32;
            if (c >= cols) break;
            uint4 lo = zero, hi = zero, b = f.a[q];
            if (c + t4 * 8 < cols) {
                lo = *reinterpret_cast<const uint4 *>(w + c * 2);
                hi = *reinterpret_cast<const uint4 *>(w + 2 * lay.four + c * 2);
            }
            uint4 rest = f.b[BOTH ? q : 0];
            if constexpr (F16) split8<T>(f.a[q], f.b[q], f.scale, b, rest);
            if (F16 && PACKED && g >= 4) b = rest;
            mma_chunk<T>(acc, lo, hi, b);
            if (!PACKED) mma_chunk<T>(rest_acc, lo, hi, rest);
        }
    };
    const Part share = part_of_down();
    for (int rt = 0; rt < row_tiles; ++rt) {
        const int r0 = row0 + (row1 - row0) * rt / row_tiles, r1 = row0 + (row1 - row0) * (rt + 1) / row_tiles;
        consumer_sync();  // the sums before these have been read
        if (PACKED) {
            for (int j = lane; j < 16 * own_pitch; j += 32) own[j] = 0.0f;
            __syncwarp();
        }
        struct Place : Part::Stage {
            int j;  // tile of entries
        };
        auto next_stage = [&](Place &p) {
            share.next(p);
            p.j = 0;
        };
        Place at{share.begin(), 0};
        if constexpr (!PACKED) {
            float one[1][4] = {};
            Block f;
            auto fetch = [&](const Place &p) { load(ls.at[p.i * 8 + g], p.k0, min(a.kc, length(p.i) - p.k0), f); };
            if (at.i < share.end) fetch(at);
            while (at.i < share.end) {
                const int K = length(at.i), cols = min(a.kc, K - at.k0);
                // a column without an entry stays out: 0 times a weight that is not finite
                const short2 there = *reinterpret_cast<const short2 *>(ls.at + at.i * 8 + 2 * t4);
                next_stage(at);
                ring.wait_full();
                float acc[4] = {}, rests[4] = {};
                products(Layout(K), cols, f, acc, rests);
                if (at.i < share.end) fetch(at);  // the next stage's, while the other group works
                ring.release(lane);
                ring.next();
#pragma unroll
                for (int q = 0; q < 4; ++q) one[0][q] += (q & 1 ? there.y : there.x) >= 0 ? acc[q] + rests[q] : 0.0f;
            }
            share_sums<1>(red, 1, one, warp, lane);
        } else {
            float acc[4] = {};
            Place ahead = at;
            auto fetch = [&](Block &f) {  // and on to the tile behind it
                if (ahead.i >= share.end) return;
                const int n = count(ahead.i), e = ahead.j * 4 + (g & 3);
                load(e < n ? ls.first[ahead.i] + e : -1, ahead.k0, min(a.kc, length(ahead.i) - ahead.k0), f);
                if (++ahead.j * 4 >= n) next_stage(ahead);
            };
            // one tile; false behind the last
            auto step = [&](const Block &now, Block &then) {
                const int K = length(at.i), n = count(at.i), first = ls.first[at.i];
                const bool last = (at.j + 1) * 4 >= n;
                fetch(then);
                if (at.j == 0) ring.wait_full();
                products(Layout(K), min(a.kc, K - at.k0), now, acc, acc);
                if (last) {
                    ring.release(lane);
                    ring.next();
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float v = acc[q] + __shfl_xor_sync(0xffffffffu, acc[q], 2);  // the rests' column
                    const int c = at.j * 4 + 2 * t4 + (q & 1);
                    if (t4 < 2 && c < n) own[(g + 8 * (q >> 1)) * own_pitch + ls.tok[first + c]] += v;
                    acc[q] = 0.0f;
                }
                __syncwarp();
                if (last)
                    next_stage(at);
                else
                    ++at.j;
                return at.i < share.end;
            };
            if (at.i < share.end) {
                Block b0, b1, b2;
                fetch(b0);
                if constexpr (F16) {  // twice the registers: a tile ahead
                    while (step(b0, b1) && step(b1, b0)) {}
                } else {
                    fetch(b1);
                    while (step(b0, b2) && step(b1, b0) && step(b2, b1)) {}
                }
            }
        }
        consumer_sync();
        if (!*reinterpret_cast<volatile int *>(&abort_flag))
            for (int j = tid; j < N * 16; j += CONSUMERS * 32) {
                const int row = j & 15, t = j >> 4, of = lane_of_row(row & 7) + (row & 8);  // the products' row
                if (r0 + row >= r1) continue;
                float v;
                if (PACKED) {
                    const float *p = reinterpret_cast<const float *>(red) + of * own_pitch + t;
                    v = p[0];
#pragma unroll
                    for (int i = 1; i < CONSUMERS; ++i) v += p[i * 16 * own_pitch];
                } else {
                    v = sum_of<CONSUMERS>(red, 1, 0, (of & 7) * 4 + (t >> 1), (of >> 3) * 2 + (t & 1));
                }
                if (F16) v *= h_scale(__ldcg(a.amax + t), true);
                if (a.residual != nullptr) {
                    Pack<T, 1> p;
                    p.load(static_cast<const T *>(a.residual) + t * a.residual_stride + r0 + row);
                    v += p.get(0);
                }
                static_cast<T *>(a.out)[t * a.out_stride + r0 + row] = elem_of<T>(v);
            }
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
    a.h = ws_ptr<void>(ws, L.h);
    a.hs = L.hs;
    a.status = ws_ptr<unsigned>(ws, 0);
    a.arrived = ws_ptr<unsigned long long>(ws, DECODE_ARRIVALS_OFFSET);
    a.barrier_ns = barrier_ns ? barrier_ns : WAIT_NS;
    a.extra_arrivals = extra_arrivals;
    const int ntm = c.N <= 8 ? 1 : c.N <= 16 ? 2 : 4;
    a.kc = std::min(KC, (std::max({c.D, c.F, c.Fs}) + 31) / 32 * 32);
    a.pitch = pitch_of(a.kc);
    a.odd_pieces = (c.F + a.kc - 1) / a.kc % 2;
    // the warps' sums, or each warp's rows x tokens
    const size_t red = std::max((size_t)CONSUMERS * 512 * ntm, (size_t)CONSUMERS * 64 * (c.N + 1));
    const size_t ring = (size_t)GROUPS * 16 * a.pitch, lists = list_bytes(c.E, c.N, c.top_k), most = SMEM_LIMIT - 5120;
    a.stages = (int)std::min<size_t>(MAX_STAGES, (most - red - lists) / ring);
    if (a.stages < 2) return MOE_ERR_UNSUPPORTED_SHAPE;
    // the activations are staged where there is room beside the rings
    const size_t xb = (size_t)c.N * pitch_of(c.D);
    a.x_pitch = a.stages * ring + red + lists + xb <= most ? pitch_of(c.D) : 0;
    a.x_at = (int)(a.stages * ring);
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
