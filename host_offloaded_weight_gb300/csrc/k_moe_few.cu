// A whole mixture-of-experts layer for a few tokens, in two kernels:
//
//   up     h[i] = SiLU(G_e x_t) * (U_e x_t)   for every routed pair i = (t, e)
//   down   out[t] = r[t] + sum_j w[t,j] D_e h[i],  w = softmax over the token's k largest logits
//
// Experts in bf16 or MXFP4. The bound is the bytes of the experts that are routed: each is read
// once (for up to 8 of its tokens), and nothing else of that size is touched.
//
// The weights are the left operand of tcgen05.mma (128 rows a tile) and the tokens the right one: 16
// or 32 columns, which are 8 tokens as bf16 (and columns that nobody reads), or, with MXFP4 experts,
// as E4M3 terms with a power of two for each block of 32 (see k_gemm_mx.cu): two for x, which
// holds a bf16's 8 bits, and three for h, 12 bits. So the weights go from memory to the tensor core as they
// are, with no instruction spent on a value, and a product (about 60 clocks for 4 KB of the stage)
// stays under the memory's time. A tile takes 64 gate rows and the 64 up rows of the same columns of h.
//
// Routing is done by every CTA of both kernels for itself (a warp a token): that costs less than a
// launch, and lets the down kernel request its first weights while the up kernel runs.
//
// Both kernels: warp 0 loads the weights by TMA into a ring of stages, warps 2-9 take turns at
// the stages and add the block scales and (up) the tokens' rows, warp 1 issues the products,
// warps 10-13 write the results. Down: a cluster has 128 output rows; its CTAs share the experts,
// keep the weighted sums [token][row] in shared memory and add one another's in CTA order. The
// same bits every time, and no atomics on data.
#include <algorithm>

#include "kernels.h"
#include "tc.cuh"

namespace ls {
namespace {

using namespace tc;

constexpr int MAX_T = 64, MAX_K = 8, MAX_E = 256;
constexpr int MAX_ROWS = MAX_T * MAX_K;
constexpr int TOK = 8;            // tokens of an expert that one pass over its weights serves
constexpr int TILE = 128;         // weight rows of a tile
constexpr int UP_F = TILE / 2;    // columns of h of a tile of the up kernel
constexpr int P_BYTES = TILE * 128;
constexpr int H_TERMS = 3;        // E4M3 terms of h (MXFP4 experts)

template <bool MX, bool UP>
struct Cfg {
    static constexpr int TERMS = !MX ? 1 : UP ? 2 : H_TERMS;
    static constexpr int BQ = TERMS <= 2 ? 16 : 32;                    // columns of a product
    static constexpr int Q_BYTES = BQ * 128;
    static constexpr int STAGE = P_BYTES + Q_BYTES + 1024;             // and 1 KB of scales
    static constexpr int STAGES = BQ == 16 ? 9 : 8;
    static constexpr int TMEM_COLS = BQ == 16 ? 128 : 256;             // two accumulators, and each stage's scales
    static_assert(2 * BQ + STAGES * 8 <= TMEM_COLS, "tensor memory");
};
constexpr int MAX_STAGES = 9;
constexpr int FEED_WARPS = 8, FIRST_EPI = 2 + FEED_WARPS;
constexpr int THREADS = 32 * (FIRST_EPI + 4);
constexpr int MAX_CLUSTER = 8;
// a wait by parity cannot tell a phase from the one two before it
static_assert(FEED_WARPS <= Cfg<true, false>::STAGES, "a feed warp's turns are within a round of the ring");

struct Routing;
struct FewParams {
    CUtensorMap map_p, map_p2;  // up: gate, up; down: down, h
    const uint8_t* scale_p;     // MXFP4: block scales of gate and up, or of down
    const uint8_t* scale_p2;
    int64_t scale_stride;       // bytes between experts
    int scale_pitch;
    const __nv_bfloat16* x;     // [T, H]
    const float* resid;         // [T, H], or NULL: x
    const float* logits;        // [T, E]
    uint8_t* h;                 // [T k][h_cols] bf16, or [H_TERMS][T k][h_cols] E4M3 terms
    uint8_t* h_scale;           // [H_TERMS][T k][h_scale_pitch]
    Routing* tables;            // the up kernel's, for the down kernel (unless small_routing)
    int h_cols, h_scale_pitch;
    int T, E, k, H, F;
    int splits;                 // CTAs of a cluster: up shares K, down the experts
    __nv_bfloat16* out;
    float* out32;
    uint32_t* err;
};

// ------------------------------------------------------------------ routing
struct alignas(16) Routing {
    uint32_t mask[MAX_E][2];      // the tokens of an expert (few rows: the logits' keys, and the experts in use)
    int first[MAX_E];             // its first row (rows are sorted by expert, then token)
    float sel_w[MAX_ROWS];
    float row_w[MAX_ROWS];        // weight and token of a row
    int16_t chunk_row[MAX_ROWS];  // first row, expert and rows of each chunk of up to TOK rows
    uint8_t sel[MAX_ROWS];
    uint8_t row_t[MAX_ROWS];
    uint8_t chunk_e[MAX_ROWS];
    uint8_t chunk_n[MAX_ROWS];
    int n_chunks;
    int pad[3];                   // 16-byte multiples: what follows is read as float4
};

// Order of floats as unsigned numbers; -0 as 0, NaN as -infinity. Never 0.
constexpr uint32_t KEY_LOWEST = 0x007fffffu;  // of -infinity
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v == v ? v + 0.f : -INFINITY);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

// Whether both kernels route for themselves. Beyond that the up kernel leaves its tables in memory, and the down
// kernel, whose CTAs mostly start when the up kernel's end, reads them: 1 us instead of 5 at 32 tokens.
__host__ __device__ __forceinline__ bool small_routing(int T, int k) { return T <= TOK && T * k <= 64; }

// Per token the k largest logits (ties to the lower expert), weights exp(l - l_max) / sum in fp32; all
// zero when every logit is -infinity. W lanes a token, PER of its logits each.
template <int PER, int W>
__device__ __forceinline__ void route_tokens(Routing& r, const FewParams& p, int warp, int lane) {
    const int l = lane % W;
    for (int t0 = warp * (32 / W); t0 < p.T; t0 += THREADS / W) {
        const int t = t0 + lane / W;
        const float* lg = p.logits + (int64_t)min(t, p.T - 1) * p.E;
        uint32_t key[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = l + W * i < p.E ? order_key(__ldg(lg + l + W * i)) : 0u;
        uint32_t mine = 0, mine_key = 0, top_key = 0;  // lane j: the j-th expert
        for (int j = 0; j < p.k; ++j) {
            uint32_t best = key[0], at = l;
#pragma unroll
            for (int i = 1; i < PER; ++i)
                if (key[i] > best) {
                    best = key[i];
                    at = l + W * i;
                }
            if (W == 32) {
                const uint32_t most = __reduce_max_sync(0xffffffffu, best);
                at = __reduce_min_sync(0xffffffffu, best == most ? at : 0xffffffffu);
                best = most;
            } else {
#pragma unroll
                for (int o = W / 2; o > 0; o >>= 1) {
                    const uint32_t ob = __shfl_xor_sync(0xffffffffu, best, o), oa = __shfl_xor_sync(0xffffffffu, at, o);
                    if (ob > best || (ob == best && oa < at)) {
                        best = ob;
                        at = oa;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (at == (uint32_t)(l + W * i)) key[i] = 0;
            if (l == j) {
                mine = at;
                mine_key = best;
            }
            if (j == 0) top_key = best;
        }
        float v = key_value(mine_key);
        if (mine_key == KEY_LOWEST) v = __ldg(lg + mine);  // -infinity, or NaN
        const float lowest = __shfl_sync(0xffffffffu, v, 0, W), top = top_key == KEY_LOWEST ? lowest : key_value(top_key);
        const float ex = l >= p.k ? 0.f : v != v ? v : top == -INFINITY ? 0.f : expf(v - top);
        float sum = 0.f;
        for (int j = 0; j < p.k; ++j) sum += __shfl_sync(0xffffffffu, ex, j, W);
        if (l < p.k && t < p.T) {
            r.sel[t * p.k + l] = (uint8_t)mine;
            r.sel_w[t * p.k + l] = sum == 0.f ? 0.f : ex / sum;
        }
    }
}

// The same when a thread can have a logit of its own: its place is the number of logits before it, and the k
// first write themselves down. No chain of maxima: one token's 128 experts take 0.5 us less so.
__device__ __forceinline__ void route_ranks(Routing& r, const FewParams& p) {
    uint32_t* keys = &r.mask[0][0];  // [T][E rounded up to 4]
    const int Ep = (p.E + 3) / 4 * 4;
    const int t = (int)threadIdx.x / Ep, e = (int)threadIdx.x % Ep;
    const float v = t < p.T && e < p.E ? __ldg(p.logits + (int64_t)t * p.E + e) : 0.f;
    const uint32_t key = order_key(v);
    if (t < p.T) keys[threadIdx.x] = e < p.E ? key : 0u;
    __syncthreads();
    float* chosen = r.row_w;  // [T][k]
    if (t < p.T && e < p.E) {
        // before: larger, or equal with a lower index. Words of four below the own one count from
        // `key` on, those above from `key` + 1 on; the own one's lower equals are added after
        const uint4* row = reinterpret_cast<const uint4*>(keys + t * Ep);
        const int own = e >> 2;
        int n0 = 0, n1 = 0, n2 = 0, n3 = 0;
#pragma unroll 8
        for (int i = 0; i < Ep / 4; ++i) {
            const uint4 o = row[i];
            const uint32_t over = i < own ? key - 1 : key;  // a key is at least 1
            n0 += o.x > over;
            n1 += o.y > over;
            n2 += o.z > over;
            n3 += o.w > over;
        }
        const uint4 o = row[own];
        const int c = e & 3;
        const int before = n0 + n1 + n2 + n3 + (c > 0 && o.x == key) + (c > 1 && o.y == key) + (c > 2 && o.z == key);
        if (before < p.k) {
            r.sel[t * p.k + before] = (uint8_t)e;
            chosen[t * p.k + before] = v;
        }
    }
    __syncthreads();
    const int i = threadIdx.x;  // T k is at most THREADS here: k is at most E
    const int first = i / p.k * p.k;
    if (i < p.T * p.k) {
        const float x = chosen[i], top = chosen[first];
        r.sel_w[i] = x != x ? x : top == -INFINITY ? 0.f : expf(x - top);
    }
    __syncthreads();
    float sum = 0.f, w = 0.f;
    if (i < p.T * p.k) {
        w = r.sel_w[i];
#pragma unroll
        for (int j = 0; j < MAX_K; ++j)
            if (j < p.k) sum += r.sel_w[first + j];
    }
    __syncthreads();
    if (i < p.T * p.k) r.sel_w[i] = sum == 0.f ? 0.f : w / sum;
}

// Rows and chunks of up to 64 routed pairs of up to TOK tokens, each by a thread that counts those before it.
__device__ __forceinline__ void small_tables(Routing& r, const FewParams& p) {
    const int n = p.T * p.k, i = threadIdx.x;
    uint32_t* used = &r.mask[MAX_E - 4][0];  // a bit for each expert
    if (i < 8) used[i] = 0;
    __syncthreads();
    if (i < n) atomicOr(&used[r.sel[i] >> 5], 1u << (r.sel[i] & 31));
    __syncthreads();
    if (i < n) {
        const int e = r.sel[i], t = i / p.k;
        int row = 0, same = 0, first = 0;
        for (int j = 0; j < n; ++j) {  // pairs are in order of their tokens
            const int o = r.sel[j];
            row += o < e || (o == e && j < i);
            first += o < e;
            same += o == e;
        }
        r.row_t[row] = (uint8_t)t;
        r.row_w[row] = r.sel_w[i];
        if (row == first) {
            int c = 0;
#pragma unroll
            for (int w = 0; w < MAX_E / 32; ++w)
                c += __popc(used[w] & (w < e >> 5 ? 0xffffffffu : w == e >> 5 ? (1u << (e & 31)) - 1u : 0u));
            r.chunk_e[c] = (uint8_t)e;
            r.chunk_n[c] = (uint8_t)same;
            r.chunk_row[c] = (int16_t)row;
        }
    }
    if (i == n) {  // fewer than THREADS pairs
        int c = 0;
#pragma unroll
        for (int w = 0; w < MAX_E / 32; ++w) c += __popc(used[w]);
        r.n_chunks = c;
    }
    __syncthreads();
}

// The same for any number: a warp has 32 experts, whose rows (low half) and chunks (high half) it sums in order.
__device__ __forceinline__ void large_tables(Routing& r, const FewParams& p, int warp, int lane) {
    for (int e = threadIdx.x; e < MAX_E; e += THREADS) r.mask[e][0] = r.mask[e][1] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * p.k; i += THREADS) atomicOr(&r.mask[r.sel[i]][i / p.k >> 5], 1u << (i / p.k & 31));
    __syncthreads();
    uint32_t n = 0, chunks = 0, sum = 0;
    const int e = 32 * warp + lane;
    uint32_t* totals = reinterpret_cast<uint32_t*>(r.chunk_row + MAX_ROWS - 16);  // free until the chunks are written
    if (warp < MAX_E / 32) {
        n = __popc(r.mask[e][0]) + __popc(r.mask[e][1]);
        chunks = (n + TOK - 1) / TOK;
        sum = n | chunks << 16;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t a = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += a;
        }
        if (lane == 31) totals[warp] = sum;
    }
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < MAX_E / 32; ++w) {
        if (w == warp) sum += before - (n | chunks << 16);
        before += totals[w];
    }
    __syncthreads();
    if (warp < MAX_E / 32) {
        const int row = sum & 0xffff, at = sum >> 16;
        r.first[e] = row;
        for (int c = 0; c < (int)chunks; ++c) {
            r.chunk_e[at + c] = (uint8_t)e;
            r.chunk_n[at + c] = (uint8_t)min(TOK, (int)n - TOK * c);
            r.chunk_row[at + c] = (int16_t)(row + TOK * c);
        }
    }
    if (threadIdx.x == 0) r.n_chunks = (int)(before >> 16);
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * p.k; i += THREADS) {
        const int t = i / p.k, x = r.sel[i];
        const uint32_t below = (1u << (t & 31)) - 1u;
        const int rank = t < 32 ? __popc(r.mask[x][0] & below) : __popc(r.mask[x][0]) + __popc(r.mask[x][1] & below);
        r.row_t[r.first[x] + rank] = (uint8_t)t;
        r.row_w[r.first[x] + rank] = r.sel_w[i];
    }
    __syncthreads();
}

// Every thread of the CTA; r is complete when it returns. The lanes of a token are chosen so that one
// pass of the CTA's warps takes all tokens.
__device__ __forceinline__ void route(Routing& r, const FewParams& p, int warp, int lane) {
    constexpr int N = THREADS / 32;
    if (p.T * ((p.E + 3) / 4 * 4) <= THREADS) {
        route_ranks(r, p);
    } else if (p.E <= 128) {
        if (p.T <= N) route_tokens<4, 32>(r, p, warp, lane);
        else if (p.T <= 2 * N) route_tokens<8, 16>(r, p, warp, lane);
        else route_tokens<16, 8>(r, p, warp, lane);
    } else {
        if (p.T <= N) route_tokens<8, 32>(r, p, warp, lane);
        else route_tokens<16, 16>(r, p, warp, lane);
    }
    __syncthreads();
    if (small_routing(p.T, p.k)) small_tables(r, p);
    else large_tables(r, p, warp, lane);
}

// ------------------------------------------------------------------ the two kernels
struct Bars {
    uint64_t full[MAX_STAGES], empty[MAX_STAGES], acc_full[2], acc_empty[2], done;
    uint32_t tmem;
};
static_assert(sizeof(Routing) % 16 == 0, "copied in 16-byte pieces");
struct UpSmem {
    Bars b;
    Routing r;
    float turn[UP_F][TOK + 1];                    // the up rows' sums, on their way to the gate rows' threads
    float red[MAX_CLUSTER - 1][TOK][TILE];        // the other CTAs' sums
};
struct alignas(16) DownSmem {
    Bars b;
    Routing r;
};
template <bool MX, bool UP>
constexpr int smem_bytes(int T) {
    return 1024 + Cfg<MX, UP>::STAGES * Cfg<MX, UP>::STAGE +
           (UP ? (int)sizeof(UpSmem) : (int)sizeof(DownSmem) + T * TILE * (int)sizeof(float));
}
static_assert(smem_bytes<true, true>(MAX_T) <= 232448 - 64 && smem_bytes<true, false>(MAX_T) <= 232448 - 64 &&
                  smem_bytes<false, false>(MAX_T) <= 232448 - 64,
              "shared memory");

__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__host__ __device__ constexpr uint32_t bf16_idesc(int M, int N) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ float4 ld_cluster(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}

// The columns f0 to f0 + 63 of h for n tokens, from a tile's sums: warps q = 0 and 1 have the gate
// rows, 2 and 3 the up rows. All four warps of the epilogue.
template <bool MX>
__device__ __forceinline__ void write_h(const FewParams& p, UpSmem& sm, const float (&v)[TOK], int q, int lane, int row0, int n,
                                        int f0) {
    if (q >= 2)
#pragma unroll
        for (int j = 0; j < TOK; ++j) sm.turn[(q - 2) * 32 + lane][j] = v[j];
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (q < 2) {
        const int f = f0 + q * 32 + lane;
        const int64_t R = (int64_t)p.T * p.k;
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
            if (j >= n) continue;
            const float g = v[j], h = g / (1.f + __expf(-g)) * sm.turn[q * 32 + lane][j];
            if (MX) {  // one block of 32: each term takes four bits of what the ones before leave
                const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7fffffffu), e = m >> 23;
                float rest = h;
#pragma unroll
                for (int i = 0; i < H_TERMS; ++i) {
                    const uint32_t low = 7 + 5 * i, b = e == 255 ? 255 : e < low ? 0 : e - low;
                    uint16_t t;
                    uint32_t back;
                    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(t) : "f"(0.f), "f"(rest * __uint_as_float((254 - min(b, 253u)) << 23)));
                    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(t));
                    rest -= __half2float(__ushort_as_half((unsigned short)(back & 0xffffu))) * e8m0_to_float(min(b, 254u));
                    p.h[(i * R + row0 + j) * p.h_cols + f] = e == 255 ? 0 : (uint8_t)t;
                    if (lane == 0) p.h_scale[(i * R + row0 + j) * p.h_scale_pitch + (f0 + q * 32) / 32] = (uint8_t)b;
                }
            } else {
                reinterpret_cast<__nv_bfloat16*>(p.h)[(int64_t)(row0 + j) * p.h_cols + f] = __float2bfloat16_rn(h);
            }
        }
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
}

// A CTA's line of work: units of ks stages (stages k0 to k0 + ks of the unit's K) each. Up: a unit is a
// (chunk, tile of h); down: a chunk.
template <bool MX, bool UP>
__global__ void __launch_bounds__(THREADS, 1) moe_few_kernel(const __grid_constant__ FewParams p) {
    using C = Cfg<MX, UP>;
    constexpr int KV = MX ? 128 : 64;  // values of K in a stage
    constexpr int BQ = C::BQ, Q_BYTES = C::Q_BYTES, STAGE = C::STAGE, STAGES = C::STAGES;
    extern __shared__ uint8_t raw_smem[];
    const uint32_t raw = smem_addr(raw_smem), base = (raw + 1023u) & ~1023u;
    uint8_t* gen = raw_smem + (base - raw) + STAGES * STAGE;
    Bars& bars = *reinterpret_cast<Bars*>(gen);
    Routing& rt = UP ? reinterpret_cast<UpSmem*>(gen)->r : reinterpret_cast<DownSmem*>(gen)->r;
    float* sums = reinterpret_cast<float*>(gen + sizeof(DownSmem));  // down: [T][TILE]
    const uint32_t full0 = smem_addr(bars.full), empty0 = smem_addr(bars.empty), acc_full0 = smem_addr(bars.acc_full),
                   acc_empty0 = smem_addr(bars.acc_empty), done = smem_addr(&bars.done);
    __shared__ volatile int stop;
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    constexpr bool FEED = MX || UP;  // down with bf16 weights has nothing to add to a stage

    if (threadIdx.x == 0) {
        stop = 0;
        for (int s = 0; s < STAGES; ++s) {
            bar_init(full0 + 8 * s, FEED ? 2 : 1);  // the TMA thread and the stage's feed warp
            bar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(acc_full0 + 8 * b, 1);
            bar_init(acc_empty0 + 8 * b, 4);
        }
        bar_init(done, 1);
        bar_init_fence();
        tma_desc_prefetch(&p.map_p);
        tma_desc_prefetch(&p.map_p2);
    }
    if (warp == 1) tmem_get(smem_addr(&bars.tmem), C::TMEM_COLS);
    if (!UP)
        for (int i = threadIdx.x; i < p.T * TILE; i += THREADS) sums[i] = 0.f;
    fence_before_sync();
    // up: everything earlier is complete after the wait, so the down kernel, which may be placed from here on, can
    // read the logits and the weights at once; only h has to wait for this kernel
    if (UP) {
        grid_wait();
        grid_release();
    }
    if (UP || small_routing(p.T, p.k)) {
        route(rt, p, warp, lane);  // ends with a barrier of the CTA
    } else {
        grid_wait();
        const uint4* from = reinterpret_cast<const uint4*>(p.tables);
        for (int i = threadIdx.x; i < (int)(sizeof(Routing) / 16); i += THREADS) reinterpret_cast<uint4*>(&rt)[i] = __ldcg(from + i);
        __syncthreads();
    }
    if (UP && blockIdx.x == 0 && !small_routing(p.T, p.k))
        for (int i = threadIdx.x; i < (int)(sizeof(Routing) / 16); i += THREADS)
            reinterpret_cast<uint4*>(p.tables)[i] = reinterpret_cast<const uint4*>(&rt)[i];
    if (p.splits > 1) {
        __syncwarp();
        cluster_barrier();
    }
    fence_after_sync();
    const uint32_t tmem = bars.tmem;

    const int rank = (int)blockIdx.x % p.splits, cluster = (int)blockIdx.x / p.splits;
    const int stages = ((UP ? p.H : p.F) + KV - 1) / KV;
    int unit0, unit_step, n_units, k0 = 0, ks = stages;
    const int n_f = (p.h_cols + UP_F - 1) / UP_F;
    if (UP) {
        k0 = rank * stages / p.splits;
        ks = (rank + 1) * stages / p.splits - k0;
        unit0 = cluster;
        unit_step = (int)gridDim.x / p.splits;
        const int units = rt.n_chunks * n_f;
        n_units = unit0 < units ? (units - 1 - unit0) / unit_step + 1 : 0;
    } else {
        unit0 = rank * rt.n_chunks / p.splits;
        unit_step = 1;
        n_units = (rank + 1) * rt.n_chunks / p.splits - unit0;
    }
    const int row_p = UP ? 0 : cluster * TILE;  // down: the tile's rows
    auto chunk_of = [&](int u) { return UP ? u / n_f : u; };
    auto f_of = [&](int u) { return UP ? u % n_f * UP_F : 0; };
    const int R = p.T * p.k;

    if (warp == 0) {
        // ------------------------------------------------------------ weights (down: and h)
        const bool one = elect_one();
        constexpr uint32_t BYTES = (MX ? P_BYTES / 2 : P_BYTES) + (UP ? 0 : C::TERMS * TOK * 128);
        auto load_p = [&](int s, int chunk, int f0, int k) {
            const uint32_t at = base + s * STAGE, bar = full0 + 8 * s;
            const int e = rt.chunk_e[chunk], x = k * KV;
            bar_expect(bar, BYTES);
            if (UP) {
                tma_3d(at, &p.map_p, bar, x, f0, e);
                tma_3d(at + P_BYTES / 2, &p.map_p2, bar, x, f0, e);
            } else {
                tma_3d(at, &p.map_p, bar, x, row_p, e);
            }
        };
        auto load_h = [&](int s, int chunk, int k) {
            if (MX) tma_3d(base + s * STAGE + P_BYTES, &p.map_p2, full0 + 8 * s, k * KV, rt.chunk_row[chunk], 0);
            else tma_2d(base + s * STAGE + P_BYTES, &p.map_p2, full0 + 8 * s, k * KV, rt.chunk_row[chunk]);
        };
        int s = 0, it = 0, u = 0, k = 0;
        uint32_t phase = 1;
        bool ok = true;
        if (!UP) {  // the first round's weights before h is complete
            const int ahead = min(STAGES, n_units * ks);
            if (one)
                for (int i = 0, v = 0, q = 0; i < ahead; ++i) {
                    load_p(i, unit0 + v, 0, q);
                    if (++q == ks) {
                        q = 0;
                        ++v;
                    }
                }
            grid_wait();
            if (one)
                for (int i = 0, v = 0, q = 0; i < ahead; ++i) {
                    load_h(i, unit0 + v, q);
                    if (++q == ks) {
                        q = 0;
                        ++v;
                    }
                }
            __syncwarp();
            it = ahead;
            u = ahead / ks;
            k = ahead % ks;
            s = ahead % STAGES;
            phase ^= ahead == STAGES ? 1u : 0u;
        }
        for (; ok && u < n_units; ++u, k = 0) {
            const int unit = unit0 + u * unit_step, chunk = chunk_of(unit), f0 = f_of(unit);
            for (; k < ks; ++k, ++it) {
                if (!bar_wait_warp(empty0 + 8 * s, phase, p.err, 1)) {
                    ok = false;
                    stop = 1;
                    break;
                }
                if (one) {
                    load_p(s, chunk, f0, k0 + k);
                    if (!UP) load_h(s, chunk, k);
                }
                __syncwarp();
                if (++s == STAGES) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
        if (stop)  // an aborted CTA waits for its own copies before it exits
            for (int i = 0; i < STAGES && i < it; ++i) {
                const int last = it - 1 - (it - 1 - i) % STAGES;
                bar_wait(full0 + 8 * i, (uint32_t)(last / STAGES) & 1u, p.err, 5);
            }
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        constexpr uint32_t IDESC = MX ? mx_idesc(5, 0, TILE, BQ) : bf16_idesc(TILE, BQ);
        const bool one = elect_one();
        int s = 0;
        uint32_t phase = 0;
        bool ok = true, ready = false;  // ready: the next stage's barrier, asked before this stage's products
        for (int u = 0; ok && u < n_units; ++u) {
            const int b = u & 1;
            if (!bar_wait_warp(acc_empty0 + 8 * b, (uint32_t)((u >> 1) + 1) & 1u, p.err, 2) || stop) {
                stop = 1;
                break;
            }
            fence_after_sync();
            const uint32_t d = tmem + (uint32_t)(b * BQ);
            for (int k = 0; k < ks; ++k) {
                if (!__all_sync(0xffffffffu, ready) && !bar_wait_warp(full0 + 8 * s, phase, p.err, 3)) {
                    ok = false;
                    stop = 1;
                    break;
                }
                fence_after_sync();
                const uint32_t sp = base + s * STAGE, sq = sp + P_BYTES, sc = sq + Q_BYTES;
                const uint32_t tp = tmem + (uint32_t)(2 * BQ + s * 8), freed = empty0 + 8 * s;
                if (++s == STAGES) {
                    s = 0;
                    phase ^= 1u;
                }
                ready = bar_test(full0 + 8 * s, phase);
                if (one) {
                    if (MX) {
                        scale_copy(tp, scale_desc(sc));
                        scale_copy(tp + 4, scale_desc(sc + 512));
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // 32 bytes of each row
                        const uint32_t acc = (k > 0 || i > 0) ? 1u : 0u;
                        if (MX) mma_mxf8(d, operand_desc(sp + 32 * i), operand_desc(sq + 32 * i), idesc_at(IDESC, i), tp, tp + 4, acc);
                        else mma_bf16(d, operand_desc(sp + 32 * i), operand_desc(sq + 32 * i), IDESC, acc);
                    }
                    mma_commit(freed);
                }
                __syncwarp();
            }
            if (ok && one) mma_commit(acc_full0 + 8 * b);
            __syncwarp();
        }
        if (one) mma_commit(done);
        __syncwarp();
        bar_wait(done, 0, p.err, 6);
    } else if (warp < FIRST_EPI) {
        // ------------------------------------------------------------ scales, and the tokens' rows
        if (FEED) {
            // a warp's turn is every eighth stage; it requests the next turn's data before this one's work
            constexpr int UNITS = MX ? 4 : 2;  // up: pieces of 8 values a lane
            const int total = n_units * ks;
            struct Turn {
                uint32_t sp[4], sq;
                uint4 x[UP ? UNITS : 1];
            };
            auto fetch = [&](Turn& to, int it, bool weights, bool rest) {
                if (it >= total) return;
                const int u = it / ks, k = k0 + it - u * ks, unit = unit0 + u * unit_step;
                const int chunk = chunk_of(unit), e = rt.chunk_e[chunk], n = rt.chunk_n[chunk], row0 = rt.chunk_row[chunk];
                if (MX && weights) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = lane + 32 * j;
                        const uint8_t* sp = UP && j >= 2 ? p.scale_p2 : p.scale_p;
                        const int row = UP ? f_of(unit) + (r & (UP_F - 1)) : row_p + r;
                        const bool in = row < (UP ? p.F : p.H);
                        to.sp[j] = in ? __ldg(reinterpret_cast<const uint32_t*>(sp + e * p.scale_stride + (int64_t)row * p.scale_pitch + 4 * k)) : 0u;
                    }
                }
                if (!rest) return;
                if (MX && !UP) {  // lane: term lane / 8 of row lane % 8
                    to.sq = lane < C::TERMS * TOK && (lane & 7) < n
                                ? __ldcg(reinterpret_cast<const uint32_t*>(p.h_scale + ((int64_t)(lane >> 3) * R + row0 + (lane & 7)) * p.h_scale_pitch + 4 * k))
                                : 0u;
                }
                if (UP) {
#pragma unroll
                    for (int j = 0; j < UNITS; ++j) {
                        // MXFP4: 16 pieces of a token's 128 values, two tokens at a time; bf16: 8 of 64, four
                        const int tok = MX ? (lane >> 4) + 2 * j : (lane >> 3) + 4 * j, at = k * KV + 8 * (MX ? lane & 15 : lane & 7);
                        const bool in = tok < n && at < p.H;  // H is a multiple of 8
                        to.x[j] = in ? __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)rt.row_t[row0 + tok] * p.H + at))
                                     : make_uint4(0, 0, 0, 0);
                    }
                }
            };
            const int first = warp - 2;
            Turn cur, nxt;
            if (UP) {
                fetch(cur, first, true, true);
            } else {
                fetch(cur, first, true, false);
                grid_wait();
                fetch(cur, first, false, true);
            }
            bool ok = true;
            for (int it = first; ok && it < total; it += FEED_WARPS) {
                fetch(nxt, it + FEED_WARPS, true, true);
                const int s = it % STAGES;
                if (!bar_wait_warp(empty0 + 8 * s, (uint32_t)(it / STAGES + 1) & 1u, p.err, 7)) {
                    ok = false;
                    stop = 1;
                    break;
                }
                const uint32_t sq = base + s * STAGE + P_BYTES, sc = sq + Q_BYTES;
                if (MX) {
                    // rows l, l + 32, l + 64, l + 96: side by side in the order that the tensor core reads
                    st_shared4(sc + 16 * lane, cur.sp[0], cur.sp[1], cur.sp[2], cur.sp[3]);
                    if (!UP)
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(sc + 512 + 16 * lane), "r"(cur.sq) : "memory");
                }
                if (UP) {
                    const int n = rt.chunk_n[chunk_of(unit0 + it / ks * unit_step)];
#pragma unroll
                    for (int j = 0; j < UNITS; ++j) {
                        if ((MX ? 2 : 4) * j >= n) continue;  // columns of tokens that do not exist hold anything
                        if (MX) {
                            uint2 o1, o2;
                            uint32_t b1, b2;
                            split8(cur.x[j], o1, o2, b1, b2);
                            const int g = lane & 15, r = (lane >> 4) + 2 * j;
                            const uint32_t at = sq + r * 128 + (uint32_t)((((g >> 1) ^ (r & 7)) << 4) + (g & 1) * 8);
                            st_shared2(at, o1.x, o1.y);
                            st_shared2(at + TOK * 128, o2.x, o2.y);
                            if ((g & 3) == 0) {
                                const uint32_t to = sc + 512 + (uint32_t)(r * 16 + (g >> 2));
                                asm volatile("st.shared.u8 [%0], %1;" ::"r"(to), "r"(b1) : "memory");
                                asm volatile("st.shared.u8 [%0], %1;" ::"r"(to + TOK * 16), "r"(b2) : "memory");
                            }
                        } else {
                            const int g = lane & 7, r = (lane >> 3) + 4 * j;
                            st_shared4(sq + r * 128 + (uint32_t)((g ^ r) << 4), cur.x[j].x, cur.x[j].y, cur.x[j].z, cur.x[j].w);
                        }
                    }
                }
                fence_smem_async();
                __syncwarp();
                if (lane == 0) bar_arrive(full0 + 8 * s);
                cur = nxt;
            }
        }
    }
    // ------------------------------------------------------------ results
    const int q = warp & 3, row = q * 32 + lane;  // the TMEM lane quarter that this warp can read
    bool bad = false;  // a wait ran out: no later one is made, and the results are void
    auto take = [&](int u, float (&v)[TOK]) {
        const int b = u & 1;
        const uint32_t t = tmem + ((uint32_t)(q * 32) << 16) + b * BQ;
        if (!bad) bad = !bar_wait_warp(acc_full0 + 8 * b, (uint32_t)(u >> 1) & 1u, p.err, 4);
        if (bad) stop = 1;
        fence_after_sync();
        uint32_t x[C::TERMS][8];
#pragma unroll
        for (int i = 0; i < C::TERMS; ++i) tmem_load8(t + i * TOK, x[i]);
        tmem_load_wait();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) bar_arrive(acc_empty0 + 8 * b);
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
            v[j] = __uint_as_float(x[C::TERMS - 1][j]);  // the smallest first
#pragma unroll
            for (int i = C::TERMS - 2; i >= 0; --i) v[j] += __uint_as_float(x[i][j]);
        }
    };
    if (UP) {
        UpSmem& sm = *reinterpret_cast<UpSmem*>(gen);
        if (p.splits == 1) {
            if (warp >= FIRST_EPI)
                for (int u = 0; u < n_units; ++u) {
                    float v[TOK];
                    take(u, v);
                    const int unit = unit0 + u * unit_step, chunk = chunk_of(unit);
                    write_h<MX>(p, sm, v, q, lane, rt.chunk_row[chunk], rt.chunk_n[chunk], f_of(unit));
                }
        } else {  // one unit a cluster: the later CTAs leave their sums in the first one's memory
            if (warp >= FIRST_EPI && rank > 0 && n_units > 0) {
                float v[TOK];
                take(0, v);
                const uint32_t to = cluster_addr(smem_addr(&sm.red[rank - 1][0][row]), 0);
#pragma unroll
                for (int j = 0; j < TOK; ++j) st_cluster(to + j * TILE * 4, v[j]);
            }
            __syncwarp();
            cluster_barrier();
            if (warp >= FIRST_EPI && rank == 0 && n_units > 0) {
                float v[TOK];
                take(0, v);
#pragma unroll
                for (int j = 0; j < TOK; ++j)
                    for (int i = 0; i < p.splits - 1; ++i) v[j] += sm.red[i][j][row];
                const int chunk = chunk_of(unit0);
                write_h<MX>(p, sm, v, q, lane, rt.chunk_row[chunk], rt.chunk_n[chunk], f_of(unit0));
            }
        }
    } else {
        if (warp >= FIRST_EPI)
            for (int u = 0; u < n_units; ++u) {
                float v[TOK];
                take(u, v);
                const int chunk = unit0 + u, n = rt.chunk_n[chunk], row0 = rt.chunk_row[chunk];
#pragma unroll
                for (int j = 0; j < TOK; ++j)
                    if (j < n) {
                        float* to = sums + rt.row_t[row0 + j] * TILE + row;
                        *to = fmaf(rt.row_w[row0 + j], v[j], *to);
                    }
            }
        // the cluster's sums, in CTA order; each CTA writes a share of the outputs
        __syncwarp();
        if (p.splits > 1) cluster_barrier();
        else __syncthreads();
        for (int i = 4 * (rank * THREADS + (int)threadIdx.x); i < p.T * TILE; i += 4 * p.splits * THREADS) {
            const int t = i / TILE, r = row_p + i % TILE;
            if (r >= p.H) continue;  // H is a multiple of 8
            float4 part[MAX_CLUSTER];
#pragma unroll
            for (int c = 0; c < MAX_CLUSTER; ++c)  // all loads before the first sum
                if (c < p.splits)
                    part[c] = p.splits > 1 ? ld_cluster(cluster_addr(smem_addr(sums + i), c)) : *reinterpret_cast<const float4*>(sums + i);
            const int64_t at = (int64_t)t * p.H + r;
            float v[4];
            if (p.resid) {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = p.resid[at + j];
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(p.x + at);
                v[0] = __uint_as_float(x.x << 16);
                v[1] = __uint_as_float(x.x & 0xffff0000u);
                v[2] = __uint_as_float(x.y << 16);
                v[3] = __uint_as_float(x.y & 0xffff0000u);
            }
            float4 sum = part[0];
#pragma unroll
            for (int c = 1; c < MAX_CLUSTER; ++c)
                if (c < p.splits) {
                    sum.x += part[c].x;
                    sum.y += part[c].y;
                    sum.z += part[c].z;
                    sum.w += part[c].w;
                }
            v[0] += sum.x;
            v[1] += sum.y;
            v[2] += sum.z;
            v[3] += sum.w;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                p.out[at + j] = __float2bfloat16_rn(v[j]);
                if (p.out32) p.out32[at + j] = v[j];
            }
        }
        __syncwarp();
        if (p.splits > 1) cluster_barrier();  // nobody goes while its sums are read
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        tmem_free(tmem, C::TMEM_COLS);
    }
}

// ------------------------------------------------------------------ host side
// View [experts][rows][pitch bytes] in boxes of one stage's K x box_rows, 128-byte swizzle.
bool map_experts(CUtensorMap* m, bool mx, const void* ptr, int64_t pitch, int64_t rows, int64_t experts, int64_t stride,
                 int box_rows) {
    const MxEncodeFn fn = mx_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)(mx ? 2 * pitch : pitch / 2), (cuuint64_t)rows, (cuuint64_t)experts};
    cuuint64_t strides[2] = {(cuuint64_t)pitch, (cuuint64_t)stride};
    cuuint32_t box[3] = {mx ? 128u : 64u, (cuuint32_t)box_rows, 1};
    cuuint32_t one[3] = {1, 1, 1};
    return fn(m, mx ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims,
              strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// h: [rows][cols] bf16 in boxes of 64 x 8, or [H_TERMS][rows][cols] bytes in boxes of 128 x 8 x H_TERMS.
bool map_h(CUtensorMap* m, bool mx, const void* ptr, int64_t rows, int64_t cols) {
    const MxEncodeFn fn = mx_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, H_TERMS};
    cuuint64_t strides[2] = {(cuuint64_t)(mx ? cols : 2 * cols), (cuuint64_t)(rows * cols)};
    cuuint32_t box[3] = {mx ? 128u : 64u, TOK, H_TERMS};
    cuuint32_t one[3] = {1, 1, 1};
    return fn(m, mx ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, mx ? 3 : 2, const_cast<void*>(ptr), dims,
              strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool MX, bool UP>
cudaError_t launch(const FewParams& p, int grid, cudaStream_t s) {
    auto kern = moe_few_kernel<MX, UP>;
    static const cudaError_t attr =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<MX, UP>(MAX_T));
    if (attr != cudaSuccess) return attr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem_bytes<MX, UP>(p.T);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = p.splits;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// Columns of a row of h: whole stages of the down kernel's K, and whole tiles of the up kernel.
int few_h_cols(bool mx, int F) { return mx ? (F + 127) / 128 * 128 : (F + 63) / 64 * 64; }
int64_t few_h_bytes(bool mx, int64_t rows, int F) {
    return (rows * few_h_cols(mx, F) * (mx ? H_TERMS : 2) + 255) / 256 * 256;
}

}  // namespace

int64_t moe_few_ws_bytes(bool mx, int T, int k, int F) {
    const int64_t rows = (int64_t)T * k;
    return (int64_t)sizeof(Routing) + 256 + few_h_bytes(mx, rows, F) + (mx ? H_TERMS * rows * mx_scale_pitch(F) : 0);
}

cudaError_t launch_moe_few(const MoeFewDesc& d, void* ws, uint32_t* err, cudaStream_t s) {
    if (d.T <= 0) return cudaSuccess;
    if (d.T > MAX_T || d.E < 1 || d.E > MAX_E || d.k < 1 || d.k > MAX_K || d.k > d.E) return cudaErrorInvalidValue;
    FewParams p;
    memset(&p, 0, sizeof(p));
    const int64_t rows = (int64_t)d.T * d.k;
    const int64_t up_pitch = d.mx ? mx_code_pitch(d.H) : 2ll * d.H, down_pitch = d.mx ? mx_code_pitch(d.F) : 2ll * d.F;
    if (!map_experts(&p.map_p, d.mx, d.gate, up_pitch, d.F, d.E, d.gate_stride, UP_F) ||
        !map_experts(&p.map_p2, d.mx, d.up, up_pitch, d.F, d.E, d.gate_stride, UP_F))
        return cudaErrorInvalidValue;
    p.scale_p = static_cast<const uint8_t*>(d.gate_scales);
    p.scale_p2 = static_cast<const uint8_t*>(d.up_scales);
    p.scale_stride = d.gate_scale_stride;
    p.scale_pitch = (int)mx_scale_pitch(d.H);
    p.x = static_cast<const __nv_bfloat16*>(d.x);
    p.resid = d.resid;
    p.logits = d.logits;
    p.h = static_cast<uint8_t*>(ws);
    p.tables = reinterpret_cast<Routing*>(p.h);
    p.h += (sizeof(Routing) + 255) / 256 * 256;
    p.h_scale = p.h + few_h_bytes(d.mx, rows, d.F);
    p.h_cols = few_h_cols(d.mx, d.F);
    p.h_scale_pitch = (int)mx_scale_pitch(d.F);
    p.T = d.T;
    p.E = d.E;
    p.k = d.k;
    p.H = d.H;
    p.F = d.F;
    p.out = static_cast<__nv_bfloat16*>(d.out);
    p.out32 = d.out32;
    p.err = err;
    FewParams q = p;
    if (!map_experts(&q.map_p, d.mx, d.down, down_pitch, d.H, d.E, d.down_stride, TILE) ||
        !map_h(&q.map_p2, d.mx, p.h, rows, p.h_cols))
        return cudaErrorInvalidValue;
    q.scale_p = static_cast<const uint8_t*>(d.down_scales);
    q.scale_stride = d.down_scale_stride;
    q.scale_pitch = (int)mx_scale_pitch(d.F);
    const int sms = gemm_num_sms();
    // up: at most rows x (h_cols / 64) units. Fewer than half the SMs: a cluster shares each along K
    const int64_t units = rows * (p.h_cols / UP_F);
    const int up_stages = (d.H + (d.mx ? 127 : 63)) / (d.mx ? 128 : 64);
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({MAX_CLUSTER, sms / units, up_stages / 2}));
    const int grid_up = (int)std::min<int64_t>(units * p.splits, sms);
    // down: clusters of as many CTAs as the SMs hold, but no more than there are rows
    const int tiles = (d.H + TILE - 1) / TILE;
    q.splits = (int)std::max<int64_t>(1, std::min<int64_t>({MAX_CLUSTER, sms / tiles, rows}));
    cudaError_t e = d.mx ? launch<true, true>(p, grid_up, s) : launch<false, true>(p, grid_up, s);
    if (e != cudaSuccess) return e;
    return d.mx ? launch<true, false>(q, tiles * q.splits, s) : launch<false, false>(q, tiles * q.splits, s);
}

}  // namespace ls
