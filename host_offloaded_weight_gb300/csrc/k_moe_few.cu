// A whole mixture-of-experts layer for a few tokens, in one launch:
//
//   h[i]   = SiLU(G_e x_t) * (U_e x_t)   for every routed pair i = (t, e)                 ("up")
//   out[t] = r[t] + sum_j w[t,j] D_e h[i],  w = softmax over the token's k largest logits ("down")
//
// Experts in bf16 or MXFP4. The bound is the bytes of the experts that are routed: each is read
// once (for up to 8 of its tokens), and nothing else of that size is touched.
//
// The weights are the left operand of tcgen05.mma (128 rows a tile) and the tokens the right one: 16
// or 32 columns, which are 8 tokens as bf16 (and columns that nobody reads), or, with MXFP4 experts,
// as E4M3 terms with a power of two for each block of 32 (see k_gemm_mx.cu): two for x, which
// holds a bf16's 8 bits, and three for h, 12 bits. So the weights go from memory to the tensor core as they
// are, with no instruction spent on a value, and a product (about 60 clocks for 4 KB of the stage)
// stays under the memory's time. A tile of up takes 64 gate rows and the 64 up rows of the same columns of h.
//
// The grid is resident as a whole (a cooperative launch): every CTA routes for itself, takes tiles of
// up, meets the others once, and takes a tile of 128 output rows for its share of the experts. Across the
// meeting the ring of stages goes on: the first weights of down are requested before it. (As two
// launches the second one's start, routing and first loads cost 8 us of 18 at one token.) The CTAs of a tile add
// their sums through memory, each a part of the outputs, in the order of the CTAs: the same bits
// every time, and no atomics on data.
//
// Roles (numbers of the code, see the kernel for the hardware's warps): 0 loads the weights by TMA into the ring,
// 2 to 9 take turns at the stages and add the block scales and (up) the tokens' rows, 1 and 14 issue the products of
// even and odd stages into accumulators of their own (one warp alone took 385 clocks a stage of 240 clocks of
// products, between its waits; the memory brings a stage in 370), 10 to 13 take the results.
//
// 128 experts of 2048 x 768, k = 8: 16 tokens bf16 124 us (6.25 TB/s of the routed experts' bytes), 32 tokens MXFP4
// 64 us (4.4 TB/s): routing 4.5, first load 3, up 31, the meeting and h on its way back 4, down 14, the tile's sums 4.
// 1 token MXFP4 16.6 us, nearly all of it those latencies, bf16 23; 64 tokens bf16 184 us (6.4 TB/s), MXFP4 73.
#include <cooperative_groups.h>

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
constexpr int FEED_WARPS = 8, FIRST_EPI = 2 + FEED_WARPS;
constexpr int SECOND_MMA = FIRST_EPI + 4;  // the warp that issues the products of odd stages
constexpr int THREADS = 32 * (SECOND_MMA + 2);  // the last warp takes part in the routing alone: 16 tokens in one pass
constexpr int P_BYTES = TILE * 128;
constexpr int X_TERMS = 2, H_TERMS = 3;  // E4M3 terms of x and of h (MXFP4 experts)

template <bool MX>
struct Cfg {
    static constexpr int Q_ROWS = MX ? 32 : 16;                        // columns of the widest product
    static constexpr int Q_BYTES = Q_ROWS * 128;
    static constexpr int STAGE = P_BYTES + Q_BYTES + 1024;             // and 1 KB of scales
    static constexpr int STAGES = 8;
    static_assert(4 * Q_ROWS + STAGES * 8 <= 256, "tensor memory: two pairs of accumulators, and each stage's scales");
    // A wait by parity cannot tell a phase from the one two before it, and stages are freed in any order (even and
    // odd ones by different warps). A feed warp that always has the same stages of the ring has waited for each phase before.
    static_assert(STAGES % FEED_WARPS == 0 && STAGES % 2 == 0, "a stage of the ring has one feed warp and one product warp");
};
constexpr int MAX_STAGES = 8, TMEM_COLS = 256;
constexpr int MAX_SHARES = 32;    // CTAs that share an output tile

struct FewParams {
    CUtensorMap gate, up, down, map_h;
    const uint8_t* gate_scale;  // MXFP4: block scales
    const uint8_t* up_scale;
    const uint8_t* down_scale;
    int64_t up_scale_stride, down_scale_stride;  // bytes between experts
    int up_scale_pitch, down_scale_pitch;
    const __nv_bfloat16* x;     // [T, H]
    const float* resid;         // [T, H], or NULL: x
    const float* logits;        // [T, E]
    uint8_t* h;                 // [T k][h_cols] bf16, or [H_TERMS][T k][h_cols] E4M3 terms
    uint8_t* h_scale;           // [H_TERMS][T k][h_scale_pitch]
    float* partial;             // [output tile][share][T][TILE]
    uint32_t* tickets;          // [output tile]
    int h_cols, h_scale_pitch;
    int T, E, k, H, F;
    int tiles, shares;          // output tiles, and the CTAs that share one
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
    uint16_t sel[MAX_ROWS];       // NONE: chosen for want of a better one, takes no part
    uint8_t row_t[MAX_ROWS];
    uint8_t chunk_e[MAX_ROWS];
    uint8_t chunk_n[MAX_ROWS];
    int n_chunks;
    int pad[3];                   // 16-byte multiples: what follows is read as float4
};

// A chosen logit of -infinity has weight 0: its pair gets no row, so that its expert is not read and what the expert or
// the token holds (0 times infinity, NaN) cannot reach the sums.
constexpr uint16_t NONE = 0xffffu;

// Order of floats as unsigned numbers; -0 as 0, NaN as -infinity. Never 0.
constexpr uint32_t KEY_LOWEST = 0x007fffffu;  // of -infinity
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v == v ? v + 0.f : -INFINITY);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

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
            r.sel[t * p.k + l] = v == -INFINITY ? NONE : (uint16_t)mine;
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
            r.sel[t * p.k + before] = v == -INFINITY ? NONE : (uint16_t)e;
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
    const int e = i < n ? r.sel[i] : NONE;
    if (e != NONE) atomicOr(&used[e >> 5], 1u << (e & 31));
    __syncthreads();
    if (e != NONE) {
        const int t = i / p.k;
        int row = 0, same = 0, first = 0;
        for (int j = 0; j < n; ++j) {  // pairs are in order of their tokens; NONE is above every expert
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
    for (int i = threadIdx.x; i < p.T * p.k; i += THREADS)
        if (r.sel[i] != NONE) atomicOr(&r.mask[r.sel[i]][i / p.k >> 5], 1u << (i / p.k & 31));
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
        if (x == NONE) continue;
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
    if (p.T <= TOK && p.T * p.k <= 64) small_tables(r, p);
    else large_tables(r, p, warp, lane);
}

// ------------------------------------------------------------------ the kernel
struct alignas(16) Smem {
    uint64_t full[MAX_STAGES], empty[MAX_STAGES], acc_full[2], acc_empty[2], done;
    uint32_t tmem, met;
    float turn[TILE][TOK + 1];  // a tile's sums, on their way to the threads that make h
    Routing r;
};
template <bool MX>
constexpr int smem_bytes(int T) {
    return 1024 + Cfg<MX>::STAGES * Cfg<MX>::STAGE + (int)sizeof(Smem) + T * TILE * (int)sizeof(float);
}
static_assert(smem_bytes<true>(MAX_T) <= 232448 - 64 && smem_bytes<false>(MAX_T) <= 232448 - 64, "shared memory");

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

// The columns f0 to f0 + 63 of h for n tokens, from the sums in sm.turn. The epilogue's 128 threads.
template <bool MX>
__device__ __forceinline__ void write_h(const FewParams& p, const Smem& sm, int tid, int row0, int n, int f0) {
    const int c = tid & 63, f = f0 + c;
    const int64_t R = (int64_t)p.T * p.k;
#pragma unroll 1
    for (int j = tid >> 6; j < n; j += 2) {
        const float g = sm.turn[c][j], h = g / (1.f + __expf(-g)) * sm.turn[UP_F + c][j];
        if (MX) {  // a warp has one block of 32: each term takes four bits of what the ones before leave
            const uint32_t e = __reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7fffffffu) >> 23;
            float rest = h * __uint_as_float((254 - min(term_byte(e, 0), 253u)) << 23);  // in units of the next term's scale
#pragma unroll
            for (int i = 0; i < H_TERMS; ++i) {
                const uint32_t b = term_byte(e, i);
                uint16_t t;
                uint32_t back;
                asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(t) : "f"(0.f), "f"(i ? rest : first_term(rest, e)));
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(t));
                rest = (rest - __half2float(__ushort_as_half((unsigned short)(back & 0xffffu)))) * pow2(b - term_byte(e, i + 1));
                p.h[(i * R + row0 + j) * p.h_cols + f] = e == 255 ? 0 : (uint8_t)t;
                if ((c & 31) == 0) p.h_scale[(i * R + row0 + j) * p.h_scale_pitch + f / 32] = (uint8_t)b;
            }
        } else {
            reinterpret_cast<__nv_bfloat16*>(p.h)[(int64_t)(row0 + j) * p.h_cols + f] = __float2bfloat16_rn(h);
        }
    }
}

// A CTA's line of work of a phase: units of ks stages each. Up: a unit is a (chunk, tile of h); down: a
// (output tile, chunk).
struct Line {
    int first, step, units, ks;
    __device__ __forceinline__ int unit(int u) const { return first + u * step; }
    __device__ __forceinline__ int stages() const { return units * ks; }
};

template <bool MX>
__global__ void __launch_bounds__(THREADS, 1) moe_few_kernel(const __grid_constant__ FewParams p) {
    using C = Cfg<MX>;
    constexpr int KV = MX ? 128 : 64;  // values of K in a stage
    constexpr int STAGE = C::STAGE, STAGES = C::STAGES;
    extern __shared__ uint8_t raw_smem[];
    const uint32_t raw = smem_addr(raw_smem), base = (raw + 1023u) & ~1023u;
    uint8_t* gen = raw_smem + (base - raw) + STAGES * STAGE;
    Smem& sm = *reinterpret_cast<Smem*>(gen);
    Routing& rt = sm.r;
    float* sums = reinterpret_cast<float*>(gen + sizeof(Smem));  // down: [T][TILE]
    const uint32_t full0 = smem_addr(sm.full), empty0 = smem_addr(sm.empty), acc_full0 = smem_addr(sm.acc_full),
                   acc_empty0 = smem_addr(sm.acc_empty), done = smem_addr(&sm.done);
    __shared__ volatile int stop;
    // A thread that waits for the other CTAs at the meeting (thread 0) can come back from it apart from its warp, and a
    // copy issued under elect_one() by a warp in two parts is issued twice. Every warp joins again after the meeting;
    // the first four warps are the epilogue's, which issue none.
    const int hw_warp = uniform_warp(), lane = threadIdx.x & 31;
    const int warp = hw_warp < 4 ? FIRST_EPI + hw_warp : hw_warp < SECOND_MMA ? hw_warp - 4 : hw_warp;

    if (threadIdx.x == 0) {
        stop = 0;
        for (int s = 0; s < STAGES; ++s) {
            bar_init(full0 + 8 * s, 2);  // the TMA thread and the stage's feed warp
            bar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(acc_full0 + 8 * b, 2);  // both product warps
            bar_init(acc_empty0 + 8 * b, 4);
        }
        bar_init(done, 2);
        bar_init_fence();
        tma_desc_prefetch(&p.gate);
        tma_desc_prefetch(&p.up);
        tma_desc_prefetch(&p.down);
        tma_desc_prefetch(&p.map_h);
    }
    if (warp == 1) tmem_get(smem_addr(&sm.tmem), TMEM_COLS);
    for (int i = threadIdx.x; i < p.T * TILE; i += THREADS) sums[i] = 0.f;
    fence_before_sync();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < p.tiles; i += THREADS) p.tickets[i] = 0;
    route(rt, p, hw_warp, lane);  // begins and ends with a barrier of the CTA
    fence_after_sync();
    const uint32_t tmem = sm.tmem;

    const int grid = (int)gridDim.x, cta = (int)blockIdx.x;
    const int n_f = (p.h_cols + UP_F - 1) / UP_F, n_chunks = rt.n_chunks;
    Line up, down;
    up.first = cta;
    up.step = grid;
    up.ks = (p.H + KV - 1) / KV;
    up.units = cta < n_chunks * n_f ? (n_chunks * n_f - 1 - cta) / grid + 1 : 0;
    // down: CTA b has share b / tiles of tile b % tiles, or (more tiles than CTAs) whole tiles b, b + grid, ...
    const int share = p.shares > 1 ? cta / p.tiles : 0;
    const int c0 = share * n_chunks / p.shares, own = share < p.shares ? (share + 1) * n_chunks / p.shares - c0 : 0;
    const int out_tiles = p.shares > 1 ? 1 : cta < p.tiles ? (p.tiles - 1 - cta) / grid + 1 : 0;
    down.first = 0;
    down.step = 1;
    down.ks = (p.F + KV - 1) / KV;
    down.units = out_tiles * own;
    auto down_chunk = [&](int u) { return c0 + u % own; };
    auto down_tile = [&](int u) { return p.shares > 1 ? cta % p.tiles : cta + u / own * grid; };
    const int R = p.T * p.k, base_it = up.stages();
    const bool one = elect_one();

    // ---- state of the roles across the meeting
    int s = 0;  // the producer's next stage
    uint32_t phase = 1;  // a new barrier's preceding phase counts as complete
    bool ok = true;
    int acc = 0;                            // accumulators used so far
    auto next_stage = [&] {
        if (++s == STAGES) {
            s = 0;
            phase ^= 1u;
        }
    };
    struct Turn {                           // a feed warp's data of a stage
        uint32_t sp[4], sq;
        uint4 x[MX ? 4 : 2];
    };
    Turn cur;

    // ---- the roles' parts of a phase
    constexpr uint32_t P_COUNT = MX ? P_BYTES / 2 : P_BYTES;  // an unpacking copy counts the packed bytes
    auto load_up = [&](int e, int f0, int k) {
        const uint32_t at = base + s * STAGE, bar = full0 + 8 * s;
        bar_expect(bar, P_COUNT);
        tma_3d(at, &p.gate, bar, k * KV, f0, e);
        tma_3d(at + P_BYTES / 2, &p.up, bar, k * KV, f0, e);
    };
    // the producer's place in down; what a unit needs is looked up once (an integer division of
    // this hardware is as long as a copy's issue)
    struct Place {
        int u, k, e, row, h_row;
    };
    auto place = [&](int u) {
        const int chunk = down_chunk(u);
        return Place{u, 0, rt.chunk_e[chunk], down_tile(u) * TILE, rt.chunk_row[chunk]};
    };
    auto advance = [&](Place& at) {
        if (++at.k == down.ks && at.u + 1 < down.units) at = place(at.u + 1);
    };
    auto load_down = [&](const Place& from) {
        const uint32_t bar = full0 + 8 * s;
        bar_expect(bar, P_COUNT + (MX ? H_TERMS : 1) * TOK * 128);
        if (!MX) bar_arrive(bar);  // no feed warp has anything to add
        tma_3d(base + s * STAGE, &p.down, bar, from.k * KV, from.row, from.e);
    };
    auto load_h = [&](int st, const Place& from) {
        const uint32_t at = base + st * STAGE + P_BYTES, bar = full0 + 8 * st;
        if (MX) tma_3d(at, &p.map_h, bar, from.k * KV, from.h_row, 0);
        else tma_2d(at, &p.map_h, bar, from.k * KV, from.h_row);
    };
    auto wait_empty = [&] {
        if (ok && !bar_wait_warp(empty0 + 8 * s, phase, p.err, 1)) {
            ok = false;
            stop = 1;
        }
        return ok;
    };
    // Stages `first` on of the ring's line: this warp's are the even or the odd ones, so that a place in the ring is
    // always the same warp's (its wait by parity for a round follows its wait for the round before).
    auto products = [&](const Line& line, int first, uint32_t idesc) {
        const int odd = warp == 1 ? 0 : 1;
        for (int u = 0; ok && u < line.units; ++u, ++acc, first += line.ks) {
            const int b = acc & 1;
            if (!bar_wait_warp(acc_empty0 + 8 * b, (uint32_t)((acc >> 1) + 1) & 1u, p.err, 2) || stop) {
                ok = false;
                stop = 1;
                break;
            }
            fence_after_sync();
            const uint32_t d = tmem + (uint32_t)((2 * b + odd) * C::Q_ROWS);
            uint32_t add = 0;
            for (int i = first + ((first ^ odd) & 1); i < first + line.ks; i += 2) {
                const int st = i % STAGES;
                if (!bar_wait_warp(full0 + 8 * st, (uint32_t)(i / STAGES) & 1u, p.err, 3)) {
                    ok = false;
                    stop = 1;
                    break;
                }
                fence_after_sync();
                const uint32_t sp = base + st * STAGE, sq = sp + P_BYTES, sc = sq + C::Q_BYTES;
                const uint32_t tp = tmem + (uint32_t)(4 * C::Q_ROWS + st * 8);
                if (one) {
                    if (MX) {
                        scale_copy(tp, scale_desc(sc));
                        scale_copy(tp + 4, scale_desc(sc + 512));
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {  // 32 bytes of each row
                        if (MX) mma_mxf8(d, operand_desc(sp + 32 * j), operand_desc(sq + 32 * j), idesc_at(idesc, j), tp, tp + 4, j ? 1u : add);
                        else mma_bf16(d, operand_desc(sp + 32 * j), operand_desc(sq + 32 * j), idesc, j ? 1u : add);
                    }
                    mma_commit(empty0 + 8 * st);
                }
                __syncwarp();
                add = 1;
            }
            if (ok && one) mma_commit(acc_full0 + 8 * b);
            __syncwarp();
        }
    };
    // the scales of a stage of 128 weight rows, lane l with rows l, l + 32, l + 64, l + 96; and in down those of h
    auto fetch_up = [&](Turn& to, int i) {
        if (i >= up.stages()) return;
        const int u = i / up.ks, k = i - u * up.ks, unit = up.unit(u), chunk = unit / n_f, f0 = unit % n_f * UP_F;
        const int e = rt.chunk_e[chunk], n = rt.chunk_n[chunk], row0 = rt.chunk_row[chunk];
        if (MX) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int f = f0 + ((lane + 32 * j) & (UP_F - 1));
                to.sp[j] = f < p.F ? __ldg(reinterpret_cast<const uint32_t*>((j < 2 ? p.gate_scale : p.up_scale) + e * p.up_scale_stride +
                                                                             (int64_t)f * p.up_scale_pitch + 4 * k))
                                   : 0u;
            }
        }
#pragma unroll
        for (int j = 0; j < (MX ? 4 : 2); ++j) {
            // MXFP4: 16 pieces of a token's 128 values, two tokens at a time; bf16: 8 of 64, four
            const int tok = MX ? (lane >> 4) + 2 * j : (lane >> 3) + 4 * j, at = k * KV + 8 * (MX ? lane & 15 : lane & 7);
            to.x[j] = tok < n && at < p.H  // H is a multiple of 8
                          ? __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)rt.row_t[row0 + tok] * p.H + at))
                          : make_uint4(0, 0, 0, 0);
        }
    };
    auto fetch_down = [&](Turn& to, int i, bool weights, bool h) {
        if (i >= down.stages()) return;
        const int u = i / down.ks, k = i - u * down.ks, chunk = down_chunk(u), e = rt.chunk_e[chunk];
        if (weights)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = down_tile(u) * TILE + lane + 32 * j;
                to.sp[j] = row < p.H ? __ldg(reinterpret_cast<const uint32_t*>(p.down_scale + e * p.down_scale_stride +
                                                                               (int64_t)row * p.down_scale_pitch + 4 * k))
                                     : 0u;
            }
        if (h)  // lane: term lane / 8 of row lane % 8
            to.sq = lane < H_TERMS * TOK && (lane & 7) < rt.chunk_n[chunk]
                        ? __ldcg(reinterpret_cast<const uint32_t*>(p.h_scale + ((int64_t)(lane >> 3) * R + rt.chunk_row[chunk] + (lane & 7)) * p.h_scale_pitch + 4 * k))
                        : 0u;
    };
    auto feed_wait = [&](int it) {
        if (!bar_wait_warp(empty0 + 8 * (it % STAGES), (uint32_t)(it / STAGES + 1) & 1u, p.err, 7)) {
            ok = false;
            stop = 1;
        }
        return ok;
    };
    auto feed_done = [&](int it) {
        fence_smem_async();
        __syncwarp();
        if (lane == 0) bar_arrive(full0 + 8 * (it % STAGES));
    };
    const int q = hw_warp, row = q * 32 + lane;  // the epilogue: the TMEM lane quarter that a warp can read
    bool bad = false;                              // a wait ran out: no later one is made, and the results are void
    // the sums of a unit of ks stages, `first` on
    auto take = [&](float (&v)[TOK], int terms, int first, int ks) {
        const int b = acc & 1;
        const uint32_t t = tmem + ((uint32_t)(q * 32) << 16) + 2 * b * C::Q_ROWS;
        if (!bad) bad = !bar_wait_warp(acc_full0 + 8 * b, (uint32_t)(acc >> 1) & 1u, p.err, 4);
        if (bad) stop = 1;
        fence_after_sync();
        uint32_t x[H_TERMS][8], y[H_TERMS][8];
#pragma unroll
        for (int i = 0; i < H_TERMS; ++i)
            if (i < terms) {
                tmem_load8(t + i * TOK, x[i]);
                tmem_load8(t + C::Q_ROWS + i * TOK, y[i]);
            }
        tmem_load_wait();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) bar_arrive(acc_empty0 + 8 * b);
        ++acc;
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
            v[j] = 0.f;
#pragma unroll
            for (int i = H_TERMS - 1; i >= 0; --i)  // the smallest first
                if (i < terms) {
                    const float even = __uint_as_float(x[i][j]), odd = __uint_as_float(y[i][j]);
                    v[j] += ks > 1 ? even + odd : first & 1 ? odd : even;
                }
        }
    };

    // ---- up
    int it = 0;     // the producer's stages so far
    int ahead = 0;  // stages of down whose weights are requested before the meeting
    Place w_at{}, h_at{};
    if (warp == 0) {
        for (int u = 0; ok && u < up.units; ++u) {
            const int unit = up.unit(u), e = rt.chunk_e[unit / n_f], f0 = unit % n_f * UP_F;
            for (int k = 0; k < up.ks && wait_empty(); ++k, ++it) {
                if (one) load_up(e, f0, k);
                __syncwarp();
                next_stage();
            }
        }
        if (down.units) w_at = h_at = place(0);
        for (; ahead < min(STAGES, down.stages()) && wait_empty(); ++ahead, ++it) {
            if (one) load_down(w_at);
            __syncwarp();
            advance(w_at);
            next_stage();
        }
    } else if (warp == 1 || warp == SECOND_MMA) {
        products(up, 0, MX ? mx_idesc(5, 0, TILE, 16) : bf16_idesc(TILE, 16));
    } else if (warp < FIRST_EPI) {
        // a turn is every eighth stage; the next turn's data are requested before this one's work
        Turn nxt;
        const int w = warp - 2;
        fetch_up(cur, w);
        for (int i = w; ok && i < up.stages(); i += FEED_WARPS) {
            fetch_up(nxt, i + FEED_WARPS);
            if (!feed_wait(i)) break;
            const uint32_t sq = base + i % STAGES * STAGE + P_BYTES, sc = sq + C::Q_BYTES;
            if (MX) st_shared4(sc + 16 * lane, cur.sp[0], cur.sp[1], cur.sp[2], cur.sp[3]);
            const int n = rt.chunk_n[up.unit(i / up.ks) / n_f];
#pragma unroll
            for (int j = 0; j < (MX ? 4 : 2); ++j) {
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
            feed_done(i);
            cur = nxt;
        }
        // the weights' scales of this warp's first turn of down: the first stage it with it % 8 = w
        if (MX) fetch_down(cur, ((w - base_it) % FEED_WARPS + FEED_WARPS) % FEED_WARPS, true, false);
    } else if (warp < SECOND_MMA) {
        for (int u = 0; u < up.units; ++u) {
            float v[TOK];
            take(v, MX ? X_TERMS : 1, u * up.ks, up.ks);
#pragma unroll
            for (int j = 0; j < TOK; ++j) sm.turn[row][j] = v[j];
            asm volatile("bar.sync 1, 128;" ::: "memory");
            const int unit = up.unit(u), chunk = unit / n_f;
            write_h<MX>(p, sm, (int)threadIdx.x, rt.chunk_row[chunk], rt.chunk_n[chunk], unit % n_f * UP_F);
            asm volatile("bar.sync 1, 128;" ::: "memory");
        }
        // h is read by tensor copies of other CTAs
        asm volatile("fence.proxy.async;" ::: "memory");
    }

    // ---- the meeting: h is complete
    __syncwarp();
    cooperative_groups::this_grid().sync();
    __syncwarp();  // whichever thread the barrier lets poll: what follows is issued by whole warps

    // ---- down
    if (warp == 0) {
        asm volatile("fence.proxy.async;" ::: "memory");
        for (int i = 0; i < ahead; ++i) {
            if (one) load_h((base_it + i) % STAGES, h_at);
            __syncwarp();
            advance(h_at);
        }
        for (int i = ahead; i < down.stages() && wait_empty(); ++i, ++it) {
            if (one) {
                load_down(w_at);
                load_h(s, w_at);
            }
            __syncwarp();
            advance(w_at);
            next_stage();
        }
        if (stop)  // an aborted CTA waits for its own copies before it exits
            for (int i = 0; i < STAGES && i < it; ++i) {
                const int last = it - 1 - (it - 1 - i) % STAGES;
                bar_wait(full0 + 8 * i, (uint32_t)(last / STAGES) & 1u, p.err, 5);
            }
    } else if (warp == 1 || warp == SECOND_MMA) {
        products(down, base_it, MX ? mx_idesc(5, 0, TILE, 32) : bf16_idesc(TILE, 16));
        if (one) mma_commit(done);
        __syncwarp();
        bar_wait(done, 0, p.err, 6);
    } else if (warp < FIRST_EPI) {
        if (MX) {
            Turn nxt;
            const int i0 = ((warp - 2 - base_it) % FEED_WARPS + FEED_WARPS) % FEED_WARPS;
            fetch_down(cur, i0, false, true);
            for (int i = i0; ok && i < down.stages(); i += FEED_WARPS) {
                fetch_down(nxt, i + FEED_WARPS, true, true);
                if (!feed_wait(base_it + i)) break;
                const uint32_t sc = base + (base_it + i) % STAGES * STAGE + P_BYTES + C::Q_BYTES;
                st_shared4(sc + 16 * lane, cur.sp[0], cur.sp[1], cur.sp[2], cur.sp[3]);
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(sc + 512 + 16 * lane), "r"(cur.sq) : "memory");
                feed_done(base_it + i);
                cur = nxt;
            }
        }
    } else if (warp < SECOND_MMA) {
        auto write_tile = [&](int tile) {  // a thread has a row of its own: no barrier
            const int r = tile * TILE + row;
            for (int t = 0; t < p.T; ++t) {
                const int64_t at = (int64_t)t * p.H + r;
                if (r < p.H) {
                    const float o = sums[t * TILE + row] + (p.resid ? p.resid[at] : __bfloat162float(p.x[at]));
                    p.out[at] = __float2bfloat16_rn(o);
                    if (p.out32) p.out32[at] = o;
                }
                sums[t * TILE + row] = 0.f;
            }
        };
        for (int u = 0; u < down.units; ++u) {
            float v[TOK];
            take(v, MX ? H_TERMS : 1, base_it + u * down.ks, down.ks);
            const int chunk = down_chunk(u), n = rt.chunk_n[chunk], row0 = rt.chunk_row[chunk];
#pragma unroll
            for (int j = 0; j < TOK; ++j)
                if (j < n) {
                    float* to = sums + rt.row_t[row0 + j] * TILE + row;
                    *to = fmaf(rt.row_w[row0 + j], v[j], *to);
                }
            if (p.shares == 1 && (u + 1) % own == 0) write_tile(down_tile(u));
        }
        if (p.shares == 1 && own == 0)  // no token has an expert
            for (int i = 0; i < out_tiles; ++i) write_tile(cta + i * grid);
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        tmem_free(tmem, TMEM_COLS);
    }
    if (p.shares == 1 || share >= p.shares) return;

    // ---- the sums of a tile's shares: its CTAs meet, and each adds a part of the outputs, in their order
    const int tile = cta % p.tiles;
    float* part = p.partial + (int64_t)tile * p.shares * p.T * TILE;
    for (int i = 4 * (int)threadIdx.x; i < p.T * TILE; i += 4 * THREADS)
        *reinterpret_cast<float4*>(part + (int64_t)share * p.T * TILE + i) = *reinterpret_cast<const float4*>(sums + i);
    __syncthreads();
    if (threadIdx.x == 0) {  // a release and an acquire by one thread, between barriers of the CTA, order every thread's parts
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.tickets + tile) : "memory");
        const uint64_t t0 = globaltimer_ns();
        uint32_t met = 0;
        while (!(met = ld_acquire_gpu(p.tickets + tile) == (uint32_t)p.shares) && globaltimer_ns() - t0 < WAIT_LIMIT_NS) {}
        if (!met) raise_error(p.err, DERR_GEMM_TIMEOUT | (10u << 8));
        sm.met = met;
    }
    __syncthreads();
    if (!sm.met) return;
    for (int i = 4 * (share * THREADS + (int)threadIdx.x); i < p.T * TILE; i += 4 * p.shares * THREADS) {
        const int t = i / TILE, r = tile * TILE + i % TILE;
        if (r >= p.H) continue;  // H is a multiple of 8
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c0 = 0; c0 < p.shares; c0 += 8) {
            float4 v[8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c0 + c < p.shares) v[c] = __ldcg(reinterpret_cast<const float4*>(part + (int64_t)(c0 + c) * p.T * TILE + i));
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c0 + c < p.shares) {
                    sum.x += v[c].x;
                    sum.y += v[c].y;
                    sum.z += v[c].z;
                    sum.w += v[c].w;
                }
        }
        const float o[4] = {sum.x, sum.y, sum.z, sum.w};
        const int64_t at = (int64_t)t * p.H + r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float v = o[j] + (p.resid ? p.resid[at + j] : __bfloat162float(p.x[at + j]));
            p.out[at + j] = __float2bfloat16_rn(v);
            if (p.out32) p.out32[at + j] = v;
        }
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

template <bool MX>
cudaError_t launch(const FewParams& p, int grid, cudaStream_t s) {
    auto kern = moe_few_kernel<MX>;
    static SmemAllowance allowed;
    const cudaError_t e = allowed.ensure(reinterpret_cast<const void*>(kern), smem_bytes<MX>(MAX_T));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem_bytes<MX>(p.T);
    cfg.stream = s;
    cudaLaunchAttribute at[1];  // programmatic stream serialization changes nothing for a cooperative launch (measured)
    at[0].id = cudaLaunchAttributeCooperative;
    at[0].val.cooperative = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// Columns of a row of h: whole stages of the down kernel's K, and whole tiles of the up kernel.
int few_h_cols(bool mx, int F) { return mx ? (F + 127) / 128 * 128 : (F + 63) / 64 * 64; }
int64_t few_h_bytes(bool mx, int64_t rows, int F) {
    return (rows * few_h_cols(mx, F) * (mx ? H_TERMS : 2) + 255) / 256 * 256;
}

}  // namespace

// Output tiles of H rows, and the CTAs that share one: as many as the SMs hold, no more than rows.
static void few_shares(int T, int k, int H, int& tiles, int& shares) {
    tiles = (H + TILE - 1) / TILE;
    shares = std::max(1, std::min({MAX_SHARES, gemm_num_sms() / tiles, T * k}));
}

int64_t moe_few_ws_bytes(bool mx, int T, int k, int H, int F) {
    const int64_t rows = (int64_t)T * k;
    int tiles, shares;
    few_shares(T, k, H, tiles, shares);
    return few_h_bytes(mx, rows, F) + (mx ? (H_TERMS * rows * mx_scale_pitch(F) + 255) / 256 * 256 : 0) +
           (4ll * tiles + 255) / 256 * 256 + (shares > 1 ? (int64_t)tiles * shares * T * TILE * 4 : 0);
}

cudaError_t launch_moe_few(const MoeFewDesc& d, void* ws, uint32_t* err, cudaStream_t s) {
    if (d.T <= 0) return cudaSuccess;
    if (d.T > MAX_T || d.E < 1 || d.E > MAX_E || d.k < 1 || d.k > MAX_K || d.k > d.E) return cudaErrorInvalidValue;
    FewParams p;
    memset(&p, 0, sizeof(p));
    const int64_t rows = (int64_t)d.T * d.k;
    const int64_t up_pitch = d.mx ? mx_code_pitch(d.H) : 2ll * d.H, down_pitch = d.mx ? mx_code_pitch(d.F) : 2ll * d.F;
    p.gate_scale = static_cast<const uint8_t*>(d.gate_scales);
    p.up_scale = static_cast<const uint8_t*>(d.up_scales);
    p.down_scale = static_cast<const uint8_t*>(d.down_scales);
    p.up_scale_stride = d.gate_scale_stride;
    p.down_scale_stride = d.down_scale_stride;
    p.up_scale_pitch = (int)mx_scale_pitch(d.H);
    p.down_scale_pitch = p.h_scale_pitch = (int)mx_scale_pitch(d.F);
    p.x = static_cast<const __nv_bfloat16*>(d.x);
    p.resid = d.resid;
    p.logits = d.logits;
    p.h_cols = few_h_cols(d.mx, d.F);
    few_shares(d.T, d.k, d.H, p.tiles, p.shares);
    uint8_t* w = static_cast<uint8_t*>(ws);
    p.h = w;
    w += few_h_bytes(d.mx, rows, d.F);
    p.h_scale = w;
    w += d.mx ? (H_TERMS * rows * p.h_scale_pitch + 255) / 256 * 256 : 0;
    p.tickets = reinterpret_cast<uint32_t*>(w);
    w += (4ll * p.tiles + 255) / 256 * 256;
    p.partial = reinterpret_cast<float*>(w);
    p.T = d.T;
    p.E = d.E;
    p.k = d.k;
    p.H = d.H;
    p.F = d.F;
    p.out = static_cast<__nv_bfloat16*>(d.out);
    p.out32 = d.out32;
    p.err = err;
    if (!map_experts(&p.gate, d.mx, d.gate, up_pitch, d.F, d.E, d.gate_stride, UP_F) ||
        !map_experts(&p.up, d.mx, d.up, up_pitch, d.F, d.E, d.gate_stride, UP_F) ||
        !map_experts(&p.down, d.mx, d.down, down_pitch, d.H, d.E, d.down_stride, TILE) ||
        !map_h(&p.map_h, d.mx, p.h, rows, p.h_cols))
        return cudaErrorInvalidValue;
    // no more CTAs than either phase can use: up has at most rows x (h_cols / 64) tiles
    const int64_t most = std::max<int64_t>(rows * (p.h_cols / UP_F), (int64_t)p.tiles * p.shares);
    const int grid = (int)std::min<int64_t>(most, gemm_num_sms());
    return d.mx ? launch<true>(p, grid, s) : launch<false>(p, grid, s);
}

}  // namespace ls
