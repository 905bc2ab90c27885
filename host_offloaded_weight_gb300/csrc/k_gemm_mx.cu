// C[M,N] = sum_k A[m,k] B[n,k] with A bf16 and B MXFP4 on the sm_103a tensor cores (kind::mxf8f6f4, block-scaled),
// for few rows of A (tokens). The weights are the left operand (128 rows a tile) and the tokens the right one, so a
// single token costs 16 columns instead of 128 padded rows. The tensor core has no bf16 x E2M1 form; a bf16 value
// has 8 significant bits and an E4M3 value 4, so A is written as two E4M3 terms with a power-of-two scale for each
// block of 32:
//   a = t1 2^s1 + t2 2^s2,  s1 = floor(log2 max|a|) - 7,  s2 = s1 - 5.
// t1 is a 2^-s1 to the nearest, t2 the rest: exact for every value down to 2^-13 of its block's largest, below that
// within 2^-22 of the largest. (A block that reaches 2^127: t1 is cut, so that t1 2^s1 stays finite, s2 = s1 - 4, and the
// smallest values are within 2^-21.) Both terms are columns of the same product and are added in fp32 in the epilogue.
//
// Structure (one persistent CTA per SM): warp 0 loads the weights by TMA, which unpacks them to a byte a value
// (128-byte rows, 128-byte swizzle), into a ring of stages; the warps after warp 1 bring the scales into the stage
// in the order that the tensor core reads them (32 rows of 16 bytes, the four 32-row groups side by side), and, up to
// 8 tokens, the tokens' terms themselves (more come from memory by TMA, split by a kernel before). One or two warps
// copy the scales to TMEM and issue the products; four write the results. The scales' TMEM columns belong to the
// stage, so the barrier that frees a stage orders their reuse too.
//
// Few tiles are shared along K by a cluster of CTAs, each of which adds the sums of every so many tokens, out of its
// shared memory. Sums are fp32 and each output is written by one thread from a fixed order of sums.
//
// What bounds it: the tensor core's reads of shared memory. Unpacked weights are 4 KB a product of K = 32 however few
// the columns: a stage takes 263 clocks with 16 columns and 362 with 64, about 68 bytes a clock, where its bytes from
// memory would take 175 of a busy SM's share; and tiles of 128 rows leave SMs without one (13824 rows: 108 of 152).
// 1 token through 13824 x 5120 takes 9.9 us (3.8 TB/s), 32 tokens through 5120 x 13824 15.2 us, of which the split
// kernel, the launch and the first load are 6. Many rows are not what it is for: through 13824 x 5120, 128 rows take 23
// us, 512 59, 1024 117 and 2048 234, where reading the weights back and the bf16 product take 65, 82, 107 and 180.
#include <algorithm>
#include <mutex>

#include "kernels.h"
#include "tc.cuh"

namespace ls {
namespace {

using namespace tc;

// ACT: the right operand is the split rows in memory.
// ACT_IN: up to 8 bf16 rows, split by the scale warps on their way into each stage (16 rows so took 16.9 us through
// 13824 x 5120, with a split kernel before 13.4; 8 rows 11.8).
enum { ACT = 1, ACT_IN = 2 };

constexpr int TILE_P = 128;               // rows of the left operand in a tile
constexpr int P_BYTES = TILE_P * 128;     // a stage of it

template <int MODE, int BQ>
struct Cfg {
    static constexpr int TN = BQ / 2;                          // tokens of a tile (two terms each)
    static constexpr int PARTS = (BQ + 127) / 128;             // 128-row parts of the right operand's scales
    static constexpr int Q_BYTES = BQ * 128;
    static constexpr int SCALE_BYTES = (1 + PARTS) * 512;
    static constexpr int STAGE = (P_BYTES + Q_BYTES + SCALE_BYTES + 1023) / 1024 * 1024;
    static constexpr int EPI_WARPS = MODE == ACT ? 8 : 4;  // ACT: 64 tokens through 13824 x 5120 from four warps 22.0 us, eight 20.0
    // CTAs that may share a tile along K, and the room for the others' sums of this one's tokens
    static constexpr int MAX_SPLIT = TN == 8 ? 8 : TN <= 32 ? 4 : TN == 64 ? 2 : 1;
    static constexpr int RED_BYTES = (MAX_SPLIT - 1) * TN * TILE_P * 4;
    // Up to 128 columns a stage's products are as short as an issuing warp's waits between them: two warps
    // take the even and the odd stages, each with an accumulator of its own.
    static constexpr int MMA_WARPS = BQ <= 128 ? 2 : 1;
    static constexpr int FIT = (232448 - 1024 - 512 - RED_BYTES) / STAGE, MOST = FIT < 10 ? FIT : 10;
    // The scale warps work in teams that take turns of RUN stages. A wait by parity cannot tell a phase from the
    // one two before it. Where one warp issues the products, stages are freed in order, and turns within a
    // round of the ring are enough; where two do, each place in the ring has a team and a product warp of its own.
    static constexpr int TEAM = MODE == ACT_IN ? 1 : 2;                     // warps of a team
    static constexpr int TEAMS = MODE == ACT_IN ? MOST / 2 * 2 : 2;
    static constexpr int RUN = MMA_WARPS == 2 ? 1 : 2;
    static constexpr int STAGES = MOST / TEAMS * TEAMS;
    static_assert(MMA_WARPS == 2 ? RUN == 1 && STAGES % TEAMS == 0 && STAGES % 2 == 0 : TEAMS * RUN <= STAGES,
                  "turns of the scale and the product warps");
    static constexpr int SCALE_WARPS = TEAM * TEAMS;
    static constexpr int SMEM = STAGES * STAGE + RED_BYTES + 1024 + 512;
    static constexpr int FIRST_EPI = 2 + SCALE_WARPS;            // the first warp of the epilogue
    static constexpr int SECOND_MMA = FIRST_EPI + EPI_WARPS;
    static constexpr int THREADS = 32 * (SECOND_MMA + MMA_WARPS - 1);
    static constexpr int ACC = MMA_WARPS * BQ;  // columns of an accumulator
    static constexpr int ACCS = 2 * ACC + STAGES * 4 * (1 + PARTS) <= 512 ? 2 : 1;
    static constexpr int SCALE_COLS = 4 * (1 + PARTS);  // TMEM columns of a stage's scales
    static_assert(ACCS * ACC + STAGES * SCALE_COLS <= 512, "tensor memory");
    static_assert(BQ % 16 == 0 && BQ <= 256, "columns of a product");
};

struct MxParams {
    CUtensorMap map_p, map_q;
    const uint8_t* scale_p;
    const uint8_t* scale_q;
    int scale_pitch;
    int rows_p, rows_q;   // rows of the weights; tokens
    int q_term_rows;      // ACT: rows between the two terms
    int k_stages;         // stages along K (128 values)
    int tiles_p, tiles_q, tiles;
    int splits;           // CTAs (a cluster) that share a tile along K
    const __nv_bfloat16* a;  // ACT_IN: the rows themselves
    int64_t lda;
    int K, vec;
    void* C;
    int64_t ldc;
    int c_f32;
    uint32_t* err;
};

// The tiles of a CTA, in order, and its stages of each: with splits > 1 a cluster has one tile,
// and its CTAs a run of whole scale groups each.
struct Work {
    int tile, step, tiles, k0, k1;
    __device__ __forceinline__ Work(const MxParams& p) {
        const int slice = (int)blockIdx.x % p.splits, groups = (p.k_stages + 3) / 4;  // 16 bytes of scales
        step = (int)gridDim.x / p.splits;
        tile = (int)blockIdx.x / p.splits - step;
        tiles = p.tiles;
        k0 = (int)((int64_t)slice * groups / p.splits) * 4;
        k1 = min(p.k_stages, (int)((int64_t)(slice + 1) * groups / p.splits) * 4);
    }
    __device__ __forceinline__ bool next() {
        tile += step;
        return tile < tiles;
    }
};

// The token tiles of one weight tile follow one another.
template <int BQ>
__device__ __forceinline__ void tile_at(const MxParams& p, int tile, int& row_p, int& row_q) {
    row_p = tile / p.tiles_q * TILE_P;
    row_q = tile % p.tiles_q * (BQ / 2);
}

// Eight tokens' sums of a weight row (an output column), tokens from `token` on.
__device__ __forceinline__ void store_tokens(const MxParams& p, int col, int token, const float (&v)[8]) {
    if (col >= p.rows_p) return;
    const int64_t at = (int64_t)token * p.ldc + col;
    if (p.c_f32) {
        float* c = static_cast<float*>(p.C) + at;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (token + j < p.rows_q) c[j * p.ldc] = v[j];
    } else {
        __nv_bfloat16* c = static_cast<__nv_bfloat16*>(p.C) + at;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (token + j < p.rows_q) c[j * p.ldc] = __float2bfloat16_rn(v[j]);
    }
}

__device__ __forceinline__ uint32_t word_of(uint32_t v, int) { return v; }
__device__ __forceinline__ uint32_t word_of(const uint2& v, int i) { return i == 0 ? v.x : v.y; }
__device__ __forceinline__ void load_words(const uint8_t* p, bool in, uint2& v) {
    v = in ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0, 0);
}
__device__ __forceinline__ void load_words(const uint8_t* p, bool in, uint32_t& v) {
    v = in ? __ldg(reinterpret_cast<const uint32_t*>(p)) : 0u;
}
template <int BYTES> struct Words;
template <> struct Words<4> { typedef uint32_t type; };
template <> struct Words<8> { typedef uint2 type; };

// A row's sums for tokens j0 to j0 + 7 of a tile of ks stages, `first` on: the smaller terms first, of even and odd stages.
template <int MODE, int BQ>
__device__ __forceinline__ void token_sums(uint32_t t, int j0, int first, int ks, float (&v)[8]) {
    using C = Cfg<MODE, BQ>;
    constexpr int N = C::MMA_WARPS;
    uint32_t x[N][8], y[N][8];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        tmem_load8(t + i * BQ + j0, x[i]);
        tmem_load8(t + i * BQ + C::TN + j0, y[i]);
    }
    tmem_load_wait();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float x0 = __uint_as_float(x[0][j]), x1 = __uint_as_float(x[N - 1][j]);
        const float y0 = __uint_as_float(y[0][j]), y1 = __uint_as_float(y[N - 1][j]);
        if (N == 1) v[j] = y0 + x0;
        else v[j] = ks > 1 ? (y0 + y1) + (x0 + x1) : first & 1 ? y1 + x1 : y0 + x0;
    }
}

template <int MODE, int BQ>
__global__ void __launch_bounds__(Cfg<MODE, BQ>::THREADS, 1) gemm_mx_kernel(const __grid_constant__ MxParams p) {
    using C = Cfg<MODE, BQ>;
    constexpr int S = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t bars = base + S * C::STAGE + C::RED_BYTES;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (S + s); };
    auto acc_full = [&](int b) { return bars + 8u * (2 * S + b); };
    auto acc_empty = [&](int b) { return bars + 8u * (2 * S + 2 + b); };
    const uint32_t done = bars + 8u * (2 * S + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (bars - base) + 8 * (2 * S + 5));
    __shared__ volatile int stop;
    const int warp = uniform_warp(), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        stop = 0;
        for (int s = 0; s < S; ++s) {
            bar_init(full(s), 1 + C::TEAM);  // the TMA thread and a team of scale warps
            bar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(acc_full(b), C::MMA_WARPS);
            bar_init(acc_empty(b), C::EPI_WARPS);
        }
        bar_init(done, C::MMA_WARPS);
        bar_init_fence();
        tma_desc_prefetch(&p.map_p);
        if (MODE != ACT_IN) tma_desc_prefetch(&p.map_q);
    }
    if (warp == 1) tmem_get(smem_addr(tmem_slot), 512);
    fence_before_sync();
    __syncwarp();
    if (p.splits > 1) cluster_barrier();
    else __syncthreads();
    fence_after_sync();
    // ACT: the kernel before this one, which splits the rows, began after everything earlier was
    // complete, so only the split rows have to be waited for; the weights start at once
    if (MODE != ACT) grid_wait();
    const uint32_t tmem = *tmem_slot;
    Work w(p);
    // the epilogue's warps: the TMEM lane quarter that a warp can read, and which of a quarter's warps it is
    constexpr int HALVES = C::EPI_WARPS / 4;
    const int q = warp & 3, half = (warp - C::FIRST_EPI) >> 2, slice = (int)blockIdx.x % p.splits;

    if (warp == 0) {
        // ------------------------------------------------------------ operand tiles
        const bool one = elect_one();
        int s = 0, it = 0;
        uint32_t phase = 1;  // a new barrier's preceding phase counts as complete
        bool ok = true;
        // an unpacking copy counts the packed bytes (it leaves every second 8 bytes alone)
        constexpr uint32_t BYTES = MODE == ACT ? P_BYTES / 2 + C::Q_BYTES : P_BYTES / 2;
        auto load_q = [&](int st, int k, int row_q) {
            const uint32_t at = base + st * C::STAGE + P_BYTES;
            if (MODE == ACT) tma_3d(at, &p.map_q, full(st), k * 128, row_q, 0);  // both terms
        };
        while (ok && w.next()) {
            int row_p, row_q, k = w.k0;
            tile_at<BQ>(p, w.tile, row_p, row_q);
            if (MODE == ACT && it == 0) {
                const int ahead = min(S, w.k1 - w.k0);
                if (one)
                    for (int i = 0; i < ahead; ++i) {
                        bar_expect(full(i), BYTES);
                        tma_2d(base + i * C::STAGE, &p.map_p, full(i), (k + i) * 128, row_p);
                    }
                grid_wait();
                if (one)
                    for (int i = 0; i < ahead; ++i) load_q(i, k + i, row_q);
                __syncwarp();
                it = ahead;
                k += ahead;
                s = ahead % S;
                phase ^= ahead == S ? 1u : 0u;
            }
            for (; k < w.k1; ++k, ++it) {
                if (!bar_wait_warp(empty(s), phase, p.err, 1)) {
                    ok = false;
                    stop = 1;
                    break;
                }
                if (one) {
                    bar_expect(full(s), BYTES);
                    tma_2d(base + s * C::STAGE, &p.map_p, full(s), k * 128, row_p);
                    load_q(s, k, row_q);
                }
                __syncwarp();
                if (++s == S) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
        grid_release();
        // an aborted CTA waits for its own copies before it exits
        if (stop)
            for (int i = 0; i < S && i < it; ++i) {
                const int last = it - 1 - (it - 1 - i) % S;
                bar_wait(full(i), (uint32_t)(last / S) & 1u, p.err, 5);
            }
    } else if (warp == 1 || (C::MMA_WARPS == 2 && warp == C::SECOND_MMA)) {
        // ------------------------------------------------------------ products
        constexpr uint32_t IDESC = mx_idesc(5, 0, TILE_P, BQ);
        const bool one = elect_one();
        const int odd = warp == 1 ? 0 : 1;
        int n = 0, it = 0;
        bool ok = true, ready = false;  // ready (one warp): the next stage's barrier, asked before this stage's products
        while (ok && w.next()) {
            const int b = n % C::ACCS;
            if (!bar_wait_warp(acc_empty(b), (uint32_t)(n / C::ACCS + 1) & 1u, p.err, 2) || stop) {
                stop = 1;
                break;
            }
            fence_after_sync();
            const uint32_t d = tmem + (uint32_t)(b * C::ACC + odd * BQ);
            uint32_t add = 0;
            const int end = it + w.k1 - w.k0;  // with two warps, this one's are the even or the odd stages of the ring's line
            for (int i = C::MMA_WARPS == 2 ? it + ((it ^ odd) & 1) : it; i < end; i += C::MMA_WARPS) {
                const int s = i % S;
                if (!__all_sync(0xffffffffu, ready) && !bar_wait_warp(full(s), (uint32_t)(i / S) & 1u, p.err, 3)) {
                    ok = false;
                    stop = 1;
                    break;
                }
                fence_after_sync();
                const uint32_t sp = base + s * C::STAGE, sq = sp + P_BYTES, sc = sq + C::Q_BYTES;
                const uint32_t tp = tmem + (uint32_t)(C::ACCS * C::ACC + s * C::SCALE_COLS), tq = tp + 4;
                if (C::MMA_WARPS == 1) ready = bar_test(full((i + 1) % S), (uint32_t)((i + 1) / S) & 1u);
                if (one) {
                    scale_copy(tp, scale_desc(sc));
#pragma unroll
                    for (int j = 0; j < C::PARTS; ++j) scale_copy(tq + 4 * j, scale_desc(sc + 512 * (1 + j)));
#pragma unroll
                    for (int j = 0; j < 4; ++j)  // 32 bytes of each row
                        mma_mxf8(d, operand_desc(sp + 32 * j), operand_desc(sq + 32 * j), idesc_at(IDESC, j), tp, tq, j ? 1u : add);
                    mma_commit(empty(s));
                }
                __syncwarp();
                add = 1;
            }
            if (ok && one) mma_commit(acc_full(b));
            __syncwarp();
            ++n;
            it = end;
        }
        if (one) mma_commit(done);
        __syncwarp();
        bar_wait(done, 0, p.err, 6);
    } else if (warp < C::FIRST_EPI) {
        // ------------------------------------------------------------ scales (and ACT_IN: the rows)
        // Teams take turns, so that the latencies of several stages' waits, stores and fences
        // overlap; a team requests later turns' scales before it starts one. A
        // team's warps share the rows: of each 128, lane l has rows l + 32 j, whose words lie side by
        // side at 16 l in the order that the tensor core reads.
        constexpr int RUN = C::RUN, TEAMS = C::TEAMS, RPW = 4 / C::TEAM;   // rows of a warp, of each 128
        constexpr int NR = RPW * (MODE == ACT_IN ? 1 : 1 + C::PARTS);
        constexpr int AHEAD = MODE == ACT && RUN == 1 ? 3 : 1;             // turns requested ahead
        constexpr int U = MODE == ACT_IN ? C::TN / 2 : 1;                  // ACT_IN: units of 8 values a lane
        typedef typename Words<4 * RUN>::type V;
        const int team = (warp - 2) / C::TEAM, first = RPW * ((warp - 2) % C::TEAM);
        w.next();
        const int stages = w.k1 - w.k0, turns = (stages + RUN - 1) / RUN;
        int tile = w.tile, u = 0, it0 = 0;                             // the turn at hand
        int f_tile = w.tile, f_u = 0;                                  // the turn to request next
        auto step = [&](int& t, int& v, int& it, int by) {
            for (v += by; v >= turns; v -= turns, t += w.step, it += stages) {}
        };
        V v[AHEAD + 1][NR];
        uint4 x[AHEAD + 1][U];
        const int xg = lane & 15;
        auto fetch = [&](V (&to)[NR], uint4 (&xto)[U], int t, int turn, int j0, int j1) {
            const bool on = t < p.tiles;
            const int k = w.k0 + turn * RUN;
            int row_p = 0, row_q = 0;
            if (on) tile_at<BQ>(p, t, row_p, row_q);
            const int64_t at = 4ll * k;
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                if (j < j0 || j >= j1) continue;
                if (j < RPW) {
                    const int row = row_p + lane + 32 * (first + j);
                    load_words(p.scale_p + (int64_t)row * p.scale_pitch + at, on && row < p.rows_p, to[j]);
                } else {
                    const int rq = lane + 128 * (j / RPW - 1) + 32 * (first + j % RPW);
                    const int64_t row = rq < BQ / 2 ? row_q + rq : (int64_t)row_q + rq - BQ / 2 + p.q_term_rows;
                    load_words(p.scale_q + row * p.scale_pitch + at, on && rq < BQ, to[j]);
                }
            }
            if (MODE == ACT_IN && j0 == 0) {
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    if (2 * i >= p.rows_q) continue;  // columns of tokens that do not exist hold anything
                    const int tok = (lane >> 4) + 2 * i;
                    xto[i] = on && tok < p.rows_q ? row8(p.a + (int64_t)tok * p.lda, k * 128 + 8 * xg, p.K, p.vec)
                                                  : make_uint4(0, 0, 0, 0);
                }
            }
        };
        int none = 0;
        step(tile, u, it0, team);
        step(f_tile, f_u, none, team);
        if (MODE == ACT) {  // the weights' scales need not wait for the split rows
            int t = f_tile, turn = f_u;
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                fetch(v[i], x[i], t, turn, 0, RPW);
                step(t, turn, none, TEAMS);
            }
            grid_wait();
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            fetch(v[i], x[i], f_tile, f_u, MODE == ACT ? RPW : 0, NR);
            step(f_tile, f_u, none, TEAMS);
        }
        bool ok = true;
        while (ok && tile < p.tiles) {
            fetch(v[AHEAD], x[AHEAD], f_tile, f_u, 0, NR);
            step(f_tile, f_u, none, TEAMS);
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                if (!ok || u * RUN + i >= stages) continue;
                const int it = it0 + u * RUN + i, s = it % S;
                if (!bar_wait_warp(empty(s), (uint32_t)(it / S + 1) & 1u, p.err, 7)) {
                    ok = false;
                    stop = 1;
                    continue;
                }
                const uint32_t sq = base + s * C::STAGE + P_BYTES, sc = sq + C::Q_BYTES, at = sc + lane * 16 + 4 * first;
#pragma unroll
                for (int j = 0; j < NR / RPW; ++j) {  // the left operand's chunk, then the right one's parts
                    if (RPW == 4)
                        st_shared4(at + 512 * j, word_of(v[0][RPW * j], i), word_of(v[0][RPW * j + 1], i),
                                   word_of(v[0][RPW * j + 2 % RPW], i), word_of(v[0][RPW * j + 3 % RPW], i));
                    else
                        st_shared2(at + 512 * j, word_of(v[0][RPW * j], i), word_of(v[0][RPW * j + 1], i));
                }
                if (MODE == ACT_IN) {
#pragma unroll
                    for (int j = 0; j < U; ++j) {
                        if (2 * j >= p.rows_q) continue;
                        uint2 o1, o2;
                        uint32_t b1, b2;
                        split8(x[0][j], o1, o2, b1, b2);
                        const int r1 = (lane >> 4) + 2 * j, r2 = r1 + C::TN;  // rows of the stage, swizzled 16 bytes
                        const uint32_t col = (uint32_t)((((xg >> 1) ^ (r1 & 7)) << 4) + (xg & 1) * 8);
                        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(sq + r1 * 128 + col), "r"(o1.x), "r"(o1.y) : "memory");
                        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(sq + r2 * 128 + col), "r"(o2.x), "r"(o2.y) : "memory");
                        if ((xg & 3) == 0) {
                            const uint32_t to = sc + 512 + (uint32_t)(xg >> 2);
                            asm volatile("st.shared.u8 [%0], %1;" ::"r"(to + r1 * 16), "r"(b1) : "memory");
                            asm volatile("st.shared.u8 [%0], %1;" ::"r"(to + r2 * 16), "r"(b2) : "memory");
                        }
                    }
                }
                fence_smem_async();
                __syncwarp();
                if (lane == 0) bar_arrive(full(s));
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
#pragma unroll
                for (int j = 0; j < NR; ++j) v[i][j] = v[i + 1][j];
#pragma unroll
                for (int j = 0; j < U; ++j) x[i][j] = x[i + 1][j];
            }
            step(tile, u, it0, TEAMS);
        }
    } else if (warp < C::SECOND_MMA) {
        // ------------------------------------------------------------ results
        int n = 0;
        while (w.next()) {
            int row_p, row_q;
            tile_at<BQ>(p, w.tile, row_p, row_q);
            const int b = n % C::ACCS;
            if (!__all_sync(0xffffffffu, bar_wait(acc_full(b), (uint32_t)(n / C::ACCS) & 1u, p.err, 4) && !stop)) {
                stop = 1;
                break;
            }
            fence_after_sync();
            const uint32_t t = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * C::ACC);
            const int row = q * 32 + lane, groups = (min(C::TN, p.rows_q - row_q) + 7) / 8;
#pragma unroll 1
            for (int g = half; g < groups; g += HALVES) {  // eight tokens
                // a cluster's CTAs take the groups in turn; the others leave their sums in the owner's memory
                const int owner = g % p.splits;
                if (p.splits > 1 && owner == slice) continue;
                float sum[8];
                token_sums<MODE, BQ>(t, 8 * g, n * (w.k1 - w.k0), w.k1 - w.k0, sum);
                if (p.splits == 1) {
                    store_tokens(p, row_p + row, row_q + 8 * g, sum);
                } else {
                    const uint32_t to = cluster_addr(base + S * C::STAGE + ((slice - (slice > owner)) * C::TN + 8 * g) * TILE_P * 4, owner);
#pragma unroll
                    for (int j = 0; j < 8; ++j) st_cluster(to + (j * TILE_P + row) * 4, sum[j]);
                }
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) bar_arrive(acc_empty(b));
            ++n;
        }
    }
    if (p.splits > 1) {
        __syncwarp();
        cluster_barrier();  // the sums are in their owners' memory; they are added in CTA order
        if (warp >= C::FIRST_EPI && warp < C::SECOND_MMA) {
            fence_after_sync();
            int row_p, row_q;
            tile_at<BQ>(p, blockIdx.x / p.splits, row_p, row_q);
            const int row = q * 32 + lane, groups = (min(C::TN, p.rows_q - row_q) + 7) / 8;
            const float* red = reinterpret_cast<const float*>(gbase + S * C::STAGE) + row;
            const uint32_t t = tmem + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
            for (int g = slice + half * p.splits; g < groups; g += HALVES * p.splits) {
                float sum[8];
                token_sums<MODE, BQ>(t, 8 * g, 0, w.k1 - w.k0, sum);
#pragma unroll 1
                for (int i = 0; i < p.splits - 1; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] += red[(i * C::TN + 8 * g + j) * TILE_P];
                store_tokens(p, row_p + row, row_q + 8 * g, sum);
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        tmem_free(tmem, 512);
    }
}

// The two terms of more rows than a stage's warps split on the way: [2][pad rows][pitch] bytes
// and their scales likewise; rows past M are zero. A thread takes 8 values, four lanes a block.
__global__ void __launch_bounds__(256)
split_rows_kernel(const __nv_bfloat16* __restrict__ a, int64_t lda, int M, int K, int vec, int pad_rows, uint32_t per_row,
                  uint8_t* __restrict__ terms, uint8_t* __restrict__ scales, int scale_pitch) {
    grid_wait();
    grid_release();  // everything earlier is complete: the product may start on the weights
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t total = (int64_t)pad_rows * per_row;
    const int row = (int)(i / per_row);
    const uint32_t g = (uint32_t)(i % per_row);
    uint2 o1, o2;
    uint32_t b1, b2;
    split8(i < total && row < M ? row8(a + row * lda, (int)g * 8, K, vec) : make_uint4(0, 0, 0, 0), o1, o2, b1, b2);
    if (i >= total) return;
    reinterpret_cast<uint2*>(terms)[i] = o1;
    reinterpret_cast<uint2*>(terms)[i + total] = o2;
    if ((g & 3) == 0) {
        uint8_t* s1 = scales + (int64_t)row * scale_pitch;
        uint8_t* s2 = s1 + (int64_t)pad_rows * scale_pitch;
        s1[g >> 2] = (uint8_t)b1;
        s2[g >> 2] = (uint8_t)b2;
        if (g + 4 == per_row)
            for (int j = (int)(per_row >> 2); j < scale_pitch; ++j) s1[j] = s2[j] = 0;
    }
}

// ------------------------------------------------------------------ host side
template <int MODE, int BQ>
cudaError_t launch(const MxParams& p, cudaStream_t s) {
    auto kern = gemm_mx_kernel<MODE, BQ>;
    using C = Cfg<MODE, BQ>;
    static SmemAllowance allowed;
    const cudaError_t e = allowed.ensure(reinterpret_cast<const void*>(kern), C::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.splits > 1 ? p.tiles * p.splits : std::min(p.tiles, gemm_num_sms()));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
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

// View [2][rows][pitch bytes] of the split rows, in boxes of 128 bytes x both terms of `tokens`, 128-byte swizzle.
bool map_terms(CUtensorMap* m, const void* ptr, int64_t rows, int64_t pitch, int tokens) {
    const MxEncodeFn fn = mx_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)pitch, (cuuint64_t)rows, 2};
    cuuint64_t strides[2] = {(cuuint64_t)pitch, (cuuint64_t)(rows * pitch)};
    cuuint32_t box[3] = {128, (cuuint32_t)tokens, 2};
    cuuint32_t one[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

// Tokens of a tile: the fewest columns that hold M, at most 128.
int act_tile(int M) { return M <= 8 ? 8 : M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

// CTAs that share a tile along K (a cluster): few tiles leave SMs idle, and joining the sums through shared memory takes
// time of its own, taken as the same for any number of CTAs, since each adds its share of the tokens. In units of a scale
// group (512 values of K, about 0.7 us of an SM's share of the memory): a CTA's groups, one to start, and three to join.
// The three are from the form in which one CTA added all sums (4 us more at 32 tokens) and have not been fitted since;
// with them K up to 2048 is never shared.
int act_splits(int tiles, int groups, int max_split) {
    int best = 1;
    double least = groups + 1.0;
    for (int n = 2; n <= max_split && n <= groups && tiles * n <= gemm_num_sms(); ++n) {
        const double cost = (groups + n - 1) / n + 1.0 + 3.0;
        if (cost < least) {
            least = cost;
            best = n;
        }
    }
    return best;
}

template <int MODE, int BQ>
cudaError_t launch_act(MxParams& p, cudaStream_t s) {
    p.splits = act_splits(p.tiles, (p.k_stages + 3) / 4, Cfg<MODE, BQ>::MAX_SPLIT);
    return launch<MODE, BQ>(p, s);
}

}  // namespace

MxEncodeFn mx_encode_fn() {
    static MxEncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<MxEncodeFn>(f);
    });
    return fn;
}

// View of `rows` rows of `pitch` bytes in boxes of 128 x box_rows, 128-byte swizzle. unpack:
// packed 4-bit values to a byte each (128 values a row of the box).
bool mx_map_rows(CUtensorMap* m, const void* ptr, int64_t rows, int64_t pitch, int box_rows, bool unpack) {
    const MxEncodeFn fn = mx_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)(unpack ? 2 * pitch : pitch), (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)pitch};
    cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    cuuint32_t one[2] = {1, 1};
    return fn(m, unpack ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr),
              dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t act_mx_ws_bytes(int M, int K) {
    const int tn = act_tile(M);
    return tn <= 8 ? 0 : 2 * up(M, tn) * (up(K, 128) + mx_scale_pitch(K));
}

cudaError_t launch_gemm_act_mx(const void* a, int64_t lda, const void* b_codes, const void* b_scales, void* C, bool c_f32,
                               int M, int N, int K, void* ws, uint32_t* err, cudaStream_t s) {
    if (M <= 0) return cudaSuccess;
    MxParams p;
    memset(&p, 0, sizeof(p));
    const int tn = act_tile(M);
    const int64_t rows = up(M, tn), kp = up(K, 128);
    p.scale_pitch = (int)mx_scale_pitch(K);
    p.tiles_p = (int)(up(N, TILE_P) / TILE_P);
    p.tiles_q = (int)(rows / tn);
    if ((int64_t)p.tiles_p * p.tiles_q > 0x3fffffffll || 2 * rows > 0x7fffffffll) return cudaErrorInvalidValue;
    p.tiles = p.tiles_p * p.tiles_q;
    if (!mx_map_rows(&p.map_p, b_codes, N, mx_code_pitch(K), TILE_P, true)) return cudaErrorInvalidValue;
    p.scale_p = static_cast<const uint8_t*>(b_scales);
    p.rows_p = N;
    p.rows_q = M;
    p.k_stages = (int)(kp / 128);
    p.a = static_cast<const __nv_bfloat16*>(a);
    p.lda = lda;
    p.K = K;
    p.vec = (reinterpret_cast<uintptr_t>(a) & 15) == 0 && lda % 8 == 0;
    p.C = C;
    p.ldc = N;
    p.c_f32 = c_f32;
    p.err = err;
    if (tn == 8) return launch_act<ACT_IN, 16>(p, s);
    uint8_t* terms = static_cast<uint8_t*>(ws);
    uint8_t* scales = terms + 2 * rows * kp;
    if (!map_terms(&p.map_q, terms, rows, kp, tn)) return cudaErrorInvalidValue;
    p.scale_q = scales;
    p.q_term_rows = (int)rows;
    const uint32_t per_row = (uint32_t)(kp / 8);
    const int64_t blocks = (rows * per_row + 255) / 256;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, split_rows_kernel, p.a, lda, M, K, p.vec, (int)rows, per_row, terms, scales,
                                             p.scale_pitch);
    if (e != cudaSuccess) return e;
    switch (tn) {
        case 16: return launch_act<ACT, 32>(p, s);
        case 32: return launch_act<ACT, 64>(p, s);
        case 64: return launch_act<ACT, 128>(p, s);
        default: return launch_act<ACT, 256>(p, s);
    }
}

}  // namespace ls
