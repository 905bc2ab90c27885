// Products of bf16 rows with MXFP4 matrices, grouped: rows g0 to g1 of a sorted order belong to group (expert) g and meet its
// matrix,  C[i] = B_g a_i  (or SiLU(G_g a_i) * (U_g a_i), or the rows scaled and put in their places), for any group sizes.
//
// As in k_gemm_mx.cu the weights are the left operand, 128 rows a tile, unpacked to a byte a value by the tensor copies, and the
// rows the right one, each as two E4M3 terms with a power of two for each block of 32 (kind::mxf8f6f4). A tile's columns
// are as many as its group needs (multiples of 32: 16 rows, two terms), so a group of three rows costs 32 columns and one of 300 three
// tiles of 112 and less. A gate/up tile takes 64 gate rows and their 64 up rows.
//
// split_sorted_kernel writes the terms in sorted order (gathering the rows by the routing's table where asked). Then persistent CTAs,
// one an SM: warp 0 loads by TMA, warp 1 copies the scales to TMEM and issues the products, eight warps in two teams bring the
// block scales, eight write the results while the next tile is computed (two accumulators).
//
// What bounds it. Groups of a few rows: 96 tokens through gate and up of 128 experts (2048 x 768, k = 8) take 46 us, 4.7 TB/s of
// the weights where the memory could bring 6.7. At 49 us, before the descriptors of a stage came by additions, a stage of 16 KB of
// unpacked weights took its issuing warp 406 clocks, the tensor pipe was active in 60 of them, and neither a second issuing warp
// (50 us), nor one product in place of four (43 us), nor no weights at all (46 us) changed that much, nor do ten stages of 16 rows at
// most in place of eight of 32 (46.5; five: 52); scales written to TMEM by their warps in place of copies of the tensor core: 47.6
// us, but 215 for 195 at 4096 tokens.
// Large groups: an SM's shared memory, about 133 bytes a clock of loads coming in and operands going out. From single CTAs a stage of 192
// columns is 41 KB in and 40 KB out, 609 clocks for 384 of products; so a pair of CTAs shares a tile of 256 weight rows
// (cta_group::2): each SM loads 128 rows of weights and one of the terms, 28 KB in and 28 KB out. 4096 tokens: up 227 -> 201 us,
// the tensor pipe active 66 % of the product's 145; the split before it takes 50. Rows fetched by the table in the product itself
// (16-byte asynchronous copies, terms written once for a token): 241 us, 288 with fewer waits. Terms of a token split once and copied
// to its experts' rows: 199 us for 201.
//
// A sum is one chain of K in its accumulator, whose cut-off is far finer than that of the bf16 products (k_gemm_lora.cu): results of values
// of either sign are off by 4e-8 of their norm at K = 768, 8e-8 at 14336, 7e-7 at 65536; of positive products by 6e-8, 1.6e-6 and 2.3e-5.
#include <algorithm>
#include <cstdlib>

#include "kernels.h"
#include "tc.cuh"

namespace ls {
namespace {

using namespace tc;

constexpr int TILE_P = 128, P_BYTES = TILE_P * 128;
constexpr int CHUNK = 16;                    // rows that a tile's columns are counted in: 32 columns with both terms
constexpr int CHUNK_BYTES = 2 * CHUNK * 128;
// A tile's chunks come in boxes of four, two and one, the larger ones first (a copy for each chunk kept the loading warp
// 45 clocks each busy, 630 a stage); a box has the first terms of its rows, then the second ones.
constexpr int BOXES = 3;
constexpr int TEAM = 4, EPI_WARPS = 8;
constexpr int PAIR = 16;                     // gate/up tiles: rows of one matrix side by side
constexpr int MAX_G = GROUPED_MX_MAX_GROUPS;

// MAXC: chunks of a tile at most. TWO: tiles of a pair of CTAs, the first of which holds the first terms and the second the second
// ones, and issues the products.
template <int MAXC, bool TWO>
struct Cfg {
    static constexpr int BQ = 32 * MAXC;                       // columns
    static constexpr int PARTS = (BQ + 127) / 128;             // 128-row parts of the right operand's scales
    static constexpr int Q_BYTES = MAXC * CHUNK_BYTES / (TWO ? 2 : 1);
    static constexpr int SCALE_BYTES = (1 + PARTS) * 512;
    static constexpr int STAGE = (P_BYTES + Q_BYTES + SCALE_BYTES + 1023) / 1024 * 1024;
    static constexpr int OWN_ROWS = (MAXC + 1) / 2 * CHUNK;    // rows of an epilogue warp
    static constexpr int FIT = (232448 - 1024 - 1024 - 20 * (MAX_G + 1) - 8 * EPI_WARPS * OWN_ROWS) / STAGE;
    static constexpr int SCALE_COLS = 4 * (1 + PARTS);
    static constexpr int FIT2 = (512 - 2 * BQ) / SCALE_COLS < FIT ? (512 - 2 * BQ) / SCALE_COLS : FIT;
    static constexpr int STAGES = FIT2 < 8 ? FIT2 : 8;
    static constexpr int TEAMS = 2, RUN = 4;                   // scale warps: teams take turns of RUN stages
    static constexpr int SMEM = STAGES * STAGE + 1024 + 512;
    static constexpr int FIRST_EPI = 2 + TEAM * TEAMS, THREADS = 32 * (FIRST_EPI + EPI_WARPS);
    static constexpr int TMEM_COLS = 512;
    static_assert(2 * BQ + STAGES * SCALE_COLS <= 512, "tensor memory: two accumulators and each stage's scales");
    // A wait by parity cannot tell a phase from the one two before it; stages are freed in order
    static_assert(RUN * (TEAMS - 1) + 1 <= STAGES, "turns of the scale warps");
};

struct GroupedParams {
    // Weights [groups][rows][K] (p2: the up matrices; both: gate and up in one map, see map_both) and terms [2][M][K]
    CUtensorMap map_p, map_p2, map_q[BOXES];
    int both, up_first;
    const uint8_t* scale_p;
    const uint8_t* scale_p2;
    int64_t scale_stride;               // bytes between groups
    const uint8_t* scale_q;             // [2][M][pitch]
    int scale_pitch;
    const int* bounds;
    int n_groups, M, N, k_stages, tiles_p, dual, epi;
    const int* row_table;
    const float* row_weight;
    void* C;
    uint32_t* err;
};

// Column of the first term of row i of a tile of `chunks`, and how many columns after it the second one's is.
__device__ __forceinline__ int column(int chunks, int i, int& apart) {
    int first = 0;
#pragma unroll
    for (int size = CHUNK << (BOXES - 1); size > CHUNK; size >>= 1)
        if (chunks & (size / CHUNK)) {
            if (i < first + size) {
                apart = size;
                return first + i;
            }
            first += size;
        }
    apart = CHUNK;
    return first + i;
}
// The row of column c, and which term.
__device__ __forceinline__ int row_of(int chunks, int c, int& term) {
    int first = 0;
#pragma unroll
    for (int size = CHUNK << (BOXES - 1); size > CHUNK; size >>= 1)
        if (chunks & (size / CHUNK)) {
            if (c < 2 * (first + size)) {
                term = c - 2 * first >= size;
                return c - first - (term ? size : 0);
            }
            first += size;
        }
    term = c - 2 * first >= CHUNK;
    return c - first - (term ? CHUNK : 0);
}

template <bool TWO>
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z) {
    if (TWO) tc::tma_3d_pair(dst, m, bar, x, y, z);
    else tc::tma_3d(dst, m, bar, x, y, z);
}
template <bool TWO>
__device__ __forceinline__ void tma_5d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z, int w, int v) {
    if (TWO) tc::tma_5d_pair(dst, m, bar, x, y, z, w, v);
    else tc::tma_5d(dst, m, bar, x, y, z, w, v);
}
template <bool TWO>
__device__ __forceinline__ void scales_to_tmem(uint32_t t, uint64_t desc) {
    if (TWO) scale_copy_pair(t, desc);
    else scale_copy(t, desc);
}
template <bool TWO>
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t add) {
    if (TWO) mma_mxf8_pair(d, a, b, idesc, sa, sb, add);
    else mma_mxf8(d, a, b, idesc, sa, sb, add);
}
template <bool TWO>
__device__ __forceinline__ void commit(uint32_t bar) {
    if (TWO) mma_commit_pair(bar);
    else mma_commit(bar);
}

// What the CTAs keep of the groups in shared memory.
struct Groups {
    int first[MAX_G + 1];   // row tiles before each group
    int row[MAX_G];         // its first row
    int end[MAX_G];
    int share[MAX_G];       // chunks of each of its row tiles, the first `more` of them have one more
    int more[MAX_G];
};

// A CTA's tiles, in order: weight tiles innermost, so that the CTAs at work share a group's rows. Steps by additions: a
// division by a number that only the launch knows takes 150 clocks.
struct Tiles {
    const Groups& s;
    int t, n, mt, g;                // tile, weight tile, row tile, group
    int step_n, step_mt;
    int p0, row, rows, chunks;      // this CTA's first output column, first sorted row, rows, chunks of 16
    int step, columns, own;         // output columns of a tile, and where in it this CTA's begin
    __device__ __forceinline__ Tiles(const GroupedParams& p, const Groups& groups, bool two) : s(groups), t((int)blockIdx.x), g(0), step((int)gridDim.x) {
        columns = p.dual ? TILE_P / 2 : TILE_P;
        own = 0;
        if (two) {
            t >>= 1;
            step >>= 1;
            own = (int)cluster_rank() * columns;
            columns *= 2;
        }
        step_mt = step / p.tiles_p;
        step_n = step - step_mt * p.tiles_p;
        mt = t / p.tiles_p;
        n = t - mt * p.tiles_p;
    }
    __device__ __forceinline__ void next(const GroupedParams& p) {
        t += step;
        mt += step_mt;
        n += step_n;
        if (n >= p.tiles_p) {
            n -= p.tiles_p;
            ++mt;
        }
    }
    // the tile's place, for t below the number of tiles
    __device__ __forceinline__ void find(const GroupedParams& p) {
        int hi = p.n_groups - 1;  // the last group with first[g] <= mt, from the one before on
        while (g < hi) {
            const int mid = (g + hi + 1) >> 1;
            if (s.first[mid] <= mt) g = mid;
            else hi = mid - 1;
        }
        const int q = mt - s.first[g], more = s.more[g];
        p0 = n * columns + own;
        chunks = s.share[g] + (q < more ? 1 : 0);
        row = s.row[g] + (q * s.share[g] + min(q, more)) * CHUNK;
        rows = min(s.end[g] - row, chunks * CHUNK);
    }
};

// g / (1 + e^-g). Far below zero the sum is e^-g, which leaves the range of a fast division at -87.3 and that of fp32 at -88.7: g e^g
// there (in 24 bits the same from -17 on).
__device__ __forceinline__ float silu(float g) {
    const bool far = g < -64.f;
    const float e = __expf(far ? g : -g);
    return far ? g * e : __fdividef(g, 1.f + e);
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ void words(const uint8_t* p, bool in, uint4& v) { v = in ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void words_now(const uint8_t* p, bool in, uint4& v) { v = in ? __ldcg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0); }

template <int MAXC, bool TWO>
__global__ void __launch_bounds__(Cfg<MAXC, TWO>::THREADS, 1) gemm_grouped_mx_kernel(const __grid_constant__ GroupedParams p) {
    using C = Cfg<MAXC, TWO>;
    constexpr int S = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t bars = base + S * C::STAGE;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (S + s); };
    auto acc_full = [&](int b) { return bars + 8u * (2 * S + b); };
    auto acc_empty = [&](int b) { return bars + 8u * (2 * S + 2 + b); };
    const uint32_t done = bars + 8u * (2 * S + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (bars - base) + 8 * (2 * S + 5));
    __shared__ volatile int stop;
    __shared__ Groups groups;
    __shared__ __align__(16) int s_to[EPI_WARPS][C::OWN_ROWS];
    __shared__ __align__(16) float s_weight[EPI_WARPS][C::OWN_ROWS];
    const int warp = uniform_warp(), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        stop = 0;
        for (int s = 0; s < S; ++s) {
            bar_init(full(s), 1 + (TWO ? 2 : 1) * TEAM);  // the (first CTA's) TMA thread and a team of scale warps (of each CTA)
            bar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(acc_full(b), 1);
            bar_init(acc_empty(b), (TWO ? 2 : 1) * EPI_WARPS);
        }
        bar_init(done, 1);
        bar_init_fence();
        tma_desc_prefetch(&p.map_p);
        for (int i = 0; i < BOXES; ++i) tma_desc_prefetch(&p.map_q[i]);
        if (p.dual && !p.both) tma_desc_prefetch(&p.map_p2);
    }
    if (warp == 1) {
        if (TWO) tmem_get_pair(smem_addr(tmem_slot), C::TMEM_COLS);
        else tmem_get(smem_addr(tmem_slot), C::TMEM_COLS);
    }
    // The kernel before this one, which splits the rows, began after everything earlier was complete: only the split rows have
    // to be waited for.
    if (warp == 2) {
        int sum = 0;
        for (int g0 = 0; g0 < p.n_groups; g0 += 32) {
            const int g = g0 + lane;
            int t = 0;
            if (g < p.n_groups) {
                // cut at both ends: the difference of an entry of the largest magnitude and one of the other sign would wrap
                const int r0 = min(max(p.bounds[g], 0), p.M), r1 = min(max(p.bounds[g + 1], 0), p.M), c = max(r1 - r0 + CHUNK - 1, 0) / CHUNK;
                t = (c + MAXC - 1) / MAXC;
                groups.row[g] = r0;
                groups.end[g] = r1;
                groups.share[g] = t ? c / t : 0;
                groups.more[g] = t ? c % t : 0;
            }
            int before = t;
#pragma unroll
            for (int i = 1; i < 32; i *= 2) {
                const int o = __shfl_up_sync(0xffffffffu, before, i);
                if (lane >= i) before += o;
            }
            if (g < p.n_groups) groups.first[g] = sum + before - t;
            sum += __shfl_sync(0xffffffffu, before, 31);
        }
        if (lane == 0) groups.first[p.n_groups] = sum;
    }
    fence_before_sync();
    __syncthreads();
    if (TWO) cluster_barrier();  // both CTAs' barriers are set up, both have their TMEM
    fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int rank = TWO ? (int)cluster_rank() : 0;
    const uint32_t full_at = TWO ? cluster_addr(full(0), 0) : full(0);  // the first CTA's
    // (Bounds out of order can give every row to half of the groups. What their matrices and C take of a card's 288 GB keeps that below
    // 2^31 tiles too: 2 10^9 at most, from 256 pairs of matrices of few values a row.)
    const int stages = p.k_stages, tiles = groups.first[p.n_groups] * p.tiles_p;

    if (warp == 0) {
        // ------------------------------------------------------------ operand tiles
        const bool one = elect_one();
        int s = 0, it = 0;
        uint32_t phase = 1;  // a new barrier's preceding phase counts as complete
        bool ok = true, waited = false;
        for (Tiles tl(p, groups, TWO); ok && tl.t < tiles; tl.next(p)) {
            tl.find(p);
            // an unpacking copy counts the packed bytes (it leaves every second 8 bytes alone)
            const uint32_t bytes = TWO ? 2 * (P_BYTES / 2 + tl.chunks * (CHUNK_BYTES / 2)) : P_BYTES / 2 + tl.chunks * CHUNK_BYTES;
            auto weights = [&](int st, int k) {
                const uint32_t at = base + st * C::STAGE, bar = full_at + 8 * st;
                if (rank == 0) bar_expect(full(st), bytes);
                if (p.both) {
                    tma_5d<TWO>(at, &p.map_p, bar, k * 128, 0, 0, tl.p0 / PAIR, tl.g);
                } else if (p.dual) {
                    for (int i = 0; i < TILE_P / 2; i += PAIR) {
                        tma_3d<TWO>(at + 2 * i * 128, &p.map_p, bar, k * 128, tl.p0 + i, tl.g);
                        tma_3d<TWO>(at + (2 * i + PAIR) * 128, &p.map_p2, bar, k * 128, tl.p0 + i, tl.g);
                    }
                } else {
                    tma_3d<TWO>(at, &p.map_p, bar, k * 128, tl.p0, tl.g);
                }
            };
            auto rows = [&](int st, int k) {
                const uint32_t at = base + st * C::STAGE + P_BYTES;
                int c = 0;
#pragma unroll
                for (int i = BOXES - 1; i >= 0; --i)
                    if (tl.chunks >> i & 1) {
                        tma_3d<TWO>(at + c * (TWO ? CHUNK_BYTES / 2 : CHUNK_BYTES), &p.map_q[i], full_at + 8 * st, k * 128, tl.row + c * CHUNK, rank);
                        c += 1 << i;
                    }
            };
            int k = 0;
            if (!waited) {  // the first stages' weights need not wait for the split rows
                const int ahead = min(S, stages);
                if (one)
                    for (int i = 0; i < ahead; ++i) weights(i, i);
                grid_wait();
                waited = true;
                if (one)
                    for (int i = 0; i < ahead; ++i) rows(i, i);
                __syncwarp();
                k = it = ahead;
                s = ahead % S;
                phase ^= ahead == S ? 1u : 0u;
            }
            for (; k < stages; ++k, ++it) {
                if (!bar_wait_warp(empty(s), phase, p.err, 1)) {
                    ok = false;
                    stop = 1;
                    break;
                }
                if (one) {
                    weights(s, k);
                    rows(s, k);
                }
                __syncwarp();
                if (++s == S) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!waited) grid_wait();
        grid_release();
        // an aborted CTA (of a pair the first, at whose barriers both CTAs' copies count) waits for its copies before it exits
        if (stop && rank == 0)
            for (int i = 0; i < S && i < it; ++i) {
                const int last = it - 1 - (it - 1 - i) % S;
                bar_wait(full(i), (uint32_t)(last / S) & 1u, p.err, 5);
            }
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        const bool one = elect_one();
        const uint32_t low_p = operand_low(base), low_q = operand_low(base + P_BYTES), low_s = scale_low(base + P_BYTES + C::Q_BYTES);
        int n = 0, it = 0;
        bool ok = rank == 0;
        for (Tiles tl(p, groups, TWO); ok && tl.t < tiles; tl.next(p), ++n) {
            tl.find(p);
            const uint32_t idesc = mx_idesc(5, 0, TWO ? 2 * TILE_P : TILE_P, 32 * tl.chunks);
            const int b = n & 1, parts = (32 * tl.chunks + 127) / 128;
            if (!bar_wait_warp(acc_empty(b), (uint32_t)((n >> 1) + 1) & 1u, p.err, 2) || stop) {
                stop = 1;
                break;
            }
            fence_after_sync();
            const uint32_t d = tmem + (uint32_t)(b * C::BQ);
            for (int k = 0; k < stages; ++k, ++it) {
                const int s = it % S;
                if (!(TWO ? bar_wait_cluster(full(s), (uint32_t)(it / S) & 1u, p.err, 3) : bar_wait_warp(full(s), (uint32_t)(it / S) & 1u, p.err, 3))) {
                    ok = false;
                    stop = 1;
                    break;
                }
                fence_after_sync();
                const uint32_t off = (uint32_t)s * (C::STAGE >> 4);
                const uint32_t tp = tmem + (uint32_t)(2 * C::BQ + s * C::SCALE_COLS), tq = tp + 4;
                if (one) {
                    scales_to_tmem<TWO>(tp, scale_from(low_s + off));
#pragma unroll
                    for (int j = 0; j < C::PARTS; ++j)
                        if (j < parts) scales_to_tmem<TWO>(tq + 4 * j, scale_from(low_s + off + (512 >> 4) * (1 + j)));
#pragma unroll
                    for (int j = 0; j < 4; ++j)  // 32 bytes of each row
                        product<TWO>(d, operand_from(low_p + off + 2 * j), operand_from(low_q + off + 2 * j), idesc_at(idesc, j), tp, tq, (k | j) ? 1u : 0u);
                    commit<TWO>(empty(s));
                }
                __syncwarp();
            }
            if (ok && one) commit<TWO>(acc_full(b));
            __syncwarp();
        }
        if (rank == 0) {
            if (one) commit<TWO>(done);
            __syncwarp();
            bar_wait(done, 0, p.err, 6);
        }
    } else if (warp < C::FIRST_EPI) {
        // ------------------------------------------------------------ scales
        // Warp w of a team has rows 32 w + lane of each 128; the words of four such rows lie side by side at 16 lane in the order
        // that the tensor core reads. A row's words for RUN stages are loaded together, while the stages before are at hand.
        constexpr int RUN = C::RUN, NR = 1 + C::PARTS;
        typedef uint4 V;
        const int team = (warp - 2) / TEAM, w = (warp - 2) % TEAM, runs = (stages + RUN - 1) / RUN;
        Tiles tl(p, groups, TWO);   // of the turn to request next
        int run = 0, at_stage = 0;                    // that turn of its tile, the tile's first stage in the ring's line
        int now_run, now_at;                          // the turn at hand
        bool now_on;
        auto skip = [&](int by) {
            for (run += by; run >= runs; run -= runs, at_stage += stages) tl.next(p);
        };
        V v[2][NR];
        auto fetch = [&](V (&to)[NR]) {
            if (tl.t >= tiles) return;
            tl.find(p);
            const int64_t at = 4ll * RUN * run;
            const int r = 32 * w + lane;
            const bool second = p.dual && ((r & PAIR) != 0) != (p.up_first != 0);
            const int row = tl.p0 + (p.dual ? r / (2 * PAIR) * PAIR + (r & (PAIR - 1)) : r);
            words((second ? p.scale_p2 : p.scale_p) + tl.g * p.scale_stride + (int64_t)row * p.scale_pitch + at, row < p.N, to[0]);
#pragma unroll
            for (int j = 0; j < C::PARTS; ++j) {
                int term = 128 * j + r >= CHUNK * tl.chunks;
                const int i = TWO ? 128 * j + r - (term ? CHUNK * tl.chunks : 0) : row_of(tl.chunks, 128 * j + r, term);
                const int64_t src = (int64_t)term * p.M + tl.row + i;
                words_now(p.scale_q + src * p.scale_pitch + at, 128 * j + r < 32 * tl.chunks && i < tl.rows, to[1 + j]);
            }
        };
        bool ok = true;
        grid_wait();
        skip(team);
        fetch(v[0]);
        now_on = tl.t < tiles;
        while (ok && now_on) {
            now_run = run;
            now_at = at_stage;
            skip(C::TEAMS);
            fetch(v[1]);
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                if (!ok || now_run * RUN + i >= stages) continue;
                const int it = now_at + now_run * RUN + i, s = it % S;
                if (!bar_wait_warp(empty(s), (uint32_t)(it / S + 1) & 1u, p.err, 7)) {
                    ok = false;
                    stop = 1;
                    continue;
                }
                const uint32_t to = base + s * C::STAGE + P_BYTES + C::Q_BYTES + lane * 16 + 4 * w;
#pragma unroll
                for (int j = 0; j < NR; ++j) st_shared1(to + 512 * j, word_of(v[0][j], i));
                fence_smem_async();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) bar_arrive(full(s));
                    else bar_arrive_cluster(full_at + 8 * s);
                }
            }
#pragma unroll
            for (int j = 0; j < NR; ++j) v[0][j] = v[1][j];
            now_on = tl.t < tiles;
        }
    } else {
        // ------------------------------------------------------------ results
        // Two warps a TMEM lane quarter, each with every second chunk of 16 rows. A lane has a weight row, an output column.
        // Gate/up tiles alternate: 16 gate rows, the 16 up rows of the same columns, so that a lane's partner is 16 lanes away;
        // each of the two finishes half of the group's rows.
        const int q = warp & 3, half = (warp - C::FIRST_EPI) >> 2, row = 32 * q + lane;  // q: the lane quarter that this warp can read
        const bool upper = lane & 16;
        int* const to = s_to[warp - C::FIRST_EPI];        // places and weights of this warp's rows
        float* const w = s_weight[warp - C::FIRST_EPI];
        int n = 0;
        for (Tiles tl(p, groups, TWO); tl.t < tiles; tl.next(p), ++n) {
            tl.find(p);
            const int b = n & 1;
            if (p.epi == EPI_SCALE_F32) {  // read while the products run; the warp's chunks are every second one
                __syncwarp();
                for (int l = lane; l < C::OWN_ROWS; l += 32) {
                    const int i = ((l >> 4) * 2 + half) * CHUNK + (l & 15);
                    int r = i < tl.rows ? __ldg(p.row_table + tl.row + i) : -1;
                    if (r >= p.M) r = -1;
                    to[l] = r;
                    w[l] = r >= 0 ? __ldg(p.row_weight + r) : 0.f;
                }
                __syncwarp();
            }
            if (!bar_wait_warp(acc_full(b), (uint32_t)(n >> 1) & 1u, p.err, 4) || stop) {
                stop = 1;
                break;
            }
            fence_after_sync();
            const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * C::BQ);
            const int col = tl.p0 + (p.dual ? 16 * q + (lane & 15) : row);
            const bool in = col < p.N;
#pragma unroll 1
            for (int i0 = half * CHUNK, l0 = 0; i0 < tl.rows; i0 += 2 * CHUNK, l0 += CHUNK) {
                uint32_t x[CHUNK], y[CHUNK];
                int apart = CHUNK * tl.chunks;
                const uint32_t c = at + (uint32_t)(TWO ? i0 : column(tl.chunks, i0, apart));
                tmem_load16(c, x);
                tmem_load16(c + apart, y);
                tmem_load_wait();
                float v[CHUNK];
#pragma unroll
                for (int j = 0; j < CHUNK; ++j) v[j] = __uint_as_float(y[j]) + __uint_as_float(x[j]);  // the smaller term first
                if (p.epi == EPI_SCALE_F32) {
                    float* const out = static_cast<float*>(p.C) + col;
#pragma unroll
                    for (int j = 0; j < CHUNK; j += 4) {
                        const int4 r = *reinterpret_cast<const int4*>(to + l0 + j);
                        const float4 f = *reinterpret_cast<const float4*>(w + l0 + j);
                        if (in && r.x >= 0) out[(uint64_t)(uint32_t)r.x * (uint32_t)p.N] = f.x * v[j];
                        if (in && r.y >= 0) out[(uint64_t)(uint32_t)r.y * (uint32_t)p.N] = f.y * v[j + 1];
                        if (in && r.z >= 0) out[(uint64_t)(uint32_t)r.z * (uint32_t)p.N] = f.z * v[j + 2];
                        if (in && r.w >= 0) out[(uint64_t)(uint32_t)r.w * (uint32_t)p.N] = f.w * v[j + 3];
                    }
                } else {
                    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.C) + (int64_t)(tl.row + i0) * p.N + col;
                    const int rows = in ? tl.rows - i0 : 0;
                    if (p.dual) {
                        if (upper) out += (int64_t)(CHUNK / 2) * p.N;
#pragma unroll
                        for (int j = 0; j < CHUNK / 2; ++j, out += p.N) {
                            const float mine = upper ? v[j + CHUNK / 2] : v[j];
                            const float other = __shfl_xor_sync(0xffffffffu, upper ? v[j] : v[j + CHUNK / 2], 16);
                            const bool swap = upper != (p.up_first != 0);
                            const float gate = swap ? other : mine, up = swap ? mine : other;
                            if (j + (upper ? CHUNK / 2 : 0) < rows) *out = __float2bfloat16_rn(silu(gate) * up);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < CHUNK; ++j, out += p.N)
                            if (j < rows) *out = __float2bfloat16_rn(v[j]);
                    }
                }
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if (TWO) bar_arrive_cluster(cluster_addr(acc_empty(b), 0));
                else bar_arrive(acc_empty(b));
            }
        }
    }
    fence_before_sync();
    __syncwarp();
    if (TWO) cluster_barrier();  // neither CTA's memory goes while the other's copies, products or arrivals may reach it
    else __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        if (TWO) tmem_free_pair(tmem, C::TMEM_COLS);
        else tmem_free(tmem, C::TMEM_COLS);
    }
}

// The row of A that an entry of the table stands for; -1: none.
__device__ __forceinline__ int64_t source_row(int entry, int k, int64_t rows) {
    const int r = entry < 0 ? -1 : entry / k;
    return r < rows ? r : -1;
}

// split8 of tc.cuh, with the scaled values and what the first term leaves as f16 pairs: both are exact there, down to 2^-24 of
// values below 2^8, far under what the second term can hold. (All in fp32: half as many instructions again.)
__device__ __forceinline__ void split8_half(uint4 raw, uint2& o1, uint2& o2, uint32_t& b1, uint32_t& b2) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    m = max(m & 0xffffu, m >> 16);
    const uint32_t e = m >> 7;
    // blocks next to either end of the range, subnormal ones among them, whose terms' scales are not 2^5 apart: the general form
    // (all lanes of the warp work together in it). Zeros, as of padding, are right in either.
    if (__any_sync(0xffffffffu, e >= TOP_FIELD || (e < 32 && m > 0))) {
        split8(raw, o1, o2, b1, b2);
        return;
    }
    b1 = e == 0 ? 0 : e - 7;
    b2 = e == 0 ? 0 : e - 12;
    const float f1 = __uint_as_float((254 - min(b1, 253u)) << 23);
    const __half2 up = __float2half2_rn(32.f);
    uint32_t t1[4], t2[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2 h = __floats2half2_rn(__uint_as_float(w[j] << 16) * f1, __uint_as_float(w[j] & 0xffff0000u) * f1);
        uint16_t q;
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(q) : "r"(*reinterpret_cast<const uint32_t*>(&h)));
        uint32_t d;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(q));
        const __half2 rest = __hmul2(__hsub2(h, *reinterpret_cast<const __half2*>(&d)), up);
        t1[j] = q;
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(q) : "r"(*reinterpret_cast<const uint32_t*>(&rest)));
        t2[j] = q;
    }
    o1 = make_uint2(__byte_perm(t1[0], t1[1], 0x5410), __byte_perm(t1[2], t1[3], 0x5410));
    o2 = make_uint2(__byte_perm(t2[0], t2[1], 0x5410), __byte_perm(t2[2], t2[3], 0x5410));
}

// The two terms of the rows in sorted order, [2][M][pitch] bytes and their scales likewise; with k > 0 row i is row table[i] / k
// of a, rows outside a are zero. A warp takes a row at a time, a lane 8 values of it, four lanes a block.
constexpr int SPLIT_WARPS = 8;
__global__ void __launch_bounds__(32 * SPLIT_WARPS)
split_sorted_kernel(const __nv_bfloat16* __restrict__ a, const int* __restrict__ table, int k, int64_t a_rows, int M, int K, int per_row,
                    uint8_t* __restrict__ terms, uint8_t* __restrict__ scales, int scale_pitch) {
    grid_wait();
    grid_release();  // everything earlier is complete: the product may start on the weights
    const int lane = threadIdx.x & 31;
    for (int row = (int)blockIdx.x * SPLIT_WARPS + (threadIdx.x >> 5); row < M; row += gridDim.x * SPLIT_WARPS) {
        const int64_t from = k > 0 ? source_row(__ldg(table + row), k, a_rows) : row < a_rows ? row : -1;
        const bool in = from >= 0;
        const __nv_bfloat16* x = a + (in ? from : 0) * K;
        uint2* t1 = reinterpret_cast<uint2*>(terms) + (int64_t)row * per_row;
        uint2* t2 = t1 + (int64_t)M * per_row;
        uint8_t* s1 = scales + (int64_t)row * scale_pitch;
        uint8_t* s2 = s1 + (int64_t)M * scale_pitch;
#pragma unroll 2
        for (int g0 = 0; g0 < per_row; g0 += 32) {
            const int g = g0 + lane;
            uint2 o1, o2;
            uint32_t b1, b2;
            split8_half(in && g * 8 < K ? __ldg(reinterpret_cast<const uint4*>(x) + g) : make_uint4(0, 0, 0, 0), o1, o2, b1, b2);  // K is a multiple of 8
            if (g >= per_row) continue;
            t1[g] = o1;
            t2[g] = o2;
            if ((g & 3) == 0) {
                s1[g >> 2] = (uint8_t)b1;
                s2[g >> 2] = (uint8_t)b2;
            }
        }
        for (int j = per_row / 4 + lane; j < scale_pitch; j += 32) s1[j] = s2[j] = 0;
    }
}

// ------------------------------------------------------------------ host side
int64_t up128(int64_t n) { return (n + 127) / 128 * 128; }

// MXFP4 codes of n matrices [rows, pitch bytes], `stride` bytes apart, unpacked to a byte a value, in boxes of 128 values x box_rows.
bool map_weights(CUtensorMap* m, const void* ptr, int64_t rows, int64_t pitch, int64_t n, int64_t stride, int box_rows) {
    const MxEncodeFn fn = mx_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)(2 * pitch), (cuuint64_t)rows, (cuuint64_t)n};
    cuuint64_t strides[2] = {(cuuint64_t)pitch, (cuuint64_t)stride};
    cuuint32_t box[3] = {128, (cuuint32_t)box_rows, 1};
    cuuint32_t one[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 3, const_cast<void*>(ptr), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Gate and up matrices of n experts as one tensor [n][rows / 16][2][16][K], the first of the two at `ptr` and the other `apart` bytes
// on, in boxes of a tile: 16 rows of one, the 16 of the other, and so on. One copy a stage in place of eight; rows a multiple of 16.
bool map_both(CUtensorMap* m, const void* ptr, int64_t apart, int64_t rows, int64_t pitch, int64_t n, int64_t stride) {
    const MxEncodeFn fn = mx_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[5] = {(cuuint64_t)(2 * pitch), (cuuint64_t)PAIR, 2, (cuuint64_t)(rows / PAIR), (cuuint64_t)n};
    cuuint64_t strides[4] = {(cuuint64_t)pitch, (cuuint64_t)apart, (cuuint64_t)(PAIR * pitch), (cuuint64_t)stride};
    cuuint32_t box[5] = {128, PAIR, 2, TILE_P / 2 / PAIR, 1};
    cuuint32_t one[5] = {1, 1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 5, const_cast<void*>(ptr), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The terms [2][rows][pitch] in boxes of 128 bytes x box_rows, of both or of one.
bool map_terms(CUtensorMap* m, const void* ptr, int64_t rows, int64_t pitch, int box_rows, int box_terms) {
    const MxEncodeFn fn = mx_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)pitch, (cuuint64_t)rows, 2};
    cuuint64_t strides[2] = {(cuuint64_t)pitch, (cuuint64_t)(rows * pitch)};
    cuuint32_t box[3] = {128, (cuuint32_t)box_rows, (cuuint32_t)box_terms};
    cuuint32_t one[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MAXC, bool TWO>
cudaError_t launch(const GroupedParams& p, int64_t most_tiles, cudaStream_t s) {
    auto kern = gemm_grouped_mx_kernel<MAXC, TWO>;
    using C = Cfg<MAXC, TWO>;
    static SmemAllowance allowed;
    const cudaError_t e = allowed.ensure(reinterpret_cast<const void*>(kern), C::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(TWO ? 2 * (unsigned)std::min<int64_t>(most_tiles, std::max(1, gemm_num_sms() / 2)) : (unsigned)std::min<int64_t>(most_tiles, gemm_num_sms()));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 2;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = TWO ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

int64_t grouped_mx_ws_bytes(int64_t M, int64_t K) { return 2 * M * (up128(K) + mx_scale_pitch(K)); }

cudaError_t launch_gemm_grouped_mx(const GroupedMxDesc& d, void* ws, uint32_t* err, cudaStream_t s) {
    GroupedParams p;
    memset(&p, 0, sizeof(p));
    const int64_t kp = up128(d.K), M = d.M;
    uint8_t* terms = static_cast<uint8_t*>(ws);
    uint8_t* scales = terms + 2 * M * kp;
    p.dual = d.epi == EPI_SWIGLU;
    p.epi = d.epi;
    const int64_t pitch = mx_code_pitch(d.K);
    const int64_t apart = static_cast<const uint8_t*>(d.b2_codes) - static_cast<const uint8_t*>(d.b_codes);
    // Groups of a few rows are bound by the stages of weights that a CTA passes and want single CTAs. 128 experts of 2048 x 768, up and
    // down: 6 rows a group take 46 and 29 us that way, 51 and 33 in pairs; 16 rows 55 and 36, 56 and 38; 24 rows down 42 and 41; 32
    // rows up 69 and 63.
    const bool two = M > 18ll * d.n_groups;
    p.both = p.dual && d.N % PAIR == 0 && apart != 0 && std::abs(apart) < (1ll << 40);
    p.up_first = p.both && apart < 0;
    bool ok = true;
    if (p.both) {
        ok = map_both(&p.map_p, p.up_first ? d.b2_codes : d.b_codes, std::abs(apart), d.N, pitch, d.n_groups, d.code_stride);
    } else {
        ok = map_weights(&p.map_p, d.b_codes, d.N, pitch, d.n_groups, d.code_stride, p.dual ? PAIR : TILE_P) &&
             (!p.dual || map_weights(&p.map_p2, d.b2_codes, d.N, pitch, d.n_groups, d.code_stride, PAIR));
    }
    for (int i = 0; i < BOXES; ++i) ok = ok && map_terms(&p.map_q[i], terms, M, kp, CHUNK << i, two ? 1 : 2);
    if (!ok)
        return cudaErrorInvalidValue;
    p.scale_p = static_cast<const uint8_t*>(d.b_scales);
    p.scale_p2 = static_cast<const uint8_t*>(d.b2_scales);
    p.scale_stride = d.scale_stride;
    p.scale_q = scales;
    p.scale_pitch = (int)mx_scale_pitch(d.K);
    p.bounds = d.bounds;
    p.n_groups = d.n_groups;
    p.M = d.M;
    p.N = d.N;
    p.k_stages = (int)(kp / 128);
    const int rows = (p.dual ? TILE_P / 2 : TILE_P) * (two ? 2 : 1);
    p.tiles_p = (d.N + rows - 1) / rows;
    p.row_table = d.row_table;
    p.row_weight = d.row_weight;
    p.C = d.C;
    p.err = err;
    const int per_row = (int)(kp / 8);
    const int64_t blocks = std::min<int64_t>((M + SPLIT_WARPS - 1) / SPLIT_WARPS, 8ll * gemm_num_sms());
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(32 * SPLIT_WARPS);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, split_sorted_kernel, static_cast<const __nv_bfloat16*>(d.A), d.gather_k > 0 ? d.row_table : nullptr,
                                             d.gather_k, d.a_rows, d.M, d.K, per_row, terms, scales, p.scale_pitch);
    if (e != cudaSuccess) return e;
    const int most = CHUNK * (two ? 7 : 2);
    const int64_t tiles = (M / most + std::min<int64_t>(d.n_groups, M)) * p.tiles_p;  // a group has at most one tile that is not full
    if (tiles > 0x3fffffffll) return cudaErrorInvalidValue;
    return two ? launch<7, true>(p, tiles, s) : launch<2, false>(p, tiles, s);
}

}  // namespace ls
