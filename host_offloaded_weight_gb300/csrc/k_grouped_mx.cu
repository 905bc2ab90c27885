// Products of bf16 rows with MXFP4 matrices, grouped: rows g0 to g1 of a sorted order belong to group (expert) g and meet its
// matrix,  C[i] = B_g a_i  (or SiLU(G_g a_i) * (U_g a_i), or the rows scaled and put in their places), for any group sizes.
//
// As in k_gemm_mx.cu the weights are the left operand, 128 rows a tile, unpacked to a byte a value by the tensor copies, and the
// rows the right one, each as two E4M3 terms with a power of two for each block of 32 (kind::mxf8f6f4). A tile's columns
// are as many as its group needs (multiples of 32: 16 rows, two terms), so a group of three rows costs 32 columns and one of 300 three
// tiles of 112 and less. A gate/up tile takes 64 gate rows and their 64 up rows.
//
// split_sorted_kernel writes the terms in sorted order (gathering the rows by the routing's table where asked). Then one persistent
// CTA an SM: warp 0 loads by TMA, warp 1 copies the scales to TMEM and issues the products, four warps at a time take turns at
// bringing the block scales, four write the results while the next tile is computed (two accumulators).
#include <algorithm>

#include "kernels.h"
#include "tc.cuh"

namespace ls {
namespace {

using namespace tc;

constexpr int TILE_P = 128, P_BYTES = TILE_P * 128;
constexpr int CHUNK = 16;                    // rows of a box: 32 columns with both terms
constexpr int CHUNK_BYTES = 2 * CHUNK * 128;
constexpr int TEAM = 4, EPI_WARPS = 8;
constexpr int PAIR = 16;                     // gate/up tiles: rows of one matrix side by side
constexpr int MAX_G = GROUPED_MX_MAX_GROUPS;

// MAXC: chunks of a tile at most.
template <int MAXC>
struct Cfg {
    static constexpr int BQ = 32 * MAXC;                       // columns
    static constexpr int PARTS = (BQ + 127) / 128;             // 128-row parts of the right operand's scales
    static constexpr int Q_BYTES = MAXC * CHUNK_BYTES;
    static constexpr int SCALE_BYTES = (1 + PARTS) * 512;
    static constexpr int STAGE = (P_BYTES + Q_BYTES + SCALE_BYTES + 1023) / 1024 * 1024;
    static constexpr int BLOCKS = (MAXC * CHUNK + 31) / 32;    // of 32 rows
    static constexpr int FIT = (232448 - 1024 - 1024 - 4 * (MAX_G + 1)) / STAGE;
    static constexpr int STAGES = FIT < 8 ? FIT / 2 * 2 : 8;
    static constexpr int TEAMS = 2, RUN = STAGES >= 5 ? 4 : 2; // scale warps: teams take turns of RUN stages
    static constexpr int SCALE_COLS = 4 * (1 + PARTS);
    static constexpr int SMEM = STAGES * STAGE + 1024 + 512;
    static constexpr int FIRST_EPI = 2 + TEAM * TEAMS, THREADS = 32 * (FIRST_EPI + EPI_WARPS);
    static constexpr int TMEM_COLS = 512;
    static_assert(2 * BQ + STAGES * SCALE_COLS <= 512, "tensor memory: two accumulators and each stage's scales");
    // A wait by parity cannot tell a phase from the one two before it; stages are freed in order
    static_assert(RUN * (TEAMS - 1) + 1 <= STAGES, "turns of the scale warps");
};

struct GroupedParams {
    CUtensorMap map_p, map_p2, map_q;   // weights [groups][rows][K] (p2: the up matrices), terms [2][M][K]
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

struct Tile {
    int g, p0, row, rows, chunks;   // group, first output column, first sorted row, rows, chunks of 16
};

// Tile t of the launch: weight tiles innermost, so that the CTAs at work share a group's rows.
template <int MAXC>
__device__ __forceinline__ Tile tile_at(const GroupedParams& p, const int* first, int t) {
    const int n = t % p.tiles_p, mt = t / p.tiles_p;
    int lo = 0, hi = p.n_groups - 1;  // the last group with first[g] <= mt
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= mt) lo = mid;
        else hi = mid - 1;
    }
    Tile r;
    r.g = lo;
    r.p0 = n * (p.dual ? TILE_P / 2 : TILE_P);
    const int r0 = max(p.bounds[lo], 0), r1 = min(p.bounds[lo + 1], p.M), c = (r1 - r0 + CHUNK - 1) / CHUNK;
    const int tiles = (c + MAXC - 1) / MAXC, q = mt - first[lo];
    const int c0 = (int)((int64_t)c * q / tiles), c1 = (int)((int64_t)c * (q + 1) / tiles);  // even shares
    r.row = r0 + c0 * CHUNK;
    r.chunks = c1 - c0;
    r.rows = min(r1 - r.row, r.chunks * CHUNK);
    return r;
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ uint32_t word_of(const uint2& v, int i) { return i == 0 ? v.x : v.y; }
__device__ __forceinline__ void words(const uint8_t* p, bool in, uint4& v) { v = in ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void words(const uint8_t* p, bool in, uint2& v) { v = in ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0, 0); }
__device__ __forceinline__ void words_now(const uint8_t* p, bool in, uint4& v) { v = in ? __ldcg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void words_now(const uint8_t* p, bool in, uint2& v) { v = in ? __ldcg(reinterpret_cast<const uint2*>(p)) : make_uint2(0, 0); }
template <int RUN> struct Words;
template <> struct Words<4> { typedef uint4 type; };
template <> struct Words<2> { typedef uint2 type; };

template <int MAXC>
__global__ void __launch_bounds__(Cfg<MAXC>::THREADS, 1) gemm_grouped_mx_kernel(const __grid_constant__ GroupedParams p) {
    using C = Cfg<MAXC>;
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
    __shared__ int first[MAX_G + 1];   // row tiles before each group
    const int warp = uniform_warp(), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        stop = 0;
        for (int s = 0; s < S; ++s) {
            bar_init(full(s), 1 + TEAM);  // the TMA thread and a team of scale warps
            bar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(acc_full(b), 1);
            bar_init(acc_empty(b), EPI_WARPS);
        }
        bar_init(done, 1);
        bar_init_fence();
        tma_desc_prefetch(&p.map_p);
        tma_desc_prefetch(&p.map_q);
        if (p.dual) tma_desc_prefetch(&p.map_p2);
    }
    if (warp == 1) tmem_get(smem_addr(tmem_slot), C::TMEM_COLS);
    // The kernel before this one, which splits the rows, began after everything earlier was complete: only the split rows have
    // to be waited for.
    if (warp == 2) {
        int sum = 0;
        for (int g0 = 0; g0 < p.n_groups; g0 += 32) {
            const int g = g0 + lane;
            int t = 0;
            if (g < p.n_groups) {
                const int n = min(p.bounds[g + 1], p.M) - max(p.bounds[g], 0);
                t = n > 0 ? ((n + CHUNK - 1) / CHUNK + MAXC - 1) / MAXC : 0;
            }
            int before = t;
#pragma unroll
            for (int i = 1; i < 32; i *= 2) {
                const int o = __shfl_up_sync(0xffffffffu, before, i);
                if (lane >= i) before += o;
            }
            if (g < p.n_groups) first[g] = sum + before - t;
            sum += __shfl_sync(0xffffffffu, before, 31);
        }
        if (lane == 0) first[p.n_groups] = sum;
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int stages = p.k_stages, tiles = first[p.n_groups] * p.tiles_p;

    if (warp == 0) {
        // ------------------------------------------------------------ operand tiles
        const bool one = elect_one();
        int s = 0, it = 0;
        uint32_t phase = 1;  // a new barrier's preceding phase counts as complete
        bool ok = true, waited = false;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            const Tile tl = tile_at<MAXC>(p, first, t);
            // an unpacking copy counts the packed bytes (it leaves every second 8 bytes alone)
            const uint32_t bytes = P_BYTES / 2 + tl.chunks * CHUNK_BYTES;
            auto weights = [&](int st, int k) {
                const uint32_t at = base + st * C::STAGE;
                bar_expect(full(st), bytes);
                if (p.dual) {
                    for (int i = 0; i < TILE_P / 2; i += PAIR) {
                        tma_3d(at + 2 * i * 128, &p.map_p, full(st), k * 128, tl.p0 + i, tl.g);
                        tma_3d(at + (2 * i + PAIR) * 128, &p.map_p2, full(st), k * 128, tl.p0 + i, tl.g);
                    }
                } else {
                    tma_3d(at, &p.map_p, full(st), k * 128, tl.p0, tl.g);
                }
            };
            auto rows = [&](int st, int k) {
                const uint32_t at = base + st * C::STAGE + P_BYTES;
                for (int c = 0; c < tl.chunks; ++c) tma_3d(at + c * CHUNK_BYTES, &p.map_q, full(st), k * 128, tl.row + c * CHUNK, 0);
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
        // an aborted CTA waits for its own copies before it exits
        if (stop)
            for (int i = 0; i < S && i < it; ++i) {
                const int last = it - 1 - (it - 1 - i) % S;
                bar_wait(full(i), (uint32_t)(last / S) & 1u, p.err, 5);
            }
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        const bool one = elect_one();
        int n = 0, it = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++n) {
            const Tile tl = tile_at<MAXC>(p, first, t);
            const uint32_t idesc = mx_idesc(5, 0, TILE_P, 32 * tl.chunks);
            const int b = n & 1, parts = (32 * tl.chunks + 127) / 128;
            if (!bar_wait_warp(acc_empty(b), (uint32_t)((n >> 1) + 1) & 1u, p.err, 2) || stop) {
                stop = 1;
                break;
            }
            fence_after_sync();
            const uint32_t d = tmem + (uint32_t)(b * C::BQ);
            for (int k = 0; k < stages; ++k, ++it) {
                const int s = it % S;
                if (!bar_wait_warp(full(s), (uint32_t)(it / S) & 1u, p.err, 3)) {
                    ok = false;
                    stop = 1;
                    break;
                }
                fence_after_sync();
                const uint32_t sp = base + s * C::STAGE, sq = sp + P_BYTES, sc = sq + C::Q_BYTES;
                const uint32_t tp = tmem + (uint32_t)(2 * C::BQ + s * C::SCALE_COLS), tq = tp + 4;
                if (one) {
                    scale_copy(tp, scale_desc(sc));
#pragma unroll
                    for (int j = 0; j < C::PARTS; ++j)
                        if (j < parts) scale_copy(tq + 4 * j, scale_desc(sc + 512 * (1 + j)));
#pragma unroll
                    for (int j = 0; j < 4; ++j)  // 32 bytes of each row
                        mma_mxf8(d, operand_desc(sp + 32 * j), operand_desc(sq + 32 * j), idesc_at(idesc, j), tp, tq, (k | j) ? 1u : 0u);
                    mma_commit(empty(s));
                }
                __syncwarp();
            }
            if (ok && one) mma_commit(acc_full(b));
            __syncwarp();
        }
        if (one) mma_commit(done);
        __syncwarp();
        bar_wait(done, 0, p.err, 6);
    } else if (warp < C::FIRST_EPI) {
        // ------------------------------------------------------------ scales
        // Warp w of a team has rows 32 w + lane of each 128; the words of four such rows lie side by side at 16 lane in the order
        // that the tensor core reads. A row's words for RUN stages are loaded together, while the stages before are at hand.
        constexpr int RUN = C::RUN, NR = 1 + C::PARTS;
        typedef typename Words<RUN>::type V;
        const int team = (warp - 2) / TEAM, w = (warp - 2) % TEAM, runs = (stages + RUN - 1) / RUN;
        struct Turn {
            int t, run, at;  // tile, turn of it, the tile's first stage in the ring's line
        };
        auto after = [&](Turn u, int by) {
            for (u.run += by; u.run >= runs; u.run -= runs, u.t += gridDim.x, u.at += stages) {}
            return u;
        };
        Tile tl;
        int tl_of = -1;
        V v[2][NR];
        auto fetch = [&](V (&to)[NR], const Turn& u) {
            if (u.t >= tiles) return;
            if (tl_of != u.t) {
                tl = tile_at<MAXC>(p, first, u.t);
                tl_of = u.t;
            }
            const int64_t at = 4ll * RUN * u.run;
            const int r = 32 * w + lane;
            const bool second = p.dual && (r & PAIR);
            const int row = tl.p0 + (p.dual ? r / (2 * PAIR) * PAIR + (r & (PAIR - 1)) : r);
            words((second ? p.scale_p2 : p.scale_p) + tl.g * p.scale_stride + (int64_t)row * p.scale_pitch + at, row < p.N, to[0]);
#pragma unroll
            for (int j = 0; j < C::PARTS; ++j) {
                const int q = 128 * j + r, i = q / 32 * CHUNK + (q & 15);  // column q: chunk, term, row of the chunk
                const int64_t src = (int64_t)((q >> 4) & 1) * p.M + tl.row + i;
                words_now(p.scale_q + src * p.scale_pitch + at, i < tl.rows, to[1 + j]);
            }
        };
        Turn u = after(Turn{(int)blockIdx.x, 0, 0}, team);
        bool ok = true;
        grid_wait();
        fetch(v[0], u);
        while (ok && u.t < tiles) {
            const Turn next = after(u, C::TEAMS);
            fetch(v[1], next);
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                if (!ok || u.run * RUN + i >= stages) continue;
                const int it = u.at + u.run * RUN + i, s = it % S;
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
                if (lane == 0) bar_arrive(full(s));
            }
#pragma unroll
            for (int j = 0; j < NR; ++j) v[0][j] = v[1][j];
            u = next;
        }
    } else {
        // ------------------------------------------------------------ results
        // Two warps a TMEM lane quarter, each with every second group of eight rows. A lane has a weight row, an output column.
        // Gate/up tiles alternate: 16 gate rows, the 16 up rows of the same columns, so that a lane's partner is 16 lanes away;
        // each of the two finishes half of the group's rows.
        const int q = warp & 3, half = (warp - C::FIRST_EPI) >> 2, row = 32 * q + lane;  // q: the lane quarter that this warp can read
        const bool upper = lane & 16;
        int n = 0;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++n) {
            const Tile tl = tile_at<MAXC>(p, first, t);
            const int b = n & 1;
            // places and weights of the rows, read while the products run: lane l has rows l, 32 + l, ...
            int to[C::BLOCKS];
            float w[C::BLOCKS];
            if (p.epi == EPI_SCALE_F32) {
#pragma unroll
                for (int c = 0; c < C::BLOCKS; ++c) {
                    to[c] = 32 * c + lane < tl.rows ? __ldg(p.row_table + tl.row + 32 * c + lane) : -1;
                    if (to[c] >= p.M) to[c] = -1;
                    w[c] = to[c] >= 0 ? __ldg(p.row_weight + to[c]) : 0.f;
                }
            }
            if (!bar_wait_warp(acc_full(b), (uint32_t)(n >> 1) & 1u, p.err, 4) || stop) {
                stop = 1;
                break;
            }
            fence_after_sync();
            const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * C::BQ);
            const int col = tl.p0 + (p.dual ? 16 * q + (lane & 15) : row);
#pragma unroll
            for (int c = 0; c < C::BLOCKS; ++c) {
#pragma unroll 1
                for (int g = half; g < 4; g += 2) {
                    const int i0 = 32 * c + 8 * g;
                    if (i0 >= tl.rows) break;
                    uint32_t x[8], y[8];
                    const uint32_t a = at + (uint32_t)(i0 / CHUNK * 32 + i0 % CHUNK);
                    tmem_load8(a, x);
                    tmem_load8(a + CHUNK, y);
                    tmem_load_wait();
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(y[j]) + __uint_as_float(x[j]);  // the smaller term first
                    if (p.epi == EPI_SCALE_F32) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int r = __shfl_sync(0xffffffffu, to[c], 8 * g + j);
                            const float wr = __shfl_sync(0xffffffffu, w[c], 8 * g + j);
                            if (r >= 0 && col < p.N) static_cast<float*>(p.C)[(int64_t)r * p.N + col] = wr * v[j];
                        }
                    } else {
                        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.C) + (int64_t)(tl.row + i0) * p.N + col;
                        const int rows = col < p.N ? tl.rows - i0 : 0;
                        if (p.dual) {
                            if (upper) out += 4ll * p.N;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float other = __shfl_xor_sync(0xffffffffu, upper ? v[j] : v[j + 4], 16);
                                const float gate = upper ? other : v[j], up = upper ? v[j + 4] : other;
                                if (j + (upper ? 4 : 0) < rows) out[(int64_t)j * p.N] = __float2bfloat16_rn(gate / (1.f + __expf(-gate)) * up);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (j < rows) out[(int64_t)j * p.N] = __float2bfloat16_rn(v[j]);
                        }
                    }
                }
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) bar_arrive(acc_empty(b));
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        tmem_free(tmem, C::TMEM_COLS);
    }
}

// The two terms of the rows in sorted order, [2][M][pitch] bytes and their scales likewise; with k > 0 row i is row table[i] / k
// of a, rows outside a are zero. A thread takes 8 values, four lanes a block; a CTA a run of the array's units.
__global__ void __launch_bounds__(256)
split_sorted_kernel(const __nv_bfloat16* __restrict__ a, const int* __restrict__ table, int k, int64_t a_rows, int M, int K, uint32_t per_row,
                    uint32_t rows_a_cta, uint8_t* __restrict__ terms, uint8_t* __restrict__ scales, int scale_pitch) {
    grid_wait();
    grid_release();  // everything earlier is complete: the product may start on the weights
    const int row0 = (int)(blockIdx.x * rows_a_cta);
    const uint32_t units = min((int)rows_a_cta, M - row0) * per_row, most = (units + 31) & ~31u;
    const int64_t total = (int64_t)M * per_row, at = (int64_t)row0 * per_row;
    for (uint32_t i = threadIdx.x; i < most; i += 256) {  // whole warps: a block's lanes work together
        const uint32_t r = i / per_row, g = i - r * per_row;
        const int row = row0 + (int)r;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (i < units) {
            const int64_t from = k > 0 ? __ldg(table + row) / k : row;
            if (from >= 0 && from < a_rows) v = row8(a + from * K, (int)g * 8, K, 1);
        }
        uint2 o1, o2;
        uint32_t b1, b2;
        split8(v, o1, o2, b1, b2);
        if (i >= units) continue;
        reinterpret_cast<uint2*>(terms)[at + i] = o1;
        reinterpret_cast<uint2*>(terms)[at + i + total] = o2;
        if ((g & 3) == 0) {
            uint8_t* s1 = scales + (int64_t)row * scale_pitch;
            uint8_t* s2 = s1 + (int64_t)M * scale_pitch;
            s1[g >> 2] = (uint8_t)b1;
            s2[g >> 2] = (uint8_t)b2;
            if (g + 4 == per_row)
                for (int j = (int)(per_row >> 2); j < scale_pitch; ++j) s1[j] = s2[j] = 0;
        }
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
// The terms [2][rows][pitch] in boxes of 128 bytes x 16 rows of both.
bool map_terms(CUtensorMap* m, const void* ptr, int64_t rows, int64_t pitch) {
    const MxEncodeFn fn = mx_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)pitch, (cuuint64_t)rows, 2};
    cuuint64_t strides[2] = {(cuuint64_t)pitch, (cuuint64_t)(rows * pitch)};
    cuuint32_t box[3] = {128, CHUNK, 2};
    cuuint32_t one[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MAXC>
cudaError_t launch(const GroupedParams& p, int64_t most_tiles, cudaStream_t s) {
    auto kern = gemm_grouped_mx_kernel<MAXC>;
    using C = Cfg<MAXC>;
    static SmemAllowance allowed;
    const cudaError_t e = allowed.ensure(reinterpret_cast<const void*>(kern), C::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(most_tiles, gemm_num_sms()));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
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
    const int box = p.dual ? PAIR : TILE_P;
    if (!map_weights(&p.map_p, d.b_codes, d.N, mx_code_pitch(d.K), d.n_groups, d.code_stride, box) ||
        (p.dual && !map_weights(&p.map_p2, d.b2_codes, d.N, mx_code_pitch(d.K), d.n_groups, d.code_stride, box)) ||
        !map_terms(&p.map_q, terms, M, kp))
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
    const int rows = p.dual ? TILE_P / 2 : TILE_P;
    p.tiles_p = (d.N + rows - 1) / rows;
    p.row_table = d.row_table;
    p.row_weight = d.row_weight;
    p.C = d.C;
    p.err = err;
    const uint32_t per_row = (uint32_t)(kp / 8);
    const uint32_t rows_a_cta = std::max<uint32_t>(1, 1024 / per_row);  // about 1024 units
    const int64_t blocks = (M + rows_a_cta - 1) / rows_a_cta;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, split_sorted_kernel, static_cast<const __nv_bfloat16*>(d.A), d.gather_k > 0 ? d.row_table : nullptr,
                                             d.gather_k, d.a_rows, d.M, d.K, per_row, rows_a_cta, terms, scales, p.scale_pitch);
    if (e != cudaSuccess) return e;
    // rows of a tile at most: groups of 32 rows and fewer are bound by the weights' bytes and want more stages of them in flight
    const bool small = M <= 32ll * d.n_groups;
    const int most = CHUNK * (small ? 2 : 7);
    const int64_t tiles = (M / most + std::min<int64_t>(d.n_groups, M)) * p.tiles_p;  // a group has at most one tile that is not full
    if (tiles > 0x3fffffffll) return cudaErrorInvalidValue;
    return small ? launch<2>(p, tiles, s) : launch<7>(p, tiles, s);
}

}  // namespace ls
