// C[M,N] = sum_k A[m,k] B[n,k] with both operands MXFP4, on the sm_103a tensor cores: kind::mxf4, 64 values of K
// an instruction, codes packed in shared memory as they lie in global memory, fp32 sums.
//
// What bounds it: an SM takes in about 60 bytes a clock (a stage of 28.7 KB took 476 clocks with the products and the
// scales left out), and at 4 bits the products of a stage are shorter than its loads. A tile's shape decides: a pair of
// CTAs shares a tile of 256 x BQ (cta_group::2), each SM loads 128 rows of A and BQ / 2 of B for 128 x BQ outputs. With
// 256 x 224 a stage is 31 KB of rows and 3 KB of scales, about 560 of the 690 clocks that it takes (products: 450; the
// tensor pipe is active 66 %; what the other 130 are spent on has not been found). One CTA with 128 x 192 tiles loaded 41 KB for 24576 outputs in place of 28672. A wider
// tile leaves no TMEM for a second accumulator.
//
// Structure (persistent pairs, one CTA an SM): warp 0 loads the CTA's operand rows by TMA (128-byte rows = 256
// values of K, 128-byte swizzle) into a ring of stages; warps 2 to 5 bring the scales, 32 bytes of a row at a time,
// in the order that the tensor core reads (32 rows of 16 bytes, the four 32-row groups side by side); the first
// CTA's warp 1 copies both CTAs' scales to TMEM and issues the products; eight warps write the results while the
// next tile is computed (two accumulators), by bulk stores of 32 rows x 128 bytes. Both CTAs' loads and scales
// count at the first CTA's `full` barriers; what frees a stage, and what completes a tile, is signalled in both.
// The scales have two sets of TMEM columns, taken in turn: the products of two stages before have to be complete.
//
// 2048 x 13824 x 5120: 50.7 us, 5.7 PFLOP/s (single CTAs: 63 us); 4096 x 4096 x 1024: 12.4 us (17.7); 333 x 1111 x
// 1000: 4.5 us (10.5); 8192 x 8192 x 8192: 6.6 PFLOP/s. fp32 results: 57, 15.7 and 4.8 us for the first three. 256 x 5120 x
// 13824, 40 tiles for 76 pairs and nothing shared along K: 19 us. One team of scale warps in place of two: 54.5 us for the
// first; results written by lanes in place of bulk stores: 14.1 us for the second. A ring of the scales' own and a warp
// that copies them to TMEM, with 192 columns: 49.9 and 12.6 us, not worth their barriers.
#include <algorithm>

#include "kernels.h"
#include "tc.cuh"

namespace ls {
namespace {

using namespace tc;

constexpr int TILE_P = 128;              // rows of A of a CTA
constexpr int P_BYTES = TILE_P * 128;    // a stage of it
constexpr int QUADS = 2;                 // words of four blocks (128 values of K) in a stage
constexpr int EPI_WARPS = 8, TEAM = 4, TEAMS = 2;  // scale warps: teams of four take turns
constexpr int RUN = 4;                   // stages of a turn: 32 bytes of a row's scales
constexpr int FIRST_EPI = 2 + TEAM * TEAMS, THREADS = 32 * (FIRST_EPI + EPI_WARPS);

template <int BQ>
struct Cfg {
    static constexpr int PARTS = (BQ + 127) / 128;          // 128-row parts of B's scales
    static constexpr int Q_BYTES = BQ / 2 * 128;
    static constexpr int SCALE_BYTES = QUADS * (1 + PARTS) * 512;
    static constexpr int STAGE = (P_BYTES + Q_BYTES + SCALE_BYTES + 1023) / 1024 * 1024;
    static constexpr int EPI_BYTES = EPI_WARPS * 4096;
    static constexpr int FIT = (232448 - 1024 - 512 - EPI_BYTES) / STAGE;
    static constexpr int STAGES = FIT < 8 ? FIT : 8;
    static constexpr int SCALE_COLS = QUADS * 4 * (1 + PARTS);  // TMEM columns of a stage's scales
    static constexpr int SMEM = STAGES * STAGE + EPI_BYTES + 1024 + 512;
    static_assert(2 * BQ + 2 * SCALE_COLS <= 512, "tensor memory");
    // A wait by parity cannot tell a phase from the one two before it. Stages are freed in order, so a team's wait for
    // one stage covers every older one: its next may be a round of the ring later, not more.
    static_assert(RUN * (TEAMS - 1) + 1 <= STAGES, "turns of the scale warps");
    static_assert(BQ % 32 == 0 && BQ <= 224, "columns of a product");
};

struct PairParams {
    CUtensorMap map_a, map_b, map_c;
    const uint8_t* scale_a;
    const uint8_t* scale_b;
    int scale_pitch, scale_wide;  // scale_wide: rows of scales are whole 32-byte sectors
    int M, N, k_stages;
    int tiles_m, tiles;   // tiles of 256 rows; all tiles
    void* C;
    int c_f32, c_bulk;    // c_bulk: rows of C are 16-byte aligned, as bulk stores want them
    uint32_t* err;
};

__device__ __forceinline__ void store_c(const PairParams& p, int64_t at, float v) {
    if (p.c_f32) static_cast<float*>(p.C)[at] = v;
    else static_cast<__nv_bfloat16*>(p.C)[at] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ uint32_t pair_bf16(uint32_t lo, uint32_t hi) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
    return *reinterpret_cast<const uint32_t*>(&t);
}

// A warp's 32 rows x 32 fp32 or 64 bf16 columns, lane l with row r0 + l: 128-byte rows with the 128-byte swizzle in
// `buf` (1024-byte aligned), written by one bulk store, which clips them to C.
template <bool F32>
__device__ __forceinline__ void store_box(const PairParams& p, uint32_t buf, const uint32_t (&v)[F32 ? 32 : 64], int r0, int col0) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) tma_store_read();  // the box before
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t at = buf + lane * 128 + ((j ^ (lane & 7)) << 4);
        if (F32) st_shared4(at, v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        else st_shared4(at, pair_bf16(v[F32 ? 0 : 8 * j], v[F32 ? 0 : 8 * j + 1]), pair_bf16(v[F32 ? 0 : 8 * j + 2], v[F32 ? 0 : 8 * j + 3]),
                        pair_bf16(v[F32 ? 0 : 8 * j + 4], v[F32 ? 0 : 8 * j + 5]), pair_bf16(v[F32 ? 0 : 8 * j + 6], v[F32 ? 0 : 8 * j + 7]));
    }
    fence_smem_async();
    __syncwarp();
    if (lane == 0 && r0 < p.M && col0 < p.N) tma_store_2d(&p.map_c, buf, col0, r0);
}

// The same for 32 columns of rows that a bulk store cannot take: turned through shared memory (float4 columns,
// exclusive-or swizzled by the row), a lane has a column and takes a row at a time.
__device__ __forceinline__ void store_chunk(const PairParams& p, float4* buf, const uint32_t (&v)[32], int r0, int col0) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        buf[lane * 8 + (j ^ (lane & 7))] = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                                       __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
    __syncwarp();
    if (col0 + lane < p.N) {
        const float* f = reinterpret_cast<const float*>(buf);
        const int rows = min(32, p.M - r0);
#pragma unroll 8
        for (int r = 0; r < rows; ++r)
            store_c(p, (int64_t)(r0 + r) * p.N + col0 + lane, f[r * 32 + 4 * ((lane >> 2) ^ (r & 7)) + (lane & 3)]);
    }
    __syncwarp();
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

template <int BQ>
__global__ void __launch_bounds__(THREADS, 1) gemm_mx4_pair_kernel(const __grid_constant__ PairParams p) {
    using C = Cfg<BQ>;
    constexpr int S = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;  // the same in both CTAs
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t bars = base + S * C::STAGE + C::EPI_BYTES;
    auto full = [&](int s) { return bars + 8u * s; };  // the first CTA's count both CTAs' loads and scales
    auto empty = [&](int s) { return bars + 8u * (S + s); };
    auto acc_full = [&](int b) { return bars + 8u * (2 * S + b); };
    auto acc_empty = [&](int b) { return bars + 8u * (2 * S + 2 + b); };
    const uint32_t done = bars + 8u * (2 * S + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (bars - base) + 8 * (2 * S + 5));
    __shared__ volatile int stop;
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank(), pair = (int)blockIdx.x >> 1, pairs = (int)gridDim.x >> 1;

    if (threadIdx.x == 0) {
        stop = 0;
        for (int s = 0; s < S; ++s) {
            bar_init(full(s), 1 + 2 * TEAM);  // the first CTA's TMA thread and a team of scale warps of each CTA
            bar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(acc_full(b), 1);
            bar_init(acc_empty(b), 2 * EPI_WARPS);
        }
        bar_init(done, 1);
        bar_init_fence();
        tma_desc_prefetch(&p.map_a);
        tma_desc_prefetch(&p.map_b);
    }
    if (warp == 1) tmem_get_pair(smem_addr(tmem_slot), 512);
    fence_before_sync();
    __syncwarp();
    cluster_barrier();  // both CTAs' barriers are set up, both have their TMEM
    fence_after_sync();
    grid_wait();
    const uint32_t tmem = *tmem_slot;
    const int stages = p.k_stages;
    auto row_a = [&](int tile) { return tile % p.tiles_m * (2 * TILE_P) + rank * TILE_P; };
    auto col_b = [&](int tile) { return tile / p.tiles_m * BQ; };

    if (warp == 0) {
        // ------------------------------------------------------------ operand tiles
        const bool one = elect_one();
        const uint32_t full_at = cluster_addr(full(0), 0);
        int s = 0, it = 0;
        uint32_t phase = 1;  // a new barrier's preceding phase counts as complete
        bool ok = true;
        for (int tile = pair; ok && tile < p.tiles; tile += pairs) {
            const int ra = row_a(tile), rb = col_b(tile) + rank * (BQ / 2);
            for (int k = 0; k < stages; ++k, ++it) {
                if (!bar_wait_warp(empty(s), phase, p.err, 1)) {
                    ok = false;
                    stop = 1;
                    break;
                }
                if (one) {
                    if (rank == 0) bar_expect(full(s), 2 * (P_BYTES + C::Q_BYTES));
                    tma_2d_pair(base + s * C::STAGE, &p.map_a, full_at + 8 * s, k * 128, ra);
                    tma_2d_pair(base + s * C::STAGE + P_BYTES, &p.map_b, full_at + 8 * s, k * 128, rb);
                }
                __syncwarp();
                if (++s == S) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
        grid_release();
        // the first CTA of an aborted pair waits for the copies that count at its barriers
        if (stop && rank == 0)
            for (int i = 0; i < S && i < it; ++i) {
                const int last = it - 1 - (it - 1 - i) % S;
                bar_wait(full(i), (uint32_t)(last / S) & 1u, p.err, 5);
            }
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        if (rank == 0) {
            constexpr uint32_t IDESC = mx_idesc(1, 1, 2 * TILE_P, BQ);
            const bool one = elect_one();
            int n = 0, it = 0;
            bool ok = true;
            for (int tile = pair; ok && tile < p.tiles; tile += pairs, ++n) {
                const int b = n & 1;
                if (!bar_wait_warp(acc_empty(b), (uint32_t)((n >> 1) + 1) & 1u, p.err, 2) || stop) {
                    stop = 1;
                    break;
                }
                fence_after_sync();
                const uint32_t d = tmem + (uint32_t)(b * BQ);
                for (int k = 0; k < stages; ++k, ++it) {
                    const int s = it % S;
                    // the products of two stages before are done with this stage's scale columns
                    if ((it >= 2 && !bar_wait_warp(empty((it - 2) % S), (uint32_t)((it - 2) / S) & 1u, p.err, 8)) ||
                        !bar_wait_cluster(full(s), (uint32_t)(it / S) & 1u, p.err, 3)) {
                        ok = false;
                        stop = 1;
                        break;
                    }
                    fence_after_sync();
                    const uint32_t sp = base + s * C::STAGE, sq = sp + P_BYTES, sc = sq + C::Q_BYTES;
                    const uint32_t tp = tmem + (uint32_t)(2 * BQ + (it & 1) * C::SCALE_COLS), tq = tp + 4 * QUADS;
                    if (one) {
#pragma unroll
                        for (int q = 0; q < QUADS; ++q) {
                            scale_copy_pair(tp + 4 * q, scale_desc(sc + 512 * q));
#pragma unroll
                            for (int j = 0; j < C::PARTS; ++j)
                                scale_copy_pair(tq + 4 * (q * C::PARTS + j), scale_desc(sc + 512 * (QUADS + q * C::PARTS + j)));
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)  // 32 bytes of each row
                            mma_mxf4_pair(d, operand_desc(sp + 32 * j), operand_desc(sq + 32 * j), idesc_at(IDESC, 2 * (j & 1)),
                                          tp + 4 * (j >> 1), tq + 4 * C::PARTS * (j >> 1), (k | j) ? 1u : 0u);
                        mma_commit_pair(empty(s));
                    }
                    __syncwarp();
                }
                if (ok && one) mma_commit_pair(acc_full(b));
                __syncwarp();
            }
            if (one) mma_commit_pair(done);
            __syncwarp();
            bar_wait(done, 0, p.err, 6);
        }
    } else if (warp < FIRST_EPI) {
        // ------------------------------------------------------------ scales
        // Warp w has rows 32 w + lane of each 128; the words of four such rows lie side by side at 16 lane in the
        // order that the tensor core reads. A row's words for RUN stages are loaded together, while the RUN stages
        // before are at hand: whole 32-byte sectors, where 16 bytes a load would fetch each sector twice.
        constexpr int NR = 1 + C::PARTS;
        const int team = (warp - 2) / TEAM, w = (warp - 2) % TEAM, runs = (stages + RUN - 1) / RUN, quarters = p.scale_pitch / 16;
        const uint32_t full_at = cluster_addr(full(0), 0);
        uint4 v[2][NR][2];
        auto fetch = [&](uint4 (&to)[NR][2], int tile, int run) {
            const bool on = tile < p.tiles;
            const int ra = on ? row_a(tile) : 0, rb = on ? col_b(tile) : 0;
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                const int r = lane + 32 * w + (j ? 128 * (j - 1) : 0), row = (j ? rb : ra) + r;
                const bool in = on && (j ? r < BQ && row < p.N : row < p.M);
                const uint4* from = reinterpret_cast<const uint4*>((j ? p.scale_b : p.scale_a) + (int64_t)row * p.scale_pitch) + 2 * run;
                to[j][0] = to[j][1] = make_uint4(0, 0, 0, 0);
                if (!in) continue;
                if (p.scale_wide) {
                    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                                 : "=r"(to[j][0].x), "=r"(to[j][0].y), "=r"(to[j][0].z), "=r"(to[j][0].w), "=r"(to[j][1].x),
                                   "=r"(to[j][1].y), "=r"(to[j][1].z), "=r"(to[j][1].w)
                                 : "l"(from));
                } else {
                    to[j][0] = __ldg(from);
                    if (2 * run + 1 < quarters) to[j][1] = __ldg(from + 1);
                }
            }
        };
        struct Turn {
            int tile, run, first;  // first: the tile's first stage in the ring's line
        };
        auto after = [&](Turn t, int by) {
            for (t.run += by; t.run >= runs; t.run -= runs, t.tile += pairs, t.first += stages) {}
            return t;
        };
        Turn at = after(Turn{pair, 0, 0}, team);
        bool ok = true;
        fetch(v[0], at.tile, at.run);
        while (ok && at.tile < p.tiles) {
            const Turn next = after(at, TEAMS);
            fetch(v[1], next.tile, next.run);
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                if (!ok || at.run * RUN + i >= stages) continue;
                const int it = at.first + at.run * RUN + i, s = it % S;
                if (!bar_wait_warp(empty(s), (uint32_t)(it / S + 1) & 1u, p.err, 7)) {
                    ok = false;
                    stop = 1;
                    continue;
                }
                const uint32_t to = base + s * C::STAGE + P_BYTES + C::Q_BYTES + lane * 16 + 4 * w;
#pragma unroll
                for (int q = 0; q < QUADS; ++q)
#pragma unroll
                    for (int j = 0; j < NR; ++j)  // A's chunk, then B's parts
                        st_shared1(to + 512 * (j == 0 ? q : QUADS + q * C::PARTS + j - 1), word_of(v[0][j][i >> 1], 2 * (i & 1) + q));
                fence_smem_async();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) bar_arrive(full(s));
                    else bar_arrive_cluster(full_at + 8 * s);
                }
            }
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                v[0][j][0] = v[1][j][0];
                v[0][j][1] = v[1][j][1];
            }
            at = next;
        }
    } else {
        // ------------------------------------------------------------ results
        const int q = warp & 3, half = (warp - FIRST_EPI) >> 2;  // q: the TMEM lane quarter that this warp can read
        const uint32_t off = S * C::STAGE + (warp - FIRST_EPI) * 4096, buf = base + off;
        const uint32_t acc_empty_at = cluster_addr(acc_empty(0), 0);
        int n = 0;
        for (int tile = pair; tile < p.tiles; tile += pairs, ++n) {
            const int b = n & 1, r0 = row_a(tile) + q * 32, c0 = col_b(tile);
            if (!bar_wait_warp(acc_full(b), (uint32_t)(n >> 1) & 1u, p.err, 4) || stop) {
                stop = 1;
                break;
            }
            fence_after_sync();
            const uint32_t t = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * BQ);
            if (p.c_bulk && !p.c_f32) {
                constexpr int BOXES = BQ / 64;
#pragma unroll 1
                for (int c = half; c < BOXES; c += 2) {
                    uint32_t v[64];
                    tmem_load32(t + 64 * c, *reinterpret_cast<uint32_t(*)[32]>(v));
                    tmem_load32(t + 64 * c + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
                    tmem_load_wait();
                    store_box<false>(p, buf, v, r0, c0 + 64 * c);
                }
                if (BQ % 64 && half == (BOXES & 1)) {  // half a box is left: each lane writes its row's 64 bytes
                    uint32_t v[32];
                    tmem_load32(t + 64 * BOXES, v);
                    tmem_load_wait();
                    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.C) + (int64_t)(r0 + lane) * p.N + c0 + 64 * BOXES;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (r0 + lane < p.M && c0 + 64 * BOXES + 8 * j < p.N)  // N is a multiple of 8
                            *reinterpret_cast<uint4*>(to + 8 * j) = make_uint4(pair_bf16(v[8 * j], v[8 * j + 1]), pair_bf16(v[8 * j + 2], v[8 * j + 3]),
                                                                               pair_bf16(v[8 * j + 4], v[8 * j + 5]), pair_bf16(v[8 * j + 6], v[8 * j + 7]));
                }
            } else {
#pragma unroll 1
                for (int c = half; c < BQ / 32; c += 2) {
                    uint32_t v[32];
                    tmem_load32(t + 32 * c, v);
                    tmem_load_wait();
                    if (p.c_bulk) store_box<true>(p, buf, v, r0, c0 + 32 * c);
                    else if (c0 + 32 * c < p.N && r0 < p.M) store_chunk(p, reinterpret_cast<float4*>(gbase + off), v, r0, c0 + 32 * c);
                }
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) bar_arrive_cluster(acc_empty_at + 8 * b);
        }
        if (lane == 0) tma_store_done();
        __syncwarp();
    }
    fence_before_sync();
    __syncwarp();
    cluster_barrier();  // neither CTA's memory goes while the other's copies, products or arrivals may reach it
    if (warp == 1) {
        fence_after_sync();
        tmem_free_pair(tmem, 512);
    }
}

// C in boxes of 128 bytes x 32 rows, 128-byte swizzle.
bool mx_map_out(CUtensorMap* m, void* C, bool f32, int64_t M, int64_t N) {
    const MxEncodeFn fn = mx_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M};
    cuuint64_t strides[1] = {(cuuint64_t)(N * (f32 ? 4 : 2))};
    cuuint32_t box[2] = {f32 ? 32u : 64u, 32};
    cuuint32_t one[2] = {1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, C, dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BQ>
cudaError_t launch(PairParams& p, const void* b_codes, int64_t pitch, cudaStream_t s) {
    auto kern = gemm_mx4_pair_kernel<BQ>;
    using C = Cfg<BQ>;
    static SmemAllowance allowed;
    const cudaError_t e = allowed.ensure(reinterpret_cast<const void*>(kern), C::SMEM);
    if (e != cudaSuccess) return e;
    if (!mx_map_rows(&p.map_b, b_codes, p.N, pitch, BQ / 2, false)) return cudaErrorInvalidValue;
    const int64_t tiles = (int64_t)p.tiles_m * ((p.N + BQ - 1) / BQ);
    if (tiles > 0x3fffffffll) return cudaErrorInvalidValue;
    p.tiles = (int)tiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * std::min(p.tiles, std::max(1, gemm_num_sms() / 2)));
    cfg.blockDim = dim3(THREADS);
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
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// Tile width: the rounds of the pairs times a tile's cost, its loaded rows for each stage and its columns'
// way out.
int tile_columns(int tiles_m, int N, int stages) {
    const int pairs = std::max(1, gemm_num_sms() / 2);
    int best = 0;
    int64_t least = 0;
    for (int bq : {224, 192, 128, 64}) {
        const int64_t tiles = (int64_t)tiles_m * ((N + bq - 1) / bq), rounds = (tiles + pairs - 1) / pairs;
        const int64_t cost = rounds * ((int64_t)stages * (TILE_P + bq / 2) + bq);
        if (!best || cost < least) {
            best = bq;
            least = cost;
        }
    }
    return best;
}

}  // namespace

cudaError_t launch_gemm_mx(const void* a_codes, const void* a_scales, const void* b_codes, const void* b_scales, void* C,
                           bool c_f32, int M, int N, int K, uint32_t* err, cudaStream_t s) {
    if (M <= 0) return cudaSuccess;
    PairParams p;
    memset(&p, 0, sizeof(p));
    const int64_t pitch = mx_code_pitch(K);
    if (!mx_map_rows(&p.map_a, a_codes, M, pitch, TILE_P, false)) return cudaErrorInvalidValue;
    p.scale_a = static_cast<const uint8_t*>(a_scales);
    p.scale_b = static_cast<const uint8_t*>(b_scales);
    p.scale_pitch = (int)mx_scale_pitch(K);
    p.scale_wide = (reinterpret_cast<uintptr_t>(a_scales) | reinterpret_cast<uintptr_t>(b_scales) | (uintptr_t)p.scale_pitch) % 32 == 0;
    p.M = M;
    p.N = N;
    p.k_stages = (K + 255) / 256;
    p.tiles_m = (M + 2 * TILE_P - 1) / (2 * TILE_P);
    p.C = C;
    p.c_f32 = c_f32;
    const int size = c_f32 ? 4 : 2;
    p.c_bulk = (reinterpret_cast<uintptr_t>(C) | (uint64_t)N * size) % 16 == 0;
    if (p.c_bulk && !mx_map_out(&p.map_c, C, c_f32, M, N)) return cudaErrorInvalidValue;
    p.err = err;
    switch (tile_columns(p.tiles_m, N, p.k_stages)) {
        case 64: return launch<64>(p, b_codes, pitch, s);
        case 128: return launch<128>(p, b_codes, pitch, s);
        case 192: return launch<192>(p, b_codes, pitch, s);
        default: return launch<224>(p, b_codes, pitch, s);
    }
}

}  // namespace ls
