// Products with MXFP4 matrices on the sm_103a tensor cores (tcgen05, block-scaled).
//
//   4-bit x 4-bit   C[M,N] = sum_k A[m,k] B[n,k], both MXFP4: kind::mxf4, 64 values of K an
//                   instruction, codes packed in shared memory as they lie in global memory.
//   bf16 x 4-bit    C[M,N] = sum_k A[m,k] B[n,k], A bf16, B MXFP4: kind::mxf8f6f4. The weights
//                   are the left operand (128 rows a tile) and the tokens the right one, so a
//                   single token costs 16 columns instead of 128 padded rows. The tensor core has no bf16 x E2M1 form;
//                   a bf16 value has 8 significant bits and an E4M3 value 4, so A is written as two
//                   E4M3 terms with a power-of-two scale for each block of 32:
//                     a = t1 2^s1 + t2 2^s2,  s1 = floor(log2 max|a|) - 7,  s2 = s1 - 5.
//                   t1 is a 2^-s1 to the nearest, t2 the rest: exact for every value down to 2^-13 of its
//                   block's largest, below that within 2^-22 of the largest. Both terms are columns
//                   of the same product and are added in fp32 in the epilogue.
//
// Structure (one persistent CTA per SM): warp 0 loads operand tiles by TMA (128-byte rows,
// 128-byte swizzle) into a ring of stages; warps 2-5 bring the scales, 16 bytes a row at a
// time, into the stage in the order that the tensor core reads them (32 rows of 16 bytes, the
// four 32-row groups side by side); warp 1 copies the scales to TMEM and issues the
// products; the others write the results. The scales' TMEM columns belong to the stage, so
// the barrier that frees a stage orders their reuse too.
//
// Sums are fp32 and each output is written by one thread from a fixed order of sums.
#include <algorithm>
#include <mutex>

#include "kernels.h"
#include "tc.cuh"

namespace ls {
namespace {

using namespace tc;

enum { MX_MX = 0, ACT_MX = 1 };

constexpr int TILE_P = 128;               // rows of the left operand in a tile
constexpr int P_BYTES = TILE_P * 128;     // a stage of it

template <int MODE, int BQ>
struct Cfg {
    static constexpr int QUADS = MODE == MX_MX ? 2 : 1;        // words of four blocks (128 values of K) in a stage
    static constexpr int PARTS = (BQ + 127) / 128;             // 128-row parts of the right operand's scales
    static constexpr int Q_BYTES = BQ * 128;
    static constexpr int SCALE_BYTES = QUADS * (1 + PARTS) * 512;
    static constexpr int STAGE = (P_BYTES + Q_BYTES + SCALE_BYTES + 1023) / 1024 * 1024;
    static constexpr int EPI_WARPS = MODE == MX_MX ? 8 : 4;
    static constexpr int EPI_BYTES = MODE == MX_MX ? EPI_WARPS * 32 * 33 * 4 : 0;
    static constexpr int FIT = (232448 - 1024 - 512 - EPI_BYTES) / STAGE;
    static constexpr int STAGES = FIT < 10 ? FIT : 10;
    static constexpr int SMEM = STAGES * STAGE + EPI_BYTES + 1024 + 512;
    static constexpr int THREADS = 32 * (6 + EPI_WARPS);
    static constexpr int ACCS = 2 * BQ + STAGES * QUADS * 4 * (1 + PARTS) <= 512 ? 2 : 1;
    static constexpr int SCALE_COLS = QUADS * 4 * (1 + PARTS);  // TMEM columns of a stage's scales
    static_assert(ACCS * BQ + STAGES * SCALE_COLS <= 512, "tensor memory");
    static_assert(BQ % 16 == 0 && BQ <= 256, "columns of a product");
};

struct MxParams {
    CUtensorMap map_p, map_q;
    const uint8_t* scale_p;
    const uint8_t* scale_q;
    int scale_pitch;
    int rows_p, rows_q;   // rows of the operands (ACT_MX: rows_q = tokens)
    int q_term_rows;      // ACT_MX: rows between the two terms
    int k_stages;         // stages along K
    int tiles_p, tiles_q, tiles;
    void* C;
    int64_t ldc;
    int c_f32;
    float* partial;       // ACT_MX: [2 * grid][BQ / 2][128] sums of tiles that several CTAs share
    uint32_t* tickets;    // ACT_MX: [tiles][4], zero before the launch
    uint32_t* err;
};

// The pieces of work of a CTA, in order. 4-bit x 4-bit: whole tiles. bf16 x 4-bit: the tiles'
// stages in one line, cut evenly over the CTAs, so that every SM streams the same share of
// the weights whatever the number of tiles; a tile that is cut is summed by its last CTA.
template <int MODE>
struct Work {
    int64_t pos, end;
    int k_stages, tile, k0, k1;
    __device__ __forceinline__ Work(const MxParams& p) : k_stages(p.k_stages), tile(0), k0(0), k1(0) {
        if (MODE == MX_MX) {
            pos = blockIdx.x;
            end = p.tiles;
        } else {
            const int64_t total = (int64_t)p.tiles * p.k_stages;
            pos = blockIdx.x * total / gridDim.x;
            end = (blockIdx.x + 1) * total / gridDim.x;
        }
    }
    __device__ __forceinline__ bool next() {
        if (pos >= end) return false;
        if (MODE == MX_MX) {
            tile = (int)pos;
            k0 = 0;
            k1 = k_stages;
            pos += gridDim.x;
        } else {
            tile = (int)(pos / k_stages);
            k0 = (int)(pos - (int64_t)tile * k_stages);
            k1 = (int)min((int64_t)k_stages, k0 + (end - pos));
            pos += k1 - k0;
        }
        return true;
    }
};

template <int MODE>
__device__ __forceinline__ void tile_at(const MxParams& p, int tile, int bq, int& row_p, int& row_q) {
    if (MODE == MX_MX) {
        row_p = tile % p.tiles_p * TILE_P;
        row_q = tile / p.tiles_p * bq;
    } else {  // the token tiles of one weight tile follow one another
        row_p = tile / p.tiles_q * TILE_P;
        row_q = tile % p.tiles_q * (bq / 2);
    }
}

__device__ __forceinline__ void store_c(const MxParams& p, int64_t at, float v) {
    if (p.c_f32) static_cast<float*>(p.C)[at] = v;
    else static_cast<__nv_bfloat16*>(p.C)[at] = __float2bfloat16_rn(v);
}

template <int MODE, int BQ>
__global__ void __launch_bounds__(Cfg<MODE, BQ>::THREADS, 1) gemm_mx_kernel(const __grid_constant__ MxParams p) {
    using C = Cfg<MODE, BQ>;
    constexpr int S = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t bars = base + S * C::STAGE + C::EPI_BYTES;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (S + s); };
    auto acc_full = [&](int b) { return bars + 8u * (2 * S + b); };
    auto acc_empty = [&](int b) { return bars + 8u * (2 * S + 2 + b); };
    const uint32_t done = bars + 8u * (2 * S + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (bars - base) + 8 * (2 * S + 5));
    __shared__ volatile int stop;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        stop = 0;
        for (int s = 0; s < S; ++s) {
            bar_init(full(s), 1 + 4);  // the TMA thread and the four scale warps
            bar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(acc_full(b), 1);
            bar_init(acc_empty(b), C::EPI_WARPS);
        }
        bar_init(done, 1);
        bar_init_fence();
    }
    if (warp == 1) tmem_get(smem_addr(tmem_slot), 512);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    grid_wait();
    const uint32_t tmem = *tmem_slot;
    Work<MODE> w(p);

    if (warp == 0) {
        // ------------------------------------------------------------ operand tiles
        if (lane == 0) {
            tma_desc_prefetch(&p.map_p);
            tma_desc_prefetch(&p.map_q);
            int it = 0;
            bool ok = true;
            while (ok && w.next()) {
                int row_p, row_q;
                tile_at<MODE>(p, w.tile, BQ, row_p, row_q);
                for (int k = w.k0; k < w.k1; ++k, ++it) {
                    const int s = it % S;
                    if (!bar_wait(empty(s), (uint32_t)(it / S + 1) & 1u, p.err, 1)) {
                        ok = false;
                        stop = 1;
                        break;
                    }
                    const uint32_t at = base + s * C::STAGE;
                    // an unpacking copy counts the packed bytes (it leaves every second 8 bytes alone)
                    bar_expect(full(s), (MODE == MX_MX ? P_BYTES : P_BYTES / 2) + C::Q_BYTES);
                    tma_2d(at, &p.map_p, full(s), k * 128, row_p);
                    if (MODE == MX_MX) {
                        tma_2d(at + P_BYTES, &p.map_q, full(s), k * 128, row_q);
                    } else {
                        tma_2d(at + P_BYTES, &p.map_q, full(s), k * 128, row_q);
                        tma_2d(at + P_BYTES + C::Q_BYTES / 2, &p.map_q, full(s), k * 128, row_q + p.q_term_rows);
                    }
                }
            }
            grid_release();
            // an aborted CTA waits for its own copies before it exits
            if (stop)
                for (int s = 0; s < S && s < it; ++s) {
                    const int last = it - 1 - (it - 1 - s) % S;
                    bar_wait(full(s), (uint32_t)(last / S) & 1u, p.err, 5);
                }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        if (lane == 0) {
            constexpr uint32_t IDESC = MODE == MX_MX ? mx_idesc(1, 1, TILE_P, BQ) : mx_idesc(5, 0, TILE_P, BQ);
            int it = 0, n = 0;
            bool ok = true;
            while (ok && w.next()) {
                const int b = n % C::ACCS;
                if (!bar_wait(acc_empty(b), (uint32_t)(n / C::ACCS + 1) & 1u, p.err, 2) || stop) {
                    stop = 1;
                    break;
                }
                fence_after_sync();
                const uint32_t d = tmem + (uint32_t)(b * BQ);
                for (int k = w.k0; k < w.k1; ++k, ++it) {
                    const int s = it % S;
                    if (!bar_wait(full(s), (uint32_t)(it / S) & 1u, p.err, 3)) {
                        ok = false;
                        stop = 1;
                        break;
                    }
                    fence_after_sync();
                    const uint32_t sp = base + s * C::STAGE, sq = sp + P_BYTES, sc = sq + C::Q_BYTES;
                    const uint32_t tp = tmem + (uint32_t)(C::ACCS * BQ + s * C::SCALE_COLS), tq = tp + 4 * C::QUADS;
#pragma unroll
                    for (int q = 0; q < C::QUADS; ++q) {
                        scale_copy(tp + 4 * q, scale_desc(sc + 512 * q));
#pragma unroll
                        for (int j = 0; j < C::PARTS; ++j)
                            scale_copy(tq + 4 * (q * C::PARTS + j), scale_desc(sc + 512 * (C::QUADS + q * C::PARTS + j)));
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // 32 bytes of each row
                        const uint32_t acc = (k > w.k0 || i > 0) ? 1u : 0u;
                        const uint64_t dp = operand_desc(sp + 32 * i), dq = operand_desc(sq + 32 * i);
                        if (MODE == MX_MX)
                            mma_mxf4(d, dp, dq, idesc_at(IDESC, 2 * (i & 1)), tp + 4 * (i >> 1),
                                     tq + 4 * C::PARTS * (i >> 1), acc);
                        else
                            mma_mxf8(d, dp, dq, idesc_at(IDESC, i), tp, tq, acc);
                    }
                    mma_commit(empty(s));
                }
                if (ok) mma_commit(acc_full(b));
                ++n;
            }
            mma_commit(done);
            bar_wait(done, 0, p.err, 6);
        }
    } else if (warp < 6) {
        // ------------------------------------------------------------ scales
        // lane l of warp w takes row 32 (l % 4) + 8 w + l / 4 of each 128: its word's place in the
        // 512 bytes is then 128 w + 4 l, free of bank conflicts
        const int r = 32 * (lane & 3) + 8 * (warp - 2) + (lane >> 2);
        const uint32_t off = (uint32_t)((warp - 2) * 128 + lane * 4);
        int it = 0;
        bool ok = true;
        while (ok && w.next()) {
            int row_p, row_q;
            tile_at<MODE>(p, w.tile, BQ, row_p, row_q);
            const uint8_t* src[1 + C::PARTS];
            src[0] = row_p + r < p.rows_p ? p.scale_p + (int64_t)(row_p + r) * p.scale_pitch : nullptr;
#pragma unroll
            for (int j = 0; j < C::PARTS; ++j) {
                const int rq = r + 128 * j;
                int64_t at = -1;
                if (rq < BQ) {
                    if (MODE == MX_MX) at = row_q + rq < p.rows_q ? row_q + rq : -1;
                    else at = rq < BQ / 2 ? row_q + rq : row_q + rq - BQ / 2 + p.q_term_rows;
                }
                src[1 + j] = at >= 0 ? p.scale_q + at * p.scale_pitch : nullptr;
            }
            uint4 cur[1 + C::PARTS], nxt[1 + C::PARTS];
            auto load = [&](uint4(&v)[1 + C::PARTS], int group) {
#pragma unroll
                for (int j = 0; j < 1 + C::PARTS; ++j)
                    v[j] = src[j] && group * 16 < p.scale_pitch
                               ? __ldg(reinterpret_cast<const uint4*>(src[j] + group * 16))
                               : make_uint4(0, 0, 0, 0);
            };
            constexpr int PER = 4 / C::QUADS;  // stages of one 16-byte load
            load(nxt, w.k0 / PER);
            for (int k = w.k0; k < w.k1; ++k, ++it) {
                if (k == w.k0 || k % PER == 0) {
#pragma unroll
                    for (int j = 0; j < 1 + C::PARTS; ++j) cur[j] = nxt[j];
                    load(nxt, k / PER + 1);
                }
                const int s = it % S;
                if (!__all_sync(0xffffffffu, bar_wait(empty(s), (uint32_t)(it / S + 1) & 1u, p.err, 7))) {
                    ok = false;
                    stop = 1;
                    break;
                }
                const uint32_t sc = base + s * C::STAGE + P_BYTES + C::Q_BYTES + off;
#pragma unroll
                for (int j = 0; j < 1 + C::PARTS; ++j) {
                    const uint4 v = cur[j];
                    if (MODE == MX_MX) {
                        const uint32_t a = k & 1 ? v.z : v.x, b = k & 1 ? v.w : v.y;
                        // the left operand's two words, then (word, part) of the right one
                        const uint32_t w0 = j == 0 ? 0 : 2 + (j - 1), w1 = j == 0 ? 1 : 2 + C::PARTS + (j - 1);
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(sc + 512 * w0), "r"(a) : "memory");
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(sc + 512 * w1), "r"(b) : "memory");
                    } else {
                        const uint32_t a = k & 2 ? (k & 1 ? v.w : v.z) : (k & 1 ? v.y : v.x);
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(sc + 512 * j), "r"(a) : "memory");
                    }
                }
                fence_smem_async();
                __syncwarp();
                if (lane == 0) bar_arrive(full(s));
            }
        }
    } else {
        // ------------------------------------------------------------ results
        const int q = warp & 3;  // the TMEM lane quarter that this warp can read
        int n = 0;
        while (w.next()) {
            int row_p, row_q;
            tile_at<MODE>(p, w.tile, BQ, row_p, row_q);
            const int b = n % C::ACCS;
            if (!__all_sync(0xffffffffu, bar_wait(acc_full(b), (uint32_t)(n / C::ACCS) & 1u, p.err, 4) && !stop)) {
                stop = 1;
                break;
            }
            fence_after_sync();
            const uint32_t t = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * BQ);
            if (MODE == MX_MX) {
                float* buf = reinterpret_cast<float*>(gbase + S * C::STAGE) + (warp - 6) * 32 * 33;
                const int r0 = row_p + q * 32;
                const int half = (warp - 6) >> 2;
#pragma unroll 1
                for (int c = half; c < BQ / 32; c += 2) {
                    uint32_t v[32];
                    tmem_load32(t + 32 * c, v);
                    tmem_load_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) buf[lane * 33 + j] = __uint_as_float(v[j]);
                    __syncwarp();
                    const int col = row_q + 32 * c + lane;
                    if (col < p.rows_q)
                        for (int i = 0; i < 32 && r0 + i < p.rows_p; ++i)
                            store_c(p, (int64_t)(r0 + i) * p.ldc + col, buf[i * 33 + lane]);
                    __syncwarp();
                }
                fence_before_sync();
                __syncwarp();
                if (lane == 0) bar_arrive(acc_empty(b));
            } else {
                constexpr int TN = BQ / 2;
                const int row = q * 32 + lane;
                const int col = row_p + row;                   // the weight row is the output column
                const int tokens = min(TN, p.rows_q - row_q);
                const bool whole = w.k0 == 0 && w.k1 == p.k_stages;
                float* mine = p.partial + ((int64_t)(2 * blockIdx.x + (w.k0 > 0 ? 0 : 1)) * TN) * 128 + row;
#pragma unroll 1
                for (int j0 = 0; j0 < tokens; j0 += 8) {
                    uint32_t x[8], y[8];
                    tmem_load8(t + j0, x);
                    tmem_load8(t + TN + j0, y);
                    tmem_load_wait();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float v = __uint_as_float(x[j]) + __uint_as_float(y[j]);
                        if (j0 + j >= tokens) continue;
                        if (!whole) mine[(j0 + j) * 128] = v;
                        else if (col < p.rows_p) store_c(p, (int64_t)(row_q + j0 + j) * p.ldc + col, v);
                    }
                }
                fence_before_sync();
                __syncwarp();
                if (lane == 0) bar_arrive(acc_empty(b));
                if (!whole) {
                    // CTA b holds the line [b total / grid, (b + 1) total / grid)
                    const int64_t total = (int64_t)p.tiles * p.k_stages, first = (int64_t)w.tile * p.k_stages;
                    const int b0 = (int)(((first + 1) * gridDim.x - 1) / total);
                    const int b1 = (int)(((first + p.k_stages) * gridDim.x - 1) / total);
                    __threadfence();
                    __syncwarp();
                    uint32_t seen = 0;
                    if (lane == 0) seen = atomicAdd(p.tickets + 4 * w.tile + q, 1u);
                    seen = __shfl_sync(0xffffffffu, seen, 0);
                    if (seen == (uint32_t)(b1 - b0)) {  // the last of the tile's CTAs: all sums, in order
                        __threadfence();
                        for (int j = 0; j < tokens; ++j) {
                            float v = 0.f;
                            for (int i = b0; i <= b1; ++i)
                                v += __ldcg(p.partial + ((int64_t)(2 * i + (i == b0 ? 1 : 0)) * TN + j) * 128 + row);
                            if (col < p.rows_p) store_c(p, (int64_t)(row_q + j) * p.ldc + col, v);
                        }
                    }
                }
            }
            ++n;
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        tmem_free(tmem, 512);
    }
}

// The two E4M3 terms of bf16 rows (see the top) and the tickets' zeros. Terms: [2][pad rows]
// [pitch] bytes, scales likewise; rows past M are zero. A thread takes 8 values, four lanes a block.
__global__ void __launch_bounds__(256)
split_rows_kernel(const __nv_bfloat16* __restrict__ a, int64_t lda, int M, int K, int vec, int pad_rows, uint32_t per_row,
                  uint8_t* __restrict__ terms, uint8_t* __restrict__ scales, int scale_pitch, uint32_t* __restrict__ tickets,
                  int n_tickets) {
    grid_release();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t total = (int64_t)pad_rows * per_row;
    if (i < n_tickets) tickets[i] = 0;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int row = (int)(i / per_row);
    const uint32_t g = (uint32_t)(i % per_row);
    if (i < total && row < M) {
        const int k = (int)g * 8;
        const __nv_bfloat16* s = a + row * lda + k;
        if (vec && k + 8 <= K) {
            const uint4 q = *reinterpret_cast<const uint4*>(s);
            const uint32_t x[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(x[j] << 16);
                v[2 * j + 1] = __uint_as_float(x[j] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k + j < K) v[j] = __bfloat162float(s[j]);
        }
    }
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (i >= total) return;
    // s1 = e - 127 - 7 and s2 = s1 - 5 as bytes, not below 0; a block with a NaN or an infinity reads as NaN
    const uint32_t e = m >> 23;
    const uint32_t b1 = e == 255 ? 255 : e < 7 ? 0 : e - 7, b2 = e == 255 ? 255 : e < 12 ? 0 : e - 12;
    const float f1 = __uint_as_float((254 - min(b1, 253u)) << 23), u1 = e8m0_to_float(min(b1, 254u));
    const float f2 = __uint_as_float((254 - min(b2, 253u)) << 23);
    uint16_t t1[4], t2[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float x = v[2 * j], y = v[2 * j + 1];
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(t1[j]) : "f"(y * f1), "f"(x * f1));
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(t1[j]));
        const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&h));
        const float rx = x - d.x * u1, ry = y - d.y * u1;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(t2[j]) : "f"(ry * f2), "f"(rx * f2));
    }
    const bool bad = e == 255;
    uint2 o1 = make_uint2(t1[0] | (uint32_t)t1[1] << 16, t1[2] | (uint32_t)t1[3] << 16);
    uint2 o2 = make_uint2(t2[0] | (uint32_t)t2[1] << 16, t2[2] | (uint32_t)t2[3] << 16);
    if (bad) o1 = o2 = make_uint2(0, 0);
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
// View of `rows` rows of `pitch` bytes in boxes of 128 x box_rows, 128-byte swizzle. codes:
// packed 4-bit values unpacked to a byte each (128 values a row of the box).
bool map_rows(CUtensorMap* m, const void* ptr, int64_t rows, int64_t pitch, int box_rows, bool unpack) {
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

template <int MODE, int BQ>
cudaError_t launch(const MxParams& p, int grid, bool pdl, cudaStream_t s) {
    auto kern = gemm_mx_kernel<MODE, BQ>;
    using C = Cfg<MODE, BQ>;
    static const cudaError_t attr = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (attr != cudaSuccess) return attr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

// Tokens of a tile: the fewest columns that hold M, at most 128.
int act_tile(int M) { return M <= 8 ? 8 : M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

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

cudaError_t launch_gemm_mx(const void* a_codes, const void* a_scales, const void* b_codes, const void* b_scales, void* C,
                           bool c_f32, int M, int N, int K, uint32_t* err, cudaStream_t s) {
    if (M <= 0) return cudaSuccess;
    constexpr int BQ = 192;
    MxParams p;
    memset(&p, 0, sizeof(p));
    const int64_t pitch = mx_code_pitch(K);
    if (!map_rows(&p.map_p, a_codes, M, pitch, TILE_P, false) || !map_rows(&p.map_q, b_codes, N, pitch, BQ, false))
        return cudaErrorInvalidValue;
    p.scale_p = static_cast<const uint8_t*>(a_scales);
    p.scale_q = static_cast<const uint8_t*>(b_scales);
    p.scale_pitch = (int)mx_scale_pitch(K);
    p.rows_p = M;
    p.rows_q = N;
    p.k_stages = (K + 255) / 256;
    p.tiles_p = (M + TILE_P - 1) / TILE_P;
    p.tiles_q = (N + BQ - 1) / BQ;
    if ((int64_t)p.tiles_p * p.tiles_q > 0x7fffffffll) return cudaErrorInvalidValue;
    p.tiles = p.tiles_p * p.tiles_q;
    p.C = C;
    p.ldc = N;
    p.c_f32 = c_f32;
    p.err = err;
    return launch<MX_MX, BQ>(p, std::min(p.tiles, gemm_num_sms()), false, s);
}

static int act_grid(int M, int N, int K) {
    const int tn = act_tile(M);
    const int64_t stages = up(N, TILE_P) / TILE_P * (up(M, tn) / tn) * (up(K, 128) / 128);
    return (int)std::min<int64_t>(stages, gemm_num_sms());
}

int64_t act_mx_ws_bytes(int M, int N, int K) {
    const int tn = act_tile(M);
    const int64_t rows = up(M, tn), tiles = up(N, TILE_P) / TILE_P * (rows / tn);
    return 2 * rows * (up(K, 128) + mx_scale_pitch(K)) + up(16 * tiles, 256) +
           2ll * act_grid(M, N, K) * tn * 128 * (int64_t)sizeof(float) + 1024;
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
    if ((int64_t)p.tiles_p * p.tiles_q > 0x7fffffffll / 4 || 2 * rows > 0x7fffffffll) return cudaErrorInvalidValue;
    p.tiles = p.tiles_p * p.tiles_q;
    uint8_t* w = static_cast<uint8_t*>(ws);
    uint8_t* terms = w;
    w += 2 * rows * kp;
    uint8_t* scales = w;
    w += 2 * rows * p.scale_pitch;
    w = reinterpret_cast<uint8_t*>(up(reinterpret_cast<intptr_t>(w), 256));
    p.tickets = reinterpret_cast<uint32_t*>(w);
    w += up(16ll * p.tiles, 256);
    p.partial = reinterpret_cast<float*>(w);
    if (!map_rows(&p.map_p, b_codes, N, mx_code_pitch(K), TILE_P, true) || !map_rows(&p.map_q, terms, 2 * rows, kp, tn, false))
        return cudaErrorInvalidValue;
    p.scale_p = static_cast<const uint8_t*>(b_scales);
    p.scale_q = scales;
    p.rows_p = N;
    p.rows_q = M;
    p.q_term_rows = (int)rows;
    p.k_stages = (int)(kp / 128);
    p.C = C;
    p.ldc = N;
    p.c_f32 = c_f32;
    p.err = err;
    const int vec = (reinterpret_cast<uintptr_t>(a) & 15) == 0 && lda % 8 == 0;
    const uint32_t per_row = (uint32_t)(kp / 8);
    const int64_t work = std::max<int64_t>(rows * per_row, 4ll * p.tiles);
    if ((work + 255) / 256 > 0x7fffffffll) return cudaErrorInvalidValue;
    split_rows_kernel<<<(unsigned)((work + 255) / 256), 256, 0, s>>>(static_cast<const __nv_bfloat16*>(a), lda, M, K, vec,
                                                                     (int)rows, per_row, terms, scales, p.scale_pitch,
                                                                     p.tickets, 4 * p.tiles);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int grid = act_grid(M, N, K);
    switch (tn) {
        case 8: return launch<ACT_MX, 16>(p, grid, true, s);
        case 16: return launch<ACT_MX, 32>(p, grid, true, s);
        case 32: return launch<ACT_MX, 64>(p, grid, true, s);
        case 64: return launch<ACT_MX, 128>(p, grid, true, s);
        default: return launch<ACT_MX, 256>(p, grid, true, s);
    }
}

}  // namespace ls
