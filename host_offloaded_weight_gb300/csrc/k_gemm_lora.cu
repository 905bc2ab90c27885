// A shared projection with low-rank adapters of many requests beside it:
//   C[t] = epi(W x_t + s_a up_a (down_a x_t)),  a = ids[t]  (none for a row whose id is not an adapter's)
//
// Two launches. lora_rows_kernel writes h_t = s_a down_a x_t as blocks: one for each tile of rows and each adapter with a row in
// it, zero in the rows of others. The shared product then takes a block with its adapter's `up` as some more columns of K. It
// starts as soon as the first kernel's CTAs run: its loads of the shared weights need nothing of it, only these last columns do.
// h is kept as two bf16 terms, 16 bits (the first term alone would be off by 2^-9, as much as the result's own rounding), and as
// three, 24 bits, where the result is asked for in fp32 too.
//
// 0 times infinity is NaN, so in a block an adapter with a NaN or an infinity would reach rows of other requests.
//
// What bounds it. 16 rows with 14 adapters of rank 16 beside 13824 x 5120: 35 us, the weights alone (ids of no adapter) 31, the floor
// 22; 64 rows and 24 adapters of rank 32 beside 5120 x 13824, fp32 results too: 50.5 us, alone 36. What the adapters add is the
// time of the first kernel, whose loads queue behind the stream of weights (14 us for the 64 rows, 21 MB of `down`; its 48 CTAs and the
// product's 120 have 152 SMs, so 6 of the product's 40 clusters of three start when h is done), and the stages of `up` at the end (5 us).
// One row beside 4096 x 1024 takes 13.5 us, a chain of latencies: ids 1, first load 2.5, sums 1.5, the next kernel's look at them 1.5,
// `up` 2, results 1.5, and two launches.
// Rows of full tiles: 2048 rows gate/up beside 13824 x 5120 take 372 us, lsk_gemm_bf16 in turn with it 341 (20 us the first kernel,
// 8 the stages of `up`); 4096 rows of 4096 x 1024 with rank 64 45 and 30. The pair kernel starts when h is computed.
// Tiles of fewer weight rows, so that all SMs have a share of the weights, changed nothing (13824 rows in 144 tiles of 96 in place
// of 108 of 128: 30.8 us both, and 41 for 35 with adapters, whose kernel then finds no SM free). That is 4.6 TB/s of the weights alone
// where a copy moves 6.7: what the other 9 us are is not known.
//
// Up to 128 rows (gemm_lora_few_kernel, below): the weights are the left operand (128 rows a tile) and the tokens the
// right one, 16 to 128 columns. Each part of `up` is looked over in shared memory before its product.
// More rows: the pair kernel of k_gemm.cu, whose operands lie in two SMs. Other CTAs of the first kernel look over the `up`
// matrices of the adapters in use (bytes that the product then finds in L2). One that is not finite is read out of bounds, which
// gives zeros, against one more term that is NaN in its own rows: they come out NaN, no others do.
#include <algorithm>

#include "kernels.h"
#include "tc.cuh"

namespace ls {
namespace {

using namespace tc;

constexpr int ROWS_THREADS = 256, ROWS_MAX_STAGES = 16;
constexpr int MAX_TILE = 256;
constexpr int MAX_SLICES = 8;         // of K
constexpr int LOOK_CTAS = 192;        // that look adapters over, at most

__device__ __forceinline__ uint32_t not_finite(uint32_t w) {  // two bf16
    return (uint32_t)((w & 0x7f80u) == 0x7f80u) | (uint32_t)((w & 0x7f800000u) == 0x7f800000u);
}

// 16 bytes, or zeros. Volatile, so that the eight of a step are all requested before the first is looked at.
__device__ __forceinline__ uint4 load16(const __nv_bfloat16* at, bool on) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(at), "r"((int)on));
    return v;
}

// The notes on the adapters in use, 16 bytes each: nonzero where a value of its `up` matrices is not finite. Which are in use is
// known by the low bits of their numbers (others that share them are looked over too).
__device__ __forceinline__ void look_over(const LoraArgs& p, int cta, int ctas) {
    constexpr int BITS = 4096;
    __shared__ uint32_t s_used[BITS / 32];
    if (threadIdx.x < BITS / 32) s_used[threadIdx.x] = 0;
    __syncthreads();
    for (int64_t t0 = threadIdx.x; t0 < p.T; t0 += 8 * ROWS_THREADS) {
        uint32_t a[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = (uint32_t)__ldg(p.ids + min(t0 + i * ROWS_THREADS, (int64_t)p.T - 1)) % BITS;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i == 0 || a[i] != a[i - 1]) atomicOr(&s_used[a[i] / 32], 1u << (a[i] % 32));
    }
    __syncthreads();
    const int64_t units = (int64_t)p.N * p.rank / 8;  // of 16 bytes
    const int bytes = 16 / p.check_parts;
    for (int64_t i = cta; i < (int64_t)p.n * p.check_parts; i += ctas) {
        const int a = (int)(i / p.check_parts), part = (int)(i % p.check_parts);
        if (!(s_used[a % BITS / 32] >> (a % 32) & 1)) continue;
        const int64_t u0 = units * part / p.check_parts, u1 = units * (part + 1) / p.check_parts;
        uint32_t bad = 0;
        for (int half = 0; half < (p.up2 ? 2 : 1); ++half) {
            const uint4* u = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(half ? p.up2 : p.up) + a * p.up_stride);
            for (int64_t k0 = u0 + threadIdx.x; k0 < u1; k0 += 8 * ROWS_THREADS) {
                uint4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = load16(reinterpret_cast<const __nv_bfloat16*>(u + k0 + i * ROWS_THREADS), k0 + i * ROWS_THREADS < u1);
#pragma unroll
                for (int i = 0; i < 8; ++i) bad |= not_finite(v[i].x) | not_finite(v[i].y) | not_finite(v[i].z) | not_finite(v[i].w);
            }
        }
        bad = __syncthreads_or((int)bad);
        if (threadIdx.x < bytes) p.notes[16ll * a + part * bytes + threadIdx.x] = bad ? 1 : 0;
    }
}

__device__ __forceinline__ uint64_t narrow_desc(uint32_t addr, int cw);
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate);

// ------------------------------------------------------------------ h
// A cluster of CTAs, a slice of K each, has a run of a tile's rows (all of a few-row tile, half of a full one) and up to 128 columns
// of h, for one adapter of the tile after the other, or for a gang of several at a time whose columns lie side by side: `down` is
// the left operand of the products (its rows, 128 with what lies behind them, whose results nobody reads), the rows of x, all of
// them, the right one. The CTAs' sums are added through their shared memory, each CTA finishing its share of the groups of eight
// rows, in the order of the CTAs. Bound by the latencies of its steps: ids, first loads, sums.
// (Register products, m16n8k16, from plain loads of a row's 64 bytes by four lanes took 55 to 110 us for 2048 rows of 5120.)
// The nearest bf16 that is finite where v is.
__device__ __forceinline__ float near_bf16(float v) {
    const float h = __bfloat162float(__float2bfloat16_rn(v));
    return isinf(h) && !isinf(v) ? __bfloat162float(__float2bfloat16_rz(v)) : h;
}
constexpr int ROWS_PROD = 0, ROWS_MMA = 1, ROWS_EPI = 2, ROWS_EPI_WARPS = 4;
constexpr int ROWS_CHAIN = 16;        // stages that an accumulator takes at most where h has three terms

// ROUNDS: h in three terms from slices too long for its chains.
template <bool ROUNDS>
__global__ void __launch_bounds__(ROWS_THREADS) lora_rows_kernel(const __grid_constant__ LoraArgs p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(16) int s_ids[MAX_TILE];
    __shared__ int s_list[MAX_TILE];
    __shared__ int s_warp[ROWS_THREADS / 32];
    __shared__ uint32_t s_tmem;
    __shared__ __align__(8) uint64_t s_bars[2 * ROWS_MAX_STAGES + 4];
    __shared__ volatile int stop;
    if ((int)blockIdx.x >= p.rows_ctas) {
        look_over(p, (int)blockIdx.x - p.rows_ctas, (int)gridDim.x - p.rows_ctas);
        return;
    }
    const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
    const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
    const int S = p.stages, down_bytes = p.block_cols * 128, stage = down_bytes + p.run * 128;
    float* red = reinterpret_cast<float*>(smem_raw + (base - raw) + S * stage);
    const uint32_t bars = smem_addr(s_bars);
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (ROWS_MAX_STAGES + s); };
    const uint32_t acc_full = bars + 8u * 2 * ROWS_MAX_STAGES, red_full = acc_full + 8u, round_full = acc_full + 16u, round_empty = acc_full + 24u;
    // slices (a cluster) innermost, then runs of columns, slots, runs of rows
    int at = (int)blockIdx.x;
    const int slice = at % p.slices;
    at /= p.slices;
    const int col0 = at % p.col_runs * 128;   // of an adapter's columns: parts of width cw side by side
    at /= p.col_runs;
    const int slot = at % p.slots;
    at /= p.slots;
    const int runs = p.tile_rows / p.run, tile = at / runs, row0 = at % runs * p.run, t0 = tile * p.tile_rows;

    if (tid == 0) {
        stop = 0;
        for (int s = 0; s < S; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
        }
        bar_init(acc_full, 1);
        bar_init(red_full, 1);
        bar_init(round_full, 1);
        bar_init(round_empty, ROWS_EPI_WARPS);
        bar_init_fence();
        tma_desc_prefetch(&p.map_x);
        tma_desc_prefetch(&p.map_down);
    }
    if (warp == ROWS_MMA) tmem_get(smem_addr(&s_tmem), p.tmem_cols);
    // the tile's adapters, in the order of their first rows
    int id = -1;
    if (tid < p.tile_rows && t0 + tid < p.T) {
        id = __ldg(p.ids + t0 + tid);
        if (id < 0 || id >= p.n) id = -1;
    }
    s_ids[tid] = id;
    __syncthreads();
    // not the first of its adapter: one of the rows before it is the same (rows of a request lie together: mostly the last one)
    bool first = id >= 0 && !(tid > 0 && s_ids[tid - 1] == id);
    if (first) {
        uint32_t seen = 0;
#pragma unroll 8
        for (int u = 0; u < tid; u += 4) {
            const int4 v = *reinterpret_cast<const int4*>(s_ids + u);
            seen |= (uint32_t)(v.x == id) | (uint32_t)(u + 1 < tid && v.y == id) | (uint32_t)(u + 2 < tid && v.z == id) | (uint32_t)(u + 3 < tid && v.w == id);
        }
        first = !seen;
    }
    __syncwarp();
    const uint32_t vote = __ballot_sync(0xffffffffu, first);
    if (lane == 0) s_warp[warp] = __popc(vote);
    __syncthreads();
    int before = 0, count = 0;
    for (int w = 0; w < ROWS_THREADS / 32; ++w) {
        if (w < warp) before += s_warp[w];
        count += s_warp[w];
    }
    if (first) s_list[before + __popc(vote & ((1u << lane) - 1u))] = id;
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (row0 == 0 && col0 == 0 && slot == 0 && slice == 0) {
        if (tid < count) p.list[(int64_t)tile * p.cap + tid] = s_list[tid];
        if (tid == 0) p.count[tile] = count;
    }
    // A product of few rows may start beside this kernel from here on (one of many waits for its memory traffic to pass: loads
    // took 15 us behind the pair kernel's first ones). Not before tensor memory is taken: the product might take all that is left.
    if (p.tile_rows != 256) grid_release();
    const uint32_t tmem = s_tmem;
    const int k0 = (int)((int64_t)slice * p.k_stages / p.slices), k1 = (int)((int64_t)(slice + 1) * p.k_stages / p.slices);
    // (divisions by numbers that only the launch knows take 150 clocks each: counters and shifts below)
    const int log_cw = p.cw == 16 ? 4 : p.cw == 32 ? 5 : 6;
    // Rounds of stages: between two, the epilogue's warps add the accumulators to the sums so far, which lie behind them.
    const int rounds = ROUNDS && k1 - k0 > p.round ? (k1 - k0 + p.round - 1) / p.round : 1;
    const int chains = min(k1 - k0 - (rounds - 1) * p.round, p.chains);   // of the last round
    const int own_cols = min(128, p.parts * p.cw - col0), part0 = col0 >> log_cw, parts = own_cols >> log_cw;   // of an adapter
    // the finish: a thread has the same two columns of every row, of an adapter of the gang
    const int log_units = 31 - __clz(own_cols * p.gang) - 1, log_own = 31 - __clz(own_cols), c = (tid & ((1 << log_units) - 1)) * 2;
    const int member = c >> log_own, own_c = c & (own_cols - 1);
    const int groups = p.run / 8, own_groups = (groups + p.slices - 1) / p.slices;
    const int q = warp & 3, col = 32 * q + lane;   // the epilogue: q the TMEM lane quarter that a warp can read, col the lane's column
    const int rows = min(p.run, p.T - t0 - row0);  // rows that exist (zero and less: none)
    int it = 0, turn = 0, joined = 0;              // stages, adapters and rounds before an adapter's last so far
    bool left = false, came = true;                // everything is sent; everything is here
    int ring = 0;                                  // the place of the next stage, and the parity of its use
    uint32_t parity = 0;
    if (p.slices > 1) cluster_barrier_smem();           // the others' shared memory is there
    for (int j = slot * p.gang; j < count; j += p.slots * p.gang) {
        const int members = min(p.gang, count - j), cols = members * own_cols;
        bool any = true;                               // few rows are one run, with a row of each adapter
        if (p.gang == 1) {
            bool mine = false;
            for (int r = tid; r < rows; r += ROWS_THREADS) mine = mine || s_ids[row0 + r] == s_list[j];
            any = __syncthreads_or(mine);              // the same in the cluster
        }
        const int a = member < members ? s_list[j + member] : -2;   // this thread's: no row has -2
        if (any) {
            auto step = [&]() {
                if (++ring == S) {
                    ring = 0;
                    parity ^= 1u;
                }
            };
            if (warp == ROWS_PROD) {
                const bool one = elect_one();
                for (int k = k0; k < k1; ++k, step()) {
                    const int s = ring;
                    if (!bar_wait_warp(empty(s), parity ^ 1u, p.err, 1)) {
                        stop = 1;
                        break;
                    }
                    if (one) {
                        const uint32_t to = base + s * stage;
                        bar_expect(full(s), cols * 128 + p.run * 128);
                        for (int i = 0, m = 0, part = part0; m < members; ++i) {
                            const int half = part >= p.chunks;
                            tma_4d(to + i * p.cw * 128, &p.map_down, full(s), k * 64, (part - half * p.chunks) * p.cw, half, s_list[j + m]);
                            if (++part == part0 + parts) {
                                part = part0;
                                ++m;
                            }
                        }
                        tma_2d(to + down_bytes, &p.map_x, full(s), k * 64, t0 + row0);
                    }
                    __syncwarp();
                }
            } else if (warp == ROWS_MMA) {
                const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(p.run >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
                const bool one = elect_one();
                int taken = 0;                     // stages of the round
                for (int k = k0; k < k1; ++k, ++taken, step()) {
                    const int s = ring;
                    if (ROUNDS && taken == p.round) {
                        if (one) mma_commit(round_full);
                        __syncwarp();
                        if (!bar_wait_warp(round_empty, (uint32_t)joined++ & 1u, p.err, 12)) {
                            stop = 1;
                            break;
                        }
                        fence_after_sync();
                        taken = 0;
                    }
                    if (!bar_wait_warp(full(s), parity, p.err, 3)) {
                        stop = 1;
                        break;
                    }
                    fence_after_sync();
                    if (one) {
                        const uint32_t sp = base + s * stage;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_bf16(tmem + (uint32_t)((taken & (p.chains - 1)) * p.run), operand_desc(sp + 32 * i), operand_desc(sp + down_bytes + 32 * i), idesc,
                                     taken >= p.chains || i ? 1u : 0u);
                        mma_commit(empty(s));
                    }
                    __syncwarp();
                }
                if (one) mma_commit(acc_full);
                __syncwarp();
            }
            it += k1 - k0;
        }
        // this CTA's rows and columns, two columns a thread: row r is row (r & 7) of its r / 8th group
        const int own = groups > slice ? (groups - slice + p.slices - 1) / p.slices * 8 : 0;
        const float scale = any && p.scale && a >= 0 ? __ldg(p.scale + a) : 1.f;
        const int64_t term = (int64_t)p.tile_rows * p.cw / 2;
        const int64_t block = ((int64_t)tile * p.cap + j + member) * p.parts + part0 + (own_c >> log_cw);
        auto each = [&](auto f) {   // f(row of the run, local row, where its pair of h goes)
            if (a == -2) return;
            for (int l = tid >> log_units; l < own; l += ROWS_THREADS >> log_units) {
                const int r = (slice + (l >> 3) * p.slices) * 8 + (l & 7);
                f(r, l, reinterpret_cast<uint32_t*>(p.h + (block * p.blocks_terms * p.tile_rows + row0 + r) * p.cw + (own_c & (p.cw - 1))));
            }
        };
        __syncwarp();
        // zeros in the rows of others, while the loads are on their way (the two warps that see to those come later)
        each([&](int r, int, uint32_t* to) {
            if (s_ids[row0 + r] == a) return;
            for (int t = 0; t < p.blocks_terms; ++t) to[t * term] = 0;
        });
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16), whole = lanes + (uint32_t)(p.chains * p.run);
        // eight rows' sums of this lane's column: of the rounds before, of so many accumulators
        auto sums = [&](int g, bool before, int accumulators, float (&v)[8]) {
            uint32_t x[8];
            if (ROUNDS && before) {
                tmem_load8(whole + 8 * g, x);
                tmem_load_wait();
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(x[i]);
            }
            for (int c = 0; c < accumulators; ++c) {
                tmem_load8(lanes + (uint32_t)(c * p.run + 8 * g), x);
                tmem_load_wait();
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = c || (ROUNDS && before) ? v[i] + __uint_as_float(x[i]) : __uint_as_float(x[i]);
            }
        };
        if (ROUNDS && any && warp >= ROWS_EPI && warp < ROWS_EPI + ROWS_EPI_WARPS)
            for (int r = 1; r < rounds; ++r) {
                if (!bar_wait_warp(round_full, (uint32_t)joined++ & 1u, p.err, 13)) {
                    stop = 1;
                    break;
                }
                fence_after_sync();
                if (32 * q < cols)
                    for (int g = 0; g < groups && 8 * g < rows; ++g) {
                        float v[8];
                        sums(g, r > 1, p.chains, v);
                        tmem_store8(whole + 8 * g, v);
                    }
                tmem_store_wait();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) bar_arrive(round_empty);
            }
        if (any) {
            const bool done = bar_wait_warp(acc_full, (uint32_t)turn & 1u, p.err, 4);   // every warp: nobody is ahead by an adapter
            if (!done) stop = 1;
            if (p.slices > 1 && tid == 0) {   // what comes to this CTA: its groups with rows, from each
                int due = 0;
                for (int g = slice; g < groups && 8 * g < rows; g += p.slices) ++due;
                bar_expect(red_full, due * p.slices * 8 * cols * 4);
            }
            __syncwarp();
            const bool last = j + p.slots * p.gang >= count;
            if (last) grid_release();
            fence_after_sync();
            ++turn;
            // every CTA's sums of a row go to the CTA that has it
            if (warp >= ROWS_EPI && warp < ROWS_EPI + ROWS_EPI_WARPS && 32 * q < cols)
                for (int g = 0, owner = 0, l = 0; g < groups && 8 * g < rows; ++g) {
                    float v[8];
                    sums(g, rounds > 1, chains, v);
                    const uint32_t to = smem_addr(red + ((slice * own_groups + l) * 8) * p.block_cols + col);
                    if (col < cols) {
                        if (p.slices == 1) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) st_shared1(to + i * p.block_cols * 4, __float_as_uint(v[i]));
                        } else {
                            const uint32_t there = cluster_addr(to, owner), counted = cluster_addr(red_full, owner);
#pragma unroll
                            for (int i = 0; i < 8; ++i) st_async(there + i * p.block_cols * 4, v[i], counted);
                        }
                    }
                    if (++owner == p.slices) {
                        owner = 0;
                        ++l;
                    }
                }
            fence_before_sync();
            __syncwarp();
            if (p.slices == 1) {
                __syncthreads();
            } else {
                left = last;
                if (left) cluster_arrive();
                came = bar_wait_cluster(red_full, (uint32_t)(turn - 1) & 1u, p.err, 10);
                if (!came) stop = 1;
            }
            each([&](int r, int l, uint32_t* to) {
                if (s_ids[row0 + r] != a) return;
                float2 v = make_float2(0.f, 0.f);
                const float* from = red + l * p.block_cols + c;
                for (int o = 0; o < p.slices; ++o, from += own_groups * 8 * p.block_cols) {
                    const float2 x = *reinterpret_cast<const float2*>(from);
                    v.x += x.x;
                    v.y += x.y;
                }
                // each term is what the ones before it leave, to the nearest bf16
                v.x *= scale;
                v.y *= scale;
                for (int t = 0; t < p.terms; ++t) {
                    const float2 h = make_float2(near_bf16(v.x), near_bf16(v.y));
                    to[t * term] = __float_as_uint(h.x) >> 16 | (__float_as_uint(h.y) & 0xffff0000u);
                    v.x = isfinite(h.x) ? v.x - h.x : 0.f;
                    v.y = isfinite(h.y) ? v.y - h.y : 0.f;
                }
                if (p.blocks_terms > p.terms) to[p.terms * term] = 0x7fc07fc0u;  // NaN
            });
        }
        fence_before_sync();
        __syncwarp();
        if (j + p.slots * p.gang >= count) break;
        // the next adapter's sums go where these were read
        if (p.slices > 1 && any) cluster_barrier_smem();
        else __syncthreads();
        fence_after_sync();
    }
    if (stop && warp == ROWS_PROD)  // an aborted CTA waits for its own copies before it exits
        for (int i = 0; i < S && i < it; ++i) bar_wait(full(i), (uint32_t)((it - 1 - (it - 1 - i) % S) / S) & 1u, p.err, 5);
    __syncwarp();
    if (left) {  // an aborted CTA's memory does not go while others' sums may reach it
        cluster_wait();
        if (!came) bar_wait_cluster(red_full, (uint32_t)(turn - 1) & 1u, p.err, 11);
    }
    fence_before_sync();
    __syncthreads();
    if (warp == ROWS_MMA) {
        fence_after_sync();
        tmem_free(tmem, p.tmem_cols);
    }
}

// ------------------------------------------------------------------ the shared product, few rows
// The tensor core cuts its fp32 sums off, so a long chain of products loses 2^-25 and more of the sum with each: an accumulator takes
// CHAIN stages at a time, and the epilogue's warps add it up in registers (64 x 5120 x 13824: off by 3.1e-6 in one chain, now 2e-7).
//
// One CTA an SM, persistent over tiles of 128 weight rows (SwiGLU: 64 gate rows and their 64 up rows). Warp 0 loads by TMA,
// warp 1 issues the products (kind::f16, 128 x NQ x 16), warps 2 to 5 write the results. Few tiles are shared along K by a
// cluster, whose CTAs add the sums of every so many groups of eight tokens out of their shared memory, in a fixed order.
// After its stages of the shared weights a CTA takes its share of the tile's adapter stages: 128 rows of `up` (rows of
// 32, 64 or 128 bytes: 16, 32 or 64 columns, whatever holds the rank) and both terms of the block of h.
constexpr int CHAIN = 4;  // stages
constexpr int TILE_P = 128, P_BYTES = TILE_P * 128, FEW_EPI = 4, FEW_THREADS = 32 * (2 + FEW_EPI);

// PACK: the right operand's room in a stage, in rows of x.
template <int NQ, int PACK>
struct Few {
    static constexpr int Q_BYTES = PACK * NQ * 128;
    static constexpr int STAGE = P_BYTES + Q_BYTES;
    static constexpr int MAX_SPLIT = NQ <= 16 ? 8 : 4;
    // the others' sums of the groups of eight tokens that this CTA of n finishes
    static constexpr int red(int n) { return (n - 1) * ((NQ / 8 + n - 1) / n) * 8 * TILE_P * 4; }
    static constexpr int most_red() {
        int most = 0;
        for (int n = 2; n <= MAX_SPLIT; ++n) most = red(n) > most ? red(n) : most;
        return most;
    }
    static constexpr int RED_BYTES = most_red();
    static constexpr int X_BYTES = 2 * 8 * 64 * 4;                // SwiGLU: the up rows' sums on their way to the gate rows' warps
    // As many as a block may have: no CTA of the first kernel (80 KB and more) finds room beside a ring of any use. 64 x 5120 x 13824,
    // 24 adapters: 49.1 us, 49.7 from 200 KB; 128 rows of 8 adapters 46.1 and 48.0; 128 rows of as many, 4096 x 4096, 36.2 and 36.9.
    static constexpr int FIT = (225 * 1024 - RED_BYTES - X_BYTES - 1024 - 512) / STAGE;
    static constexpr int STAGES = FIT < 9 ? FIT : 9;
    static constexpr int SMEM = STAGES * STAGE + RED_BYTES + X_BYTES + 1024 + 512;
    static constexpr int COLS = 4 * NQ;                           // of tensor memory: two accumulators, a tile's sums (and a quarter not used)
    static_assert(STAGES >= 4 && SMEM + 1024 <= 232448, "shared memory, with the static arrays");
};

struct FewLora {
    CUtensorMap map_w, map_x, map_h, map_up, map_up2;
    int M, N, K;
    int k_stages, tiles, splits;
    int dual, b2_row_off, epi;
    int cw, chunks, parts, rank;   // columns of a part of h; parts of a rank, of an adapter
    int terms, fit, pack, split;   // terms of h, of a stage; blocks of a stage, or stages of a block
    const int* count;
    const int* list;
    const int* ids;
    const __nv_bfloat16* bias;
    const void* resid;
    int resid_f32;
    __nv_bfloat16* C;
    float* C32;
    uint32_t* err;
};

// Operand with rows of cw bf16 values along K and the swizzle of that width.
__device__ __forceinline__ uint64_t narrow_desc(uint32_t addr, int cw) {
    const uint64_t layout = cw == 64 ? 2 : cw == 32 ? 4 : 6;
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)1 << 16) | ((uint64_t)((16 * cw) >> 4) << 32) | ((uint64_t)1 << 46) | (layout << 61);
}
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// A CTA's adapter stages: every so many stages of the tile's; first: the stage's first block, part `part` of adapter j of the
// tile. p.pack blocks and all their terms, or (p.split > 1 stages a block) p.fit terms of one block, `term` and up.
struct Blocks {
    const FewLora& p;
    int all, first, term, j, part;
    __device__ __forceinline__ Blocks(const FewLora& q, int slice, int count) : p(q), all(count), first(0), term(0), j(0), part(0) { step(slice); }
    __device__ __forceinline__ void step(int stages) {
        if (p.split > 1) {
            int blocks = 0;
            for (term += stages * p.fit; term >= p.split * p.fit; term -= p.split * p.fit) ++blocks;
            stages = blocks;
        } else {
            stages *= p.pack;
        }
        first += stages;
        for (part += stages; part >= p.parts; part -= p.parts) ++j;
    }
    __device__ __forceinline__ void next() { step(p.splits); }
    __device__ __forceinline__ bool left() const { return first < all; }
    __device__ __forceinline__ int blocks() const { return min(p.pack, all - first); }
    __device__ __forceinline__ int terms() const { return min(p.fit, p.terms - term); }  // (a copy brings p.fit)
};

// GELU(v) = v Phi(v), SiLU(v) = v / (1 + e^-v)
__device__ __forceinline__ float gelu(float v) { return 0.5f * v * (1.f + erff(v * 0.70710678118654752f)); }
__device__ __forceinline__ float silu(float v) { return v / (1.f + __expf(-v)); }

template <int NQ, int PACK>
__global__ void __launch_bounds__(FEW_THREADS, 1) gemm_lora_few_kernel(const __grid_constant__ FewLora p) {
    using F = Few<NQ, PACK>;
    constexpr int S = F::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t bars = base + S * F::STAGE + F::RED_BYTES + F::X_BYTES;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (S + s); };
    auto acc_full = [&](int b) { return bars + 8u * (2 * S + b); };
    auto acc_empty = [&](int b) { return bars + 8u * (2 * S + 2 + b); };
    const uint32_t done = bars + 8u * (2 * S + 4);
    auto checked = [&](int s) { return bars + 8u * (2 * S + 5 + s); };  // an adapter stage's values are finite
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (bars - base) + 8 * (3 * S + 5));
    __shared__ volatile int stop;
    __shared__ int s_list[LORA_FEW_ROWS];  // the loading warp's copy of the adapters
    const int warp = uniform_warp(), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        stop = 0;
        for (int s = 0; s < S; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
            bar_init(checked(s), FEW_EPI);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(acc_full(b), 1);
            bar_init(acc_empty(b), FEW_EPI);
        }
        bar_init(done, 1);
        bar_init_fence();
        tma_desc_prefetch(&p.map_w);
        tma_desc_prefetch(&p.map_x);
        tma_desc_prefetch(&p.map_h);
        tma_desc_prefetch(&p.map_up);
    }
    if (warp == 1) tmem_get(smem_addr(tmem_slot), F::COLS);
    fence_before_sync();
    __syncwarp();
    if (p.splits > 1) cluster_barrier();
    else __syncthreads();
    fence_after_sync();
    // The kernel before this one is this call's own and began when everything earlier was complete: the weights and the rows
    // of x may be read at once, only the blocks have to be waited for.
    const uint32_t tmem = *tmem_slot;
    const int slice = (int)blockIdx.x % p.splits, tile0 = (int)blockIdx.x / p.splits, step = (int)gridDim.x / p.splits;
    const int k0 = (int)((int64_t)slice * p.k_stages / p.splits), k1 = (int)((int64_t)(slice + 1) * p.k_stages / p.splits);
    const int rows = p.dual ? TILE_P / 2 : TILE_P;  // columns of C of a tile

    if (warp == 0) {
        // ------------------------------------------------------------ loads
        const bool one = elect_one();
        int s = 0, it = 0, more = -1;
        uint32_t phase = 1;  // a new barrier's preceding phase counts as complete
        bool ok = true;
        auto turn = [&]() {  // waits for a stage to be free
            if (!bar_wait_warp(empty(s), phase, p.err, 1)) {
                ok = false;
                stop = 1;
            }
            return ok;
        };
        auto next = [&]() {
            __syncwarp();
            ++it;
            if (++s == S) {
                s = 0;
                phase ^= 1u;
            }
        };
        for (int tile = tile0; ok && tile < p.tiles; tile += step) {
            const int n0 = tile * rows;
            for (int k = k0; k < k1 && turn(); ++k, next()) {
                if (!one) continue;
                const uint32_t at = base + s * F::STAGE;
                bar_expect(full(s), P_BYTES + NQ * 128);
                tma_2d(at, &p.map_w, full(s), k * 64, n0);  // a box of 128 rows, or two of 64
                if (p.dual) tma_2d(at + P_BYTES / 2, &p.map_w, full(s), k * 64, p.b2_row_off + n0);
                tma_2d(at + P_BYTES, &p.map_x, full(s), k * 64, 0);
            }
            if (!ok) break;
            if (more < 0) {
                grid_wait();
                const int count = *p.count;
                for (int j = lane; j < count; j += 32) s_list[j] = p.list[j];
                __syncwarp();
                more = count * p.parts;
            }
            const int up_bytes = TILE_P * p.cw * 2, h_bytes = NQ * p.cw * 2;
            Blocks at_block(p, slice, more);
            for (; at_block.left() && turn(); at_block.next(), next()) {
                if (!one) continue;
                const uint32_t at = base + s * F::STAGE;
                const int blocks = at_block.blocks();
                bar_expect(full(s), blocks * (up_bytes + p.fit * h_bytes));
                int j = at_block.j, part = at_block.part;
                for (int i = 0; i < blocks; ++i) {
                    const int half = part >= p.chunks, col = (part - (half ? p.chunks : 0)) * p.cw, a = s_list[j];
                    // out of bounds: zeros, for the other half of a SwiGLU tile
                    const CUtensorMap* up = half ? &p.map_up2 : &p.map_up;
                    const uint32_t to = at + i * up_bytes;
                    tma_3d(to, up, full(s), col, half ? p.N : n0, a);
                    if (p.dual) tma_3d(to + up_bytes / 2, up, full(s), col, half ? n0 : p.N, a);
                    tma_2d(at + P_BYTES + i * p.fit * h_bytes, &p.map_h, full(s), 0, ((at_block.first + i) * p.terms + at_block.term) * NQ);
                    if (++part == p.parts) {
                        part = 0;
                        ++j;
                    }
                }
            }
        }
        if (more < 0) grid_wait();
        grid_release();
        // an aborted CTA waits for its own copies before it exits
        if (stop)
            for (int i = 0; i < S && i < it; ++i) {
                const int last = it - 1 - (it - 1 - i) % S;
                bar_wait(full(i), (uint32_t)(last / S) & 1u, p.err, 5);
            }
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(NQ >> 3) << 17) | ((uint32_t)(TILE_P >> 4) << 24);
        const bool one = elect_one();
        int n = 0, it = 0, more = -1;
        uint32_t uses = 0;
        bool ok = true;
        const uint32_t low_p = operand_low(base), low_q = operand_low(base + P_BYTES);
        uint32_t d = 0, add = 0;
        int left = 0;                   // stages that this chain still takes
        auto chain = [&]() {            // the accumulator for the next stage
            if (left > 0) return true;
            const int b = n & 1;
            if (!bar_wait_warp(acc_empty(b), (uint32_t)((n >> 1) + 1) & 1u, p.err, 2) || stop) {
                ok = false;
                stop = 1;
                return false;
            }
            fence_after_sync();
            d = tmem + (uint32_t)(b * NQ);
            add = 0;
            left = CHAIN;
            return true;
        };
        auto close = [&](bool last) {   // after a stage's products
            __syncwarp();
            add = 1;
            if (--left > 0 && !last) return;
            if (one) mma_commit(acc_full(n & 1));
            __syncwarp();
            left = 0;
            ++n;
        };
        for (int tile = tile0; ok && tile < p.tiles; tile += step) {
            for (int k = k0; k < k1 && chain(); ++k, ++it) {
                const int s = it % S;
                if (!bar_wait_warp(full(s), (uint32_t)(it / S) & 1u, p.err, 3)) {
                    ok = false;
                    stop = 1;
                    break;
                }
                fence_after_sync();
                const uint32_t off = (uint32_t)s * (F::STAGE >> 4);
                if (one) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) mma_bf16(d, operand_from(low_p + off + 2 * i), operand_from(low_q + off + 2 * i), IDESC, i ? 1u : add);
                    mma_commit(empty(s));
                }
                close(k + 1 == k1);
            }
            if (ok && more < 0) {
                grid_wait();
                more = *p.count * p.parts;
            }
            const int up_bytes = TILE_P * p.cw * 2, h_bytes = NQ * p.cw * 2;
            Blocks at_block(p, slice, more);
            while (ok && at_block.left() && chain()) {
                const int s = it % S;
                if (!bar_wait_warp(checked(s), uses >> s & 1u, p.err, 9)) {  // the stage's uses for adapters have a count of their own
                    ok = false;
                    stop = 1;
                    break;
                }
                uses ^= 1u << s;
                fence_after_sync();
                const uint32_t sp = base + s * F::STAGE, sq = sp + P_BYTES;
                const int blocks = at_block.blocks(), terms = at_block.terms();
                if (one) {
                    int part = at_block.part;
                    for (int i = 0; i < blocks; ++i) {
                        const int chunk = part >= p.chunks ? part - p.chunks : part, steps = (min(p.cw, p.rank - chunk * p.cw) + 15) / 16;
                        for (int k = 0; k < steps; ++k)
                            for (int t = 0; t < terms; ++t) {
                                mma_bf16(d, narrow_desc(sp + i * up_bytes + 32 * k, p.cw), narrow_desc(sq + (i * p.fit + t) * h_bytes + 32 * k, p.cw),
                                         IDESC, add);
                                add = 1;
                            }
                        if (++part == p.parts) part = 0;
                    }
                    mma_commit(empty(s));
                }
                at_block.next();
                ++it;
                close(!at_block.left());
            }
        }
        if (one) mma_commit(done);
        __syncwarp();
        bar_wait(done, 0, p.err, 6);
    } else {
        // ------------------------------------------------------------ results
        const int q = warp & 3, row = 32 * q + lane;  // q: the TMEM lane quarter that this warp can read
        const int groups = (p.M + 7) / 8, own_groups = (NQ / 8 + p.splits - 1) / p.splits;
        float* red = reinterpret_cast<float*>(gbase + S * F::STAGE);
        float* swap = reinterpret_cast<float*>(gbase + S * F::STAGE + F::RED_BYTES);
        // An aborted warp goes through the same steps, without waits and results: the others meet it at the barrier below.
        bool dead = false;
        int turn = 0;
        // eight tokens' sums of this lane's weight row, whole: on to C
        auto finish = [&](int n0, int g, float (&v)[8]) {
            const int col = n0 + (p.dual ? row & 63 : row);
            if (p.dual) {
                float* x = swap + (turn++ & 1) * 8 * 64 + (row & 63);
                if (q >= 2) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[64 * j] = v[j];
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (q >= 2) return;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = silu(v[j]) * x[64 * j];
            }
            if (col >= p.N || dead) return;
            const bool has_bias = p.epi == EPI_BIAS_GELU || p.epi == EPI_BIAS_RESID;
            const bool has_resid = p.epi == EPI_BIAS_RESID || p.epi == EPI_RESID;
            const float bias = has_bias ? __bfloat162float(p.bias[col]) : 0.f;
            const int64_t at = (int64_t)8 * g * p.N + col;
            float r[8] = {};
            if (has_resid) {  // all loads before the first store: the residual may be what C32 or C overwrites
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (8 * g + j < p.M)
                        r[j] = p.resid_f32 ? static_cast<const float*>(p.resid)[at + (int64_t)j * p.N]
                                           : __bfloat162float(static_cast<const __nv_bfloat16*>(p.resid)[at + (int64_t)j * p.N]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (8 * g + j >= p.M) continue;
                float y = v[j] + bias;
                if (p.epi == EPI_BIAS_GELU) y = gelu(y);
                y += r[j];
                if (has_resid && p.C32) p.C32[at + (int64_t)j * p.N] = y;
                p.C[at + (int64_t)j * p.N] = __float2bfloat16_rn(y);
            }
        };
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16), whole = lanes + 2 * NQ;  // whole: this warp's place for a tile's sums
        auto sums = [&](int g, float (&v)[8]) {
            uint32_t x[8];
            tmem_load8(whole + 8 * g, x);
            tmem_load_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(x[j]);
        };
        float sum[NQ];
        int n = 0, it = 0, more = -1;   // chains, stages, adapter blocks of a tile
        auto collect = [&](bool first) {
            const int b = n & 1;
            if (!dead && (!bar_wait_warp(acc_full(b), (uint32_t)(n >> 1) & 1u, p.err, 4) || stop)) {
                stop = 1;
                dead = true;
            }
            fence_after_sync();
#pragma unroll
            for (int g = 0; g < NQ / 8; ++g) {
                if (g >= groups) break;
                uint32_t x[8];
                tmem_load8(lanes + (uint32_t)(b * NQ + 8 * g), x);
                tmem_load_wait();
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[8 * g + j] = first ? __uint_as_float(x[j]) : sum[8 * g + j] + __uint_as_float(x[j]);
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) bar_arrive(acc_empty(b));
            ++n;
        };
        for (int tile = tile0; tile < p.tiles; tile += step) {
            for (int k = k0; k < k1; k += CHAIN) collect(k == k0);
            // Adapter stages first pass by these warps, a quarter each. 0 times infinity is NaN: a value that is not finite would
            // reach rows of other adapters. It becomes zero, and the adapter's own rows of h NaN.
            // (A wait by parity cannot tell a use of a stage from the one two before it. The last chain above is complete, so every use
            // before these is over.)
            it += k1 - k0;
            if (more < 0) {
                grid_wait();
                more = *p.count * p.parts;
            }
            const int up_bytes = TILE_P * p.cw * 2, h_bytes = NQ * p.cw * 2;
            Blocks at_block(p, slice, more);
            for (int in_chain = 0; at_block.left(); ++it) {
                const int s = it % S;
                if (!dead && !bar_wait_warp(full(s), (uint32_t)(it / S) & 1u, p.err, 8)) {
                    stop = 1;
                    dead = true;
                }
                int j = at_block.j, part = at_block.part;
                for (int i = 0; !dead && i < at_block.blocks(); ++i) {
                    uint8_t* v = gbase + s * F::STAGE + i * up_bytes + q * (up_bytes / 4);
                    uint32_t bad = 0;
#pragma unroll 4
                    for (int o = lane * 16; o < up_bytes / 4; o += 512) {
                        const uint4 w = *reinterpret_cast<const uint4*>(v + o);
                        bad |= not_finite(w.x) | not_finite(w.y) | not_finite(w.z) | not_finite(w.w);
                    }
                    if (__any_sync(0xffffffffu, bad)) {
                        for (int o = lane * 2; o < up_bytes / 4; o += 64) {
                            uint16_t* w = reinterpret_cast<uint16_t*>(v + o);
                            if ((*w & 0x7f80) == 0x7f80) *w = 0;
                        }
                        const int a = p.list[j];
                        uint8_t* h = gbase + s * F::STAGE + P_BYTES + i * p.fit * h_bytes;  // its rows, whatever the order within one
                        for (int t = 0; t < p.M; ++t)
                            if (p.ids[t] == a && lane < p.cw / 2) *reinterpret_cast<uint32_t*>(h + (t * p.cw + lane * 2) * 2) = 0x7fc07fc0u;
                    }
                    if (++part == p.parts) {
                        part = 0;
                        ++j;
                    }
                }
                fence_smem_async();
                __syncwarp();
                if (lane == 0) bar_arrive(checked(s));
                at_block.next();
                if (++in_chain == CHAIN || !at_block.left()) {
                    collect(false);
                    in_chain = 0;
                }
            }
#pragma unroll
            for (int g = 0; g < NQ / 8; ++g) {
                if (g >= groups) break;
                tmem_store8(whole + 8 * g, sum + 8 * g);
            }
            tmem_store_wait();
#pragma unroll 1
            for (int g = 0, owner = -1, l = 0; g < groups; ++g) {  // l: the owner's groups before this one
                if (++owner == p.splits) {
                    owner = 0;
                    ++l;
                }
                if (p.splits > 1 && owner == slice) continue;
                float v[8];
                sums(g, v);
                if (p.splits == 1) {
                    finish(tile * rows, g, v);
                } else {
                    const int at = (slice - (slice > owner)) * own_groups + l;
                    const uint32_t to = cluster_addr(base + S * F::STAGE + at * 8 * TILE_P * 4, owner);
#pragma unroll
                    for (int j = 0; j < 8; ++j) st_cluster(to + (j * TILE_P + row) * 4, v[j]);
                }
            }
        }
        if (p.splits > 1) {
            // a cluster has one tile; its sums are added in the order of the CTAs, this one's own first
            __syncwarp();
            cluster_barrier();
#pragma unroll 1
            for (int g = slice, l = 0; g < groups; g += p.splits, ++l) {
                float v[8];
                sums(g, v);
#pragma unroll 1
                for (int o = 0; o < p.splits - 1; ++o)
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += red[((o * own_groups + l) * 8 + j) * TILE_P + row];
                finish(tile0 * rows, g, v);
            }
        }
    }
    if (p.splits > 1 && warp < 2) {
        __syncwarp();
        cluster_barrier();
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        tmem_free(tmem, F::COLS);
    }
}

// ------------------------------------------------------------------ host side
// The `down` matrices [n][two][rank, K] in boxes of 64 values x cw rows, 128-byte swizzle.
bool map_down(CUtensorMap* m, const LoraArgs& p, int two) {
    const MxEncodeFn fn = mx_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[4] = {(cuuint64_t)p.K, (cuuint64_t)p.rank, (cuuint64_t)two, (cuuint64_t)p.n};
    cuuint64_t strides[3] = {(cuuint64_t)p.K * 2, (cuuint64_t)p.K * 2 * p.rank, (cuuint64_t)p.down_stride};
    cuuint32_t box[4] = {64, (cuuint32_t)p.cw, 1, 1};
    cuuint32_t one[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p.down), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int few_rows(int M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

// CTAs (a cluster) that share a tile along K: a CTA's stages (64 values of K, about a third of a microsecond each), and
// what joining the sums takes, in stages.
int few_splits(int tiles, int k_stages, int most) {
    int best = 1, least = k_stages;
    for (int n = 2; n <= most && n <= k_stages && tiles * n <= gemm_num_sms(); ++n) {
        const int cost = (k_stages + n - 1) / n + 6;
        if (cost < least) {
            least = cost;
            best = n;
        }
    }
    return best;
}

cudaLaunchConfig_t config(dim3 grid, int threads, int smem, cudaStream_t s, cudaLaunchAttribute* at, bool early) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = early ? 1 : 0;
    return cfg;
}

// The grid of lora_rows_kernel and its maps.
cudaError_t launch_rows(LoraArgs& p, bool dual, cudaStream_t s) {
    const int cols = p.parts * p.cw;
    p.run = std::min(p.tile_rows, 128);
    // Adapters of few rows go together, as many as 128 columns hold: x is read once for them, and more SMs are left for the product
    // to start on. 128 rows of as many adapters of rank 16, 4096 x 4096: 44 us one by one, now 36; 8 rows 21.7 and 17.4; 128 rows
    // of 8 adapters of rank 32, 5120 x 13824: 53 and 42. (64 columns at most: 24 adapters of rank 32 49 us for 51, but the last 51.)
    const bool few = p.tile_rows != 256;
    const int most_adapters = (int)std::min<int64_t>(p.cap, p.T);
    p.gang = 1;
    while (few && 2 * p.gang * cols <= 128 && p.gang < most_adapters) p.gang *= 2;
    p.block_cols = std::min(p.gang * cols, 128);
    p.col_runs = (cols + 127) / 128;
    p.k_stages = (p.K + 63) / 64;
    // Accumulators that the stages take in turn (the tensor core cuts its sums off, see CHAIN below). Two CTAs of an SM get by with
    // its tensor memory: one that waited for another's could hold up its cluster, and that the other.
    p.chains = std::min(4, 256 / p.run);
    p.tmem_cols = p.chains * p.run;
    // 80 KB of loads in flight; the products read 128 rows of the last stage's left operand, whatever lies behind it
    const int stage = (p.block_cols + p.run) * 128;
    p.stages = std::max(3, std::min(ROWS_MAX_STAGES, 81920 / stage));
    // A cluster for each run of rows and columns and each gang that there may be (few rows) or two adapters (a full tile has few), over
    // slices of 96 KB and more; as many as are resident together, two an SM, beside some that look adapters over (1024 rows of 16
    // adapters, 5120 x 13824: 161 us; 174 with 48 more places left to those and 64 KB in flight).
    const int64_t runs = p.tiles * (p.tile_rows / p.run) * p.col_runs, room = 2 * gemm_num_sms() - (few ? 0 : LOOK_CTAS / 4);
    p.slots = few ? (most_adapters + p.gang - 1) / p.gang : std::min(p.cap, 2);
    p.slices = (int)std::max<int64_t>(1, std::min<int64_t>({MAX_SLICES, (int64_t)p.k_stages * stage / 98304, room / (runs * p.slots)}));
    if (few && runs * p.slots * p.slices <= gemm_num_sms()) p.stages = std::min(ROWS_MAX_STAGES, 131072 / stage);  // an SM to itself
    while (!few && 2 * p.slots <= p.cap && runs * p.slices * 2 * p.slots <= room) p.slots *= 2;
    // Slices that are long all the same (many rows or adapters, K beyond 8 slices) are taken in rounds where h has three terms, with
    // half of the accumulators and the sums so far in place of the others. The adapters' part of fp32 results at K = 13824, of its norm
    // (us beside 5120, 2048 and 1024 weight rows): 128 rows, as many adapters of rank 256, off by 7.8e-6 in one round (524), 1.1e-6
    // now (570); 4096 rows, 64 of rank 64, 2.0 and 1.2e-6 (1303, 1436); 16384 rows, 2 of rank 16, 7.7 and 1.1e-6 (474, 498).
    p.round = p.k_stages;
    if (p.terms == 3 && (p.k_stages + p.slices - 1) / p.slices > ROWS_CHAIN * p.chains) {
        p.chains /= 2;
        p.round = ROWS_CHAIN * p.chains;
    }
    const int groups = p.run / 8, red = p.slices * ((groups + p.slices - 1) / p.slices) * 8 * p.block_cols * 4;
    // not less than 80 KB: a third CTA of an SM would wait for tensor memory
    const int smem = std::max(80 * 1024, 1024 + p.stages * stage + std::max(red, 128 * 128));
    const int64_t rows = runs * p.slots * p.slices, most = std::max<int64_t>(LOOK_CTAS / 6, std::min<int64_t>(LOOK_CTAS, 2 * gemm_num_sms() - rows));
    const int64_t looks = few ? 0 : std::min<int64_t>((most + p.slices - 1) / p.slices, ((int64_t)p.n * p.check_parts + p.slices - 1) / p.slices) * p.slices;
    if (rows + looks > 0x7fffffffll) return cudaErrorInvalidValue;
    p.rows_ctas = (int)rows;
    if (!lora_map(&p.map_x, p.x, p.T, p.K, 64, p.run, 0, 0) || !map_down(&p.map_down, p, dual ? 2 : 1)) return cudaErrorInvalidValue;
    const bool rounds = p.round < p.k_stages;
    auto kern = rounds ? lora_rows_kernel<true> : lora_rows_kernel<false>;
    static SmemAllowance allowed[2];
    const cudaError_t e = allowed[rounds].ensure(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t cfg = config(dim3((unsigned)(rows + looks)), ROWS_THREADS, smem, s, at, false);
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = p.slices;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.numAttrs = p.slices > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int NQ, int PACK>
cudaError_t launch_few(FewLora& p, int rows, const void* h, int64_t h_rows, cudaStream_t s) {
    auto kern = gemm_lora_few_kernel<NQ, PACK>;
    using F = Few<NQ, PACK>;
    static SmemAllowance allowed;
    const cudaError_t e = allowed.ensure(reinterpret_cast<const void*>(kern), F::SMEM);
    if (e != cudaSuccess) return e;
    p.tiles = (p.N + rows - 1) / rows;
    // what a stage has room for beside 128 rows of `up`, of term rows as long as those of x; a copy has up to 256 rows
    const int room = F::Q_BYTES / (NQ * p.cw * 2);
    p.fit = std::min({p.terms, room, 256 / NQ});
    p.split = (p.terms + p.fit - 1) / p.fit;
    p.pack = p.split > 1 ? 1 : std::min(room / p.fit, 64 / p.cw);
    if (!lora_map(&p.map_h, h, h_rows, p.cw, p.cw, p.fit * NQ, 0, 0)) return cudaErrorInvalidValue;
    p.splits = few_splits(p.tiles, p.k_stages, F::MAX_SPLIT);
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t cfg = config(dim3(p.splits > 1 ? p.tiles * p.splits : std::min(p.tiles, gemm_num_sms())), FEW_THREADS, F::SMEM, s, at, true);
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = p.splits;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    if (p.splits > 1) cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

struct Layout {  // of a call's scratch
    int64_t count, list, notes, h, bytes;
};

Layout layout(const LoraArgs& p) {
    Layout l;
    l.count = 0;
    l.list = up256(4 * p.tiles);
    l.notes = l.list + up256(4 * p.tiles * p.cap);
    l.h = l.notes + up256(16ll * p.n);
    l.bytes = l.h + p.tiles * p.cap * p.parts * 2ll * p.blocks_terms * p.tile_rows * p.cw;
    return l;
}

}  // namespace

bool lora_map(CUtensorMap* m, const void* ptr, int64_t rows, int64_t cols, int box_cols, int box_rows, int64_t n, int64_t stride) {
    const MxEncodeFn fn = mx_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)n};
    cuuint64_t strides[2] = {(cuuint64_t)(2 * cols), (cuuint64_t)stride};
    cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
    cuuint32_t one[3] = {1, 1, 1};
    const CUtensorMapSwizzle sw = box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, n ? 3 : 2, const_cast<void*>(ptr), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool lora_plan(LoraArgs& p, bool dual, bool fp32) {
    p.cw = p.rank <= 16 ? 16 : p.rank <= 32 ? 32 : 64;
    p.chunks = (p.rank + p.cw - 1) / p.cw;
    p.parts = p.chunks * (dual ? 2 : 1);
    p.tile_rows = p.T <= LORA_FEW_ROWS ? few_rows(p.T) : 256;
    p.tiles = ((int64_t)p.T + p.tile_rows - 1) / p.tile_rows;
    p.cap = std::min(p.n, p.tile_rows);
    // CTAs that look an adapter over, 16 KB and more each
    p.check_parts = 1;
    while (p.check_parts < 16 && (int64_t)p.N * p.rank * 2 / p.check_parts > 24576) p.check_parts *= 2;
    // blocks are rows of one tensor map, counted in 32 bits
    p.terms = fp32 ? 3 : 2;
    p.blocks_terms = p.terms + (p.tile_rows == 256 ? 1 : 0);
    return p.tiles * p.cap * p.parts * p.blocks_terms * p.tile_rows <= 0x7fffffffll && (int64_t)p.n * p.check_parts <= 0x3fffffffll;
}

int64_t lora_ws_bytes(const LoraArgs& p) { return layout(p).bytes; }

cudaError_t launch_gemm_lora(const GemmDesc& d, LoraArgs& p, void* ws, cudaStream_t s) {
    const bool dual = d.epi == EPI_SWIGLU;
    const Layout l = layout(p);
    uint8_t* w = static_cast<uint8_t*>(ws);
    p.count = reinterpret_cast<int*>(w + l.count);
    p.list = reinterpret_cast<int*>(w + l.list);
    p.notes = w + l.notes;
    p.h = reinterpret_cast<__nv_bfloat16*>(w + l.h);
    const bool few = p.tile_rows != 256;
    const cudaError_t e = launch_rows(p, dual, s);
    if (e != cudaSuccess) return e;
    const int64_t h_rows = p.tiles * p.cap * p.parts * p.blocks_terms * p.tile_rows;
    if (!few) return launch_gemm_bf16_lora(d, p, h_rows, s);
    const int rows = dual ? TILE_P / 2 : TILE_P;
    FewLora f;
    memset(&f, 0, sizeof(f));
    if (!lora_map(&f.map_w, d.B, d.b_rows, d.K, 64, rows, 0, 0) || !lora_map(&f.map_x, d.A, d.M, d.K, 64, p.tile_rows, 0, 0) ||
        !lora_map(&f.map_up, p.up, d.N, p.rank, p.cw, rows, p.n, p.up_stride) ||
        (dual && !lora_map(&f.map_up2, p.up2, d.N, p.rank, p.cw, rows, p.n, p.up_stride)))
        return cudaErrorInvalidValue;
    f.M = d.M;
    f.N = d.N;
    f.K = d.K;
    f.k_stages = (d.K + 63) / 64;
    f.dual = dual;
    f.b2_row_off = d.b2_row_off;
    f.epi = d.epi;
    f.cw = p.cw;
    f.chunks = p.chunks;
    f.parts = p.parts;
    f.rank = p.rank;
    f.terms = p.terms;
    f.count = p.count;
    f.list = p.list;
    f.ids = p.ids;
    f.bias = static_cast<const __nv_bfloat16*>(d.bias);
    f.resid = d.resid;
    f.resid_f32 = d.resid_f32;
    f.C = static_cast<__nv_bfloat16*>(d.C);
    f.C32 = static_cast<float*>(d.C32);
    f.err = d.err_word;
    // 64 rows: room for all terms of a block beside its `up`, where the smaller stage has it not and the block would be two stages
    // that both read `up` (64 adapters of rank 64 beside 13824 x 5120: 108 us, now 79). Elsewhere the smaller stage, of which there
    // are seven in place of five: 36.6 us for 37.5 without adapters (64 x 5120 x 13824).
    switch (p.tile_rows) {
        case 16: return launch_few<16, 2>(f, rows, p.h, h_rows, s);
        case 32: return launch_few<32, 2>(f, rows, p.h, h_rows, s);
        case 64: return p.terms * p.cw > 64 ? launch_few<64, 2>(f, rows, p.h, h_rows, s) : launch_few<64, 1>(f, rows, p.h, h_rows, s);
        default: return launch_few<128, 1>(f, rows, p.h, h_rows, s);
    }
}

}  // namespace ls
