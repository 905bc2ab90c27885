// A shared projection with low-rank adapters of many requests beside it:
//   C[t] = epi(W x_t + s_a up_a (down_a x_t)),  a = ids[t]  (none for a row whose id is not an adapter's)
//
// Two launches. lora_rows_kernel writes h_t = s_a down_a x_t as blocks: one for each tile of rows and each adapter with a row in
// it, zero in the rows of others. The shared product then takes a block with its adapter's `up` as some more columns of K. It
// starts as soon as the first kernel's CTAs run: its loads of the shared weights need nothing of it, only these last columns do.
// h is kept as two bf16 terms (16 bits: the first term alone would be off by 2^-9, more than the fp32 sums lose).
//
// 0 times infinity is NaN, so in a block an adapter with a NaN or an infinity would reach rows of other requests. Other CTAs of the
// first kernel look over the `up` matrices of the adapters in use (bytes that the product then finds in L2). One that is not finite is
// read out of bounds, which gives zeros, against a third term that is NaN in its own rows: they come out NaN, no others do.
//
// Up to 128 rows (gemm_lora_few_kernel, below): the weights are the left operand (128 rows a tile) and the tokens the
// right one, 16 to 128 columns. More rows: the pair kernel of k_gemm.cu.
#include <algorithm>

#include "kernels.h"
#include "tc.cuh"

namespace ls {
namespace {

using namespace tc;

constexpr int DOWN_THREADS = 256, DOWN_WARPS = 8, SUB = 16;  // rows of a CTA of the down kernel
constexpr int MAX_TILE = 256;
constexpr int MAX_SLICES = 8;         // of K

__device__ __forceinline__ uint32_t not_finite(uint32_t w) {  // two bf16
    return (uint32_t)((w & 0x7f80u) == 0x7f80u) | (uint32_t)((w & 0x7f800000u) == 0x7f800000u);
}

// A part of an adapter's `up` matrices: its notes, 16 bytes an adapter, are nonzero where a value is not finite.
__device__ __forceinline__ void look_over(const LoraArgs& p, int cta) {
    const int a = cta / p.check_parts, part = cta % p.check_parts;
    int used = 0;
#pragma unroll 4
    for (int t = threadIdx.x; t < p.T; t += DOWN_THREADS) used |= __ldg(p.ids + t) == a;
    if (!__syncthreads_or(used)) return;
    const int64_t units = (int64_t)p.N * p.rank / 8;  // of 16 bytes
    const int64_t u0 = units * part / p.check_parts, u1 = units * (part + 1) / p.check_parts;
    uint32_t bad = 0;
    for (int half = 0; half < (p.up2 ? 2 : 1); ++half) {
        const uint4* u = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(half ? p.up2 : p.up) + a * p.up_stride);
#pragma unroll 8
        for (int64_t i = u0 + threadIdx.x; i < u1; i += DOWN_THREADS) {
            const uint4 v = __ldg(u + i);
            bad |= not_finite(v.x) | not_finite(v.y) | not_finite(v.z) | not_finite(v.w);
        }
    }
    bad = __syncthreads_or((int)bad);
    const int bytes = 16 / p.check_parts;
    if (threadIdx.x < bytes) p.notes[16ll * a + part * bytes + threadIdx.x] = bad ? 1 : 0;
}

// ------------------------------------------------------------------ h
// A CTA has 16 of the rows that an adapter has in a tile, 8 NT columns of h and a slice of K (a cluster has all of it), for one
// adapter of the tile after the other: m16n8k16 products (bound by the loads: the shared product's tensor core form would want 128 rows and a TMA ring for 16
// columns), K dealt to eight warps. The sums of the warps and of the cluster's CTAs are added in their order. A lane's 16 bytes of
// a row of x and of `down` are the same eight values of K, so which of them a product calls its first does not matter: a warp's
// load takes 64 bytes of each of eight rows.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int NT>
__global__ void __launch_bounds__(DOWN_THREADS) lora_rows_kernel(const __grid_constant__ LoraArgs p) {
    constexpr int COLS = 8 * NT, UNITS = SUB * COLS / 2;  // units: two columns of a row
    __shared__ __align__(16) int s_ids[MAX_TILE];
    __shared__ int s_list[MAX_TILE];
    __shared__ int s_warp[2][DOWN_WARPS];
    __shared__ int s_rows[SUB];
    __shared__ float s_sum[DOWN_WARPS][SUB][COLS + 1];
    __shared__ float2 s_red[2][UNITS + MAX_SLICES];
    grid_release();
    if ((int)blockIdx.x >= p.rows_ctas) {
        look_over(p, (int)blockIdx.x - p.rows_ctas);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // slices (a cluster) innermost, then columns, slots, 16 rows
    int at = (int)blockIdx.x;
    const int slice = at % p.slices;
    at /= p.slices;
    const int col0 = at % p.col_ctas * COLS;
    at /= p.col_ctas;
    const int slot = at % p.slots;
    at /= p.slots;
    const int subs = p.tile_rows / SUB, tile = at / subs, row0 = at % subs * SUB, t0 = tile * p.tile_rows;

    // the tile's adapters, in the order of their first rows
    int id = -1;
    if (tid < p.tile_rows && t0 + tid < p.T) {
        id = __ldg(p.ids + t0 + tid);
        if (id < 0 || id >= p.n) id = -1;
    }
    s_ids[tid] = id;
    __syncthreads();
    bool first = id >= 0;
    for (int u = 0; first && u < tid; u += 4) {
        const int4 v = *reinterpret_cast<const int4*>(s_ids + u);
        if ((v.x == id) || (u + 1 < tid && v.y == id) || (u + 2 < tid && v.z == id) || (u + 3 < tid && v.w == id)) first = false;
    }
    const uint32_t vote = __ballot_sync(0xffffffffu, first);
    if (lane == 0) s_warp[1][warp] = __popc(vote);
    __syncthreads();
    int before = 0, count = 0;
    for (int w = 0; w < DOWN_WARPS; ++w) {
        if (w < warp) before += s_warp[1][w];
        count += s_warp[1][w];
    }
    if (first) s_list[before + __popc(vote & ((1u << lane) - 1u))] = id;
    __syncthreads();
    const bool writes_list = row0 == 0 && col0 == 0 && slot == 0 && slice == 0;
    if (writes_list) {
        if (tid < count) p.list[(int64_t)tile * p.cap + tid] = s_list[tid];
        if (tid == 0) p.count[tile] = count;
    }
    if (p.slices > 1) cluster_barrier();  // the others' shared memory is there

    const int g = lane >> 2, q = lane & 3;
    const int part = col0 / p.cw, half = part / p.chunks, c0 = col0 % p.cw, r0 = part % p.chunks * p.cw + c0;  // parts of width cw, side by side
    const int k_first = slice * p.slice_k, k_end = min(p.K, k_first + p.slice_k);
    auto owner_first = [&](int o) { return (UNITS * o + p.slices - 1) / p.slices; };  // a CTA of the cluster finishes these units and up
    const int own0 = owner_first(slice), own1 = owner_first(slice + 1);
    int turn = 0;
    for (int j = slot; j < count; j += p.slots, ++turn) {
        const int a = s_list[j];
        // the adapter's rows row0, row0 + 1, ... of the tile, of however many it has
        const uint32_t mine = __ballot_sync(0xffffffffu, s_ids[tid] == a);
        if (lane == 0) s_warp[turn & 1][warp] = __popc(mine);
        __syncthreads();
        int rank = __popc(mine & ((1u << lane) - 1u)) - row0, rows = -row0;
        for (int w = 0; w < DOWN_WARPS; ++w) {
            if (w < warp) rank += s_warp[turn & 1][w];
            rows += s_warp[turn & 1][w];
        }
        if (s_ids[tid] == a && rank >= 0 && rank < SUB) s_rows[rank] = tid;
        __syncthreads();
        const bool any = rows > 0;   // the same in the cluster
        if (any) {
            const bool on0 = g < rows, on1 = g + 8 < rows;
            float acc[NT][4] = {};
            const __nv_bfloat16* x0 = p.x + (int64_t)(t0 + (on0 ? s_rows[g] : 0)) * p.K;
            const __nv_bfloat16* x1 = p.x + (int64_t)(t0 + (on1 ? s_rows[g + 8] : 0)) * p.K;
            const uint8_t* down = static_cast<const uint8_t*>(p.down) + a * p.down_stride;
            const __nv_bfloat16* d[NT];
            bool in[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int r = r0 + 8 * n + g;
                in[n] = r < p.rank;
                d[n] = reinterpret_cast<const __nv_bfloat16*>(down) + ((int64_t)half * p.rank + (in[n] ? r : 0)) * p.K;
            }
            const uint4 zero = make_uint4(0, 0, 0, 0);
            constexpr int U = NT <= 2 ? 4 : 2;
            for (int k0 = k_first + 32 * warp; k0 < k_end; k0 += 32 * DOWN_WARPS * U) {
                uint4 va[U], vb[U], vd[U][NT];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int k = k0 + 32 * DOWN_WARPS * u + 8 * q;
                    const bool k_in = k < k_end;  // K and the slices are multiples of 8
                    va[u] = on0 && k_in ? __ldg(reinterpret_cast<const uint4*>(x0 + k)) : zero;
                    vb[u] = on1 && k_in ? __ldg(reinterpret_cast<const uint4*>(x1 + k)) : zero;
#pragma unroll
                    for (int n = 0; n < NT; ++n) vd[u][n] = in[n] && k_in ? __ldg(reinterpret_cast<const uint4*>(d[n] + k)) : zero;
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma16816(acc[n], va[u].x, vb[u].x, va[u].y, vb[u].y, vd[u][n].x, vd[u][n].y);
                        mma16816(acc[n], va[u].z, vb[u].z, va[u].w, vb[u].w, vd[u][n].z, vd[u][n].w);
                    }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                s_sum[warp][g][8 * n + 2 * q] = acc[n][0];
                s_sum[warp][g][8 * n + 2 * q + 1] = acc[n][1];
                s_sum[warp][g + 8][8 * n + 2 * q] = acc[n][2];
                s_sum[warp][g + 8][8 * n + 2 * q + 1] = acc[n][3];
            }
            __syncthreads();
            float2* red = s_red[turn & 1];
            for (int i = tid; i < UNITS; i += DOWN_THREADS) {
                const int r = i / (COLS / 2), c = i % (COLS / 2) * 2;
                float2 v = make_float2(0.f, 0.f);
#pragma unroll
                for (int w = 0; w < DOWN_WARPS; ++w) {
                    v.x += s_sum[w][r][c];
                    v.y += s_sum[w][r][c + 1];
                }
                if (p.slices == 1) {
                    red[i] = v;
                } else {
                    const int o = i * p.slices / UNITS, o0 = owner_first(o), share = owner_first(o + 1) - o0;
                    const uint32_t to = cluster_addr(smem_addr(red + slice * share + i - o0), o);
                    st_cluster(to, v.x);
                    st_cluster(to + 4, v.y);
                }
            }
            if (p.slices > 1) cluster_barrier();
            else __syncthreads();
        }
        const float scale = p.scale ? p.scale[a] : 1.f;
        const float2* red = s_red[turn & 1];
        const int64_t block = (((int64_t)tile * p.cap + j) * p.parts + part) * LORA_TERMS;
        const int64_t term = (int64_t)p.tile_rows * p.cw / 2;
        for (int i = own0 + tid; i < own1; i += DOWN_THREADS) {
            const int r = i / (COLS / 2), c = i % (COLS / 2) * 2;
            uint32_t* to = reinterpret_cast<uint32_t*>(p.h + block * p.tile_rows * p.cw + c0 + c);
            // rows row0 and up of the tile that are not the adapter's are zero
            if (s_ids[row0 + r] != a) {
                uint32_t* z = to + (int64_t)(row0 + r) * p.cw / 2;
                z[0] = z[term] = z[2 * term] = 0;
            }
            if (r >= rows) continue;
            float2 v = make_float2(0.f, 0.f);
            for (int o = 0; o < p.slices; ++o) {
                const float2 x = red[o * (own1 - own0) + i - own0];
                v.x += x.x;
                v.y += x.y;
            }
            uint32_t hi = 0, lo = 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float h = r0 + c + e < p.rank ? (e ? v.y : v.x) * scale : 0.f;
                float t1 = __bfloat162float(__float2bfloat16_rn(h));
                if (isinf(t1) && !isinf(h)) t1 = __bfloat162float(__float2bfloat16_rz(h));
                const float t2 = isfinite(t1) ? h - t1 : 0.f;
                hi |= (__float_as_uint(t1) >> 16) << (16 * e);
                lo |= (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(t2)) << (16 * e);
            }
            to += (int64_t)s_rows[r] * p.cw / 2;
            to[0] = hi;
            to[term] = lo;
            to[2 * term] = 0x7fc07fc0u;  // NaN
        }
    }
}

// ------------------------------------------------------------------ the shared product, few rows
// One CTA an SM, persistent over tiles of 128 weight rows (SwiGLU: 64 gate rows and their 64 up rows). Warp 0 loads by TMA,
// warp 1 issues the products (kind::f16, 128 x NQ x 16), warps 2 to 5 write the results. Few tiles are shared along K by a
// cluster, whose CTAs add the sums of every so many groups of eight tokens out of their shared memory, in a fixed order.
// After its stages of the shared weights a CTA takes its share of the tile's adapter stages: 128 rows of `up` (rows of
// 32, 64 or 128 bytes: 16, 32 or 64 columns, whatever holds the rank) and both terms of the block of h.
constexpr int TILE_P = 128, P_BYTES = TILE_P * 128, FEW_EPI = 4, FEW_THREADS = 32 * (2 + FEW_EPI);

template <int NQ>
struct Few {
    static constexpr int Q_BYTES = 2 * NQ * 128;                  // an adapter stage's two terms
    static constexpr int STAGE = P_BYTES + Q_BYTES;
    static constexpr int MAX_SPLIT = NQ <= 16 ? 8 : NQ <= 64 ? 4 : 2;
    static constexpr int RED_BYTES = (MAX_SPLIT - 1) * NQ * TILE_P * 4;
    static constexpr int X_BYTES = 2 * 8 * 64 * 4;                // SwiGLU: the up rows' sums on their way to the gate rows' warps
    // the kernels before it need room on the same SM
    static constexpr int FIT = (200 * 1024 - RED_BYTES - X_BYTES - 1024 - 512) / STAGE;
    static constexpr int STAGES = FIT < 9 ? FIT : 9;
    static constexpr int SMEM = STAGES * STAGE + RED_BYTES + X_BYTES + 1024 + 512;
    static constexpr int COLS = 2 * NQ < 32 ? 32 : 2 * NQ;        // of tensor memory: two accumulators
    static_assert(STAGES >= 2 && SMEM <= 232448, "shared memory");
};

struct FewLora {
    CUtensorMap map_w, map_x, map_h, map_up, map_up2;
    int M, N, K;
    int k_stages, tiles, splits;
    int dual, b2_row_off, epi;
    int cw, chunks, parts, rank;   // columns of a part of h; parts of a rank, of a block
    const int* count;
    const int* list;
    const uint8_t* notes;
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

// GELU(v) = v Phi(v), SiLU(v) = v / (1 + e^-v)
__device__ __forceinline__ float gelu(float v) { return 0.5f * v * (1.f + erff(v * 0.70710678118654752f)); }
__device__ __forceinline__ float silu(float v) { return v / (1.f + __expf(-v)); }

template <int NQ>
__global__ void __launch_bounds__(FEW_THREADS, 1) gemm_lora_few_kernel(const __grid_constant__ FewLora p) {
    using F = Few<NQ>;
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
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (bars - base) + 8 * (2 * S + 5));
    __shared__ volatile int stop;
    __shared__ int s_list[LORA_FEW_ROWS];  // adapters; those that are not finite as -1 - a
    const int warp = uniform_warp(), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        stop = 0;
        for (int s = 0; s < S; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
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
                tma_2d(at, &p.map_w, full(s), k * 64, n0);  // boxes of 64 rows
                tma_2d(at + P_BYTES / 2, &p.map_w, full(s), k * 64, p.dual ? p.b2_row_off + n0 : n0 + 64);
                tma_2d(at + P_BYTES, &p.map_x, full(s), k * 64, 0);
            }
            if (!ok) break;
            if (more < 0) {
                grid_wait();
                const int count = *p.count;
                for (int j = lane; j < count; j += 32) {
                    const int a = p.list[j];
                    const uint4 n = *reinterpret_cast<const uint4*>(p.notes + 16ll * a);
                    s_list[j] = n.x | n.y | n.z | n.w ? -1 - a : a;
                }
                __syncwarp();
                more = count * p.parts;
            }
            const int up_bytes = TILE_P * p.cw * 2;
            for (int e = slice; e < more && turn(); e += p.splits, next()) {
                const int j = e / p.parts, part = e % p.parts, half = part / p.chunks, col = part % p.chunks * p.cw;
                const int a = s_list[j];
                if (!one) continue;
                const uint32_t at = base + s * F::STAGE;
                bar_expect(full(s), up_bytes + 2 * NQ * p.cw * 2);
                // out of bounds: zeros, for an adapter that is not finite and for the other half of a SwiGLU tile
                const int none = p.N;
                const CUtensorMap* up = half ? &p.map_up2 : &p.map_up;
                tma_3d(at, up, full(s), col, a < 0 || half ? none : n0, max(a, 0));
                tma_3d(at + up_bytes / 2, up, full(s), col, a < 0 || (p.dual && !half) ? none : p.dual ? n0 : n0 + 64, max(a, 0));
                tma_2d(at + P_BYTES, &p.map_h, full(s), 0, (e * LORA_TERMS + (a < 0 ? 2 : 0)) * NQ);  // two terms; the third with the next block's first
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
        bool ok = true;
        for (int tile = tile0; ok && tile < p.tiles; tile += step, ++n) {
            const int b = n & 1;
            if (!bar_wait_warp(acc_empty(b), (uint32_t)((n >> 1) + 1) & 1u, p.err, 2) || stop) {
                stop = 1;
                break;
            }
            fence_after_sync();
            const uint32_t d = tmem + (uint32_t)(b * NQ);
            uint32_t add = 0;
            auto ready = [&]() {
                if (!bar_wait_warp(full(it % S), (uint32_t)(it / S) & 1u, p.err, 3)) {
                    ok = false;
                    stop = 1;
                }
                fence_after_sync();
                return ok;
            };
            for (int k = k0; k < k1 && ready(); ++k, ++it) {
                const uint32_t sp = base + it % S * F::STAGE, sq = sp + P_BYTES;
                if (one) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) mma_bf16(d, operand_desc(sp + 32 * i), operand_desc(sq + 32 * i), IDESC, i ? 1u : add);
                    mma_commit(empty(it % S));
                }
                __syncwarp();
                add = 1;
            }
            if (ok && more < 0) {
                grid_wait();
                more = *p.count * p.parts;
            }
            for (int e = slice; ok && e < more && ready(); e += p.splits, ++it) {
                const uint32_t sp = base + it % S * F::STAGE, sq = sp + P_BYTES;
                const int left = min(p.cw, p.rank - e % p.parts % p.chunks * p.cw), steps = (left + 15) / 16;
                if (one) {
                    for (int i = 0; i < steps; ++i) {
                        const uint64_t a = narrow_desc(sp + 32 * i, p.cw);
                        mma_bf16(d, a, narrow_desc(sq + 32 * i, p.cw), IDESC, i ? 1u : add);
                        mma_bf16(d, a, narrow_desc(sq + NQ * p.cw * 2 + 32 * i, p.cw), IDESC, 1u);
                    }
                    mma_commit(empty(it % S));
                }
                __syncwarp();
                add = 1;
            }
            if (ok && one) mma_commit(acc_full(b));
            __syncwarp();
        }
        if (one) mma_commit(done);
        __syncwarp();
        bar_wait(done, 0, p.err, 6);
    } else {
        // ------------------------------------------------------------ results
        const int q = warp & 3, row = 32 * q + lane;  // q: the TMEM lane quarter that this warp can read
        const int groups = (p.M + 7) / 8;
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
            const float bias = has_bias ? __bfloat162float(p.bias[col]) : 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int t = 8 * g + j;
                if (t >= p.M) continue;
                const int64_t at = (int64_t)t * p.N + col;
                float r = v[j] + bias;
                if (p.epi == EPI_BIAS_GELU) r = gelu(r);
                if (p.epi == EPI_BIAS_RESID || p.epi == EPI_RESID) {
                    r += p.resid_f32 ? static_cast<const float*>(p.resid)[at] : __bfloat162float(static_cast<const __nv_bfloat16*>(p.resid)[at]);
                    if (p.C32) p.C32[at] = r;
                }
                p.C[at] = __float2bfloat16_rn(r);
            }
        };
        auto sums = [&](int b, int g, float (&v)[8]) {
            uint32_t x[8];
            tmem_load8(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * NQ + 8 * g), x);
            tmem_load_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(x[j]);
        };
        int n = 0;
        for (int tile = tile0; tile < p.tiles; tile += step, ++n) {
            const int b = n & 1;
            if (!dead && (!bar_wait_warp(acc_full(b), (uint32_t)(n >> 1) & 1u, p.err, 4) || stop)) {
                stop = 1;
                dead = true;
            }
            fence_after_sync();
#pragma unroll 1
            for (int g = 0; g < groups; ++g) {
                const int owner = g % p.splits;
                if (p.splits > 1 && owner == slice) continue;
                float v[8];
                sums(b, g, v);
                if (p.splits == 1) {
                    finish(tile * rows, g, v);
                } else {
                    const uint32_t to = cluster_addr(base + S * F::STAGE + ((slice - (slice > owner)) * NQ + 8 * g) * TILE_P * 4, owner);
#pragma unroll
                    for (int j = 0; j < 8; ++j) st_cluster(to + (j * TILE_P + row) * 4, v[j]);
                }
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) bar_arrive(acc_empty(b));
        }
        if (p.splits > 1) {
            // a cluster has one tile; its sums are added in the order of the CTAs, this one's own first
            __syncwarp();
            cluster_barrier();
            fence_after_sync();
#pragma unroll 1
            for (int g = slice; g < groups; g += p.splits) {
                float v[8];
                sums(0, g, v);
#pragma unroll 1
                for (int o = 0; o < p.splits - 1; ++o)
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += red[(o * NQ + 8 * g + j) * TILE_P + row];
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

template <int NT>
cudaError_t launch_rows(LoraArgs& p, cudaStream_t s) {
    const int64_t subs = p.tiles * (p.tile_rows / SUB);
    p.col_ctas = p.parts * p.cw / (8 * NT);
    // Slices of 1024 and more values of K, what a CTA's eight warps have in flight at a time; no more than fill the SMs twice
    // with CTAs that have work: one for each adapter with few rows, one for each 16 rows else.
    const int64_t busy = p.col_ctas * (p.tile_rows == 256 ? subs : std::min<int64_t>(p.cap, p.T));
    p.slices = (int)std::max<int64_t>(1, std::min<int64_t>({MAX_SLICES, (p.K + 1023) / 1024, 2 * gemm_num_sms() / busy}));
    p.slice_k = ((p.K + p.slices - 1) / p.slices + 31) / 32 * 32;
    const int64_t each = subs * p.col_ctas * p.slices;
    p.slots = (int)std::min<int64_t>(p.cap, std::max<int64_t>(1, 1024 / each));
    const int64_t rows = each * p.slots, looks = ((int64_t)p.n * p.check_parts + p.slices - 1) / p.slices * p.slices;
    if (rows + looks > 0x7fffffffll) return cudaErrorInvalidValue;
    p.rows_ctas = (int)rows;
    auto kern = lora_rows_kernel<NT>;
    static SmemCarveout wide;
    wide.ask(reinterpret_cast<const void*>(kern));
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t cfg = config(dim3((unsigned)(rows + looks)), DOWN_THREADS, 0, s, at, false);
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = p.slices;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.numAttrs = p.slices > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int NQ>
cudaError_t launch_few(FewLora& p, int rows, cudaStream_t s) {
    auto kern = gemm_lora_few_kernel<NQ>;
    using F = Few<NQ>;
    static SmemAllowance allowed;
    const cudaError_t e = allowed.ensure(reinterpret_cast<const void*>(kern), F::SMEM);
    if (e != cudaSuccess) return e;
    p.tiles = (p.N + rows - 1) / rows;
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
    l.bytes = l.h + p.tiles * p.cap * p.parts * 2ll * LORA_TERMS * p.tile_rows * p.cw;
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

bool lora_plan(LoraArgs& p, bool dual) {
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
    return p.tiles * p.cap * p.parts * LORA_TERMS * p.tile_rows <= 0x7fffffffll && (int64_t)p.n * p.check_parts <= 0x3fffffffll;
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
    // few rows: more CTAs of 16 columns each, and room beside the product's shared memory
    const cudaError_t e = p.cw == 16 || few ? launch_rows<2>(p, s) : p.cw == 32 ? launch_rows<4>(p, s) : launch_rows<8>(p, s);
    if (e != cudaSuccess) return e;
    const int64_t h_rows = p.tiles * p.cap * p.parts * LORA_TERMS * p.tile_rows;
    if (!few) return launch_gemm_bf16_lora(d, p, h_rows, s);
    FewLora f;
    memset(&f, 0, sizeof(f));
    if (!lora_map(&f.map_w, d.B, d.b_rows, d.K, 64, 64, 0, 0) || !lora_map(&f.map_x, d.A, d.M, d.K, 64, p.tile_rows, 0, 0) ||
        !lora_map(&f.map_h, p.h, h_rows, p.cw, p.cw, 2 * p.tile_rows, 0, 0) ||
        !lora_map(&f.map_up, p.up, d.N, p.rank, p.cw, 64, p.n, p.up_stride) ||
        (dual && !lora_map(&f.map_up2, p.up2, d.N, p.rank, p.cw, 64, p.n, p.up_stride)))
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
    f.count = p.count;
    f.list = p.list;
    f.notes = p.notes;
    f.bias = static_cast<const __nv_bfloat16*>(d.bias);
    f.resid = d.resid;
    f.resid_f32 = d.resid_f32;
    f.C = static_cast<__nv_bfloat16*>(d.C);
    f.C32 = static_cast<float*>(d.C32);
    f.err = d.err_word;
    const int rows = dual ? 64 : 128;
    switch (p.tile_rows) {
        case 16: return launch_few<16>(f, rows, s);
        case 32: return launch_few<32>(f, rows, s);
        case 64: return launch_few<64>(f, rows, s);
        default: return launch_few<128>(f, rows, s);
    }
}

}  // namespace ls
