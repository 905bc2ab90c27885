// A whole mixture-of-experts layer for a few tokens, in two kernels:
//
//   up     h[i] = SiLU(G_e x_t) * (U_e x_t)   for every routed pair i = (t, e)
//   down   out[t] = x[t] + sum_j w[t,j] D_e h[i],  w = softmax over the token's k largest logits
//
// Experts in bf16 or MXFP4. Bound by the bytes of the experts that are routed: each is read once
// (per 16 of its tokens), and nothing else of that size is touched. Tokens are the 8-wide side
// of mma.sync (m16n8k16): with one to a few tokens an expert the 128-row tiles of tcgen05
// would be padding, and the tensor work is far from being the bound.
//
// Routing is done by every CTA of both kernels for itself (a warp a token): it costs less
// than a launch, and lets the down kernel request its first weights while the up kernel runs.
//
// up: a unit is 32 columns f of one expert (32 gate and 32 up rows) for up to 16 of its
// tokens. Four warps split K in boxes of 128 bytes a row; each keeps its own ring of TMA stages
// and refills a stage itself, so the main loop has no barrier between warps. In a 16-row
// product rows 0-7 are gate rows and rows 8-15 the up rows of the same f. The four sums are joined in
// shared memory in a fixed order.
// down: a CTA has 16 output rows for all experts; the (expert, box) pairs are split
// over its warps in order, sums go to a private [token][row] array and are added in warp
// order: the same bits every time, and no atomics on data.
//
// MXFP4 products: E2M1 codes become f16 exactly (one conversion instruction for two), the other
// side is f16 times a power of two: x scaled by its row's largest value, h by the largest of
// its block of 32 (11 bits; what is under 2^-22 of that largest vanishes). A block's product is multiplied by
// the block's scales in fp32.
#include <algorithm>

#include "kernels.h"
#include "tc.cuh"

namespace ls {
namespace {

using namespace tc;

constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr int MAX_T = 64, MAX_K = 8, MAX_E = 256;
constexpr int MAX_ROWS = MAX_T * MAX_K;
constexpr int CHUNK = 16;         // tokens of an expert that one pass over its weights serves
constexpr int UP_F = 32;          // columns of h in a unit of the up kernel
constexpr int UP_STAGE = 2 * UP_F * 128;
constexpr int UP_DEPTH = 2;
constexpr int DOWN_ROWS = 16;     // output rows of a CTA of the down kernel
constexpr int DOWN_STAGE = DOWN_ROWS * 128;
constexpr int DOWN_DEPTH = 6;

struct FewParams {
    CUtensorMap map_a, map_b;  // up: gate, up; down: down (map_a)
    const uint8_t* scale_a;    // MXFP4: block scales of the same matrices
    const uint8_t* scale_b;
    int64_t scale_stride;      // bytes between experts
    int scale_pitch;
    const __nv_bfloat16* x;    // [T, H]
    const float* resid;        // [T, H], or NULL: x
    const float* logits;       // [T, E]
    void* h;                   // [T k][h_pitch] bf16, or f16 with block scales
    float* h_scale;            // [T k][hs_pitch]
    int h_pitch, hs_pitch;
    int T, E, k, H, F;
    __nv_bfloat16* out;
    float* out32;
    uint32_t* err;
};

// ------------------------------------------------------------------ routing
struct Routing {
    uint32_t mask[MAX_E][2];      // the tokens of an expert
    int first[MAX_E];             // its first row (rows are sorted by expert, then token)
    uint8_t sel[MAX_ROWS];
    float sel_w[MAX_ROWS];
    uint8_t row_t[MAX_ROWS];      // token and weight of a row
    float row_w[MAX_ROWS];
    int n_chunks;
    uint8_t chunk_e[MAX_ROWS];    // expert, first row and rows of each chunk
    uint8_t chunk_n[MAX_ROWS];
    int16_t chunk_row[MAX_ROWS];
};

// Order of floats as unsigned numbers; -0 as 0, NaN as -infinity. Never 0.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v == v ? v + 0.f : -INFINITY);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Every thread of the CTA; r is complete when it returns. Per token the k largest logits (ties to the lower
// expert), weights exp(l - l_max) / sum in fp32; all zero when every logit is -infinity.
__device__ void route(Routing& r, const FewParams& p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < p.E; e += THREADS) r.mask[e][0] = r.mask[e][1] = 0;
    __syncthreads();
    for (int t = warp; t < p.T; t += WARPS) {
        uint32_t key[MAX_E / 32];
#pragma unroll
        for (int i = 0; i < MAX_E / 32; ++i) {
            const int e = lane + 32 * i;
            key[i] = e < p.E ? order_key(p.logits[(int64_t)t * p.E + e]) : 0u;
        }
        int mine = 0;  // lane j: the j-th expert
        for (int j = 0; j < p.k; ++j) {
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < MAX_E / 32; ++i) best = max(best, key[i]);
            best = __reduce_max_sync(0xffffffffu, best);
            uint32_t at = 0xffffffffu;
#pragma unroll
            for (int i = MAX_E / 32 - 1; i >= 0; --i)
                if (key[i] == best) at = lane + 32 * i;
            at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
            for (int i = 0; i < MAX_E / 32; ++i)
                if (at == (uint32_t)(lane + 32 * i)) key[i] = 0;
            if (lane == j) mine = (int)at;
        }
        const float l = lane < p.k ? p.logits[(int64_t)t * p.E + mine] : -INFINITY;
        const float top = __shfl_sync(0xffffffffu, l, 0);
        const float ex = top == -INFINITY ? 0.f : expf(l - top);
        float sum = 0.f;
        for (int j = 0; j < p.k; ++j) sum += __shfl_sync(0xffffffffu, ex, j);
        if (lane < p.k) {
            r.sel[t * p.k + lane] = (uint8_t)mine;
            r.sel_w[t * p.k + lane] = top == -INFINITY ? 0.f : ex / sum;
            atomicOr(&r.mask[mine][t >> 5], 1u << (t & 31));
        }
    }
    __syncthreads();
    if (warp == 0) {  // rows and chunks of the experts, in order
        int rows = 0, chunks = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < p.E ? __popc(r.mask[e][0]) + __popc(r.mask[e][1]) : 0;
            const int c = (n + CHUNK - 1) / CHUNK;
            int sn = n, sc = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(0xffffffffu, sn, o), b = __shfl_up_sync(0xffffffffu, sc, o);
                if (lane >= o) {
                    sn += a;
                    sc += b;
                }
            }
            if (e < p.E) r.first[e] = rows + sn - n;
            for (int i = 0; i < c; ++i) {
                const int at = chunks + sc - c + i;
                r.chunk_e[at] = (uint8_t)e;
                r.chunk_n[at] = (uint8_t)min(CHUNK, n - CHUNK * i);
                r.chunk_row[at] = (int16_t)(rows + sn - n + CHUNK * i);
            }
            rows += __shfl_sync(0xffffffffu, sn, 31);
            chunks += __shfl_sync(0xffffffffu, sc, 31);
        }
        if (lane == 0) r.n_chunks = chunks;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * p.k; i += THREADS) {
        const int t = i / p.k, e = r.sel[i];
        const uint32_t below = (1u << (t & 31)) - 1u;
        const int rank = t < 32 ? __popc(r.mask[e][0] & below) : __popc(r.mask[e][0]) + __popc(r.mask[e][1] & below);
        r.row_t[r.first[e] + rank] = (uint8_t)t;
        r.row_w[r.first[e] + rank] = r.sel_w[i];
    }
    __syncthreads();
}

// ------------------------------------------------------------------ products
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&q)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
// Two neighbouring scales (bytes 2 i and 2 i + 1 of v) as floats.
__device__ __forceinline__ float2 scale_pair(uint2 v, int i) {
    const uint32_t w = i < 2 ? v.x : v.y;
    const uint16_t b = (uint16_t)(i & 1 ? w >> 16 : w);
    uint32_t d;
    asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(d) : "h"(b));
    return make_float2(__uint_as_float(d << 16), __uint_as_float(d & 0xffff0000u));
}
// Row of a group of 8 that lane group g takes in 16-byte reads of bf16 weights: with the
// 128-byte swizzle, neighbouring lane groups then read different halves of their rows.
__device__ __forceinline__ int mix_row(int g) { return (g >> 1) | ((g & 1) << 2); }

// Eight bf16 times 2^e as f16 pairs.
__device__ __forceinline__ uint4 bf16_to_half(uint4 v, float f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
        o[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// A power of two that brings values up to |v| (fp32 bits, finite) to [256, 512), and its inverse.
__device__ __forceinline__ void half_scale(uint32_t bits, float& f, float& inv) {
    int e = (int)(bits >> 23) - 127 - 8;      // v 2^-e in [256, 512)
    e = max(-126, min(e, 126));
    f = __uint_as_float((uint32_t)(127 - e) << 23);
    inv = __uint_as_float((uint32_t)(127 + e) << 23);
}

// A warp's own ring of TMA stages. Only this warp fills and empties it.
template <int DEPTH, int STAGE>
struct Ring {
    uint32_t base, bars;
    int issued, taken;
    bool bad;
    // after a timeout: let the copies in flight land (again with a limit) before the CTA goes
    __device__ __forceinline__ void drain(uint32_t* err) const {
        if (!bad) return;
        for (int i = max(0, issued - DEPTH); i < issued; ++i) bar_wait(bar(i), (uint32_t)(i / DEPTH) & 1u, err, 9);
    }
    __device__ __forceinline__ uint32_t stage(int i) const { return base + (uint32_t)(i % DEPTH) * STAGE; }
    __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8u * (i % DEPTH); }
    // the next stage's data, as an address; on a timeout the error word is set and no later wait is made
    __device__ __forceinline__ uint32_t take(uint32_t* err) {
        if (!bad) bad = !__all_sync(0xffffffffu, bar_wait(bar(taken), (uint32_t)(taken / DEPTH) & 1u, err, 8));
        return stage(taken);
    }
};

// ------------------------------------------------------------------ up
struct UpSmem {
    uint64_t bars[WARPS][UP_DEPTH];
    float red[WARPS / 4][4][32][32];   // [group][warp][accumulator][lane]
    uint32_t x_max[MAX_T];             // largest |x| of a token, as bits
    Routing r;
};

// One unit's products over this warp's boxes.
template <bool MX, int NT, class Refill>
__device__ __forceinline__ void up_products(float (&acc)[4][2][4], const FewParams& p, UpSmem& sm, Ring<UP_DEPTH, UP_STAGE>& ring,
                                            Refill refill, int chunk, int f0, int n_box) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, wg = (threadIdx.x >> 5) & 3;
    const int e = sm.r.chunk_e[chunk], n = sm.r.chunk_n[chunk], row0 = sm.r.chunk_row[chunk];
    constexpr int BLOCKS = MX ? 8 : 2;   // blocks of 32 values in a box
    constexpr int SUB = MX ? 4 : 2;      // of which x is loaded at a time
    const __nv_bfloat16* xr[NT];
    float xf[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int tok = 8 * i + g;
        xr[i] = nullptr;
        xf[i] = 0.f;
        if (tok < n) {
            const int t = sm.r.row_t[row0 + tok];
            xr[i] = p.x + (int64_t)t * p.H + 8 * c;
            float inv;
            half_scale(sm.x_max[t], xf[i], inv);
        }
    }
    uint4 raw[NT][SUB];
    auto load_x = [&](int box, int sub) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int b = 0; b < SUB; ++b) {
                const int k = (box * BLOCKS + sub * SUB + b) * 32;
                raw[i][b] = xr[i] && k + 8 * c < p.H ? __ldg(reinterpret_cast<const uint4*>(xr[i] + k)) : make_uint4(0, 0, 0, 0);
            }
    };
    const uint8_t* sg = nullptr;
    const uint8_t* su = nullptr;
    uint2 scale[8];
    auto load_scales = [&](int box) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const bool in = f0 + 8 * m + g < p.F && 8 * box < p.scale_pitch;
            const int64_t at = (int64_t)(f0 + 8 * m + g) * p.scale_pitch + 8 * box;
            scale[2 * m] = in ? __ldg(reinterpret_cast<const uint2*>(sg + at)) : make_uint2(0, 0);
            scale[2 * m + 1] = in ? __ldg(reinterpret_cast<const uint2*>(su + at)) : make_uint2(0, 0);
        }
    };
    if (wg >= n_box) return;
    if (MX) {
        sg = p.scale_a + (int64_t)e * p.scale_stride;
        su = p.scale_b + (int64_t)e * p.scale_stride;
        load_scales(wg);
    }
    load_x(wg, 0);
    for (int box = wg; box < n_box; box += 4) {
        const uint32_t st = ring.take(p.err);
#pragma unroll
        for (int sub = 0; sub < BLOCKS / SUB; ++sub) {
            uint4 xb[NT][SUB];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int b = 0; b < SUB; ++b) xb[i][b] = MX ? bf16_to_half(raw[i][b], xf[i]) : raw[i][b];
            if (sub + 1 < BLOCKS / SUB) load_x(box, sub + 1);
            else if (box + 4 < n_box) load_x(box + 4, 0);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if (MX) {
#pragma unroll
                    for (int bp = 0; bp < SUB / 2; ++bp) {
                        // matrices: gate and up rows of block b, then of block b + 1
                        const int b0 = sub * SUB + 2 * bp;
                        const int mi = lane >> 3, r = lane & 7;
                        uint32_t q[4];
                        ldmatrix4(st + (mi & 1) * (UP_F * 128) + (8 * m + r) * 128 + (((b0 + (mi >> 1)) ^ r) << 4), q);
                        const float2 fg = scale_pair(scale[2 * m], b0 / 2), fu = scale_pair(scale[2 * m + 1], b0 / 2);
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            uint32_t a[4], u[4];
                            e2m1_to_half(q[2 * b], a);
                            e2m1_to_half(q[2 * b + 1], u);
                            const float s0 = b ? fg.y : fg.x, s1 = b ? fu.y : fu.x;
#pragma unroll
                            for (int i = 0; i < NT; ++i) {
                                float d[4] = {0.f, 0.f, 0.f, 0.f};
                                const uint4 x = xb[i][2 * bp + b];
                                mma_f16(d, a[0], u[0], a[1], u[1], x.x, x.y);
                                mma_f16(d, a[2], u[2], a[3], u[3], x.z, x.w);
                                acc[m][i][0] = fmaf(s0, d[0], acc[m][i][0]);
                                acc[m][i][1] = fmaf(s0, d[1], acc[m][i][1]);
                                acc[m][i][2] = fmaf(s1, d[2], acc[m][i][2]);
                                acc[m][i][3] = fmaf(s1, d[3], acc[m][i][3]);
                            }
                        }
                    }
                } else {
                    const int r = mix_row(g);
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const uint32_t at = st + (8 * m + r) * 128 + (((4 * b + c) ^ r) << 4);
                        const uint4 a = lds128(at), u = lds128(at + UP_F * 128);
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            const uint4 x = xb[i][b];
                            mma_bf16(acc[m][i], a.x, u.x, a.y, u.y, x.x, x.y);
                            mma_bf16(acc[m][i], a.z, u.z, a.w, u.w, x.z, x.w);
                        }
                    }
                }
            }
        }
        if (MX && box + 4 < n_box) load_scales(box + 4);
        __syncwarp();
        ring.taken++;
        refill();
    }
}

template <bool MX>
__global__ void __launch_bounds__(THREADS, 1) moe_few_up_kernel(const __grid_constant__ FewParams p) {
    extern __shared__ uint8_t raw_smem[];
    const uint32_t base = (smem_addr(raw_smem) + 1023u) & ~1023u;
    UpSmem& sm = *reinterpret_cast<UpSmem*>(raw_smem + (base - smem_addr(raw_smem)) + WARPS * UP_DEPTH * UP_STAGE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp & 3, group = warp >> 2;
    if (threadIdx.x == 0) {
        for (int w = 0; w < WARPS; ++w)
            for (int s = 0; s < UP_DEPTH; ++s) bar_init(smem_addr(&sm.bars[w][s]), 1);
        bar_init_fence();
        tma_desc_prefetch(&p.map_a);
        tma_desc_prefetch(&p.map_b);
    }
    grid_wait();
    grid_release();  // the down kernel may be placed: everything before this kernel is complete
    route(sm.r, p);

    const int n_f = (p.h_pitch + UP_F - 1) / UP_F;                 // h_pitch is a multiple of 32
    const int row_bytes = MX ? (int)((p.H + 127) / 128 * 64) : 2 * p.H;
    const int n_box = (row_bytes + 127) / 128;
    const int units = sm.r.n_chunks * n_f, step = gridDim.x * (WARPS / 4);
    const int u0 = blockIdx.x + gridDim.x * group;

    Ring<UP_DEPTH, UP_STAGE> ring;
    ring.base = base + warp * UP_DEPTH * UP_STAGE;
    ring.bars = smem_addr(&sm.bars[warp][0]);
    ring.issued = ring.taken = 0;
    ring.bad = false;
    int pu = u0, pb = wg;   // the next box to request
    auto refill = [&]() {
        if (pu >= units || wg >= n_box || ring.bad) return;
        if (lane == 0) {
            const int e = sm.r.chunk_e[pu / n_f], f0 = pu % n_f * UP_F;
            const uint32_t st = ring.stage(ring.issued), bar = ring.bar(ring.issued);
            bar_expect(bar, UP_STAGE);
            tma_3d(st, &p.map_a, bar, pb * 128, f0, e);
            tma_3d(st + UP_F * 128, &p.map_b, bar, pb * 128, f0, e);
        }
        ring.issued++;
        pb += 4;
        if (pb >= n_box) {
            pb = wg;
            pu += step;
        }
    };
    for (int i = 0; i < UP_DEPTH; ++i) refill();

    if (MX) {  // the largest |x| of each token (infinities and NaN aside: they stay what they are in f16)
        for (int t = warp; t < p.T; t += WARPS) {
            uint32_t m = 0;
            for (int k = 8 * lane; k < p.H; k += 256) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)t * p.H + k));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t lo = (w[i] << 16) & 0x7fffffffu, hi = w[i] & 0x7fff0000u;
                    if (lo < 0x7f800000u) m = max(m, lo);
                    if (hi < 0x7f800000u) m = max(m, hi);
                }
            }
            m = __reduce_max_sync(0xffffffffu, m);
            if (lane == 0) sm.x_max[t] = m;
        }
        __syncthreads();
    }

    for (int u = u0; u < units; u += step) {
        const int chunk = u / n_f, f0 = u % n_f * UP_F;
        const int n = sm.r.chunk_n[chunk], row0 = sm.r.chunk_row[chunk];
        float acc[4][2][4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[m][i][j] = 0.f;
        if (n <= 8) up_products<MX, 1>(acc, p, sm, ring, refill, chunk, f0, n_box);
        else up_products<MX, 2>(acc, p, sm, ring, refill, chunk, f0, n_box);
        // join the four warps' sums
        const int tiles = n <= 8 ? 1 : 2;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (i < tiles)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sm.red[group][wg][(m * 2 + i) * 4 + j][lane] = acc[m][i][j];
        asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
        const int tid = threadIdx.x & 127;
        for (int i = 0; i < tiles; ++i) {  // 16 threads a token, 2 columns each
            const int tok = 8 * i + (tid >> 4), f = (tid & 15) * 2;
            float h[2];
            const int t = tok < n ? sm.r.row_t[row0 + tok] : 0;
            float xf = 1.f, xi = 1.f;
            if (MX) half_scale(sm.x_max[t], xf, xi);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int fr = (f + j) & 7, m = (f + j) >> 3;
                const int gg = MX ? fr : ((fr & 3) << 1) | (fr >> 2);  // the lane group of this row
                const int ln = gg * 4 + ((tok & 7) >> 1), a = (m * 2 + i) * 4 + (tok & 1);
                float gs = 0.f, us = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    gs += sm.red[group][w][a][ln];
                    us += sm.red[group][w][a + 2][ln];
                }
                gs *= xi;
                us *= xi;
                h[j] = gs / (1.f + __expf(-gs)) * us;
            }
            if (MX) {
                // block of 32 columns: f16 times a power of two from its largest value
                uint32_t m = max(__float_as_uint(h[0]) & 0x7fffffffu, __float_as_uint(h[1]) & 0x7fffffffu);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                float hf, hi;
                half_scale(m, hf, hi);
                const bool bad = m >= 0x7f800000u;
                if (tok < n) {
                    const __half2 v = __floats2half2_rn(bad ? 0.f : h[0] * hf, bad ? 0.f : h[1] * hf);
                    *reinterpret_cast<__half2*>(static_cast<__half*>(p.h) + (int64_t)(row0 + tok) * p.h_pitch + f0 + f) = v;
                    if ((tid & 15) == 0) {
                        float* to = p.h_scale + (int64_t)(row0 + tok) * p.hs_pitch + f0 / 32;
                        to[0] = bad ? __uint_as_float(0x7fc00000u) : hi;
                        if (f0 + UP_F == p.h_pitch)  // the row's padding is read with it
                            for (int j = 1; j < p.hs_pitch - f0 / 32; ++j) to[j] = 0.f;
                    }
                }
            } else if (tok < n) {
                *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.h) + (int64_t)(row0 + tok) * p.h_pitch + f0 + f) =
                    __floats2bfloat162_rn(h[0], h[1]);
            }
        }
        asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
    }
    ring.drain(p.err);
}

// ------------------------------------------------------------------ down
struct DownSmem {
    uint64_t bars[WARPS][DOWN_DEPTH];
    Routing r;
};

template <bool MX, int NT, class Refill>
__device__ __forceinline__ void down_products(float (&acc)[2][4], const FewParams& p, const Routing& r,
                                              Ring<DOWN_DEPTH, DOWN_STAGE>& ring, Refill refill, int chunk, int box0, int box1,
                                              int r0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int e = r.chunk_e[chunk], n = r.chunk_n[chunk], row0 = r.chunk_row[chunk];
    constexpr int BLOCKS = MX ? 8 : 2, SUB = MX ? 4 : 2;
    const uint16_t* hr[NT];
    const float* hs0[NT];
    const float* hs1[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int tok = 8 * i + g, t0 = 8 * i + 2 * c;
        hr[i] = tok < n ? static_cast<const uint16_t*>(p.h) + (int64_t)(row0 + tok) * p.h_pitch + 8 * c : nullptr;
        hs0[i] = MX && t0 < n ? p.h_scale + (int64_t)(row0 + t0) * p.hs_pitch : nullptr;
        hs1[i] = MX && t0 + 1 < n ? p.h_scale + (int64_t)(row0 + t0 + 1) * p.hs_pitch : nullptr;
    }
    uint4 raw[NT][SUB];
    float4 s0[NT], s1[NT];
    auto load_h = [&](int box, int sub) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int b0 = box * BLOCKS + sub * SUB;
#pragma unroll
            for (int b = 0; b < SUB; ++b)
                raw[i][b] = hr[i] && (b0 + b) * 32 < p.h_pitch ? __ldcg(reinterpret_cast<const uint4*>(hr[i] + (b0 + b) * 32))
                                                               : make_uint4(0, 0, 0, 0);
            if (MX) {
                s0[i] = hs0[i] && b0 < p.hs_pitch ? __ldcg(reinterpret_cast<const float4*>(hs0[i] + b0)) : make_float4(0, 0, 0, 0);
                s1[i] = hs1[i] && b0 < p.hs_pitch ? __ldcg(reinterpret_cast<const float4*>(hs1[i] + b0)) : make_float4(0, 0, 0, 0);
            }
        }
    };
    const uint8_t* sc = MX ? p.scale_a + (int64_t)e * p.scale_stride : nullptr;
    uint2 sa = make_uint2(0, 0), sb = make_uint2(0, 0);
    auto load_scales = [&](int box) {
        if (!MX || 8 * box >= p.scale_pitch) {
            sa = sb = make_uint2(0, 0);
            return;
        }
        sa = r0 + g < p.H ? __ldg(reinterpret_cast<const uint2*>(sc + (int64_t)(r0 + g) * p.scale_pitch + 8 * box)) : make_uint2(0, 0);
        sb = r0 + g + 8 < p.H ? __ldg(reinterpret_cast<const uint2*>(sc + (int64_t)(r0 + g + 8) * p.scale_pitch + 8 * box))
                              : make_uint2(0, 0);
    };
    load_scales(box0);
    load_h(box0, 0);
    for (int box = box0; box < box1; ++box) {
        const uint32_t st = ring.take(p.err);
#pragma unroll
        for (int sub = 0; sub < BLOCKS / SUB; ++sub) {
            uint4 hb[NT][SUB];
            float4 u0[NT], u1[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                u0[i] = s0[i];
                u1[i] = s1[i];
#pragma unroll
                for (int b = 0; b < SUB; ++b) hb[i][b] = raw[i][b];
            }
            if (sub + 1 < BLOCKS / SUB) load_h(box, sub + 1);
            else if (box + 1 < box1) load_h(box + 1, 0);
            if (MX) {
#pragma unroll
                for (int bp = 0; bp < SUB / 2; ++bp) {
                    const int b0 = sub * SUB + 2 * bp;
                    const int mi = lane >> 3, rr = lane & 7;
                    uint32_t q[4];
                    ldmatrix4(st + ((mi & 1) * 8 + rr) * 128 + (((b0 + (mi >> 1)) ^ rr) << 4), q);
                    const float2 fa = scale_pair(sa, b0 / 2), fb = scale_pair(sb, b0 / 2);
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        uint32_t a[4], u[4];
                        e2m1_to_half(q[2 * b], a);
                        e2m1_to_half(q[2 * b + 1], u);
                        const float w0 = b ? fa.y : fa.x, w1 = b ? fb.y : fb.x;
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            float d[4] = {0.f, 0.f, 0.f, 0.f};
                            const uint4 x = hb[i][2 * bp + b];
                            mma_f16(d, a[0], u[0], a[1], u[1], x.x, x.y);
                            mma_f16(d, a[2], u[2], a[3], u[3], x.z, x.w);
                            const float h0 = bp ? (b ? u0[i].w : u0[i].z) : (b ? u0[i].y : u0[i].x);
                            const float h1 = bp ? (b ? u1[i].w : u1[i].z) : (b ? u1[i].y : u1[i].x);
                            acc[i][0] = fmaf(w0 * h0, d[0], acc[i][0]);
                            acc[i][1] = fmaf(w0 * h1, d[1], acc[i][1]);
                            acc[i][2] = fmaf(w1 * h0, d[2], acc[i][2]);
                            acc[i][3] = fmaf(w1 * h1, d[3], acc[i][3]);
                        }
                    }
                }
            } else {
                const int rr = mix_row(g);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const uint32_t at = st + rr * 128 + (((4 * b + c) ^ rr) << 4);
                    const uint4 a = lds128(at), u = lds128(at + 8 * 128);
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const uint4 x = hb[i][b];
                        mma_bf16(acc[i], a.x, u.x, a.y, u.y, x.x, x.y);
                        mma_bf16(acc[i], a.z, u.z, a.w, u.w, x.z, x.w);
                    }
                }
            }
        }
        if (box + 1 < box1) load_scales(box + 1);
        __syncwarp();
        ring.taken++;
        refill();
    }
}

template <bool MX>
__global__ void __launch_bounds__(THREADS, 1) moe_few_down_kernel(const __grid_constant__ FewParams p) {
    extern __shared__ uint8_t raw_smem[];
    const uint32_t base = (smem_addr(raw_smem) + 1023u) & ~1023u;
    uint8_t* gen = raw_smem + (base - smem_addr(raw_smem));
    DownSmem& sm = *reinterpret_cast<DownSmem*>(gen + WARPS * DOWN_DEPTH * DOWN_STAGE);
    float* sums = reinterpret_cast<float*>(gen + WARPS * DOWN_DEPTH * DOWN_STAGE + sizeof(DownSmem));  // [warp][T][16]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    if (threadIdx.x == 0) {
        for (int w = 0; w < WARPS; ++w)
            for (int s = 0; s < DOWN_DEPTH; ++s) bar_init(smem_addr(&sm.bars[w][s]), 1);
        bar_init_fence();
        tma_desc_prefetch(&p.map_a);
    }
    // this kernel starts once every CTA of the up kernel has seen all earlier work complete, so the
    // routing and the weights can be read; only h has to wait
    float* mine = sums + warp * p.T * DOWN_ROWS;
    for (int i = lane; i < p.T * DOWN_ROWS; i += 32) mine[i] = 0.f;
    route(sm.r, p);

    const int r0 = blockIdx.x * DOWN_ROWS;
    const int row_bytes = MX ? (int)((p.F + 127) / 128 * 64) : 2 * p.F;
    const int n_box = (row_bytes + 127) / 128;
    const int total = sm.r.n_chunks * n_box;
    const int i0 = warp * total / WARPS, i1 = (warp + 1) * total / WARPS;

    Ring<DOWN_DEPTH, DOWN_STAGE> ring;
    ring.base = base + warp * DOWN_DEPTH * DOWN_STAGE;
    ring.bars = smem_addr(&sm.bars[warp][0]);
    ring.issued = ring.taken = 0;
    ring.bad = false;
    auto refill = [&]() {
        const int i = i0 + ring.issued;
        if (i >= i1 || ring.bad) return;
        if (lane == 0) {
            const uint32_t bar = ring.bar(ring.issued);
            bar_expect(bar, DOWN_STAGE);
            tma_3d(ring.stage(ring.issued), &p.map_a, bar, i % n_box * 128, r0, sm.r.chunk_e[i / n_box]);
        }
        ring.issued++;
    };
    for (int i = 0; i < DOWN_DEPTH; ++i) refill();
    grid_wait();

    for (int i = i0; i < i1;) {
        const int chunk = i / n_box, box0 = i % n_box, box1 = min(n_box, box0 + i1 - i);
        const int n = sm.r.chunk_n[chunk], row0 = sm.r.chunk_row[chunk];
        float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        if (n <= 8) down_products<MX, 1>(acc, p, sm.r, ring, refill, chunk, box0, box1, r0);
        else down_products<MX, 2>(acc, p, sm.r, ring, refill, chunk, box0, box1, r0);
        const int ra = MX ? g : mix_row(g);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int tok = 8 * j + 2 * c + q;
                if (tok < n) {
                    const float w = sm.r.row_w[row0 + tok];
                    float* to = mine + sm.r.row_t[row0 + tok] * DOWN_ROWS + ra;
                    to[0] = fmaf(w, acc[j][q], to[0]);
                    to[8] = fmaf(w, acc[j][2 + q], to[8]);
                }
            }
        __syncwarp();
        i += box1 - box0;
    }
    ring.drain(p.err);
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * DOWN_ROWS; i += THREADS) {
        const int t = i / DOWN_ROWS, row = r0 + i % DOWN_ROWS;
        if (row >= p.H) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += sums[w * p.T * DOWN_ROWS + i];
        const int64_t at = (int64_t)t * p.H + row;
        v += p.resid ? p.resid[at] : __bfloat162float(p.x[at]);
        p.out[at] = __float2bfloat16_rn(v);
        if (p.out32) p.out32[at] = v;
    }
}

// ------------------------------------------------------------------ host side
// View [experts][rows][pitch] of bytes, boxes of 128 bytes x box_rows, 128-byte swizzle.
bool map_experts(CUtensorMap* m, const void* ptr, int64_t pitch, int64_t rows, int64_t experts, int64_t stride, int box_rows) {
    const MxEncodeFn fn = mx_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)pitch, (cuuint64_t)rows, (cuuint64_t)experts};
    cuuint64_t strides[2] = {(cuuint64_t)pitch, (cuuint64_t)stride};
    cuuint32_t box[3] = {128, (cuuint32_t)box_rows, 1};
    cuuint32_t one[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int UP_SMEM = 1024 + WARPS * UP_DEPTH * UP_STAGE + (int)sizeof(UpSmem);
constexpr int down_smem(int T) {
    return 1024 + WARPS * DOWN_DEPTH * DOWN_STAGE + (int)sizeof(DownSmem) + (int)sizeof(float) * WARPS * DOWN_ROWS * T;
}
static_assert(UP_SMEM <= 232448 && down_smem(MAX_T) <= 232448, "shared memory");

template <bool MX>
cudaError_t allow_smem() {
    static const cudaError_t e = [] {
        const cudaError_t a = cudaFuncSetAttribute(moe_few_up_kernel<MX>, cudaFuncAttributeMaxDynamicSharedMemorySize, UP_SMEM);
        return a != cudaSuccess ? a
                                : cudaFuncSetAttribute(moe_few_down_kernel<MX>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       down_smem(MAX_T));
    }();
    return e;
}

template <class Kernel>
cudaError_t launch(Kernel kern, const FewParams& p, int grid, size_t smem, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

int few_h_pitch(int F) { return (F + 31) / 32 * 32; }
int few_hs_pitch(int F) { return (F + 255) / 256 * 8; }

}  // namespace

int64_t moe_few_ws_bytes(int T, int k, int F) {
    return (int64_t)T * k * (2ll * few_h_pitch(F) + 4ll * few_hs_pitch(F)) + 512;
}

cudaError_t launch_moe_few(const MoeFewDesc& d, void* ws, uint32_t* err, cudaStream_t s) {
    if (d.T <= 0) return cudaSuccess;
    if (d.T > MAX_T || d.E < 1 || d.E > MAX_E || d.k < 1 || d.k > MAX_K || d.k > d.E) return cudaErrorInvalidValue;
    FewParams p;
    memset(&p, 0, sizeof(p));
    const int64_t up_pitch = d.mx ? mx_code_pitch(d.H) : 2ll * d.H, down_pitch = d.mx ? mx_code_pitch(d.F) : 2ll * d.F;
    FewParams q;
    if (!map_experts(&p.map_a, d.gate, up_pitch, d.F, d.E, d.gate_stride, UP_F) ||
        !map_experts(&p.map_b, d.up, up_pitch, d.F, d.E, d.gate_stride, UP_F))
        return cudaErrorInvalidValue;
    p.scale_a = static_cast<const uint8_t*>(d.gate_scales);
    p.scale_b = static_cast<const uint8_t*>(d.up_scales);
    p.scale_stride = d.gate_scale_stride;
    p.scale_pitch = (int)mx_scale_pitch(d.H);
    p.x = static_cast<const __nv_bfloat16*>(d.x);
    p.resid = d.resid;
    p.logits = d.logits;
    p.h = ws;
    p.h_pitch = few_h_pitch(d.F);
    p.hs_pitch = few_hs_pitch(d.F);
    p.h_scale = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + ((int64_t)d.T * d.k * p.h_pitch * 2 + 255) / 256 * 256);
    p.T = d.T;
    p.E = d.E;
    p.k = d.k;
    p.H = d.H;
    p.F = d.F;
    p.out = static_cast<__nv_bfloat16*>(d.out);
    p.out32 = d.out32;
    p.err = err;
    q = p;
    if (!map_experts(&q.map_a, d.down, down_pitch, d.H, d.E, d.down_stride, DOWN_ROWS)) return cudaErrorInvalidValue;
    q.scale_a = static_cast<const uint8_t*>(d.down_scales);
    q.scale_stride = d.down_scale_stride;
    q.scale_pitch = (int)mx_scale_pitch(d.F);
    cudaError_t e = d.mx ? allow_smem<true>() : allow_smem<false>();
    if (e != cudaSuccess) return e;
    const int grid_up = gemm_num_sms(), grid_down = (d.H + DOWN_ROWS - 1) / DOWN_ROWS;
    e = d.mx ? launch(moe_few_up_kernel<true>, p, grid_up, UP_SMEM, s)
             : launch(moe_few_up_kernel<false>, p, grid_up, UP_SMEM, s);
    if (e != cudaSuccess) return e;
    return d.mx ? launch(moe_few_down_kernel<true>, q, grid_down, down_smem(d.T), s)
                : launch(moe_few_down_kernel<false>, q, grid_down, down_smem(d.T), s);
}

}  // namespace ls
