// Device helpers of the 4-bit and few-token kernels: mbarriers with bounded waits, TMA loads,
// tensor memory, block-scaled tcgen05 products and the conversions of the MXFP4 format.
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace ls {
namespace tc {

constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;  // bound of every mbarrier wait, far above any legitimate one

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// ------------------------------------------------------------------ mbarriers
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_init_fence() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Whether a phase is complete, without waiting (a try may be suspended for a while).
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// The slow half of a wait: polls until the phase completes or the limit passes; then records
// the role that gave up and returns false.
static __device__ __noinline__ bool bar_wait_long(uint32_t bar, uint32_t parity, uint32_t* err, uint32_t role) {
    const uint64_t t0 = globaltimer_ns();
    while (!bar_try(bar, parity)) {
        if (globaltimer_ns() - t0 > WAIT_LIMIT_NS) {
            raise_error(err, DERR_GEMM_TIMEOUT | (role << 8));
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, uint32_t* err, uint32_t role) {
    return bar_try(bar, parity) || bar_wait_long(bar, parity, err, role);
}

// The same for a whole warp, with one outcome.
__device__ __forceinline__ bool bar_wait_warp(uint32_t bar, uint32_t parity, uint32_t* err, uint32_t role) {
    if (__all_sync(0xffffffffu, bar_try(bar, parity))) return true;
    return __all_sync(0xffffffffu, bar_wait_long(bar, parity, err, role));
}
// True in one lane of a converged warp. Tensor copies and products issued under it, in control flow that
// the whole warp shares, take their operands from uniform registers: four products and six scale copies
// are issued in 384 clocks (their time on the tensor core), against 559 from a branch on the lane.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0); }

// ------------------------------------------------------------------ launch order
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void fence_smem_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ------------------------------------------------------------------ clusters
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address, in the cluster's window, of CTA `rank`'s shared memory at this CTA's address `a`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t a, uint32_t rank) {
    uint32_t out;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(out) : "r"(a), "r"(rank));
    return out;
}
__device__ __forceinline__ void st_cluster(uint32_t a, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// An arrival at a barrier of another CTA of the cluster, after this CTA's writes to its shared memory. The order is
// asked for shared memory alone: a release of everything waits for the SM's global stores, a microsecond each time.
__device__ __forceinline__ void bar_arrive_cluster(uint32_t bar) {
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A wait of a whole warp that also orders what other CTAs of the cluster wrote to shared memory before they arrived.
__device__ __forceinline__ bool bar_wait_cluster(uint32_t bar, uint32_t parity, uint32_t* err, uint32_t role) {
    if (!bar_wait_warp(bar, parity, err, role)) return false;
    asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
    return true;
}

// ------------------------------------------------------------------ TMA
__device__ __forceinline__ void tma_desc_prefetch(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// A box out of shared memory, clipped to the tensor; x and y at least 0. Issued, committed and waited for by one lane.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }  // memory free again
__device__ __forceinline__ void tma_store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// ------------------------------------------------------------------ tensor memory
__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_get(uint32_t slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t t, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(cols) : "memory");
}
__device__ __forceinline__ void tmem_load8(uint32_t t, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(t));
}
__device__ __forceinline__ void tmem_load32(uint32_t t, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t));
}
__device__ __forceinline__ void tmem_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ------------------------------------------------------------------ block-scaled products
// Shared-memory operand of a product: K along the rows, 128-byte rows with the 128-byte
// swizzle, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// 512 bytes of scales: 32 rows of 16 bytes, no swizzle, groups of 8 rows 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)1 << 16) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}
// Scales into 4 TMEM columns, replicated for the four lane quarters: row r of a 128-row
// operand lies in lane r % 32, column r / 32, its four consecutive blocks in the word's bytes.
__device__ __forceinline__ void scale_copy(uint32_t tmem, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
// 8- and 4-bit operands, a value a byte; a scale for every 32 values; K = 32 an instruction.
__device__ __forceinline__ void mma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// Instruction descriptor: fp32 sums, E8M0 scales, operands along K; the scales' first byte
// within the TMEM words goes to bits 29 (A) and 4 (B).
__host__ __device__ constexpr uint32_t mx_idesc(uint32_t a_type, uint32_t b_type, int M, int N) {
    return (a_type << 7) | (b_type << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t idesc_at(uint32_t idesc, uint32_t byte) {
    return idesc | (byte << 29) | (byte << 4);
}

// ------------------------------------------------------------------ the same for a pair of CTAs (cta_group::2)
// Products of 256 rows, 128 of each CTA; each CTA holds half of the right operand's rows, its own left scales and
// all of the right operand's scales. One CTA issues for both.
// A copy into this CTA's memory that counts at a barrier of either CTA of the pair (`bar`: in the cluster's window).
__device__ __forceinline__ void tma_2d_pair(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tmem_get_pair(uint32_t slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t t, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(cols) : "memory");
}
// From the same address of each CTA's memory to the same columns of its TMEM.
__device__ __forceinline__ void scale_copy_pair(uint32_t tmem, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
// Both operands E2M1, packed; a scale for every 32 values of K; K = 64 an instruction.
__device__ __forceinline__ void mma_mxf4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}
// An arrival at the barrier at this address in both CTAs when the products so far are complete.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
    const uint16_t mask = 3;
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"(mask)
                 : "memory");
}

// ------------------------------------------------------------------ formats
// The four byte pairs of a word of eight E2M1 codes as f16 pairs (exact), in order of k.
__device__ __forceinline__ void e2m1_to_half(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// Eight fp32 values rounded to E2M1 (nearest, ties to even, saturating), low nibble first.
__device__ __forceinline__ uint32_t e2m1_pack(const float (&v)[8]) {
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return w;
}
// 2^(byte - 127): 0 is the subnormal 2^-127, 255 is NaN.
__device__ __forceinline__ float e8m0_to_float(uint32_t byte) {
    return byte == 0 ? __uint_as_float(0x00400000u) : byte == 255 ? __uint_as_float(0x7fc00000u)
                                                                  : __uint_as_float(byte << 23);
}

// ------------------------------------------------------------------ bf16 rows as two E4M3 terms
// Eight values of a bf16 row from k on, zeros past K.
__device__ __forceinline__ uint4 row8(const __nv_bfloat16* row, int k, int K, int vec) {
    if (vec && k + 8 <= K) return __ldg(reinterpret_cast<const uint4*>(row + k));
    uint32_t w[4] = {0, 0, 0, 0};
    const uint16_t* s = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (k + j < K) w[j >> 1] |= (uint32_t)s[k + j] << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The first term of a block whose largest magnitude has exponent field 254 is cut to its four bits: rounded up, it could
// be 2^128, whose products with weights of 1 and more are infinite. It leaves up to twice as much, so the next terms'
// scales are a bit larger.
constexpr uint32_t TOP_FIELD = 254;
__device__ __forceinline__ float first_term(float v, uint32_t field) {
    return __uint_as_float(__float_as_uint(v) & (field == TOP_FIELD ? 0xfff00000u : 0xffffffffu));
}
// The scale byte of term i: the field - 127 - 7 - 5 i as a byte, not below 0; a block with a NaN or an infinity reads as NaN.
__device__ __forceinline__ uint32_t term_byte(uint32_t field, int i) {
    const uint32_t low = 7 + 5 * i - (i > 0 && field == TOP_FIELD ? 1 : 0);
    return field == 255 ? 255 : field < low ? 0 : field - low;
}
__device__ __forceinline__ float pow2(uint32_t e) { return __uint_as_float((127 + e) << 23); }

// The two E4M3 terms of eight values and the scale bytes of their block (a 2^-s1 to the nearest, then the rest 2^-s2,
// exact in units of 2^s1: an unscaled first term could overflow). Four
// neighbouring lanes hold a block; every lane of the warp takes part.
__device__ __forceinline__ void split8(uint4 raw, uint2& o1, uint2& o2, uint32_t& b1, uint32_t& b2) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = __vmaxu2(m, w[j] & 0x7fff7fffu);
    m = max(m & 0xffffu, m >> 16);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t e = m >> 7;
    b1 = term_byte(e, 0);
    b2 = term_byte(e, 1);
    const float f1 = __uint_as_float((254 - min(b1, 253u)) << 23), f2 = pow2(b1 - b2);
    uint16_t t1[4], t2[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float x = __uint_as_float(w[j] << 16) * f1, y = __uint_as_float(w[j] & 0xffff0000u) * f1;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(t1[j]) : "f"(first_term(y, e)), "f"(first_term(x, e)));
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(t1[j]));
        const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&h));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(t2[j]) : "f"((y - d.y) * f2), "f"((x - d.x) * f2));
    }
    o1 = make_uint2(t1[0] | (uint32_t)t1[1] << 16, t1[2] | (uint32_t)t1[3] << 16);
    o2 = make_uint2(t2[0] | (uint32_t)t2[1] << 16, t2[2] | (uint32_t)t2[3] << 16);
    if (e == 255) o1 = o2 = make_uint2(0, 0);
}

// ------------------------------------------------------------------ shared memory
__device__ __forceinline__ void st_shared1(uint32_t a, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ void st_shared2(uint32_t at, uint32_t a, uint32_t b) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void st_shared4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

}  // namespace tc
}  // namespace ls
