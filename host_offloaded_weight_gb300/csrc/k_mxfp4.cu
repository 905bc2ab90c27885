// MXFP4 conversion: blocks of 32 values along a row, E2M1 elements and one E8M0 scale a block
// (OCP Microscaling Formats 1.0, section 5.3 and the conversion of section 6.3):
//
//   s = floor(log2 max|v|) - 2 (2 = the largest E2M1 exponent), clamped to -127 and above
//   element = round_nearest_even(v 2^-s), saturating at 6;   value read back = element 2^s
//
// floor(log2) is the fp32 exponent field, so the scale byte is that field minus 2, and v 2^-s
// is exact (a power of two). A block with a NaN or an infinity gets the scale byte 255, which
// reads back as NaN: it cannot pass unseen as a large finite block.
//
// Bound by memory: 2 or 4 bytes a value one way, 17/32 the other. A thread takes 8 values (16
// bytes of bf16 in, 4 bytes of codes out, both contiguous across the warp); four neighbouring
// lanes hold a block and join its maximum by two shuffles.
#include "kernels.h"
#include "tc.cuh"

namespace ls {
namespace {

constexpr int THREADS = 256;

__device__ __forceinline__ void split_index(int64_t i, int64_t total, uint32_t per_row, int64_t& row, uint32_t& g) {
    if (total <= 0xffffffffll) {
        row = (uint32_t)i / per_row;
        g = (uint32_t)i % per_row;
    } else {
        row = i / per_row;
        g = (uint32_t)(i % per_row);
    }
}

template <bool F32>
__device__ __forceinline__ void load8(const void* src, int64_t at, int left, int vec, float (&v)[8]) {
    if (F32) {
        const float* p = static_cast<const float*>(src) + at;
        if (vec && left >= 8) {
            const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
            const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = j < left ? p[j] : 0.f;
        }
    } else {
        const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(src) + at;
        if (vec && left >= 8) {
            const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(w[j] << 16);
                v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = j < left ? __bfloat162float(p[j]) : 0.f;
        }
    }
}

template <bool F32, int U>
__global__ void __launch_bounds__(THREADS)
mx_quantize_kernel(const void* __restrict__ src, int64_t rows, int K, int64_t ld, int vec, uint32_t per_row,
                   uint32_t* __restrict__ codes, uint8_t* __restrict__ scales, int scale_pitch) {
    tc::grid_wait();
    tc::grid_release();
    const int64_t total = rows * per_row;  // a multiple of 16: a block's four lanes are in or out together
    const int64_t first = (int64_t)blockIdx.x * (THREADS * U) + threadIdx.x;
    float v[U][8];
    int64_t row[U];
    uint32_t g[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {  // all loads before the first use
        const int64_t i = first + u * THREADS;
        split_index(i < total ? i : 0, total, per_row, row[u], g[u]);
        load8<F32>(src, row[u] * ld + (int64_t)g[u] * 8, K - (int)g[u] * 8, vec, v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * THREADS;
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[u][j]) & 0x7fffffffu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        if (i >= total) continue;
        const uint32_t e = m >> 23;
        const uint32_t byte = e == 255 ? 255 : e < 2 ? 0 : e - 2;
        const float inv = __uint_as_float((254 - min(byte, 253u)) << 23);  // 2^-s
#pragma unroll
        for (int j = 0; j < 8; ++j) v[u][j] *= inv;
        codes[i] = byte == 255 ? 0u : tc::e2m1_pack(v[u]);
        if ((g[u] & 3) == 0) {
            uint8_t* s = scales + row[u] * scale_pitch;
            s[g[u] >> 2] = (uint8_t)byte;
            if (g[u] + 4 == per_row)  // the row's padding
                for (int j = (int)(per_row >> 2); j < scale_pitch; ++j) s[j] = 0;
        }
    }
}

template <bool F32, int U>
__global__ void __launch_bounds__(THREADS)
mx_dequantize_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, int scale_pitch,
                     int64_t rows, int K, uint32_t per_row, void* __restrict__ dst, int64_t ld, int vec) {
    tc::grid_wait();
    tc::grid_release();
    const int64_t total = rows * per_row;
    const int64_t first = (int64_t)blockIdx.x * (THREADS * U) + threadIdx.x;
    uint32_t code[U], byte[U], g[U];
    int64_t row[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * THREADS < total ? first + u * THREADS : 0;
        split_index(i, total, per_row, row[u], g[u]);
        code[u] = __ldcs(codes + i);
        byte[u] = __ldg(scales + row[u] * scale_pitch + (g[u] >> 2));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int k = (int)g[u] * 8;
        if (first + u * THREADS >= total || k >= K) continue;
        uint32_t h[4];
        tc::e2m1_to_half(code[u], h);
        const float s = tc::e8m0_to_float(byte[u]);
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
            v[2 * j] = f.x * s;
            v[2 * j + 1] = f.y * s;
        }
        if (F32) {
            float* p = static_cast<float*>(dst) + row[u] * ld + k;
            if (vec && k + 8 <= K) {
                __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
                __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (k + j < K) p[j] = v[j];
            }
        } else {  // exact: two significant bits, and bf16 has fp32's exponents (subnormals too)
            __nv_bfloat16* p = static_cast<__nv_bfloat16*>(dst) + row[u] * ld + k;
            if (vec && k + 8 <= K) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                    w[j] = *reinterpret_cast<const uint32_t*>(&t);
                }
                __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (k + j < K) p[j] = __float2bfloat16_rn(v[j]);
            }
        }
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// 16-byte accesses of 8 values: the base and every row start on 16 bytes.
int vec_ok(const void* p, int64_t ld, bool f32) { return aligned16(p) && ld % (f32 ? 4 : 8) == 0; }

// Launched behind the kernel before it (programmatic stream serialization). A thread takes
// four groups of 8 where that still fills the device, else one.
template <class Kernel, class... Args>
cudaError_t launch_groups(Kernel one, Kernel four, int64_t groups, cudaStream_t s, Args... args) {
    const bool many = groups >= 4ll * THREADS * 8 * gemm_num_sms();
    const int64_t blocks = (groups + (many ? 4 : 1) * THREADS - 1) / ((many ? 4 : 1) * THREADS);
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, many ? four : one, args...);
}

}  // namespace

cudaError_t launch_mx_quantize(const void* src, bool f32, int64_t rows, int K, int64_t ld, void* codes, void* scales,
                               cudaStream_t s) {
    if (rows <= 0) return cudaSuccess;
    const uint32_t per_row = (uint32_t)(mx_code_pitch(K) / 4);
    const int vec = vec_ok(src, ld, f32), sp = (int)mx_scale_pitch(K);
    uint32_t* c = static_cast<uint32_t*>(codes);
    uint8_t* sc = static_cast<uint8_t*>(scales);
    return f32 ? launch_groups(mx_quantize_kernel<true, 1>, mx_quantize_kernel<true, 4>, rows * per_row, s, src, rows, K,
                               ld, vec, per_row, c, sc, sp)
               : launch_groups(mx_quantize_kernel<false, 1>, mx_quantize_kernel<false, 4>, rows * per_row, s, src, rows, K,
                               ld, vec, per_row, c, sc, sp);
}

cudaError_t launch_mx_dequantize(const void* codes, const void* scales, int64_t rows, int K, void* dst, bool f32,
                                 int64_t ld, cudaStream_t s) {
    if (rows <= 0) return cudaSuccess;
    const uint32_t per_row = (uint32_t)(mx_code_pitch(K) / 4);
    const int vec = vec_ok(dst, ld, f32), sp = (int)mx_scale_pitch(K);
    const uint32_t* c = static_cast<const uint32_t*>(codes);
    const uint8_t* sc = static_cast<const uint8_t*>(scales);
    return f32 ? launch_groups(mx_dequantize_kernel<true, 1>, mx_dequantize_kernel<true, 4>, rows * per_row, s, c, sc, sp,
                               rows, K, per_row, dst, ld, vec)
               : launch_groups(mx_dequantize_kernel<false, 1>, mx_dequantize_kernel<false, 4>, rows * per_row, s, c, sc, sp,
                               rows, K, per_row, dst, ld, vec);
}

}  // namespace ls
