// MXFP4 conversion: blocks of 32 values along a row, E2M1 elements and one E8M0 scale a block
// (OCP Microscaling Formats 1.0, section 5.3 and the conversion of section 6.3):
//
//   s = floor(log2 max|v|) - 2 (2 = the largest E2M1 exponent), clamped to -127 and above
//   element = round_nearest_even(v 2^-s), saturating at 6;   value read back = element 2^s
//
// floor(log2) is the exponent field, so the scale byte is that field minus 2, and v 2^-s is exact
// (a power of two; what underflows in bf16 is below half of the smallest element). A block with a
// NaN or an infinity gets the scale byte 255, which reads back as NaN: it cannot pass unseen as a
// large finite block.
//
// Bound by memory: 2 or 4 bytes a value one way, 17/32 the other. A thread takes half a block, 16
// values: 32 bytes of bf16 in one access, 8 bytes of codes; two neighbouring lanes join their
// maxima by one shuffle, and the index arithmetic (no division: a block of threads is columns x
// rows) and the scale are paid once for 16 values.
// 13824 x 5120 bf16: 27.9 us there and 29.0 us back (6.4 and 6.2 TB/s; 8 values a thread and an index division
// took 89 for both); fp32 47 and 48 us (6.8 and 6.6 TB/s). fp32 back in 16-byte accesses: 69 us.
#include "kernels.h"
#include "tc.cuh"

namespace ls {
namespace {

// 32 bytes of a row; vec: 2 with 32-byte alignment, 1 with 16.
__device__ __forceinline__ void load32(const void* p, int vec, uint32_t (&w)[8]) {
    if (vec == 2) {
        asm volatile("ld.global.cs.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    } else {
        const uint4 a = __ldcs(static_cast<const uint4*>(p)), b = __ldcs(static_cast<const uint4*>(p) + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
}
__device__ __forceinline__ void store32(void* p, int vec, const uint32_t (&w)[8]) {
    if (vec == 2) {
        asm volatile("st.global.cs.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(p)
                     : "memory");
    } else {
        __stcs(static_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
        __stcs(static_cast<uint4*>(p) + 1, make_uint4(w[4], w[5], w[6], w[7]));
    }
}

// Half a block as it lies in memory, zeros past the row's end.
template <bool F32>
struct Half {
    uint32_t w[F32 ? 16 : 8];
};
template <bool F32>
__device__ __forceinline__ void load_half(Half<F32>& h, const void* src, int64_t at, int64_t left, int vec) {
    if (vec && left >= 16) {
        const uint8_t* p = static_cast<const uint8_t*>(src) + at * (F32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) load32(p + 32 * i, vec, *reinterpret_cast<uint32_t(*)[8]>(h.w + 8 * i));
    } else if (F32) {
#pragma unroll
        for (int j = 0; j < 16; ++j) h.w[F32 ? j : 0] = j < left ? static_cast<const uint32_t*>(src)[at + j] : 0u;
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(src) + at;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            h.w[j] = (2 * j < left ? p[2 * j] : 0u) | (uint32_t)(2 * j + 1 < left ? p[2 * j + 1] : 0u) << 16;
    }
}

// The exponent field of the largest of a thread's magnitudes, or 255 with a NaN or an infinity.
__device__ __forceinline__ uint32_t top_exponent(const Half<true>& h) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) m = max(m, h.w[j] & 0x7fffffffu);
    return m >> 23;
}
__device__ __forceinline__ uint32_t top_exponent(const Half<false>& h) {
    __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&h.w[0]));
#pragma unroll
    for (int j = 1; j < 8; ++j) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&h.w[j])));
    const uint32_t b = *reinterpret_cast<const uint32_t*>(&m);
    return max((b & 0x7fffu) >> 7, (b & 0x7fffffffu) >> 23);
}

template <bool F32, int U>
__global__ void __launch_bounds__(512)
mx_quantize_kernel(const void* __restrict__ src, int64_t rows, int64_t K, int64_t ld, int vec, int64_t per_row,
                   uint2* __restrict__ codes, uint8_t* __restrict__ scales, int64_t scale_pitch) {
    tc::grid_wait();
    tc::grid_release();
    const int64_t first = (int64_t)blockIdx.x * (blockDim.y * U) + threadIdx.y;
    for (int64_t g0 = (int64_t)blockIdx.y * blockDim.x; g0 < per_row; g0 += (int64_t)gridDim.y * blockDim.x) {
        const int64_t g = g0 + threadIdx.x;  // per_row is even: a block's two lanes are in or out together
        Half<F32> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {  // all loads before the first use
            const int64_t row = first + u * blockDim.y;
            load_half<F32>(v[u], src, row * ld + 16 * g, row < rows && g < per_row ? K - 16 * g : 0, vec);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = first + u * blockDim.y;
            uint32_t e = top_exponent(v[u]);
            e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
            if (row >= rows || g >= per_row) continue;
            const uint32_t byte = e == 255 ? 255 : e < 2 ? 0 : e - 2, inv = 254 - min(byte, 253u);  // 2^-s
            float x[2][8];
            if (F32) {
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j >> 3][j & 7] = __uint_as_float(v[u].w[F32 ? j : 0]) * __uint_as_float(inv << 23);
            } else {
                const uint32_t f = inv << 23 | inv << 7;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const __nv_bfloat162 t = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v[u].w[j]),
                                                     *reinterpret_cast<const __nv_bfloat162*>(&f));
                    const uint32_t b = *reinterpret_cast<const uint32_t*>(&t);
                    x[j >> 2][2 * (j & 3)] = __uint_as_float(b << 16);
                    x[j >> 2][2 * (j & 3) + 1] = __uint_as_float(b & 0xffff0000u);
                }
            }
            codes[row * per_row + g] = byte == 255 ? make_uint2(0, 0) : make_uint2(tc::e2m1_pack(x[0]), tc::e2m1_pack(x[1]));
            if ((g & 1) == 0) {
                uint8_t* s = scales + row * scale_pitch;
                s[g >> 1] = (uint8_t)byte;
                if (g + 2 == per_row)  // the row's padding
                    for (int64_t j = per_row >> 1; j < scale_pitch; ++j) s[j] = 0;
            }
        }
    }
}

template <bool F32, int U>
__global__ void __launch_bounds__(512)
mx_dequantize_kernel(const uint2* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t scale_pitch,
                     int64_t rows, int64_t K, int64_t per_row, void* __restrict__ dst, int64_t ld, int vec) {
    tc::grid_wait();
    tc::grid_release();
    const int64_t first = (int64_t)blockIdx.x * (blockDim.y * U) + threadIdx.y;
    for (int64_t g0 = (int64_t)blockIdx.y * blockDim.x; g0 < per_row; g0 += (int64_t)gridDim.y * blockDim.x) {
        const int64_t g = g0 + threadIdx.x, k = 16 * g;
        uint2 code[U];
        uint32_t byte[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = first + u * blockDim.y;
            if (row >= rows || k >= K) continue;
            code[u] = __ldcs(codes + row * per_row + g);
            byte[u] = __ldg(scales + row * scale_pitch + (g >> 1));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = first + u * blockDim.y;
            if (row >= rows || k >= K) continue;
            const float s = tc::e8m0_to_float(byte[u]);
            float v[16];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t h[4];
                tc::e2m1_to_half(i ? code[u].y : code[u].x, h);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
                    v[8 * i + 2 * j] = f.x * s;
                    v[8 * i + 2 * j + 1] = f.y * s;
                }
            }
            const int64_t at = row * ld + k;
            uint32_t w[8];
            if (F32) {
                float* p = static_cast<float*>(dst) + at;
                if (vec && k + 16 <= K) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[8 * i + j]);
                        store32(p + 8 * i, vec, w);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (k + j < K) p[j] = v[j];
                }
            } else {  // exact: two significant bits, and bf16 has fp32's exponents (subnormals too)
                __nv_bfloat16* p = static_cast<__nv_bfloat16*>(dst) + at;
                if (vec && k + 16 <= K) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                        w[j] = *reinterpret_cast<const uint32_t*>(&t);
                    }
                    store32(p, vec, w);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (k + j < K) p[j] = __float2bfloat16_rn(v[j]);
                }
            }
        }
    }
}

// Widest access of half a block: 32 bytes (2) or 16 (1) where the base and every row start there, else none.
int vec_of(const void* p, int64_t ld, bool f32) {
    const uint64_t at = reinterpret_cast<uintptr_t>(p) | (uint64_t)(ld * (f32 ? 4 : 2));
    return at % 32 == 0 ? 2 : at % 16 == 0 ? 1 : 0;
}

// A block of threads is bx half blocks of a row x by rows, launched behind the kernel before it
// (programmatic stream serialization). `per` rows a thread where that still fills the device. 13824 x 5120 bf16, rows a
// thread and us: there 1 30.0, 2 27.9, 4 28.8; back in 32-byte accesses 1 31.6, 2 30.3, 4 29.0, in 16-byte ones 2 33.3, 4
// 36.1; fp32 the same with 2 and 4 back, 47.1 and 49.4 there.
template <class Kernel, class... Args>
cudaError_t launch_halves(Kernel one, Kernel several, int per, int64_t rows, int64_t per_row, cudaStream_t s, Args... args) {
    int64_t segments = (per_row + 255) / 256, bx = per_row, by = 1;
    if (per_row >= 128) bx = ((per_row + segments - 1) / segments + 31) / 32 * 32;  // whole warps
    else by = 256 / per_row >= 4 ? 256 / per_row / 4 * 4 : 4;  // per_row is a multiple of 8
    if (segments > 65535) segments = 65535;
    const bool many = rows * per_row >= 2ll * 2048 * 4 * gemm_num_sms();
    const int64_t blocks = (rows + by * (many ? per : 1) - 1) / (by * (many ? per : 1));
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)segments);
    cfg.blockDim = dim3((unsigned)bx, (unsigned)by);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, many ? several : one, args...);
}

}  // namespace

cudaError_t launch_mx_quantize(const void* src, bool f32, int64_t rows, int K, int64_t ld, void* codes, void* scales,
                               cudaStream_t s) {
    if (rows <= 0) return cudaSuccess;
    const int64_t per_row = mx_code_pitch(K) / 8, sp = mx_scale_pitch(K);
    const int vec = vec_of(src, ld, f32);
    uint2* c = static_cast<uint2*>(codes);
    uint8_t* sc = static_cast<uint8_t*>(scales);
    return f32 ? launch_halves(mx_quantize_kernel<true, 1>, mx_quantize_kernel<true, 2>, 2, rows, per_row, s, src, rows,
                               (int64_t)K, ld, vec, per_row, c, sc, sp)
               : launch_halves(mx_quantize_kernel<false, 1>, mx_quantize_kernel<false, 2>, 2, rows, per_row, s, src, rows,
                               (int64_t)K, ld, vec, per_row, c, sc, sp);
}

cudaError_t launch_mx_dequantize(const void* codes, const void* scales, int64_t rows, int K, void* dst, bool f32,
                                 int64_t ld, cudaStream_t s) {
    if (rows <= 0) return cudaSuccess;
    const int64_t per_row = mx_code_pitch(K) / 8, sp = mx_scale_pitch(K);
    const int vec = vec_of(dst, ld, f32);
    const uint2* c = static_cast<const uint2*>(codes);
    const uint8_t* sc = static_cast<const uint8_t*>(scales);
    const bool four = !f32 && vec == 2;
    return f32 ? launch_halves(mx_dequantize_kernel<true, 1>, mx_dequantize_kernel<true, 2>, 2, rows, per_row, s, c, sc, sp,
                               rows, (int64_t)K, per_row, dst, ld, vec)
               : launch_halves(mx_dequantize_kernel<false, 1>, four ? mx_dequantize_kernel<false, 4> : mx_dequantize_kernel<false, 2>,
                               four ? 4 : 2, rows, per_row, s, c, sc, sp, rows, (int64_t)K, per_row, dst, ld, vec);
}

}  // namespace ls
