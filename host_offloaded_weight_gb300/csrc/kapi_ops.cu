// C entry points of the 4-bit and few-token operators (see ls_kernels.h).
#include <cuda_runtime.h>

#include "kernels.h"
#include "ls_kernels.h"

using namespace ls;

namespace {

ls_status status_of(cudaError_t e) {
    if (e == cudaSuccess) return LS_OK;
    if (e == cudaErrorInvalidValue) return LS_ERR_INVALID_ARG;
    return LS_ERR_CUDA;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Stream-ordered scratch of one call, from the entry points' pool.
struct Scratch {
    void* p = nullptr;
    cudaStream_t s;
    explicit Scratch(cudaStream_t stream) : s(stream) {}
    bool take(int64_t bytes) {
        cudaMemPool_t pool = entry_scratch_pool();
        if (!pool || cudaMallocFromPoolAsync(&p, (size_t)bytes, pool, s) != cudaSuccess) {
            cudaGetLastError();
            p = nullptr;
            return false;
        }
        return true;
    }
    ~Scratch() {
        if (p) cudaFreeAsync(p, s);
    }
};

constexpr int32_t MX_MAX_K = 1 << 24;

}  // namespace

extern "C" {

int64_t lsk_mxfp4_code_pitch(int32_t K) { return K > 0 ? mx_code_pitch(K) : 0; }

int64_t lsk_mxfp4_scale_pitch(int32_t K) { return K > 0 ? mx_scale_pitch(K) : 0; }

ls_status lsk_mxfp4_quantize(const void* src, int32_t src_f32, int64_t rows, int32_t K, int64_t ld, void* codes,
                             void* scales, void* stream) {
    if (rows < 0 || K < 1 || K > MX_MAX_K || ld < K) return LS_ERR_INVALID_ARG;
    if (rows == 0) return LS_OK;
    if (!src || !codes || !scales || !aligned(src, src_f32 ? 4 : 2) || !aligned(codes, 32) || !aligned(scales, 16))
        return LS_ERR_INVALID_ARG;
    return status_of(launch_mx_quantize(src, src_f32 != 0, rows, K, ld, codes, scales, (cudaStream_t)stream));
}

ls_status lsk_mxfp4_dequantize(const void* codes, const void* scales, int64_t rows, int32_t K, void* dst, int32_t dst_f32,
                               int64_t ld, void* stream) {
    if (rows < 0 || K < 1 || K > MX_MAX_K || ld < K) return LS_ERR_INVALID_ARG;
    if (rows == 0) return LS_OK;
    if (!dst || !codes || !scales || !aligned(dst, dst_f32 ? 4 : 2) || !aligned(codes, 32) || !aligned(scales, 16))
        return LS_ERR_INVALID_ARG;
    return status_of(launch_mx_dequantize(codes, scales, rows, K, dst, dst_f32 != 0, ld, (cudaStream_t)stream));
}

ls_status lsk_gemm_mxfp4(const void* a_codes, const void* a_scales, const void* b_codes, const void* b_scales, void* C,
                         int32_t c_f32, int32_t M, int32_t N, int32_t K, void* stream) {
    if (M < 0 || N < 1 || K < 1 || K > MX_MAX_K) return LS_ERR_INVALID_ARG;
    if (M == 0) return LS_OK;
    if (!a_codes || !a_scales || !b_codes || !b_scales || !C || !aligned(a_codes, 32) || !aligned(b_codes, 32) ||
        !aligned(a_scales, 16) || !aligned(b_scales, 16) || !aligned(C, c_f32 ? 4 : 2))
        return LS_ERR_INVALID_ARG;
    return status_of(launch_gemm_mx(a_codes, a_scales, b_codes, b_scales, C, c_f32 != 0, M, N, K, entry_error_word(),
                                    (cudaStream_t)stream));
}

ls_status lsk_gemm_bf16_mxfp4(const void* A, int64_t lda, const void* b_codes, const void* b_scales, void* C,
                              int32_t c_f32, int32_t M, int32_t N, int32_t K, void* stream) {
    if (M < 0 || N < 1 || K < 1 || K > MX_MAX_K || lda < K) return LS_ERR_INVALID_ARG;
    if (M == 0) return LS_OK;
    if (!A || !b_codes || !b_scales || !C || !aligned(A, 2) || !aligned(b_codes, 32) || !aligned(b_scales, 16) ||
        !aligned(C, c_f32 ? 4 : 2))
        return LS_ERR_INVALID_ARG;
    Scratch ws((cudaStream_t)stream);
    if (!ws.take(act_mx_ws_bytes(M, N, K))) return LS_ERR_OOM;
    return status_of(launch_gemm_act_mx(A, lda, b_codes, b_scales, C, c_f32 != 0, M, N, K, ws.p, entry_error_word(),
                                        (cudaStream_t)stream));
}

}  // extern "C"
