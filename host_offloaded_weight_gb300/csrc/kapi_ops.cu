// C entry points of the 4-bit, few-token and per-row operators (see ls_kernels.h).
#include <cuda_runtime.h>

#include <string.h>

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
// Rows are counted in 32 bits, whole tiles of them (256 rows of A and 224 of B; 128 rows of A twice).
constexpr int32_t MX_MAX_M = 0x7fffffff - 255, MX_MAX_N = 0x7fffffff - 223, ACT_MAX_M = (1 << 30) - 128;
constexpr int32_t LORA_MAX_M = 0x7fffffff - 255;  // tiles of 256 rows and columns

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
    if (M > MX_MAX_M || N > MX_MAX_N) return LS_ERR_UNSUPPORTED;
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
    if (M > ACT_MAX_M) return LS_ERR_UNSUPPORTED;
    if (M == 0) return LS_OK;
    if (!A || !b_codes || !b_scales || !C || !aligned(A, 2) || !aligned(b_codes, 32) || !aligned(b_scales, 16) ||
        !aligned(C, c_f32 ? 4 : 2))
        return LS_ERR_INVALID_ARG;
    Scratch ws((cudaStream_t)stream);
    const int64_t need = act_mx_ws_bytes(M, K);
    if (need > 0 && !ws.take(need)) return LS_ERR_OOM;
    return status_of(launch_gemm_act_mx(A, lda, b_codes, b_scales, C, c_f32 != 0, M, N, K, ws.p, entry_error_word(),
                                        (cudaStream_t)stream));
}

ls_status lsk_moe_few(const void* x, const float* resid, const float* logits, const lsk_moe_experts* w, int32_t T,
                      int32_t E, int32_t k, int32_t H, int32_t F, void* out, float* out32, void* stream) {
    if (!w || T < 0 || E < 1 || k < 1 || k > E || H < 8 || F < 8 || (H % 8) || (F % 8) || H > MX_MAX_K || F > MX_MAX_K)
        return LS_ERR_INVALID_ARG;
    if (T > 64 || E > 256 || k > 8) return LS_ERR_UNSUPPORTED;
    if (T == 0) return LS_OK;
    const bool mx = w->mxfp4 != 0;
    const int al = mx ? 32 : 16;
    if (!x || !logits || !out || !w->gate || !w->up || !w->down || !aligned(x, 16) || !aligned(resid, 4) ||
        !aligned(logits, 4) || !aligned(out, 2) || !aligned(out32, 4) || !aligned(w->gate, al) || !aligned(w->up, al) ||
        !aligned(w->down, al))
        return LS_ERR_INVALID_ARG;
    const int64_t up_bytes = (int64_t)F * (mx ? mx_code_pitch(H) : 2ll * H);
    const int64_t down_bytes = (int64_t)H * (mx ? mx_code_pitch(F) : 2ll * F);
    // a stride may be anything with one expert; the tensor copies want multiples of 16 bytes (of 32 where they unpack
    // 4-bit codes) below 2^40
    const int64_t gs = E == 1 ? up_bytes : w->gate_stride, ds = E == 1 ? down_bytes : w->down_stride;
    if (gs < up_bytes || ds < down_bytes || (gs % al) || (ds % al) || gs >= (1ll << 40) || ds >= (1ll << 40))
        return LS_ERR_INVALID_ARG;
    MoeFewDesc d;
    if (mx) {
        const int64_t ub = F * mx_scale_pitch(H), db = H * mx_scale_pitch(F);
        d.gate_scale_stride = E == 1 ? ub : w->gate_scale_stride;
        d.down_scale_stride = E == 1 ? db : w->down_scale_stride;
        if (!w->gate_scales || !w->up_scales || !w->down_scales || !aligned(w->gate_scales, 16) ||
            !aligned(w->up_scales, 16) || !aligned(w->down_scales, 16) || d.gate_scale_stride < ub ||
            d.down_scale_stride < db || (d.gate_scale_stride % 16) || (d.down_scale_stride % 16))
            return LS_ERR_INVALID_ARG;
    }
    d.x = x;
    d.resid = resid;
    d.logits = logits;
    d.mx = mx;
    d.gate = w->gate;
    d.up = w->up;
    d.down = w->down;
    d.gate_stride = gs;
    d.down_stride = ds;
    d.gate_scales = w->gate_scales;
    d.up_scales = w->up_scales;
    d.down_scales = w->down_scales;
    d.T = T;
    d.E = E;
    d.k = k;
    d.H = H;
    d.F = F;
    d.out = out;
    d.out32 = out32;
    Scratch ws((cudaStream_t)stream);
    if (!ws.take(moe_few_ws_bytes(mx, T, k, H, F))) return LS_ERR_OOM;
    return status_of(launch_moe_few(d, ws.p, entry_error_word(), (cudaStream_t)stream));
}

ls_status lsk_gemm_lora_bf16(int32_t epilogue, const void* A, const void* B, int64_t b_rows, int32_t b2_row_off,
                             const lsk_lora* l, const int32_t* ids, const void* bias, const void* resid, int32_t resid_f32,
                             void* C, void* C32, int32_t M, int32_t N, int32_t K, void* stream) {
    const bool dual = epilogue == LSK_EPI_SWIGLU, has_bias = epilogue == LSK_EPI_BIAS_GELU || epilogue == LSK_EPI_BIAS_RESID;
    const bool has_resid = epilogue == LSK_EPI_BIAS_RESID || epilogue == LSK_EPI_RESID;
    if (epilogue < LSK_EPI_STORE || epilogue > LSK_EPI_RESID || !l || M < 0 || N < 8 || K < 8 || (N % 8) || (K % 8) || K > MX_MAX_K)
        return LS_ERR_INVALID_ARG;
    if (b2_row_off < 0 || b_rows < (dual ? (int64_t)b2_row_off + N : N) || l->n < 1 || l->rank < 8 || (l->rank % 8)) return LS_ERR_INVALID_ARG;
    if (M > LORA_MAX_M || N > LORA_MAX_M || l->rank > LORA_MAX_RANK || b_rows > 0x7fffffffll) return LS_ERR_UNSUPPORTED;
    if (M == 0) return LS_OK;
    const int64_t down_bytes = 2ll * l->rank * K * (dual ? 2 : 1), up_bytes = 2ll * N * l->rank;
    const int64_t ds = l->n == 1 ? down_bytes : l->down_stride, us = l->n == 1 ? up_bytes : l->up_stride;
    if (!A || !B || !ids || !C || !l->down || !l->up || (dual && !l->up2) || (has_bias && !bias) || (has_resid && !resid) || (C32 && !has_resid))
        return LS_ERR_INVALID_ARG;
    if (!aligned(A, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(ids, 4) || !aligned(l->down, 16) || !aligned(l->up, 16) ||
        (dual && !aligned(l->up2, 16)) || !aligned(l->scale, 4) || (has_bias && !aligned(bias, 16)) || (has_resid && !aligned(resid, 16)) ||
        !aligned(C32, 16))
        return LS_ERR_INVALID_ARG;
    if (ds < down_bytes || us < up_bytes || (ds % 16) || (us % 16) || ds >= (1ll << 40) || us >= (1ll << 40)) return LS_ERR_INVALID_ARG;
    LoraArgs p;
    memset(&p, 0, sizeof(p));
    p.x = static_cast<const __nv_bfloat16*>(A);
    p.ids = ids;
    p.down = l->down;
    p.up = l->up;
    p.up2 = dual ? l->up2 : nullptr;
    p.scale = l->scale;
    p.down_stride = ds;
    p.up_stride = us;
    p.T = M;
    p.N = N;
    p.K = K;
    p.n = l->n;
    p.rank = l->rank;
    p.err = entry_error_word();
    if (!lora_plan(p, dual, C32 != nullptr)) return LS_ERR_UNSUPPORTED;
    GemmDesc d;
    d.epi = epilogue;
    d.A = A; d.lda = K; d.a_rows = M;
    d.B = B; d.ldb = K; d.b_rows = b_rows;
    d.b2_row_off = b2_row_off;
    d.bias = has_bias ? bias : nullptr;
    d.resid = has_resid ? resid : nullptr; d.ldr = N;
    d.resid_f32 = resid_f32 != 0;
    d.C = C; d.ldc = N;
    d.C32 = C32;
    d.M = M; d.N = N; d.K = K;
    d.err_word = entry_error_word();
    Scratch ws((cudaStream_t)stream);
    if (!ws.take(lora_ws_bytes(p))) return LS_ERR_OOM;
    return status_of(launch_gemm_lora(d, p, ws.p, (cudaStream_t)stream));
}

ls_status lsk_gemm_grouped_bf16_mxfp4(int32_t epilogue, const void* A, int64_t a_rows, const void* b_codes, const void* b_scales,
                                      const void* b2_codes, const void* b2_scales, int64_t code_stride, int64_t scale_stride,
                                      const int32_t* bounds, int32_t n_groups, const int32_t* row_table, const float* row_weight,
                                      int32_t gather_k, void* C, int32_t M, int32_t N, int32_t K, void* stream) {
    const bool dual = epilogue == LSK_EPI_SWIGLU, scaled = epilogue == LSK_EPI_SCALE_F32;
    if ((epilogue != LSK_EPI_STORE && !dual && !scaled) || M < 0 || N < 1 || K < 8 || (K % 8) || K > MX_MAX_K || n_groups < 1 || gather_k < 0 ||
        a_rows < 0 || (gather_k == 0 && a_rows < M))
        return LS_ERR_INVALID_ARG;
    if (n_groups > GROUPED_MX_MAX_GROUPS || M > (1 << 30) || N > MX_MAX_N) return LS_ERR_UNSUPPORTED;
    if (M == 0) return LS_OK;
    if (!A || !b_codes || !b_scales || (dual && (!b2_codes || !b2_scales)) || !bounds || !C || ((scaled || gather_k > 0) && !row_table) ||
        (scaled && !row_weight))
        return LS_ERR_INVALID_ARG;
    const int64_t code_bytes = N * mx_code_pitch(K), scale_bytes = N * mx_scale_pitch(K);
    const int64_t cs = n_groups == 1 ? code_bytes : code_stride, ss = n_groups == 1 ? scale_bytes : scale_stride;
    if (!aligned(A, 16) || !aligned(b_codes, 32) || !aligned(b_scales, 16) || (dual && (!aligned(b2_codes, 32) || !aligned(b2_scales, 16))) ||
        !aligned(bounds, 4) || !aligned(row_table, 4) || !aligned(row_weight, 4) || !aligned(C, scaled ? 4 : 2) || cs < code_bytes ||
        ss < scale_bytes || (cs % 32) || (ss % 16) || cs >= (1ll << 40) || ss >= (1ll << 40))
        return LS_ERR_INVALID_ARG;
    GroupedMxDesc d;
    d.epi = epilogue;
    d.A = A;
    d.a_rows = a_rows;
    d.b_codes = b_codes;
    d.b_scales = b_scales;
    d.b2_codes = b2_codes;
    d.b2_scales = b2_scales;
    d.code_stride = cs;
    d.scale_stride = ss;
    d.bounds = bounds;
    d.n_groups = n_groups;
    d.row_table = row_table;
    d.row_weight = row_weight;
    d.gather_k = gather_k;
    d.C = C;
    d.M = M;
    d.N = N;
    d.K = K;
    Scratch ws((cudaStream_t)stream);
    if (!ws.take(grouped_mx_ws_bytes(M, K))) return LS_ERR_OOM;
    return status_of(launch_gemm_grouped_mx(d, ws.p, entry_error_word(), (cudaStream_t)stream));
}

}  // extern "C"
