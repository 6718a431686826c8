// Entry points of the INT8 x INT8 (W8A8) products: argument checks and the choice of kernel by size.
#include "w8a8_common.cuh"
#include "w8a8_ptx.cuh"

PFN_cuTensorMapEncodeTiled_v12000 w8::tensor_map_encoder()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void* f = nullptr;
        const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f) : nullptr;
    }();
    return fn;
}

int w8a8_gemm_launch(const w8::Problem& p, cudaStream_t s);
int w8a8_small_launch(const w8::Problem& p, cudaStream_t s);

namespace {

int run(const w8::Problem& p, int32_t out_dtype, cudaStream_t s)
{
    if (p.m < 0 || p.n < 0 || p.k < 16 || p.k > Q8_MAX_K || p.k % 16) return Q4_ERR_SHAPE;
    if (out_dtype != Q4_OUT_F32 && out_dtype != Q4_OUT_BF16) return Q4_ERR_UNSUPPORTED;
    if (p.m == 0 || p.n == 0) return Q4_OK;   // an empty product reads and writes nothing
    if (!p.xq || !p.scale_a || !p.w0 || !p.scale_0 || !p.y || (p.w1 && !p.scale_1)) return Q4_ERR_NULL;
    if (!q4_aligned16(p.xq) || !q4_aligned16(p.w0) || !q4_aligned16(p.w1) || !q4_aligned16(p.y) ||
        (((uintptr_t)p.scale_a | (uintptr_t)p.scale_0 | (uintptr_t)p.scale_1 | (uintptr_t)p.bias) & 3u))
        return Q4_ERR_ALIGN;
    return p.m <= 64 ? w8a8_small_launch(p, s) : w8a8_gemm_launch(p, s);
}

}  // namespace

extern "C" int q8_linear_w8a8(const int8_t* xq, const float* scale_a, int32_t m, const int8_t* wq, const float* scale_w,
                              int32_t n, int32_t k, const float* bias, void* y, int32_t out_dtype, int32_t* dev_status,
                              void* stream)
{
    const w8::Problem p = {xq, scale_a, wq, scale_w, nullptr, nullptr, bias, y, m, n, k, out_dtype == Q4_OUT_BF16, 0, dev_status};
    return run(p, out_dtype, (cudaStream_t)stream);
}

extern "C" int q8_linear_w8a8_gated(const int8_t* xq, const float* scale_a, int32_t m, const int8_t* wq_gate,
                                    const float* scale_gate, const int8_t* wq_up, const float* scale_up, int32_t n, int32_t k,
                                    int32_t act, void* h, int32_t out_dtype, int32_t* dev_status, void* stream)
{
    if (act != Q8_ACT_SILU && act != Q8_ACT_GELU) return Q4_ERR_UNSUPPORTED;
    if (m > 0 && n > 0 && !wq_up) return Q4_ERR_NULL;
    const w8::Problem p = {xq, scale_a, wq_gate, scale_gate, wq_up, scale_up, nullptr, h, m, n, k, out_dtype == Q4_OUT_BF16, act, dev_status};
    return run(p, out_dtype, (cudaStream_t)stream);
}
