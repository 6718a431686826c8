// Entry points of the INT8 x INT8 (W8A8) products: argument checks and the choice of kernel by size.
#include <atomic>

#include "w8a8_common.cuh"
#include "w8a8_ptx.cuh"

PFN_cuTensorMapEncodeTiled_v12000 w8::tensor_map_encoder()
{
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> kept{nullptr};   // (a failed look-up is tried again)
    PFN_cuTensorMapEncodeTiled_v12000 fn = kept.load(std::memory_order_relaxed);
    if (!fn) {
        cudaDriverEntryPointQueryResult q;
        void* f = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess && q == cudaDriverEntryPointSuccess) {
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
            kept.store(fn, std::memory_order_relaxed);
        }
    }
    return fn;
}

int w8a8_gemm_launch(const w8::Problem& p, cudaStream_t s);
int w8a8_split_launch(const w8::Problem& p, int bn, int splits, cudaStream_t s);
int w8a8_small_launch(const w8::Problem& p, cudaStream_t s);

namespace {

// Which kernel: the streaming one for few tokens, else the faster of the split and the pair kernel by their times.
//
// Streaming: its tokens come in groups of 16 that each read the weights again.  It is the faster one up to 8 tokens, and
// beyond while the groups read about 24 MB in all (us, streaming / split: 2048 x 2048, 64 tokens 4.7 / 5.5; 8192 x 2048, 17 tokens
// 6.7 / 6.9, 32 tokens 7.9 / 6.8; gated 8192 x 2048, 16 tokens 12.0 / 9.5).
//
// The other two by what was measured on B200 (16 and 64 blocks of K, 8 to 1024 tokens), in us:
//   split: 3.3 + bn / (36 splits) + bn / 128 for the exchange + 0.24 to 0.43 a block of K, for each wave of CTAs
//   pair:  5.3 + 0.27 a block of K a wave, and 3 more from the second wave on
// (2048 x 8192, 65 tokens: split 9.2, pair 22.4; 2048 x 2048, 512 tokens: 9.2 / 9.9; 8192 x 2048, 256 tokens: 13.3 / 10.5.)
struct Choice {
    int kernel;       // Q8_KERNEL_*
    int bn, splits;   // the split kernel's
};

Choice choose(const w8::Problem& p, bool gated)
{
    const int64_t groups = (p.m + 15) / 16;
    if (p.m <= 8 || (p.m <= 64 && groups * p.n * p.k * (gated ? 2 : 1) <= (24 << 20))) return {Q8_KERNEL_STREAM, 0, 0};
    const int kb = (p.k + 127) / 128, sms = q4_num_sms();
    auto ceil_div = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const int64_t pair_waves = ceil_div(ceil_div(p.m, 256) * ceil_div(p.n, gated ? 128 : 256), sms / 2);
    double best = 5.3 + 0.27 * kb * pair_waves + 3.0 * (pair_waves - 1);
    Choice c = {Q8_KERNEL_PAIR, 0, 0};
    const int64_t tiles_n = ceil_div(p.n, gated ? 64 : 128);
    for (int i = 0; i < 4; i++) {
        const int bn = 32 << i;
        const double block[4] = {0.24, 0.26, 0.36, 0.43};
        if (i > 0 && bn / 2 >= p.m) break;   // (a narrower tile holds every token)
        for (int splits = 1; splits <= 4 && splits <= kb; splits *= 2) {
            const int64_t waves = ceil_div(tiles_n * ceil_div(p.m, bn) * splits, sms);
            const double t = 1.5 + waves * (1.8 + bn / (36.0 * splits) + (splits > 1 ? bn / 128.0 : 0.0) + block[i] * ceil_div(kb, splits));
            if (t < best) {
                best = t;
                c = {Q8_KERNEL_SPLIT, bn, splits};
            }
        }
    }
    return c;
}

bool sizes_ok(int m, int n, int k)
{
    return m >= 0 && n >= 0 && m <= Q8_MAX_ROWS && n <= Q8_MAX_ROWS && k >= 16 && k <= Q8_MAX_K && k % 16 == 0;
}

int run(const w8::Problem& p, int32_t out_dtype, cudaStream_t s)
{
    if (!sizes_ok(p.m, p.n, p.k)) return Q4_ERR_SHAPE;
    if (out_dtype != Q4_OUT_F32 && out_dtype != Q4_OUT_BF16) return Q4_ERR_UNSUPPORTED;
    if (p.m == 0 || p.n == 0) return Q4_OK;   // an empty product reads and writes nothing
    if (!p.xq || !p.scale_a || !p.w0 || !p.scale_0 || !p.y || (p.w1 && !p.scale_1)) return Q4_ERR_NULL;
    if (!q4_aligned16(p.xq) || !q4_aligned16(p.w0) || !q4_aligned16(p.w1) || !q4_aligned16(p.y) ||
        (((uintptr_t)p.scale_a | (uintptr_t)p.scale_0 | (uintptr_t)p.scale_1 | (uintptr_t)p.bias) & 3u))
        return Q4_ERR_ALIGN;
    const int64_t m = p.m, n = p.n, ny = m * n * (p.out_bf16 ? 2 : 4);
    if (q4_overlap(p.y, ny, p.xq, m * p.k) || q4_overlap(p.y, ny, p.w0, n * p.k) || q4_overlap(p.y, ny, p.w1, n * p.k) ||
        q4_overlap(p.y, ny, p.scale_a, 4 * m) || q4_overlap(p.y, ny, p.scale_0, 4 * n) || q4_overlap(p.y, ny, p.scale_1, 4 * n) ||
        q4_overlap(p.y, ny, p.bias, 4 * n))
        return Q4_ERR_UNSUPPORTED;   // tiles are written while others' inputs are still read
    const Choice c = choose(p, p.w1 != nullptr);
    return c.kernel == Q8_KERNEL_STREAM  ? w8a8_small_launch(p, s)
           : c.kernel == Q8_KERNEL_SPLIT ? w8a8_split_launch(p, c.bn, c.splits, s)
                                         : w8a8_gemm_launch(p, s);
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

extern "C" int q8_linear_w8a8_kernel(int32_t m, int32_t n, int32_t k, int32_t gated)
{
    if (!sizes_ok(m, n, k) || m == 0 || n == 0) return Q4_ERR_SHAPE;
    w8::Problem p = {};
    p.m = m;
    p.n = n;
    p.k = k;
    return choose(p, gated != 0).kernel;
}
