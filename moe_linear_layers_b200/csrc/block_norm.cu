// The boundary between two blocks of a layer stack in one pass (block_norm): the norm after a block, its gate,
// the residual update with its scales, the norm before the next block and, where the next product takes INT8
// activations, their codes and scales.
//
//   b  = x * rstd(x) * post_w            (b = x without post_w)       rstd(v) = (mean v^2 + eps)^(-1/2)
//   r' = res_scale * residual + gate * (branch_scale * b)
//   n  = r' * rstd(r') * pre_w
//
// HBM-bound: x and residual are read once and each output is written once; a row's values stay in registers
// between the two reductions and the quantizer's.  One CTA per row.
//
// Every elementwise step is one fp32 operation rounded to nearest, in the order written in the header, and the
// sums of squares run in fp64 (their rounding error stays below a quarter of an fp32 ulp of rstd by nine
// orders of magnitude, so rstd does not depend on the order of the sum).  That pins n, and with it the
// codes, which change by a whole step when a value crosses a rounding border.  The fp64 work is a conversion and a
// multiply-add per value and norm, a few per cent of the fp64 pipe at the memory floor.
#include "q4_common.cuh"

namespace {

struct Args {
    const void *x, *residual, *post_w, *gate, *pre_w;
    void *residual_out, *y;
    int8_t* xq;
    float* scale_a;
    int x_dt, r_dt, w_dt, g_dt, y_dt;
    int T, H, tokens_per_gate;
    float eps, res_scale, branch_scale;
    int32_t* status;
};

// V consecutive values at element i of an array of type dt (V = 8: 16-byte aligned; V = 1: any element)
template <int V> __device__ __forceinline__ void load(const void* p, int dt, int64_t i, float (&v)[V])
{
    if constexpr (V == 8) {
        if (dt == Q4_F32) {
            const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
            const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + 4);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
            const uint32_t e[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (dt == Q4_BF16) {
                    v[2 * j] = __uint_as_float(e[j] << 16);
                    v[2 * j + 1] = __uint_as_float(e[j] & 0xFFFF0000u);
                } else {
                    const float2 f = __half22float2(u32_as_h2(e[j]));
                    v[2 * j] = f.x;
                    v[2 * j + 1] = f.y;
                }
            }
        }
    } else {
        if (dt == Q4_F32) v[0] = static_cast<const float*>(p)[i];
        else if (dt == Q4_BF16) v[0] = bf16_bits_to_float(static_cast<const uint16_t*>(p)[i]);
        else v[0] = __half2float(__ushort_as_half(static_cast<const uint16_t*>(p)[i]));
    }
}

// v rounded to dt (and widened again): what a store of it holds
__device__ __forceinline__ float as_stored(float v, int dt)
{
    if (dt == Q4_BF16) return __bfloat162float(__float2bfloat16_rn(v));
    if (dt == Q4_F16) return __half2float(__float2half_rn(v));
    return v;
}

template <int V> __device__ __forceinline__ void store(void* p, int dt, int64_t i, const float (&v)[V])
{
    if constexpr (V == 8) {
        if (dt == Q4_F32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
            o[0] = make_float4(v[0], v[1], v[2], v[3]);
            o[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint32_t e[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (dt == Q4_BF16) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                    e[j] = *reinterpret_cast<const uint32_t*>(&h);
                } else {
                    e[j] = h2_as_u32(__floats2half2_rn(v[2 * j], v[2 * j + 1]));
                }
            }
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(e[0], e[1], e[2], e[3]);
        }
    } else {
        if (dt == Q4_F32) static_cast<float*>(p)[i] = v[0];
        else if (dt == Q4_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v[0]);
        else static_cast<__half*>(p)[i] = __float2half_rn(v[0]);
    }
}

constexpr int kMaxWarps = 32;

// sum over the CTA (every thread gets the same bits); `red` is free for reuse after the next barrier
__device__ __forceinline__ double block_sum(double v, double* red)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int nw = blockDim.x / 32, lane = threadIdx.x & 31;
    if (nw == 1) return v;
    if (lane == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    v = lane < nw ? red[lane] : 0.0;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red)
{
    v = __reduce_max_sync(0xffffffffu, v);
    const int nw = blockDim.x / 32, lane = threadIdx.x & 31;
    if (nw == 1) return v;
    if (lane == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, lane < nw ? red[lane] : 0u);
}

// V values a load, P loads a thread: V * P * blockDim.x >= H
template <int V, int P>
__global__ void __launch_bounds__(1024) block_norm_kernel(const Args a)
{
    __shared__ double red[2][kMaxWarps];
    __shared__ uint32_t redm[kMaxWarps];
    q4_pdl_start();
    const int64_t row = blockIdx.x, base = row * a.H;
    const int nt = blockDim.x;
    const double inv_h = 1.0 / a.H;
    float v[P][V];
#pragma unroll
    for (int i = 0; i < P; i++) {
        const int c = (i * nt + threadIdx.x) * V;
#pragma unroll
        for (int j = 0; j < V; j++) v[i][j] = 0.0f;
        if (a.x && c < a.H) load<V>(a.x, a.x_dt, base + c, v[i]);
    }
    if (a.x) {
        if (a.post_w) {
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < P; i++)
#pragma unroll
                for (int j = 0; j < V; j++) s = fma((double)v[i][j], (double)v[i][j], s);
            const float rs = (float)rsqrt(block_sum(s, red[0]) * inv_h + (double)a.eps);
#pragma unroll
            for (int i = 0; i < P; i++) {
                const int c = (i * nt + threadIdx.x) * V;
                if (c >= a.H) continue;
                float w[V];
                load<V>(a.post_w, a.w_dt, c, w);
#pragma unroll
                for (int j = 0; j < V; j++) v[i][j] = __fmul_rn(__fmul_rn(v[i][j], rs), w[j]);
            }
        }
        const int64_t grow = a.gate ? (row / a.tokens_per_gate) * a.H : 0;
#pragma unroll
        for (int i = 0; i < P; i++) {
            const int c = (i * nt + threadIdx.x) * V;
            if (c >= a.H) continue;
#pragma unroll
            for (int j = 0; j < V; j++) v[i][j] = __fmul_rn(v[i][j], a.branch_scale);
            if (a.gate) {
                float g[V];
                load<V>(a.gate, a.g_dt, grow + c, g);
#pragma unroll
                for (int j = 0; j < V; j++) v[i][j] = __fmul_rn(v[i][j], g[j]);
            }
        }
    }
    if (a.residual) {
#pragma unroll
        for (int i = 0; i < P; i++) {
            const int c = (i * nt + threadIdx.x) * V;
            if (c >= a.H) continue;
            float r[V];
            load<V>(a.residual, a.r_dt, base + c, r);
#pragma unroll
            for (int j = 0; j < V; j++) {
                r[j] = __fmul_rn(r[j], a.res_scale);
                v[i][j] = a.x ? __fadd_rn(r[j], v[i][j]) : r[j];
            }
        }
    }
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < P; i++)
#pragma unroll
        for (int j = 0; j < V; j++) s = fma((double)v[i][j], (double)v[i][j], s);
    if (a.residual_out) {
#pragma unroll
        for (int i = 0; i < P; i++) {
            const int c = (i * nt + threadIdx.x) * V;
            if (c < a.H && q4_in_bounds(base + c + V - 1, (int64_t)a.T * a.H, a.status))
                store<V>(a.residual_out, a.r_dt, base + c, v[i]);
        }
    }
    if (!a.y && !a.xq) return;
    const double ss = block_sum(s, red[1]);
    const float rs = (float)rsqrt(ss * inv_h + (double)a.eps);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < P; i++) {
        const int c = (i * nt + threadIdx.x) * V;
        if (c >= a.H) continue;
        float w[V];
        if (a.pre_w) load<V>(a.pre_w, a.w_dt, c, w);
#pragma unroll
        for (int j = 0; j < V; j++) {
            v[i][j] = __fmul_rn(v[i][j], rs);
            if (a.pre_w) v[i][j] = __fmul_rn(v[i][j], w[j]);
        }
        if (a.y && q4_in_bounds(base + c + V - 1, (int64_t)a.T * a.H, a.status)) store<V>(a.y, a.y_dt, base + c, v[i]);
        if (a.xq) {
#pragma unroll
            for (int j = 0; j < V; j++) {
                v[i][j] = as_stored(v[i][j], a.y_dt);
                top = max(top, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);   // (bit order = magnitude order, NaN on top)
            }
        }
    }
    if (!a.xq) return;
    top = block_max(top, redm);
    const float scale = __uint_as_float(top) / 127.0f;
    if (threadIdx.x == 0) {
        a.scale_a[row] = scale;
        if (top >= 0x7F800000u) q4_set_status(a.status, Q4_ERR_NONFINITE);
    }
    const bool exact_div = !(scale >= 0x1p-100f);
    const float inv = exact_div ? 0.0f : 1.0f / scale;
#pragma unroll
    for (int i = 0; i < P; i++) {
        const int c = (i * nt + threadIdx.x) * V;
        if (c >= a.H) continue;
        uint32_t o[V == 8 ? 2 : 1] = {};
#pragma unroll
        for (int j = 0; j < V; j++)
            o[j / 4] |= (scale == 0.0f ? 0u : (uint32_t)q4_code8(v[i][j], scale, inv, exact_div) & 0xFFu) << (8 * (j & 3));
        if (!q4_in_bounds(base + c + V - 1, (int64_t)a.T * a.H, a.status)) continue;
        if constexpr (V == 8) *reinterpret_cast<uint2*>(a.xq + base + c) = make_uint2(o[0], o[1]);
        else a.xq[base + c] = (int8_t)o[0];
    }
}

template <int V> int launch(const Args& a, cudaStream_t s)
{
    const int words = (a.H + V - 1) / V;
    const int p = (words + 1023) / 1024;
    const dim3 grid(a.T), block(p > 1 ? 1024 : (words + 31) / 32 * 32);
    if (p <= 1) return q4_launch_pdl(block_norm_kernel<V, 1>, grid, block, 0, s, a);
    if (p <= 2) return q4_launch_pdl(block_norm_kernel<V, 2>, grid, block, 0, s, a);
    if (p <= 4) return q4_launch_pdl(block_norm_kernel<V, 4>, grid, block, 0, s, a);
    if constexpr (V == 1) {
        if (p <= 16) return q4_launch_pdl(block_norm_kernel<V, 16>, grid, block, 0, s, a);
        return q4_launch_pdl(block_norm_kernel<V, 32>, grid, block, 0, s, a);
    }
    return Q4_ERR_SHAPE;
}

int64_t dtype_size(int dt) { return dt == Q4_F32 ? 4 : 2; }

// two arrays share memory (NULL shares none)
bool overlap(const void* a, int64_t na, const void* b, int64_t nb)
{
    const uintptr_t p = (uintptr_t)a, q = (uintptr_t)b;
    return a && b && p < q + nb && q < p + na;
}

bool known_dtype(int dt) { return dt == Q4_F32 || dt == Q4_BF16 || dt == Q4_F16; }
bool aligned_to(const void* p, int dt) { return ((uintptr_t)p & (dt == Q4_F32 ? 3u : 1u)) == 0; }

}  // namespace

extern "C" int block_norm(const q4_block_norm* d, int32_t T, int32_t H, int32_t* dev_status, void* stream)
{
    if (!d) return Q4_ERR_NULL;
    if (T < 0 || H < 1 || H > Q4_BLOCK_NORM_MAX_H) return Q4_ERR_SHAPE;
    if (!known_dtype(d->x_dtype) || !known_dtype(d->residual_dtype) || !known_dtype(d->w_dtype) ||
        !known_dtype(d->gate_dtype) || !known_dtype(d->y_dtype))
        return Q4_ERR_UNSUPPORTED;
    if (!(d->eps >= 0.0f) || isinf(d->eps)) return Q4_ERR_SHAPE;
    if (d->gate && (d->gate_rows < 1 || T % d->gate_rows)) return Q4_ERR_SHAPE;
    if (T == 0) return Q4_OK;   // no rows: the arrays hold nothing and may be NULL
    if (!d->x && !d->residual) return Q4_ERR_NULL;
    if (!d->x && (d->post_w || d->gate)) return Q4_ERR_NULL;   // a gate or a norm after a block that is not there
    if (!d->residual_out && !d->y && !d->xq) return Q4_ERR_NULL;
    if (!d->xq != !d->scale_a) return Q4_ERR_NULL;
    if (!aligned_to(d->x, d->x_dtype) || !aligned_to(d->residual, d->residual_dtype) ||
        !aligned_to(d->residual_out, d->residual_dtype) || !aligned_to(d->post_w, d->w_dtype) ||
        !aligned_to(d->pre_w, d->w_dtype) || !aligned_to(d->gate, d->gate_dtype) || !aligned_to(d->y, d->y_dtype) ||
        ((uintptr_t)d->scale_a & 3u))
        return Q4_ERR_ALIGN;
    // an output may replace the input of the same rows and element size, and overlap nothing else
    const int64_t n = (int64_t)T * H;
    const void* in[5] = {d->x, d->residual, d->post_w, d->pre_w, d->gate};
    const int64_t in_n[5] = {n * dtype_size(d->x_dtype), n * dtype_size(d->residual_dtype), H * dtype_size(d->w_dtype),
                             H * dtype_size(d->w_dtype), (int64_t)d->gate_rows * H * dtype_size(d->gate_dtype)};
    const void* out[4] = {d->residual_out, d->y, d->xq, d->scale_a};
    const int64_t out_n[4] = {n * dtype_size(d->residual_dtype), n * dtype_size(d->y_dtype), n, 4 * (int64_t)T};
    for (int o = 0; o < 4; o++) {
        for (int i = 0; i < 5; i++) {
            const bool in_place = o < 2 && i < 2 && out[o] == in[i] && out_n[o] == in_n[i];
            if (!in_place && overlap(out[o], out_n[o], in[i], in_n[i])) return Q4_ERR_UNSUPPORTED;
        }
        for (int q = 0; q < o; q++)
            if (overlap(out[o], out_n[o], out[q], out_n[q])) return Q4_ERR_UNSUPPORTED;
    }
    Args a = {};
    a.x = d->x;
    a.residual = d->residual;
    a.post_w = d->post_w;
    a.gate = d->gate;
    a.pre_w = d->pre_w;
    a.residual_out = d->residual_out;
    a.y = d->y;
    a.xq = d->xq;
    a.scale_a = d->scale_a;
    a.x_dt = d->x_dtype;
    a.r_dt = d->residual_dtype;
    a.w_dt = d->w_dtype;
    a.g_dt = d->gate_dtype;
    a.y_dt = d->y_dtype;
    a.T = T;
    a.H = H;
    a.tokens_per_gate = d->gate ? T / d->gate_rows : 1;
    a.eps = d->eps;
    a.res_scale = d->res_scale;
    a.branch_scale = d->branch_scale;
    a.status = dev_status;
    // 16-byte accesses need rows and arrays that start on 16 bytes (8 for the codes); otherwise one value at a time
    const bool vec = H % 8 == 0 && q4_aligned16(d->x) && q4_aligned16(d->residual) && q4_aligned16(d->residual_out) &&
                     q4_aligned16(d->post_w) && q4_aligned16(d->pre_w) && q4_aligned16(d->gate) && q4_aligned16(d->y) &&
                     ((uintptr_t)d->xq & 7u) == 0;
    return vec ? launch<8>(a, (cudaStream_t)stream) : launch<1>(a, (cudaStream_t)stream);
}
