// The boundary between two blocks of a layer stack in one pass (block_norm): the norm after a block, its gate,
// the residual update with its scales, the norm before the next block and, where the next product takes INT8
// activations, their codes and scales.
//
//   b  = x * rstd(x) * post_w            (b = x without post_w)       rstd(v) = (mean v^2 + eps)^(-1/2)
//   r' = res_scale * residual + gate * (branch_scale * b)
//   n  = r' * rstd(r') * pre_w
//
// HBM-bound: x and residual are read once and each output is written once; a row's values stay in registers
// between the two reductions and the quantizer's.
//
// Every elementwise step is one fp32 operation rounded to nearest, in the order written in the header, and the
// sums of squares run in fp64 (their rounding error stays below a quarter of an fp32 ulp of rstd by nine
// orders of magnitude, so rstd does not depend on the order of the sum).  That pins n, and with it the
// codes, which change by a whole step when a value crosses a rounding border.  The fp64 work is a conversion and a
// multiply-add per value and norm, a few per cent of the fp64 pipe at the memory floor.
#include <type_traits>

#include "tc_ptx.cuh"

namespace {

struct Args {
    const void *x, *residual, *post_w, *gate, *pre_w;
    void *residual_out, *y;
    int8_t* xq;
    float* scale_a;
    int x_dt, r_dt, w_dt, g_dt, y_dt;
    int T, H, tokens_per_gate;   // tokens_per_gate 0: one gate for all
    float res_scale, branch_scale;
    double eps, inv_h;
    uint64_t ones;      // the fp32 pair (1, 1)
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

// the gate's row of a token (T < 2^31, and a 64-bit division would be a fifth of a short row's instructions)
__device__ __forceinline__ int64_t gate_row(const Args& a, int64_t row)
{
    return a.tokens_per_gate ? (int64_t)((uint32_t)row / (uint32_t)a.tokens_per_gate) : 0;
}

__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// sum over the CTA; every thread gets the same bits
__device__ __forceinline__ double cta_sum(double v, double* red)
{
    v = warp_sum(v);
    const int nw = blockDim.x / 32, lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    return warp_sum(lane < nw ? red[lane] : 0.0);
}

__device__ __forceinline__ uint32_t cta_max(uint32_t v, uint32_t* red)
{
    v = __reduce_max_sync(0xffffffffu, v);
    const int nw = blockDim.x / 32, lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, lane < nw ? red[lane] : 0u);
}

template <int V> __device__ __forceinline__ void add_squares(const float (&v)[V], double& s)
{
#pragma unroll
    for (int j = 0; j < V; j++) s = fma((double)v[j], (double)v[j], s);
}

__device__ __forceinline__ float rstd_of(double sum, const Args& a)
{
    const double m = fma(sum, a.inv_h, a.eps);
    if (m > 1e-30 && m < 1e30) {
        // the fp32 root (off by a relative d of 2^-22 or so) and one third-order step in fp64: off by d^3, and a
        // fraction of the fp64 root's instructions, which every warp of a row would issue
        const double r0 = (double)rsqrtf((float)m);
        const double e = fma(-(m * r0), r0, 1.0);
        return (float)fma(r0, fma(0.375, e, 0.5) * e, r0);
    }
    return (float)rsqrt(m);
}

template <int V> __device__ __forceinline__ void scale_by(float (&v)[V], float f)
{
#pragma unroll
    for (int j = 0; j < V; j++) v[j] = __fmul_rn(v[j], f);
}
template <int V> __device__ __forceinline__ void scale_by(float (&v)[V], const float (&f)[V])
{
#pragma unroll
    for (int j = 0; j < V; j++) v[j] = __fmul_rn(v[j], f[j]);
}

// amax / 127, from the bits of amax, as a product with the fp32 reciprocal.  That is what a division by the constant 127 is in
// tensor operations on a GPU, so a row quantized by them has these codes and this scale bit for bit; act_quant_per_token divides
// (IEEE), and where the two scales differ (in about 5 % of rows, by an ulp: each is off by at most 2^-23 of itself) a
// value whose quotient lies on a rounding border gets the neighbouring code.
__device__ __forceinline__ float scale_of(uint32_t top) { return __fmul_rn(__uint_as_float(top), 1.0f / 127.0f); }

// v = what y_dt holds of v; the largest magnitude's bits (their order is the magnitudes', NaN on top)
template <int V> __device__ __forceinline__ void settle(float (&v)[V], int dt, uint32_t& top)
{
#pragma unroll
    for (int j = 0; j < V; j++) {
        v[j] = as_stored(v[j], dt);
        top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    }
}

// The codes of V values.  With a scale of at least 2^-100 the rounded quotient is at most 127 in magnitude (scale is amax /
// 127 to 2^-23), so there is nothing to clamp and q + 1.5 * 2^23, rounded to nearest even like rint, holds the
// code in its low byte.
template <int V> __device__ __forceinline__ void store_codes(int8_t* p, const float (&v)[V], float scale, float inv, bool exact_div)
{
    uint32_t o[V == 8 ? 2 : 1] = {};
    if (exact_div) {
#pragma unroll
        for (int j = 0; j < V; j++)
            o[j / 4] |= (scale == 0.0f ? 0u : (uint32_t)q4_code8(v[j], scale, inv, true) & 0xFFu) << (8 * (j & 3));
    } else {
        uint32_t c[V];
#pragma unroll
        for (int j = 0; j < V; j++) {
            const float t = v[j] * inv;
            c[j] = __float_as_uint(fmaf(fmaf(-scale, t, v[j]), inv, t) + 12582912.0f);
        }
        if constexpr (V == 2) {
            o[0] = prmt(c[0], c[1], 0x0040u);
        } else if constexpr (V == 8) {
#pragma unroll
            for (int h = 0; h < 2; h++)
                o[h] = prmt(prmt(c[4 * h], c[4 * h + 1], 0x0040u), prmt(c[4 * h + 2], c[4 * h + 3], 0x0040u), 0x5410u);
        } else {
            o[0] = c[0];
        }
    }
    if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(o[0], o[1]);
    else if constexpr (V == 2) *reinterpret_cast<uint16_t*>(p) = (uint16_t)o[0];
    else *p = (int8_t)o[0];
}

// Rows of more than 16384 values (where the persistent form does not take them, see launch_many): a CTA of 1024 threads a row, V
// values a load, P loads a thread.  A thread's 32 values of x and of the residual do not fit its 64 registers: 296 bytes of spill
// stores with V = 8, 588 with V = 1, and a branch on a type stands at every access.  2048 x 32768 with every part: bf16 223 us, fp32
// 251 (3.5 TB/s); odd widths, 2048 x 32767: 1016 and 982 us.
template <int V, int P>
__global__ void __launch_bounds__(1024) block_norm_wide_kernel(const Args a)
{
    __shared__ double red_sum[2][32];
    __shared__ uint32_t red_top[32];
    q4_pdl_start();
    const int64_t row = blockIdx.x;
    const int64_t base = row * a.H;
    const int tid = threadIdx.x, nt = blockDim.x;
    float v[P][V], r[P][V];
    // both rows' loads go out before either is used
#pragma unroll
    for (int i = 0; i < P; i++) {
        const int c = (i * nt + tid) * V;
#pragma unroll
        for (int j = 0; j < V; j++) v[i][j] = r[i][j] = 0.0f;
        if (a.x && c < a.H) load<V>(a.x, a.x_dt, base + c, v[i]);
        if (a.residual && c < a.H) load<V>(a.residual, a.r_dt, base + c, r[i]);
    }
    if (a.post_w) {
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < P; i++) add_squares<V>(v[i], s);
        const float rs = rstd_of(cta_sum(s, red_sum[0]), a);
#pragma unroll
        for (int i = 0; i < P; i++) {
            const int c = (i * nt + tid) * V;
            if (c >= a.H) continue;
            float w[V];
            load<V>(a.post_w, a.w_dt, c, w);
            scale_by<V>(v[i], rs);
            scale_by<V>(v[i], w);
        }
    }
    const int64_t grow = a.gate ? gate_row(a, row) * a.H : 0;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < P; i++) {
        const int c = (i * nt + tid) * V;
        if (c >= a.H) continue;
        if (a.x) scale_by<V>(v[i], a.branch_scale);
        if (a.gate) {
            float g[V];
            load<V>(a.gate, a.g_dt, grow + c, g);
            scale_by<V>(v[i], g);
        }
        if (a.residual) {
#pragma unroll
            for (int j = 0; j < V; j++) {
                r[i][j] = __fmul_rn(r[i][j], a.res_scale);
                v[i][j] = a.x ? __fadd_rn(r[i][j], v[i][j]) : r[i][j];
            }
        }
        add_squares<V>(v[i], s);
        if (a.residual_out && q4_in_bounds(base + c + V - 1, (int64_t)a.T * a.H, a.status))
            store<V>(a.residual_out, a.r_dt, base + c, v[i]);
    }
    if (!a.y && !a.xq) return;
    const float rs = rstd_of(cta_sum(s, red_sum[1]), a);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < P; i++) {
        const int c = (i * nt + tid) * V;
        if (c >= a.H) continue;
        scale_by<V>(v[i], rs);
        if (a.pre_w) {
            float w[V];
            load<V>(a.pre_w, a.w_dt, c, w);
            scale_by<V>(v[i], w);
        }
        if (a.y && q4_in_bounds(base + c + V - 1, (int64_t)a.T * a.H, a.status)) store<V>(a.y, a.y_dt, base + c, v[i]);
        if (a.xq) settle<V>(v[i], a.y_dt, top);
    }
    if (!a.xq) return;
    top = cta_max(top, red_top);
    const float scale = scale_of(top);
    if (tid == 0) {
        a.scale_a[row] = scale;
        if (top >= 0x7F800000u) q4_set_status(a.status, Q4_ERR_NONFINITE);
    }
    const bool exact_div = !(scale >= 0x1p-100f && scale < INFINITY);
    const float inv = exact_div ? 0.0f : 1.0f / scale;
#pragma unroll
    for (int i = 0; i < P; i++) {
        const int c = (i * nt + tid) * V;
        if (c < a.H && q4_in_bounds(base + c + V - 1, (int64_t)a.T * a.H, a.status))
            store_codes<V>(a.xq + base + c, v[i], scale, inv, exact_div);
    }
}

__device__ __forceinline__ float max_nan(float a, float b)   // max(a, |b|), NaN wins
{
    float d;
    asm("{\n\t.reg .f32 m;\n\tabs.f32 m, %2;\n\tmax.NaN.f32 %0, %1, m;\n\t}" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

__device__ __forceinline__ uint64_t pair(float lo, float hi) { return tc::f2_pack(__float_as_uint(lo), __float_as_uint(hi)); }

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// V values (8 or 1) of type DT at p
template <int V, int DT> __device__ __forceinline__ void get(const uint8_t* p, float (&v)[V]) { load<V>(p, DT, 0, v); }

template <int V, int DT> __device__ __forceinline__ void put(uint8_t* p, const float (&v)[V])
{
    if constexpr (V == 2) {
        if constexpr (DT == Q4_F32) *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
        else if constexpr (DT == Q4_BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]);
            *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(&h);
        } else *reinterpret_cast<uint32_t*>(p) = h2_as_u32(__floats2half2_rn(v[0], v[1]));
    } else {
        store<V>(p, DT, 0, v);
    }
}

// f(DT) for the type dt: one branch around a whole row's work instead of one per value
template <typename F> __device__ __forceinline__ void by_type(int dt, F f)
{
    if (dt == Q4_BF16) f(std::integral_constant<int, Q4_BF16>());
    else if (dt == Q4_F32) f(std::integral_constant<int, Q4_F32>());
    else f(std::integral_constant<int, Q4_F16>());
}

// a pair as DT holds it, and the largest magnitude so far
template <int DT> __device__ __forceinline__ uint64_t settle_pair(uint64_t x, float& top)
{
    float lo = tc::f2_lo(x), hi = tc::f2_hi(x);
    if constexpr (DT == Q4_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        const uint32_t e = *reinterpret_cast<const uint32_t*>(&h);
        lo = __uint_as_float(e << 16);
        hi = __uint_as_float(e & 0xFFFF0000u);
    } else {
        lo = as_stored(lo, DT);
        hi = as_stored(hi, DT);
    }
    top = max_nan(max_nan(top, lo), hi);
    return pair(lo, hi);
}

// store_codes' quotient and rounding, two values at a time: the codes are the low bytes of the two halves
struct Coder {
    uint64_t inv2, neg2, magic;
    __device__ __forceinline__ explicit Coder(float scale)
    {
        const float inv = 1.0f / scale;
        inv2 = pair(inv, inv);
        neg2 = pair(-scale, -scale);
        magic = pair(12582912.0f, 12582912.0f);
    }
    __device__ __forceinline__ uint64_t operator()(uint64_t x) const
    {
        const uint64_t t = f2_mul(x, inv2);
        return tc::f2_add(tc::f2_fma(tc::f2_fma(neg2, t, x), inv2, t), magic);
    }
};

__device__ __forceinline__ uint32_t code_bytes(uint64_t pair) { return prmt((uint32_t)pair, (uint32_t)(pair >> 32), 0x0040u); }

// Raw words of V values of a 16-bit or 32-bit type, loaded before anything depends on the type
template <int V> struct Raw {
    uint32_t w[V];
    __device__ __forceinline__ void load(const void* base, bool wide, int64_t at)
    {
        const uint32_t* p32 = static_cast<const uint32_t*>(base) + at;
        const uint16_t* p16 = static_cast<const uint16_t*>(base) + at;
        if constexpr (V == 8) {
            const uint4 a = wide ? *reinterpret_cast<const uint4*>(p32) : *reinterpret_cast<const uint4*>(p16);
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
            if (wide) {
                const uint4 b = *reinterpret_cast<const uint4*>(p32 + 4);
                w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
            }
        } else if constexpr (V == 2) {
            if (wide) {
                const uint2 a = *reinterpret_cast<const uint2*>(p32);
                w[0] = a.x; w[1] = a.y;
            } else {
                w[0] = *reinterpret_cast<const uint32_t*>(p16);
            }
        } else {
            w[0] = wide ? *p32 : *p16;
        }
    }
    // pair j of the values (V == 1: the value and 0)
    template <int DT> __device__ __forceinline__ uint64_t get(int j) const
    {
        if constexpr (V == 1) {
            return pair(DT == Q4_F32    ? __uint_as_float(w[0])
                        : DT == Q4_BF16 ? __uint_as_float(w[0] << 16)
                                        : __half2float(__ushort_as_half((unsigned short)w[0])), 0.0f);
        } else if constexpr (DT == Q4_F32) {
            return tc::f2_pack(w[2 * j], w[2 * j + 1]);
        } else if constexpr (DT == Q4_BF16) {
            return tc::f2_pack(w[j] << 16, w[j] & 0xFFFF0000u);
        } else {
            const float2 f = __half22float2(u32_as_h2(w[j]));
            return pair(f.x, f.y);
        }
    }
};

// r * res + b, two values at a time.  The sum is a multiply-add by a one the compiler does not know: a packed product that
// feeds a packed sum was seen to be contracted with it into one rounding (mul.rn.f32x2, add.rn.f32x2, CUDA 12.9), which
// moves r' by more than an ulp where the residual and the branch cancel.
__device__ __forceinline__ uint64_t add_scaled(uint64_t r, uint64_t res2, uint64_t b, const Args& a)
{
    return tc::f2_fma(f2_mul(r, res2), a.ones, b);
}

// Up to a few thousand rows: a team of W warps a row, 256 threads or a row a CTA, E values a lane in registers (V at a time,
// chunks of a warp side by side).  x and the residual are loaded before either is used, the vectors come through L1.  One
// branch on a type stands around a row's work, not around a value's, and the fp32 arithmetic is packed in pairs (a CTA of 256
// threads with 8 values each and neither of the two took 78 instructions a value; CTAs of 128 threads instead of 256 cost 4800
// x 2048 rows 34 us instead of 24).  FULL: the lanes' values make up the row exactly (V = 8), without bound checks.
template <int V, int E, bool FULL>
__global__ void __launch_bounds__(512) block_norm_row_kernel(const Args a, const int W)
{
    constexpr int C = E / V, Q = (V + 1) / 2, D = 32 * V;   // D: between a lane's chunks
    __shared__ double red_sum[2][16];
    __shared__ float red_top[16];
    // (the block's second dimension counts the teams: no division by W)
    const int H = a.H, tl = threadIdx.x, lane = tl & 31, team = threadIdx.y, first_warp = team * W, warp = first_warp + tl / 32;
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + team;
    q4_pdl_start();
    if (row >= a.T) return;      // (whole teams)
    const int64_t base = row * H;
    const int c0 = tl / 32 * (32 * E) + lane * V, left = H - c0;
    auto each = [&](auto f) {    // f(chunk) for this lane's chunks of the row
#pragma unroll
        for (int i = 0; i < C; i++)
            if (FULL || i * D < left) f(i);
    };
    auto team_sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * W) : "memory"); };
    auto team_sum = [&](double v, double* red) {
        v = warp_sum(v);
        if (W == 1) return v;
        if (lane == 0) red[warp] = v;
        team_sync();
        v = red[first_warp];
        for (int i = 1; i < W; i++) v += red[first_warp + i];
        return v;
    };
    Raw<V> rx[C], rr[C];
    if (a.x) each([&](int i) { rx[i].load(a.x, a.x_dt == Q4_F32, base + c0 + i * D); });
    if (a.residual) each([&](int i) { rr[i].load(a.residual, a.r_dt == Q4_F32, base + c0 + i * D); });
    // the lane's values; what is not of the row stays 0 (-0 without x: a sum with -0 keeps every value as it is)
    uint64_t v[C][Q];
    auto all = [&](auto f) {
#pragma unroll
        for (int i = 0; i < C; i++)
#pragma unroll
            for (int j = 0; j < Q; j++) v[i][j] = f(v[i][j]);
    };
    auto times = [&](float f) {
        const uint64_t f2 = pair(f, f);
        all([&](uint64_t x) { return f2_mul(x, f2); });
    };
    auto times_vector = [&](const void* p, int dt) {
        by_type(dt, [&](auto DT) {
            each([&](int i) {
                Raw<V> w;
                w.load(p, DT() == Q4_F32, c0 + i * D);
#pragma unroll
                for (int j = 0; j < Q; j++) v[i][j] = f2_mul(v[i][j], w.template get<DT()>(j));
            });
        });
    };
    auto squares = [&] {   // four chains: one would wait for each multiply-add
        double s4[4] = {};
#pragma unroll
        for (int i = 0; i < C; i++)
#pragma unroll
            for (int j = 0; j < Q; j++) {
                const int k = 2 * ((i * Q + j) & 1);
                const double lo = (double)tc::f2_lo(v[i][j]);
                s4[k] = fma(lo, lo, s4[k]);
                if constexpr (V > 1) {
                    const double hi = (double)tc::f2_hi(v[i][j]);
                    s4[k + 1] = fma(hi, hi, s4[k + 1]);
                }
            }
        return (s4[0] + s4[1]) + (s4[2] + s4[3]);
    };
    all([&](uint64_t) { return a.x ? 0ull : 0x8000000080000000ull; });
    if (a.x) {
        by_type(a.x_dt, [&](auto DT) {
            each([&](int i) {
#pragma unroll
                for (int j = 0; j < Q; j++) v[i][j] = rx[i].template get<DT()>(j);
            });
        });
        if (a.post_w) {
            times(rstd_of(team_sum(squares(), red_sum[0]), a));
            times_vector(a.post_w, a.w_dt);
        }
        if (a.branch_scale != 1.0f) times(a.branch_scale);
        if (a.gate) times_vector(static_cast<const uint8_t*>(a.gate) + gate_row(a, row) * H * (a.g_dt == Q4_F32 ? 4 : 2), a.g_dt);
    }
    if (a.residual) {
        const uint64_t res2 = pair(a.res_scale, a.res_scale);
        by_type(a.r_dt, [&](auto DT) {
            each([&](int i) {
#pragma unroll
                for (int j = 0; j < Q; j++) v[i][j] = add_scaled(rr[i].template get<DT()>(j), res2, v[i][j], a);
            });
        });
    }
    auto chunk = [&](int i, float (&w)[V]) {
#pragma unroll
        for (int j = 0; j < V; j++) w[j] = j & 1 ? tc::f2_hi(v[i][j / 2]) : tc::f2_lo(v[i][j / 2]);
    };
    auto write = [&](void* out, auto DT) {
        constexpr int es = DT() == Q4_F32 ? 4 : 2;
        uint8_t* p = static_cast<uint8_t*>(out) + (base + c0) * es;
        each([&](int i) {
            float w[V];
            chunk(i, w);
            if (q4_in_bounds(base + c0 + i * D + V - 1, (int64_t)a.T * H, a.status)) put<V, DT()>(p + i * (D * es), w);
        });
    };
    if (a.residual_out) by_type(a.r_dt, [&](auto DT) { write(a.residual_out, DT); });
    if (!a.y && !a.xq) return;
    times(rstd_of(team_sum(squares(), red_sum[1]), a));
    if (a.pre_w) times_vector(a.pre_w, a.w_dt);
    float top = 0.0f;
    by_type(a.y_dt, [&](auto DT) {
        if (a.y) write(a.y, DT);
        if (a.xq) all([&](uint64_t x) { return settle_pair<DT()>(x, top); });
    });
    if (!a.xq) return;
    uint32_t tb = __reduce_max_sync(0xffffffffu, __float_as_uint(top));   // (bit order = order of magnitudes, NaN on top)
    if (W > 1) {
        if (lane == 0) red_top[warp] = __uint_as_float(tb);
        team_sync();
        for (int i = 0; i < W; i++) tb = max(tb, __float_as_uint(red_top[first_warp + i]));
    }
    const float scale = scale_of(tb);
    if (tl == 0) {
        a.scale_a[row] = scale;
        if (tb >= 0x7F800000u) q4_set_status(a.status, Q4_ERR_NONFINITE);
    }
    int8_t* out = a.xq + base + c0;
    if (!(scale >= 0x1p-100f && scale < INFINITY)) {
        each([&](int i) {
            float w[V];
            chunk(i, w);
            if (q4_in_bounds(base + c0 + i * D + V - 1, (int64_t)a.T * H, a.status)) store_codes<V>(out + i * D, w, scale, 0.0f, true);
        });
        return;
    }
    const Coder code(scale);
    each([&](int i) {
        if (!q4_in_bounds(base + c0 + i * D + V - 1, (int64_t)a.T * H, a.status)) return;
        if constexpr (V == 8)
            *reinterpret_cast<uint2*>(out + i * D) =
                make_uint2(prmt(code_bytes(code(v[i][0])), code_bytes(code(v[i][1])), 0x5410u),
                           prmt(code_bytes(code(v[i][2])), code_bytes(code(v[i][3])), 0x5410u));
        else if constexpr (V == 2) *reinterpret_cast<uint16_t*>(out + i * D) = (uint16_t)code_bytes(code(v[i][0]));
        else out[i * D] = (int8_t)code(v[i][0]);
    });
}

// Many rows: one persistent CTA of 16 or 20 warps an SM.  A team of W warps (1 up to 2048 values a row) owns a row at a time, E
// values a lane in registers, so a row's two sums and its maximum cost a lane a few instructions for E values
// and, with one warp a team, no barrier.  (With 256 threads a row the reductions alone were a fifth of 78 instructions a
// value: 2.1 TB/s.)  Rows come ahead of use by bulk copies into the team's ring in shared memory: x, the residual, and
// the gate's row where it changes with the token.  A copy covers the 16-byte pieces that hold the row, so rows of odd
// width take this path too, one value at a time (V = 1; else V = 8).  What every row
// shares (the norms' weights, a single gate) is kept as fp32 in shared memory.
struct Ring {
    int stages, warps, teams;        // slots a team, warps a team, teams a CTA
    int slot[3];                     // bytes of a slot's x, residual and gate pieces (0: not in the ring)
    int post, gate, pre;             // where the shared vectors start (bytes; -1: none)
    int rings;                       // where the rings start
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(tc::smem_u32(dst)), "l"(src), "r"(bytes), "r"(tc::smem_u32(bar)) : "memory");
}

// 64 values a lane need 128 registers, fewer fit in 100
__host__ __device__ constexpr int team_threads(int e) { return e == 64 ? 512 : 640; }
constexpr int kMaxSlots = 48;   // stages x teams
constexpr int kTeamSmem = 224 * 1024;   // shared memory a CTA for the vectors and the rings, at most

// A shared vector in fp32: V == 8 keeps the two halves of each 8 values apart, so that a warp's 16-byte reads of
// consecutive pieces touch every bank once.
template <int V> __device__ __forceinline__ int shared_at(int c, int j, int H)
{
    return V == 8 ? (j >> 2) * (H / 2) + (c >> 1) + (j & 3) : c + j;
}

template <int V, int E, bool FULL>
__global__ void __launch_bounds__(team_threads(E), 1) block_norm_team_kernel(const Args a, const Ring q)
{
    constexpr int C = E / V, kTeamThreads = team_threads(E);
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kMaxSlots];
    __shared__ double red_sum[2][2][kTeamThreads / 32];
    __shared__ float red_top[2][kTeamThreads / 32];
    __shared__ volatile int abort_flag;   // one lane's wait ran out: the others' end too
    const int H = a.H, W = q.warps, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int team = warp / W, first_warp = team * W, tl = (warp - first_warp) * 32 + lane, tt = 32 * W;
    const int slot_bytes = q.slot[0] + q.slot[1] + q.slot[2];
    if (threadIdx.x == 0) {
        for (int i = 0; i < q.stages * q.teams; i++) tc::mbar_init(&full[i], 1);
        abort_flag = 0;
        tc::fence_mbar_init();
    }
    __syncthreads();
    q4_pdl_start();
    const bool live = team < q.teams;
    const int64_t step = (int64_t)gridDim.x * q.teams, row0 = (int64_t)blockIdx.x * q.teams + team;
    uint8_t* ring = smem + q.rings + (int64_t)team * q.stages * slot_bytes;
    const int xs = a.x_dt == Q4_F32 ? 4 : 2, rs_ = a.r_dt == Q4_F32 ? 4 : 2, gs = a.g_dt == Q4_F32 ? 4 : 2;
    const int64_t g_rows = q.slot[2] ? a.T / a.tokens_per_gate : 0;

    // the 16-byte pieces of row i of an array of n rows; the array's last bytes past a whole piece are left out (tail)
    auto piece = [&](const void* base, int64_t i, int64_t n, int es, const uint8_t*& src, uint32_t& bytes) {
        const int64_t b0 = i * H * es & ~(int64_t)15, end = n * H * es & ~(int64_t)15;
        const int64_t b1 = ((i + 1) * H * es + 15) & ~(int64_t)15;
        src = static_cast<const uint8_t*>(base) + b0;
        bytes = (uint32_t)((b1 < end ? b1 : end) - b0);
    };
    auto fetch = [&](int64_t row, int s) {   // one lane
        uint8_t* dst = ring + (int64_t)s * slot_bytes;
        uint64_t* bar = &full[team * q.stages + s];
        const uint8_t *px = nullptr, *pr = nullptr, *pg = nullptr;
        uint32_t bx = 0, br = 0, bg = 0;
        if (q.slot[0]) piece(a.x, row, a.T, xs, px, bx);
        if (q.slot[1]) piece(a.residual, row, a.T, rs_, pr, br);
        if (q.slot[2]) piece(a.gate, gate_row(a, row), g_rows, gs, pg, bg);
        tc::mbar_arrive_expect_tx(bar, bx + br + bg);
        if (bx) bulk_load(dst, px, bx, bar);
        if (br) bulk_load(dst + q.slot[0], pr, br, bar);
        if (bg) bulk_load(dst + q.slot[0] + q.slot[1], pg, bg, bar);
    };
    if (live && tl == 0)
        for (int i = 0; i < q.stages; i++)
            if (row0 + i * step < a.T) fetch(row0 + i * step, i);
    // the shared vectors into shared memory, the three vectors' loads side by side
    for (int c = threadIdx.x * V; c < H; c += kTeamThreads * V) {
        float w[3][V];
        auto read = [&](const void* p, int dt, bool on, float (&f)[V]) {
            if (on) by_type(dt, [&](auto DT) { get<V, DT()>(static_cast<const uint8_t*>(p) + (int64_t)c * (DT() == Q4_F32 ? 4 : 2), f); });
        };
        auto keep = [&](int at, const float (&f)[V]) {
            if (at >= 0)
#pragma unroll
                for (int j = 0; j < V; j++) reinterpret_cast<float*>(smem + at)[shared_at<V>(c, j, H)] = f[j];
        };
        read(a.post_w, a.w_dt, q.post >= 0, w[0]);
        read(a.gate, a.g_dt, q.gate >= 0, w[1]);
        read(a.pre_w, a.w_dt, q.pre >= 0, w[2]);
        keep(q.post, w[0]);
        keep(q.gate, w[1]);
        keep(q.pre, w[2]);
    }
    __syncthreads();
    if (!live) return;
    const float* s_post = reinterpret_cast<const float*>(smem + (q.post < 0 ? 0 : q.post));
    const float* s_gate = reinterpret_cast<const float*>(smem + (q.gate < 0 ? 0 : q.gate));
    const float* s_pre = reinterpret_cast<const float*>(smem + (q.pre < 0 ? 0 : q.pre));

    auto team_sync = [&] {
        if (W == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(tt) : "memory");
    };
    auto team_sum = [&](double v, double* red) {
        v = warp_sum(v);
        if (W == 1) return v;
        if (lane == 0) red[warp] = v;
        team_sync();
        v = red[first_warp];
        for (int i = 1; i < W; i++) v += red[first_warp + i];
        return v;
    };

    // A warp owns E * 32 consecutive values of the row, a lane V of each 32 V: chunk i is at a constant offset from the
    // lane's first value c0, and in the row while i * 32 V < left.
    const int c0 = (warp - first_warp) * (32 * E) + lane * V, left = H - c0;
    constexpr int D = 32 * V;   // between a lane's chunks
    // the first row of each array whose end lies behind the array's last whole piece
    auto first_cut = [&](int64_t n, int es) { return (n * H * es & ~(int64_t)15) / ((int64_t)H * es); };
    const int64_t cut[3] = {q.slot[0] ? first_cut(a.T, xs) : a.T, q.slot[1] ? first_cut(a.T, rs_) : a.T, first_cut(g_rows, gs)};
    int s = -1, par = 1;
    uint32_t phase = 1;
    bool ok = true;   // (a thread that gives up still meets its team; the row is then undefined)
    for (int64_t row = row0; row < a.T; row += step) {
        par ^= 1;
        if (++s == q.stages) s = 0;
        if (s == 0) phase ^= 1;
        const int64_t base = row * H;
        uint8_t* src = ring + (int64_t)s * slot_bytes;
        ok = ok && tc::mbar_wait(&full[team * q.stages + s], phase, a.status, &abort_flag);
        if (V != 8 && (row >= cut[0] || row >= cut[1] || (q.slot[2] && gate_row(a, row) >= cut[2]))) {
            // the bytes past an array's last whole piece (the end of its last row, for short rows of several)
            auto tail = [&](const void* p, int64_t i, int64_t n, int es, uint8_t* dst) {
                const int64_t b0 = i * H * es & ~(int64_t)15, end = n * H * es & ~(int64_t)15;
                const int64_t hi = (i + 1) * H * es;
                for (int64_t b = (end > b0 ? end : b0) + 2 * tl; b < hi; b += 2 * tt)
                    *reinterpret_cast<uint16_t*>(dst + (b - b0)) = *reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(p) + b);
            };
            if (q.slot[0]) tail(a.x, row, a.T, xs, src);
            if (q.slot[1]) tail(a.residual, row, a.T, rs_, src + q.slot[0]);
            if (q.slot[2]) tail(a.gate, gate_row(a, row), g_rows, gs, src + q.slot[0] + q.slot[1]);
            team_sync();
        }
        // the lane's E values in pairs, for the packed fp32 instructions (each half rounds like the scalar one); a
        // chunk's V values are consecutive, and what is not of the row stays 0
        uint64_t v[E / 2];
#pragma unroll
        for (int i = 0; i < E / 2; i++) v[i] = q.slot[0] ? 0 : 0x8000000080000000ull;
        // each: f(chunk) for this lane's chunks of the row
        auto each = [&](auto f) {
#pragma unroll
            for (int i = 0; i < C; i++)
                if (FULL || i * D < left) f(i);
        };
        auto all = [&](auto f) {
#pragma unroll
            for (int i = 0; i < E / 2; i++) v[i] = f(v[i]);
        };
        auto times = [&](float f) {
            const uint64_t f2 = pair(f, f);
            all([&](uint64_t x) { return f2_mul(x, f2); });
        };
        // values of type DT at p (chunk i at p + i * D values) combined with v pair by pair: v = f(v, value)
        auto with = [&](const uint8_t* p, auto DT, auto f) {
            constexpr int es = DT() == Q4_F32 ? 4 : 2;
            if constexpr (V == 1) {
#pragma unroll
                for (int i = 0; i < C; i += 2) {
                    float lo[1] = {0.0f}, hi[1] = {0.0f};
                    if (i * D < left) get<1, DT()>(p + i * (D * es), lo);
                    if ((i + 1) * D < left) get<1, DT()>(p + (i + 1) * (D * es), hi);
                    v[i / 2] = f(v[i / 2], pair(lo[0], hi[0]));
                }
            } else {
                each([&](int i) {
                    float w[V];
                    get<V, DT()>(p + i * (D * es), w);
#pragma unroll
                    for (int j = 0; j < V; j += 2) v[(i * V + j) / 2] = f(v[(i * V + j) / 2], pair(w[j], w[j + 1]));
                });
            }
        };
        auto times_shared = [&](const float* sm) {
            if constexpr (V == 8) {
                const float* p0 = sm + (c0 >> 1);
                const float* p1 = p0 + H / 2;
                each([&](int i) {
                    const ulonglong2 lo = *reinterpret_cast<const ulonglong2*>(p0 + i * (D / 2));
                    const ulonglong2 hi = *reinterpret_cast<const ulonglong2*>(p1 + i * (D / 2));
                    v[4 * i] = f2_mul(v[4 * i], lo.x);
                    v[4 * i + 1] = f2_mul(v[4 * i + 1], lo.y);
                    v[4 * i + 2] = f2_mul(v[4 * i + 2], hi.x);
                    v[4 * i + 3] = f2_mul(v[4 * i + 3], hi.y);
                });
            } else {
                with(reinterpret_cast<const uint8_t*>(sm + c0), std::integral_constant<int, Q4_F32>(), f2_mul);
            }
        };
        auto squares = [&] {   // four chains: one would wait for each multiply-add
            double s4[4] = {};
#pragma unroll
            for (int i = 0; i < E / 2; i++) {
                const double lo = (double)tc::f2_lo(v[i]), hi = (double)tc::f2_hi(v[i]);
                s4[2 * (i & 1)] = fma(lo, lo, s4[2 * (i & 1)]);
                s4[2 * (i & 1) + 1] = fma(hi, hi, s4[2 * (i & 1) + 1]);
            }
            return (s4[0] + s4[1]) + (s4[2] + s4[3]);
        };
        if (q.slot[0]) {
            by_type(a.x_dt, [&](auto DT) {
                constexpr int es = DT() == Q4_F32 ? 4 : 2;
                with(src + (base * es & 15) + c0 * es, DT, [](uint64_t, uint64_t x) { return x; });
            });
            if (a.post_w) {
                times(rstd_of(team_sum(squares(), red_sum[par][0]), a));
                times_shared(s_post);
            }
            if (a.branch_scale != 1.0f) times(a.branch_scale);
            if (q.slot[2])
                by_type(a.g_dt, [&](auto DT) {
                    constexpr int es = DT() == Q4_F32 ? 4 : 2;
                    with(src + q.slot[0] + q.slot[1] + (gate_row(a, row) * H * es & 15) + c0 * es, DT, f2_mul);
                });
            else if (q.gate >= 0) times_shared(s_gate);
        }
        if (q.slot[1]) {
            const uint64_t rs2 = pair(a.res_scale, a.res_scale);
            by_type(a.r_dt, [&](auto DT) {
                constexpr int es = DT() == Q4_F32 ? 4 : 2;
                with(src + q.slot[0] + (base * es & 15) + c0 * es, DT,
                     [&](uint64_t x, uint64_t r) { return add_scaled(r, rs2, x, a); });
            });
        }
        const float rs = rstd_of(team_sum(squares(), red_sum[par][1]), a);
        // every lane of the team has read the slot (the sum's barrier, or the warp's shuffles, lie behind the reads)
        {
            __syncwarp();
            const int64_t next = row + q.stages * step;
            if (tl == 0 && ok && next < a.T) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                fetch(next, s);
            }
        }
        auto chunk = [&](int i, float (&w)[V]) {
#pragma unroll
            for (int j = 0; j < V; j++) w[j] = (i * V + j) & 1 ? tc::f2_hi(v[(i * V + j) / 2]) : tc::f2_lo(v[(i * V + j) / 2]);
        };
        auto write = [&](void* out, auto DT) {
            constexpr int es = DT() == Q4_F32 ? 4 : 2;
            uint8_t* p = static_cast<uint8_t*>(out) + (base + c0) * es;
            each([&](int i) {
                float w[V];
                chunk(i, w);
                if (q4_in_bounds(base + c0 + i * D + V - 1, (int64_t)a.T * H, a.status)) put<V, DT()>(p + i * (D * es), w);
            });
        };
        if (a.residual_out) by_type(a.r_dt, [&](auto DT) { write(a.residual_out, DT); });
        if (!a.y && !a.xq) continue;
        times(rs);
        if (q.pre >= 0) times_shared(s_pre);
        float top = 0.0f;
        by_type(a.y_dt, [&](auto DT) {
            if (a.y) write(a.y, DT);
            if (a.xq) all([&](uint64_t x) { return settle_pair<DT()>(x, top); });
        });
        if (!a.xq) continue;
        uint32_t tb = __reduce_max_sync(0xffffffffu, __float_as_uint(top));   // (bit order = order of magnitudes, NaN on top)
        if (W > 1) {
            if (lane == 0) red_top[par][warp] = __uint_as_float(tb);
            team_sync();
            for (int i = 0; i < W; i++) tb = max(tb, __float_as_uint(red_top[par][first_warp + i]));
        }
        const float scale = scale_of(tb);
        if (tl == 0) {
            a.scale_a[row] = scale;
            if (tb >= 0x7F800000u) q4_set_status(a.status, Q4_ERR_NONFINITE);
        }
        const bool exact_div = !(scale >= 0x1p-100f && scale < INFINITY);
        int8_t* out = a.xq + base + c0;
        if (exact_div) {
            each([&](int i) {
                float w[V];
                chunk(i, w);
                if (q4_in_bounds(base + c0 + i * D + V - 1, (int64_t)a.T * H, a.status)) store_codes<V>(out + i * D, w, scale, 0.0f, true);
            });
        } else {
            const Coder code(scale);
            all([&](uint64_t x) { return code(x); });
            each([&](int i) {
                if (!q4_in_bounds(base + c0 + i * D + V - 1, (int64_t)a.T * H, a.status)) return;
                auto bytes = [&](int j) { return code_bytes(v[j]); };
                if constexpr (V == 8)
                    *reinterpret_cast<uint2*>(out + i * D) = make_uint2(prmt(bytes(4 * i), bytes(4 * i + 1), 0x5410u),
                                                                        prmt(bytes(4 * i + 2), bytes(4 * i + 3), 0x5410u));
                else out[i * D] = (int8_t)(i & 1 ? v[i / 2] >> 32 : v[i / 2]);
            });
        }
    }
    if (!ok && tl == 0) {   // given up: no copy may land in the memory of the CTA that follows
        const uint64_t t0 = tc::globaltimer_ns();
        for (uint32_t i = 0; !tc::wait_expired(t0, 100000000ull, i, 64); i++) __nanosleep(1000);
    }
}

int launch_rows(const Args& a, bool whole, cudaStream_t s)
{
    const int V = !whole || a.H % 2 ? 1 : a.H % 8 ? 2 : 8;
    if (a.H > 16384) {
        const dim3 grid(a.T), block(1024);
        return V == 8 ? q4_launch_pdl(block_norm_wide_kernel<8, 4>, grid, block, 0, s, a)
                      : q4_launch_pdl(block_norm_wide_kernel<1, 32>, grid, block, 0, s, a);
    }
    // values a lane: 8 in rows of up to 256 (and one at a time: 16 take 110 registers, and 32, for rows above 8192 values, spill
    // 76 bytes), else 16; 16 warps a row at most
    int E = a.H <= 256 || V == 1 ? 8 : 16;
    while (32 * E * 16 < a.H) E *= 2;
    const int W = (a.H + 32 * E - 1) / (32 * E), teams = (8 + W - 1) / W;   // (8 warps a CTA or the next multiple: 2400 x 3000 in 20.0 us with 12 warps, 23.3 with 6)
    const dim3 grid((unsigned)((a.T + (int64_t)teams - 1) / teams)), block(32 * W, teams);
    auto go = [&](auto kern) { return q4_launch_pdl(kern, grid, block, 0, s, a, W); };
    if (V == 8 && a.H == 32 * E * W)
        return E == 8 ? go(block_norm_row_kernel<8, 8, true>) : E == 16 ? go(block_norm_row_kernel<8, 16, true>) : go(block_norm_row_kernel<8, 32, true>);
    if (V == 8)
        return E == 8 ? go(block_norm_row_kernel<8, 8, false>) : E == 16 ? go(block_norm_row_kernel<8, 16, false>) : go(block_norm_row_kernel<8, 32, false>);
    if (V == 2)
        return E == 8 ? go(block_norm_row_kernel<2, 8, false>) : E == 16 ? go(block_norm_row_kernel<2, 16, false>) : go(block_norm_row_kernel<2, 32, false>);
    return E == 8 ? go(block_norm_row_kernel<1, 8, false>) : E == 16 ? go(block_norm_row_kernel<1, 16, false>) : go(block_norm_row_kernel<1, 32, false>);
}

int elem_bytes(int dt) { return dt == Q4_F32 ? 4 : 2; }

// The persistent form for E values a lane: Q4_ERR_UNSUPPORTED where the shape does not suit it
int launch_teams(const Args& a, int E, int min_rows, bool many_gates, cudaStream_t s)
{
    const int sms = q4_num_sms();
    const int V = a.H % 8 == 0 ? 8 : 1;
    Ring q = {};
    q.warps = (a.H + 32 * E - 1) / (32 * E);
    if (q.warps > team_threads(E) / 32) return Q4_ERR_UNSUPPORTED;
    const bool full = V == 8 && a.H == 32 * E * q.warps;
    auto slot = [&](bool on, int dt) { return on ? (a.H * elem_bytes(dt) + 15) / 16 * 16 + (V == 8 ? 0 : 16) : 0; };
    q.slot[0] = slot(a.x, a.x_dt);
    q.slot[1] = slot(a.residual, a.r_dt);
    q.slot[2] = slot(many_gates, a.g_dt);
    const int row = q.slot[0] + q.slot[1] + q.slot[2];
    int at = 0;
    auto vec = [&](bool on) {
        const int here = at;
        if (!on) return -1;
        at += (4 * a.H + 15) / 16 * 16;
        return here;
    };
    q.post = vec(a.post_w);
    q.gate = vec(a.gate && !many_gates);
    q.pre = vec(a.pre_w);
    q.rings = at;
    const int room = kTeamSmem - at;
    q.teams = std::min(team_threads(E) / 32 / q.warps, room / row);
    if (q.teams < 1 || a.T < (int64_t)min_rows * sms * q.teams) return Q4_ERR_UNSUPPORTED;
    q.stages = std::min({3, room / (row * q.teams), kMaxSlots / q.teams});
    const int smem = at + q.stages * q.teams * row;
    auto go = [&](auto kern) {
        // the attribute is the kernel's on this device, not the call's: one value for every shape, or a call with a smaller
        // shape on another thread would lower it between this call's two lines and the launch be refused
        if (const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kTeamSmem)) return q4_cuda_status(e);
        return q4_launch_pdl(kern, dim3(sms), dim3(team_threads(E)), smem, s, a, q);
    };
    if (full) return E == 64 ? go(block_norm_team_kernel<8, 64, true>) : E == 32 ? go(block_norm_team_kernel<8, 32, true>)
                                                                                 : go(block_norm_team_kernel<8, 16, true>);
    if (V == 8) return E == 64 ? go(block_norm_team_kernel<8, 64, false>) : E == 32 ? go(block_norm_team_kernel<8, 32, false>)
                                                                                    : go(block_norm_team_kernel<8, 16, false>);
    if (E == 64) return Q4_ERR_UNSUPPORTED;   // (not instantiated: 64 values a lane, one at a time, spilled)
    return E == 32 ? go(block_norm_team_kernel<1, 32, false>) : go(block_norm_team_kernel<1, 16, false>);
}

// When the persistent form takes the rows.  It issues about half the instructions a value, the team a row moves bytes faster
// (6.7 against 5.3 TB/s), so it pays where little is moved for much work.  16384 x 2048, persistent / team a row, us:
//   bf16 in and out (7 bytes a value), codes: 43 / 49; with the norm after the block 51 / 63; with a gate too 53 / 67
//   the same without codes (8 bytes): 51 / 49     fp32 block output (9 bytes), codes: 55 / 52; with both 58 / 70
//   fp32 residual (11 bytes), codes: 71 / 59      all fp32 (13 bytes), codes: 85 / 65; with both, no codes 90 / 82
// Fitted to 16384 x 2048 values, the persistent form's time is 6.3 us a byte and the other's 33 and what is below.
// It also needs rows enough (bf16 with every part): H 1024, 12000 rows 25.7 / 26.1, 32768 rows 53 / 64; H 2048, 4800 rows 25.1 / 22.6, 12000 rows
// 44.1 / 50; H 4096, 2400 rows 26.2 / 24.1, 4800 rows 39 / 46; H 8192, 600 rows 20.8 / 17.0, 1200 rows 28 / 30: three rows a
// team, two above 4096 values, five below 1536.  Rows of odd width (a value at a time): H 1001, 1111 rows 12.2 / 7.0, 1600 rows 12.5 / 11.9, 2400
// rows 12.8 / 16.4; H 5001, 900 rows 26 / 48: from 12 rows an SM on, 4 above 4096 values; rows of pairs never (H 1002, 9600
// rows 40 / 29).  The most values a lane that make up the row, or else leave the lanes four fifths full, cost the fewest
// instructions.
int launch_many(const Args& a, bool many_gates, cudaStream_t s)
{
    if (a.H % 2) {
        if (a.H <= 256 || a.T < (a.H > 4096 ? 4 : 12) * q4_num_sms()) return Q4_ERR_UNSUPPORTED;
        return launch_teams(a, a.H <= 512 ? 16 : 32, 0, many_gates, s);
    }
    if (a.H % 8 || a.H < 1024) return Q4_ERR_UNSUPPORTED;
    const int bytes = (a.x ? elem_bytes(a.x_dt) : 0) + (a.residual ? elem_bytes(a.r_dt) : 0) + (a.residual_out ? elem_bytes(a.r_dt) : 0) +
                      (a.y ? elem_bytes(a.y_dt) : 0) + (a.xq ? 1 : 0) + (many_gates ? elem_bytes(a.g_dt) : 0);
    if (63 * bytes >= 10 * (33 + (a.post_w ? 14 : 0) + (a.gate ? 4 : 0) + (a.xq ? 16 : 0))) return Q4_ERR_UNSUPPORTED;
    // (5120 values: 32 a lane make up the row, 9600 rows 95 us; 64 fill it to five sixths, 104)
    const int full = a.H % 2048 == 0 ? 64 : a.H % 1024 == 0 ? 32 : 0;
    const int min_rows = a.H > 4096 ? 2 : a.H >= 1536 ? 3 : 5;
    if (full) return launch_teams(a, full, min_rows, many_gates, s);
    for (int E = 64; E >= 16; E /= 2) {
        const int cap = (a.H + 32 * E - 1) / (32 * E) * 32 * E;
        if (5 * a.H >= 4 * cap || E == 16) return launch_teams(a, E, min_rows, many_gates, s);
    }
    return Q4_ERR_UNSUPPORTED;
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
    if (!(d->eps >= 0.0) || isinf(d->eps)) return Q4_ERR_SHAPE;
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
    const int64_t in_n[5] = {n * (int64_t)elem_bytes(d->x_dtype), n * (int64_t)elem_bytes(d->residual_dtype), H * (int64_t)elem_bytes(d->w_dtype),
                             H * (int64_t)elem_bytes(d->w_dtype), (int64_t)d->gate_rows * H * (int64_t)elem_bytes(d->gate_dtype)};
    const void* out[4] = {d->residual_out, d->y, d->xq, d->scale_a};
    const int64_t out_n[4] = {n * (int64_t)elem_bytes(d->residual_dtype), n * (int64_t)elem_bytes(d->y_dtype), n, 4 * (int64_t)T};
    for (int o = 0; o < 4; o++) {
        for (int i = 0; i < 5; i++) {
            const bool in_place = o < 2 && i < 2 && out[o] == in[i] && out_n[o] == in_n[i];
            if (!in_place && q4_overlap(out[o], out_n[o], in[i], in_n[i])) return Q4_ERR_UNSUPPORTED;
        }
        for (int q = 0; q < o; q++)
            if (q4_overlap(out[o], out_n[o], out[q], out_n[q])) return Q4_ERR_UNSUPPORTED;
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
    a.tokens_per_gate = d->gate && d->gate_rows > 1 ? T / d->gate_rows : 0;
    a.eps = d->eps;
    a.res_scale = d->res_scale;
    a.branch_scale = d->branch_scale;
    a.inv_h = 1.0 / H;
    a.ones = 0x3F8000003F800000ull;
    a.status = dev_status;
    // Arrays that start on 16 bytes (8 for the codes) take the persistent form when there are rows enough, and
    // 16-byte accesses when H % 8 == 0 keeps the rows so (pairs when H is even); anything else goes one value at a time.
    const bool whole = q4_aligned16(d->x) && q4_aligned16(d->residual) && q4_aligned16(d->residual_out) &&
                       q4_aligned16(d->post_w) && q4_aligned16(d->pre_w) && q4_aligned16(d->gate) && q4_aligned16(d->y) &&
                       ((uintptr_t)d->xq & 7u) == 0;
    if (whole) {
        const int rc = launch_many(a, d->gate && d->gate_rows > 1, (cudaStream_t)stream);
        if (rc != Q4_ERR_UNSUPPORTED) return rc;
    }
    return launch_rows(a, whole, (cudaStream_t)stream);
}
