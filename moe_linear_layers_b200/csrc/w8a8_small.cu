// W8A8 products for few tokens: the weights stream through registers once.
//
// acc[n][j] = sum_k wq[n][k] * xq[j][k] for 16 weight rows a CTA (16 of each matrix when gated) and up to 8 * MT tokens,
// exact in int32 on the warp-level int8 MMA (16 x 8 x 32): 8 tokens cost what one does, and a thread's
// operand registers are filled by plain 16-byte loads.  The order of k inside a sum is free, so the MMA's
// k slots are given the bytes that a 16-byte load brings: lane (g, t) takes bytes 16 t .. 16 t + 15 of each 64-byte
// block of rows g and g + 8 (weights) and of token g (activations), and the four words fill two MMAs' slots.
//
// Memory-bound: n * k bytes of weights.  The CTA's warps split k in 128-byte blocks, and meet
// once through shared memory.  Measured on B200, back to back: 1 x 2048 x 2048 2.3 us, 1 x 8192 x 2048 3.2 us (5.2 TB/s, weights
// partly in L2), gated 8.1 us (4.1 TB/s), 16 x 2048 x 8192 6.4 us.
#include "w8a8_common.cuh"

namespace {

using w8::Problem;

constexpr int kRows = 16;

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ld16(const int8_t* p, bool ok)
{
    return ok ? *reinterpret_cast<const uint4*>(p) : make_uint4(0u, 0u, 0u, 0u);
}

// MT: groups of 8 tokens a CTA; MATS: 1, or 2 = gate and up; U: blocks of k whose loads are in flight together
template <int MT, int MATS, int kWarps>
__global__ void __launch_bounds__(kWarps * 32) w8a8_small_kernel(const Problem p)
{
    constexpr int U = MT * MATS == 1 ? 4 : 2;
    __shared__ int part[kWarps][MATS * kRows * 8 * MT];
    const int n0 = blockIdx.x * kRows, m0 = blockIdx.y * 8 * MT;
    // The CTA's weight rows (one stretch of memory) start towards L2 while the previous kernel still runs: a prefetch reads
    // nothing into the kernel, so it may pass the wait.  Weights from DRAM, 1 x 8192 x 2048: 5.0 -> 4.1 us, 1 x 2048 x 8192
    // 6.7 -> 5.3, gated 1 x 8192 x 2048 8.8 -> 8.9.
    q4_pdl_trigger();
    if (threadIdx.x < MATS && blockIdx.y == 0) {
        const uint32_t bytes = (uint32_t)min(kRows, p.n - n0) * (uint32_t)p.k;
        const int8_t* w = (threadIdx.x ? p.w1 : p.w0) + (int64_t)n0 * p.k;
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(w), "r"(bytes) : "memory");
    }
    q4_pdl_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int g = lane / 4, t = lane % 4;
    int acc[MATS][MT][4] = {};
    const int8_t* wr[MATS][2];
    bool wok[2], xok[MT];
#pragma unroll
    for (int h = 0; h < 2; h++) {
        wok[h] = n0 + g + 8 * h < p.n;
        const int64_t row = wok[h] ? n0 + g + 8 * h : 0;
        wr[0][h] = p.w0 + row * p.k;
        if constexpr (MATS == 2) wr[1][h] = p.w1 + row * p.k;
    }
    const int8_t* xr[MT];
#pragma unroll
    for (int i = 0; i < MT; i++) {
        xok[i] = m0 + 8 * i + g < p.m;
        xr[i] = p.xq + (int64_t)(xok[i] ? m0 + 8 * i + g : 0) * p.k;
    }
#pragma unroll U
    for (int k0 = warp * 128; k0 < p.k; k0 += kWarps * 128) {
        uint4 w[2][MATS][2], x[2][MT];
#pragma unroll
        for (int c = 0; c < 2; c++) {
            const int kk = k0 + 64 * c + 16 * t;
            const bool in = kk < p.k;   // (k is a multiple of 16)
#pragma unroll
            for (int q = 0; q < MATS; q++)
#pragma unroll
                for (int h = 0; h < 2; h++) w[c][q][h] = ld16(wr[q][h] + kk, in && wok[h]);
#pragma unroll
            for (int i = 0; i < MT; i++) x[c][i] = ld16(xr[i] + kk, in && xok[i]);
        }
#pragma unroll
        for (int c = 0; c < 2; c++)
#pragma unroll
            for (int i = 0; i < MT; i++)
#pragma unroll
                for (int q = 0; q < MATS; q++) {
                    mma_s8(acc[q][i], w[c][q][0].x, w[c][q][1].x, w[c][q][0].y, w[c][q][1].y, x[c][i].x, x[c][i].y);
                    mma_s8(acc[q][i], w[c][q][0].z, w[c][q][1].z, w[c][q][0].w, w[c][q][1].w, x[c][i].z, x[c][i].w);
                }
    }
    // part[warp][matrix][token][row]: rows of a token side by side, as y stores them
#pragma unroll
    for (int q = 0; q < MATS; q++)
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                part[warp][(q * 8 * MT + 8 * i + 2 * t + (e & 1)) * kRows + g + 8 * (e >> 1)] = acc[q][i][e];
    __syncthreads();
    for (int o = threadIdx.x; o < 8 * MT * kRows; o += kWarps * 32) {
        const int j = m0 + o / kRows, n = n0 + o % kRows;
        if (j >= p.m || n >= p.n) continue;
        int s[MATS] = {};
#pragma unroll
        for (int q = 0; q < MATS; q++)
#pragma unroll
            for (int w = 0; w < kWarps; w++) s[q] += part[w][q * 8 * MT * kRows + o];
        const float sa = p.scale_a[j];
        float v = w8::rescale(s[0], p.scale_0[n], sa);
        if constexpr (MATS == 2) v = w8::gated(v, w8::rescale(s[1], p.scale_1[n], sa), p.act);
        else if (p.bias) v = __fadd_rn(v, p.bias[n]);
        const int64_t at = (int64_t)j * p.n + n;
        if (!q4_in_bounds(at, (int64_t)p.m * p.n, p.status)) continue;
        if (p.out_bf16) static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
        else static_cast<float*>(p.y)[at] = v;
    }
}

// 8 warps a CTA, or 16 where 8 would leave an SM fewer than 16 and k gives each of the 16 a block or more (2048 rows, k 8192,
// one token: 6.2 us with 8 warps)
template <int MT> int launch(const Problem& p, cudaStream_t s)
{
    const dim3 grid((p.n + kRows - 1) / kRows, (p.m + 8 * MT - 1) / (8 * MT));
    if (grid.y > 65535) return Q4_ERR_SHAPE;
    const bool more = (int64_t)grid.x * grid.y <= q4_num_sms() && p.k >= 16 * 128;
    auto go = [&](auto kern, int warps) { return q4_launch_pdl(kern, grid, dim3(32 * warps), 0, s, p); };
    if (p.w1) return more ? go(w8a8_small_kernel<MT, 2, 16>, 16) : go(w8a8_small_kernel<MT, 2, 8>, 8);
    return more ? go(w8a8_small_kernel<MT, 1, 16>, 16) : go(w8a8_small_kernel<MT, 1, 8>, 8);
}

}  // namespace

int w8a8_small_launch(const w8::Problem& p, cudaStream_t s) { return p.m <= 8 ? launch<1>(p, s) : launch<2>(p, s); }
