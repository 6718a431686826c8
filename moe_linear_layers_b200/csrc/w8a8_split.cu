// W8A8 products whose 256 x 256 output tiles would leave most of the GPU idle: few tokens, or few weight rows.
//
// The weights are the MMA's M side here (128 rows a tile; gated: 64 of gate and 64 of up), the tokens its N side (a tile of
// 32 to 256), so that a batch of any size reads the weights once per token tile and pays for no empty rows of M.  A cluster
// of up to 4 CTAs shares a tile: CTA r sums its part of K in its own TMEM, the int32 sums go to its shared memory, and each
// CTA then adds up one slice of the tokens over the cluster (distributed shared memory), rescales and stores it.  Integer sums
// do not depend on the split, so the result is the same for every cluster size, and no workspace is needed.
//
// What bounds it is latency: one TMA ring fill, K / cluster of MMAs, and the exchange.  Measured on B200: 65 x 2048 x 2048
// 5.8 us, 256 x 2048 x 2048 7.1, 128 x 2048 x 8192 9.1, gated 200 x 1024 x 2048 7.1 (the pair kernel: 9.1, 9.5, 22.7, 9.8).
// Warps (12): 0 TMA producer, 1 MMA issuer, 2 TMEM owner, 4-11 from TMEM to shared memory, and all of them in the
// rescale.  Every wait is bounded (Q4_ERR_TIMEOUT).
#include "tc_ptx.cuh"
#include "w8a8_common.cuh"
#include "w8a8_ptx.cuh"

namespace {

using w8::Problem;

constexpr int BM = 128;       // weight rows a tile
constexpr int BK = 128;       // codes of K a block (one swizzled 128-byte row)
constexpr int kMaxStages = 8;
constexpr int kThreads = 384;
constexpr int kRing = 200 * 1024;

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full;
    uint32_t tmem;
    int abort_flag;
};

struct Shape {
    int bn;            // tokens a tile: 32, 64, 128 or 256
    int blocks;        // K blocks a stage
    int stages;
    int splits;        // CTAs a cluster
    int per;           // K blocks a CTA
    int tiles_m;       // token tiles
    int wide;          // rows of y let four outputs be stored at once
};

template <bool GATED>
__global__ void __launch_bounds__(kThreads, 1)
w8a8_split_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w0,
                  const __grid_constant__ CUtensorMap tm_w1, const Problem p, const Shape g)
{
    extern __shared__ __align__(1024) uint8_t smem[];   // (whole 1024-byte swizzle atoms)
    Shared* sh = reinterpret_cast<Shared*>(smem + kRing);
    volatile int* abort_flag = &sh->abort_flag;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int rank = g.splits > 1 ? (int)w8::cluster_rank() : 0;
    const int tile = blockIdx.x / g.splits;
    constexpr int ROWS = GATED ? BM / 2 : BM;   // outputs a tile
    const int m0 = (tile % g.tiles_m) * g.bn, n0 = (tile / g.tiles_m) * ROWS;
    const int kblocks = (p.k + BK - 1) / BK;
    const int kb0 = min(rank * g.per, kblocks), kb1 = min(kb0 + g.per, kblocks);
    const int block_bytes = (BM + g.bn) * BK, stage_bytes = g.blocks * block_bytes;
    if (tc::smem_u32(smem) & 1023u) {           // (never seen: the declared alignment is kept)
        q4_set_status(p.status, Q4_ERR_ALIGN);
        return;
    }

    if (threadIdx.x == 0) {
        for (int i = 0; i < g.stages; i++) {
            tc::mbar_init(&sh->full[i], 1);
            tc::mbar_init(&sh->empty[i], 1);
        }
        tc::mbar_init(&sh->acc_full, 1);
        sh->abort_flag = 0;
        tc::fence_mbar_init();
        tc::tma_prefetch_desc(&tm_x);
        tc::tma_prefetch_desc(&tm_w0);
    }
    if (warp == 2) tc::tmem_alloc(&sh->tmem, (uint32_t)g.bn);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = sh->tmem;
    q4_pdl_start();

    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            for (int kb = kb0, it = 0; kb < kb1; kb += g.blocks, it++) {
                const int s = it % g.stages, nb = min(g.blocks, kb1 - kb);
                if (it >= g.stages && !(ok = tc::mbar_wait(&sh->empty[s], ((it / g.stages) & 1) ^ 1, p.status, abort_flag))) break;
                tc::mbar_arrive_expect_tx(&sh->full[s], nb * block_bytes);
                for (int j = 0; j < nb; j++) {
                    uint8_t* dst = smem + s * stage_bytes + j * block_bytes;
                    tc::tma_load_2d(dst, &tm_w0, &sh->full[s], (kb + j) * BK, n0);
                    if constexpr (GATED) tc::tma_load_2d(dst + ROWS * BK, &tm_w1, &sh->full[s], (kb + j) * BK, n0);
                    tc::tma_load_2d(dst + BM * BK, &tm_x, &sh->full[s], (kb + j) * BK, m0);
                }
            }
            if (!ok) w8::pause_ns(100000000ull);   // given up: let the copies in flight land before the memory is used again
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t idesc = w8::idesc_s8(BM, (uint32_t)g.bn);
        for (int kb = kb0, it = 0; kb < kb1; kb += g.blocks, it++) {
            const int s = it % g.stages, nb = min(g.blocks, kb1 - kb);
            if (!w8::warp_wait(&sh->full[s], (it / g.stages) & 1, p.status, abort_flag)) break;
            tc::fence_after_sync();
            for (int j = 0; j < nb; j++) {
                const uint32_t a = tc::smem_u32(smem + s * stage_bytes + j * block_bytes);
                const uint64_t ad = tc::smem_desc_sw128(a), bd = tc::smem_desc_sw128(a + BM * BK);
#pragma unroll
                for (int i = 0; i < BK / 32; i++)
                    if (lane == 0) w8::mma_i8(tbase, ad + 2 * i, bd + 2 * i, idesc, it > 0 || j > 0 || i > 0);
            }
            if (lane == 0) tc::mma_commit(&sh->empty[s]);
            __syncwarp();
        }
        if (lane == 0) tc::mma_commit(&sh->acc_full);   // (also after a wait that gave up: the MMAs issued so far retire)
        __syncwarp();
    }
    // every warp: the accumulator is complete, and the ring is free
    bool ok = tc::mbar_wait(&sh->acc_full, 0, p.status, nullptr);
    tc::fence_after_sync();
    ok = __syncthreads_and(ok);   // (one answer for every lane: the TMEM reads take whole warps)
    if (warp >= 4 && ok) {
        // TMEM lane = weight row, column = token; sums [token][128 rows] in shared memory.  (A CTA without a part of K has zeros.)
        const int q = warp & 3, half = (warp - 4) >> 2;
        int* st = reinterpret_cast<int*>(smem) + 32 * q + lane;
        for (int c = 32 * half; c < g.bn; c += 64) {
            uint32_t r[32];
            if (kb1 > kb0) {
                tc::tmem_ld32(tbase + ((uint32_t)(32 * q) << 16) + c, r);
                w8::tmem_wait_ld32(r);
            } else {
#pragma unroll
                for (int j = 0; j < 32; j++) r[j] = 0;
            }
#pragma unroll
            for (int j = 0; j < 32; j++) st[(c + j) * BM] = (int)r[j];
        }
    }
    tc::fence_before_sync();
    __syncwarp();
    if (g.splits > 1) w8::cluster_sync();
    else __syncthreads();
    tc::fence_after_sync();

    // this CTA's slice of the tokens: four outputs a thread
    const int slice = g.bn / g.splits, j0 = rank * slice;
    constexpr int QUADS = ROWS / 4;
    const uint32_t base = tc::smem_u32(smem);
    for (int i = threadIdx.x; i < slice * QUADS; i += kThreads) {
        const int j = j0 + i / QUADS, c = 4 * (i % QUADS);
        const int m = m0 + j, n = n0 + c;
        if (m >= p.m || n >= p.n) continue;
        int4 s = make_int4(0, 0, 0, 0), u = s;
        for (int r = 0; r < g.splits; r++) {
            const uint32_t at = base + (uint32_t)(j * BM + c) * 4;
            const int4 a = w8::ld_cluster(at, (uint32_t)r, g.splits > 1);
            s.x += a.x; s.y += a.y; s.z += a.z; s.w += a.w;
            if constexpr (GATED) {
                const int4 b = w8::ld_cluster(at + ROWS * 4, (uint32_t)r, g.splits > 1);
                u.x += b.x; u.y += b.y; u.z += b.z; u.w += b.w;
            }
        }
        const float sa = p.scale_a[m];
        const int si[4] = {s.x, s.y, s.z, s.w}, ui[4] = {u.x, u.y, u.z, u.w};
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int ne = min(n + e, p.n - 1);
            v[e] = w8::rescale(si[e], p.scale_0[ne], sa);
            if constexpr (GATED) v[e] = w8::gated(v[e], w8::rescale(ui[e], p.scale_1[ne], sa), p.act);
            else if (p.bias) v[e] = __fadd_rn(v[e], p.bias[ne]);
        }
        const int64_t at = (int64_t)m * p.n + n;
        if (!q4_in_bounds(min(at + 3, (int64_t)(m + 1) * p.n - 1), (int64_t)p.m * p.n, p.status)) continue;
        if (g.wide) {   // (n and p.n are multiples of 4)
            if (p.out_bf16)
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + at) = make_uint2(w8::bf16_pair(v[0], v[1]), w8::bf16_pair(v[2], v[3]));
            else
                *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++) {
                if (n + e >= p.n) continue;
                if (p.out_bf16) static_cast<__nv_bfloat16*>(p.y)[at + e] = __float2bfloat16_rn(v[e]);
                else static_cast<float*>(p.y)[at + e] = v[e];
            }
        }
    }
    __syncwarp();
    if (g.splits > 1) w8::cluster_sync();   // no CTA leaves while another may still read its sums
    if (warp == 2) tc::tmem_dealloc(tbase, (uint32_t)g.bn);
}

}  // namespace

// bn tokens a tile, splits CTAs a cluster (both powers of two)
int w8a8_split_launch(const Problem& p, int bn, int splits, cudaStream_t s)
{
    const bool gated = p.w1 != nullptr;
    const int rows = gated ? BM / 2 : BM;
    CUtensorMap mx, m0, m1;
    if (!w8::make_code_map(&mx, p.xq, p.k, p.m, bn) || !w8::make_code_map(&m0, p.w0, p.k, p.n, rows) ||
        (gated && !w8::make_code_map(&m1, p.w1, p.k, p.n, rows)))
        return Q4_ERR_CUDA;
    if (!gated) m1 = m0;
    Shape g;
    g.bn = bn;
    g.splits = splits;
    const int kblocks = (p.k + BK - 1) / BK;
    g.per = (kblocks + splits - 1) / splits;
    // A stage costs its waits about 0.25 us whatever its size, so it holds several blocks, and the ring two stages or three.
    g.blocks = bn <= 64 ? 4 : 2;
    g.stages = std::min(kMaxStages, kRing / (g.blocks * (BM + bn) * BK));
    g.tiles_m = (p.m + bn - 1) / bn;
    g.wide = p.n % 4 == 0;
    const int64_t ctas = (int64_t)g.tiles_m * ((p.n + rows - 1) / rows) * splits;
    if (ctas > INT32_MAX) return Q4_ERR_SHAPE;
    constexpr int smem = kRing + (int)sizeof(Shared);
    static_assert(smem <= 227 * 1024 && 256 * BM * 4 <= kRing, "shared memory");
    auto go = [&](auto kern) {
        if (const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) return q4_cuda_status(e);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)ctas);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)splits;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return q4_cuda_status(cudaLaunchKernelEx(&cfg, kern, mx, m0, m1, p, g));
    };
    return gated ? go(w8a8_split_kernel<true>) : go(w8a8_split_kernel<false>);
}
