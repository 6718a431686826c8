// W8A8 products for many tokens: int8 tcgen05 MMAs on CTA pairs.
//
// A pair of CTAs (cluster of 2, cta_group::2) owns a tile of 256 tokens x 256 weight rows: each CTA brings its own 128
// token rows and 128 of the weight rows into shared memory (TMA, 128-byte swizzle, K-major), the pair's
// MMA (M 256, N 256, K 32) reads both halves, and each CTA's TMEM receives its 128 token rows x 256 int32 sums.
// Per 128 codes of K a CTA thus loads 32 KB for 4 MMAs of 128 cycles (64 bytes a cycle; a lone CTA with a 128 x 256
// tile would need 96).  Gated: the first CTA's weight rows are the gate's, the second's the same rows of up, so a
// thread finds a token's g and u in columns c and 128 + c of its TMEM lane and h needs no exchange.
//
// The whole sum over K stays in the int32 accumulators (exact), so the epilogue touches each output once.
// Two accumulators (2 x 256 TMEM columns): the epilogue of one tile runs under the MMAs of the next.  Persistent: one
// pair per two SMs walks the tiles, tokens fastest, so that concurrent pairs share weight rows in L2.
//
// Warps (12): 0 TMA producer, 1 MMA issuer (leader CTA only), 2 TMEM owner, 4-11 epilogue (two warps per TMEM lane
// quarter, each half of the columns).  Every wait is bounded (Q4_ERR_TIMEOUT).
//
// Measured on B200: 4096 x 2048 x 8192 in 51 to 56 us (2.45 to 2.67 PTOP/s), 4096 x 8192 x 2048 in 56 us, gated 98 to 108 us
// (2.55 to 2.8 PTOP/s), the spread being the clock, which falls from 1965 to about 1.5 GHz at the power cap; tensor pipe 71 %
// (gated) and 81 % active.  Without loads the gated problem takes 105 us to this kernel's 123 with 128 codes a stage; with 256
// codes a stage and neither loads nor epilogue 75 us: what is left is the drain at each of the issuer's waits.
#include "tc_ptx.cuh"
#include "w8a8_common.cuh"
#include "w8a8_ptx.cuh"

namespace {

using w8::Problem;

constexpr int BM = 128;                 // token rows a CTA
constexpr int BNC = 128;                // weight rows a CTA loads
constexpr int BN = 2 * BNC;             // accumulator columns
constexpr int BK = 128;                 // codes of K a block (one swizzled 128-byte row)
constexpr int kBlocks = 2;              // blocks a stage
constexpr int kStages = 3;
constexpr int kBlockBytes = (BM + BNC) * BK;
constexpr int kStageBytes = kBlocks * kBlockBytes;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kStageOut = 4096;         // output staging bytes an epilogue warp: 32 rows x 128 bytes

struct Shared {
    uint64_t full[kStages], empty[kStages];   // full: the leader's (both CTAs' copies); empty: each CTA's
    uint64_t acc_full[2], acc_empty[2];       // acc_full: each CTA's; acc_empty: the leader's (both CTAs' epilogues)
    uint64_t done;
    uint32_t tmem;
    int abort_flag;
    alignas(16) float sw[BN], bias[BN];       // the tile's channel scales (gated: gate's, up's) and biases
};

constexpr int kSmem = kStages * kStageBytes + kEpiWarps * kStageOut + (int)sizeof(Shared);
static_assert(kSmem <= 227 * 1024, "shared memory");

struct Grid {
    int tiles_m, tiles;
    int tma_out;    // rows of y start on 16 bytes: stored by TMA
};

template <bool GATED, bool OUT32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
w8a8_gemm_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w0,
                 const __grid_constant__ CUtensorMap tm_w1, const __grid_constant__ CUtensorMap tm_y, const Problem p,
                 const Grid g)
{
    extern __shared__ __align__(1024) uint8_t smem[];   // (whole 1024-byte swizzle atoms)
    if (tc::smem_u32(smem) & 1023u) {                   // (never seen: the declared alignment is kept)
        q4_set_status(p.status, Q4_ERR_ALIGN);
        return;
    }
    uint8_t* out_stage = smem + kStages * kStageBytes;
    Shared* sh = reinterpret_cast<Shared*>(out_stage + kEpiWarps * kStageOut);
    volatile int* abort_flag = &sh->abort_flag;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t rank = w8::cluster_rank();
    const int kblocks = (p.k + BK - 1) / BK, kstages = (kblocks + kBlocks - 1) / kBlocks;
    const int first = blockIdx.x / 2, step = gridDim.x / 2;
    constexpr int ROWS = GATED ? BNC : BN;   // weight rows (of each matrix) a tile covers

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; i++) {
            tc::mbar_init(&sh->full[i], 1);
            tc::mbar_init(&sh->empty[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            tc::mbar_init(&sh->acc_full[i], 1);
            tc::mbar_init(&sh->acc_empty[i], 2 * kEpiWarps);
        }
        tc::mbar_init(&sh->done, 1);
        sh->abort_flag = 0;
        tc::fence_mbar_init();
        tc::tma_prefetch_desc(&tm_x);
        tc::tma_prefetch_desc(&tm_w0);
    }
    if (warp == 2) w8::tmem_alloc_pair(&sh->tmem, 512);
    tc::fence_before_sync();
    __syncthreads();
    w8::cluster_sync();       // both CTAs' barriers are initialised before either is signalled
    tc::fence_after_sync();
    const uint32_t tbase = sh->tmem;
    q4_pdl_start();

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = first; t < g.tiles && ok; t += step) {
                const int m0 = (t % g.tiles_m) * (2 * BM) + (int)rank * BM;
                const int n0 = (t / g.tiles_m) * ROWS + (GATED ? 0 : (int)rank * BNC);
                const CUtensorMap* mw = GATED && rank ? &tm_w1 : &tm_w0;
                for (int ks = 0; ks < kstages; ks++, it++) {
                    const int s = it % kStages;
                    if (!(ok = tc::mbar_wait(&sh->empty[s], ((it / kStages) & 1) ^ 1, p.status, abort_flag))) break;
                    const int nb = min(kBlocks, kblocks - ks * kBlocks);
                    if (rank == 0) tc::mbar_arrive_expect_tx(&sh->full[s], 2 * nb * kBlockBytes);
                    const uint32_t bar = w8::map_to_rank(&sh->full[s], 0);
                    for (int j = 0; j < nb; j++) {
                        uint8_t* dst = smem + s * kStageBytes + j * kBlockBytes;
                        w8::tma_load_pair(dst, &tm_x, bar, (ks * kBlocks + j) * BK, m0);
                        w8::tma_load_pair(dst + BM * BK, mw, bar, (ks * kBlocks + j) * BK, n0);
                    }
                }
            }
            if (!ok) w8::pause_ns(100000000ull);   // given up: let the copies in flight land before the CTA leaves
        }
    } else if (warp == 1) {
        // The whole warp runs this loop and lane 0's predicate is on the instructions alone: measured 340 ns per four
        // MMAs against 390 with the loop inside a branch of lane 0.  A barrier wait costs the issuer another ~130 ns (the
        // MMAs before it drain), hence eight MMAs (two blocks of K) a wait.
        if (rank == 0) {
            constexpr uint32_t idesc = w8::idesc_s8(2 * BM, BN);
            uint32_t it = 0, tl = 0;
            bool ok = true;
            for (int t = first; t < g.tiles && ok; t += step, tl++) {
                const uint32_t b = tl & 1;
                if (!(ok = w8::warp_wait(&sh->acc_empty[b], ((tl >> 1) & 1) ^ 1, p.status, abort_flag))) break;
                tc::fence_after_sync();
                for (int ks = 0; ks < kstages; ks++, it++) {
                    const int s = it % kStages;
                    if (!(ok = w8::warp_wait(&sh->full[s], (it / kStages) & 1, p.status, abort_flag))) break;
                    tc::fence_after_sync();
                    const int nb = min(kBlocks, kblocks - ks * kBlocks);
#pragma unroll
                    for (int j = 0; j < kBlocks; j++) {
                        if (j >= nb) continue;
                        const uint32_t a = tc::smem_u32(smem + s * kStageBytes + j * kBlockBytes);
                        const uint64_t ad = tc::smem_desc_sw128(a), bd = tc::smem_desc_sw128(a + BM * BK);
#pragma unroll
                        for (int i = 0; i < BK / 32; i++)
                            if (lane == 0) w8::mma_i8_pair(tbase + b * BN, ad + 2 * i, bd + 2 * i, idesc, ks > 0 || j > 0 || i > 0);
                    }
                    if (lane == 0) w8::commit_pair(&sh->empty[s]);
                    __syncwarp();
                }
                if (ok && lane == 0) w8::commit_pair(&sh->acc_full[b]);
                __syncwarp();
            }
            // every MMA issued has retired before TMEM is freed (a wait that does not honour the abort flag: the operands
            // are in place, so it ends)
            if (lane == 0) w8::commit_one_of_pair(&sh->done);
            __syncwarp();
            tc::mbar_wait(&sh->done, 0, p.status, nullptr);
            __syncwarp();
        }
    } else if (warp >= 4) {
        const int e = warp - 4, q = warp & 3, half = e >> 2;
        uint8_t* stage = out_stage + e * kStageOut;
        uint32_t tl = 0;
        bool ok = true;   // (a warp that gave up still meets the others at the barriers)
        // a tile's channel scales and biases, one a thread (256 epilogue threads, 256 columns), and its lane's token scale come
        // a tile ahead (4096 x 8192 x 512: 28.8 -> 28.1 us; the outputs alone, 67 MB, take 20 us at the rate of writes)
        float next_sw = 0.0f, next_bias = 0.0f, next_sa = 0.0f;
        auto fetch = [&](int t) {
            if (t >= g.tiles) return;
            const int m = (t % g.tiles_m) * (2 * BM) + (int)rank * BM + 32 * q + lane;
            const int c = threadIdx.x - 128, n = (t / g.tiles_m) * ROWS + (GATED ? c % BNC : c);
            next_sw = n < p.n ? (GATED && c >= BNC ? p.scale_1 : p.scale_0)[n] : 0.0f;
            if (!GATED) next_bias = p.bias && n < p.n ? p.bias[n] : 0.0f;
            next_sa = m < p.m ? p.scale_a[m] : 0.0f;
        };
        fetch(first);
        for (int t = first; t < g.tiles; t += step, tl++) {
            const uint32_t b = tl & 1;
            const int m0 = (t % g.tiles_m) * (2 * BM) + (int)rank * BM + 32 * q;
            const int n0 = (t / g.tiles_m) * ROWS;
            w8::named_barrier(1, 32 * kEpiWarps);   // the last tile's scales are no longer read
            sh->sw[threadIdx.x - 128] = next_sw;
            if (!GATED) sh->bias[threadIdx.x - 128] = next_bias;
            const float sa = next_sa;
            w8::named_barrier(1, 32 * kEpiWarps);
            fetch(t + step);
            ok = ok && w8::warp_wait(&sh->acc_full[b], (tl >> 1) & 1, p.status, abort_flag);
            if (!ok) continue;
            tc::fence_after_sync();
            const uint32_t tcol = tbase + ((uint32_t)(32 * q) << 16) + b * BN;
            constexpr int CHUNKS = GATED ? 2 : 4;
            constexpr int PER = OUT32 ? 1 : 2;                    // chunks a box: 128-byte rows
#pragma unroll 1
            for (int c0 = 0; c0 < CHUNKS; c0 += PER) {
#pragma unroll
                for (int c1 = 0; c1 < PER; c1++) {
                    const int c = c0 + c1;
                    const int col = half * (32 * CHUNKS) + 32 * c;   // the first of 32 output columns of the tile
                    uint32_t r[32], u[32];
                    tc::tmem_ld32(tcol + col, r);
                    if constexpr (GATED) tc::tmem_ld32(tcol + BNC + col, u);
                    w8::tmem_wait_ld32(r);
                    if constexpr (GATED) w8::tmem_wait_ld32(u);
                    if (c == CHUNKS - 1) {   // this warp's last read: the accumulator may be overwritten
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) w8::arrive_remote(w8::map_to_rank(&sh->acc_empty[b], 0));
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 s0 = *reinterpret_cast<const float4*>(sh->sw + col + j);
                        const float4 s1 = *reinterpret_cast<const float4*>(GATED ? sh->sw + BNC + col + j : sh->bias + col + j);
                        const float f0[4] = {s0.x, s0.y, s0.z, s0.w}, f1[4] = {s1.x, s1.y, s1.z, s1.w};
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            float v = w8::rescale((int)r[j + i], f0[i], sa);
                            if constexpr (GATED) v = w8::gated(v, w8::rescale((int)u[j + i], f1[i], sa), p.act);
                            else if (p.bias) v = __fadd_rn(v, f1[i]);
                            r[j + i] = __float_as_uint(v);
                        }
                    }
                    // 32 rows into this warp's staging box (16-byte pieces in the TMA swizzle's places)
                    if (c1 == 0) {
                        if (lane == 0) w8::bulk_wait_read<0>();   // the copy that last read it
                        __syncwarp();
                    }
                    if constexpr (OUT32) {
#pragma unroll
                        for (int k = 0; k < 8; k++)
                            *reinterpret_cast<uint4*>(stage + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                                make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            uint32_t o[4];
#pragma unroll
                            for (int j = 0; j < 4; j++)
                                o[j] = w8::bf16_pair(__uint_as_float(r[8 * k + 2 * j]), __uint_as_float(r[8 * k + 2 * j + 1]));
                            *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * c1 + k) ^ (lane & 7)) << 4)) =
                                make_uint4(o[0], o[1], o[2], o[3]);
                        }
                    }
                }
                const int nc = n0 + half * (32 * CHUNKS) + 32 * c0;
                constexpr int W = 32 * PER;             // columns of the box
                const bool any = nc < p.n && m0 < p.m;   // (warp-uniform)
                if (any && g.tma_out) {
                    w8::fence_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        w8::tma_store(&tm_y, stage, nc, m0);
                        w8::bulk_commit();
                    }
                } else if (any) {
                    __syncwarp();
                    // rows that do not start on 16 bytes: a warp stores 32 columns of a row at a time, or 32 pairs of bf16
                    // columns where the rows start on 4 bytes
                    constexpr int ES = OUT32 ? 4 : 2;
                    const int rows = min(32, p.m - m0);
                    auto columns = [&](int x, auto WORD) {
                        using Word = decltype(WORD);
                        const int piece = x * ES >> 4, inner = x * ES & 15;
                        uint8_t* dst = static_cast<uint8_t*>(p.y) + ((int64_t)m0 * p.n + nc + x) * ES;
#pragma unroll 8
                        for (int i = 0; i < rows; i++, dst += (int64_t)p.n * ES) {
                            if (!q4_in_bounds((int64_t)(m0 + i) * p.n + nc + x + (int)sizeof(Word) / ES - 1, (int64_t)p.m * p.n, p.status)) continue;
                            *reinterpret_cast<Word*>(dst) = *reinterpret_cast<const Word*>(stage + i * 128 + ((piece ^ (i & 7)) << 4) + inner);
                        }
                    };
                    if constexpr (OUT32) {
                        if (nc + lane < p.n) columns(lane, uint32_t());
                    } else if (p.n % 2 == 0) {
                        if (nc + 2 * lane < p.n) columns(2 * lane, uint32_t());
                    } else {
                        for (int x = lane; x < W; x += 32)
                            if (nc + x < p.n) columns(x, uint16_t());
                    }
                }
                __syncwarp();
            }
        }
        if (lane == 0) w8::bulk_wait_all();   // the output is written before the grid can count as complete
    }
    tc::fence_before_sync();
    __syncwarp();
    w8::cluster_sync();       // no CTA leaves while its peer may still signal or read it
    tc::fence_after_sync();
    if (warp == 2) w8::tmem_dealloc_pair(tbase, 512);
}

}  // namespace

int w8a8_gemm_launch(const Problem& p, cudaStream_t s)
{
    const bool gated = p.w1 != nullptr;
    CUtensorMap mx, m0, m1, my;
    if (!w8::make_code_map(&mx, p.xq, p.k, p.m, BM) || !w8::make_code_map(&m0, p.w0, p.k, p.n, BNC) ||
        (gated && !w8::make_code_map(&m1, p.w1, p.k, p.n, BNC)))
        return Q4_ERR_CUDA;
    if (!gated) m1 = m0;
    Grid g;
    g.tiles_m = (p.m + 2 * BM - 1) / (2 * BM);
    const int rows = gated ? BNC : BN;
    const int64_t tiles = (int64_t)g.tiles_m * ((p.n + rows - 1) / rows);
    if (tiles > INT32_MAX) return Q4_ERR_SHAPE;
    g.tiles = (int)tiles;
    const int es = p.out_bf16 ? 2 : 4;
    g.tma_out = ((int64_t)p.n * es) % 16 == 0;
    if (g.tma_out) {
        if (!w8::make_out_map(&my, p.y, p.n, p.m, p.out_bf16)) return Q4_ERR_CUDA;
    } else {
        my = mx;
    }
    const int pairs = (int)std::min<int64_t>(tiles, q4_num_sms() / 2);
    auto go = [&](auto kern) {
        if (const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) return q4_cuda_status(e);
        return q4_launch_pdl(kern, dim3(2 * pairs), dim3(kThreads), kSmem, s, mx, m0, m1, my, p, g);
    };
    if (gated) return p.out_bf16 ? go(w8a8_gemm_kernel<true, false>) : go(w8a8_gemm_kernel<true, true>);
    return p.out_bf16 ? go(w8a8_gemm_kernel<false, false>) : go(w8a8_gemm_kernel<false, true>);
}
