// q4k_experts_gemm.cu -- the experts' packed products for many rows an expert, on
// the 5th-generation tensor cores: each expert's Q4_K matrix (or its gate and up
// matrices) with its own rows of x.
//
// Y^T = W X^T as in the dense GEMM: the MMA's A operand is 128 weight rows,
// dequantised to bf16 in TMEM, its B operand up to 192 rows of x in shared memory,
// the accumulator 128 TMEM lanes x the rows of x. A unit is (expert, rows of x,
// two tiles of 128 weight rows): 256 rows of the matrix, or of a gated product 128
// of gate and 128 of up, so that the two factors of an output lie in the same lane
// at the end. The rows of an expert are cut into tiles of equal height, and a
// tile's MMAs are as wide as the tile (a multiple of 16).
//
// Why two tiles, and A in TMEM: shared memory moves 128 bytes a cycle, and an MMA of
// 128 rows at full rate reads its B operand at half of that; x coming in from L2
// for one tile takes the other half, and the A operand through shared memory
// (written, then read) more than is left. With A in TMEM and x read by two tiles,
// what is left carries the packed words. And why two issuing warps, one a tile: the
// wait before a step and the commit behind it hold a warp some 400 cycles, the four
// MMAs of a step 2 cycles a row of x, so one warp alone leaves the tensor cores
// idle below 200 rows.
//
// A block stays on its SM and takes every gridDim-th unit; its warps run ahead
// of one another through rings, from one unit into the next:
//   warp 0       W producer: {144 B, 128 rows} of packed words per tile and 256 k (TMA)
//   warps 1, 2   MMA issuers, one a tile
//   warp 3       X producer: the tile's rows x 64 k (TMA, 128-byte swizzle)
//   warps 4..11  the end of a unit: TMEM -> registers -> (silu(g) u) -> bf16 -> Y, four
//                warps with a tile each, or with half of a gated unit's rows of x
//   warps 12..27 dequantisers, four groups of 128 threads: two a tile, each with every
//                other 64 k, a thread with a weight row of them and 32 columns of TMEM
// All waits are bounded (see mbar_wait).
//
// 4096 tokens to 8 of 128 experts, gated 768 x 2048: 152 us, 1.35 PFLOP/s; 2048 tokens to 4 of 16,
// 4096 x 2048: 98 us, 1.40 PFLOP/s (70 and 73 % of cuBLAS's rate; tensor core busy 67 and 71 %,
// dequantisers' issue slots 67 %). Over many calls the power cap takes a tenth.
#include <cuda_bf16.h>

#include <type_traits>

#include "q4k_device.cuh"
#include "q4k_experts.h"
#include "q4k_serve.h"

namespace q4k {

constexpr int kEgBM = 128;                    // weight rows of a tile
constexpr int kEgBN = 192;                    // rows of x of a unit at most
constexpr int kEgStep = 64;                   // k of a step
constexpr int kEgXStages = 4, kEgWStages = 3;  // W stages of each tile
constexpr int kEgXStage = kEgBN * 128;
constexpr int kEgWStage = kEgBM * kBlockBytes;
constexpr int kEgEpiWarp = 4, kEgDeqWarp = 12, kEgDeqWarps = 16;
constexpr int kEgThreads = 32 * (kEgDeqWarp + kEgDeqWarps);
constexpr int kEgOffW = kEgXStages * kEgXStage;
constexpr int kEgOffBar = kEgOffW + 2 * kEgWStages * kEgWStage;
// w_full[2][W], w_empty[2][W], x_full, x_empty, a_full[2][2], a_empty[2][2], acc_full[2],
// acc_empty[2], end
constexpr int kEgBars = 4 * kEgWStages + 2 * kEgXStages + 8 + 5;
constexpr int kEgOffTmem = kEgOffBar + 8 * kEgBars;
constexpr int kEgOffTab = (kEgOffTmem + 8 + 15) / 16 * 16;
// the two accumulators, then two stages of A of 32 columns for each tile
constexpr uint32_t kEgTmemCols = 512, kEgTmemA = 2 * kEgBN;
static_assert(kEgTmemA + 128 <= kEgTmemCols, "TMEM");

__host__ __device__ constexpr int eg_smem(int experts) { return kEgOffTab + 8 * (experts + 1) + 1024; }
static_assert(eg_smem(kMaxExperts) <= 232448, "shared memory per CTA");

struct XMaps {
    CUtensorMap box[kEgBN / 32];  // boxes of 32, 64, .. rows x 64 k
};

// The scale and min of 32 weights as bf16 pairs for dequant8: w = d1 q - m1 =
// d1 (q - c) + r with c the 16th of a code nearest to w = 0 and r = c d1 - m1, d1 the sum of two bf16.
// (16 (q - c) has 8 bits, so q - c is exact in bf16; with whole codes for c, r is up to 16 times as large, and
// its two roundings show.)
struct EgScale {
    __nv_bfloat162 dh, dl, r, c;
};
// unit: the q - c of dequant8 come as this much of themselves, 2^-6 for low nibbles, 2^-2 for high ones
__device__ __forceinline__ EgScale eg_scale(float d1, float m1, float unit) {
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(d1));
    const float c = fminf(fmaxf(rintf(m1 * inv * 16.f), 0.f), 255.f);  // 16ths (0 where the quotient is not a number)
    const float d = d1 * (1.f / unit);
    EgScale s;
    s.dh = __float2bfloat162_rn(d);
    s.dl = __float2bfloat162_rn(d - __low2float(s.dh));
    s.r = __float2bfloat162_rn(fmaf(c, d1 * 0.0625f, -m1));
    s.c = __float2bfloat162_rn(-c * (unit * 0.0625f));
    return s;
}

// The eight weights of a qs word: o[0], o[1] its low nibbles, o[2], o[3] its high
// ones, two bf16 each. A byte spread to 16 bits and masked is a bf16 number as it
// stands, q 2^-133 or 16 q 2^-133 (bit patterns below 256 count on evenly); one FMA makes
// (q - c) 2^-6 or 2^-2 of it, exactly, and w = (q - c) dh + ((q - c) dl + r) takes two more: per
// weight 0.75 integer instructions, at half the rate of the FMAs' 1.5 (masks, fp32
// FMAs and conversions take 1.75, and that pipe bound the kernel: 4096 tokens to 8 of 128
// experts, gated 196 us, 182 this way). Roundings: r, the inner FMA (about |r| too) and w, and
// what is left of d1 (2^-16): off by 2^-8 (|w| + 2 |r|) to within 2 %. |r| <= |d1| / 32 where the weight 0
// lies among the codes (0 <= m1 <= 15.96 d1); elsewhere c is at an end and |r| <= |w|.
__device__ __forceinline__ void dequant8(uint32_t w, const EgScale& lo, const EgScale& hi, uint32_t* o) {
    const __nv_bfloat162 up = __float2bfloat162_rn(exp2i(127));
    const uint32_t p[2] = {__byte_perm(w, 0, 0x4140), __byte_perm(w, 0, 0x4342)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t a = p[i] & 0x000F000Fu, b = p[i] & 0x00F000F0u;
        const __nv_bfloat162 x = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&a), up, lo.c);
        const __nv_bfloat162 y = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&b), up, hi.c);
        const __nv_bfloat162 u = __hfma2(x, lo.dh, __hfma2(x, lo.dl, lo.r)), v = __hfma2(y, hi.dh, __hfma2(y, hi.dl, hi.r));
        o[i] = *reinterpret_cast<const uint32_t*>(&u);
        o[2 + i] = *reinterpret_cast<const uint32_t*>(&v);
    }
}

// After a timeout the barriers tell nothing: a while for the copies that are still landing.
__device__ __forceinline__ void eg_drain() {
    const unsigned long long t0 = globaltimer();
    while (globaltimer() - t0 < kDrainLimitNs) {
    }
}

template <bool kGated>
__global__ void __launch_bounds__(kEgThreads, 1)
    q4k_experts_gemm_kernel(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapW2,
                            const __grid_constant__ XMaps mapX, const ExpertRows rows, int N, int K, uint16_t* Y,
                            unsigned int* err) {
    constexpr int kCols = kGated ? kEgBM : 2 * kEgBM;  // output columns of a unit
    extern __shared__ uint8_t eg_raw[];
    const uint32_t raw = smem_u32(eg_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t* smem = eg_raw + pad;
    const uint32_t sbase = raw + pad;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bwf = sbase + kEgOffBar, bwe = bwf + 16 * kEgWStages, bxf = bwe + 16 * kEgWStages,
                   bxe = bxf + 8 * kEgXStages, baf = bxe + 8 * kEgXStages, bae = baf + 32, bcf = bae + 32, bce = bcf + 16,
                   bend = bce + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kEgOffTmem);
    int* starts = reinterpret_cast<int*>(smem + kEgOffTab);
    int* tiles = starts + rows.experts + 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * kEgWStages; ++i) mbar_init(bwf + 8 * i, 1), mbar_init(bwe + 8 * i, kEgDeqWarps / 2);
        for (int i = 0; i < kEgXStages; ++i) mbar_init(bxf + 8 * i, 1), mbar_init(bxe + 8 * i, 2);
        for (int i = 0; i < 4; ++i) mbar_init(baf + 8 * i, kEgDeqWarps / 4), mbar_init(bae + 8 * i, 1);
        for (int i = 0; i < 2; ++i) mbar_init(bcf + 8 * i, 1), mbar_init(bce + 8 * i, kGated ? 8 : 4);
        mbar_init(bend, 2);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), kEgTmemCols);
        tmem_relinquish();
    }
    pdl_wait();
    for (int e = threadIdx.x; e <= rows.experts; e += blockDim.x) starts[e] = min(max(rows.starts[e], 0), rows.pairs);
    if (threadIdx.x == 0) tmem_slot[1] = 0u;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // only now that this block has its TMEM: a later kernel's block beside it could
    // take what it still needs, and wait for it
    if (threadIdx.x == 0) pdl_launch_dependents();
    if (warp == 0) expert_tiles<kEgBN>(starts, tiles, rows.experts, lane);
    __syncthreads();
    const uint32_t tmem = *tmem_slot;
    const int ntiles = (N + kCols - 1) / kCols;
    const int64_t units = static_cast<int64_t>(tiles[rows.experts]) * ntiles;
    const int KB = K / kBlockWeights;

    // unit u: (expert, row tile, columns), the columns of a row tile side by side, so
    // that its rows of x come from memory once
    struct Unit {
        int e, n0, p0, rows;
    };
    auto unit_of = [&](int64_t u) {
        const int tile = static_cast<int>(u / ntiles);
        Unit r;
        r.e = expert_of(tiles, rows.experts, tile);
        r.n0 = static_cast<int>(u % ntiles) * kCols;
        const int all = starts[r.e + 1] - starts[r.e], mt = tiles[r.e + 1] - tiles[r.e];
        const int h = ((all + mt - 1) / mt + 15) & ~15;  // <= kEgBN
        const int off = (tile - tiles[r.e]) * h;
        r.p0 = starts[r.e] + off;
        r.rows = max(0, min(h, all - off));
        return r;
    };

    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&mapW);
            // (kept in L2: the words of an expert with several row tiles are read for each; 155 us, 159)
            const uint64_t pol = policy_evict_last();
            uint32_t it = 0;
            bool ok = true;
            for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const Unit w = unit_of(u);
                for (int sb = 0; sb < KB && ok; ++sb, ++it) {
#pragma unroll 1
                    for (int tile = 0; tile < 2; ++tile) {
                        const uint32_t s = tile * kEgWStages + it % kEgWStages;
                        if (!mbar_wait_idle(bwe + 8 * s, ((it / kEgWStages) & 1) ^ 1, err)) { ok = false; break; }
                        mbar_arrive_expect_tx(bwf + 8 * s, kEgWStage);
                        const uint32_t dst = sbase + kEgOffW + s * kEgWStage;
                        const int row = w.e * N + w.n0 + (kGated ? 0 : tile * kEgBM);
                        tma_load_2d_hint(dst, kGated && tile == 1 ? &mapW2 : &mapW, sb * kBlockBytes, row, bwf + 8 * s, pol);
                    }
                }
            }
            if (!ok) eg_drain();
        }
        __syncwarp();
    } else if (warp == 3) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_last();
            uint32_t it = 0;
            bool ok = true;
            for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const Unit w = unit_of(u);
                const int q = (max(w.rows, 1) - 1) / 32;  // a box of 32 (q + 1) rows
                const uint32_t bytes = 32u * 128u * (q + 1);
                for (int ks = 0; ks < 4 * KB; ++ks, ++it) {
                    const uint32_t s = it % kEgXStages;
                    if (!mbar_wait_idle(bxe + 8 * s, ((it / kEgXStages) & 1) ^ 1, err)) { ok = false; break; }
                    mbar_arrive_expect_tx(bxf + 8 * s, bytes);
                    tma_load_2d_hint(sbase + s * kEgXStage, &mapX.box[q], ks * kEgStep, w.p0, bxf + 8 * s, pol);
                }
            }
            if (!ok) eg_drain();
        }
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        // a copy of the loop each: what depends on the tile is a constant there
        auto issue = [&](auto which) {
            constexpr int tile = decltype(which)::value;
            constexpr uint32_t d = tile * kEgBN, a_tmem = kEgTmemA + 64 * tile;  // (the allocation is all of TMEM: from 0)
            uint32_t it = 0, n = 0;  // super-blocks, units
            bool ok = true;
            for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x, ++n) {
                const Unit w = unit_of(u);
                const uint32_t idesc = idesc_bf16_f32(kEgBM, max(16, (w.rows + 15) & ~15));
                ok = __all_sync(0xffffffffu, mbar_wait_idle(bce + 8 * tile, (n & 1) ^ 1, err));
                for (int sb = 0; sb < KB && ok; ++sb, ++it) {
                    // the four steps of a super-block: with as many X stages, and two of A, every address is a constant
                    static_assert(kEgXStages == 4, "steps of a super-block");
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        ok = ok && __all_sync(0xffffffffu, mbar_wait_idle(bxf + 8 * c, it & 1, err) &&
                                                               mbar_wait_idle(baf + 8 * (2 * tile + (c & 1)), c >> 1, err));
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t b0 = sw128_desc(sbase + c * kEgXStage);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                tc_mma_bf16_ts(d, a_tmem + 32 * (c & 1) + 8 * kk, b0 + 2 * kk, idesc, c != 0 || kk != 0 || sb != 0);
                            tc_commit(bae + 8 * (2 * tile + (c & 1)));
                            tc_commit(bxe + 8 * c);
                            if (c == 3 && sb == KB - 1) tc_commit(bcf + 8 * tile);
                        }
                        __syncwarp();
                    }
                }
            }
        };
        if (warp == 1) issue(std::integral_constant<int, 0>{});
        else issue(std::integral_constant<int, 1>{});
        if (elect_one()) tc_commit(bend);
        __syncwarp();
    } else if (warp >= kEgDeqWarp) {
        const int t = threadIdx.x - 32 * kEgDeqWarp;
        const int group = t >> 7, tile = group & 1, half = group >> 1;  // chunks half and half + 2 of each super-block
        const int r = t & (kEgBM - 1);  // the weight row of this thread and its TMEM lane
        const uint32_t a_tmem = tmem + kEgTmemA + 64 * tile + 32 * half + (static_cast<uint32_t>(r & ~31) << 16);
        const uint32_t bfull = baf + 8 * (2 * tile + half), bfree = bae + 8 * (2 * tile + half);
        const int sh = 16 * half;
        // 0, read from shared memory so that the compiler cannot see through the
        // dependence that is built from it below
        const uint32_t zero = *reinterpret_cast<volatile uint32_t*>(tmem_slot + 1);
        uint32_t it = 0;
        bool ok = true;
        for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
            for (int sb = 0; sb < KB && ok; ++sb, ++it) {
                const uint32_t s = tile * kEgWStages + it % kEgWStages;
                if (!__all_sync(0xffffffffu, mbar_wait_idle(bwf + 8 * s, (it / kEgWStages) & 1, err))) { ok = false; break; }
                const uint8_t* P = smem + kEgOffW + s * kEgWStage + r * kBlockBytes;
                const uint4 hd = *reinterpret_cast<const uint4*>(P);
                uint4 q[2][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    q[i][0] = *reinterpret_cast<const uint4*>(P + 16 + 32 * (half + 2 * i));
                    q[i][1] = *reinterpret_cast<const uint4*>(P + 32 + 32 * (half + 2 * i));
                }
                // the stage is given back once every lane has its words: the vote
                // needs all of them, so the arrival cannot come before the loads
                const unsigned all = __ballot_sync(0xffffffffu, (hd.x | q[0][0].x | q[0][1].x | q[1][0].x | q[1][1].x) != 0u);
                if (lane == 0) mbar_arrive(bwe + 8 * s + (all & zero));
                const float dd = half_lo(hd.x), dmin = half_hi(hd.x);
                const uint32_t s0 = hd.y >> sh, s1 = hd.z >> sh, s2 = hd.w >> sh;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // the two scales and mins of the chunk's sub-blocks, a byte each
                    const uint32_t sc = i == 0 ? s0 & 0x3F3Fu : (s2 & 0x0F0Fu) | ((s0 >> 2) & 0x3030u);
                    const uint32_t mn = i == 0 ? s1 & 0x3F3Fu : ((s2 >> 4) & 0x0F0Fu) | ((s1 >> 2) & 0x3030u);
                    const uint32_t qw[8] = {q[i][0].x, q[i][0].y, q[i][0].z, q[i][0].w, q[i][1].x, q[i][1].y, q[i][1].z, q[i][1].w};
                    uint32_t o[32];  // the row's 64 k, two to a column
                    const EgScale lo = eg_scale(dd * byte_to_float(sc, 0), dmin * byte_to_float(mn, 0), 0x1p-6f);
                    const EgScale hi = eg_scale(dd * byte_to_float(sc, 1), dmin * byte_to_float(mn, 1), 0x1p-2f);
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        uint32_t w[4];
                        dequant8(qw[v], lo, hi, w);
                        o[2 * v] = w[0];
                        o[2 * v + 1] = w[1];
                        o[16 + 2 * v] = w[2];
                        o[16 + 2 * v + 1] = w[3];
                    }
                    if (!__all_sync(0xffffffffu, mbar_wait_idle(bfree, (i & 1) ^ 1, err))) { ok = false; break; }
                    tc_fence_after();
                    tmem_st_32x32b_x32(a_tmem, o);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bfull);
                }
            }
        }
    } else if (warp >= kEgEpiWarp) {
        const int q = warp & 3, part = (warp - kEgEpiWarp) >> 2;
        uint32_t n = 0;
        bool ok = true;
        for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x, ++n) {
            const Unit w = unit_of(u);
            const uint32_t acc = tmem + (static_cast<uint32_t>(32 * q) << 16), step = 2u * static_cast<uint32_t>(N);
            uint8_t* base = reinterpret_cast<uint8_t*>(Y + static_cast<int64_t>(w.p0) * N + w.n0 + 32 * q + lane);
            // 16 rows of x at a time, from row c0 on; `left` of them have an output
            auto store = [&](uint8_t* y, const float (&v)[16], int left) {
                if (left >= 16) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        *reinterpret_cast<uint16_t*>(y + static_cast<uint64_t>(step) * j) = __bfloat16_as_ushort(__float2bfloat16_rn(v[j]));
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (j < left) *reinterpret_cast<uint16_t*>(y + static_cast<uint64_t>(step) * j) = __bfloat16_as_ushort(__float2bfloat16_rn(v[j]));
                }
            };
            if (kGated) {
                ok = __all_sync(0xffffffffu, mbar_wait_idle(bcf, n & 1, err) && mbar_wait_idle(bcf + 8, n & 1, err));
                if (!ok) break;
                tc_fence_after();
                const int rows_out = w.n0 + 32 * q + lane < N ? w.rows : 0;
                for (int c0 = 16 * part; c0 < w.rows; c0 += 32) {
                    uint32_t g[16], up[16];
                    tmem_ld_32x32b(acc + c0, g);
                    tmem_ld_32x32b(acc + kEgBN + c0, up);
                    tmem_ld_wait();
                    float v[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = silu(__uint_as_float(g[j])) * __uint_as_float(up[j]);
                    store(base + static_cast<uint64_t>(step) * c0, v, rows_out - c0);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bce), mbar_arrive(bce + 8);
            } else {
                if (!__all_sync(0xffffffffu, mbar_wait_idle(bcf + 8 * part, n & 1, err))) break;
                tc_fence_after();
                const int rows_out = w.n0 + part * kEgBM + 32 * q + lane < N ? w.rows : 0;
                for (int c0 = 0; c0 < w.rows; c0 += 16) {
                    uint32_t a[16];
                    tmem_ld_32x32b(acc + part * kEgBN + c0, a);
                    tmem_ld_wait();
                    float v[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(a[j]);
                    store(base + 2 * kEgBM * part + static_cast<uint64_t>(step) * c0, v, rows_out - c0);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bce + 8 * part);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        mbar_wait_idle(bend, 0, err);  // no MMA is under way when the accumulators are given back
        tc_fence_after();
        tmem_dealloc(tmem, kEgTmemCols);
    }
}

// ------------------------------------------------------------------ host ---

namespace {

template <bool kGated>
cudaError_t launch_gated(const ExpertArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    constexpr int cols = kGated ? kEgBM : 2 * kEgBM;
    CUtensorMap mapW, mapW2;
    if (weight_map(&mapW, a.W, a.rows.experts * a.N, a.K, kEgBM) != Q4K_OK) return cudaErrorInvalidValue;
    mapW2 = mapW;
    if (kGated && weight_map(&mapW2, a.W2, a.rows.experts * a.N, a.K, kEgBM) != Q4K_OK) return cudaErrorInvalidValue;
    XMaps mapX;
    for (int i = 0; i < kEgBN / 32; ++i)
        if (rows_map(&mapX.box[i], a.X, a.rows.pairs, a.K, 32 * (i + 1)) != Q4K_OK) return cudaErrorInvalidValue;
    const int64_t busy = a.rows.pairs < a.rows.experts ? a.rows.pairs : a.rows.experts;
    const int64_t most = (a.rows.pairs / kEgBN + busy) * ((a.N + cols - 1) / cols);
    return launch_serve(q4k_experts_gemm_kernel<kGated>, dim3(static_cast<unsigned>(most < dev.num_sms ? most : dev.num_sms)),
                        dim3(kEgThreads), eg_smem(a.rows.experts), stream, pdl, 1, mapW, mapW2, mapX, a.rows,
                        static_cast<int>(a.N), static_cast<int>(a.K), a.Y, dev.err);
}

}  // namespace

cudaError_t experts_gemm_setup() {
    const cudaError_t e = cudaFuncSetAttribute(q4k_experts_gemm_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               eg_smem(kMaxExperts));
    const cudaError_t r = cudaFuncSetAttribute(q4k_experts_gemm_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               eg_smem(kMaxExperts));
    return e != cudaSuccess ? e : r;
}

// See launch_experts.
double experts_gemm_us(const ExpertArgs& a, const DeviceInfo& dev) {
    const int64_t pairs = a.rows.pairs, busy = pairs < a.rows.experts ? pairs : a.rows.experts;
    const int64_t cols = a.W2 != nullptr ? kEgBM : 2 * kEgBM, each = (pairs + busy - 1) / busy;
    const double units = static_cast<double>(busy) * ((each + kEgBN - 1) / kEgBN) * ((a.N + cols - 1) / cols);
    const double rounds = units <= dev.num_sms ? 1.0 : units / dev.num_sms + 0.5;
    return 4.0 + rounds * (1.6 + 1.55 * static_cast<double>(a.K / kBlockWeights));
}

cudaError_t launch_experts_gemm(const ExpertArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    return a.W2 != nullptr ? launch_gated<true>(a, stream, dev, pdl) : launch_gated<false>(a, stream, dev, pdl);
}

}  // namespace q4k
