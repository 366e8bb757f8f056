// q4k_experts_gemm.cu -- the experts' packed products for many rows an expert, on
// the 5th-generation tensor cores: each expert's Q4_K matrix (or its gate and up
// matrices) with its own rows of x.
//
// Y^T = W X^T as in the dense GEMM: the MMA's A operand is 128 weight rows,
// dequantised to bf16 in TMEM, its B operand up to 192 rows of x, the
// accumulator 128 TMEM lanes x the rows of x. A unit is (expert, rows of x,
// 128 weight rows); of a gated product the 128 are 64 gate and 64 up rows,
// sixteen and sixteen in turn, so that the two factors of an output lie in one
// warp's lanes at the end. The rows of an expert are cut into tiles of equal
// height, and a tile's MMAs are as wide as the tile (a multiple of 16).
//
// A block stays on its SM and takes every gridDim-th unit; its warps run ahead
// of one another through rings, from one unit into the next:
//   warp 0       W producer: {144 B, 128 rows} of packed words per 256 k (TMA)
//   warp 1       MMA issuer, TMEM (two accumulators: a unit's end overlaps the next)
//   warp 2       X producer: the tile's rows x 128 k (TMA, 128-byte swizzle)
//   warps 4..7   the end of a unit: TMEM -> registers -> (silu(g) u) -> bf16 -> Y
//   warps 8..23  dequantisers, four groups of 128 threads: group c has the 64 k
//                chunk c of every super-block, thread r of it a weight row, and
//                32 columns of TMEM: half the A operand of a step of 128 k
// All waits are bounded (see mbar_wait).
#include <cuda_bf16.h>

#include "q4k_device.cuh"
#include "q4k_experts.h"
#include "q4k_serve.h"

namespace q4k {

constexpr int kEgBM = 128;                    // weight rows of a unit
constexpr int kEgBN = 192;                    // rows of x of a unit at most
// k of a step, the work of one commit: a commit and its wait take the issuing warp
// some 320 cycles whatever they cover, the eight MMAs of a step 4 cycles a row of x
constexpr int kEgStep = 128;
constexpr int kEgAStages = 2, kEgXStages = 3, kEgWStages = 4;
constexpr int kEgXHalf = kEgBN * 128;         // 64 k of the rows of x
constexpr int kEgXStage = 2 * kEgXHalf;
constexpr int kEgWStage = kEgBM * kBlockBytes;
constexpr int kEgEpiWarp = 4, kEgDeqWarp = 8, kEgDeqWarps = 16;
constexpr int kEgThreads = 32 * (kEgDeqWarp + kEgDeqWarps);
constexpr int kEgOffW = kEgXStages * kEgXStage;
constexpr int kEgOffBar = kEgOffW + kEgWStages * kEgWStage;
// w_full, w_empty, x_full, a_full, done (of a step's MMAs), acc_full[2], acc_empty[2], end
constexpr int kEgBars = 2 * (kEgWStages + kEgXStages) + kEgAStages + 5;
constexpr int kEgOffTmem = kEgOffBar + 8 * kEgBars;
constexpr int kEgOffTab = (kEgOffTmem + 8 + 15) / 16 * 16;
constexpr uint32_t kEgTmemCols = 512, kEgTmemA = 2 * kEgBN;  // the accumulators, then 64 columns a stage of A
static_assert(kEgTmemA + 64 * kEgAStages <= kEgTmemCols, "TMEM");

__host__ __device__ constexpr int eg_smem(int experts) { return kEgOffTab + 8 * (experts + 1) + 1024; }
static_assert(eg_smem(kMaxExperts) <= 232448, "shared memory per CTA");

struct XMaps {
    CUtensorMap box[kEgBN / 32];  // boxes of 32, 64, .. rows x 64 k
};

// Eight weights of one nibble half (hh) from the qs words w0 and w1, as bf16 pairs.
// A nibble at bit s of a word, under the bits of 1.0, is the float 1 + q 2^(s-23),
// and d1 q - m1 = (1 + q 2^(s-23)) E - (E + m1) with E = d1 2^(23-s): one masking
// and half a paired FMA a weight. The constant's rounding, 2^-24 E, is 2^-8 d1
// at most (s >= 7) and mostly far less, beside the rounding to 8 significant bits
// that the weight meets anyway. Bytes 0 and 1 are brought to bits 7 and 15, bytes
// 2 and 3 too. E0, C0 and E1, C1: (E, E) and -(E + m1, E + m1) for s = 7 + 4 hh and 15 + 4 hh.
__device__ __forceinline__ void dequant8(uint32_t w0, uint32_t w1, int hh, uint64_t E0, uint64_t C0, uint64_t E1,
                                         uint64_t C1, uint32_t* o) {
    const uint32_t one = 0x3F800000u, m0 = 0x780u << (4 * hh), m1 = 0x78000u << (4 * hh);
    const uint32_t u0 = w0 << 7, u1 = w1 << 7, v0 = w0 >> 9, v1 = w1 >> 9;
    auto two = [&](uint32_t a, uint32_t b, uint32_t m) {
        return static_cast<uint64_t>((a & m) | one) | static_cast<uint64_t>((b & m) | one) << 32;
    };
    const float2 a = unpack2(fma2(two(u0, u1, m0), E0, C0)), b = unpack2(fma2(two(u0, u1, m1), E1, C1));
    const float2 c = unpack2(fma2(two(v0, v1, m0), E0, C0)), d = unpack2(fma2(two(v0, v1, m1), E1, C1));
    const __nv_bfloat162 r[4] = {__floats2bfloat162_rn(a.x, b.x), __floats2bfloat162_rn(c.x, d.x),
                                 __floats2bfloat162_rn(a.y, b.y), __floats2bfloat162_rn(c.y, d.y)};
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = *reinterpret_cast<const uint32_t*>(&r[i]);
}

template <bool kGated>
__global__ void __launch_bounds__(kEgThreads, 1)
    q4k_experts_gemm_kernel(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapW2,
                            const __grid_constant__ XMaps mapX, const ExpertRows rows, int N, int K, uint16_t* Y,
                            unsigned int* err) {
    constexpr int kCols = kGated ? kEgBM / 2 : kEgBM;  // output columns of a unit
    extern __shared__ uint8_t eg_raw[];
    const uint32_t raw = smem_u32(eg_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t* smem = eg_raw + pad;
    const uint32_t sbase = raw + pad;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bwf = sbase + kEgOffBar, bwe = bwf + 8 * kEgWStages, bxf = bwe + 8 * kEgWStages,
                   baf = bxf + 8 * kEgXStages, bdone = baf + 8 * kEgAStages,
                   bcf = bdone + 8 * kEgXStages, bce = bcf + 16, bend = bce + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kEgOffTmem);
    int* starts = reinterpret_cast<int*>(smem + kEgOffTab);
    int* tiles = starts + rows.experts + 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kEgWStages; ++i) mbar_init(bwf + 8 * i, 1), mbar_init(bwe + 8 * i, kEgDeqWarps);
        for (int i = 0; i < kEgXStages; ++i) mbar_init(bxf + 8 * i, 1), mbar_init(bdone + 8 * i, 1);
        for (int i = 0; i < kEgAStages; ++i) mbar_init(baf + 8 * i, kEgDeqWarps / 2);
        for (int i = 0; i < 2; ++i) mbar_init(bcf + 8 * i, 1), mbar_init(bce + 8 * i, 4);
        mbar_init(bend, 1);
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

    // unit u: (expert, row tile, column tile), the column tiles of a row tile side
    // by side, so that its rows of x come from memory once
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
            const uint64_t pol = policy_evict_first();
            uint32_t it = 0;
            bool ok = true;
            for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const Unit w = unit_of(u);
                for (int sb = 0; sb < KB; ++sb, ++it) {
                    const uint32_t s = it % kEgWStages;
                    if (!mbar_wait(bwe + 8 * s, ((it / kEgWStages) & 1) ^ 1, err)) { ok = false; break; }
                    mbar_arrive_expect_tx(bwf + 8 * s, kEgWStage);
                    const uint32_t dst = sbase + kEgOffW + s * kEgWStage;
                    tma_load_2d_hint(dst, &mapW, sb * kBlockBytes, w.e * N + w.n0, bwf + 8 * s, pol);
                    if (kGated) tma_load_2d_hint(dst + kEgWStage / 2, &mapW2, sb * kBlockBytes, w.e * N + w.n0, bwf + 8 * s, pol);
                }
            }
            // the copies that may still be landing after a timeout
            if (!ok)
                for (uint32_t i = it < kEgWStages ? 0 : it - kEgWStages; i < it; ++i)
                    mbar_wait(bwf + 8 * (i % kEgWStages), (i / kEgWStages) & 1, err, kDrainLimitNs);
        }
        __syncwarp();
    } else if (warp == 2) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_last();
            uint32_t it = 0;
            bool ok = true;
            for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const Unit w = unit_of(u);
                const int q = (max(w.rows, 1) - 1) / 32;  // a box of 32 (q + 1) rows
                const uint32_t bytes = 2u * 32u * 128u * (q + 1);
                for (int ks = 0; ks < 2 * KB; ++ks, ++it) {
                    const uint32_t s = it % kEgXStages;
                    // free once the MMAs of step it - kEgXStages are done (that barrier's next phase
                    // is step it's own: no wait finds its barrier two phases on)
                    if (it >= kEgXStages && !mbar_wait(bdone + 8 * s, (it / kEgXStages - 1) & 1, err)) { ok = false; break; }
                    mbar_arrive_expect_tx(bxf + 8 * s, bytes);
                    const uint32_t dst = sbase + s * kEgXStage;
                    tma_load_2d_hint(dst, &mapX.box[q], ks * kEgStep, w.p0, bxf + 8 * s, pol);
                    tma_load_2d_hint(dst + kEgXHalf, &mapX.box[q], ks * kEgStep + 64, w.p0, bxf + 8 * s, pol);
                }
            }
            if (!ok)
                for (uint32_t i = it < kEgXStages ? 0 : it - kEgXStages; i < it; ++i)
                    mbar_wait(bxf + 8 * (i % kEgXStages), (i / kEgXStages) & 1, err, kDrainLimitNs);
        }
        __syncwarp();
    } else if (warp == 1) {
        // the whole warp goes through the loop, so that addresses and descriptors stay
        // the warp's own; one lane issues
        uint32_t it = 0, n = 0;
        bool ok = true;
        for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x, ++n) {
            const Unit w = unit_of(u);
            const uint32_t idesc = idesc_bf16_f32(kEgBM, max(16, (w.rows + 15) & ~15));
            const uint32_t d = tmem + (n & 1) * kEgBN;
            if (!__all_sync(0xffffffffu, mbar_wait(bce + 8 * (n & 1), ((n >> 1) & 1) ^ 1, err))) break;
            for (int ks = 0; ks < 2 * KB; ++ks, ++it) {
                const uint32_t sa = it % kEgAStages, sx = it % kEgXStages;
                const bool in = mbar_wait(bxf + 8 * sx, (it / kEgXStages) & 1, err) &&
                                mbar_wait(baf + 8 * sa, (it / kEgAStages) & 1, err);
                if (!__all_sync(0xffffffffu, in)) { ok = false; break; }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t a0 = tmem + kEgTmemA + 64 * sa;
                    const uint64_t b0 = sw128_desc(sbase + sx * kEgXStage);
#pragma unroll
                    for (int kk = 0; kk < kEgStep / 16; ++kk)
                        tc_mma_bf16_ts(d, a0 + 8 * kk, b0 + (kk >> 2) * (kEgXHalf >> 4) + 2 * (kk & 3), idesc, ks != 0 || kk != 0);
                    tc_commit(bdone + 8 * sx);
                    if (ks == 2 * KB - 1) tc_commit(bcf + 8 * (n & 1));
                }
                __syncwarp();
            }
        }
        if (elect_one()) tc_commit(bend);
        __syncwarp();
    } else if (warp >= kEgDeqWarp) {
        const int t = threadIdx.x - 32 * kEgDeqWarp;
        const int c = t >> 7;
        // the TMEM lane of this thread, and the row of packed words that goes there: of a gated
        // unit 16 gate rows, then the 16 up rows that go with them
        const int ra = t & (kEgBM - 1);
        const int r = kGated ? (ra & 16) * 4 + (ra >> 5) * 16 + (ra & 15) : ra;
        const uint32_t a_tmem = tmem + kEgTmemA + 32 * c + (static_cast<uint32_t>(ra & ~31) << 16);
        const int sh = 16 * (c & 1);
        // 0, read from shared memory so that the compiler cannot see through the
        // dependence that is built from it below
        const uint32_t zero = *reinterpret_cast<volatile uint32_t*>(tmem_slot + 1);
        uint32_t it = 0;
        bool ok = true;
        for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
            for (int sb = 0; sb < KB; ++sb, ++it) {
                const uint32_t s = it % kEgWStages;
                if (!__all_sync(0xffffffffu, mbar_wait(bwf + 8 * s, (it / kEgWStages) & 1, err))) { ok = false; break; }
                const uint8_t* P = smem + kEgOffW + s * kEgWStage + r * kBlockBytes;
                const uint4 hd = *reinterpret_cast<const uint4*>(P);
                const uint4 qa = *reinterpret_cast<const uint4*>(P + 16 + 32 * c);
                const uint4 qb = *reinterpret_cast<const uint4*>(P + 32 + 32 * c);
                // the stage is given back once every lane has its words: the vote
                // needs all of them, so the arrival cannot come before the loads
                const unsigned all = __ballot_sync(0xffffffffu, (hd.x | qa.x | qb.x) != 0u);
                if (lane == 0) mbar_arrive(bwe + 8 * s + (all & zero));
                // the two scales and mins of sub-blocks 2c and 2c + 1, a byte each
                const uint32_t s0 = hd.y >> sh, s1 = hd.z >> sh, s2 = hd.w >> sh;
                const uint32_t sc = c < 2 ? s0 & 0x3F3Fu : (s2 & 0x0F0Fu) | ((s0 >> 2) & 0x3030u);
                const uint32_t mn = c < 2 ? s1 & 0x3F3Fu : ((s2 >> 4) & 0x0F0Fu) | ((s1 >> 2) & 0x3030u);
                const float d = half_lo(hd.x), dmin = half_hi(hd.x);
                const uint32_t qw[8] = {qa.x, qa.y, qa.z, qa.w, qb.x, qb.y, qb.z, qb.w};
                uint32_t o[32];  // the row's 64 k, two to a column
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const float d1 = d * byte_to_float(sc, hh), m1 = dmin * byte_to_float(mn, hh);
                    const float e0 = d1 * exp2i(16 - 4 * hh), e1 = d1 * exp2i(8 - 4 * hh);
                    const float c0 = -(e0 + m1), c1 = -(e1 + m1);
                    const uint64_t E0 = pack2(e0, e0), C0 = pack2(c0, c0), E1 = pack2(e1, e1), C1 = pack2(c1, c1);
#pragma unroll
                    for (int v = 0; v < 4; ++v) dequant8(qw[2 * v], qw[2 * v + 1], hh, E0, C0, E1, C1, o + 16 * hh + 4 * v);
                }
                // the stage is free once the MMAs of two steps before are done (the barrier's next
                // phase is a step behind this one's: it cannot be further)
                const uint32_t step = 2 * it + (c >> 1), was = step - kEgAStages;
                if (step >= kEgAStages &&
                    !__all_sync(0xffffffffu, mbar_wait(bdone + 8 * (was % kEgXStages), (was / kEgXStages) & 1, err))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                tmem_st_32x32b_x32(a_tmem, o);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(baf + 8 * (c >> 1));
            }
        }
    } else if (warp >= kEgEpiWarp) {
        const int q = warp & 3;
        uint32_t n = 0;
        for (int64_t u = blockIdx.x; u < units; u += gridDim.x, ++n) {
            const Unit w = unit_of(u);
            if (!__all_sync(0xffffffffu, mbar_wait(bcf + 8 * (n & 1), (n >> 1) & 1, err))) break;
            tc_fence_after();
            const uint32_t acc = tmem + (n & 1) * kEgBN + (static_cast<uint32_t>(32 * q) << 16);
            // gated: lane i < 16 has gate row i, lane i + 16 the up row of the same column: they
            // swap one value for two rows of x, and each has one output
            const int col = w.n0 + (kGated ? 16 * q + (lane & 15) : 32 * q + lane);
            uint16_t* y = Y + static_cast<int64_t>(w.p0 + (kGated ? lane >> 4 : 0)) * N + col;
            for (int c0 = 0; c0 < w.rows; c0 += 32) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(acc + c0, v);
                tmem_ld_wait();
                const int left = col < N ? w.rows - c0 : 0;
                if (kGated) {
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float mine = __uint_as_float(lane < 16 ? v[j] : v[j + 1]);
                        const float away = __uint_as_float(__shfl_xor_sync(0xffffffffu, lane < 16 ? v[j + 1] : v[j], 16));
                        const uint16_t o = __bfloat16_as_ushort(__float2bfloat16_rn(lane < 16 ? silu(mine) * away : silu(away) * mine));
                        if (j + (lane >> 4) < left) *y = o;
                        y += 2 * N;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (j < left) *y = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(v[j])));
                        y += N;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bce + 8 * (n & 1));
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        mbar_wait(bend, 0, err);  // no MMA is under way when the accumulators are given back
        tc_fence_after();
        tmem_dealloc(tmem, kEgTmemCols);
    }
}

// ------------------------------------------------------------------ host ---

namespace {

template <bool kGated>
cudaError_t launch_gated(const ExpertArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    constexpr int cols = kGated ? kEgBM / 2 : kEgBM;
    CUtensorMap mapW, mapW2;
    if (weight_map(&mapW, a.W, a.rows.experts * a.N, a.K, cols) != Q4K_OK) return cudaErrorInvalidValue;
    mapW2 = mapW;
    if (kGated && weight_map(&mapW2, a.W2, a.rows.experts * a.N, a.K, cols) != Q4K_OK) return cudaErrorInvalidValue;
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

cudaError_t launch_experts_gemm(const ExpertArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    return a.W2 != nullptr ? launch_gated<true>(a, stream, dev, pdl) : launch_gated<false>(a, stream, dev, pdl);
}

}  // namespace q4k
