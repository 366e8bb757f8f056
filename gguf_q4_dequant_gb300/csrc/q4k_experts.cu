// q4k_experts.cu -- the experts' packed products for few rows an expert: each
// expert's Q4_K matrix (or its gate and up matrices) with its own rows, on the
// tensor cores, straight from the packed words in registers.
//
// y[p][n] = sum_k x[p][k] w(n,k) with w = d sc_j q - dmin m_j over the sub-blocks j
// of 32 k is, for each super-block of 256 k,
//   d * sum_j sc_j (sum_k q x) - dmin * sum_j m_j (sum_k x).
// A warp holds 16 weight rows x 32 k of codes as the A fragments of two
// m16n8k16 products with 8 rows of x as B. A code needs no conversion: the
// integers 0..255 as bf16 bit patterns are the numbers q 2^-133 (the patterns
// of the subnormal numbers and of the first binade count on evenly), so a byte
// spread to 16 bits and masked is the operand, the high nibble 16 times its
// code. x is multiplied by 2^64 (exact), which keeps the products in fp32's
// normal range, and the scales by 2^69. The sums of x come from products too, with
// x as the A operand (its first and second 16 k in the upper and lower eight rows) and a
// column of ones for each sub-block, so that they end where one more product with
// the m_j wants its B operand: 42 products a step (m_j against all of x took 64, and 7 us
// of the 62 for 64 tokens to 8 of 128 experts). Rows of x with values of 2^64 and more are
// out of range.
//
// What bounds it: few rows leave the memory's rate for the packed words (each
// read once) and the issue slots. So the work is laid out for the words: a warp
// owns 32 weight rows of one matrix (of a gated product gate or up) and a share of
// the super-blocks, and streams them through a ring of its own with TMA. The wk
// warps of a unit add their sums in shared memory, in warp order; with wk = 1
// warps never wait for one another. A unit is (up to 8 rows of x of an expert, 32 output
// columns); units are dealt out to resident warps, the next unit's words on their
// way during this one's end. 64 tokens to 8 of 128 experts, gated 768 x 2048: 51 us, 4.2 TB/s
// of words (38 without the products, 48 with them alone); 5 tokens to 2 of 8 experts, 4096 x
// 12288: 43 us, 4.0 TB/s; one token to 8 of 128, gated: 8.9 us.
#include <cuda_bf16.h>

#include "q4k_device.cuh"
#include "q4k_experts.h"
#include "q4k_serve.h"

namespace q4k {

// Warps of a block, blocks of an SM: 12 warps with 168 registers each (128 experts
// with four rows each, gated: 55 us; 16 warps with 128, 62).
constexpr int kExWarps = 4, kExBlocks = 3;
constexpr int kExRows = 32;                            // weight rows of a step, output columns of a unit
constexpr int kExStage = kExRows * kBlockBytes;        // 4608
constexpr int kExTile = 8;                             // rows of x of a unit
constexpr int kExStages = 2;
constexpr int kExPitch = kExRows + 8;                  // floats of a row of partial sums

struct ExSmem {
    int ring, red, bars, starts, tiles, total;
};
__host__ __device__ inline ExSmem ex_smem(int wk, int experts) {
    ExSmem s;
    s.ring = 0;
    s.red = s.ring + kExWarps * kExStages * kExStage;
    s.bars = s.red + (wk > 1 ? kExWarps * kExTile * kExPitch * 4 : 0);
    s.starts = s.bars + kExWarps * kExStages * 8;
    s.tiles = s.starts + 4 * (experts + 1);
    s.total = s.tiles + 4 * (experts + 1);
    return s;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The first product of a sum.
__device__ __forceinline__ void mma_bf16_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Physical row of an MMA operand's row: consecutive weight rows of a fragment two
// rows apart, so that eight lanes' words of a 144-byte row lie in different banks.
__device__ __forceinline__ int ex_row(int g) { return ((g & 3) << 1) | (g >> 2); }

// This lane's x of 64 k: k = off + 32 h + 8 t4 .. + 7 of its row.
__device__ __forceinline__ void ex_load(const uint16_t* x, int off, uint4 (&v)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
        v[h] = *reinterpret_cast<const uint4*>(x + off + 32 * h);
}

// One super-block of 32 weight rows (a stage, at wrow for this lane) with eight rows
// of x: acc += this step's products. x: this lane's row of x at this super-block
// and the lane's 8 k of 32; xv[0] holds its first 64 k.
__device__ __forceinline__ void ex_step(const uint8_t* wrow, const uint16_t* x, int g, int t4, uint4 (&xv)[2][2],
                                        float (&acc)[2][4]) {
    uint32_t hx[2][2];
    ScaleBytes sb[2][2];
    float d[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint4 head = *reinterpret_cast<const uint4*>(wrow + (16 * m + 8 * r) * kBlockBytes);
            sb[m][r] = decode_scales(head.y, head.z, head.w);
            hx[m][r] = head.x;
            d[m][r] = half_lo(head.x) * exp2i(69);
        }
    float sums[4];  // of x (2^59 x) over sub-blocks 2 t4 and 2 t4 + 1: their first, then their second 16 k
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (c < 3) ex_load(x, 64 * (c + 1), xv[(c + 1) & 1]);
        uint32_t xs[2][4];  // x 2^64 as B fragments
        const __nv_bfloat162 up = __floats2bfloat162_rn(exp2i(64), exp2i(64));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w[4] = {xv[c & 1][h].x, xv[c & 1][h].y, xv[c & 1][h].z, xv[c & 1][h].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), up);
                xs[h][i] = *reinterpret_cast<const uint32_t*>(&y);
            }
        }
        uint32_t a[2][2][2][4];  // [row tile][nibble half][which 16 k]
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const uint2 q0 = *reinterpret_cast<const uint2*>(wrow + 16 * m * kBlockBytes + 16 + 32 * c + 8 * t4);
            const uint2 q1 = *reinterpret_cast<const uint2*>(wrow + (16 * m + 8) * kBlockBytes + 16 + 32 * c + 8 * t4);
            // bytes of a word to 16 bits each, (0, 1) and (2, 3); the low nibbles by a mask, the high ones
            // (16 times their codes) as what is left: exact, and a subtraction goes to the FMA pipe, where
            // masks alone fill the integer one (73 us for the 77 of masks, 128 experts with four rows each)
            const uint32_t p[2][4] = {{__byte_perm(q0.x, 0, 0x4140), __byte_perm(q1.x, 0, 0x4140),
                                       __byte_perm(q0.x, 0, 0x4342), __byte_perm(q1.x, 0, 0x4342)},
                                      {__byte_perm(q0.y, 0, 0x4140), __byte_perm(q1.y, 0, 0x4140),
                                       __byte_perm(q0.y, 0, 0x4342), __byte_perm(q1.y, 0, 0x4342)}};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    a[m][0][i][k] = p[i][k] & 0x000F000Fu;
                    const __nv_bfloat162 y = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&p[i][k]),
                                                     *reinterpret_cast<const __nv_bfloat162*>(&a[m][0][i][k]));
                    a[m][1][i][k] = *reinterpret_cast<const uint32_t*>(&y);
                }
        }
        float s[2][2][2], f[2][2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = 2 * c + h;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t scw = j < 4 ? sb[m][r].sc_lo : sb[m][r].sc_hi;
                    // (2^23 + sc) d - 2^23 d: both exact, so the FMA rounds sc d once
                    const float dh = h ? d[m][r] * 0.0625f : d[m][r];
                    s[m][h][r] = fmaf(__uint_as_float(__byte_perm(scw, 0x4B000000u, 0x7440u | (j & 3))), dh, -8388608.f * dh);
                }
            }
        // a sum's next product comes some products later: the tensor core takes them one behind the other
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) mma_bf16_zero(f[m][h], a[m][h][0], xs[h][0], xs[h][1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t rows[4] = {xs[h][0], xs[h][2], xs[h][1], xs[h][3]};
            const uint32_t one = g == 2 * c + h ? 0x3D003D00u : 0u;  // 2^-5 in column j
            if (c == 0 && h == 0) mma_bf16_zero(sums, rows, one, one);
            else mma_bf16(sums, rows, one, one);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) mma_bf16(f[m][h], a[m][h][1], xs[h][2], xs[h][3]);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][i] = fmaf(f[m][h][i], s[m][h][i >> 1], acc[m][i]);
    }
    // the mins: one product over the eight sub-blocks, each sum as two bf16 (off by 2^-16 at most), m_j as m_j 2^-33
    const float even = sums[0] + sums[2], odd = sums[1] + sums[3];
    const __nv_bfloat162 top = __floats2bfloat162_rn(even, odd);
    const __nv_bfloat162 rest = __floats2bfloat162_rn(even - __low2float(top), odd - __high2float(top));
    const __nv_bfloat162 up = __floats2bfloat162_rn(exp2i(100), exp2i(100));
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        uint32_t mn[4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint32_t pair = __byte_perm(t4 < 2 ? sb[m][r].m_lo : sb[m][r].m_hi, 0, t4 & 1 ? 0x4342 : 0x4140);
            const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&pair), up);
            mn[r] = mn[r + 2] = *reinterpret_cast<const uint32_t*>(&v);
        }
        float low[4];  // 2^26 sum over j of m_j (sum of x)
        mma_bf16_zero(low, mn, *reinterpret_cast<const uint32_t*>(&top), *reinterpret_cast<const uint32_t*>(&rest));
        const float lo0 = half_hi(hx[m][0]) * exp2i(-26), lo1 = half_hi(hx[m][1]) * exp2i(-26);
        acc[m][0] = fmaf(-lo0, low[0], acc[m][0]);
        acc[m][1] = fmaf(-lo0, low[1], acc[m][1]);
        acc[m][2] = fmaf(-lo1, low[2], acc[m][2]);
        acc[m][3] = fmaf(-lo1, low[3], acc[m][3]);
    }
}

template <bool kGated>
__global__ void __launch_bounds__(32 * kExWarps, kExBlocks)
    q4k_experts_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap map2, const uint16_t* X,
                       const ExpertRows rows, int N, int K, int wk, uint16_t* Y, unsigned int* err) {
    extern __shared__ __align__(128) uint8_t ex_smem_raw[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const ExSmem at = ex_smem(wk, rows.experts);
    const int group = warp / wk, kw = warp - group * wk, groups = kExWarps / wk;
    // this warp's share of K; of a gated product's warps (two at least) the even ones have gate, the odd ones up
    const int k0 = kGated ? kw >> 1 : kw, nk = kGated ? wk >> 1 : wk;
    const CUtensorMap* words = kGated && (kw & 1) ? &map2 : &map;
    float* red = reinterpret_cast<float*>(ex_smem_raw + at.red) + group * wk * kExTile * kExPitch;
    int* starts = reinterpret_cast<int*>(ex_smem_raw + at.starts);
    int* tiles = reinterpret_cast<int*>(ex_smem_raw + at.tiles);
    const uint32_t bar = smem_u32(ex_smem_raw + at.bars) + warp * kExStages * 8;
    const uint32_t ring = smem_u32(ex_smem_raw + at.ring) + warp * kExStages * kExStage;
    const uint8_t* ring_ptr = ex_smem_raw + at.ring + warp * kExStages * kExStage;
    if (lane == 0) {
        for (int i = 0; i < kExStages; ++i) mbar_init(bar + 8 * i, 1);
        fence_barrier_init();
        tma_prefetch_desc(words);
    }
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    for (int e = threadIdx.x; e <= rows.experts; e += blockDim.x) starts[e] = min(max(rows.starts[e], 0), rows.pairs);
    __syncthreads();
    if (warp == 0) expert_tiles<kExTile>(starts, tiles, rows.experts, lane);
    __syncthreads();
    const int slabs = (N + kExRows - 1) / kExRows, all = tiles[rows.experts];
    const int KB = K / kBlockWeights;
    // this group's units: every (gridDim.x * groups)-th of (row tile, slab)
    const int every = gridDim.x * groups, first = blockIdx.x * groups + group;
    const int dt = every / slabs, ds = every - dt * slabs;

    // the producer's place: the next (unit, super-block) to be asked for
    int pt = first / slabs, ps = first - pt * slabs, pkb = k0, prow = 0;
    if (pt < all) prow = expert_at(tiles, rows.experts, pt, lane) * N + ps * kExRows;
    const uint64_t policy = policy_evict_first();
    uint32_t asked = 0, step = 0;
    auto ask = [&](int stage) {  // the whole warp; nothing when the units are through
        if (pt >= all) return;
        ++asked;
        if (lane == 0) {
            mbar_arrive_expect_tx(bar + 8 * stage, kExStage);
            tma_load_2d_hint(ring + stage * kExStage, words, pkb * kBlockBytes, prow, bar + 8 * stage, policy);
        }
        pkb += nk;
        if (pkb >= KB) {
            pkb = k0;
            pt += dt;
            ps += ds;
            if (ps >= slabs) ps -= slabs, ++pt;
            if (pt < all) prow = expert_at(tiles, rows.experts, pt, lane) * N + ps * kExRows;
        }
    };
#pragma unroll
    for (int i = 0; i < kExStages; ++i) ask(i);

    const int g = lane >> 2, t4 = lane & 3;
    const bool vec = (N & 3) == 0;
    bool ok = true;
    int t = first / slabs, s = first - t * slabs;
    while (t < all) {
        const int e = expert_at(tiles, rows.experts, t, lane), n0 = s * kExRows;
        const int p0 = starts[e] + (t - tiles[e]) * kExTile, p1 = min(p0 + kExTile, starts[e + 1]);
        float acc[2][4] = {};
        // (lanes without a row have the last one again: its products go nowhere)
        const uint16_t* x = X + static_cast<int64_t>(min(p0 + g, p1 - 1)) * K + k0 * kBlockWeights + 8 * t4;
        for (int kb = k0; kb < KB; kb += nk, ++step) {
            const int stage = step % kExStages;
            uint4 xv[2][2];
            ex_load(x, 0, xv[0]);
            if (ok && !__all_sync(0xffffffffu, mbar_wait(bar + 8 * stage, (step / kExStages) & 1, err))) {
                // the words did not come: nothing more is asked for (the sums are worth nothing), and
                // the block does not end while a copy is on its way
                ok = false;
                pt = all;
                for (uint32_t i = step; i < asked; ++i)
                    mbar_wait(bar + 8 * (i % kExStages), (i / kExStages) & 1, err, kDrainLimitNs);
            }
            ex_step(ring_ptr + stage * kExStage + ex_row(g) * kBlockBytes, x, g, t4, xv, acc);
            // every word of the stage has gone through a product that has been issued
            __syncwarp();
            ask(stage);
            x += nk * kBlockWeights;
        }
        if (!kGated && wk == 1) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int p = p0 + 2 * t4 + (i & 1), n = n0 + 16 * m + 8 * (i >> 1) + ex_row(g);
                    if (p < p1 && n < N)
                        Y[static_cast<int64_t>(p) * N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[m][i]));
                }
        } else {
            // the warps' sums: red[warp][row of x][weight row]
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    red[(kw * kExTile + 2 * t4 + (i & 1)) * kExPitch + 16 * m + 8 * (i >> 1) + ex_row(g)] = acc[m][i];
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * wk) : "memory");
            for (int i = 32 * kw + lane; i < kExTile * kExRows / 4; i += 32 * wk) {
                const int r = i / (kExRows / 4), n = 4 * (i % (kExRows / 4));
                if (p0 + r >= p1 || n0 + n >= N) continue;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f), w = v;
                for (int k = 0; k < wk; k += kGated ? 2 : 1) {
                    const float* src = red + (k * kExTile + r) * kExPitch + n;
                    const float4 a = *reinterpret_cast<const float4*>(src);
                    v.x += a.x; v.y += a.y; v.z += a.z; v.w += a.w;
                    if (kGated) {
                        const float4 b = *reinterpret_cast<const float4*>(src + kExTile * kExPitch);
                        w.x += b.x; w.y += b.y; w.z += b.z; w.w += b.w;
                    }
                }
                if (kGated) {
                    v.x = silu(v.x) * w.x;
                    v.y = silu(v.y) * w.y;
                    v.z = silu(v.z) * w.z;
                    v.w = silu(v.w) * w.w;
                }
                const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
                const uint2 o = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                uint16_t* y = Y + static_cast<int64_t>(p0 + r) * N + n0 + n;
                if (vec) {
                    *reinterpret_cast<uint2*>(y) = o;
                } else {
                    y[0] = static_cast<uint16_t>(o.x);
                    if (n0 + n + 1 < N) y[1] = static_cast<uint16_t>(o.x >> 16);
                    if (n0 + n + 2 < N) y[2] = static_cast<uint16_t>(o.y);
                    if (n0 + n + 3 < N) y[3] = static_cast<uint16_t>(o.y >> 16);
                }
            }
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * wk) : "memory");
        }
        t += dt;
        s += ds;
        if (s >= slabs) s -= slabs, ++t;
    }
}

// ------------------------------------------------------------------ host ---

namespace {

template <bool kGated>
cudaError_t launch_few(const ExpertArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    CUtensorMap map, map2;
    if (weight_map(&map, a.W, a.rows.experts * a.N, a.K, kExRows) != Q4K_OK) return cudaErrorInvalidValue;
    map2 = map;
    if (kGated && weight_map(&map2, a.W2, a.rows.experts * a.N, a.K, kExRows) != Q4K_OK) return cudaErrorInvalidValue;
    const int64_t busy = a.rows.pairs < a.rows.experts ? a.rows.pairs : a.rows.experts, slabs = (a.N + kExRows - 1) / kExRows;
    const int KB = static_cast<int>(a.K / kBlockWeights);
    // wk, the warps that share K: few units are split further, so that every warp
    // of the GPU has some of the words on their way (8 experts of 128 with one row
    // each, gated 768 x 2048: 10.7 us with 4, 12.6 with 2); many are not, as the warps of
    // a unit wait for one another (four rows for each of 128 experts of 2048 x 768: 32 us
    // with 1, 38 with 2). In between it counts how full the last round is (5 tokens to
    // 2 of 8 experts of 4096 x 12288: 61, 45, 45 us with 1, 2, 4).
    const int64_t tiles = busy > a.rows.pairs / kExTile ? busy : a.rows.pairs / kExTile;
    int wk = kGated ? 2 : 1, per = 1;
    double best = 1e300;
    for (int w = wk; w <= kExWarps; w *= 2) {
        const int nk = kGated ? w / 2 : w;
        if (nk > KB) break;
        int p = static_cast<int>((228 * 1024) / (ex_smem(w, a.rows.experts).total + 1024));
        p = p < 1 ? 1 : p < kExBlocks ? p : kExBlocks;
        const double groups = static_cast<double>(dev.num_sms) * p * kExWarps / w;
        // the experts with rows are known on the device only: half a round is lost on average
        const double rounds = static_cast<double>(tiles * slabs) / groups + 0.5;
        const double cost = (rounds > 1.0 ? rounds : 1.0) * ((KB + nk - 1) / nk + (w > 1 ? 0.5 : 0.25));
        if (cost < best * 0.999) best = cost, wk = w, per = p;
    }
    const int64_t units = (a.rows.pairs / kExTile + busy) * slabs, groups = kExWarps / wk;
    const int64_t blocks = (units + groups - 1) / groups, slots = static_cast<int64_t>(dev.num_sms) * per;
    return launch_serve(q4k_experts_kernel<kGated>, dim3(static_cast<unsigned>(blocks < slots ? blocks : slots)),
                        dim3(32 * kExWarps), ex_smem(wk, a.rows.experts).total, stream, pdl, 1, map, map2, a.X, a.rows,
                        static_cast<int>(a.N), static_cast<int>(a.K), wk, a.Y, dev.err);
}

template <bool kGated>
cudaError_t setup_few() {
    return cudaFuncSetAttribute(q4k_experts_kernel<kGated>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                ex_smem(kExWarps, kMaxExperts).total);
}

}  // namespace

cudaError_t experts_setup(DeviceInfo&) {
    cudaError_t e = experts_gemm_setup(), r;
    if ((r = setup_few<false>()) != cudaSuccess) e = r;
    if ((r = setup_few<true>()) != cudaSuccess) e = r;
    return e;
}

// The two kernels' times in us, from the sizes that the host knows: experts with
// rows are taken to be all of them or as many as there are rows, with equal
// shares. The one for few rows goes over the words again for every eight rows of
// an expert, 0.92 ns a step of 32 weight rows and 256 k on all of the GPU; the
// tcgen05 kernel's blocks take 1.55 us for 256 k of a unit, whatever rows it has, and 1.6
// for its end, and have nothing to share out when there are few units. 128 experts, gated
// 768 x 2048: 8 rows each 70 us for 84 (here 73, 83), 12 rows 97 for 84 (95, 83); down 2048 x
// 768: 8 rows 41 us for 46 (39, 49), 12 rows 53 for 47 (50, 49); 8 experts of 4096 x 12288: 8 rows
// 68 for 82 (73, 80), 12 rows 90 for 82 (95, 80); 2 experts of 144 x 7168, 300 rows: 17 for 49 (15, 49).
// (Tiles of 16 and 32 rows in the first kernel were slower than its 8 or the second at every size.)
static bool many_rows(const ExpertArgs& a, const DeviceInfo& dev) {
    const double pairs = a.rows.pairs, busy = pairs < a.rows.experts ? pairs : a.rows.experts, mats = a.W2 != nullptr ? 2 : 1;
    const double KB = static_cast<double>(a.K / kBlockWeights);
    const double slabs = static_cast<double>((a.N + kExRows - 1) / kExRows);
    double tiles = pairs / kExTile + 0.5 * busy;
    tiles = tiles > busy ? tiles : busy;
    const double few = 5.0 + 0.92e-3 * tiles * slabs * KB * mats;
    return experts_gemm_us(a, dev) < few;
}

cudaError_t launch_experts(const ExpertArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    if (many_rows(a, dev)) return launch_experts_gemm(a, stream, dev, pdl);
    return a.W2 != nullptr ? launch_few<true>(a, stream, dev, pdl) : launch_few<false>(a, stream, dev, pdl);
}

}  // namespace q4k
