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
// normal range, and the scales by 2^69. The mins are the same trick: m_j as
// the A operand for all 32 k of its sub-block, one accumulator for all of them.
// Rows of x with values of 2^64 and more are out of range.
//
// What bounds it: few rows leave the memory's rate for the packed words (each
// read once) and the issue slots. So the work is laid out for the words: a warp
// owns 32 weight rows (of a gated product 32 of each matrix) and every wk-th
// super-block, and streams them through a ring of its own with TMA. The wk warps
// of a unit add their sums in shared memory, in warp order; with wk = 1 warps
// never wait for one another. A unit is (8 NB rows of x of an expert, 32 output
// columns); units are dealt out to resident warps, the next unit's words on their
// way during this one's end.
#include <cuda_bf16.h>

#include "q4k_device.cuh"
#include "q4k_experts.h"
#include "q4k_serve.h"

namespace q4k {

constexpr int kExWarps = 8;                            // warps of a block
constexpr int kExRows = 32;                            // weight rows of a step, output columns of a unit
constexpr int kExStage = kExRows * kBlockBytes;        // 4608
constexpr int kExStages = 2;
constexpr int kExPitch = kExRows + 8;                  // floats of a row of partial sums

struct ExSmem {
    int ring, red, bars, starts, tiles, total;
};
__host__ __device__ inline ExSmem ex_smem(int NB, bool gated, int wk, int experts) {
    ExSmem s;
    s.ring = 0;
    s.red = s.ring + kExWarps * kExStages * kExStage;
    s.bars = s.red + (wk > 1 ? kExWarps * 8 * NB * kExPitch * 4 * (gated ? 2 : 1) : 0);
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

// One super-block of 32 weight rows (a stage, at wrow for this lane) with 8 NB rows
// of x: acc += this step's products. xrow: this lane's row of x of each eight, at
// this super-block and the lane's 8 k; live: whether there is one.
template <int NB>
__device__ __forceinline__ void ex_step(const uint8_t* wrow, const uint16_t* const (&xrow)[NB], const bool (&live)[NB],
                                        int t4, uint4 (&xv)[2][NB][2], float (&acc)[2][NB][4]) {
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
    float low[2][NB][4];  // sum over j of m_j (sum of x)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (c < 3) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    xv[(c + 1) & 1][b][h] = live[b] ? *reinterpret_cast<const uint4*>(xrow[b] + 64 * (c + 1) + 32 * h)
                                                    : make_uint4(0, 0, 0, 0);
        }
        uint32_t xs[NB][2][4];  // x 2^64 as B fragments
        const __nv_bfloat162 up = __floats2bfloat162_rn(exp2i(64), exp2i(64));
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t w[4] = {xv[c & 1][b][h].x, xv[c & 1][b][h].y, xv[c & 1][b][h].z, xv[c & 1][b][h].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), up);
                    xs[b][h][i] = *reinterpret_cast<const uint32_t*>(&y);
                }
            }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const uint2 q0 = *reinterpret_cast<const uint2*>(wrow + 16 * m * kBlockBytes + 16 + 32 * c + 8 * t4);
            const uint2 q1 = *reinterpret_cast<const uint2*>(wrow + (16 * m + 8) * kBlockBytes + 16 + 32 * c + 8 * t4);
            // bytes of a word to 16 bits each: (0, 1) and (2, 3)
            const uint32_t p[2][4] = {{__byte_perm(q0.x, 0, 0x4140), __byte_perm(q1.x, 0, 0x4140),
                                       __byte_perm(q0.x, 0, 0x4342), __byte_perm(q1.x, 0, 0x4342)},
                                      {__byte_perm(q0.y, 0, 0x4140), __byte_perm(q1.y, 0, 0x4140),
                                       __byte_perm(q0.y, 0, 0x4342), __byte_perm(q1.y, 0, 0x4342)}};
            // the low nibbles by a mask, the high ones (16 times their codes) as what is left: exact, and
            // a subtraction goes to the FMA pipe, the masks fill the integer one
            uint32_t a[2][2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    a[0][i][k] = p[i][k] & 0x000F000Fu;
                    const __nv_bfloat162 y = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&p[i][k]), *reinterpret_cast<const __nv_bfloat162*>(&a[0][i][k]));
                    a[1][i][k] = *reinterpret_cast<const uint32_t*>(&y);
                }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = 2 * c + h;
                float s[2];
                uint32_t mn[4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t scw = j < 4 ? sb[m][r].sc_lo : sb[m][r].sc_hi;
                    const uint32_t mw = j < 4 ? sb[m][r].m_lo : sb[m][r].m_hi;
                    // (2^23 + sc) d - 2^23 d: both exact, so the FMA rounds sc d once
                    const float dh = h ? d[m][r] * 0.0625f : d[m][r];
                    s[r] = fmaf(__uint_as_float(__byte_perm(scw, 0x4B000000u, 0x7440u | (j & 3))), dh, -8388608.f * dh);
                    mn[r] = mn[r + 2] = __byte_perm(mw, 0, (j & 3) * 0x0101 | 0x4040);
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float f[4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (i == 0) mma_bf16_zero(f, a[h][i], xs[b][h][0], xs[b][h][1]); else mma_bf16(f, a[h][i], xs[b][h][2], xs[b][h][3]);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (j == 0 && i == 0) mma_bf16_zero(low[m][b], mn, xs[b][h][0], xs[b][h][1]);
                        else mma_bf16(low[m][b], mn, xs[b][h][2 * i], xs[b][h][2 * i + 1]);
                    }
                    acc[m][b][0] = fmaf(f[0], s[0], acc[m][b][0]);
                    acc[m][b][1] = fmaf(f[1], s[0], acc[m][b][1]);
                    acc[m][b][2] = fmaf(f[2], s[1], acc[m][b][2]);
                    acc[m][b][3] = fmaf(f[3], s[1], acc[m][b][3]);
                }
            }
        }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const float lo0 = half_hi(hx[m][0]) * exp2i(69), lo1 = half_hi(hx[m][1]) * exp2i(69);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            acc[m][b][0] = fmaf(-lo0, low[m][b][0], acc[m][b][0]);
            acc[m][b][1] = fmaf(-lo0, low[m][b][1], acc[m][b][1]);
            acc[m][b][2] = fmaf(-lo1, low[m][b][2], acc[m][b][2]);
            acc[m][b][3] = fmaf(-lo1, low[m][b][3], acc[m][b][3]);
        }
    }
}

// Blocks of an SM: two, as far as a thread's sums leave it 128 registers.
__host__ __device__ constexpr int ex_blocks(int NB, bool gated) { return NB == 1 || (NB == 2 && !gated) ? 2 : 1; }

template <int NB, bool kGated>
__global__ void __launch_bounds__(32 * kExWarps, ex_blocks(NB, kGated))
    q4k_experts_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap map2, const uint16_t* X,
                       const ExpertRows rows, int N, int K, int wk, uint16_t* Y, unsigned int* err) {
    constexpr int NT = 8 * NB;              // rows of x of a unit
    constexpr int kMats = kGated ? 2 : 1;   // matrices of a unit
    extern __shared__ __align__(128) uint8_t ex_smem_raw[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const ExSmem at = ex_smem(NB, kGated, wk, rows.experts);
    const int group = warp / wk, kw = warp - group * wk, groups = kExWarps / wk;
    float* red = reinterpret_cast<float*>(ex_smem_raw + at.red) + group * wk * kMats * NT * kExPitch;
    int* starts = reinterpret_cast<int*>(ex_smem_raw + at.starts);
    int* tiles = reinterpret_cast<int*>(ex_smem_raw + at.tiles);
    const uint32_t bar = smem_u32(ex_smem_raw + at.bars) + warp * kExStages * 8;
    const uint32_t ring = smem_u32(ex_smem_raw + at.ring) + warp * kExStages * kExStage;
    const uint8_t* ring_ptr = ex_smem_raw + at.ring + warp * kExStages * kExStage;
    if (lane == 0) {
        for (int i = 0; i < kExStages; ++i) mbar_init(bar + 8 * i, 1);
        fence_barrier_init();
    }
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    for (int e = threadIdx.x; e <= rows.experts; e += blockDim.x) starts[e] = min(max(rows.starts[e], 0), rows.pairs);
    __syncthreads();
    if (warp == 0) expert_tiles<NT>(starts, tiles, rows.experts, lane);
    __syncthreads();
    const int slabs = (N + kExRows - 1) / kExRows, all = tiles[rows.experts];
    const int KB = K / kBlockWeights;
    // this group's units: every (gridDim.x * groups)-th of (row tile, slab)
    const int every = gridDim.x * groups, first = blockIdx.x * groups + group;
    const int dt = every / slabs, ds = every - dt * slabs;

    // the producer's place: the next (unit, super-block, matrix) to be asked for
    int pt = first / slabs, ps = first - pt * slabs, pkb = kw, pm = 0, prow = 0;
    if (pt < all) prow = expert_at(tiles, rows.experts, pt, lane) * N + ps * kExRows;
    const uint64_t policy = policy_evict_first();
    uint32_t asked = 0, step = 0;
    auto ask = [&](int stage) {  // the whole warp; nothing when the units are through
        if (pt >= all) return;
        ++asked;
        if (lane == 0) {
            mbar_arrive_expect_tx(bar + 8 * stage, kExStage);
            tma_load_2d_hint(ring + stage * kExStage, kGated && pm ? &map2 : &map, pkb * kBlockBytes, prow, bar + 8 * stage, policy);
        }
        if (kGated && pm == 0) {
            pm = 1;
            return;
        }
        pm = 0;
        pkb += wk;
        if (pkb >= KB) {
            pkb = kw;
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
        const int p0 = starts[e] + (t - tiles[e]) * NT, p1 = min(p0 + NT, starts[e + 1]);
        float acc[kMats][2][NB][4] = {};
        const uint16_t* xrow[NB];
        bool live[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            live[b] = p0 + 8 * b + g < p1;
            xrow[b] = X + static_cast<int64_t>(live[b] ? p0 + 8 * b + g : p0) * K + 8 * t4 + kw * kBlockWeights;
        }
        for (int kb = kw; kb < KB; kb += wk) {
#pragma unroll
            for (int mat = 0; mat < kMats; ++mat, ++step) {
                const int stage = step % kExStages;
                uint4 xv[2][NB][2];  // this lane's x of 64 k at a time: k = 64 c + 32 h + 8 t4 .. + 7
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        xv[0][b][h] = live[b] ? *reinterpret_cast<const uint4*>(xrow[b] + 32 * h) : make_uint4(0, 0, 0, 0);
                if (ok && !__all_sync(0xffffffffu, mbar_wait(bar + 8 * stage, (step / kExStages) & 1, err))) {
                    // the words did not come: nothing more is asked for (the sums are worth nothing), and
                    // the block does not end while a copy is on its way
                    ok = false;
                    pt = all;
                    for (uint32_t i = step; i < asked; ++i)
                        mbar_wait(bar + 8 * (i % kExStages), (i / kExStages) & 1, err, kDrainLimitNs);
                }
                ex_step<NB>(ring_ptr + stage * kExStage + ex_row(g) * kBlockBytes, xrow, live, t4, xv, acc[mat]);
                // every word of the stage has gone through a product that has been issued
                __syncwarp();
                ask(stage);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) xrow[b] += wk * kBlockWeights;
        }
        if (wk == 1) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int p = p0 + 8 * b + 2 * t4 + (i & 1), n = n0 + 16 * m + 8 * (i >> 1) + ex_row(g);
                        const float v = kGated ? silu(acc[0][m][b][i]) * acc[kMats - 1][m][b][i] : acc[0][m][b][i];
                        if (p < p1 && n < N) Y[static_cast<int64_t>(p) * N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
                    }
        } else {
            // the warps' sums: red[warp][matrix][row of x][weight row]
#pragma unroll
            for (int mat = 0; mat < kMats; ++mat)
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            red[((kw * kMats + mat) * NT + 8 * b + 2 * t4 + (i & 1)) * kExPitch + 16 * m + 8 * (i >> 1) + ex_row(g)] =
                                acc[mat][m][b][i];
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * wk) : "memory");
            for (int i = 32 * kw + lane; i < NT * kExRows / 4; i += 32 * wk) {
                const int r = i / (kExRows / 4), n = 4 * (i % (kExRows / 4));
                if (p0 + r >= p1 || n0 + n >= N) continue;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f), w = v;
                for (int k = 0; k < wk; ++k) {
                    const float* src = red + (k * kMats * NT + r) * kExPitch + n;
                    const float4 a = *reinterpret_cast<const float4*>(src);
                    v.x += a.x; v.y += a.y; v.z += a.z; v.w += a.w;
                    if (kGated) {
                        const float4 b = *reinterpret_cast<const float4*>(src + NT * kExPitch);
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

template <int NB, bool kGated>
cudaError_t launch_nb(const ExpertArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    CUtensorMap map, map2;
    if (weight_map(&map, a.W, a.rows.experts * a.N, a.K, kExRows) != Q4K_OK) return cudaErrorInvalidValue;
    map2 = map;
    if (kGated && weight_map(&map2, a.W2, a.rows.experts * a.N, a.K, kExRows) != Q4K_OK) return cudaErrorInvalidValue;
    const int64_t busy = a.rows.pairs < a.rows.experts ? a.rows.pairs : a.rows.experts, slabs = (a.N + kExRows - 1) / kExRows;
    const int KB = static_cast<int>(a.K / kBlockWeights);
    // wk, the warps that share K: few units are split further, so that every warp
    // of the GPU has some of the words on their way (8 experts of 128 with one row
    // each, gated 768 x 2048: 12.6 us with 8, 32 with 1); many are not, as the warps of
    // a unit wait for one another (64 rows for each of 128 experts of 2048 x 768: 37 us
    // with 1, 44 with 2). In between the units' count decides how full the last
    // round is (128 experts with four rows each, gated: 76, 73, 68, 72 us with 1, 2, 4, 8).
    const int64_t tiles = busy > a.rows.pairs / (8 * NB) ? busy : a.rows.pairs / (8 * NB);
    int wk = 1, per = 1;
    double best = 1e300;
    for (int w = 1; w <= kExWarps && w <= KB; w *= 2) {
        int p = static_cast<int>((228 * 1024) / (ex_smem(NB, kGated, w, a.rows.experts).total + 1024));
        const int most = ex_blocks(NB, kGated);
        p = p < most ? p : most;
        const double groups = static_cast<double>(dev.num_sms) * p * kExWarps / w;
        // the experts with rows are known on the device only: half a round is lost on average
        const double rounds = static_cast<double>(tiles * slabs) / groups + 0.5;
        const double cost = (rounds > 1.0 ? rounds : 1.0) * ((KB + w - 1) / w * (kGated ? 2 : 1) + (w > 1 ? 0.5 : 0.25));
        if (cost < best * 0.999) best = cost, wk = w, per = p;
    }
    const int64_t units = (a.rows.pairs / (8 * NB) + busy) * slabs, groups = kExWarps / wk;
    const int64_t blocks = (units + groups - 1) / groups, slots = static_cast<int64_t>(dev.num_sms) * per;
    return launch_serve(q4k_experts_kernel<NB, kGated>, dim3(static_cast<unsigned>(blocks < slots ? blocks : slots)),
                        dim3(32 * kExWarps), ex_smem(NB, kGated, wk, a.rows.experts).total, stream, pdl, 1, map, map2, a.X, a.rows,
                        static_cast<int>(a.N), static_cast<int>(a.K), wk, a.Y, dev.err);
}

template <int NB, bool kGated>
cudaError_t setup_nb() {
    return cudaFuncSetAttribute(q4k_experts_kernel<NB, kGated>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                ex_smem(NB, kGated, kExWarps, kMaxExperts).total);
}

}  // namespace

cudaError_t experts_setup(DeviceInfo&) {
    cudaError_t e = experts_gemm_setup(), r;
    if ((r = setup_nb<1, false>()) != cudaSuccess) e = r;
    if ((r = setup_nb<2, false>()) != cudaSuccess) e = r;
    if ((r = setup_nb<4, false>()) != cudaSuccess) e = r;
    if ((r = setup_nb<1, true>()) != cudaSuccess) e = r;
    if ((r = setup_nb<2, true>()) != cudaSuccess) e = r;
    if ((r = setup_nb<4, true>()) != cudaSuccess) e = r;
    return e;
}

cudaError_t launch_experts(const ExpertArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    // rows of x that an expert with rows has, if they are spread evenly
    const double mean = static_cast<double>(a.rows.pairs) / (a.rows.pairs < a.rows.experts ? a.rows.pairs : a.rows.experts);
    const bool gated = a.W2 != nullptr;
    if (mean > 24.0) return launch_experts_gemm(a, stream, dev, pdl);
    if (mean <= 5.0) return gated ? launch_nb<1, true>(a, stream, dev, pdl) : launch_nb<1, false>(a, stream, dev, pdl);
    if (mean <= 12.0) return gated ? launch_nb<2, true>(a, stream, dev, pdl) : launch_nb<2, false>(a, stream, dev, pdl);
    return gated ? launch_nb<4, true>(a, stream, dev, pdl) : launch_nb<4, false>(a, stream, dev, pdl);
}

}  // namespace q4k
