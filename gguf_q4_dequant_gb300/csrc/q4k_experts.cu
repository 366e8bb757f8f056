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
// read once) and the issue slots; per 16 rows x 256 k a warp issues about 240
// instructions for 8 rows of x. So the work is laid out for the words: a warp
// owns 32 weight rows (a gated product's 16 of each matrix) and every W-th
// super-block, streams them through a ring of its own with TMA, and the warps
// of a block meet once per unit, to add their sums in shared memory in warp
// order. A unit is (expert, 32 weight rows, up to 8 NB rows of x); units are dealt
// out to resident blocks, the next unit's words on their way during this one's
// end.
#include <cuda_bf16.h>

#include "q4k_device.cuh"
#include "q4k_experts.h"
#include "q4k_serve.h"

namespace q4k {

constexpr int kExWarps = 8;                            // warps of a block at most (each a share of K)
constexpr int kExRows = 32;                            // weight rows of a unit
constexpr int kExStage = kExRows * kBlockBytes;        // 4608
constexpr int kExStages = 2;
constexpr int kExPitch = kExRows + 8;                  // floats of a token's row of partial sums

struct ExSmem {
    int ring, red, starts, tiles, bars, total;
};
__host__ __device__ inline ExSmem ex_smem(int warps, int NB, int experts) {
    ExSmem s;
    s.ring = 0;
    s.red = s.ring + warps * kExStages * kExStage;
    s.bars = s.red + warps * 8 * NB * kExPitch * 4;
    s.starts = s.bars + warps * kExStages * 8;
    s.tiles = s.starts + 4 * (experts + 1);
    s.total = s.tiles + 4 * (experts + 1);
    return s;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Physical row of an MMA operand's row: consecutive weight rows of a fragment two
// rows apart, so that eight lanes' words of a 144-byte row lie in different banks.
__device__ __forceinline__ int ex_row(int g) { return ((g & 3) << 1) | (g >> 2); }

template <int NB, bool kGated>
__global__ void __launch_bounds__(32 * kExWarps, NB == 4 ? 1 : 2)
    q4k_experts_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap map2, const uint16_t* X,
                       const ExpertRows rows, int N, int K, uint16_t* Y, unsigned int* err) {
    constexpr int NT = 8 * NB;                        // rows of x of a unit
    constexpr int kSlab = kGated ? kExRows / 2 : kExRows;  // output columns of a unit
    extern __shared__ __align__(128) uint8_t ex_smem_raw[];
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const ExSmem at = ex_smem(warps, NB, rows.experts);
    float* red = reinterpret_cast<float*>(ex_smem_raw + at.red);
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
    // the experts' rows (whatever the array holds, inside [0, pairs] and ascending),
    // and the row tiles before each expert
    for (int e = threadIdx.x; e <= rows.experts; e += blockDim.x) starts[e] = min(max(rows.starts[e], 0), rows.pairs);
    __syncthreads();
    if (warp == 0) expert_tiles<NT>(starts, tiles, rows.experts, lane);
    __syncthreads();
    const int slabs = (N + kSlab - 1) / kSlab;
    const int64_t units = static_cast<int64_t>(tiles[rows.experts]) * slabs;
    const int KB = K / kBlockWeights;

    // A unit: its expert by bisection, then (column slab, row tile), the row tiles
    // of a slab side by side so that its words come from memory once.
    auto unit_of = [&](int64_t u, int& e, int& n0, int& p0, int& p1) {
        e = expert_of(tiles, rows.experts, static_cast<int>(u / slabs));
        const int mt = tiles[e + 1] - tiles[e];
        const int in = static_cast<int>(u - static_cast<int64_t>(tiles[e]) * slabs);
        n0 = in / mt * kSlab;
        p0 = starts[e] + in % mt * NT;
        p1 = min(p0 + NT, starts[e + 1]);
    };

    // the producer's place: the next (unit, super-block) of this warp to be asked for
    int64_t pu = blockIdx.x;
    int pkb = warp, prow = 0;
    if (pu < units) {
        int e, n0, p0, p1;
        unit_of(pu, e, n0, p0, p1);
        prow = e * N + n0;
    }
    const uint64_t policy = policy_evict_first();
    uint32_t asked = 0, step = 0;
    auto ask = [&](int stage) {  // the whole warp; nothing when the units are through
        if (pu >= units) return;
        ++asked;
        if (lane == 0) {
            mbar_arrive_expect_tx(bar + 8 * stage, kExStage);
            const uint32_t dst = ring + stage * kExStage;
            tma_load_2d_hint(dst, &map, pkb * kBlockBytes, prow, bar + 8 * stage, policy);
            if (kGated) tma_load_2d_hint(dst + kExStage / 2, &map2, pkb * kBlockBytes, prow, bar + 8 * stage, policy);
        }
        pkb += warps;
        if (pkb >= KB) {
            pkb = warp;
            pu += gridDim.x;
            if (pu < units) {
                int e, n0, p0, p1;
                unit_of(pu, e, n0, p0, p1);
                prow = e * N + n0;
            }
        }
    };
#pragma unroll
    for (int i = 0; i < kExStages; ++i) ask(i);

    const int g = lane >> 2, t4 = lane & 3;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        int e, n0, p0, p1;
        unit_of(u, e, n0, p0, p1);
        float acc[2][NB][4] = {};
        const uint16_t* xrow[NB];
        bool live[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            live[b] = p0 + 8 * b + g < p1;
            xrow[b] = X + static_cast<int64_t>(live[b] ? p0 + 8 * b + g : p0) * K + 8 * t4;
        }
        for (int kb = warp; kb < KB; kb += warps, ++step) {
            const int stage = step % kExStages;
            // this lane's x of a chunk of 64 k: k = 64 c + 32 h + 8 t4 .. + 7 of row g
            uint4 xv[2][NB][2];
            auto load_x = [&](int c, uint4 (&v)[NB][2]) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        v[b][h] = live[b] ? *reinterpret_cast<const uint4*>(xrow[b] + kb * kBlockWeights + 64 * c + 32 * h)
                                          : make_uint4(0, 0, 0, 0);
            };
            load_x(0, xv[0]);
            if (ok && !__all_sync(0xffffffffu, mbar_wait(bar + 8 * stage, (step / kExStages) & 1, err))) {
                // the words did not come: nothing more is asked for (the sums are worth nothing), and
                // the block does not end while a copy is on its way
                ok = false;
                pu = units;
                for (uint32_t s = step; s < asked; ++s)
                    mbar_wait(bar + 8 * (s % kExStages), (s / kExStages) & 1, err, kDrainLimitNs);
            }
            const uint8_t* wrow = ring_ptr + stage * kExStage + ex_row(g) * kBlockBytes;
            uint4 head[2][2];
            ScaleBytes sb[2][2];
            float d[2][2];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    head[m][r] = *reinterpret_cast<const uint4*>(wrow + (16 * m + 8 * r) * kBlockBytes);
                    sb[m][r] = decode_scales(head[m][r].y, head[m][r].z, head[m][r].w);
                    d[m][r] = half_lo(head[m][r].x) * exp2i(69);
                }
            float low[2][NB][4] = {};  // sum over j of m_j (sum of x)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (c < 3) load_x(c + 1, xv[(c + 1) & 1]);
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
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int j = 2 * c + h;
                        const uint32_t mask = h ? 0x00F000F0u : 0x000F000Fu;
                        float s[2];
                        uint32_t mn[4];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const uint32_t scw = j < 4 ? sb[m][r].sc_lo : sb[m][r].sc_hi;
                            const uint32_t mw = j < 4 ? sb[m][r].m_lo : sb[m][r].m_hi;
                            s[r] = byte_to_float(scw, j & 3) * (h ? d[m][r] * 0.0625f : d[m][r]);
                            mn[r] = mn[r + 2] = __byte_perm(mw, 0, (j & 3) * 0x0101 | 0x4040);
                        }
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            float f[4] = {};
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t a4[4] = {p[i][0] & mask, p[i][1] & mask, p[i][2] & mask, p[i][3] & mask};
                                mma_bf16(f, a4, xs[b][h][2 * i], xs[b][h][2 * i + 1]);
                            }
#pragma unroll
                            for (int i = 0; i < 2; ++i) mma_bf16(low[m][b], mn, xs[b][h][2 * i], xs[b][h][2 * i + 1]);
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
                const float lo0 = half_hi(head[m][0].x) * exp2i(69), lo1 = half_hi(head[m][1].x) * exp2i(69);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    acc[m][b][0] = fmaf(-lo0, low[m][b][0], acc[m][b][0]);
                    acc[m][b][1] = fmaf(-lo0, low[m][b][1], acc[m][b][1]);
                    acc[m][b][2] = fmaf(-lo1, low[m][b][2], acc[m][b][2]);
                    acc[m][b][3] = fmaf(-lo1, low[m][b][3], acc[m][b][3]);
                }
            }
            // every word of the stage has gone through a product that has been issued
            __syncwarp();
            ask(stage);
        }
        // the warps' sums: red[warp][row of x][weight row]
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    red[(warp * NT + 8 * b + 2 * t4 + (i & 1)) * kExPitch + 16 * m + 8 * (i >> 1) + ex_row(g)] = acc[m][b][i];
        __syncthreads();
        const bool vec = (N & 3) == 0;
        for (int i = threadIdx.x; i < NT * kSlab / 4; i += blockDim.x) {
            const int r = i / (kSlab / 4), n = 4 * (i % (kSlab / 4));
            if (p0 + r >= p1 || n0 + n >= N) continue;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f), v = s;
            for (int w = 0; w < warps; ++w) {
                const float* src = red + (w * NT + r) * kExPitch + n;
                const float4 a = *reinterpret_cast<const float4*>(src);
                s.x += a.x; s.y += a.y; s.z += a.z; s.w += a.w;
                if (kGated) {
                    const float4 b = *reinterpret_cast<const float4*>(src + kSlab);
                    v.x += b.x; v.y += b.y; v.z += b.z; v.w += b.w;
                }
            }
            if (kGated) {
                s.x = silu(s.x) * v.x;
                s.y = silu(s.y) * v.y;
                s.z = silu(s.z) * v.z;
                s.w = silu(s.w) * v.w;
            }
            const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
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
        __syncthreads();
    }
}

// ------------------------------------------------------------------ host ---

namespace {

template <int NB, bool kGated>
cudaError_t launch_nb(const ExpertArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    constexpr int slab = kGated ? kExRows / 2 : kExRows;
    CUtensorMap map, map2;
    if (weight_map(&map, a.W, a.rows.experts * a.N, a.K, slab) != Q4K_OK) return cudaErrorInvalidValue;
    map2 = map;
    if (kGated && weight_map(&map2, a.W2, a.rows.experts * a.N, a.K, slab) != Q4K_OK) return cudaErrorInvalidValue;
    // the warps of a block share out the super-blocks evenly
    const int KB = static_cast<int>(a.K / kBlockWeights), rounds = (KB + kExWarps - 1) / kExWarps;
    const int warps = (KB + rounds - 1) / rounds;
    const int smem = ex_smem(warps, NB, a.rows.experts).total;
    int per = 228 * 1024 / (smem + 1024), by_warps = (NB == 4 ? 8 : 16) / warps;
    per = per < by_warps ? per : by_warps;
    const int64_t busy = a.rows.pairs < a.rows.experts ? a.rows.pairs : a.rows.experts;
    const int64_t most = (a.rows.pairs / (8 * NB) + busy) * ((a.N + slab - 1) / slab);
    const int64_t slots = static_cast<int64_t>(dev.num_sms) * (per < 1 ? 1 : per);
    return launch_serve(q4k_experts_kernel<NB, kGated>, dim3(static_cast<unsigned>(most < slots ? most : slots)),
                        dim3(32 * warps), smem, stream, pdl, 1, map, map2, a.X, a.rows, static_cast<int>(a.N),
                        static_cast<int>(a.K), a.Y, dev.err);
}

template <int NB, bool kGated>
cudaError_t setup_nb() {
    return cudaFuncSetAttribute(q4k_experts_kernel<NB, kGated>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                ex_smem(kExWarps, NB, kMaxExperts).total);
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
