// q4k_attn_decode.cu -- attention for few rows per kv head: the single tokens
// of a decode step (tokens x query heads of a kv head up to 16 per row tile).
//
// Every key and value is read once and used by a handful of rows, so the bound
// is the memory's rate: 4 D G flops per 4 D bytes leave the tensor pipe mostly
// idle whichever instruction feeds it. What matters is that loads never pause.
// One CTA per SM: a producer warp keeps a ring of three 128-position K and V
// tiles (192 KB at head_dim 128) on its way, across item boundaries, and eight
// consumer warps take 16 positions of each tile. A warp works alone on its
// positions -- scores, running reference and sum, weighted values, all in
// registers (mma.sync, 16 rows) -- so the warps meet only at the end of a row
// tile, in shared memory. The row count is too small for tcgen05 (128 rows per
// MMA, and a round trip through TMEM and barriers per tile).
#include <cuda_bf16.h>

#include "q4k_attn.cuh"

namespace q4k {

constexpr int kDecKeys = 128;
constexpr int kDecWarps = 8;                    // consumers; one more warp produces
constexpr int kDecThreads = 32 * (kDecWarps + 1);

template <int D>
struct DecodeCfg {
    static constexpr int kTileBytes = kDecKeys * D * 2;
    static constexpr int kStageBytes = 2 * kTileBytes;  // K, V
    static constexpr int kRing = D == 128 ? 3 : 6;
    static constexpr int kOffJoin = kRing * kStageBytes;          // [8 warps][8 rows][D]
    static constexpr int kOffRef = kOffJoin + kDecWarps * 8 * D * 4;   // [8 warps][16] references, sums
    static constexpr int kOffBar = kOffRef + kDecWarps * 16 * 8;  // full[kRing] empty[kRing] join ifull[] iempty[]
    static constexpr int kOffMisc = kOffBar + 8 * (2 * kRing + 2 + 2 * kItemRing);
    static constexpr int kSmem = kOffMisc + 112 + kItemRing * sizeof(AttnItem) + 1024;
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(kMaxBatch * 8 <= kRing * kStageBytes, "the plan's scratch is the ring");
    static constexpr int kPartFloats = 16 * (D + 2);
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// d (16 x 8) += a (16 x 16) b (16 x 8), bf16 in, fp32 out.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(kDecThreads, 1)
    q4k_attn_decode_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap map_k,
                           const __grid_constant__ CUtensorMap map_v) {
    using Cfg = DecodeCfg<D>;
    constexpr int KT = kDecKeys, R = Cfg::kRing;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t* smem = smem_raw + pad;
    const uint32_t sbase = raw + pad;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const uint32_t b_full = sbase + Cfg::kOffBar;
    const uint32_t b_empty = b_full + 8 * R;
    const uint32_t b_join = b_empty + 8 * R;
    const uint32_t b_ifull = b_join + 8;
    const uint32_t b_iempty = b_ifull + 8 * kItemRing;
    AttnWalk* walk_s = reinterpret_cast<AttnWalk*>(smem + Cfg::kOffMisc);
    volatile int* last_s = reinterpret_cast<volatile int*>(smem + Cfg::kOffMisc + 96);
    AttnItem* items = reinterpret_cast<AttnItem*>(smem + Cfg::kOffMisc + 112);
    static_assert(sizeof(AttnWalk) <= 96 && sizeof(AttnItem) % 8 == 0, "layout");
    if (threadIdx.x == 0) {
        for (int i = 0; i < R; ++i) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, kDecWarps);
        }
        mbar_init(b_join, kDecWarps);
        for (int i = 0; i < kItemRing; ++i) {
            mbar_init(b_ifull + 8 * i, 1);
            mbar_init(b_iempty + 8 * i, kDecWarps);
        }
        fence_barrier_init();
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
    }
    pdl_wait();
    const int tt = 16 / p.group;  // tokens of a row tile
    plan_units<KT>(p, tt, reinterpret_cast<int64_t*>(smem), walk_s);
    fence_proxy_async_smem();  // the plan's scratch becomes the ring
    __syncthreads();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const int page = 1 << p.c.page_shift;

    if (warp == kDecWarps) {
        // ---------------------------------------------------- TMA producer ---
        AttnWalk w = *walk_s;
        AttnItem it{};
        int slot = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        const int pages = KT >> p.c.page_shift;
        const uint32_t page_bytes = static_cast<uint32_t>(page) * D * 2;
        for (int n_items = 0; ok; ++n_items) {
            const bool more = next_item<KT>(p, w, tt, it);
            const int k = n_items % kItemRing;
            ok = __all_sync(0xffffffffu, mbar_wait(b_iempty + 8 * k, ((n_items / kItemRing) & 1) ^ 1, p.err));
            if (!ok) break;
            if (lane == 0) {
                items[k] = it;
                mbar_arrive(b_ifull + 8 * k);
            }
            if (!more) break;
            for (int i = it.i0; i < it.i1; ++i) {
                const int tile = it.keys.tile(i);
                const int pg = lane % pages;
                const int64_t idx = static_cast<int64_t>(tile) * pages + pg;
                int id = -1;
                if (idx << p.c.page_shift < it.len) id = p.c.table[it.row + idx];
                if (id < 0 || id >= p.c.n_pages) id = -1;  // fills zeros
                ok = __all_sync(0xffffffffu, mbar_wait(b_empty + 8 * slot, phase ^ 1, p.err));
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(b_full + 8 * slot, Cfg::kStageBytes);
                __syncwarp();
                if (lane < 2 * pages)
                    tma_load_5d(sbase + slot * Cfg::kStageBytes + (lane < pages ? 0 : Cfg::kTileBytes) + pg * page_bytes,
                                lane < pages ? &map_k : &map_v, 0, 0, 0, it.h, id, b_full + 8 * slot);
                ++issued;
                if (++slot == R) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
        for (int k = 0; k < R && k < issued; ++k) {  // every copy has landed before the CTA ends
            if (slot == 0) phase ^= 1;
            slot = slot == 0 ? R - 1 : slot - 1;
            mbar_wait(b_full + 8 * slot, phase, p.err, kDrainLimitNs);
        }
        return;
    }

    // ------------------------------------------------------------ consumers ---
    int slot = 0;
    uint32_t phase = 0, join_phase = 0;
    auto join = [&] {  // all consumer warps
        __syncwarp();
        if (lane == 0) mbar_arrive(b_join);
        const bool done = __all_sync(0xffffffffu, mbar_wait(b_join, join_phase, p.err));
        join_phase ^= 1;
        return done;
    };
    // this warp's 16 positions of a tile
    const uint32_t slice = static_cast<uint32_t>((16 * warp) / page) * page * D * 2 + ((16 * warp) % page) * 128;
    const uint32_t block_stride = static_cast<uint32_t>(page) * 128;  // the next 64 dimensions
    const int k_key = ((lane >> 4) << 3) + (lane & 7), k_chunk = (lane >> 3) & 1;
    const int v_key = (((lane >> 3) & 1) << 3) + (lane & 7), v_chunk = lane >> 4;
    const int ra = lane >> 2, rb = ra + 8;
    float* join_o = reinterpret_cast<float*>(smem + Cfg::kOffJoin);
    float* join_ref = reinterpret_cast<float*>(smem + Cfg::kOffRef);
    float* join_sum = join_ref + kDecWarps * 16;

    for (int n_items = 0;; ++n_items) {
        // done with the item before
        __syncwarp();
        if (n_items > 0 && lane == 0) mbar_arrive(b_iempty + 8 * ((n_items - 1) % kItemRing));
        const int ik = n_items % kItemRing;
        if (!__all_sync(0xffffffffu, mbar_wait(b_ifull + 8 * ik, (n_items / kItemRing) & 1, p.err))) return;
        const AttnItem it = items[ik];
        if (it.i1 == it.i0) return;
        const int rows = it.tokens * p.group, p1 = it.p0 + it.tokens - 1;
        uint32_t q[D / 16][4];
        {
            const uint16_t* qa = p.Q + (static_cast<int64_t>(it.t_first + ra / p.group) * p.heads + it.h * p.group + ra % p.group) * D + 2 * (lane & 3);
            const uint16_t* qb = p.Q + (static_cast<int64_t>(it.t_first + rb / p.group) * p.heads + it.h * p.group + rb % p.group) * D + 2 * (lane & 3);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                q[k][0] = ra < rows ? *reinterpret_cast<const uint32_t*>(qa + 16 * k) : 0u;
                q[k][1] = rb < rows ? *reinterpret_cast<const uint32_t*>(qb + 16 * k) : 0u;
                q[k][2] = ra < rows ? *reinterpret_cast<const uint32_t*>(qa + 16 * k + 8) : 0u;
                q[k][3] = rb < rows ? *reinterpret_cast<const uint32_t*>(qb + 16 * k + 8) : 0u;
            }
        }
        const int pa = ra < rows ? it.p0 + ra / p.group : -1, pb = rb < rows ? it.p0 + rb / p.group : -1;
        float o[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
        float ref_a = -INFINITY, ref_b = -INFINITY, sum_a = 0.f, sum_b = 0.f;
        bool poison = false;
        for (int i = it.i0; i < it.i1; ++i) {
            const int j0 = it.keys.tile(i) * KT + 16 * warp;
            if (!__all_sync(0xffffffffu, mbar_wait(b_full + 8 * slot, phase, p.err))) return;
            const uint32_t ks = sbase + slot * Cfg::kStageBytes + slice, vs = ks + Cfg::kTileBytes;
            const bool none = j0 > p1 || (p.window > 0 && j0 + 15 <= it.p0 - p.window && j0 >= p.sinks);
            if (!none) {
                float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t kf[4];
                    const int chunk = 2 * k + k_chunk;
                    ldmatrix_x4(ks + (chunk >> 3) * block_stride + k_key * 128 + (((chunk & 7) ^ (k_key & 7)) << 4), kf);
                    mma_16816(s[0], q[k], kf[0], kf[1]);
                    mma_16816(s[1], q[k], kf[2], kf[3]);
                }
                const bool full = tile_is_full<16>(j0 >> 4, it.p0, p1, p.window, p.sinks);
                if (!full) {
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int key = j0 + 8 * b + 2 * (lane & 3) + e;
                            if (!sees(pa, key, p.window, p.sinks)) s[b][e] = -INFINITY;
                            if (!sees(pb, key, p.window, p.sinks)) s[b][2 + e] = -INFINITY;
                        }
                    // values that are not finite: zero here, and remembered for the end
                    bool bad = false;
                    for (int e = lane; e < 16 * (D / 8); e += 32) {
                        const int row = e & 15, chunk = e >> 4;  // (the order of the chunks does not matter)
                        uint4* x = reinterpret_cast<uint4*>(smem + (vs - sbase) + (chunk >> 3) * block_stride + row * 128 + ((chunk & 7) << 4));
                        uint4 v = *x;
                        uint32_t* vw = &v.x;
                        uint32_t any = 0;
#pragma unroll
                        for (int c = 0; c < 4; ++c) any |= bf16x2_non_finite(vw[c]);
                        if (any) {
                            bad = true;
#pragma unroll
                            for (int c = 0; c < 4; ++c) vw[c] &= ~((bf16x2_non_finite(vw[c]) >> 15) * 0xFFFFu);
                            *x = v;
                        }
                    }
                    bad = __any_sync(0xffffffffu, bad);
                    if (bad) fence_proxy_async_smem();  // before the stage is written again
                    poison |= bad;
                    __syncwarp();
                }
                float ma = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
                float mb = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
                for (int d = 1; d < 4; d <<= 1) {
                    ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, d));
                    mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, d));
                }
                ma *= p.scale_log2;
                mb *= p.scale_log2;
                const bool ga = ma > ref_a + 8.f || (ref_a == -INFINITY && ma > ref_a);
                const bool gb = mb > ref_b + 8.f || (ref_b == -INFINITY && mb > ref_b);
                if (__any_sync(0xffffffffu, ga || gb)) {
                    const float fa = ga ? ex2(ref_a - ma) : 1.f, fb = gb ? ex2(ref_b - mb) : 1.f;
                    if (ga) ref_a = ma;
                    if (gb) ref_b = mb;
                    sum_a *= fa;
                    sum_b *= fb;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][0] *= fa;
                        o[n][1] *= fa;
                        o[n][2] *= fb;
                        o[n][3] *= fb;
                    }
                }
                const float za = ref_a == -INFINITY ? 0.f : ref_a, zb = ref_b == -INFINITY ? 0.f : ref_b;
                uint32_t a[4];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float x0 = ex2(fmaf(s[b][0], p.scale_log2, -za)), x1 = ex2(fmaf(s[b][1], p.scale_log2, -za));
                    const float y0 = ex2(fmaf(s[b][2], p.scale_log2, -zb)), y1 = ex2(fmaf(s[b][3], p.scale_log2, -zb));
                    sum_a += x0 + x1;
                    sum_b += y0 + y1;
                    const __nv_bfloat162 xp = __floats2bfloat162_rn(x0, x1), yp = __floats2bfloat162_rn(y0, y1);
                    a[2 * b] = *reinterpret_cast<const uint32_t*>(&xp);
                    a[2 * b + 1] = *reinterpret_cast<const uint32_t*>(&yp);
                }
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    uint32_t vf[4];
                    const int chunk = 2 * n + v_chunk;
                    ldmatrix_x4_trans(vs + (chunk >> 3) * block_stride + v_key * 128 + (((chunk & 7) ^ (v_key & 7)) << 4), vf);
                    mma_16816(o[2 * n], a, vf[0], vf[1]);
                    mma_16816(o[2 * n + 1], a, vf[2], vf[3]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(b_empty + 8 * slot);
            if (++slot == R) {
                slot = 0;
                phase ^= 1;
            }
        }
        if (poison) {  // the zeroed values, back into the rows that see them
            for (int i = it.i0; i < it.i1; ++i) {
                const int j0 = it.keys.tile(i) * KT + 16 * warp;
                if (tile_is_full<16>(j0 >> 4, it.p0, p1, p.window, p.sinks)) continue;
                for (int k = j0; k < j0 + 16 && k < it.len; ++k) {
                    const bool sa = sees(pa, k, p.window, p.sinks), sb = sees(pb, k, p.window, p.sinks);
                    const int id = p.c.table[it.row + (k >> p.c.page_shift)];
                    if (id < 0 || id >= p.c.n_pages) continue;
                    const uint16_t* v = p.c.v + id * p.c.page_stride + ((static_cast<int64_t>(it.h) << p.c.page_shift) + (k & (page - 1))) * D + 2 * (lane & 3);
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float x = __uint_as_float(static_cast<uint32_t>(v[8 * n + e]) << 16);
                            if (!isfinite(x)) {
                                if (sa) o[n][e] += x;
                                if (sb) o[n][2 + e] += x;
                            }
                        }
                }
            }
        }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            sum_a += __shfl_xor_sync(0xffffffffu, sum_a, d);
            sum_b += __shfl_xor_sync(0xffffffffu, sum_b, d);
        }
        if ((lane & 3) == 0) {
            join_ref[16 * warp + ra] = ref_a;
            join_ref[16 * warp + rb] = ref_b;
            join_sum[16 * warp + ra] = sum_a;
            join_sum[16 * warp + rb] = sum_b;
        }
        // the warps' results: eight rows at a time through shared memory, a warp
        // per row adds them up
        const bool whole = it.i0 == 0 && it.i1 == it.keys.n;
        constexpr int V = D / 32;  // consecutive columns per lane
        auto out_row = [&](int r) {
            return p.out + (static_cast<int64_t>(it.t_first + r / p.group) * p.heads + it.h * p.group + r % p.group) * D + V * lane;
        };
        auto store = [&](int r, const float (&x)[V], float sum) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            uint32_t y[V / 2];
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * e] * inv, x[2 * e + 1] * inv);
                y[e] = *reinterpret_cast<const uint32_t*>(&v);
            }
            if constexpr (V == 4)
                *reinterpret_cast<uint2*>(out_row(r)) = make_uint2(y[0], y[1]);
            else
                *reinterpret_cast<uint32_t*>(out_row(r)) = y[0];
        };
        for (int half = 0; half < (rows > 8 ? 2 : 1); ++half) {
            float* mine = join_o + (warp * 8 + ra) * D + 2 * (lane & 3);
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                *reinterpret_cast<float2*>(mine + 8 * n) = half ? make_float2(o[n][2], o[n][3]) : make_float2(o[n][0], o[n][1]);
            if (!join()) return;
            const int r = 8 * half + warp;
            if (r < rows) {
                float top = -INFINITY;
#pragma unroll
                for (int k = 0; k < kDecWarps; ++k) top = fmaxf(top, join_ref[16 * k + r]);
                const float z = top == -INFINITY ? 0.f : top;
                float x[V], sum = 0.f;
#pragma unroll
                for (int e = 0; e < V; ++e) x[e] = 0.f;
#pragma unroll
                for (int k = 0; k < kDecWarps; ++k) {
                    const float f = ex2(join_ref[16 * k + r] - z);
                    sum = fmaf(join_sum[16 * k + r], f, sum);
                    const float* from = join_o + (k * 8 + warp) * D + V * lane;
#pragma unroll
                    for (int e = 0; e < V; ++e) x[e] = fmaf(from[e], f, x[e]);
                }
                if (whole) {
                    store(r, x, sum);
                } else {
                    float* to = p.scratch + static_cast<int64_t>(it.slot(blockIdx.x)) * Cfg::kPartFloats;
#pragma unroll
                    for (int e = 0; e < V; ++e) __stcg(to + r * D + V * lane + e, x[e]);
                    if (lane == 0) {
                        __stcg(to + 16 * D + r, top);
                        __stcg(to + 16 * D + 16 + r, sum);
                    }
                }
            }
            if (rows > 8 && !join()) return;  // the buffer is written again
        }
        if (whole) {
            if (rows <= 8 && !join()) return;
            continue;
        }
        // part of a row tile: the last CTA to arrive adds the parts up in the CTAs' order
        __threadfence();
        if (!join()) return;
        if (threadIdx.x == 0) {
            uint32_t* count = p.counters + it.first;
            const bool last = atomicAdd(count, 1u) == static_cast<uint32_t>(it.last - it.first);
            if (last) *count = 0u;  // as the next call expects it
            __threadfence();
            *last_s = last;
        }
        if (!join()) return;
        if (!*last_s) continue;
        for (int r = warp; r < rows; r += kDecWarps) {
            auto part = [&](int cta) { return p.scratch + static_cast<int64_t>(it.slot(cta)) * Cfg::kPartFloats; };
            float top = -INFINITY;
            for (int cta = it.first + lane; cta <= it.last; cta += 32) top = fmaxf(top, __ldcg(part(cta) + 16 * D + r));
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float z = top == -INFINITY ? 0.f : top;
            float x[V], sum = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) x[e] = 0.f;
#pragma unroll 4
            for (int cta = it.first; cta <= it.last; ++cta) {
                const float* from = part(cta);
                const float f = ex2(__ldcg(from + 16 * D + r) - z);
                sum = fmaf(__ldcg(from + 16 * D + 16 + r), f, sum);
#pragma unroll
                for (int e = 0; e < V; ++e) x[e] = fmaf(__ldcg(from + r * D + V * lane + e), f, x[e]);
            }
            store(r, x, sum);
        }
    }
}

// ------------------------------------------------------------------ host ---

template <int D>
static cudaError_t launch_d(const AttnParams& p, cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    CUtensorMap mk, mv;
    if (!encode_pages(&mk, p.c.k, p.c, D, D / 64) || !encode_pages(&mv, p.c.v, p.c, D, D / 64))
        return cudaErrorInvalidValue;
    return launch_serve(q4k_attn_decode_kernel<D>, dim3(dev.num_sms), dim3(kDecThreads), DecodeCfg<D>::kSmem, stream,
                        pdl, 1, p, mk, mv);
}

cudaError_t launch_attn_decode(const AttnParams& p, int head_dim, cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    return head_dim == 64 ? launch_d<64>(p, stream, dev, pdl) : launch_d<128>(p, stream, dev, pdl);
}

cudaError_t attn_decode_setup() {
    cudaError_t e = cudaFuncSetAttribute(q4k_attn_decode_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         DecodeCfg<64>::kSmem);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(q4k_attn_decode_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                DecodeCfg<128>::kSmem);
}

}  // namespace q4k
