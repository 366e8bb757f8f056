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
// registers -- so the warps meet only at the end of a row tile, in shared
// memory. The positions and dimensions are the M of the products (mma.sync,
// S^T = K Q^T and O^T = V^T P^T), the rows their N of 8 or 16: few rows waste
// little, and P^T comes from S^T by one 8x8 transpose in registers. (128 rows
// per tcgen05 MMA, with a round trip through TMEM and barriers per tile, would
// be idle for the most part: the chunk kernel takes 468 us where this one takes
// 156.)
//
// 64 tokens of 40 heads over 1.02 GB of keys and values: 156 us, 6.6 TB/s (with
// rows as the M of 16-row products, twice the products and registers: 197 us);
// 2 tokens over 217 k positions, 64 wide, 445 MB: 77 us, 5.8 TB/s -- the rest is
// the plan at the start and the joining of ten parts per row tile; one token over
// 517 positions: 9.1 us, five tiles through one SM per kv head.
#include <cuda_bf16.h>

#include "q4k_attn.cuh"

namespace q4k {

constexpr int kDecKeys = 128;
constexpr int kDecWarps = 8;                    // consumers; one more warp produces
constexpr int kDecThreads = 32 * (kDecWarps + 1);
constexpr AttnCost kDecCost{2, 3, 4};  // item, snap, q_min

template <int D>
struct DecodeCfg {
    static constexpr int kTileBytes = kDecKeys * D * 2;
    static constexpr int kStageBytes = 2 * kTileBytes;  // K, V
    static constexpr int kRing = D == 128 ? 3 : 6;
    // [8 warps][8 rows][D values, reference, sum, 2 unused]: the four extra words
    // keep the eight rows and dimensions that a warp writes at once in 32 banks
    static constexpr int kJoinRow = D + 4;
    static constexpr int kOffJoin = kRing * kStageBytes;
    static constexpr int kOffBar = kOffJoin + kDecWarps * 8 * kJoinRow * 4;  // full[kRing] empty[kRing] join ifull[] iempty[]
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

// The transpose of an 8x8 matrix of 16-bit values (lane = row, column pair).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// NB: blocks of 8 rows in a row tile. U: what units of work are counted in.
template <int D, int NB, typename U>
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
    AttnWalk<U>* walk_s = reinterpret_cast<AttnWalk<U>*>(smem + Cfg::kOffMisc);
    volatile int* last_s = reinterpret_cast<volatile int*>(smem + Cfg::kOffMisc + 96);
    AttnItem* items = reinterpret_cast<AttnItem*>(smem + Cfg::kOffMisc + 112);
    static_assert(sizeof(AttnWalk<U>) <= 96 && Cfg::kOffMisc % 8 == 0 && sizeof(AttnItem) % 8 == 0, "layout");
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
    const int tt = 8 * NB / p.group;  // tokens of a row tile
    if (p.b.n > 32) {
        plan_block<KT, U>(p, tt, kDecCost, reinterpret_cast<U*>(smem), walk_s);
        fence_proxy_async_smem();  // the plan's scratch becomes the ring
    }
    __syncthreads();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const int page = 1 << p.c.page_shift;

    if (warp == kDecWarps) {
        // ---------------------------------------------------- TMA producer ---
        AttnWalk<U> w = p.b.n > 32 ? *walk_s : plan_warp<KT, U>(p, tt, kDecCost);
        AttnItem it{};
        PageIds ids;
        int slot = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        const int pages = KT >> p.c.page_shift;
        const uint32_t page_bytes = static_cast<uint32_t>(page) * D * 2;
        for (int n_items = 0; ok; ++n_items) {
            const bool more = next_item<KT, U>(p, w, tt, kDecCost, it);
            const int k = n_items % kItemRing;
            ok = __all_sync(0xffffffffu, mbar_wait(b_iempty + 8 * k, ((n_items / kItemRing) & 1) ^ 1, p.err));
            if (!ok) break;
            if (lane == 0) {
                items[k] = it;
                mbar_arrive(b_ifull + 8 * k);
            }
            if (!more) break;
            ids.begin();
            for (int i = it.i0; i < it.i1; ++i) {
                const int tile = it.keys.tile(i);
                const int pg = lane % pages, id = ids.get(p, it, tile * pages, pg);
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
    const int k_key = (((lane >> 3) & 1) << 3) + (lane & 7), k_chunk = lane >> 4;
    const int v_key = ((lane >> 4) << 3) + (lane & 7), v_chunk = (lane >> 3) & 1;
    const int l4 = lane >> 2, r2 = 2 * (lane & 3);
    constexpr int JR = Cfg::kJoinRow;
    float* join_buf = reinterpret_cast<float*>(smem + Cfg::kOffJoin);

    // the next item, and its rows' queries (lane: row l4 of each block, dimensions r2, r2 + 1, ...)
    AttnItem it{};
    uint32_t q[NB][D / 16][2];
    int n_items = 0;
    auto fetch = [&] {
        const int ik = n_items % kItemRing;
        if (!__all_sync(0xffffffffu, mbar_wait(b_ifull + 8 * ik, (n_items / kItemRing) & 1, p.err))) return false;
        it = items[ik];
        __syncwarp();
        if (lane == 0) mbar_arrive(b_iempty + 8 * ik);
        ++n_items;
        if (it.i0 == it.i1) return false;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int r = 8 * b + l4;
            const bool in = r < it.tokens * p.group;
            const uint16_t* from = p.Q + (static_cast<int64_t>(it.t_first + r / p.group) * p.heads +
                                          it.h * p.group + r % p.group) * D + r2;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                q[b][k][0] = in ? *reinterpret_cast<const uint32_t*>(from + 16 * k) : 0u;
                q[b][k][1] = in ? *reinterpret_cast<const uint32_t*>(from + 16 * k + 8) : 0u;
            }
        }
        return true;
    };
    // (one block of rows: the next item's queries are fetched while this one's
    // parts are put together; two leave no registers for that)
    bool more = fetch();
    for (; more; more = NB == 1 ? more : fetch()) {
        const AttnItem cur = it;
        const int rows = cur.tokens * p.group, p1 = cur.p0 + cur.tokens - 1;
        int pos[NB][2];  // of this lane's rows 8 b + r2, 8 b + r2 + 1
        float ref[NB][2], sum[NB][2], o[D / 16][NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * b + r2 + e;
                pos[b][e] = r < rows ? cur.p0 + r / p.group : -1;
                ref[b][e] = -INFINITY;
                sum[b][e] = 0.f;
            }
#pragma unroll
        for (int n = 0; n < D / 16; ++n)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][b][e] = 0.f;
        bool poison = false;
        for (int i = cur.i0; i < cur.i1; ++i) {
            const int j0 = cur.keys.tile(i) * KT + 16 * warp;
            if (!__all_sync(0xffffffffu, mbar_wait(b_full + 8 * slot, phase, p.err))) return;
            const uint32_t ks = sbase + slot * Cfg::kStageBytes + slice, vs = ks + Cfg::kTileBytes;
            // (positions below 0 see nothing; less a large window they would pass -2^31)
            const bool none = j0 > p1 || (p.window > 0 && j0 + 15 <= max(cur.p0, 0) - p.window && j0 >= p.sinks);
            if (!none) {
                // scores: one block of rows in two chains of products, added at the end
                float s[NB][4], s1[NB][4];
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[b][e] = s1[b][e] = 0.f;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t kf[4];
                    const int chunk = 2 * k + k_chunk;
                    ldmatrix_x4(ks + (chunk >> 3) * block_stride + k_key * 128 + (((chunk & 7) ^ (k_key & 7)) << 4), kf);
#pragma unroll
                    for (int b = 0; b < NB; ++b) mma_16816(NB == 1 && (k & 1) ? s1[b] : s[b], kf, q[b][k][0], q[b][k][1]);
                }
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4 && NB == 1; ++e) s[b][e] += s1[b][e];
                const bool full = tile_is_full<16>(j0 >> 4, cur.p0, p1, p.window, p.sinks);
                if (!full) {
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!sees(pos[b][e & 1], j0 + l4 + 8 * (e >> 1), p.window, p.sinks)) s[b][e] = -INFINITY;
                    // values that are not finite: zero here, and remembered for the end
                    bool bad = false;
                    for (int e = lane; e < 16 * (D / 8); e += 32) {
                        const int row = e & 15, chunk = e >> 4;  // (the order of the chunks does not matter)
                        uint4* x = reinterpret_cast<uint4*>(smem + (vs - sbase) + (chunk >> 3) * block_stride + row * 128 + ((chunk & 7) << 4));
                        const uint4 v = *x;
                        const uint4 m = make_uint4(bf16x2_non_finite(v.x), bf16x2_non_finite(v.y), bf16x2_non_finite(v.z),
                                                   bf16x2_non_finite(v.w));
                        if ((m.x | m.y | m.z | m.w) == 0u) continue;
                        bad = true;
                        *x = make_uint4(v.x & ~((m.x >> 15) * 0xFFFFu), v.y & ~((m.y >> 15) * 0xFFFFu),
                                        v.z & ~((m.z >> 15) * 0xFFFFu), v.w & ~((m.w >> 15) * 0xFFFFu));
                    }
                    bad = __any_sync(0xffffffffu, bad);
                    if (bad) fence_proxy_async_smem();  // before the stage is written again
                    poison |= bad;
                    __syncwarp();
                }
                float top[NB][2];
                bool grow = false;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = fmaxf(s[b][e], s[b][2 + e]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                        top[b][e] = m * p.scale_log2;
                        grow |= top[b][e] > ref[b][e] + 8.f || (ref[b][e] == -INFINITY && top[b][e] > ref[b][e]);
                    }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const bool g = top[b][e] > ref[b][e] + 8.f || (ref[b][e] == -INFINITY && top[b][e] > ref[b][e]);
                            const float f = g ? ex2(ref[b][e] - top[b][e]) : 1.f;
                            if (g) ref[b][e] = top[b][e];
                            sum[b][e] *= f;
#pragma unroll
                            for (int n = 0; n < D / 16; ++n) {
                                o[n][b][e] *= f;
                                o[n][b][2 + e] *= f;
                            }
                        }
                }
                // A weight is the sum of two bf16, 16 bits: one would add as much error
                // as the output's own rounding, and here the tensor core has time for
                // both. The upper is cut off, not rounded, and the lower is not 0 unless
                // the weight is, so that both parts of an infinite value's product have its sign.
                uint32_t pt[NB][2], pt_lo[NB][2];
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const float z0 = ref[b][0] == -INFINITY ? 0.f : ref[b][0], z1 = ref[b][1] == -INFINITY ? 0.f : ref[b][1];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x0 = ex2(fmaf(s[b][2 * e], p.scale_log2, -z0)), x1 = ex2(fmaf(s[b][2 * e + 1], p.scale_log2, -z1));
                        sum[b][0] += x0;
                        sum[b][1] += x1;
                        const uint32_t u0 = __float_as_uint(x0) & 0xFFFF0000u, u1 = __float_as_uint(x1) & 0xFFFF0000u;
                        constexpr float kLeast = 1.17549435e-38f;  // 2^-126
                        const __nv_bfloat162 lo = __floats2bfloat162_rn(
                            fmaxf(x0 - __uint_as_float(u0), fminf(x0, kLeast)), fmaxf(x1 - __uint_as_float(u1), fminf(x1, kLeast)));
                        pt[b][e] = transpose_8x8(u0 >> 16 | u1);
                        pt_lo[b][e] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&lo));
                    }
                }
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    uint32_t vf[4];
                    const int chunk = 2 * n + v_chunk;
                    ldmatrix_x4_trans(vs + (chunk >> 3) * block_stride + v_key * 128 + (((chunk & 7) ^ (v_key & 7)) << 4), vf);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        mma_16816(o[n][b], vf, pt[b][0], pt[b][1]);
                        mma_16816(o[n][b], vf, pt_lo[b][0], pt_lo[b][1]);
                    }
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
            for (int i = cur.i0; i < cur.i1; ++i) {
                const int j0 = cur.keys.tile(i) * KT + 16 * warp;
                if (tile_is_full<16>(j0 >> 4, cur.p0, p1, p.window, p.sinks)) continue;
                for (int k = j0; k < j0 + 16 && k < cur.len; ++k) {
                    const int id = p.c.table[cur.row + (k >> p.c.page_shift)];
                    if (id < 0 || id >= p.c.n_pages) continue;
                    const uint16_t* v = p.c.v + id * p.c.page_stride + ((static_cast<int64_t>(cur.h) << p.c.page_shift) + (k & (page - 1))) * D + l4;
#pragma unroll
                    for (int n = 0; n < D / 16; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = __uint_as_float(static_cast<uint32_t>(v[16 * n + 8 * (e >> 1)]) << 16);
                            if (!isfinite(x)) {
#pragma unroll
                                for (int b = 0; b < NB; ++b)
                                    if (sees(pos[b][e & 1], k, p.window, p.sinks)) o[n][b][e] += x;
                            }
                        }
                }
            }
        }
        if (NB == 1) more = fetch();
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) sum[b][e] += __shfl_xor_sync(0xffffffffu, sum[b][e], d);
        // the warps' results: eight rows at a time through shared memory, a warp
        // per row adds them up
        const bool whole = cur.i0 == 0 && cur.i1 == cur.keys.n;
        constexpr int V = D / 32;  // consecutive columns per lane
        auto store = [&](int r, const float (&x)[V], float total) {
            const float inv = total == 0.f ? 0.f : 1.f / total;
            uint16_t* to = p.out + (static_cast<int64_t>(cur.t_first + r / p.group) * p.heads + cur.h * p.group + r % p.group) * D + V * lane;
            uint32_t y[V / 2];
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * e] * inv, x[2 * e + 1] * inv);
                y[e] = *reinterpret_cast<const uint32_t*>(&v);
            }
            if constexpr (V == 4)
                *reinterpret_cast<uint2*>(to) = make_uint2(y[0], y[1]);
            else
                *reinterpret_cast<uint32_t*>(to) = y[0];
        };
        auto part = [&](int cta) { return p.scratch + static_cast<int64_t>(cur.slot(cta)) * Cfg::kPartFloats; };
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if (8 * b >= rows) break;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float* mine = join_buf + (warp * 8 + r2 + e) * JR;
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    mine[16 * n + l4] = o[n][b][e];
                    mine[16 * n + 8 + l4] = o[n][b][2 + e];
                }
                if (l4 == 0) {
                    mine[D] = ref[b][e];
                    mine[D + 1] = sum[b][e];
                }
            }
            if (!join()) return;
            const int r = 8 * b + warp;
            if (r < rows) {
                float top = -INFINITY;
#pragma unroll
                for (int k = 0; k < kDecWarps; ++k) top = fmaxf(top, join_buf[(k * 8 + warp) * JR + D]);
                const float z = top == -INFINITY ? 0.f : top;
                float x[V], total = 0.f;
#pragma unroll
                for (int e = 0; e < V; ++e) x[e] = 0.f;
#pragma unroll
                for (int k = 0; k < kDecWarps; ++k) {
                    const float* from = join_buf + (k * 8 + warp) * JR;
                    const float f = ex2(from[D] - z);
                    total = fmaf(from[D + 1], f, total);
#pragma unroll
                    for (int e = 0; e < V; ++e) x[e] = fmaf(from[V * lane + e], f, x[e]);
                }
                if (whole) {
                    store(r, x, total);
                } else {
                    float* to = part(blockIdx.x);
#pragma unroll
                    for (int e = 0; e < V; ++e) __stcg(to + r * D + V * lane + e, x[e]);
                    if (lane == 0) {
                        __stcg(to + 16 * D + r, top);
                        __stcg(to + 16 * D + 16 + r, total);
                    }
                }
            }
            if ((whole || 8 * (b + 1) < rows) && !join()) return;  // the buffer is written again
        }
        if (whole) continue;
        // part of a row tile: the last CTA to arrive adds the parts up in the CTAs' order
        __threadfence();
        if (!join()) return;
        if (threadIdx.x == 0) {
            uint32_t* count = p.counters + cur.first;
            const bool last = atomicAdd(count, 1u) == static_cast<uint32_t>(cur.last - cur.first);
            if (last) *count = 0u;  // as the next call expects it
            __threadfence();
            *last_s = last;
        }
        if (!join()) return;
        if (!*last_s) continue;
        for (int r = warp; r < rows; r += kDecWarps) {
            float top = -INFINITY;
            for (int cta = cur.first + lane; cta <= cur.last; cta += 32) top = fmaxf(top, __ldcg(part(cta) + 16 * D + r));
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float z = top == -INFINITY ? 0.f : top;
            float x[V], total = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) x[e] = 0.f;
#pragma unroll 4
            for (int cta = cur.first; cta <= cur.last; ++cta) {
                const float* from = part(cta);
                const float f = ex2(__ldcg(from + 16 * D + r) - z);
                total = fmaf(__ldcg(from + 16 * D + 16 + r), f, total);
#pragma unroll
                for (int e = 0; e < V; ++e) x[e] = fmaf(__ldcg(from + r * D + V * lane + e), f, x[e]);
            }
            store(r, x, total);
        }
    }
}

// ------------------------------------------------------------------ host ---

template <int D>
static cudaError_t launch_d(const AttnParams& p, int rows, cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    CUtensorMap mk, mv;
    if (!encode_pages(&mk, p.c.k, p.c, D, D / 64) || !encode_pages(&mv, p.c.v, p.c, D, D / 64))
        return cudaErrorInvalidValue;
    const int blocks = rows <= 8 ? 1 : 2;
    const bool wide = count_wide(p, 8 * blocks / p.group, kDecKeys, kDecCost);
    auto kernel = blocks == 1 ? (wide ? q4k_attn_decode_kernel<D, 1, uint64_t> : q4k_attn_decode_kernel<D, 1, uint32_t>)
                              : (wide ? q4k_attn_decode_kernel<D, 2, uint64_t> : q4k_attn_decode_kernel<D, 2, uint32_t>);
    return launch_serve(kernel, dim3(dev.num_sms),
                        dim3(kDecThreads), DecodeCfg<D>::kSmem, stream, pdl, 1, p, mk, mv);
}

cudaError_t launch_attn_decode(const AttnParams& p, int rows, int head_dim, cudaStream_t stream,
                               const DeviceInfo& dev, int pdl) {
    return head_dim == 64 ? launch_d<64>(p, rows, stream, dev, pdl) : launch_d<128>(p, rows, stream, dev, pdl);
}

cudaError_t attn_decode_setup() {
    cudaError_t e = cudaSuccess, r;
#define Q4K_SET(D, NB, U)                                                                                      \
    if ((r = cudaFuncSetAttribute(q4k_attn_decode_kernel<D, NB, U>, cudaFuncAttributeMaxDynamicSharedMemorySize, \
                                  DecodeCfg<D>::kSmem)) != cudaSuccess)                                        \
        e = r;
    Q4K_SET(64, 1, uint32_t) Q4K_SET(64, 2, uint32_t) Q4K_SET(128, 1, uint32_t) Q4K_SET(128, 2, uint32_t)
    Q4K_SET(64, 1, uint64_t) Q4K_SET(64, 2, uint64_t) Q4K_SET(128, 1, uint64_t) Q4K_SET(128, 2, uint64_t)
#undef Q4K_SET
    return e;
}

}  // namespace q4k
