// q4k_attn.cu -- attention of a step's new tokens over the pages of one layer:
// the chunk kernel, for many rows (tokens x query heads) per kv head.
//
// out = (sum_j 2^(s_j - r) v_j) / (sum_j 2^(s_j - r)) with s_j = scale log2(e)
// q.k_j and a running reference r per row: r follows the row's largest score,
// but only once it has grown by 2^8 or more, so that the accumulated sums are
// rarely rescaled (the weights stay below 2^8, exact as far as fp32 and bf16 go).
//
// An item is 2 x 128 rows of one kv head: each half is whole tokens times the
// G query heads that share the kv head, so every key and value tile (128
// positions) is used by 256 rows. Two products per half and key tile, both
// 128 x 128 x head_dim on tcgen05:
//   S = Q K^T   Q and K from shared memory (K-major, 128-byte swizzle), S in TMEM
//   O += P V    P (bf16) in TMEM over S's columns, V from shared memory as the
//               pages hold it (rows are k: MN-major)
// P is rounded to bf16, as much error again as the output's own rounding (0.0023
// of the values together, 0.0017 alone): its lower half as a second product would
// be half as much work again.
// While the tensor core works for one half, the other half's 128 threads (one
// row each) turn S into P: the two halves take turns.
//
// 4096 tokens of 32 heads over 16384 positions, 128 wide: 0.59-0.60 ms for a dozen
// calls, 1.59 to 1.63 PFLOP/s; 0.62-0.64, 1.52, call after call (1380 W, power
// capped, 1.93 GHz). A key tile takes 3000 cycles for both halves, 2048 of them
// products (tensor pipe 65 %); with the softmax reduced to a copy the whole
// still takes 0.58 ms: the products are held up by shared memory, of which Q and K are read at
// 64 KB and V at 32 KB per half while the next tiles come in at 64 KB, together
// 2048 cycles at 128 bytes. Sharing K between two SMs (cta_group::2) is what
// would lift that. Two threads per row, P handed over in parts, a pipeline over
// TMEM loads and hand-ordered exponentials were no faster (0.60 to 0.88 ms).
// 2017 tokens in 8 sequences with a window of 1024: 49-52 us; 14 key tiles a CTA
// are 22 us of it, the first loads, row tiles' ends and the joining the rest.
// Joining: the half that comes last keeps its own part in TMEM, and does not
// write it out if it sees that the others have come; parts are read and written 16 bytes a
// thread (2048 tokens of one sequence 42 us; all parts written and read back, 4
// bytes a thread: 48).
//
// Warp roles: 0-3 softmax of half 0, 4-7 of half 1, 8 TMA producer (pages of
// K and V tiles, Q), 9 MMA issuer, 10-11 scan (below). K and V tiles go through one ring of
// buffers, filled page by page: the tensor map's last coordinate is the page,
// and pages past a sequence's end are asked for at page -1, which fills zeros.
//
// Values that no row may see can be NaN (pages are not cleared): scores are
// selected, not added to, and V tiles that some row sees only in part are
// searched, by two warps ahead of the MMAs, for infinities and NaN, which are
// zeroed in shared memory and added back, at the end, to the rows that do see
// them.
#include <cuda_bf16.h>

#include <algorithm>

#include "q4k_attn.cuh"

namespace q4k {

constexpr int kChunkKeys = 128;
constexpr int kChunkThreads = 384;
constexpr int kScanWarps = 2;
// Registers: the block starts with 168 a thread; the last warpgroup gives some to the softmax.
constexpr int kSoftRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftRegs + kOtherRegs <= 3 * 168, "registers");
// item, snap, q_min. With a range of 3, 4 or 5 units at least: a prompt of 512
// tokens 17.9, 15.0, 17.7 us; 64 tokens over 4000 positions 31.5, 30.4, 28.4 us
// (every part more costs the joining CTA 128 KB); steps that fill the GPU alike.
constexpr AttnCost kChunkCost{3, 1, 4};

template <int D>
struct ChunkCfg {
    static constexpr int kHalves = D / 64;                 // 64-element column blocks of a row
    static constexpr int kTileBytes = kChunkKeys * D * 2;  // one K or V tile, one half of Q
    static constexpr int kRing = D == 128 ? 4 : 8;
    static constexpr int kOffQ = 0;
    static constexpr int kOffRing = 2 * kTileBytes;
    static constexpr int kOffStage = kOffRing + kRing * kTileBytes;  // output rows, 4 KB per softmax warp
    static constexpr int kOffBar = kOffStage + 8 * 4096;
    // full[kRing] empty[kRing] qfull qempty sfull[2] pfull[2] ofull[2] wg[2] fin ifull[kItemRing] iempty[kItemRing]
    // vclean[kRing]
    static constexpr int kNumBars = 3 * kRing + 11 + 2 * kItemRing;
    static constexpr int kOffMisc = kOffBar + 8 * ((kNumBars + 1) / 2 * 2);  // walk, tmem address, flags, items
    static constexpr int kMiscBytes = 144 + kItemRing * sizeof(AttnItem);
    static constexpr int kSmem = kOffMisc + kMiscBytes + 1024;  // + alignment slack
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(kMaxBatch * 8 <= kRing * kTileBytes, "the plan's scratch is the ring");
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kColS = 0, kColO = 256;        // S (and P) 2 x 128, O 2 x D
    static constexpr int kPartFloats = (D + 2) * 128;        // a partial result of one half
};

template <int kRegs>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// U: what units of work are counted in.
template <int D, typename U>
__global__ void __launch_bounds__(kChunkThreads, 1)
    q4k_attn_chunk_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap map_q,
                          const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
    using Cfg = ChunkCfg<D>;
    constexpr int KT = kChunkKeys, R = Cfg::kRing;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t* smem = smem_raw + pad;
    const uint32_t sbase = raw + pad;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const uint32_t b_full = sbase + Cfg::kOffBar;
    const uint32_t b_empty = b_full + 8 * R;
    const uint32_t b_qfull = b_empty + 8 * R;
    const uint32_t b_qempty = b_qfull + 8;
    const uint32_t b_sfull = b_qempty + 8;
    const uint32_t b_pfull = b_sfull + 16;
    const uint32_t b_ofull = b_pfull + 16;
    const uint32_t b_wg = b_ofull + 16;
    const uint32_t b_fin = b_wg + 16;
    const uint32_t b_ifull = b_fin + 8;
    const uint32_t b_iempty = b_ifull + 8 * kItemRing;
    const uint32_t b_vclean = b_iempty + 8 * kItemRing;
    AttnWalk<U>* walk_s = reinterpret_cast<AttnWalk<U>*>(smem + Cfg::kOffMisc);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + Cfg::kOffMisc + 96);
    volatile int* poison = reinterpret_cast<volatile int*>(smem + Cfg::kOffMisc + 112);  // [4] item tags
    volatile int* last_s = reinterpret_cast<volatile int*>(smem + Cfg::kOffMisc + 128);  // [2]
    AttnItem* items = reinterpret_cast<AttnItem*>(smem + Cfg::kOffMisc + 144);
    static_assert(sizeof(AttnWalk<U>) <= 96 && Cfg::kOffMisc % 8 == 0 && sizeof(AttnItem) % 8 == 0, "layout");

    if (threadIdx.x == 0) {
        for (int i = 0; i < R; ++i) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, 1 + kScanWarps);  // the MMA's commit, the scan warps
            mbar_init(b_vclean + 8 * i, kScanWarps);
        }
        mbar_init(b_qfull, 1);
        mbar_init(b_qempty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_sfull + 8 * i, 1);
            mbar_init(b_pfull + 8 * i, 128);
            mbar_init(b_ofull + 8 * i, 1);
            mbar_init(b_wg + 8 * i, 128);
            poison[2 * i] = poison[2 * i + 1] = 0;
        }
        mbar_init(b_fin, 1);
        for (int i = 0; i < kItemRing; ++i) {
            mbar_init(b_ifull + 8 * i, 1);
            mbar_init(b_iempty + 8 * i, 9 + kScanWarps);  // MMA, softmax and scan warps
        }
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), Cfg::kTmemCols);
        tmem_relinquish();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_desc(&map_q);
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
    }
    pdl_wait();
    const int tph = 128 / p.group, tt = 2 * tph;  // tokens per half and per item
    if (p.b.n > 32) {
        plan_block<KT, U>(p, tt, kChunkCost, reinterpret_cast<U*>(smem + Cfg::kOffRing), walk_s);
        fence_proxy_async_smem();  // the plan's scratch (generic accesses) becomes the ring (TMA writes)
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (threadIdx.x == 0) pdl_launch_dependents();

    if (warp >= 8) {
        regs_dec<kOtherRegs>();
        if (warp == 8) {
            // ------------------------------------------------ TMA producer ---
            AttnWalk<U> w = p.b.n > 32 ? *walk_s : plan_warp<KT, U>(p, tt, kChunkCost);
            AttnItem it{};
            PageIds ids;
            int slot = 0, n_items = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            const int pages = KT >> p.c.page_shift;   // per key tile
            const int boxes = pages * Cfg::kHalves;
            const uint32_t page_bytes = 128u << p.c.page_shift;  // of one column block
            auto load_tile = [&](const CUtensorMap* map, int page) {
                if (!__all_sync(0xffffffffu, mbar_wait(b_empty + 8 * slot, phase ^ 1, p.err))) return false;
                if (lane == 0) mbar_arrive_expect_tx(b_full + 8 * slot, Cfg::kTileBytes);
                __syncwarp();
                if (lane < boxes) {
                    const int pg = lane % pages, cb = lane / pages;
                    tma_load_5d(sbase + Cfg::kOffRing + slot * Cfg::kTileBytes + cb * (KT * 128) + pg * page_bytes, map,
                                0, 0, cb, it.h, page, b_full + 8 * slot);
                }
                ++issued;
                if (++slot == R) {
                    slot = 0;
                    phase ^= 1;
                }
                return true;
            };
            for (;;) {
                const bool more = next_item<KT, U>(p, w, tt, kChunkCost, it);
                const int k = n_items % kItemRing;
                ok = __all_sync(0xffffffffu, mbar_wait(b_iempty + 8 * k, ((n_items / kItemRing) & 1) ^ 1, p.err));
                if (!ok) break;
                if (lane == 0) {
                    items[k] = it;
                    mbar_arrive(b_ifull + 8 * k);
                }
                if (!more) break;
                ok = __all_sync(0xffffffffu, mbar_wait(b_qempty, (n_items & 1) ^ 1, p.err));
                if (!ok) break;
                const int halves = it.tokens > tph ? 2 : 1;
                if (lane == 0)
                    mbar_arrive_expect_tx(b_qfull, static_cast<uint32_t>(halves * tph * p.group * D * 2));
                __syncwarp();
                if (lane < halves * Cfg::kHalves) {
                    const int hf = lane / Cfg::kHalves, cb = lane % Cfg::kHalves;
                    tma_load_4d(sbase + Cfg::kOffQ + hf * Cfg::kTileBytes + cb * (128 * 128), &map_q, 0,
                                it.h * p.group, it.t_first + hf * tph, cb, b_qfull);
                }
                ++n_items;
                ids.begin();
                for (int i = it.i0; ok && i < it.i1; ++i) {
                    const int tile = it.keys.tile(i);
                    const int page = ids.get(p, it, tile * pages, lane % pages);
                    ok = load_tile(&map_k, page) && load_tile(&map_v, page);
                }
                if (!ok) break;
            }
            // before the CTA may end, every copy has landed: at most the last R
            // tiles and the last Q can be on their way
            for (int k = 0; k < R && k < issued; ++k) {
                if (slot == 0) phase ^= 1;
                slot = slot == 0 ? R - 1 : slot - 1;
                mbar_wait(b_full + 8 * slot, phase, p.err, kDrainLimitNs);
            }
            if (n_items > 0) mbar_wait(b_qfull, (n_items - 1) & 1, p.err, kDrainLimitNs);
        } else if (warp == 9) {
            // -------------------------------------------------- MMA issuer ---
            constexpr uint32_t idesc_s = idesc_bf16_f32(128, KT);
            constexpr uint32_t idesc_o = idesc_bf16_f32(128, D) | kIdescBMnMajor;
            int n_items = 0, slot = 0;
            uint32_t phase = 0, p_phase[2] = {0, 0}, clean_phase = 0;  // (a bit per ring slot)
            bool ok = true;
            auto wait = [&](uint32_t bar, uint32_t ph) {
                const bool r = __all_sync(0xffffffffu, mbar_wait(bar, ph, p.err));
                tc_fence_after();
                return r;
            };
            auto scores = [&](int hf, int kslot) {  // S = Q K^T
                if (elect_one()) {
#pragma unroll
                    for (int cb = 0; cb < Cfg::kHalves; ++cb) {
                        const uint64_t a = sw128_desc(sbase + Cfg::kOffQ + hf * Cfg::kTileBytes + cb * (128 * 128));
                        const uint64_t b = sw128_desc(sbase + Cfg::kOffRing + kslot * Cfg::kTileBytes + cb * (KT * 128));
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma_bf16(tmem + Cfg::kColS + hf * 128, a + 2 * kk, b + 2 * kk, idesc_s, cb + kk > 0);
                    }
                    tc_commit(b_sfull + 8 * hf);
                }
                __syncwarp();
            };
            auto values = [&](int hf, int vslot, bool first) {  // O += P V
                if (elect_one()) {
                    const uint64_t b = sw128_desc_mn(sbase + Cfg::kOffRing + vslot * Cfg::kTileBytes, KT * 128);
#pragma unroll
                    for (int kk = 0; kk < KT / 16; ++kk)
                        tc_mma_bf16_ts(tmem + Cfg::kColO + hf * D, tmem + Cfg::kColS + hf * 128 + 8 * kk,
                                       b + kk * (16 * 128 / 16), idesc_o, !first || kk > 0);
                }
                __syncwarp();
            };
            auto commit = [&](uint32_t bar) {
                if (elect_one()) tc_commit(bar);
                __syncwarp();
            };
            for (;;) {
                const int ik = n_items % kItemRing;
                ok = wait(b_ifull + 8 * ik, (n_items / kItemRing) & 1);
                if (!ok) break;
                const int halves = items[ik].tokens > tph ? 2 : 1, n = items[ik].i1 - items[ik].i0;
                const int i0 = items[ik].i0, p0 = items[ik].p0, p1 = p0 + items[ik].tokens - 1;
                const KeyTiles keys = items[ik].keys;
                __syncwarp();
                if (lane == 0) mbar_arrive(b_iempty + 8 * ik);
                if (n == 0) break;
                ok = wait(b_qfull, n_items & 1) && wait(b_full + 8 * slot, phase);
                if (!ok) break;
                for (int hf = 0; hf < halves; ++hf) scores(hf, slot);
                commit(b_empty + 8 * slot);
                if (n == 1) commit(b_qempty);
                for (int j = 0; ok && j < n; ++j) {
                    int vslot = slot + 1 == R ? 0 : slot + 1;
                    const uint32_t vphase = vslot == 0 ? phase ^ 1 : phase;
                    int kslot = vslot + 1 == R ? 0 : vslot + 1;
                    const uint32_t kphase = kslot == 0 ? vphase ^ 1 : vphase;
                    const bool more = j + 1 < n;
                    ok = wait(b_full + 8 * vslot, vphase);
                    if (ok && !tile_is_full<KT>(keys.tile(i0 + j), p0, p1, p.window, p.sinks)) {
                        ok = wait(b_vclean + 8 * vslot, clean_phase >> vslot & 1);
                        clean_phase ^= 1u << vslot;
                    }
                    if (ok && more) ok = wait(b_full + 8 * kslot, kphase);
                    for (int hf = 0; ok && hf < halves; ++hf) {
                        ok = wait(b_pfull + 8 * hf, p_phase[hf]);
                        if (!ok) break;
                        p_phase[hf] ^= 1;
                        values(hf, vslot, j == 0);
                        if (more)
                            scores(hf, kslot);
                        else
                            commit(b_ofull + 8 * hf);
                    }
                    if (!ok) break;
                    commit(b_empty + 8 * vslot);
                    slot = vslot;
                    phase = vphase;
                    if (more) {
                        commit(b_empty + 8 * kslot);
                        if (j + 2 == n) commit(b_qempty);
                        slot = kslot;
                        phase = kphase;
                    }
                }
                if (!ok) break;
                if (++slot == R) {
                    slot = 0;
                    phase ^= 1;
                }
                ++n_items;
            }
            commit(b_fin);  // every MMA of this CTA has completed
        } else {
            // ---------------------------------------------------------- scan ---
            int slot = 0;
            uint32_t phase = 0;
            for (int n_items = 0;; ++n_items) {
                const int ik = n_items % kItemRing;
                if (!__all_sync(0xffffffffu, mbar_wait(b_ifull + 8 * ik, (n_items / kItemRing) & 1, p.err))) break;
                const int i0 = items[ik].i0, n = items[ik].i1 - i0, p0 = items[ik].p0, p1 = p0 + items[ik].tokens - 1;
                const KeyTiles keys = items[ik].keys;
                __syncwarp();
                if (lane == 0) mbar_arrive(b_iempty + 8 * ik);
                if (n == 0) break;
                bool ok = true;
                // every buffer of the ring in its turn (so that none is passed over
                // or met a round late), the V tiles of partly seen key tiles read
                for (int j = 0; ok && j < 2 * n; ++j) {
                    const int vslot = slot;
                    ok = __all_sync(0xffffffffu, mbar_wait(b_full + 8 * vslot, phase, p.err));
                    if (!ok) break;
                    if (++slot == R) {
                        slot = 0;
                        phase ^= 1;
                    }
                    if (!(j & 1) || tile_is_full<KT>(keys.tile(i0 + (j >> 1)), p0, p1, p.window, p.sinks)) {
                        if (lane == 0) mbar_arrive(b_empty + 8 * vslot);
                        continue;
                    }
                    uint4* v4 = reinterpret_cast<uint4*>(smem + Cfg::kOffRing + vslot * Cfg::kTileBytes) +
                                (threadIdx.x - 32 * 10);
                    constexpr int kStep = 32 * kScanWarps;
#pragma unroll 1
                    for (int e = 0; e < Cfg::kTileBytes / 16 / kStep; e += 8) {
                        uint4 x[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = v4[kStep * (e + i)];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint4 m = make_uint4(bf16x2_non_finite(x[i].x), bf16x2_non_finite(x[i].y),
                                                       bf16x2_non_finite(x[i].z), bf16x2_non_finite(x[i].w));
                            if ((m.x | m.y | m.z | m.w) == 0u) continue;
                            poison[(n_items + 1) & 3] = n_items + 1;
                            v4[kStep * (e + i)] = make_uint4(
                                x[i].x & ~((m.x >> 15) * 0xFFFFu), x[i].y & ~((m.y >> 15) * 0xFFFFu),
                                x[i].z & ~((m.z >> 15) * 0xFFFFu), x[i].w & ~((m.w >> 15) * 0xFFFFu));
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(b_vclean + 8 * vslot);
                        mbar_arrive(b_empty + 8 * vslot);
                    }
                }
                if (!ok) break;
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- softmax ---
        regs_inc<kSoftRegs>();
        const int hf = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lane_base + Cfg::kColS + hf * 128;
        const uint32_t t_o = tmem + lane_base + Cfg::kColO + hf * D;
        const int tok = r / p.group, g = r % p.group;
        int n_items = 0;
        uint32_t s_phase = 0, o_phase = 0, wg_phase = 0;
        bool ok = true;
        for (;;) {
            // done with the item before
            __syncwarp();
            if (n_items > 0 && lane == 0) mbar_arrive(b_iempty + 8 * ((n_items - 1) % kItemRing));
            const int ik = n_items % kItemRing;
            if (!__all_sync(0xffffffffu, mbar_wait(b_ifull + 8 * ik, (n_items / kItemRing) & 1, p.err))) break;
            const AttnItem& it = items[ik];
            const int n = it.i1 - it.i0;
            if (n == 0) break;
            ++n_items;
            const int mine = min(it.tokens - hf * tph, tph);  // tokens of this half
            if (mine <= 0) continue;
            const int h0 = it.p0 + hf * tph, h1 = h0 + mine - 1;  // positions of the half's tokens
            const int pos = tok < mine ? h0 + tok : -1;
            float ref = -INFINITY, sum = 0.f;
            for (int j = 0; j < n; ++j) {
                const int tile = it.keys.tile(it.i0 + j);
                if (!__all_sync(0xffffffffu, mbar_wait(b_sfull + 8 * hf, s_phase, p.err))) {
                    ok = false;
                    break;
                }
                s_phase ^= 1;
                tc_fence_after();
                uint32_t sv[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(t_s + 32 * c, sv[c]);
                tmem_ld_wait();
                if (!tile_is_full<KT>(tile, h0, h1, p.window, p.sinks)) {
                    // columns of this tile that the row sees: [0, sink) and (low, high], as 32 bits per block
                    const int j0 = tile * KT, high = pos - j0;
                    const int low = p.window > 0 ? max(max(pos, 0) - p.window, -1) - j0 : -1;
                    const int sink = p.window > 0 ? p.sinks - j0 : 0;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        auto below = [&](int col) {  // bits of the columns under col
                            const int k = min(max(col - 32 * c, 0), 32);
                            return static_cast<uint32_t>((1ull << k) - 1);
                        };
                        const uint32_t seen = below(high + 1) & (~below(low + 1) | below(sink));
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(seen >> e & 1u)) sv[c][e] = 0xFF800000u;
                    }
                }
                float part_max[4];  // four chains: one would be 64 steps long
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    part_max[c] = __uint_as_float(sv[c][0]);
#pragma unroll
                    for (int e = 1; e < 32; ++e) part_max[c] = fmaxf(part_max[c], __uint_as_float(sv[c][e]));
                }
                const float mx = fmaxf(fmaxf(part_max[0], part_max[1]), fmaxf(part_max[2], part_max[3])) * p.scale_log2;
                const bool grow = mx > ref + 8.f || (ref == -INFINITY && mx > ref);
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = grow ? ex2(ref - mx) : 1.f;
                    if (grow) ref = mx;
                    sum *= f;
                    if (j > 0) {
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld_32x32b_x32(t_o + 32 * c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st_32x32b_x32(t_o + 32 * c, o);
                        }
                        tmem_st_wait();
                    }
                }
                const float base = ref == -INFINITY ? 0.f : ref;
                uint64_t acc[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
                const uint64_t k2 = pack2(p.scale_log2, p.scale_log2), b2 = pack2(-base, -base);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t pw[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 x = unpack2(fma2(
                            pack2(__uint_as_float(sv[c][2 * e]), __uint_as_float(sv[c][2 * e + 1])), k2, b2));
                        const float a0 = ex2(x.x), a1 = ex2(x.y);
                        acc[e & 1] = add2(acc[e & 1], pack2(a0, a1));
                        const __nv_bfloat162 pr = __floats2bfloat162_rn(a0, a1);
                        pw[e] = *reinterpret_cast<const uint32_t*>(&pr);
                    }
                    tmem_st_32x32b_x16(t_s + 16 * c, pw);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(b_pfull + 8 * hf);
                const float2 a = unpack2(add2(acc[0], acc[1]));
                sum += a.x + a.y;
            }
            if (!ok) break;
            const bool whole = it.i0 == 0 && it.i1 == it.keys.n;
            const int first = it.first, last = it.last, me = blockIdx.x;
            uint32_t* count = p.counters + 2 * first + hf;
            uint32_t arrived = 0;
            if (!whole && r == 0) arrived = ld_acquire(count);
            if (!__all_sync(0xffffffffu, mbar_wait(b_ofull + 8 * hf, o_phase, p.err))) {
                ok = false;
                break;
            }
            o_phase ^= 1;
            tc_fence_after();
            const bool fix = poison[n_items & 3] == n_items;
            // the non-finite values that were zeroed, back into 64 columns of the rows that see them
            auto add_back = [&](float (&o)[64], int c0) {
                for (int j = 0; j < n; ++j) {
                    const int tile = it.keys.tile(it.i0 + j);
                    if (tile_is_full<KT>(tile, it.p0, it.p0 + it.tokens - 1, p.window, p.sinks)) continue;
                    for (int k = 0; k < KT; ++k) {
                        const int key = tile * KT + k;
                        if (pos < 0 || !sees(pos, key, p.window, p.sinks)) continue;
                        const int page = p.c.table[it.row + (key >> p.c.page_shift)];
                        if (page < 0 || page >= p.c.n_pages) continue;
                        const uint16_t* v = p.c.v + page * p.c.page_stride +
                                            ((static_cast<int64_t>(it.h) << p.c.page_shift) +
                                             (key & ((1 << p.c.page_shift) - 1))) * D + c0;
#pragma unroll
                        for (int e = 0; e < 64; ++e) {
                            const float x = __uint_as_float(static_cast<uint32_t>(v[e]) << 16);
                            if (!isfinite(x)) o[e] += x;
                        }
                    }
                }
            };
            auto accumulators = [&](float (&o)[64], int c0) {
                uint32_t ov[2][32];
                tmem_ld_32x32b_x32(t_o + c0, ov[0]);
                tmem_ld_32x32b_x32(t_o + c0 + 32, ov[1]);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 64; ++e) o[e] = __uint_as_float(ov[e >> 5][e & 31]);
                if (fix) add_back(o, c0);
            };
            // 64 columns of the warp's 32 rows: turned in shared memory (16-byte
            // chunk index XOR row % 8), so that eight lanes write a row's 128 bytes
            const int out_row = tok < mine && r < tph * p.group
                                    ? (it.t_first + hf * tph + tok) * p.heads + it.h * p.group + g : -1;
            uint8_t* stage = smem + Cfg::kOffStage + warp * 4096;
            auto store = [&](const float (&o)[64], int c0, float inv) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint32_t y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __nv_bfloat162 q = __floats2bfloat162_rn(o[8 * c + 2 * i] * inv, o[8 * c + 2 * i + 1] * inv);
                        y[i] = *reinterpret_cast<const uint32_t*>(&q);
                    }
                    *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int row = 4 * k + (lane >> 3), to = __shfl_sync(0xffffffffu, out_row, row);
                    const uint4 v = *reinterpret_cast<const uint4*>(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
                    if (to >= 0) *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(to) * D + c0 + 8 * (lane & 7)) = v;
                }
                __syncwarp();
            };
            if (whole) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 64) {
                    float o[64];
                    accumulators(o, c0);
                    store(o, c0, inv);
                }
                continue;
            }
            // part of a row tile: the partial sums go to the scratch, the last
            // CTA to arrive adds them up in the CTAs' order, its own from TMEM
            auto part = [&](int cta) {
                return p.scratch + (static_cast<int64_t>(it.slot(cta)) * 2 + hf) * Cfg::kPartFloats;
            };
            auto wg_sync = [&] {
                mbar_arrive(b_wg + 8 * hf);
                const bool done = __all_sync(0xffffffffu, mbar_wait(b_wg + 8 * hf, wg_phase, p.err));
                wg_phase ^= 1;
                return done;
            };
            // (all threads of the half have read last_s of the item before: their P has been used)
            if (r == 0) last_s[hf] = arrived == static_cast<uint32_t>(last - first);
            if (!(ok = wg_sync())) break;
            if (!last_s[hf]) {
                float* out_part = part(me);
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 64) {
                    float o[64];
                    accumulators(o, c0);
#pragma unroll
                    for (int e = 0; e < 64; e += 4)
                        __stcg(reinterpret_cast<float4*>(out_part + (c0 + e) * 128) + r,
                               make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]));
                }
                __stcg(out_part + D * 128 + r, ref);
                __stcg(out_part + (D + 1) * 128 + r, sum);
                __threadfence();
                if (!(ok = wg_sync())) break;
                if (r == 0) {
                    last_s[hf] = atomicAdd(count, 1u) == static_cast<uint32_t>(last - first);
                    __threadfence();
                }
                if (!(ok = wg_sync())) break;
                if (!last_s[hf]) continue;
            }
            if (r == 0) *count = 0u;  // as the next call expects it
            float top = ref;
            for (int cta = first; cta <= last; ++cta)
                if (cta != me) top = fmaxf(top, __ldcg(part(cta) + D * 128 + r));
            const float base = top == -INFINITY ? 0.f : top;
            float all = 0.f;
            for (int cta = first; cta <= last; ++cta) {
                const bool own = cta == me;
                const float its_ref = own ? ref : __ldcg(part(cta) + D * 128 + r);
                const float its_sum = own ? sum : __ldcg(part(cta) + (D + 1) * 128 + r);
                all = fmaf(its_sum, ex2(its_ref - base), all);
            }
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 64) {
                float o[64] = {};
#pragma unroll 1
                for (int cta = first; cta <= last; ++cta) {
                    const float* from = part(cta);
                    float x[64], its_ref = ref;
                    if (cta == me) {
                        accumulators(x, c0);
                    } else {
                        its_ref = __ldcg(from + D * 128 + r);
#pragma unroll
                        for (int e = 0; e < 64; e += 4) {
                            const float4 y = __ldcg(reinterpret_cast<const float4*>(from + (c0 + e) * 128) + r);
                            x[e] = y.x;
                            x[e + 1] = y.y;
                            x[e + 2] = y.z;
                            x[e + 3] = y.w;
                        }
                    }
                    const float w = ex2(its_ref - base);
#pragma unroll
                    for (int e = 0; e < 64; ++e) o[e] = fmaf(x[e], w, o[e]);
                }
                store(o, c0, all == 0.f ? 0.f : 1.f / all);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        mbar_wait(b_fin, 0, p.err);
        tc_fence_after();
        tmem_dealloc(tmem, Cfg::kTmemCols);
    }
}

// ------------------------------------------------------------------ host ---

// Q: {64 of head_dim, query head, token, column block}; a box is the rows of half an item.
static bool encode_q(CUtensorMap* map, const AttnArgs& a, int tokens, int group) {
    const uint64_t row = static_cast<uint64_t>(a.head_dim) * 2;
    const uint64_t dims[4] = {64, static_cast<uint64_t>(a.heads), static_cast<uint64_t>(tokens),
                              static_cast<uint64_t>(a.head_dim / 64)};
    const uint64_t strides[3] = {row, row * a.heads, 128};
    const uint32_t box[4] = {64, static_cast<uint32_t>(group), static_cast<uint32_t>(128 / group), 1};
    return encode_bf16_sw128(map, a.Q, 4, dims, strides, box);
}

template <int D>
static cudaError_t launch_chunk(const AttnParams& p, const AttnArgs& a, cudaStream_t stream, const DeviceInfo& dev,
                                int pdl) {
    CUtensorMap mq, mk, mv;
    if (!encode_q(&mq, a, p.b.tokens, p.group) || !encode_pages(&mk, p.c.k, p.c, D, 1) ||
        !encode_pages(&mv, p.c.v, p.c, D, 1))
        return cudaErrorInvalidValue;
    auto kernel = count_wide(p, 2 * (128 / p.group), kChunkKeys, kChunkCost) ? q4k_attn_chunk_kernel<D, uint64_t>
                                                                             : q4k_attn_chunk_kernel<D, uint32_t>;
    return launch_serve(kernel, dim3(dev.num_sms), dim3(kChunkThreads), ChunkCfg<D>::kSmem, stream,
                        pdl, 1, p, mq, mk, mv);
}

cudaError_t launch_attention(const CacheLayer& c, const Batch& b, const AttnArgs& a, int max_new,
                             cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    AttnParams p;
    p.c = c;
    p.b = b;
    p.out = a.out;
    p.Q = a.Q;
    p.heads = a.heads;
    p.group = a.heads / c.kv_heads;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.window = a.window;
    p.sinks = a.sinks;
    p.counters = a.counters;
    p.scratch = static_cast<float*>(a.scratch);
    p.err = dev.err;
    // at most one row tile of 16 per sequence and kv head: bound by the memory,
    // not by the tensor core
    const int64_t rows = std::max(static_cast<int64_t>(max_new) * p.group, static_cast<int64_t>(p.group));
    if (rows <= 16) return launch_attn_decode(p, static_cast<int>(rows), a.head_dim, stream, dev, pdl);
    return a.head_dim == 64 ? launch_chunk<64>(p, a, stream, dev, pdl) : launch_chunk<128>(p, a, stream, dev, pdl);
}

int64_t attn_scratch_bytes(const DeviceInfo& dev, int head_dim) {
    const int64_t part = head_dim == 64 ? ChunkCfg<64>::kPartFloats : ChunkCfg<128>::kPartFloats;
    return static_cast<int64_t>(dev.num_sms) * 4 * part * 4;
}

cudaError_t attn_setup(DeviceInfo& dev) {
    if (2 * dev.num_sms > kPageTicket) return cudaErrorInvalidValue;  // counters of the workspace
    cudaError_t e = attn_decode_setup();
    if (e != cudaSuccess) return e;
    cudaError_t r;
#define Q4K_SET(D, U)                                                                                     \
    if ((r = cudaFuncSetAttribute(q4k_attn_chunk_kernel<D, U>, cudaFuncAttributeMaxDynamicSharedMemorySize, \
                                  ChunkCfg<D>::kSmem)) != cudaSuccess)                                    \
        e = r;
    Q4K_SET(64, uint32_t) Q4K_SET(64, uint64_t) Q4K_SET(128, uint32_t) Q4K_SET(128, uint64_t)
#undef Q4K_SET
    return e;
}

}  // namespace q4k
