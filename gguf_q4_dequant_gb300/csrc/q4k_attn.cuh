// q4k_attn.cuh -- how the attention kernels share out a step's work.
//
// The rows of a kv head (its G query heads of each new token) are cut into row
// tiles of whole tokens, the positions into key tiles. One unit of work is one
// (row tile, key tile) that the mask does not rule out; the units of all
// sequences, kv heads and row tiles are numbered in that order, and CTA c of
// the grid takes about units [c*q, (c+1)*q) with q = ceil(total / grid). So every
// CTA has about the same number of key tiles whatever the sequences' lengths
// are, on the device's own numbers. Units are counted in 32 bits (U) unless the
// step may have 2^32 of them, as a prompt of two million tokens with 8 query heads
// for each of 8 kv heads has (some 40 s of work): then in 64. Counting in 64 always
// cost 0.7 us at one token (11.0 for 10.3 in a stream) and 2 % of a prompt chunk.
// Those of one row tile fit 24 bits.
// A row tile that lies in several CTAs' ranges is put
// together from their partial results by whichever of them finishes last, in
// the order of the CTAs: the result does not depend on which one that is.
#pragma once

#include "q4k_device.cuh"
#include "q4k_serve.h"

namespace q4k {

struct AttnParams {
    CacheLayer c;
    Batch b;
    uint16_t* out;
    const uint16_t* Q;
    int heads, group;     // query heads; query heads per kv head
    float scale_log2;     // scale * log2(e): weights are 2^(s * scale_log2 - reference)
    int window, sinks;
    uint32_t* counters;
    float* scratch;
    unsigned int* err;
};

// Key tiles that some row of a row tile with positions p0 .. p1 sees: tiles
// 0 .. st-1 (first tokens), then w0, w0 + 1, ...; n in all, at least 1 (a row
// tile that sees nothing still writes its zeros).
struct KeyTiles {
    int st, w0, n;
    __device__ __forceinline__ int tile(int i) const { return i < st ? i : w0 + (i - st); }
};

template <int KT>
__device__ __forceinline__ KeyTiles key_tiles(int p0, int p1, int window, int sinks) {
    KeyTiles k{0, 0, 1};
    if (p1 < 0) return k;
    const int end = p1 / KT + 1;
    if (window > 0) {
        const int64_t lo = static_cast<int64_t>(p0) - window + 1;
        k.w0 = lo > 0 ? static_cast<int>(lo) / KT : 0;
        k.st = min((min(sinks, p1 + 1) + KT - 1) / KT, k.w0);
    }
    k.n = k.st + end - k.w0;
    return k;
}

// Every row with a position in p0 .. p1 sees every key of the tile.
template <int KT>
__device__ __forceinline__ bool tile_is_full(int tile, int p0, int p1, int window, int sinks) {
    const int j0 = tile * KT, j1 = j0 + KT - 1;
    return j1 <= p0 && (window == 0 || j0 > p1 - window || j1 < sinks);
}

__device__ __forceinline__ bool sees(int p, int j, int window, int sinks) {
    return j <= p && (window == 0 || j > p - window || j < sinks);
}

// How a range's units are counted: a row tile counts as `item` units more than
// it has key tiles (its start and its end take about that long), and a range's
// end that falls into a row tile within `snap` key tiles of one of its ends
// moves there, since putting two parts together costs about as much. So
// boundary c, at first c * q, lies inside a row tile of units [a, b) only if
// a + item + snap < c * q < b - snap. A range has q_min units at least.
struct AttnCost {
    int item, snap, q_min;
};

// A counter that other CTAs add to after they have written their parts.
__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
    uint32_t x;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(x) : "l"(p) : "memory");
    return x;
}

// What one CTA does, item by item.
struct AttnItem {
    int t_first, tokens;  // rows of the step's arrays
    int p0;               // position of the first token (negative: sees nothing)
    int h;                // kv head
    int64_t row;          // the sequence's row of the table
    int len;
    KeyTiles keys;
    int i0, i1;           // this CTA's part of the key tiles' list
    int first, last;      // CTAs that share the row tile (equal: this one has all of it)

    // Where a partial result goes: a CTA has at most two split row tiles, one
    // that began in an earlier CTA (slot 0) and one that goes on in a later (slot 1).
    __device__ __forceinline__ int slot(int cta) const { return 2 * cta + (cta == first); }
};

// The producer warp works the items out and hands them to the other warps
// through a small ring in shared memory; an item without key tiles is the end.
constexpr int kItemRing = 4;

template <typename U>
struct AttnWalk {
    U u, u_end;  // units left to do
    U q;
    int b, h, tile, off;
    SeqView s;
};

// The next item, or false. `tt`: tokens of a row tile.
template <int KT, typename U>
__device__ __forceinline__ bool next_item(const AttnParams& p, AttnWalk<U>& w, int tt, AttnCost cost, AttnItem& it) {
    it.i0 = it.i1 = 0;
    if (w.u >= w.u_end) return false;
    while (w.tile * tt >= w.s.m) {  // the sequence's row tiles are done for this head
        w.tile = 0;
        if (w.s.m == 0 || ++w.h == p.c.kv_heads) {
            w.h = 0;
            w.s = seq_view(p.c, p.b, ++w.b);  // exists: there are units left
        }
    }
    it.t_first = w.s.t0 + w.tile * tt;
    it.tokens = min(tt, w.s.m - w.tile * tt);
    it.p0 = w.s.len - w.s.m + w.tile * tt;
    it.h = w.h;
    it.row = w.s.row;
    it.len = w.s.len;
    it.keys = key_tiles<KT>(it.p0, it.p0 + it.tokens - 1, p.window, p.sinks);
    const U u0 = w.u - w.off, u1 = u0 + cost.item + it.keys.n;  // the row tile's units
    it.i0 = w.off > 0 ? w.off - cost.item : 0;
    it.i1 = w.u_end < u1 ? static_cast<int>(w.u_end - u0) - cost.item : it.keys.n;
    it.first = it.last = blockIdx.x;
    if (it.i0 > 0 || it.i1 < it.keys.n) {
        it.first = static_cast<int>((u0 + cost.item + cost.snap) / w.q);  // one before the first boundary inside
        it.last = static_cast<int>((u1 - cost.snap - 1) / w.q);           // the last boundary inside
    }
    w.u = min(u1, w.u_end);
    w.off = 0;
    ++w.tile;
    return true;
}

// Units of a row tile of a sequence.
template <int KT>
__device__ __forceinline__ int tile_units(const AttnParams& p, const SeqView& s, int tile, int tt, AttnCost cost) {
    const int p0 = s.len - s.m + tile * tt;
    return cost.item + key_tiles<KT>(p0, p0 + min(tt, s.m - tile * tt) - 1, p.window, p.sinks).n;
}

template <typename U>
struct AttnCut {
    U u;               // the boundary, moved
    int b, h, tile, off;  // where it lies (off > 0: inside the row tile)
    SeqView s;
};

// Inclusive sum over the lanes of a warp.
template <typename U>
__device__ __forceinline__ U warp_scan(U x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const U v = __shfl_up_sync(0xffffffffu, x, k);
        if (lane >= k) x += v;
    }
    return x;
}

// Sum over the lanes of a warp.
__device__ __forceinline__ uint32_t warp_sum(uint32_t x) { return __reduce_add_sync(0xffffffffu, x); }
__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
    return x;
}

// By one warp: where unit u of the step lies in sequence b, which has per_head
// units per kv head from unit `at` on.
template <int KT, typename U>
__device__ __forceinline__ AttnCut<U> cut_in(const AttnParams& p, int tt, int b, const SeqView& s, U per_head, U at, U u,
                                             AttnCost cost) {
    const int lane = threadIdx.x & 31;
    AttnCut<U> c;
    c.b = b;
    c.s = s;
    c.tile = 0;
    c.h = static_cast<int>((u - at) / per_head);
    U rest = (u - at) - c.h * per_head;
    int n = static_cast<int>(per_head);  // (of the row tile that is cut, if the sequence has only one)
    if (s.m > tt) {
        for (int t0 = 0; t0 < (s.m + tt - 1) / tt; t0 += 32) {
            const int t = t0 + lane;
            const uint32_t mine = static_cast<int64_t>(t) * tt < s.m ? tile_units<KT>(p, s, t, tt, cost) : 0;
            const uint32_t incl = warp_scan(mine);
            const uint32_t past = __ballot_sync(0xffffffffu, incl > rest);
            if (past) {
                const int l = __ffs(past) - 1;
                c.tile = t0 + l;
                n = __shfl_sync(0xffffffffu, mine, l);
                rest -= __shfl_sync(0xffffffffu, incl - mine, l);
                break;
            }
            rest -= __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    c.u = u;
    c.off = static_cast<int>(rest);
    if (c.off <= cost.item + cost.snap) {
        c.u -= c.off;
        c.off = 0;
    } else if (n - c.off <= cost.snap) {
        c.u += n - c.off;
        c.off = 0;
        ++c.tile;  // (one past the last: the walk goes on to the next head or sequence)
    }
    return c;
}

// By one warp: units per kv head of the lanes' sequences.
template <int KT, typename U>
__device__ __forceinline__ U lane_units(const AttnParams& p, int tt, const SeqView& s, AttnCost cost) {
    const int lane = threadIdx.x & 31, tiles = (s.m + tt - 1) / tt;
    U u = 0;
    if (tiles <= 4)
        for (int t = 0; t < tiles; ++t) u += tile_units<KT>(p, s, t, tt, cost);
    // many row tiles: the warp counts them together
    uint32_t many = __ballot_sync(0xffffffffu, tiles > 4);
    while (many) {
        const int l = __ffs(many) - 1;
        many &= many - 1;
        SeqView o;
        o.m = __shfl_sync(0xffffffffu, s.m, l);
        o.len = __shfl_sync(0xffffffffu, s.len, l);
        const int ot = (o.m + tt - 1) / tt;
        U x = 0;
        for (int t = lane; t < ot; t += 32) x += tile_units<KT>(p, o, t, tt, cost);
        x = warp_sum(x);
        if (lane == l) u = x;
    }
    return u;
}

// The CTA's range by one warp, for at most 32 sequences.
template <int KT, typename U>
__device__ __forceinline__ AttnWalk<U> plan_warp(const AttnParams& p, int tt, AttnCost cost) {
    const int lane = threadIdx.x & 31;
    SeqView s{0, 0, 0, 0};
    if (lane < p.b.n) s = seq_view(p.c, p.b, lane);
    const U per_head = lane_units<KT, U>(p, tt, s, cost), mine = per_head * p.c.kv_heads;
    const U incl = p.b.n > 1 ? warp_scan(mine) : __shfl_sync(0xffffffffu, mine, 0);
    const U total = __shfl_sync(0xffffffffu, incl, 31);
    AttnWalk<U> w;
    w.q = max((total + gridDim.x - 1) / gridDim.x, static_cast<U>(cost.q_min));
    w.u = w.u_end = total;
    w.b = w.h = w.tile = w.off = 0;
    w.s = SeqView{0, 0, 0, 0};
    auto cut = [&](U u) {
        const int l = __ffs(__ballot_sync(0xffffffffu, incl > u)) - 1;
        SeqView o;
        o.t0 = __shfl_sync(0xffffffffu, s.t0, l);
        o.m = __shfl_sync(0xffffffffu, s.m, l);
        o.len = __shfl_sync(0xffffffffu, s.len, l);
        o.row = __shfl_sync(0xffffffffu, s.row, l);
        return cut_in<KT, U>(p, tt, l, o, __shfl_sync(0xffffffffu, per_head, l), __shfl_sync(0xffffffffu, incl - mine, l), u, cost);
    };
    const uint64_t u0 = static_cast<uint64_t>(blockIdx.x) * w.q, u1 = u0 + w.q;
    if (u0 < total) {
        const AttnCut<U> c = cut(static_cast<U>(u0));
        w.u = c.u;
        w.b = c.b;
        w.h = c.h;
        w.tile = c.tile;
        w.off = c.off;
        w.s = c.s;
        if (u1 < total) w.u_end = cut(static_cast<U>(u1)).u;
    }
    return w;
}

// The same by all threads of the block, for any number of sequences: `units`
// holds n counts in shared memory, `found` takes the result. Ends with
// __syncthreads().
template <int KT, typename U>
__device__ __forceinline__ void plan_block(const AttnParams& p, int tt, AttnCost cost, U* units,
                                           AttnWalk<U>* found) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    for (int i0 = warp * 32; i0 < p.b.n; i0 += nwarps * 32) {
        const int i = i0 + lane;
        SeqView s{0, 0, 0, 0};
        if (i < p.b.n) s = seq_view(p.c, p.b, i);
        const U u = lane_units<KT, U>(p, tt, s, cost);
        if (i < p.b.n) units[i] = u * p.c.kv_heads;
    }
    __syncthreads();
    // warp 0 finds where the range begins, warp 1 where it ends
    if (warp < 2) {
        U total = 0;
        for (int i = lane; i < p.b.n; i += 32) total += units[i];
        total = warp_sum(total);
        const U q = max((total + gridDim.x - 1) / gridDim.x, static_cast<U>(cost.q_min));
        const uint64_t u64 = static_cast<uint64_t>(blockIdx.x + warp) * q;
        AttnCut<U> c;
        c.u = total;
        c.b = c.h = c.tile = c.off = 0;
        c.s = SeqView{0, 0, 0, 0};
        if (u64 < total) {
            const U u = static_cast<U>(u64);
            U at = 0;
            int b = 0;
            for (int i0 = 0; i0 < p.b.n; i0 += 32) {
                const U mine = i0 + lane < p.b.n ? units[i0 + lane] : 0, incl = warp_scan(mine);
                const uint32_t past = __ballot_sync(0xffffffffu, at + incl > u);
                if (past) {
                    const int l = __ffs(past) - 1;
                    b = i0 + l;
                    at += __shfl_sync(0xffffffffu, incl - mine, l);
                    break;
                }
                at += __shfl_sync(0xffffffffu, incl, 31);
            }
            c = cut_in<KT, U>(p, tt, b, seq_view(p.c, p.b, b), units[b] / p.c.kv_heads, at, u, cost);
        }
        if (lane == 0) {
            if (warp == 0) {
                found->u = c.u;
                found->q = q;
                found->b = c.b;
                found->h = c.h;
                found->tile = c.tile;
                found->off = c.off;
                found->s = c.s;
            } else {
                found->u_end = c.u;
            }
        }
    }
    __syncthreads();
}

// K or V of one layer as a tensor map: {64 of head_dim, row of the page, column
// block, kv head, page}; a box is `blocks` column blocks of one page of one head.
inline bool encode_pages(CUtensorMap* map, const uint16_t* base, const CacheLayer& c, int head_dim, int blocks) {
    const int page = 1 << c.page_shift;
    const uint64_t dims[5] = {64, static_cast<uint64_t>(page), static_cast<uint64_t>(head_dim / 64),
                              static_cast<uint64_t>(c.kv_heads), static_cast<uint64_t>(c.n_pages)};
    const uint64_t strides[4] = {static_cast<uint64_t>(head_dim) * 2, 128,
                                 static_cast<uint64_t>(page) * head_dim * 2,
                                 static_cast<uint64_t>(c.page_stride) * 2};
    const uint32_t box[5] = {64, static_cast<uint32_t>(page), static_cast<uint32_t>(blocks), 1, 1};
    return encode_bf16_sw128(map, base, 5, dims, strides, box);
}

// Whether units are to be counted in 64 bits: the step has fewer than 2^32 (and the
// grid's rounding) if every sequence may have all the tokens, as offsets that make no
// sense may say, and every row tile (of tt tokens) all the key tiles that the
// table has room for.
inline bool count_wide(const AttnParams& p, int tt, int keys, AttnCost cost) {
    const double row_tiles = static_cast<double>(p.b.n) * (p.b.tokens / tt + 1) * p.c.kv_heads;
    const int key_tiles = ((p.c.width << p.c.page_shift) + keys - 1) / keys;
    return row_tiles * (key_tiles + cost.item) > 4.2e9;
}

// The kernel for few rows per kv head: `rows` <= 16 of them in a row tile (group <= rows).
cudaError_t launch_attn_decode(const AttnParams& p, int rows, int head_dim, cudaStream_t stream,
                               const DeviceInfo& dev, int pdl);
cudaError_t attn_decode_setup();

// The page ids of a sequence's key tiles, for one warp: 32 entries of its table
// row at a time, a lane each, and the next 32 already on their way.
struct PageIds {
    int base, ids, next;

    __device__ __forceinline__ int load(const AttnParams& p, const AttnItem& it, int64_t at) const {
        if (at << p.c.page_shift >= it.len) return -1;  // (asked for as page -1: reads as zeros)
        const int id = p.c.table[it.row + at];
        return id < p.c.n_pages ? max(id, -1) : -1;
    }
    __device__ __forceinline__ void begin() { base = -1; }
    // Entry first + k of the row, for the lanes' own k < 32; first is the same for all and a multiple of `pages` | 32.
    __device__ __forceinline__ int get(const AttnParams& p, const AttnItem& it, int first, int k) {
        if (base < 0 || first < base || first >= base + 32) {
            const int lane = threadIdx.x & 31;
            ids = base >= 0 && first == base + 32 ? next : load(p, it, static_cast<int64_t>(first) + lane);
            base = first;
            next = load(p, it, static_cast<int64_t>(first) + 32 + lane);
        }
        return __shfl_sync(0xffffffffu, ids, first - base + k);
    }
};

// 2^x by the special function unit (flushes subnormal results to zero, which a
// softmax weight may be).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Bit 15 and 31: that half of a bf16 pair is an infinity or NaN.
__device__ __forceinline__ uint32_t bf16x2_non_finite(uint32_t w) {
    return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}

}  // namespace q4k
