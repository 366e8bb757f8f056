// q4k_route.cu -- the k largest router logits of each token, their weights, and
// the tokens' rows in the order of their experts: the sort, the gathering of the
// rows, and the way back with the weights applied.
//
// The sort counts: how many pairs go to each expert, how many of them come before
// a pair in the numbering, both by whole warps, so the order hangs on no timing. Its
// arrays are small (8192 tokens, 128 experts: 4 MB of logits, 0.8 MB of results), its time
// is launches, dependent loads and the picks' integer instructions: 48 tokens and
// their rows 7.6 us, 8192 tokens 71 us, 49 of them the rows (286 MB, 5.8 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "q4k_device.cuh"
#include "q4k_experts.h"
#include "q4k_serve.h"

namespace q4k {

constexpr int kRouteTokens = 64;    // tokens of a block of the sort
constexpr int kRouteThreads = 1024;
// Threads of a block that picks: a lane holds R logits and their keys.
__host__ __device__ constexpr int pick_threads(int R) { return R <= 8 ? 1024 : 512; }
// Steps of up to so many blocks have no scan of their own: each block adds up the
// counts of the blocks before it (128 of them and 128 experts: two rounds of eight loads).
constexpr int kRouteFew = 128;
// Logits below this are masks, not scores (programs mask with -1e4, -1e9 or the type's lowest value, -65504 in
// fp16): sigmoids over their sum are 0 for a token that has nothing else, as they are for one with only -inf.
constexpr float kRouteMask = -1000.f;

// ------------------------------------------------------------------- top k ---

// An unsigned integer that orders like the logit; 0 for -inf and NaN, which are
// never picked. (x + 0 makes -0 of 0, so that they tie.)
__device__ __forceinline__ uint32_t logit_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    const uint32_t key = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return x != x || u == 0xFF800000u ? 0u : key;
}

// exp(x - top) for live logits x <= top, an infinite top included.
__device__ __forceinline__ float rel_exp(float x, float top) { return x == top ? 1.f : expf(x - top); }

// A warp picks the k largest of a token's logits: expert 32 r + lane is held in
// key[r]; each round takes the warp's largest key and, of the lanes that hold
// it, the lowest expert. Lane j returns the j-th pick's expert (-1: none left)
// and its weight.
template <int R>
__device__ __forceinline__ int pick_experts(const float* row, int E, int k, int weighting, float scale, int lane,
                                            float* weight) {
    float x[R];
    uint32_t key[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int e = 32 * r + lane;
        x[r] = e < E ? row[e] : -INFINITY;
        key[r] = logit_key(x[r]);
    }
    int mine = -1;
    float mine_x = 0.f, top = 0.f;
    for (int j = 0; j < k; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (key[r] > best) best = key[r], at = r;  // the lowest r of the lane's largest
        const uint32_t most = __reduce_max_sync(0xffffffffu, best);
        if (most == 0u) break;
        const unsigned e = __reduce_min_sync(0xffffffffu, best == most ? 32u * at + lane : 0xffffffffu);
        const float xe = __uint_as_float((most & 0x80000000u) ? most & 0x7FFFFFFFu : ~most);
        if (j == 0) top = xe;
        if (lane == j) mine = static_cast<int>(e), mine_x = xe;
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (32u * r + lane == e) key[r] = 0u;
    }
    float rel = 0.f, total = 1.f;
    if (weighting == Q4K_ROUTE_SOFTMAX || weighting == Q4K_ROUTE_SOFTMAX_TOP) {
        if (mine >= 0) rel = rel_exp(mine_x, top);
        total = rel;
        if (weighting == Q4K_ROUTE_SOFTMAX) {
            total = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (logit_key(x[r]) != 0u) total += rel_exp(x[r], top);
        }
    } else {
        // Where the sigmoids are divided by their sum and the largest logit is below 0, they are taken as
        // e^(x - top) / (1 + e^x): the common factor e^top of sigmoid(x) goes with the sum, and
        // nothing leaves fp32's range that the quotient does not. (From 0 up their sum is at least 1/2: what
        // 1 / (1 + e^-x) loses below x = -88 is below 2^-125.)
        const bool part = weighting == Q4K_ROUTE_SIGMOID_TOP && top < 0.f && top >= kRouteMask;
        if (mine >= 0) rel = part ? rel_exp(mine_x, top) / (1.f + expf(mine_x)) : 1.f / (1.f + expf(-mine_x));
        total = rel;
    }
    if (weighting != Q4K_ROUTE_SIGMOID) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    } else {
        total = 1.f;
    }
    *weight = total > 0.f ? rel / total * scale : 0.f;
    return mine;
}

// The picks of every `step`-th of tokens t0 .. t0 + n - 1 from the i0-th on, a warp
// each: to ids and weights, and to put(pair of the block, expert).
template <int R, typename Put>
__device__ __forceinline__ void pick_tokens(const RouteArgs& a, int t0, int n, int i0, int step, Put put) {
    const int lane = threadIdx.x & 31;
    for (int i = i0; i < n; i += step) {
        float w;
        const int64_t t = t0 + i;
        const int e = pick_experts<R>(a.logits + t * a.E, a.E, a.k, a.weighting, a.scale, lane, &w);
        if (lane < a.k) {
            a.ids[t * a.k + lane] = e;
            a.weights[t * a.k + lane] = w;
            put(i * a.k + lane, e);
        }
    }
}

// How many of the block's pairs before each pair go to its expert, in the order
// of the pairs. Each warp takes a run of whole 32 pairs: it counts its own in
// `hist[warp]`, the counts are summed over the warps before it, and it goes
// over its run again, 32 pairs at a time (lanes with the same expert find one
// another). hist: [warps][E], zeros; `used` warps have pairs.
__device__ __forceinline__ void count_pairs(const int16_t* chosen, int pairs, int E, int* hist, int run) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i0 = warp * run; i0 < min((warp + 1) * run, pairs); i0 += 32) {
        const int i = i0 + lane;
        const int e = i < pairs ? chosen[i] : -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && lane == __ffs(same) - 1) hist[warp * E + e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
}

__device__ __forceinline__ void place_pairs(const RouteArgs& a, const int16_t* chosen, int64_t first, int pairs, int E,
                                            int* hist, const int* base, int run) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i0 = warp * run; i0 < min((warp + 1) * run, pairs); i0 += 32) {
        const int i = i0 + lane;
        const int e = i < pairs ? chosen[i] : -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        int at = -1;
        if (e >= 0) at = base[e] + hist[warp * E + e] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1) hist[warp * E + e] += __popc(same);
        __syncwarp();
        if (i < pairs) {
            a.slots[first + i] = at;
            if (at >= 0) a.order[at] = static_cast<int>(first + i);
        }
    }
}

// Exclusive scan of the counts cnt[0 .. E-1] (shared memory) by the block, to
// base[0 .. E] (base[E]: the total): a lane of the first warp has E / 32 of them
// side by side. E <= 1024.
__device__ __forceinline__ void scan_experts(const int* cnt, int E, int* base) {
    if (threadIdx.x < 32) {
        const int per = (E + 31) / 32, e0 = threadIdx.x * per, e1 = min(e0 + per, E);
        int sum = 0;
        for (int e = e0; e < e1; ++e) sum += cnt[e];
        int s = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, s, o);
            if (static_cast<int>(threadIdx.x) >= o) s += t;
        }
        int at = s - sum;
        for (int e = e0; e < e1; ++e) {
            base[e] = at;
            at += cnt[e];
        }
        if (threadIdx.x == 31) base[E] = s;
    }
    __syncthreads();
}

// A step of a few tokens is one launch: a cluster's blocks share the picks, which
// fill a block's integer pipe (48 tokens: 5.7 us, 8.4 by one block), and hand them
// to the first one's shared memory, which does the rest.
template <int R>
__global__ void __launch_bounds__(pick_threads(R)) q4k_route_one_kernel(const RouteArgs a) {
    extern __shared__ int route_smem[];
    const int blocks = gridDim.x;  // of the one cluster
    if (blocks > 1) cluster_arrive_relaxed();
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, pairs = a.T * a.k;
    int* hist = route_smem;             // [warps][E]
    int* cnt = hist + warps * a.E;      // [E]
    int* base = cnt + a.E;              // [E + 1]
    int16_t* chosen = reinterpret_cast<int16_t*>(base + a.E + 1);
    const int run = ((pairs + warps - 1) / warps + 31) / 32 * 32, used = (pairs + run - 1) / run;
    if (blocks > 1) {
        const uint32_t first = map_shared_rank(smem_u32(chosen), 0);
        cluster_wait();  // every block of the cluster has begun
        pick_tokens<R>(a, 0, a.T, blockIdx.x + blocks * warp, blocks * warps, [&](int i, int e) {
            asm volatile("st.shared::cluster.u16 [%0], %1;" ::"r"(first + 2 * i), "h"(static_cast<int16_t>(e)) : "memory");
        });
        __syncwarp();
        cluster_sync_all();
        if (blockIdx.x != 0) return;
    } else {
        pick_tokens<R>(a, 0, a.T, warp, warps, [&](int i, int e) { chosen[i] = static_cast<int16_t>(e); });
    }
    for (int i = threadIdx.x; i < used * a.E; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    count_pairs(chosen, pairs, a.E, hist, run);
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int s = 0;
        for (int w = 0; w < used; ++w) {
            const int c = hist[w * a.E + e];
            hist[w * a.E + e] = s;
            s += c;
        }
        cnt[e] = s;
    }
    __syncthreads();
    scan_experts(cnt, a.E, base);
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) a.starts[e] = base[e];
    for (int i = base[a.E] + threadIdx.x; i < pairs; i += blockDim.x) a.order[i] = -1;
    place_pairs(a, chosen, 0, pairs, a.E, hist, base, run);
}

// Many tokens: groups of kRouteTokens are picked and counted (counts: [groups][E]), by a
// block each or, while there are SMs for it, by a cluster of `spread`, counted in the first one's
// shared memory, ...
template <int R>
__global__ void __launch_bounds__(pick_threads(R)) q4k_route_pick_kernel(const RouteArgs a, int spread) {
    extern __shared__ int route_smem[];
    int* hist = route_smem;  // [E]
    const int group = blockIdx.x / spread, rank = blockIdx.x - group * spread;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) hist[e] = 0;
    if (spread > 1) cluster_sync_all();
    else __syncthreads();
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const int t0 = group * kRouteTokens, n = min(kRouteTokens, a.T - t0);
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    // (counts: their order does not matter)
    if (spread > 1) {
        const uint32_t first = map_shared_rank(smem_u32(hist), 0);
        pick_tokens<R>(a, t0, n, rank + spread * warp, spread * warps, [&](int, int e) {
            if (e >= 0) asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(first + 4 * e), "r"(1) : "memory");
        });
        __syncwarp();
        cluster_sync_all();
        if (rank != 0) return;
    } else {
        pick_tokens<R>(a, t0, n, warp, warps, [&](int, int e) {
            if (e >= 0) atomicAdd(&hist[e], 1);
        });
        __syncthreads();
    }
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.ws[static_cast<int64_t>(group) * a.E + e] = hist[e];
}

// ... the counts become, for each expert, the sums over the blocks before (in
// place; totals to row `blocks`): a block for 32 experts, each warp a run of
// blocks ...
__global__ void __launch_bounds__(1024) q4k_route_scan_kernel(int32_t* counts, int blocks, int E) {
    __shared__ int part[32][33];
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    const int run = (blocks + 31) / 32, b0 = min(warp * run, blocks), b1 = min(b0 + run, blocks);
    int s = 0;
    if (e < E)
        for (int b = b0; b < b1; ++b) s += counts[static_cast<int64_t>(b) * E + e];
    part[warp][lane] = s;
    __syncthreads();
    int at = 0;
    for (int w = 0; w < warp; ++w) at += part[w][lane];
    if (e < E) {
        for (int b = b0; b < b1; ++b) {
            const int64_t i = static_cast<int64_t>(b) * E + e;
            const int c = counts[i];
            counts[i] = at;
            at += c;
        }
        if (warp == 31) counts[static_cast<int64_t>(blocks) * E + e] = at;
    }
}

// ... and each block places its pairs. kScanned: ws holds those sums and totals,
// else the counts of each block.
template <bool kScanned>
__global__ void __launch_bounds__(kRouteThreads) q4k_route_place_kernel(const RouteArgs a, int most) {
    extern __shared__ int route_smem[];
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const int E = a.E, blocks = gridDim.x;
    int* hist = route_smem;        // [most][E], most: warps with pairs
    int* cnt = hist + most * E;    // [E]
    int* before = cnt + E;         // [E]
    int* base = before + E;        // [E + 1]
    int16_t* chosen = reinterpret_cast<int16_t*>(base + E + 1);
    const int t0 = blockIdx.x * kRouteTokens, n = min(kRouteTokens, a.T - t0), pairs = n * a.k;
    const int64_t first = static_cast<int64_t>(t0) * a.k;
    const int run = ((kRouteTokens * a.k + most - 1) / most + 31) / 32 * 32, used = (pairs + run - 1) / run;
    for (int i = threadIdx.x; i < used * E; i += blockDim.x) hist[i] = 0;
    for (int i = threadIdx.x; i < pairs; i += blockDim.x) chosen[i] = static_cast<int16_t>(a.ids[first + i]);
    if (kScanned) {
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            cnt[e] = a.ws[static_cast<int64_t>(blocks) * E + e];
            before[e] = a.ws[static_cast<int64_t>(blockIdx.x) * E + e];
        }
        __syncthreads();
    } else {
        for (int e = threadIdx.x; e < E; e += blockDim.x) cnt[e] = before[e] = 0;
        __syncthreads();
        // as many slices of the blocks as there are threads for; sums of integers: any order
        const int slices = max(1, static_cast<int>(blockDim.x) / E);
        for (int i = threadIdx.x; i < slices * E; i += blockDim.x) {
            const int e = i % E, slice = i / E;
            int all = 0, mine = 0;
#pragma unroll 8
            for (int b = slice; b < blocks; b += slices) {
                const int c = a.ws[static_cast<int64_t>(b) * E + e];
                all += c;
                if (b < static_cast<int>(blockIdx.x)) mine += c;
            }
            atomicAdd(&cnt[e], all);
            atomicAdd(&before[e], mine);
        }
        __syncthreads();
    }
    scan_experts(cnt, E, base);
    count_pairs(chosen, pairs, E, hist, run);
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int s = before[e];
        for (int w = 0; w < used; ++w) {
            const int c = hist[w * E + e];
            hist[w * E + e] = s;
            s += c;
        }
    }
    __syncthreads();
    place_pairs(a, chosen, first, pairs, E, hist, base, run);
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= E; e += blockDim.x) a.starts[e] = base[e];
    // what is behind the last row: each block its share
    const int64_t all = static_cast<int64_t>(a.T) * a.k;
    for (int64_t i = base[E] + static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < all;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x)
        a.order[i] = -1;
}

// ------------------------------------------------------------------ gather ---

// Eight columns of a row as bf16: copied, or e4m3 codes times their power of two
// (a code has 4 significant bits: exact in bf16 above its smallest normal
// number). Scale byte 255 is NaN.
__device__ __forceinline__ uint4 row8(const uint16_t* x, const uint8_t*, int64_t i) {
    return *reinterpret_cast<const uint4*>(x + i);
}
__device__ __forceinline__ uint4 row8(const uint8_t* x, const uint8_t* scales, int64_t i) {
    const uint2 c = *reinterpret_cast<const uint2*>(x + i);
    const uint32_t s = scales[i >> 5];
    const float f = __uint_as_float(s == 255u ? 0x7FC00000u : s == 0u ? 0x00400000u : s << 23);
    const uint32_t w[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[j]), __NV_E4M3);
        const float2 v = __half22float2(__half2(h));
        const __nv_bfloat162 b = __floats2bfloat162_rn(v.x * f, v.y * f);
        o[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Results that outgrow half of L2 pass it by: 8192 tokens to 8 experts each, 268 MB, 71 us
// for the sort of a prompt chunk instead of 87; smaller ones stay for the product that reads them.
__device__ __forceinline__ void store16(uint16_t* p, uint4 v, bool stream) {
    if (stream) __stcs(reinterpret_cast<uint4*>(p), v);
    else *reinterpret_cast<uint4*>(p) = v;
}

// A warp takes rows in turn, kGatherLoads loads of a lane in flight, the next
// row's place asked for meanwhile; the rows of a token are read once from memory
// and from L2 for its other experts.
constexpr int kGatherWarps = 4, kGatherLoads = 8, kGatherBlocks = 16;

template <typename X>
__global__ void __launch_bounds__(32 * kGatherWarps) q4k_gather_kernel(const GatherArgs a) {
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t every = static_cast<int64_t>(gridDim.x) * kGatherWarps;
    const X* x = static_cast<const X*>(a.x);
    int64_t p = static_cast<int64_t>(blockIdx.x) * kGatherWarps + (threadIdx.x >> 5);
    int pair = p < a.pairs ? a.order[p] : -1;
    for (; p < a.pairs; p += every) {
        const int now = pair;
        if (p + every < a.pairs) pair = a.order[p + every];
        if (now < 0 || now >= a.pairs) continue;
        const int64_t src = static_cast<int64_t>(now / a.k) * a.C, dst = p * a.C;
        for (int c0 = 0; c0 < a.C; c0 += 256 * kGatherLoads) {
            uint4 v[kGatherLoads];
#pragma unroll
            for (int j = 0; j < kGatherLoads; ++j) {
                const int c = c0 + 256 * j + 8 * lane;
                if (c < a.C) v[j] = row8(x, a.scales, src + c);
            }
#pragma unroll
            for (int j = 0; j < kGatherLoads; ++j) {
                const int c = c0 + 256 * j + 8 * lane;
                if (c < a.C) store16(a.out + dst + c, v[j], a.stream);
            }
        }
    }
}

// ----------------------------------------------------------------- combine ---

// Eight columns of a token a thread: the rows of its experts, kCombineLoads of
// them in flight, added in the order of the picks (one result whatever runs when).
// The rows' bytes are the bound: 8192 tokens, 8 rows of 2048 each, 63 us, 6.4 TB/s (94 % of
// a copy's rate); 48 tokens 2.9 us.
constexpr int kCombineLoads = 8;

__global__ void __launch_bounds__(256) q4k_combine_kernel(const CombineArgs a) {
    pdl_wait();
    if (threadIdx.x == 0 && threadIdx.y == 0) pdl_launch_dependents();
    const int per = (a.C / 8 + blockDim.x - 1) / blockDim.x;  // blocks along a row
    const int64_t t = static_cast<int64_t>(blockIdx.x / per) * blockDim.y + threadIdx.y;
    const int c = 8 * ((blockIdx.x % per) * blockDim.x + threadIdx.x);
    if (t >= a.T || c >= a.C) return;
    float s[8] = {};
    if (a.base != nullptr) {
        const float4* b = reinterpret_cast<const float4*>(a.base + t * a.C + c);
        const float4 p = b[0], q = b[1];
        s[0] = p.x; s[1] = p.y; s[2] = p.z; s[3] = p.w;
        s[4] = q.x; s[5] = q.y; s[6] = q.z; s[7] = q.w;
    }
    for (int j0 = 0; j0 < a.k; j0 += kCombineLoads) {
        uint4 v[kCombineLoads];
        float w[kCombineLoads];
#pragma unroll
        for (int j = 0; j < kCombineLoads; ++j) {
            const int64_t i = t * a.k + j0 + j;
            const int slot = j0 + j < a.k ? a.slots[i] : -1;
            const bool live = slot >= 0 && slot < a.pairs;
            // a row that is not there adds nothing, whatever its weight holds
            w[j] = live ? a.weights[i] : 0.f;
            v[j] = live ? __ldcs(reinterpret_cast<const uint4*>(a.y + static_cast<int64_t>(slot) * a.C + c)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < kCombineLoads; ++j) {
            const uint32_t x[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[2 * i] = fmaf(w[j], __uint_as_float(x[i] << 16), s[2 * i]);
                s[2 * i + 1] = fmaf(w[j], __uint_as_float(x[i] & 0xFFFF0000u), s[2 * i + 1]);
            }
        }
    }
    float4* o = reinterpret_cast<float4*>(a.out + t * a.C + c);
    const float4 lo = make_float4(s[0], s[1], s[2], s[3]), hi = make_float4(s[4], s[5], s[6], s[7]);
    if (a.stream) __stcs(o, lo), __stcs(o + 1, hi);
    else o[0] = lo, o[1] = hi;
}

// ------------------------------------------------------------------ host ---

namespace {

// Steps of up to so many tokens and pairs take one launch (128 experts, 8 picks: 128 tokens 8.3 us
// for 8.4, 192 tokens 9.6 for 8.5; 16 experts, one pick: 512 tokens 6.2 for 6.8, 2048 13.3 for 7.0).
constexpr int kOneTokens = 512, kOnePairs = 1024;
// Fewer tokens stay with one block, whose warps have room (8 tokens: 4.3 us either way), unless a
// token alone keeps it busy (8 tokens to 32 of 1024 experts: 28 us, 16 shared out).
constexpr int kOneSpread = 8, kOneSpreadExperts = 256;

template <int R>
cudaError_t route_r(const RouteArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    const int64_t pairs = static_cast<int64_t>(a.T) * a.k;
    if (a.T <= kOneTokens && pairs <= kOnePairs) {
        // a warp per token, as many as the counts of a warp leave room for in the 48 KB that need no attribute
        const int most = (40960 - 4 * (2 * a.E + 1)) / (4 * a.E);
        int warps = a.T < pick_threads(R) / 32 ? a.T : pick_threads(R) / 32;
        warps = warps < most ? warps : most;
        const size_t smem = 4 * (static_cast<size_t>(warps) * a.E + 2 * a.E + 1) + 2 * pairs;
        const int spread = a.T > (a.E <= kOneSpreadExperts ? kOneSpread : 1) ? 8 : 1;
        return launch_serve(q4k_route_one_kernel<R>, dim3(spread), dim3(32 * warps), smem, stream, pdl, spread, a);
    }
    const int blocks = (a.T - 1) / kRouteTokens + 1;  // (T may be 2^31 - 1)
    const size_t chosen = 2 * static_cast<size_t>(kRouteTokens) * a.k;
    int spread = 1;  // (1003 tokens, 61 experts: 8.1 us, 9.4 with 1)
    while (spread < 8 && 2 * spread * blocks <= dev.num_sms) spread *= 2;
    const int threads = pick_threads(R) < 32 * kRouteTokens / spread ? pick_threads(R) : 32 * kRouteTokens / spread;
    cudaError_t e = launch_serve(q4k_route_pick_kernel<R>, dim3(blocks * spread), dim3(threads), 4 * a.E, stream, pdl, spread, a, spread);
    if (e != cudaSuccess) return e;
    // counts for as many warps as have 32 pairs each, within 48 KB
    int most = (44 * 1024 - static_cast<int>(chosen) - 4 * (3 * a.E + 1)) / (4 * a.E);
    const int runs = (kRouteTokens * a.k + 31) / 32;
    most = most < runs ? most : runs;
    most = most < kRouteThreads / 32 ? most : kRouteThreads / 32;
    const size_t smem = 4 * (static_cast<size_t>(most) * a.E + 3 * a.E + 1) + chosen;
    if (blocks <= kRouteFew)
        return launch_serve(q4k_route_place_kernel<false>, dim3(blocks), dim3(kRouteThreads), smem, stream, pdl, 1, a, most);
    e = launch_serve(q4k_route_scan_kernel, dim3((a.E + 31) / 32), dim3(1024), 0, stream, pdl, 1, a.ws, blocks, a.E);
    if (e != cudaSuccess) return e;
    return launch_serve(q4k_route_place_kernel<true>, dim3(blocks), dim3(kRouteThreads), smem, stream, pdl, 1, a, most);
}

}  // namespace

int64_t route_scratch_bytes(int64_t T, int E) { return 4 * E * ((T + kRouteTokens - 1) / kRouteTokens + 1); }

cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    if (a.E <= 32) return route_r<1>(a, stream, dev, pdl);
    if (a.E <= 64) return route_r<2>(a, stream, dev, pdl);
    if (a.E <= 128) return route_r<4>(a, stream, dev, pdl);
    if (a.E <= 256) return route_r<8>(a, stream, dev, pdl);
    if (a.E <= 512) return route_r<16>(a, stream, dev, pdl);
    return route_r<32>(a, stream, dev, pdl);
}

cudaError_t launch_gather(const GatherArgs& args, cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    GatherArgs a = args;
    a.stream = passes_l2(2 * static_cast<int64_t>(a.pairs) * a.C);
    const int64_t rows = (static_cast<int64_t>(a.pairs) + kGatherWarps - 1) / kGatherWarps, most = static_cast<int64_t>(dev.num_sms) * kGatherBlocks;
    const dim3 grid(static_cast<unsigned>(rows < most ? rows : most)), block(32 * kGatherWarps);
    if (a.scales != nullptr) return launch_serve(q4k_gather_kernel<uint8_t>, grid, block, 0, stream, pdl, 1, a);
    return launch_serve(q4k_gather_kernel<uint16_t>, grid, block, 0, stream, pdl, 1, a);
}

cudaError_t launch_combine(const CombineArgs& args, cudaStream_t stream, int pdl) {
    CombineArgs a = args;
    a.stream = passes_l2(4 * a.T * a.C);
    const int c8 = a.C / 8;
    int bx = 1;
    while (bx < c8 && bx < 256) bx *= 2;
    const int by = 256 / bx, per = (c8 + bx - 1) / bx;
    const int64_t grid = (a.T + by - 1) / by * per;
    return launch_serve(q4k_combine_kernel, dim3(static_cast<unsigned>(grid)), dim3(bx, by), 0, stream, pdl, 1, a);
}

}  // namespace q4k
