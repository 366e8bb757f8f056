// q4k_logits.cu -- penalties for repeated tokens, biases and a grammar mask on
// the logits, and the greedy pick, in one pass.
//
// A logit is read once (and written once if kept): the bound is the memory's
// rate for many rows, and latency for one. A cluster of CTAs shares a row, so
// that one row is spread over several SMs without a second launch: the CTAs'
// best candidates meet in the first one's shared memory.
//
// Few tokens of a row are penalised or biased, so these are taken apart, by four
// warps of their own, while the other warps stream all logits past the grammar
// mask at a few instructions each, four at a time, with one comparison per four.
// The four warps count the history into a table of the CTA's part of the row in
// shared memory (integer atomics: their order does not matter; 16 bits per logit
// unless the history is long enough to overflow them); tokens counted for the
// first time go on a list, and the tokens of the list are adjusted one by one
// and go over the streamed logits at the end. A thread whose largest logit turns
// out to be one of them has its logits looked through again, by a warp, without
// the ones on the list.
// (Penalties applied where the logits stream by took 68 instructions per logit,
// half of the warps dividing for one lane's token: 43 us for 64 rows of 151936,
// issue-bound. The same steps before or after the stream, by all warps: 33 and 35
// us, 27 with the row asked for into L2 before. Beside the stream an access of
// shared memory takes about half a microsecond, as it queues behind the stream's:
// with the tables cleared by all warps first, one atomic operation per
// history entry, eight of them in flight, and one per warp and batch for the
// list's places, 22 us, 3.6 TB/s; one entry after another, three atomics each:
// 26 us. 200 rows of 50257, not kept: 13.4 us, 3.1 TB/s; one row of 128256: 5.8 us.
// Of the 22 us the stream is 13; the rest is the chain before and after
// it: starts, the list, the look again, the cluster's exchange.)
//
// Rows start at any multiple of 4 bytes (V may be odd), so a row is cut into
// the 16-byte groups of the memory, the first and last of them partly used.
#include <algorithm>

#include "q4k_device.cuh"
#include "q4k_serve.h"

namespace q4k {

namespace {

constexpr int kPickThreads = 512;
constexpr int kPickApart = 128;          // threads that see to the penalised and biased tokens
constexpr int kPickBatch = 3;            // groups of 4 logits that a thread has in flight
constexpr int kPickTableGroups = 7168;   // groups that the tables cover at most
constexpr int kPickList = 1024;          // adjusted tokens that wait for the end of the stream
constexpr int kPickMaxCluster = 8;

// Bytes of the tables of `groups` groups (a multiple of 32): a 16-bit count per
// logit, a bit per logit that is not on the list for want of room; the list.
__host__ __device__ constexpr int pick_late_bytes(int groups) { return groups / 2; }
__host__ __device__ constexpr int pick_tables_bytes(int groups) {
    return pick_late_bytes(groups) + 8 * groups + 8 * kPickList;
}

// The largest number met and its token: by value, then by lower token.
struct Best {
    float x;
    uint32_t v;
    __device__ __forceinline__ void take(float y, uint32_t w) {
        if (y > x || (y == x && w < v)) {
            x = y;
            v = w;
        }
    }
    // Larger is better as an unsigned integer; no number above -infinity: 1 if a
    // token was allowed, else 0. (-0 counts as 0.)
    __device__ __forceinline__ unsigned long long key(bool any) const {
        if (!(x > -INFINITY)) return any;
        const uint32_t u = __float_as_uint(x + 0.f);
        const uint32_t o = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
        return static_cast<unsigned long long>(o) << 32 | (0xFFFFFFFFu - v);
    }
};

struct RowRules {
    int h0, h1, b0, b1;  // the row's history and biases
    float repeat, presence, frequency;
    const uint32_t* mask;

    __device__ __forceinline__ bool allowed(int64_t v) const { return mask == nullptr || (mask[v >> 5] >> (v & 31) & 1u); }
    __device__ __forceinline__ float penalise(float x, uint32_t count) const {
        const float y = x > 0.f ? __fdiv_rn(x, repeat) : __fmul_rn(x, repeat);
        return __fsub_rn(__fsub_rn(y, __fmul_rn(static_cast<float>(count), frequency)), presence);
    }
    // the last entry of the token counts
    __device__ __forceinline__ float add_bias(const PickArgs& a, float x, int v) const {
        for (int i = b1 - 1; i >= b0; --i)
            if (a.bias_ids[i] == v) return __fadd_rn(x, a.bias[i]);
        return x;
    }
};

// The pick of a row that allows some token, but has no number above -infinity:
// the lowest allowed -infinity, else the lowest allowed NaN. One CTA looks
// through the row.
__device__ __noinline__ int64_t pick_rest(const PickArgs& a, RowRules rules, int64_t row) {
    __shared__ int lowest[2];
    if (threadIdx.x < 2) lowest[threadIdx.x] = 0x7FFFFFFF;
    __syncthreads();
    constexpr int kEach = 8;
    for (int64_t v0 = 0; v0 < a.V; v0 += kEach * kPickThreads) {
        for (int e = 0; e < kEach; ++e) {
            const int64_t v = v0 + e * kPickThreads + threadIdx.x;
            if (v >= a.V || !rules.allowed(v)) continue;
            float x;
            if (a.out != nullptr) {
                x = __ldcg(a.out + row + v);  // adjusted already
            } else {
                x = a.logits[row + v];
                if (x == x) {
                    uint32_t count = 0;
                    for (int i = rules.h0; i < rules.h1; ++i) count += a.history[i] == v;
                    if (count) x = rules.penalise(x, count);
                    x = rules.add_bias(a, x, static_cast<int>(v));
                }
            }
            atomicMin(lowest + (x != x), static_cast<int>(v));
        }
        __syncthreads();
        if (lowest[0] != 0x7FFFFFFF) break;  // (read by all before anyone writes again: the loop's barrier is next)
        __syncthreads();
    }
    __syncthreads();
    return lowest[0] != 0x7FFFFFFF ? lowest[0] : lowest[1];
}

}  // namespace

// kAligned: rows begin at multiples of 16 bytes. kApart: there are histories or biases.
template <bool kAligned, bool kApart>
__global__ void __launch_bounds__(kPickThreads, 3)
    q4k_pick_kernel(const __grid_constant__ PickArgs a, int C, int table_groups) {
    constexpr int T = kApart ? kPickThreads - kPickApart : kPickThreads;  // threads that stream
    extern __shared__ __align__(16) uint8_t tables[];
    __shared__ unsigned long long best_s[kPickThreads / 32];
    __shared__ unsigned long long cluster_best[kPickMaxCluster];
    __shared__ int again_s[kApart ? kPickThreads : 1], listed, again;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto clear = [&] {
        for (int i = tid; i < (pick_late_bytes(table_groups) + 8 * table_groups) / 16; i += kPickThreads)
            reinterpret_cast<uint4*>(tables)[i] = make_uint4(0u, 0u, 0u, 0u);
        if (tid == 0) listed = again = 0;
    };
    if (C > 1) cluster_arrive_relaxed();
    if (kApart) clear();
    pdl_wait();
    if (tid == 0) pdl_launch_dependents();
    const int rank = blockIdx.x % C;
    const int64_t m = blockIdx.x / C;
    const int64_t V = a.V, row = m * V;
    const int s = kAligned ? 0 : static_cast<int>(row & 3);  // the row begins s logits into its first group
    const int groups = static_cast<int>((V + s + 3) >> 2), per = (groups + C - 1) / C;
    const int g_begin = min(rank * per, groups), g_end = min(g_begin + per, groups);

    RowRules rules{0, 0, 0, 0, 1.f, 0.f, 0.f, a.mask != nullptr ? a.mask + m * ((V + 31) >> 5) : nullptr};
    if (kApart && a.history != nullptr) {
        rules.h0 = a.hist_starts[m];
        rules.h1 = a.hist_starts[m + 1];
        rules.repeat = a.penalties[3 * m];
        rules.presence = a.penalties[3 * m + 1];
        rules.frequency = a.penalties[3 * m + 2];
    }
    if (kApart && a.bias_ids != nullptr) {
        rules.b0 = a.bias_starts[m];
        rules.b1 = a.bias_starts[m + 1];
    }
    // A token's entry: how often the history has it, and the highest bit if it has a bias.
    const bool wide = rules.h1 - rules.h0 > 32767;
    uint32_t* late = reinterpret_cast<uint32_t*>(tables);
    uint32_t* counts = late + pick_late_bytes(table_groups) / 4;
    int2* list = reinterpret_cast<int2*>(counts + 2 * table_groups);  // token, its bias entry or -1; then its value's bits
    const int step = kApart ? (wide ? table_groups / 2 : table_groups) : groups;  // groups that the tables cover at a time

    Best best{-INFINITY, 0xFFFFFFFFu};
    uint32_t any = rules.mask == nullptr;  // bits 0..3: some token is allowed
    for (int g_tab = g_begin; g_tab < g_end; g_tab += step) {
        if (kApart) __syncthreads();  // the tables are clear
        const int n = min(step, g_end - g_tab);
        const int64_t first = s - 4 * static_cast<int64_t>(g_tab);  // logit v is entry v + first of the tables
        // a token's place in the tables, or -1
        auto place = [&](int v) {
            const int64_t at = v + first;
            return v >= 0 && v < V && at >= 0 && at < 4 * n ? static_cast<int>(at) : -1;
        };
        auto entry = [&](int at) { return counts + (wide ? at : at >> 1); };
        auto shift = [&](int at) { return wide ? 0 : 16 * (at & 1); };
        const uint32_t field = wide ? 0xFFFFFFFFu : 0xFFFFu, flag = field ^ (field >> 1);
        auto adjusted = [&](int at, int v, float bias, bool has_bias) {
            float y = a.logits[row + v];
            const bool ok = rules.allowed(v);
            if (rules.h1 > rules.h0) {
                const uint32_t c = *entry(at) >> shift(at) & (field ^ flag);
                if (c) y = rules.penalise(y, c);
            }
            if (has_bias) y = __fadd_rn(y, bias);
            if (!ok) y = -INFINITY;
            any |= ok;  // (a token in a group that the row fills in part is seen as allowed only here)
            best.take(y, v);
            return y;
        };
        float top = -INFINITY;  // the largest of this thread's groups, and the first logit that has it
        uint32_t top_v = 0xFFFFFFFFu;
        const float4* in = reinterpret_cast<const float4*>(a.logits + (row - s));
        float4* out = reinterpret_cast<float4*>(a.out != nullptr ? a.out + (row - s) : nullptr);
        // groups that the row fills
        const int f0 = max(g_tab, s != 0 ? 1 : 0), f1 = min(g_tab + n, static_cast<int>((V + s) >> 2));
        auto masked = [&](float4 y, const uint32_t* word, uint32_t sh) {
            uint32_t ok = word[0];
            if (kAligned)
                ok >>= sh;
            else
                ok = __funnelshift_r(ok, sh > 28u ? word[1] : 0u, sh);
            any |= ok & 15u;
            y.x = ok & 1u ? y.x : -INFINITY;
            y.y = ok & 2u ? y.y : -INFINITY;
            y.z = ok & 4u ? y.z : -INFINITY;
            y.w = ok & 8u ? y.w : -INFINITY;
            return y;
        };
        if (!kApart || tid < T) {
            // ------------------------------------------------------- the stream ---
            // A thread's groups are T apart, a multiple of 8: their mask bits lie
            // at the same place of words T / 8 apart.
            int g = f0 + tid, top_g = -1;
            // asked for at once, into L2: a thread's own loads are too few to fill the memory's queue
            if (tid == 0 && f1 > f0)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(in + f0), "r"(16 * (f1 - f0)) : "memory");
            const uint32_t mask_sh = (4u * g - s) & 31u;
            const uint32_t* mask_p = rules.mask + ((4u * g - s) >> 5);
            float4 top_y = make_float4(0.f, 0.f, 0.f, 0.f);
            for (; g < f1; g += kPickBatch * T, mask_p += kPickBatch * (T / 8)) {
                float4 x[kPickBatch] = {};
                auto each = [&](int e) {
                    float4 y = x[e];
                    if (rules.mask != nullptr) y = masked(y, mask_p + e * (T / 8), mask_sh);
                    if (out != nullptr) __stcs(out + (g + e * T), y);
                    const float t = fmaxf(fmaxf(y.x, y.y), fmaxf(y.z, y.w));
                    if (t > top) {
                        top = t;
                        top_y = y;
                        top_g = g + e * T;
                    }
                };
                if (g + (kPickBatch - 1) * T < f1) {
#pragma unroll
                    for (int e = 0; e < kPickBatch; ++e) x[e] = __ldcs(in + g + e * T);
#pragma unroll
                    for (int e = 0; e < kPickBatch; ++e) each(e);
                } else {
#pragma unroll
                    for (int e = 0; e < kPickBatch; ++e)
                        if (g + e * T < f1) x[e] = __ldcs(in + g + e * T);
#pragma unroll
                    for (int e = 0; e < kPickBatch; ++e)
                        if (g + e * T < f1) each(e);
                }
            }
            if (top_g >= 0)
                top_v = 4u * top_g - s + (top_y.x == top ? 0u : top_y.y == top ? 1u : top_y.z == top ? 2u : 3u);
        } else {
            // -------------------------------------------- the tokens set apart ---
            const int t = tid - T;
            auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kPickApart) : "memory"); };
            const int h0 = rules.h0, h1 = rules.h1, b0 = rules.b0, b1 = rules.b1;
            // (by whole warps) puts tokens on the list, at places from `to` on
            auto put = [&](int to, int at, int v, int bias_at) {
                if (to < kPickList)
                    list[to] = make_int2(v, bias_at);
                else
                    atomicOr(late + (at >> 5), 1u << (at & 31));
            };
            auto places = [&](int k) { return __shfl_sync(0xffffffffu, lane == 0 ? atomicAdd(&listed, k) : 0, 0); };
            const uint32_t below = (1u << lane) - 1;
            constexpr int kUnroll = 8;  // history entries in flight
            auto history = [&](int i) { return i < h1 ? a.history[i] : -1; };
            int v[kUnroll];
#pragma unroll
            for (int e = 0; e < kUnroll; ++e) v[e] = history(h0 + t + e * kPickApart);
            // biases, by one warp: the last entry of a token counts, so the entries go by from the end
            if (t < 32) {
                for (int i1 = b1; i1 > b0; i1 -= 32) {
                    const int i = i1 - 1 - lane, w = i >= b0 ? a.bias_ids[i] : -1, at = place(w);
                    const bool last = (__match_any_sync(0xffffffffu, w) & below) == 0u;
                    bool is = false;
                    if (at >= 0 && last) is = !(atomicOr(entry(at), flag << shift(at)) >> shift(at) & flag);
                    const uint32_t m = __ballot_sync(0xffffffffu, is);
                    if (m == 0u) continue;
                    const int to = places(__popc(m));
                    if (is) put(to + __popc(m & below), at, w, i);
                }
            }
            sync();
            for (int i0 = h0; i0 < h1; i0 += kUnroll * kPickApart) {
                uint32_t first[kUnroll];
                if (i0 != h0)
#pragma unroll
                    for (int e = 0; e < kUnroll; ++e) v[e] = history(i0 + t + e * kPickApart);
#pragma unroll
                for (int e = 0; e < kUnroll; ++e) {  // (a bias has its token on the list already)
                    const int at = place(v[e]);
                    first[e] = at >= 0 ? atomicAdd(entry(at), 1u << shift(at)) >> shift(at) & field : 1u;
                }
                int news = 0;
#pragma unroll
                for (int e = 0; e < kUnroll; ++e) {
                    first[e] = __ballot_sync(0xffffffffu, first[e] == 0u);
                    news += __popc(first[e]);
                }
                if (news == 0) continue;
                int to = places(news);
#pragma unroll
                for (int e = 0; e < kUnroll; ++e) {
                    if (first[e] >> lane & 1u) put(to + __popc(first[e] & below), place(v[e]), v[e], -1);
                    to += __popc(first[e]);
                }
            }
            sync();
            for (int i = t; i < min(listed, kPickList); i += kPickApart) {
                const int2 e = list[i];
                const float bias = e.y >= 0 ? a.bias[e.y] : 0.f;
                list[i].y = __float_as_int(adjusted(place(e.x), e.x, bias, e.y >= 0));
            }
        }
        auto marked = [&](int64_t v) {
            const int at = static_cast<int>(v + first);
            return kApart && (*entry(at) >> shift(at) & field) != 0u;
        };
        if (kApart) {
            __syncthreads();  // all is listed, and the logits are written
            if (a.out != nullptr)
                for (int i = tid; i < min(listed, kPickList); i += kPickThreads)
                    a.out[row + list[i].x] = __int_as_float(list[i].y);
            if (listed > kPickList) {  // the others, by whoever takes them first
                auto take = [&](int v) {
                    const int at = place(v);
                    if (at < 0) return;
                    const uint32_t bit = 1u << (at & 31);
                    if (!(atomicAnd(late + (at >> 5), ~bit) & bit)) return;
                    float bias = 0.f;
                    bool has_bias = false;
                    for (int i = rules.b1 - 1; i >= rules.b0 && !has_bias; --i)
                        if (a.bias_ids[i] == v) {
                            bias = a.bias[i];
                            has_bias = true;
                        }
                    const float y = adjusted(at, v, bias, has_bias);
                    if (a.out != nullptr) a.out[row + v] = y;
                };
                for (int i = rules.h0 + tid; i < rules.h1; i += kPickThreads) take(a.history[i]);
                for (int i = rules.b0 + tid; i < rules.b1; i += kPickThreads) take(a.bias_ids[i]);
            }
        }
        if (top_v != 0xFFFFFFFFu) {
            if (!marked(top_v))
                best.take(top, top_v);
            else
                again_s[atomicAdd(&again, 1)] = tid;
        }
        if (kApart) {
            __syncthreads();
            // the logits of a thread whose largest was set apart, without those that were
            for (int i = warp; i < again; i += kPickThreads / 32)
                for (int g = f0 + again_s[i] + lane * T; g < f1; g += 32 * T) {
                    float4 y = out != nullptr ? __ldcg(out + g) : in[g];
                    const uint32_t v0 = 4u * g - s;
                    if (out == nullptr && rules.mask != nullptr) y = masked(y, rules.mask + (v0 >> 5), v0 & 31u);
                    const float z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (!marked(v0 + k)) best.take(z[k], v0 + k);
                }
        }
        // the logits of the groups at the row's ends that it fills in part
        if (tid < 8) {
            const int64_t v = tid < 4 ? tid : ((V + s) >> 2 << 2) - s + (tid - 4);
            const int64_t at = v + first;
            const bool mine = tid < 4 ? s != 0 && tid < 4 - s : v >= (s != 0 ? 4 - s : 0);
            if (mine && v < V && at >= 0 && at < 4 * n && !marked(v)) {
                const bool ok = rules.allowed(v);
                any |= ok;
                const float y = ok ? a.logits[row + v] : -INFINITY;
                if (a.out != nullptr) a.out[row + v] = y;
                best.take(y, static_cast<uint32_t>(v));
            }
        }
        if (kApart && g_tab + step < g_end) {
            __syncthreads();  // the tables are read
            clear();
        }
    }

    if (a.pick == nullptr) {
        if (C > 1) cluster_wait();  // (each arrival waits once)
        return;
    }
    unsigned long long key = best.key(any != 0u);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long k = __shfl_xor_sync(0xffffffffu, key, o);
        key = k > key ? k : key;
    }
    if (lane == 0) best_s[warp] = key;
    __syncthreads();
    key = lane < kPickThreads / 32 ? best_s[lane] : 0ull;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long k = __shfl_xor_sync(0xffffffffu, key, o);
        key = k > key ? k : key;
    }
    if (C > 1) {
        cluster_wait();  // every CTA of the cluster has begun
        if (tid == 0)
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(map_shared_rank(smem_u32(cluster_best + rank), 0)),
                         "l"(key)
                         : "memory");
        cluster_sync_all();
        if (rank == 0)
            for (int r = 0; r < C; ++r) key = cluster_best[r] > key ? cluster_best[r] : key;
    }
    if (rank != 0) return;
    int64_t pick = key == 0ull ? -1 : static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
    if (key == 1ull) {
        __syncthreads();
        pick = pick_rest(a, rules, row);
    }
    if (tid == 0) a.pick[m] = pick;
}

cudaError_t launch_pick(const PickArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    // as many CTAs per row as still run at once, and none without a batch for every thread
    const int64_t groups = (a.V + 6) / 4;
    int64_t C = std::min<int64_t>(groups / (kPickThreads * kPickBatch) + 1, kPickMaxCluster);
    while (C > 1 && a.M > dev.pick_clusters[C]) --C;
    const int64_t per = (groups + C - 1) / C;
    const int table_groups = static_cast<int>(std::min<int64_t>(kPickTableGroups, (per + 31) / 32 * 32));
    const bool aligned = a.V % 4 == 0, apart = a.history != nullptr || a.bias_ids != nullptr;
    auto kernel = aligned ? (apart ? q4k_pick_kernel<true, true> : q4k_pick_kernel<true, false>)
                          : (apart ? q4k_pick_kernel<false, true> : q4k_pick_kernel<false, false>);
    return launch_serve(kernel, dim3(static_cast<unsigned>(a.M * C)), dim3(kPickThreads),
                        apart ? pick_tables_bytes(table_groups) : 0, stream, pdl, static_cast<int>(C), a,
                        static_cast<int>(C), table_groups);
}

cudaError_t pick_setup(DeviceInfo& dev) {
    const int smem = pick_tables_bytes(kPickTableGroups);
    cudaError_t e = cudaFuncSetAttribute(q4k_pick_kernel<true, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(q4k_pick_kernel<false, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    for (int c = 2; c <= kPickMaxCluster; ++c) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(c);
        cfg.blockDim = dim3(kPickThreads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = c;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, q4k_pick_kernel<true, true>, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            n = 0;
        }
        dev.pick_clusters[c] = n;
    }
    return cudaSuccess;
}

}  // namespace q4k
