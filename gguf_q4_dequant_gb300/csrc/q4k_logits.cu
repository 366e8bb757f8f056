// q4k_logits.cu -- penalties for repeated tokens, biases and a grammar mask on
// the logits, and the greedy pick, in one pass.
//
// A logit is read once (and written once if kept): the bound is the memory's
// rate for many rows, and latency for one. A cluster of CTAs shares a row, so
// that one row is spread over several SMs without a second launch: the CTAs'
// best candidates meet in the first one's shared memory. A CTA takes its part
// of the row in chunks of 16 logits per thread, loaded into registers first;
// while they are on their way, the row's history is counted into a table of the
// chunk in shared memory (integer atomics: order does not matter), and the
// bias entries leave their index there (the largest wins).
//
// Rows start at any multiple of 4 bytes (V may be odd), so a row is cut into
// the 16-byte groups of the memory, the first and last of them partly used.
#include "q4k_device.cuh"
#include "q4k_serve.h"

namespace q4k {

namespace {

constexpr int kPickThreads = 512;
constexpr int kPickGroups = 4;  // groups of 4 logits per thread and chunk
constexpr int kPickChunk = kPickThreads * kPickGroups;  // groups
constexpr int kPickMaxCluster = 8;

// Orders floats as unsigned integers: numbers by value (-0 as 0) above NaN (1)
// above a token that is not allowed (0).
__device__ __forceinline__ uint32_t pick_order(float x, bool allowed) {
    const uint32_t u = __float_as_uint(x + 0.f);
    const uint32_t o = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
    return !allowed ? 0u : x != x ? 1u : o;
}

}  // namespace

__global__ void __launch_bounds__(kPickThreads)
    q4k_pick_kernel(const PickArgs a, int C) {
    extern __shared__ uint32_t tables[];  // counts, bias indices: one word per logit of the chunk
    __shared__ unsigned long long best_s[kPickThreads / 32];
    __shared__ unsigned long long cluster_best[kPickMaxCluster];
    if (C > 1) cluster_arrive_relaxed();
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x % C;
    const int64_t m = blockIdx.x / C;
    const int64_t V = a.V, row = m * V;
    const int s = static_cast<int>(row & 3);  // the row begins s logits into its first group
    const float* in = a.logits + (row - s);
    float* out = a.out != nullptr ? a.out + (row - s) : nullptr;
    const int64_t groups = (V + s + 3) >> 2, per = (groups + C - 1) / C;
    const int64_t g_end = min(groups, (rank + 1) * per);

    int h0 = 0, h1 = 0, b0 = 0, b1 = 0;
    float repeat = 1.f, presence = 0.f, frequency = 0.f;
    if (a.history != nullptr) {
        h0 = a.hist_starts[m];
        h1 = a.hist_starts[m + 1];
        repeat = a.penalties[3 * m];
        presence = a.penalties[3 * m + 1];
        frequency = a.penalties[3 * m + 2];
    }
    if (a.bias_ids != nullptr) {
        b0 = a.bias_starts[m];
        b1 = a.bias_starts[m + 1];
    }
    const bool counted = h1 > h0, biased = b1 > b0;
    uint32_t* counts = tables;
    uint32_t* places = tables + (a.history != nullptr ? 4 * kPickChunk : 0);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int e = 0; e < kPickGroups; ++e) {
        if (counted) reinterpret_cast<uint4*>(counts)[tid + e * kPickThreads] = zero;
        if (biased) reinterpret_cast<uint4*>(places)[tid + e * kPickThreads] = zero;
    }
    const uint32_t* mask = a.mask != nullptr ? a.mask + m * ((V + 31) >> 5) : nullptr;

    uint32_t top = 0u, top_at = 0u;
    for (int64_t ga = rank * per; ga < g_end; ga += kPickChunk) {
        float x[kPickGroups][4];
        uint32_t bits[kPickGroups];
#pragma unroll
        for (int e = 0; e < kPickGroups; ++e) {
            const int64_t g = ga + tid + e * kPickThreads, v0 = 4 * g - s;
            bits[e] = 0u;
            if (g >= g_end) continue;
            if (v0 >= 0 && v0 + 4 <= V) {
                const float4 f = __ldcs(reinterpret_cast<const float4*>(in) + g);
                x[e][0] = f.x;
                x[e][1] = f.y;
                x[e][2] = f.z;
                x[e][3] = f.w;
                bits[e] = 15u;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const bool is = v0 + k >= 0 && v0 + k < V;
                    x[e][k] = is ? in[4 * g + k] : 0.f;
                    bits[e] |= is ? 1u << k : 0u;
                }
            }
            if (mask != nullptr) {
                const int64_t w = (v0 < 0 ? 0 : v0) >> 5;
                const int sh = static_cast<int>(v0 & 31);
                const uint32_t lo = mask[w];
                uint32_t ok;
                if (v0 < 0)
                    ok = lo << -v0;
                else
                    ok = __funnelshift_r(lo, sh > 28 && 32 * (w + 1) < V ? mask[w + 1] : 0u, sh);
                bits[e] |= (~ok & 15u) << 4;  // forbidden
            }
        }
        if (counted || biased) {
            __syncthreads();  // the tables are clear
            // logit v of the row is entry v + first of the chunk's tables
            const int64_t first = s - 4 * ga;
            const int64_t entries = 4 * min(static_cast<int64_t>(kPickChunk), g_end - ga);
            for (int i = h0 + tid; i < h1; i += kPickThreads) {
                const int v = a.history[i];
                const int64_t at = v + first;
                if (v >= 0 && v < V && at >= 0 && at < entries) atomicAdd(counts + at, 1u);
            }
            for (int i = b0 + tid; i < b1; i += kPickThreads) {
                const int v = a.bias_ids[i];
                const int64_t at = v + first;
                if (v >= 0 && v < V && at >= 0 && at < entries) atomicMax(places + at, static_cast<uint32_t>(i - b0) + 1u);
            }
            __syncthreads();
        }
#pragma unroll
        for (int e = 0; e < kPickGroups; ++e) {
            const int64_t g = ga + tid + e * kPickThreads, v0 = 4 * g - s;
            if (g >= g_end) continue;
            if (counted) {
                uint4* slot = reinterpret_cast<uint4*>(counts) + tid + e * kPickThreads;
                const uint4 c4 = *slot;
                if ((c4.x | c4.y | c4.z | c4.w) != 0u) {
                    *slot = zero;  // for the next chunk
                    const uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (c[k] != 0u) {
                            const float y = x[e][k] > 0.f ? __fdiv_rn(x[e][k], repeat) : __fmul_rn(x[e][k], repeat);
                            x[e][k] = __fsub_rn(__fsub_rn(y, __fmul_rn(static_cast<float>(c[k]), frequency)), presence);
                        }
                }
            }
            if (biased) {
                uint4* slot = reinterpret_cast<uint4*>(places) + tid + e * kPickThreads;
                const uint4 p4 = *slot;
                if ((p4.x | p4.y | p4.z | p4.w) != 0u) {
                    *slot = zero;
                    const uint32_t p[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (p[k] != 0u) x[e][k] = __fadd_rn(x[e][k], a.bias[b0 + p[k] - 1u]);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool allowed = (bits[e] >> k & 0x11u) == 1u;
                if ((bits[e] >> (k + 4)) & 1u) x[e][k] = -INFINITY;
                const uint32_t o = pick_order(x[e][k], allowed);
                if (o > top) {
                    top = o;
                    top_at = static_cast<uint32_t>(v0 + k);
                }
            }
            if (out != nullptr) {
                if ((bits[e] & 15u) == 15u) {
                    __stcs(reinterpret_cast<float4*>(out) + g, make_float4(x[e][0], x[e][1], x[e][2], x[e][3]));
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (bits[e] >> k & 1u) out[4 * g + k] = x[e][k];
                }
            }
        }
    }

    // larger value first, then lower index
    unsigned long long key = static_cast<unsigned long long>(top) << 32 | (0xFFFFFFFFu - top_at);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long k = __shfl_xor_sync(0xffffffffu, key, o);
        key = k > key ? k : key;
    }
    if (lane == 0) best_s[warp] = key;
    __syncthreads();
    if (warp == 0) {
        key = lane < kPickThreads / 32 ? best_s[lane] : 0ull;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long k = __shfl_xor_sync(0xffffffffu, key, o);
            key = k > key ? k : key;
        }
    }
    if (C > 1) {
        cluster_wait();  // every CTA of the cluster has begun
        if (tid == 0)
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(map_shared_rank(smem_u32(cluster_best + rank), 0)),
                         "l"(key)
                         : "memory");
        cluster_sync_all();
        if (rank == 0 && tid == 0)
            for (int r = 0; r < C; ++r) key = cluster_best[r] > key ? cluster_best[r] : key;
    }
    if (rank == 0 && tid == 0 && a.pick != nullptr)
        a.pick[m] = (key >> 32) == 0ull ? -1 : static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
}

cudaError_t launch_pick(const PickArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    // as many CTAs per row as still run at once, and no more than have a chunk's worth
    int C = kPickMaxCluster;
    while (C > 1 && (a.M * C > 3 * dev.num_sms || (a.V + 3) / 4 <= static_cast<int64_t>(kPickChunk) * (C / 2))) C /= 2;
    const size_t smem = static_cast<size_t>((a.history != nullptr) + (a.bias_ids != nullptr)) * 16 * kPickChunk;
    return launch_serve(q4k_pick_kernel, dim3(static_cast<unsigned>(a.M * C)), dim3(kPickThreads), smem, stream, pdl, C,
                        a, C);
}

cudaError_t pick_setup() {
    return cudaFuncSetAttribute(q4k_pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * 16 * kPickChunk);
}

}  // namespace q4k
