// q4k_experts.h -- what the kernels of an expert layer share: the device view of
// the rows sorted by expert, and the host-side launchers. Not part of the public
// interface.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "q4k.h"
#include "q4k_internal.h"

namespace q4k {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTop = 32;

// Whether results of so many bytes are written past L2 (129 MB): more than about half of it.
inline bool passes_l2(int64_t bytes) { return bytes > (int64_t(64) << 20); }

// The rows of a step in the order of their experts: expert e has rows
// starts[e] .. starts[e+1]-1 of `pairs` rows.
struct ExpertRows {
    const int32_t* starts;  // [experts + 1]
    int experts, pairs;
};

#ifdef __CUDACC__
// The row tiles (of up to NT rows) of every expert, by one warp: starts[0 .. E]
// (shared memory, inside [0, pairs] whatever the caller's array held) are made
// ascending, tiles[e] becomes the number of tiles before expert e, tiles[E] of all.
// A lane has (E + 32) / 32 entries side by side.
template <int NT>
__device__ __forceinline__ void expert_tiles(int* starts, int* tiles, int E, int lane) {
    const int per = E / 32 + 1, e0 = lane * per, e1 = min(e0 + per, E + 1);
    int high = 0;  // the highest up to this lane's last
    for (int e = e0; e < e1; ++e) high = max(high, starts[e]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, high, o);
        if (lane >= o) high = max(high, t);
    }
    int prev = __shfl_up_sync(0xffffffffu, high, 1);
    if (lane == 0) prev = e1 > e0 ? starts[0] : 0;
    // the tiles of experts e0 - 1 .. e1 - 2, whose rows end at starts[e0 .. e1 - 1]
    int sum = 0;
    for (int e = e0, p = prev; e < e1; ++e) {
        const int hi = max(p, starts[e]);
        starts[e] = hi;
        sum += (hi - p + NT - 1) / NT;
        p = hi;
    }
    int at = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += t;
    }
    at -= sum;
    for (int e = e0, p = prev; e < e1; ++e) {
        at += (starts[e] - p + NT - 1) / NT;
        p = starts[e];
        tiles[e] = at;
    }
}

// g / (1 + exp(-g)) with the approximate base-2 exponential and reciprocal, results
// below 2^-126 as 0: a few units in the last place of fp32, for a result that is
// rounded to bf16; 0 where exp(-g) overflows.
__device__ __forceinline__ float silu(float g) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return g * r;
}

// The expert of row tile `tile` < tiles[E]: the last e with tiles[e] <= tile.
__device__ __forceinline__ int expert_of(const int* tiles, int E, int tile) {
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tiles[mid] <= tile) lo = mid; else hi = mid;
    }
    return lo;
}

// The same by a whole warp: of every 32nd expert, then of the 32 from there.
__device__ __forceinline__ int expert_at(const int* tiles, int E, int tile, int lane) {
    const int i = 32 * lane;
    const int b = 32 * (__popc(__ballot_sync(0xffffffffu, i < E && tiles[i] <= tile)) - 1), j = b + lane;
    return b + __popc(__ballot_sync(0xffffffffu, j < E && tiles[j] <= tile)) - 1;
}
#endif

struct NormArgs {
    const void* x;
    const float* delta;
    const float* weight;
    void* sum;
    void* out;
    uint8_t* codes;
    uint8_t* scales;
    int64_t T;
    int C;
    float eps;
    bool x_bf16, out_bf16;
    bool stream = false;  // set by the launcher
};
cudaError_t launch_add_norm(const NormArgs& a, cudaStream_t stream, int pdl);

struct RouteArgs {
    const float* logits;
    int T, E, k, weighting;
    float scale;
    int32_t* ids;
    float* weights;
    int32_t *order, *slots, *starts;
    int32_t* ws;
};
int64_t route_scratch_bytes(int64_t T, int E);
cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl);

struct GatherArgs {
    const void* x;
    const uint8_t* scales;  // NULL: bf16 rows, else e4m3 codes and these exponents
    const int32_t* order;
    uint16_t* out;
    int T, C, k, pairs;
    bool stream = false;  // set by the launcher
};
cudaError_t launch_gather(const GatherArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl);

struct CombineArgs {
    const uint16_t* y;
    const int32_t* slots;
    const float* weights;
    const float* base;
    float* out;
    int64_t T;
    int C, k, pairs;
    bool stream = false;  // set by the launcher
};
cudaError_t launch_combine(const CombineArgs& a, cudaStream_t stream, int pdl);

struct ExpertArgs {
    const uint8_t* W;
    const uint8_t* W2;  // the up matrices of a gated product, or NULL
    int64_t N, K;
    const uint16_t* X;
    ExpertRows rows;
    uint16_t* Y;
};
cudaError_t launch_experts(const ExpertArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl);
cudaError_t experts_setup(DeviceInfo& dev);
cudaError_t launch_experts_gemm(const ExpertArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl);
double experts_gemm_us(const ExpertArgs& a, const DeviceInfo& dev);  // its time, about
cudaError_t experts_gemm_setup();

// A 2-D byte map {K/256*144, N} of packed rows, box one super-block of `rows` rows
// (a q4k_status; cached per host thread).
int weight_map(CUtensorMap* map, const void* W, int64_t N, int64_t K, int rows);
// Rows of bf16 [rows][K], box 64 k x box_rows rows with the 128-byte swizzle (the same).
int rows_map(CUtensorMap* map, const void* X, int64_t rows, int64_t K, int box_rows);

}  // namespace q4k
