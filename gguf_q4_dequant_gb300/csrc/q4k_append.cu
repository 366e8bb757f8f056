// q4k_append.cu -- a step's keys and values into the pages of one layer, and
// its queries for the attention: per-head norm, rotary positions, one rounding
// to bf16.
//
// Nothing is reused: 4 bytes are read and 2 written per element, so the bound
// is the memory's rate, and for a decode batch the launch. A row of head_dim
// elements is held by head_dim/4 lanes, four adjacent elements each (one
// 16-byte load, one 8-byte store): adjacent pairs lie in one lane, and the
// partner of a pair (i, i + head_dim/2) is half a row's lanes away, so both
// pairings and the norm's sum stay inside the row's lanes. One block per token
// finds the token's sequence and page once for all heads.
#include <cuda_bf16.h>

#include "q4k_device.cuh"
#include "q4k_serve.h"

namespace q4k {

constexpr int kAppThreads = 256;

__device__ __forceinline__ uint2 bf16x4(float4 x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

template <int D>
__global__ void __launch_bounds__(kAppThreads)
    q4k_append_kernel(const CacheLayer c, const Batch b, const float* __restrict__ Yq,
                      const float* __restrict__ Yk, const float* __restrict__ Yv,
                      uint16_t* __restrict__ q_out, int heads, const float* __restrict__ rope, int pairs,
                      const float* __restrict__ q_norm, const float* __restrict__ k_norm, float eps) {
    constexpr int L = D / 4;  // lanes per row
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const int t = blockIdx.x;
    // the sequence: as many of starts[1 ..] as are not above t
    int i = 0;
    for (int j = 0; j < b.n; j += kAppThreads)
        i += __syncthreads_count(j + threadIdx.x < b.n && b.starts[j + threadIdx.x + 1] <= t);
    int64_t pos = -1, off = -1;
    if (i < b.n) {
        const SeqView s = seq_view(c, b, i);
        const int r = t - s.t0;
        if (r >= 0 && r < s.m) pos = static_cast<int64_t>(s.len) - s.m + r;
        if (pos >= 0) {
            const int page = c.table[s.row + (pos >> c.page_shift)];
            if (page >= 0 && page < c.n_pages)
                off = page * c.page_stride + (pos & ((1 << c.page_shift) - 1)) * D;
        }
    }
    const int lane = threadIdx.x % L;
    float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool turn = pairs != 0 && pos >= 0;
    if (turn) {
        const float* row = rope + pos * D;
        if (pairs == 1) {
            const float2 c2 = *reinterpret_cast<const float2*>(row + 2 * lane);
            const float2 s2 = *reinterpret_cast<const float2*>(row + D / 2 + 2 * lane);
            cs = make_float4(c2.x, c2.x, c2.y, c2.y);
            sn = make_float4(-s2.x, s2.x, -s2.y, s2.y);
        } else {
            const int k = 4 * (lane % (L / 2));
            cs = *reinterpret_cast<const float4*>(row + k);
            sn = *reinterpret_cast<const float4*>(row + D / 2 + k);
            if (lane < L / 2) sn = make_float4(-sn.x, -sn.y, -sn.z, -sn.w);
        }
    }
    const int G = c.kv_heads, rows = heads + 2 * G;
    // whole warps keep together: the shuffles need every lane of a row
    for (int h0 = 0; h0 < rows; h0 += kAppThreads / L) {
        const int h = h0 + threadIdx.x / L;
        const bool in = h < rows;
        const bool is_q = h < heads, is_v = h >= heads + G;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (in) {
            const float* src = is_q   ? Yq + (static_cast<int64_t>(t) * heads + h) * D
                               : is_v ? Yv + (static_cast<int64_t>(t) * G + h - heads - G) * D
                                      : Yk + (static_cast<int64_t>(t) * G + h - heads) * D;
            x = __ldcs(reinterpret_cast<const float4*>(src) + lane);
        }
        const float* w = is_q ? q_norm : is_v ? nullptr : k_norm;
        float ss = x.x * x.x + x.y * x.y + x.z * x.z + x.w * x.w;
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (w != nullptr) {
            const float4 wv = *reinterpret_cast<const float4*>(w + 4 * lane);
            const float f = 1.f / sqrtf(ss * (1.f / D) + eps);
            x = make_float4(x.x * f * wv.x, x.y * f * wv.y, x.z * f * wv.z, x.w * f * wv.w);
        }
        float4 y;  // the other element of each pair
        if (pairs == 2) {
            y.x = __shfl_xor_sync(0xffffffffu, x.x, L / 2);
            y.y = __shfl_xor_sync(0xffffffffu, x.y, L / 2);
            y.z = __shfl_xor_sync(0xffffffffu, x.z, L / 2);
            y.w = __shfl_xor_sync(0xffffffffu, x.w, L / 2);
        } else {
            y = make_float4(x.y, x.x, x.w, x.z);
        }
        if (turn && !is_v)
            x = make_float4(x.x * cs.x + y.x * sn.x, x.y * cs.y + y.y * sn.y, x.z * cs.z + y.z * sn.z,
                            x.w * cs.w + y.w * sn.w);
        if (!in) continue;
        if (is_q) {
            *(reinterpret_cast<uint2*>(q_out + (static_cast<int64_t>(t) * heads + h) * D) + lane) = bf16x4(x);
        } else if (off >= 0) {
            const int g = is_v ? h - heads - G : h - heads;
            uint16_t* dst = (is_v ? c.v : c.k) + off + (static_cast<int64_t>(g) << c.page_shift) * D;
            *(reinterpret_cast<uint2*>(dst) + lane) = bf16x4(x);
        }
    }
}

cudaError_t launch_append(const CacheLayer& c, const Batch& b, const float* Yq, const float* Yk,
                          const float* Yv, uint16_t* q_out, int heads, int head_dim, const float* rope,
                          int pairs, const float* q_norm, const float* k_norm, float eps,
                          cudaStream_t stream, int pdl) {
    auto kernel = head_dim == 64 ? q4k_append_kernel<64> : q4k_append_kernel<128>;
    return launch_serve(kernel, dim3(b.tokens), dim3(kAppThreads), 0, stream, pdl, 1, c, b, Yq, Yk, Yv, q_out,
                        heads, rope, pairs, q_norm, k_norm, eps);
}

}  // namespace q4k
