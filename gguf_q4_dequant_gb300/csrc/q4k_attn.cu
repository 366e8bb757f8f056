// q4k_attn.cu -- attention of a step's new tokens over the pages of one layer.
//
// One warp per (token, head): 32 keys at a time, a lane each for the scores
// (running maximum and sum over the blocks), then the lanes share the
// dimensions of V for the weighted sum, over the visible keys only.
#include <cuda_bf16.h>

#include "q4k_device.cuh"
#include "q4k_serve.h"

namespace q4k {

constexpr int kAttnWarps = 4;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <int D>
__global__ void __launch_bounds__(32 * kAttnWarps)
    q4k_attn_simple_kernel(const CacheLayer c, const Batch b, const uint16_t* __restrict__ Q,
                           uint16_t* __restrict__ out, int heads, float scale, int window, int sinks) {
    __shared__ float q_s[kAttnWarps][D];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kAttnWarps + warp;
    if (item >= static_cast<int64_t>(b.tokens) * heads) return;
    const int t = static_cast<int>(item / heads), h = static_cast<int>(item % heads);
    int i = 0;
    for (int j = lane; j < b.n; j += 32) i += b.starts[j + 1] <= t;
    i = __reduce_add_sync(0xffffffffu, i);
    if (i >= b.n) return;
    const SeqView s = seq_view(c, b, i);
    if (t < s.t0 || t >= s.t0 + s.m) return;
    const int p = s.len - s.m + (t - s.t0);
    const int g = h / (heads / c.kv_heads);
    for (int d = lane; d < D; d += 32) q_s[warp][d] = bf16_lo(Q[item * D + d]);
    __syncwarp();
    float acc[D / 32], top = -INFINITY, total = 0.f;
    for (int d = 0; d < D / 32; ++d) acc[d] = 0.f;
    const int mask = (1 << c.page_shift) - 1;
    for (int j0 = 0; j0 <= p; j0 += 32) {
        if (window > 0 && j0 >= sinks && j0 + 31 <= p - window) continue;
        const int j = j0 + lane;
        const bool sees = j <= p && (window == 0 || j > p - window || j < sinks);
        int page = sees ? c.table[s.row + (j >> c.page_shift)] : -1;
        if (page >= c.n_pages) page = -1;
        const int64_t off = page < 0 ? -1 : page * c.page_stride + ((static_cast<int64_t>(g) << c.page_shift) + (j & mask)) * D;
        float x = -INFINITY;
        if (sees) {
            x = 0.f;
            if (off >= 0)
                for (int d = 0; d < D; d += 8) {
                    const uint4 kv = *reinterpret_cast<const uint4*>(c.k + off + d);
                    const uint32_t w[4] = {kv.x, kv.y, kv.z, kv.w};
                    for (int e = 0; e < 4; ++e) {
                        x = fmaf(bf16_lo(w[e]), q_s[warp][d + 2 * e], x);
                        x = fmaf(bf16_hi(w[e]), q_s[warp][d + 2 * e + 1], x);
                    }
                }
            x *= scale;
        }
        float m = x;
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = fmaxf(m, top);
        const float base = m == -INFINITY ? 0.f : m;
        const float keep = expf(top - base);
        const float a = sees ? expf(x - base) : 0.f;
        top = m;
        total = total * keep + a;
        for (int d = 0; d < D / 32; ++d) acc[d] *= keep;
        uint32_t vis = __ballot_sync(0xffffffffu, sees);
        while (vis) {
            const int l = __ffs(vis) - 1;
            vis &= vis - 1;
            const float al = __shfl_sync(0xffffffffu, a, l);
            const int64_t ol = __shfl_sync(0xffffffffu, off, l);
            if (ol >= 0)
                for (int d = 0; d < D / 32; ++d) acc[d] = fmaf(al, bf16_lo(c.v[ol + d * 32 + lane]), acc[d]);
        }
    }
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    for (int d = 0; d < D / 32; ++d) {
        const __nv_bfloat16 y = __float2bfloat16_rn(total == 0.f ? 0.f : acc[d] / total);
        out[item * D + d * 32 + lane] = __bfloat16_as_ushort(y);
    }
}

cudaError_t launch_attention(const CacheLayer& c, const Batch& b, const AttnArgs& a, int max_new,
                             cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    (void)max_new;
    (void)dev;
    auto kernel = a.head_dim == 64 ? q4k_attn_simple_kernel<64> : q4k_attn_simple_kernel<128>;
    const int64_t items = static_cast<int64_t>(b.tokens) * a.heads;
    return launch_serve(kernel, dim3(static_cast<unsigned>((items + kAttnWarps - 1) / kAttnWarps)),
                        dim3(32 * kAttnWarps), 0, stream, pdl, 1, c, b, a.Q, a.out, a.heads, a.scale, a.window,
                        a.sinks);
}

int64_t attn_scratch_bytes(const DeviceInfo&, int) { return 0; }
cudaError_t attn_setup(DeviceInfo&) { return cudaSuccess; }

}  // namespace q4k
