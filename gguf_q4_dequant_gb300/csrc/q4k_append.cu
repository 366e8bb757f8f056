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
// finds the token's sequence and page once for all heads, while the first rows
// are on their way: that takes four loads, each from the result of the one
// before. 2894 tokens of 48 rows, 108 MB: 21 us, 5.2 TB/s (26 us when the rows
// were loaded after the place was known and the norm's and rotation's steps were
// taken whether wanted or not); with a norm 2894 tokens of 56 rows take 28 us for 23,
// with rotation 33: five shuffles per row, and registers for 4 blocks per SM only.
// 64 tokens of 56 rows: 3.8 us, the launch and the four loads.
#include <cuda_bf16.h>

#include "q4k_device.cuh"
#include "q4k_serve.h"

namespace q4k {

__device__ __forceinline__ uint2 bf16x4(float4 x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// A token is one block's, of one of two widths: wide, with all rows on their way
// at once, for up to one token per SM (64 tokens of 56 rows 3.8 us, 5.4 in the other
// width; 152 tokens 4.3, 5.9), else so that blocks in different phases share an
// SM (200 tokens 6.2 us, 6.6 wide; 2894 tokens of 48 rows 21 us, 43 wide).
__host__ __device__ constexpr int app_threads(bool wide) { return wide ? 1024 : 256; }
__host__ __device__ constexpr int app_rows(bool wide) { return wide ? 2 : 6; }  // rows that a thread has in flight

template <int D, int kPairs, bool kNorm, bool kWide>
__global__ void __launch_bounds__(app_threads(kWide), kWide ? 1 : 4)
    q4k_append_kernel(const CacheLayer c, const Batch b, const float* Yq,
                      const float* Yk, const float* Yv,
                      uint16_t* q_out, int heads, const float* rope,
                      const float* q_norm, const float* k_norm, float eps) {
    constexpr int kAppThreads = app_threads(kWide), kAppRows = app_rows(kWide);
    constexpr int L = D / 4;                // lanes per row
    constexpr int kStep = kAppThreads / L;  // rows that the block holds at a time
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const int t = blockIdx.x, G = c.kv_heads, rows = heads + 2 * G;
    const int lane = threadIdx.x % L, r = threadIdx.x / L;
    float4 x[kAppRows];
    auto load = [&](int h0) {
#pragma unroll
        for (int e = 0; e < kAppRows; ++e) {
            const int h = h0 + e * kStep;
            if (h >= rows) continue;
            const float* src = h < heads       ? Yq + (static_cast<int64_t>(t) * heads + h) * D
                               : h < heads + G ? Yk + (static_cast<int64_t>(t) * G + h - heads) * D
                                               : Yv + (static_cast<int64_t>(t) * G + h - heads - G) * D;
            x[e] = __ldcs(reinterpret_cast<const float4*>(src) + lane);
        }
    };
    load(r);
    // the sequence: as many of starts[1 ..] as are not above t; of more than the
    // block has threads, every `every`-th first, then those between two of them
    const int every = (b.n + kAppThreads - 1) / kAppThreads, last = min((static_cast<int>(threadIdx.x) + 1) * every, b.n);
    int i = every * __syncthreads_count(static_cast<int>(threadIdx.x) * every < b.n && b.starts[last] <= t);
    if (every > 1) {
        const int j = i + static_cast<int>(threadIdx.x);
        i += __syncthreads_count(static_cast<int>(threadIdx.x) < every && j < b.n && b.starts[j + 1] <= t);
    }
    int64_t pos = -1, off = -1;
    if (i < b.n) {
        const SeqView s = seq_view(c, b, i);
        const int at = t - s.t0;
        if (at >= 0 && at < s.m) pos = static_cast<int64_t>(s.len) - s.m + at;
        if (pos >= 0) {
            const int page = c.table[s.row + (pos >> c.page_shift)];
            if (page >= 0 && page < c.n_pages)
                off = page * c.page_stride + (pos & ((1 << c.page_shift) - 1)) * D;
        }
    }
    // the new element is x * cs + (the pair's other element) * sn
    float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
    if (kPairs != 0 && pos >= 0) {
        const float* row = rope + pos * D;
        if (kPairs == 1) {
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
    const bool turn = kPairs != 0 && pos >= 0;
    float4 wq = make_float4(0.f, 0.f, 0.f, 0.f), wk = wq;
    if (kNorm) {
        if (q_norm != nullptr) wq = *(reinterpret_cast<const float4*>(q_norm) + lane);
        if (k_norm != nullptr) wk = *(reinterpret_cast<const float4*>(k_norm) + lane);
    }
    // whole warps keep together: the shuffles need every lane of a row
    for (int h0 = r; h0 - r < rows; h0 += kAppRows * kStep) {
        if (h0 != r) load(h0);
#pragma unroll
        for (int e = 0; e < kAppRows; ++e) {
            if (h0 - r + e * kStep >= rows) break;
            const int h = h0 + e * kStep;
            const bool in = h < rows, is_q = h < heads, is_v = h >= heads + G;
            float4 y = in ? x[e] : make_float4(0.f, 0.f, 0.f, 0.f);
            if (kNorm) {
                const bool scaled = is_q ? q_norm != nullptr : !is_v && k_norm != nullptr;
                float ss = y.x * y.x + y.y * y.y + y.z * y.z + y.w * y.w;
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (scaled) {
                    const float f = rsqrtf(ss * (1.f / D) + eps);  // (within 2 ulp, before a rounding to 8 bits)
                    const float4 w = is_q ? wq : wk;
                    y = make_float4(y.x * f * w.x, y.y * f * w.y, y.z * f * w.z, y.w * f * w.w);
                }
            }
            if (kPairs != 0) {
                float4 z;  // the other element of each pair
                if (kPairs == 2) {
                    z.x = __shfl_xor_sync(0xffffffffu, y.x, L / 2);
                    z.y = __shfl_xor_sync(0xffffffffu, y.y, L / 2);
                    z.z = __shfl_xor_sync(0xffffffffu, y.z, L / 2);
                    z.w = __shfl_xor_sync(0xffffffffu, y.w, L / 2);
                } else {
                    z = make_float4(y.y, y.x, y.w, y.z);
                }
                if (turn && !is_v)
                    y = make_float4(y.x * cs.x + z.x * sn.x, y.y * cs.y + z.y * sn.y, y.z * cs.z + z.z * sn.z,
                                    y.w * cs.w + z.w * sn.w);
            }
            if (is_q) {
                *(reinterpret_cast<uint2*>(q_out + (static_cast<int64_t>(t) * heads + h) * D) + lane) = bf16x4(y);
            } else if (in && off >= 0 && !(kWide && is_v)) {
                const int g = is_v ? h - heads - G : h - heads;
                uint16_t* dst = (is_v ? c.v : c.k) + off + (static_cast<int64_t>(g) << c.page_shift) * D;
                *(reinterpret_cast<uint2*>(dst) + lane) = bf16x4(y);
            }
        }
        if (kWide) {
            // values after keys: what a cache of one tensor for both holds is then the
            // values (in the other width no order holds between a key and its value)
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kAppRows; ++e) {
                const int h = h0 + e * kStep;
                if (h < heads + G || h >= rows || off < 0) continue;
                uint16_t* dst = c.v + off + (static_cast<int64_t>(h - heads - G) << c.page_shift) * D;
                *(reinterpret_cast<uint2*>(dst) + lane) = bf16x4(x[e]);
            }
        }
    }
}

template <int D, bool kWide>
static cudaError_t launch_d(const CacheLayer& c, const Batch& b, const float* Yq, const float* Yk, const float* Yv,
                            uint16_t* q_out, int heads, const float* rope, int pairs, const float* q_norm,
                            const float* k_norm, float eps, cudaStream_t stream, int pdl) {
    const bool norm = q_norm != nullptr || k_norm != nullptr;
    auto kernel = pairs == 0   ? (norm ? q4k_append_kernel<D, 0, true, kWide> : q4k_append_kernel<D, 0, false, kWide>)
                  : pairs == 1 ? (norm ? q4k_append_kernel<D, 1, true, kWide> : q4k_append_kernel<D, 1, false, kWide>)
                               : (norm ? q4k_append_kernel<D, 2, true, kWide> : q4k_append_kernel<D, 2, false, kWide>);
    return launch_serve(kernel, dim3(b.tokens), dim3(app_threads(kWide)), 0, stream, pdl, 1, c, b, Yq, Yk, Yv, q_out,
                        heads, rope, q_norm, k_norm, eps);
}

cudaError_t launch_append(const CacheLayer& c, const Batch& b, const float* Yq, const float* Yk,
                          const float* Yv, uint16_t* q_out, int heads, int head_dim, const float* rope,
                          int pairs, const float* q_norm, const float* k_norm, float eps,
                          cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    // A cache of one tensor for K and V takes the width that writes the values last.
    // (To leave its keys unwritten instead costs the others: 2894 tokens of 56 rows
    // with norm 28.1 us for 27.6.)
    const bool wide = b.tokens <= dev.num_sms || c.k == c.v;
    auto launch = head_dim == 64 ? (wide ? launch_d<64, true> : launch_d<64, false>)
                                 : (wide ? launch_d<128, true> : launch_d<128, false>);
    return launch(c, b, Yq, Yk, Yv, q_out, heads, rope, pairs, q_norm, k_norm, eps, stream, pdl);
}

}  // namespace q4k
