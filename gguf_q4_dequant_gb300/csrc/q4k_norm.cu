// q4k_norm.cu -- the residual's addition, the RMS norm, and its rows in fp32 or
// bf16 and in 8 bits (e4m3 codes with one power of two for 32 columns).
//
// A row is read once into registers, eight adjacent columns a thread: the sum of
// squares goes through the row's threads, then every output is written from the
// registers. Nothing is reused, so the memory's rate is the bound, or for a few
// rows the launch and one trip to memory. Four adjacent threads hold the 32
// columns of a scale: its maximum takes two shuffles. 4096 rows of 5120, bf16 and an
// fp32 addition to fp32 and 8 bits: 45 us, 6.1 TB/s (90 % of a copy's rate); one row of
// 4096: 2.8 us.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "q4k_device.cuh"
#include "q4k_experts.h"
#include "q4k_serve.h"

namespace q4k {

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8], bool stream) {
    float4* o = reinterpret_cast<float4*>(p);
    const float4 lo = make_float4(v[0], v[1], v[2], v[3]), hi = make_float4(v[4], v[5], v[6], v[7]);
    if (stream) __stcs(o, lo), __stcs(o + 1, hi);
    else o[0] = lo, o[1] = hi;
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8], bool stream) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    const uint4 o = make_uint4(w[0], w[1], w[2], w[3]);
    if (stream) __stcs(reinterpret_cast<uint4*>(p), o);
    else *reinterpret_cast<uint4*>(p) = o;
}

// Eight of the 32 columns of a scale (the lanes 4i .. 4i+3 hold them): the
// smallest power of two s with max |v| <= 448 s, from the maximum's bits (|v|
// as an integer orders like |v|, with infinities and NaN above the rest), and
// the codes of v / s. 448 = 1.75 * 2^8 is the largest e4m3 value, so no code
// saturates; 2^-127 is the smallest scale. A block with an infinity or a NaN has
// scale byte 255 and NaN codes.
// Every lane of the warp takes part; those with `in` store.
__device__ __forceinline__ void store_eight(const float (&v)[8], uint8_t* codes, uint8_t* scale, bool in, bool first) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const bool finite = m < 0x7F800000u;
    const int e = max(static_cast<int>(m >> 23) - 127 - 8 + ((m & 0x7FFFFFu) > 0x600000u ? 1 : 0), -127);
    const float inv = exp2i(-min(e, 120));  // e <= 120 where m is finite
    uint2 w = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    if (finite) {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        w = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    }
    if (in) {
        *reinterpret_cast<uint2*>(codes) = w;
        if (first) *scale = static_cast<uint8_t>(finite ? e + 127 : 255);
    }
}

// The sum over a row's threads: a warp, or the whole block through `part` (32 floats).
template <bool kWarp>
__device__ __forceinline__ float row_sum(float s, float* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (!kWarp) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) part[threadIdx.x >> 5] = s;
        __syncthreads();
        s = lane < static_cast<int>(blockDim.x >> 5) ? part[lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    }
    return s;
}

// Rows of up to 8 * R columns a thread. kWarp: a warp per row, several rows a
// block (the sum stays in the warp); else a block per row.
template <typename X, typename O, int R, bool kWarp>
__global__ void __launch_bounds__(1024) q4k_add_norm_kernel(const NormArgs a) {
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = kWarp ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
    if (kWarp && row >= a.T) return;
    const int at = kWarp ? lane : threadIdx.x, n = kWarp ? 32 : blockDim.x;
    const int64_t off = row * a.C;
    float v[R][8];
    float ss = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = 8 * (at + r * n);
        if (c < a.C) {
            load8(static_cast<const X*>(a.x) + off + c, v[r]);
            if (a.delta != nullptr) {
                float d[8];
                load8(a.delta + off + c, d);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[r][i] += d[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[r][i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[r][i], v[r][i], ss);
    }
    __shared__ float part[2][32];
    float mean = row_sum<kWarp>(ss, part[0]) / static_cast<float>(a.C);
    if (!(mean < INFINITY)) {  // (the same for the whole row) the sum may pass fp32 where the mean does not
        ss = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(v[r][i] * 0x1p-8f, v[r][i] * 0x1p-8f, ss);
        mean = row_sum<kWarp>(ss, part[1]) / static_cast<float>(a.C) * 0x1p16f;
    }
    mean += a.eps;
    // 1 / sqrt(mean + eps) as the sum of two floats (a Newton step's correction of the rounded
    // root), and r times that as a product with its error, which nothing makes overflow (it is below
    // sqrt(C)) before it meets the weight: y is the exact value but for its last bit, so that codes and
    // scales, which jump at borders, are those of the exact y almost always
    const float rs = 1.f / sqrtf(mean);
    const float t = mean * rs, rest = fmaf(-t, rs, fmaf(-fmaf(mean, rs, -t), rs, 1.f));
    const float rs_lo = mean > 0.f && rs < INFINITY ? 0.5f * rs * rest : 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = 8 * (at + r * n);
        const bool in = c < a.C;  // C is a multiple of 32: the same for the four lanes of a scale
        float w[8] = {};
        if (in) {
            if (a.sum != nullptr) store8(static_cast<X*>(a.sum) + off + c, v[r], a.stream);
            const float4 p = *reinterpret_cast<const float4*>(a.weight + c), q = *(reinterpret_cast<const float4*>(a.weight + c) + 1);
            w[0] = p.x; w[1] = p.y; w[2] = p.z; w[3] = p.w;
            w[4] = q.x; w[5] = q.y; w[6] = q.z; w[7] = q.w;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float u = v[r][i] * rs, off_u = fmaf(v[r][i], rs_lo, fmaf(v[r][i], rs, -u));
                const float y = fmaf(u, w[i], off_u * w[i]);
                w[i] = isfinite(y) ? y : u * w[i];  // (a mean past fp32: rs = 0, its correction NaN)
            }
            if (a.out != nullptr) store8(static_cast<O*>(a.out) + off + c, w, a.stream);
        }
        if (a.codes != nullptr) store_eight(w, a.codes + off + c, a.scales + (off + c) / 32, in, (lane & 3) == 0);
    }
}

// ------------------------------------------------------------------ host ---

namespace {

template <typename X, typename O>
cudaError_t launch_xo(const NormArgs& a, cudaStream_t stream, int pdl) {
    // a warp per row up to 1024 columns; then a block, of one round of eight
    // columns a thread as far as that goes (all of a row on its way at once)
    if (a.C <= 1024) {
        const int rows = 4;
        const dim3 grid(static_cast<unsigned>((a.T + rows - 1) / rows)), block(32 * rows);
        if (a.C <= 256) return launch_serve(q4k_add_norm_kernel<X, O, 1, true>, grid, block, 0, stream, pdl, 1, a);
        if (a.C <= 512) return launch_serve(q4k_add_norm_kernel<X, O, 2, true>, grid, block, 0, stream, pdl, 1, a);
        return launch_serve(q4k_add_norm_kernel<X, O, 4, true>, grid, block, 0, stream, pdl, 1, a);
    }
    const dim3 grid(static_cast<unsigned>(a.T));
    const int rounds = a.C <= 8192 ? 1 : a.C <= 16384 ? 2 : 4;
    const dim3 block((a.C / 8 + 32 * rounds - 1) / (32 * rounds) * 32);
    if (rounds == 1) return launch_serve(q4k_add_norm_kernel<X, O, 1, false>, grid, block, 0, stream, pdl, 1, a);
    if (rounds == 2) return launch_serve(q4k_add_norm_kernel<X, O, 2, false>, grid, block, 0, stream, pdl, 1, a);
    return launch_serve(q4k_add_norm_kernel<X, O, 4, false>, grid, block, 0, stream, pdl, 1, a);
}

}  // namespace

cudaError_t launch_add_norm(const NormArgs& args, cudaStream_t stream, int pdl) {
    NormArgs a = args;
    const int64_t x = a.x_bf16 ? 2 : 4, o = a.out_bf16 ? 2 : 4;
    a.stream = passes_l2(a.T * a.C * ((a.sum != nullptr ? x : 0) + (a.out != nullptr ? o : 0)));
    if (a.x_bf16)
        return a.out_bf16 ? launch_xo<uint16_t, uint16_t>(a, stream, pdl) : launch_xo<uint16_t, float>(a, stream, pdl);
    return a.out_bf16 ? launch_xo<float, uint16_t>(a, stream, pdl) : launch_xo<float, float>(a, stream, pdl);
}

}  // namespace q4k
