// q4k_experts_api.cu -- the C ABI of the expert layer's calls: argument checks on
// the host, then one launcher each.
#include <cuda_runtime.h>

#include <cmath>

#include "q4k.h"
#include "q4k_experts.h"
#include "q4k_internal.h"

namespace q4k {
namespace {

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool in_type(int t) { return t == Q4K_F32 || t == Q4K_BF16; }

constexpr int64_t kMaxCols = 32768;
constexpr int64_t kInt = int64_t(1) << 31;

bool bad_pairs(int64_t T, int k) { return k < 1 || k > kMaxTop || T < 1 || T >= (kInt + k - 1) / k; }

int status(cudaError_t e) { return e == cudaSuccess ? Q4K_OK : Q4K_ERR_CUDA; }

int run_experts(const void* W, const void* W2, bool gated, int64_t E, int64_t N, int64_t K, const uint16_t* X,
                const int32_t* starts, int64_t pairs, uint16_t* Y, void* stream) {
    if (!W || (gated && !W2) || !X || !starts || !Y) return Q4K_ERR_NULL;
    if (E < 1 || E > kMaxExperts || N < 1 || N >= kInt || E * N >= kInt || K < 256 || K % 256 != 0 ||
        K > (int64_t(1) << 24) || pairs < 1 || pairs >= kInt)
        return Q4K_ERR_BAD_DIM;
    if (!aligned(W, 16) || !aligned(W2, 16) || !aligned(X, 16) || !aligned(Y, 16) || !aligned(starts, 4))
        return Q4K_ERR_ALIGN;
    const DeviceInfo* dev = nullptr;
    const int rc = device_info(&dev);
    if (rc != Q4K_OK) return rc;
    ExpertArgs a;
    a.W = static_cast<const uint8_t*>(W);
    a.W2 = static_cast<const uint8_t*>(W2);
    a.N = N;
    a.K = K;
    a.X = X;
    a.rows = ExpertRows{starts, static_cast<int>(E), static_cast<int>(pairs)};
    a.Y = Y;
    return status(launch_experts(a, static_cast<cudaStream_t>(stream), *dev, pdl_mode()));
}

}  // namespace
}  // namespace q4k

using namespace q4k;

extern "C" {

int q4k_add_norm(const void* x, int x_type, const float* delta, const float* weight, float eps, int64_t T, int64_t C,
                 void* sum, void* out, int out_type, uint8_t* codes, uint8_t* scales, void* stream) {
    if (!x || !weight || (!out && !codes) || (codes == nullptr) != (scales == nullptr)) return Q4K_ERR_NULL;
    if (!in_type(x_type) || (out && !in_type(out_type)) || T < 1 || T >= kInt || C < 32 || C % 32 != 0 || C > kMaxCols ||
        !(eps >= 0.f) || !std::isfinite(eps))
        return Q4K_ERR_BAD_DIM;
    if (!aligned(x, 16) || !aligned(delta, 16) || !aligned(weight, 16) || !aligned(sum, 16) || !aligned(out, 16) ||
        !aligned(codes, 8))
        return Q4K_ERR_ALIGN;
    const DeviceInfo* dev = nullptr;
    const int rc = device_info(&dev);
    if (rc != Q4K_OK) return rc;
    const NormArgs a{x,    delta, weight,               sum, out,
                     codes, scales, T, static_cast<int>(C), eps, x_type == Q4K_BF16, out && out_type == Q4K_BF16};
    return status(launch_add_norm(a, static_cast<cudaStream_t>(stream), pdl_mode()));
}

int64_t q4k_route_workspace(int64_t T, int64_t E) {
    if (T < 1 || T >= kInt || E < 1 || E > kMaxExperts) return Q4K_ERR_BAD_DIM;
    return route_scratch_bytes(T, static_cast<int>(E));
}

int q4k_route(const float* logits, int64_t T, int64_t E, int k, int weighting, float scale, int32_t* ids, float* weights,
              int32_t* order, int32_t* slots, int32_t* starts, void* ws, int64_t ws_bytes, void* stream) {
    if (!logits || !ids || !weights || !order || !slots || !starts || !ws) return Q4K_ERR_NULL;
    if (bad_pairs(T, k) || E < k || E > kMaxExperts || weighting < Q4K_ROUTE_SOFTMAX ||
        weighting > Q4K_ROUTE_SIGMOID_TOP || !std::isfinite(scale))
        return Q4K_ERR_BAD_DIM;
    if (!aligned(logits, 4) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(order, 4) || !aligned(slots, 4) ||
        !aligned(starts, 4) || !aligned(ws, 4))
        return Q4K_ERR_ALIGN;
    if (ws_bytes < route_scratch_bytes(T, static_cast<int>(E))) return Q4K_ERR_SPACE;
    const DeviceInfo* dev = nullptr;
    const int rc = device_info(&dev);
    if (rc != Q4K_OK) return rc;
    const RouteArgs a{logits,  static_cast<int>(T), static_cast<int>(E), k, weighting, scale, ids, weights, order, slots,
                      starts, static_cast<int32_t*>(ws)};
    return status(launch_route(a, static_cast<cudaStream_t>(stream), *dev, pdl_mode()));
}

int q4k_experts_gather(const void* X, const uint8_t* scales, const int32_t* order, int64_t T, int k, int64_t C,
                       uint16_t* out, void* stream) {
    if (!X || !order || !out) return Q4K_ERR_NULL;
    if (bad_pairs(T, k) || C < 8 || C % (scales ? 32 : 8) != 0 || C > kMaxCols) return Q4K_ERR_BAD_DIM;
    if (!aligned(X, scales ? 8 : 16) || !aligned(order, 4) || !aligned(out, 16)) return Q4K_ERR_ALIGN;
    const DeviceInfo* dev = nullptr;
    const int rc = device_info(&dev);
    if (rc != Q4K_OK) return rc;
    const GatherArgs a{X, scales, order, out, static_cast<int>(T), static_cast<int>(C), k, static_cast<int>(T * k)};
    return status(launch_gather(a, static_cast<cudaStream_t>(stream), *dev, pdl_mode()));
}

int q4k_experts_matmul(const void* W, int64_t E, int64_t N, int64_t K, const uint16_t* X, const int32_t* starts,
                       int64_t pairs, uint16_t* Y, void* stream) {
    return run_experts(W, nullptr, false, E, N, K, X, starts, pairs, Y, stream);
}

int q4k_experts_gated(const void* gate, const void* up, int64_t E, int64_t N, int64_t K, const uint16_t* X,
                      const int32_t* starts, int64_t pairs, uint16_t* Y, void* stream) {
    return run_experts(gate, up, true, E, N, K, X, starts, pairs, Y, stream);
}

int q4k_experts_combine(const uint16_t* Y, int64_t pairs, const int32_t* slots, const float* weights, const float* base,
                        int64_t T, int k, int64_t C, float* out, void* stream) {
    if (!Y || !slots || !weights || !out) return Q4K_ERR_NULL;
    if (bad_pairs(T, k) || pairs < 1 || pairs >= kInt || C < 8 || C % 8 != 0 || C > kMaxCols) return Q4K_ERR_BAD_DIM;
    if (!aligned(Y, 16) || !aligned(slots, 4) || !aligned(weights, 4) || !aligned(base, 16) || !aligned(out, 16))
        return Q4K_ERR_ALIGN;
    const DeviceInfo* dev = nullptr;
    const int rc = device_info(&dev);
    if (rc != Q4K_OK) return rc;
    const CombineArgs a{Y, slots, weights, base, out, T, static_cast<int>(C), k, static_cast<int>(pairs)};
    return status(launch_combine(a, static_cast<cudaStream_t>(stream), pdl_mode()));
}

}  // extern "C"
