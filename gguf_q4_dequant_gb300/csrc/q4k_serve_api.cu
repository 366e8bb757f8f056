// q4k_serve_api.cu -- the C ABI of the calls between the products: argument
// checks on the host, then one launcher each.
#include <cuda_runtime.h>

#include <cmath>

#include "q4k.h"
#include "q4k_internal.h"
#include "q4k_serve.h"

namespace q4k {
namespace {

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

int page_shift(int page_size) {
    switch (page_size) {
        case 16: return 4;
        case 32: return 5;
        case 64: return 6;
        case 128: return 7;
    }
    return -1;
}

int check_cache(const q4k_cache* c) {
    if (!c || !c->k || !c->v || !c->refs || !c->table || !c->lens) return Q4K_ERR_NULL;
    if (page_shift(c->page_size) < 0 || (c->head_dim != 64 && c->head_dim != 128)) return Q4K_ERR_BAD_DIM;
    if (c->n_pages < 1 || c->n_pages > (int64_t(1) << 30) || c->layers < 1 || c->layers > 65535 ||
        c->kv_heads < 1 || c->kv_heads > 1024 || c->n_seqs < 1 || c->n_seqs > (1 << 24) || c->width < 1 ||
        static_cast<int64_t>(c->width) * c->page_size > (int64_t(1) << 30))
        return Q4K_ERR_BAD_DIM;
    const int64_t page = static_cast<int64_t>(c->kv_heads) * c->page_size * c->head_dim;
    // strides below 2^39 elements (the tensor map's limit), so that the products below fit
    const int64_t lim = int64_t(1) << 39;
    if (c->page_stride < page || c->layer_stride < page || c->page_stride >= lim || c->layer_stride >= lim ||
        c->page_stride % 8 != 0 || c->layer_stride % 8 != 0)
        return Q4K_ERR_BAD_DIM;
    // either the layers follow one another, each with all its pages, or every
    // page holds all its layers
    const bool layers_apart = c->layers == 1 || c->layer_stride / c->page_stride >= c->n_pages ||
                              c->layer_stride >= (c->n_pages - 1) * static_cast<double>(c->page_stride) + page;
    const bool pages_apart = c->n_pages == 1 || c->page_stride >= (c->layers - 1) * static_cast<double>(c->layer_stride) + page;
    if (!layers_apart && !pages_apart) return Q4K_ERR_BAD_DIM;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->refs, 4) || !aligned(c->table, 4) ||
        !aligned(c->lens, 4))
        return Q4K_ERR_ALIGN;
    return Q4K_OK;
}

int64_t workspace_bytes(const q4k_cache& c, const DeviceInfo& dev) {
    const int64_t a = attn_scratch_bytes(dev, c.head_dim), p = pages_scratch_bytes(c.n_pages);
    return kWsCounterBytes + (a > p ? a : p);
}

int check_workspace(const q4k_cache& c, const void* ws, int64_t bytes, const DeviceInfo& dev) {
    return bytes < workspace_bytes(c, dev) ? Q4K_ERR_SPACE : Q4K_OK;
}

uint32_t* ws_counters(void* ws) { return static_cast<uint32_t*>(ws); }
void* ws_scratch(void* ws) { return static_cast<uint8_t*>(ws) + kWsCounterBytes; }

CacheLayer layer_view(const q4k_cache& c, int layer) {
    CacheLayer l;
    l.k = c.k + layer * c.layer_stride;
    l.v = c.v + layer * c.layer_stride;
    l.page_stride = c.page_stride;
    l.table = c.table;
    l.lens = c.lens;
    l.n_pages = static_cast<int32_t>(c.n_pages);
    l.n_seqs = c.n_seqs;
    l.width = c.width;
    l.page_shift = page_shift(c.page_size);
    l.kv_heads = c.kv_heads;
    return l;
}

// The parts of a step that append and attention share.
int check_step(const q4k_cache* c, int layer, const int32_t* seqs, int n, const int32_t* starts,
               int64_t tokens, int heads) {
    const int rc = check_cache(c);
    if (rc != Q4K_OK) return rc;
    if (!starts) return Q4K_ERR_NULL;
    if (layer < 0 || layer >= c->layers || n < 1 || n > kMaxBatch || heads < c->kv_heads ||
        heads % c->kv_heads != 0 || heads > 65535 || tokens < 1 || tokens >= (int64_t(1) << 31) / heads)
        return Q4K_ERR_BAD_DIM;
    if (seqs == nullptr && n > c->n_seqs) return Q4K_ERR_BAD_DIM;
    if (!aligned(starts, 4) || !aligned(seqs, 4)) return Q4K_ERR_ALIGN;
    return Q4K_OK;
}

}  // namespace
}  // namespace q4k

using namespace q4k;

extern "C" {

int64_t q4k_cache_workspace(const q4k_cache* c) {
    int rc = check_cache(c);
    if (rc != Q4K_OK) return rc;
    const DeviceInfo* dev = nullptr;
    if ((rc = device_info(&dev)) != Q4K_OK) return rc;
    return workspace_bytes(*c, *dev);
}

int q4k_cache_append(const q4k_cache* c, int layer, const int32_t* seqs, int n, const int32_t* starts,
                     int64_t tokens, const float* Yq, const float* Yk, const float* Yv,
                     uint16_t* q_out, int heads, const float* rope, int64_t rope_rows, int pairs,
                     const float* q_norm, const float* k_norm, float eps, void* stream) {
    int rc = check_step(c, layer, seqs, n, starts, tokens, heads);
    if (rc != Q4K_OK) return rc;
    if (!Yq || !Yk || !Yv || !q_out) return Q4K_ERR_NULL;
    if (pairs < 0 || pairs > 2) return Q4K_ERR_BAD_DIM;
    if (pairs != 0) {
        if (!rope) return Q4K_ERR_NULL;
        if (rope_rows < static_cast<int64_t>(c->width) * c->page_size) return Q4K_ERR_BAD_DIM;
    }
    if ((q_norm || k_norm) && !(eps >= 0.f && std::isfinite(eps))) return Q4K_ERR_BAD_DIM;
    if (!aligned(Yq, 16) || !aligned(Yk, 16) || !aligned(Yv, 16) || !aligned(q_out, 16) ||
        !aligned(rope, 16) || !aligned(q_norm, 16) || !aligned(k_norm, 16))
        return Q4K_ERR_ALIGN;
    const DeviceInfo* dev = nullptr;
    if ((rc = device_info(&dev)) != Q4K_OK) return rc;
    const Batch b{seqs, starts, n, static_cast<int32_t>(tokens)};
    return launch_append(layer_view(*c, layer), b, Yq, Yk, Yv, q_out, heads, c->head_dim, rope, pairs,
                         q_norm, k_norm, eps, static_cast<cudaStream_t>(stream), *dev, pdl_mode()) == cudaSuccess
               ? Q4K_OK
               : Q4K_ERR_CUDA;
}

int q4k_cache_attention(const q4k_cache* c, int layer, const int32_t* seqs, int n,
                        const int32_t* starts, int64_t tokens, const uint16_t* Q, uint16_t* out,
                        int heads, int max_new, float scale, int window, int sinks, void* ws,
                        int64_t ws_bytes, void* stream) {
    int rc = check_step(c, layer, seqs, n, starts, tokens, heads);
    if (rc != Q4K_OK) return rc;
    if (!Q || !out || !ws) return Q4K_ERR_NULL;
    if (heads / c->kv_heads > 128 || max_new < 0 || window < 0 || sinks < 0 || !(scale > 0.f) ||
        !std::isfinite(scale))
        return Q4K_ERR_BAD_DIM;
    if (!aligned(Q, 16) || !aligned(out, 16) || !aligned(ws, 256)) return Q4K_ERR_ALIGN;
    const DeviceInfo* dev = nullptr;
    if ((rc = device_info(&dev)) != Q4K_OK) return rc;
    if ((rc = check_workspace(*c, ws, ws_bytes, *dev)) != Q4K_OK) return rc;
    const Batch b{seqs, starts, n, static_cast<int32_t>(tokens)};
    AttnArgs a;
    a.Q = Q;
    a.out = out;
    a.heads = heads;
    a.head_dim = c->head_dim;
    a.scale = scale;
    a.window = window;
    a.sinks = sinks;
    a.counters = ws_counters(ws);
    a.scratch = ws_scratch(ws);
    return launch_attention(layer_view(*c, layer), b, a, max_new, static_cast<cudaStream_t>(stream), *dev,
                            pdl_mode()) == cudaSuccess
               ? Q4K_OK
               : Q4K_ERR_CUDA;
}

int q4k_pages_reserve(const q4k_cache* c, const int32_t* seqs, int n, const int32_t* starts,
                      int32_t* status, void* stream) {
    int rc = check_cache(c);
    if (rc != Q4K_OK) return rc;
    if (!starts || !status) return Q4K_ERR_NULL;
    if (n < 1 || n > kMaxBatch || (seqs == nullptr && n > c->n_seqs)) return Q4K_ERR_BAD_DIM;
    if (!aligned(starts, 4) || !aligned(seqs, 4) || !aligned(status, 4)) return Q4K_ERR_ALIGN;
    const DeviceInfo* dev = nullptr;
    if ((rc = device_info(&dev)) != Q4K_OK) return rc;
    return launch_pages_reserve(*c, seqs, n, starts, status, static_cast<cudaStream_t>(stream), pdl_mode()) ==
                   cudaSuccess
               ? Q4K_OK
               : Q4K_ERR_CUDA;
}

int q4k_pages_fork(const q4k_cache* c, const int32_t* parents, const int32_t* children, int n,
                   int32_t* status, void* ws, int64_t ws_bytes, void* stream) {
    int rc = check_cache(c);
    if (rc != Q4K_OK) return rc;
    if (!parents || !children || !status || !ws) return Q4K_ERR_NULL;
    if (n < 1 || n > kMaxBatch) return Q4K_ERR_BAD_DIM;
    if (!aligned(parents, 4) || !aligned(children, 4) || !aligned(status, 4) || !aligned(ws, 256))
        return Q4K_ERR_ALIGN;
    const DeviceInfo* dev = nullptr;
    if ((rc = device_info(&dev)) != Q4K_OK) return rc;
    if ((rc = check_workspace(*c, ws, ws_bytes, *dev)) != Q4K_OK) return rc;
    return launch_pages_fork(*c, parents, children, n, status, ws_counters(ws),
                             static_cast<cudaStream_t>(stream), *dev, pdl_mode()) == cudaSuccess
               ? Q4K_OK
               : Q4K_ERR_CUDA;
}

int q4k_pages_free(const q4k_cache* c, const int32_t* seqs, int n, void* stream) {
    int rc = check_cache(c);
    if (rc != Q4K_OK) return rc;
    if (!seqs) return Q4K_ERR_NULL;
    if (n < 1 || n > (1 << 24)) return Q4K_ERR_BAD_DIM;
    if (!aligned(seqs, 4)) return Q4K_ERR_ALIGN;
    const DeviceInfo* dev = nullptr;
    if ((rc = device_info(&dev)) != Q4K_OK) return rc;
    return launch_pages_free(*c, seqs, n, static_cast<cudaStream_t>(stream), pdl_mode()) == cudaSuccess
               ? Q4K_OK
               : Q4K_ERR_CUDA;
}

int q4k_pages_copy(const q4k_cache* c, const int32_t* src, const int32_t* dst, int64_t n, void* stream) {
    int rc = check_cache(c);
    if (rc != Q4K_OK) return rc;
    if (!src || !dst) return Q4K_ERR_NULL;
    if (n < 1 || n > (int64_t(1) << 31) - 1) return Q4K_ERR_BAD_DIM;
    if (!aligned(src, 4) || !aligned(dst, 4)) return Q4K_ERR_ALIGN;
    const DeviceInfo* dev = nullptr;
    if ((rc = device_info(&dev)) != Q4K_OK) return rc;
    return launch_pages_copy(*c, src, dst, n, static_cast<cudaStream_t>(stream), *dev, pdl_mode()) == cudaSuccess
               ? Q4K_OK
               : Q4K_ERR_CUDA;
}

int q4k_pages_compact(const q4k_cache* c, void* ws, int64_t ws_bytes, void* stream) {
    int rc = check_cache(c);
    if (rc != Q4K_OK) return rc;
    if (!ws) return Q4K_ERR_NULL;
    if (!aligned(ws, 256)) return Q4K_ERR_ALIGN;
    const DeviceInfo* dev = nullptr;
    if ((rc = device_info(&dev)) != Q4K_OK) return rc;
    if ((rc = check_workspace(*c, ws, ws_bytes, *dev)) != Q4K_OK) return rc;
    return launch_pages_compact(*c, ws_scratch(ws), static_cast<cudaStream_t>(stream), *dev, pdl_mode()) ==
                   cudaSuccess
               ? Q4K_OK
               : Q4K_ERR_CUDA;
}

int q4k_logits_pick(const float* logits, int64_t M, int64_t V, float* out, int64_t* pick,
                    const int32_t* history, const int32_t* hist_starts, const float* penalties,
                    const int32_t* bias_ids, const float* bias, const int32_t* bias_starts,
                    const uint32_t* mask, void* stream) {
    if (!logits || (!out && !pick)) return Q4K_ERR_NULL;
    if (history && (!hist_starts || !penalties)) return Q4K_ERR_NULL;
    if (bias_ids && (!bias || !bias_starts)) return Q4K_ERR_NULL;
    if (M < 1 || M > 65535 || V < 1 || V > (int64_t(1) << 31) - 1) return Q4K_ERR_BAD_DIM;
    if (!aligned(logits, 16) || !aligned(out, 16) || !aligned(pick, 8) || !aligned(history, 4) ||
        !aligned(hist_starts, 4) || !aligned(penalties, 4) || !aligned(bias_ids, 4) || !aligned(bias, 4) ||
        !aligned(bias_starts, 4) || !aligned(mask, 4))
        return Q4K_ERR_ALIGN;
    const DeviceInfo* dev = nullptr;
    int rc = device_info(&dev);
    if (rc != Q4K_OK) return rc;
    PickArgs a{logits, out, pick, history, hist_starts, penalties, bias_ids, bias, bias_starts, mask, M, V};
    return launch_pick(a, static_cast<cudaStream_t>(stream), *dev, pdl_mode()) == cudaSuccess ? Q4K_OK
                                                                                              : Q4K_ERR_CUDA;
}

}  // extern "C"
