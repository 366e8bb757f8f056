// q4k_serve.h -- what the kernels between the products share: the device view
// of a paged cache and of a step's batch, and their host-side launchers. Not
// part of the public interface.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "q4k.h"
#include "q4k_internal.h"

namespace q4k {

constexpr int kMaxBatch = 4096;         // sequences of a step
constexpr int kWsCounterBytes = 16384;  // zeroed words at the front of the workspace
constexpr int kPageTicket = 4095;       // the word that the page calls count in

// One layer's pages (see q4k_cache in q4k.h).
struct CacheLayer {
    uint16_t* k;
    uint16_t* v;
    int64_t page_stride;
    const int32_t* table;
    const int32_t* lens;
    int32_t n_pages, n_seqs, width, page_shift, kv_heads;
};

struct Batch {
    const int32_t* seqs;    // NULL: 0 .. n-1
    const int32_t* starts;  // [n + 1]
    int32_t n, tokens;
};

// A sequence of the batch: its new tokens are rows t0 .. t0+m-1 at positions
// len-m .. len-1, its pages are table[row ..]. Whatever the device arrays hold,
// the rows lie in [0, tokens) and the positions below the table's capacity; a
// sequence id out of range has len = 0.
struct SeqView {
    int t0, m, len;
    int64_t row;
};

#ifdef __CUDACC__
__device__ __forceinline__ SeqView seq_view(const CacheLayer& c, const Batch& b, int i) {
    SeqView s;
    s.t0 = min(max(b.starts[i], 0), b.tokens);
    s.m = min(max(b.starts[i + 1], s.t0), b.tokens) - s.t0;
    const int id = b.seqs != nullptr ? b.seqs[i] : i;
    const bool ok = id >= 0 && id < c.n_seqs;
    s.row = ok ? static_cast<int64_t>(id) * c.width : 0;
    s.len = ok ? min(max(c.lens[id], 0), c.width << c.page_shift) : 0;
    return s;
}
#endif

cudaError_t launch_append(const CacheLayer& c, const Batch& b, const float* Yq, const float* Yk,
                          const float* Yv, uint16_t* q_out, int heads, int head_dim, const float* rope,
                          int pairs, const float* q_norm, const float* k_norm, float eps,
                          cudaStream_t stream, const DeviceInfo& dev, int pdl);

struct AttnArgs {
    const uint16_t* Q;
    uint16_t* out;
    int heads, head_dim;
    float scale;
    int window, sinks;
    uint32_t* counters;  // kWsCounterBytes of zeros, left as zeros
    void* scratch;       // attn_scratch_bytes
};
cudaError_t launch_attention(const CacheLayer& c, const Batch& b, const AttnArgs& a, int max_new,
                             cudaStream_t stream, const DeviceInfo& dev, int pdl);
int64_t attn_scratch_bytes(const DeviceInfo& dev, int head_dim);
cudaError_t attn_setup(DeviceInfo& dev);

cudaError_t launch_pages_reserve(const q4k_cache& c, const int32_t* seqs, int n, const int32_t* starts,
                                 int32_t* status, cudaStream_t stream, int pdl);
cudaError_t launch_pages_fork(const q4k_cache& c, const int32_t* parents, const int32_t* children, int n,
                              int32_t* status, uint32_t* counters, cudaStream_t stream,
                              const DeviceInfo& dev, int pdl);
cudaError_t launch_pages_free(const q4k_cache& c, const int32_t* seqs, int n, cudaStream_t stream, int pdl);
cudaError_t launch_pages_copy(const q4k_cache& c, const int32_t* src, const int32_t* dst, int64_t n,
                              cudaStream_t stream, const DeviceInfo& dev, int pdl);
cudaError_t launch_pages_compact(const q4k_cache& c, void* scratch, cudaStream_t stream,
                                 const DeviceInfo& dev, int pdl);
int64_t pages_scratch_bytes(int64_t n_pages);
cudaError_t pages_setup();

struct PickArgs {
    const float* logits;
    float* out;
    int64_t* pick;
    const int32_t *history, *hist_starts;
    const float* penalties;
    const int32_t* bias_ids;
    const float* bias;
    const int32_t* bias_starts;
    const uint32_t* mask;
    int64_t M, V;
};
cudaError_t pick_setup(DeviceInfo& dev);  // fills dev.pick_clusters
cudaError_t launch_pick(const PickArgs& a, cudaStream_t stream, const DeviceInfo& dev, int pdl);

// Launch with programmatic stream serialisation when the PDL mode asks for it
// (every kernel launched this way begins with pdl_wait()), and with a cluster
// of `cluster` CTAs along x when that is above 1. A kernel's arrays are not
// declared __restrict__: the kernel before may write them after this one has
// begun, so they may not be read as data that is constant while it runs.
template <typename... P, typename... A>
cudaError_t launch_serve(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                         int pdl, int cluster, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (pdl) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = cluster;
        attr[na].val.clusterDim.y = 1;
        attr[na++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = na;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace q4k
