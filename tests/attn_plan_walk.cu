// attn_plan_walk.cu -- the attention kernels' sharing of a step's work, on its
// own: every block writes out its range and the first items of its walk, and no
// key, value or query is touched. Built and read by tests/test_gpu_attn_plan.py.
#include "q4k_attn.cuh"

using namespace q4k;

constexpr int kKeys = 128;       // positions of a key tile in both kernels
constexpr int kHead = 8;         // words of a block: u, u_end, q, b, h, tile, off, items
constexpr int kItemWords = 10;   // words of an item

template <typename U>
__global__ void plan_walk_kernel(AttnParams p, int tt, AttnCost cost, int most, int64_t* out) {
    extern __shared__ uint64_t units[];
    __shared__ AttnWalk<U> found;
    if (p.b.n > 32) {
        plan_block<kKeys, U>(p, tt, cost, reinterpret_cast<U*>(units), &found);
    } else if (threadIdx.x < 32) {
        const AttnWalk<U> w = plan_warp<kKeys, U>(p, tt, cost);
        if (threadIdx.x == 0) found = w;
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    AttnWalk<U> w = found;
    int64_t* o = out + static_cast<int64_t>(blockIdx.x) * (kHead + most * kItemWords);
    o[0] = w.u;
    o[1] = w.u_end;
    o[2] = w.q;
    o[3] = w.b;
    o[4] = w.h;
    o[5] = w.tile;
    o[6] = w.off;
    AttnItem it;
    int n = 0;
    for (int64_t* x = o + kHead; n < most && next_item<kKeys, U>(p, w, tt, cost, it); ++n, x += kItemWords) {
        x[0] = it.t_first;
        x[1] = it.tokens;
        x[2] = it.p0;
        x[3] = it.h;
        x[4] = it.row;
        x[5] = it.keys.n;
        x[6] = it.i0;
        x[7] = it.i1;
        x[8] = it.first;
        x[9] = it.last;
    }
    o[7] = n;
}

// lens [n_seqs], starts [n + 1] and out [grid][kHead + most * kItemWords] on the
// device; sequences 0 .. n-1. wide: units counted in 64 bits; 2: as the kernels' own
// rule says. The count's bytes are returned, or 0.
extern "C" int plan_walk(const int32_t* lens, const int32_t* starts, int n, int tokens, int width, int kv_heads,
                         int group, int tt, int item, int snap, int q_min, int window, int sinks, int grid, int most,
                         int wide, int64_t* out) {
    AttnParams p = {};
    p.c.lens = lens;
    p.c.n_seqs = n;
    p.c.n_pages = 1;
    p.c.width = width;
    p.c.page_shift = 7;
    p.c.kv_heads = kv_heads;
    p.b.starts = starts;
    p.b.n = n;
    p.b.tokens = tokens;
    p.heads = kv_heads * group;
    p.group = group;
    p.window = window;
    p.sinks = sinks;
    const AttnCost cost{item, snap, q_min};
    if (wide == 2) wide = count_wide(p, tt, kKeys, cost);
    auto kernel = wide ? plan_walk_kernel<uint64_t> : plan_walk_kernel<uint32_t>;
    kernel<<<grid, 128, kMaxBatch * 8>>>(p, tt, cost, most, out);
    if (cudaGetLastError() != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) return 0;
    return wide ? 8 : 4;
}
