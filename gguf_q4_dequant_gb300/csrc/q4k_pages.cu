// q4k_pages.cu -- the pages of a cache: handing out, sharing, giving back,
// copying and moving together. All state lives on the device, so a step's
// bookkeeping needs no host round trip and can be captured.
//
// Free pages are always taken lowest id first, by ranking the free entries of
// refs (ballots and a block scan): the outcome is a function of the state
// alone. What takes time is the copying of page contents in every layer, bound
// by the memory's rate (a compaction that moves 512 MB: 6.5 TB/s of reads and
// writes in the copying kernel, 167 us with the plan before it); the bookkeeping
// is a few microseconds of latency (16 beams freed and forked anew in 28 layers,
// 29 MB of copies: 10.8 us, of which the copies need 4.3).
#include "q4k_device.cuh"
#include "q4k_serve.h"

namespace q4k {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;  // 16-byte vectors that a thread has in flight

// Rank of each thread's flag among the block's set flags (exclusive), and
// their number. Every thread of the block calls it; `warp_sums` holds 32 words.
template <int kThreads>
__device__ __forceinline__ int block_rank(bool flag, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t votes = __ballot_sync(0xffffffffu, flag);
    if (lane == 0) warp_sums[warp] = __popc(votes);
    __syncthreads();
    const int mine = lane < kThreads / 32 ? warp_sums[lane] : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
    const int before = __shfl_sync(0xffffffffu, incl - mine, warp);
    __syncthreads();  // warp_sums may be written again
    return before + __popc(votes & ((1u << lane) - 1));
}

struct PageGeom {
    uint4 *k, *v;
    int64_t layer_stride, page_stride;  // in 16-byte vectors
    int32_t layers, page_vecs;
};

PageGeom geom(const q4k_cache& c) {
    PageGeom g;
    g.k = reinterpret_cast<uint4*>(c.k);
    g.v = reinterpret_cast<uint4*>(c.v);
    g.layer_stride = c.layer_stride / 8;
    g.page_stride = c.page_stride / 8;
    g.layers = c.layers;
    g.page_vecs = c.kv_heads * c.page_size * (c.head_dim / 8);
    return g;
}

// One block copies part `part` (kCopyThreads * kCopyVecs vectors) of one page
// of one layer, K (kv = 0) or V (kv = 1).
__device__ __forceinline__ void copy_part(const PageGeom& g, int64_t src, int64_t dst, int layer, int kv, int part) {
    uint4* base = (kv ? g.v : g.k) + layer * g.layer_stride;
    const uint4* s = base + src * g.page_stride;
    uint4* d = base + dst * g.page_stride;
    const int o = part * (kCopyThreads * kCopyVecs) + threadIdx.x;
    uint4 x[kCopyVecs];
#pragma unroll
    for (int e = 0; e < kCopyVecs; ++e)
        if (o + e * kCopyThreads < g.page_vecs) x[e] = __ldcs(s + o + e * kCopyThreads);
#pragma unroll
    for (int e = 0; e < kCopyVecs; ++e)
        if (o + e * kCopyThreads < g.page_vecs) __stcs(d + o + e * kCopyThreads, x[e]);
}

int parts_per_page(const PageGeom& g) { return (g.page_vecs + kCopyThreads * kCopyVecs - 1) / (kCopyThreads * kCopyVecs); }

}  // namespace

// Copies n pairs of pages in every layer (n from the device if n_dev is given);
// blocks take parts of (pair, layer, K or V) in turn.
__global__ void __launch_bounds__(kCopyThreads)
    q4k_pages_copy_kernel(const PageGeom g, const int32_t* src, const int32_t* dst,
                          int64_t n, int64_t n_pages, int parts) {
    pdl_wait();
    const int64_t per_pair = static_cast<int64_t>(g.layers) * 2 * parts, total = n * per_pair;
    for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
        const int64_t i = w / per_pair;
        const int r = static_cast<int>(w - i * per_pair);
        const int from = src[i], to = dst[i];
        if (from < 0 || to < 0 || from >= n_pages || to >= n_pages) continue;
        copy_part(g, from, to, r / (2 * parts), (r / parts) & 1, r % parts);
    }
}

__global__ void __launch_bounds__(256)
    q4k_pages_free_kernel(const int32_t* seqs, int n_seqs, int width, int64_t n_pages,
                          int32_t* refs, int32_t* table, int32_t* lens) {
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const int id = seqs[blockIdx.x];
    if (id < 0 || id >= n_seqs) return;
    int32_t* row = table + static_cast<int64_t>(id) * width;
    for (int j = threadIdx.x; j < width; j += blockDim.x) {
        const int page = row[j];
        if (page >= 0 && page < n_pages) atomicSub(refs + page, 1);
        row[j] = -1;
    }
    if (threadIdx.x == 0) lens[id] = 0;
}

// One block: needs of the sequences, their running total, then the free pages
// in ascending order to the sequences in order.
__global__ void __launch_bounds__(kPlanThreads)
    q4k_pages_reserve_kernel(const int32_t* seqs, int n, const int32_t* starts,
                             int32_t* status, int n_seqs, int width, int page_size,
                             int64_t n_pages, int32_t* refs, int32_t* table, int32_t* lens) {
    __shared__ int64_t upto[kMaxBatch + 1];  // pages that the sequences before i need
    __shared__ int warp_sums[32];
    __shared__ int64_t warp_tot[32];
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t cap = static_cast<int64_t>(width) * page_size;
    auto old_len = [&](int id) { return min(max(static_cast<int64_t>(lens[id]), int64_t(0)), cap); };
    auto seq_of = [&](int i) { return seqs != nullptr ? seqs[i] : i; };
    auto grows = [&](int i) { return max(static_cast<int64_t>(starts[i + 1]) - starts[i], int64_t(0)); };
    constexpr int kPer = kMaxBatch / kPlanThreads;
    int64_t need[kPer], sum = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int i = threadIdx.x * kPer + e;
        need[e] = 0;
        if (i < n) {
            const int id = seq_of(i);
            if (id >= 0 && id < n_seqs) {
                const int64_t len = old_len(id), want = len + grows(i);
                if (want <= cap) need[e] = (want + page_size - 1) / page_size - (len + page_size - 1) / page_size;
            }
        }
        sum += need[e];
    }
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    int64_t at = incl - sum;
    for (int w = 0; w < warp; ++w) at += warp_tot[w];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        upto[threadIdx.x * kPer + e] = at;
        at += need[e];
    }
    if (threadIdx.x == kPlanThreads - 1) upto[kMaxBatch] = at;
    __syncthreads();
    const int64_t all = upto[n];
    int64_t free_pages = 0;
    for (int64_t p0 = 0; p0 < n_pages && free_pages < all; p0 += kPlanThreads)
        free_pages += __syncthreads_count(p0 + threadIdx.x < n_pages && refs[p0 + threadIdx.x] == 0);
    // the needs that fit: sequences whose running total does not pass the free pages
    int64_t given = 0;
    for (int64_t p0 = 0; p0 < n_pages && given < all; p0 += kPlanThreads) {
        const int64_t p = p0 + threadIdx.x;
        const bool is_free = p < n_pages && refs[p] == 0;
        int here;
        const int64_t r = given + block_rank<kPlanThreads>(is_free, warp_sums, here);
        if (is_free && r < all) {
            int lo = 0, hi = n;  // the sequence with upto[lo] <= r < upto[lo + 1]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (upto[mid] <= r) lo = mid; else hi = mid;
            }
            if (upto[lo + 1] <= free_pages) {
                const int id = seq_of(lo);
                const int64_t col = (old_len(id) + page_size - 1) / page_size + (r - upto[lo]);
                table[static_cast<int64_t>(id) * width + col] = static_cast<int32_t>(p);
                refs[p] = 1;
            }
        }
        given += here;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int id = seq_of(i);
        int bad = 1;
        if (id >= 0 && id < n_seqs) {
            const int64_t want = old_len(id) + grows(i);
            if (want <= cap && (upto[i + 1] == upto[i] || upto[i + 1] <= free_pages)) {
                lens[id] = static_cast<int32_t>(want);
                bad = 0;
            }
        }
        status[i] = bad;
    }
}

// Forks. Every block works out the whole plan for itself from the state (a few
// loads; the plan lies in shared memory, three words per fork) and counts itself
// in. The block that counts in last, when no block reads any more what it
// changes, writes the new tables, lengths, references and the statuses; all copy
// their share of the pages. (Parents' lengths and tables do not change.)
__global__ void __launch_bounds__(kCopyThreads)
    q4k_pages_fork_kernel(const PageGeom g, const int32_t* parents,
                          const int32_t* children, int n, int32_t* status, int n_seqs,
                          int width, int page_size, int64_t n_pages, int32_t* refs, int32_t* table,
                          int32_t* lens, int parts, uint32_t* ticket) {
    extern __shared__ int32_t plan_s[];
    int32_t* rank_s = plan_s;        // copies before i, or ~that where i may not fork
    int32_t* src_s = plan_s + n;     // the parent's last page if it is copied, else -1
    int32_t* fresh = plan_s + 2 * n; // the lowest free pages
    __shared__ int warp_sums[32];
    __shared__ bool last;
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const int64_t cap = static_cast<int64_t>(width) * page_size;
    auto length = [&](int id) { return static_cast<int>(min(max(static_cast<int64_t>(lens[id]), int64_t(0)), cap)); };
    int copies = 0;
    for (int i0 = 0; i0 < n; i0 += kCopyThreads) {
        const int i = i0 + threadIdx.x;
        bool may = false;
        int src = -1;
        if (i < n) {
            const int p = parents[i], ch = children[i];
            if (p >= 0 && p < n_seqs && ch >= 0 && ch < n_seqs && lens[ch] == 0) {
                const int len = length(p);
                may = true;
                if (len % page_size != 0) {
                    src = table[static_cast<int64_t>(p) * width + len / page_size];
                    if (src >= n_pages) src = -1;
                    may = src >= 0;
                }
            }
        }
        int here;
        const int r = copies + block_rank<kCopyThreads>(src >= 0, warp_sums, here);
        if (i < n) {
            rank_s[i] = may ? r : ~r;
            src_s[i] = src;
        }
        copies += here;
    }
    int found = 0;
    for (int64_t p0 = 0; p0 < n_pages && found < copies; p0 += kCopyThreads) {
        const int64_t p = p0 + threadIdx.x;
        const bool is_free = p < n_pages && refs[p] == 0;
        int here;
        const int r = found + block_rank<kCopyThreads>(is_free, warp_sums, here);
        if (is_free && r < copies) fresh[r] = static_cast<int32_t>(p);
        found += here;
    }
    found = min(found, copies);
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(ticket, 1u) == gridDim.x - 1;
        if (last) *ticket = 0u;
    }
    // this block's share of the copies: (child, layer, K or V, part)
    const int per_child = g.layers * 2 * parts;
    const int64_t total = static_cast<int64_t>(n) * per_child;
    for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
        const int i = total <= 0x7FFFFFFF ? static_cast<int>(w) / per_child : static_cast<int>(w / per_child);
        const int r = rank_s[i];
        if (src_s[i] < 0 || r < 0 || r >= found) continue;
        const int u = static_cast<int>(w - static_cast<int64_t>(i) * per_child);
        copy_part(g, src_s[i], fresh[r], u / (2 * parts), (u / parts) & 1, u % parts);
    }
    __syncthreads();
    if (!last) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = warp; i < n; i += kCopyThreads / 32) {
        const int r = rank_s[i];
        bool ok = r >= 0;
        if (ok) {
            const int p = parents[i], ch = children[i], len = length(p);
            const int full = len / page_size;
            const bool part = src_s[i] >= 0;
            ok = !part || r < found;
            if (ok) {
                const int32_t* from = table + static_cast<int64_t>(p) * width;
                int32_t* to = table + static_cast<int64_t>(ch) * width;
                for (int j = lane; j < width; j += 32) {
                    int page = -1;
                    if (j < full) {
                        page = from[j];
                        if (page >= 0 && page < n_pages) atomicAdd(refs + page, 1);
                    } else if (j == full && part) {
                        page = fresh[r];
                        refs[page] = 1;
                    }
                    to[j] = page;
                }
                if (lane == 0) lens[ch] = len;
            }
        }
        if (lane == 0) status[i] = ok ? 0 : 1;
    }
}

// Compaction, first kernel (one block): the free pages below L (holes) and the
// used ones from L on (movers) by rank, refs, and where each mover goes.
//   plan[0] = L, plan[1] = moves; src, dst [n_pages/2 + 1]; to [n_pages]
__global__ void __launch_bounds__(kPlanThreads)
    q4k_pages_plan_kernel(int64_t n_pages, int32_t* refs, int32_t* plan, int32_t* src, int32_t* dst, int32_t* to) {
    __shared__ int warp_sums[32];
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    int used = 0;
    for (int64_t p0 = 0; p0 < n_pages; p0 += kPlanThreads)
        used += __syncthreads_count(p0 + threadIdx.x < n_pages && refs[p0 + threadIdx.x] > 0);
    int holes = 0, movers = 0;
    for (int64_t p0 = 0; p0 < n_pages; p0 += kPlanThreads) {
        const int64_t p = p0 + threadIdx.x;
        const bool in = p < n_pages, live = in && refs[p] > 0;
        int here;
        const bool hole = in && !live && p < used, mover = live && p >= used;
        if (p0 < used) {
            const int r = holes + block_rank<kPlanThreads>(hole, warp_sums, here);
            if (hole) dst[r] = static_cast<int32_t>(p);
            holes += here;
        }
        if (p0 + kPlanThreads > used) {
            const int r = movers + block_rank<kPlanThreads>(mover, warp_sums, here);
            if (mover) src[r] = static_cast<int32_t>(p);
            movers += here;
        }
    }
    __syncthreads();
    for (int r = threadIdx.x; r < movers; r += kPlanThreads) {
        const int s = src[r], d = dst[r];
        to[s] = d;
        refs[d] = refs[s];
        refs[s] = 0;
    }
    if (threadIdx.x == 0) {
        plan[0] = used;
        plan[1] = movers;
    }
}

// Second kernel: the copies, and the tables' entries that moved.
__global__ void __launch_bounds__(kCopyThreads)
    q4k_pages_move_kernel(const PageGeom g, const int32_t* plan, const int32_t* src,
                          const int32_t* dst, const int32_t* to, int64_t n_pages,
                          int n_seqs, int width, int page_size, int32_t* table, const int32_t* lens,
                          int parts) {
    pdl_wait();
    const int used = plan[0], moves = plan[1];
    const int64_t per_pair = static_cast<int64_t>(g.layers) * 2 * parts, total = moves * per_pair;
    for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
        const int i = static_cast<int>(w / per_pair);
        const int r = static_cast<int>(w - i * per_pair);
        copy_part(g, src[i], dst[i], r / (2 * parts), (r / parts) & 1, r % parts);
    }
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (kCopyThreads / 32);
    for (int s = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); s < n_seqs; s += warps) {
        const int64_t len = min(max(static_cast<int64_t>(lens[s]), int64_t(0)), static_cast<int64_t>(width) * page_size);
        const int pages = static_cast<int>((len + page_size - 1) / page_size);
        int32_t* row = table + static_cast<int64_t>(s) * width;
        for (int j = lane; j < pages; j += 32) {
            const int page = row[j];
            if (page >= used && page < n_pages) {
                const int d = to[page];  // (an entry that names a free page has no place to go)
                if (d >= 0 && d < used) row[j] = d;
            }
        }
    }
}

// ------------------------------------------------------------------ host ---

// Four blocks per SM, 16 KB on the way in each (compaction 167 us, forks 10.8;
// eight: 171 and 11.3, two: 177 and 11.5).
static int copy_grid(int64_t parts, const DeviceInfo& dev) {
    const int64_t most = static_cast<int64_t>(dev.num_sms) * (1024 / kCopyThreads);
    return static_cast<int>(parts < most ? (parts < 1 ? 1 : parts) : most);
}

cudaError_t launch_pages_copy(const q4k_cache& c, const int32_t* src, const int32_t* dst, int64_t n,
                              cudaStream_t stream, const DeviceInfo& dev, int pdl) {
    const PageGeom g = geom(c);
    const int parts = parts_per_page(g);
    return launch_serve(q4k_pages_copy_kernel, dim3(copy_grid(n * g.layers * 2 * parts, dev)), dim3(kCopyThreads),
                        0, stream, pdl, 1, g, src, dst, n, c.n_pages, parts);
}

cudaError_t launch_pages_free(const q4k_cache& c, const int32_t* seqs, int n, cudaStream_t stream, int pdl) {
    return launch_serve(q4k_pages_free_kernel, dim3(n), dim3(256), 0, stream, pdl, 1, seqs, c.n_seqs, c.width,
                        c.n_pages, c.refs, c.table, c.lens);
}

cudaError_t launch_pages_reserve(const q4k_cache& c, const int32_t* seqs, int n, const int32_t* starts,
                                 int32_t* status, cudaStream_t stream, int pdl) {
    return launch_serve(q4k_pages_reserve_kernel, dim3(1), dim3(kPlanThreads), 0, stream, pdl, 1, seqs, n, starts,
                        status, c.n_seqs, c.width, c.page_size, c.n_pages, c.refs, c.table, c.lens);
}

cudaError_t launch_pages_fork(const q4k_cache& c, const int32_t* parents, const int32_t* children, int n,
                              int32_t* status, uint32_t* counters, cudaStream_t stream, const DeviceInfo& dev,
                              int pdl) {
    const PageGeom g = geom(c);
    const int parts = parts_per_page(g);
    return launch_serve(q4k_pages_fork_kernel,
                        dim3(copy_grid(static_cast<int64_t>(n) * g.layers * 2 * parts, dev)), dim3(kCopyThreads),
                        12 * static_cast<size_t>(n), stream, pdl, 1, g, parents, children, n, status, c.n_seqs, c.width, c.page_size,
                        c.n_pages, c.refs, c.table, c.lens, parts, counters + kPageTicket);
}

cudaError_t pages_setup() {
    // 48 KB of plan for the most forks, beside the kernel's own
    return cudaFuncSetAttribute(q4k_pages_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 12 * kMaxBatch);
}

int64_t pages_scratch_bytes(int64_t n_pages) { return 256 + 4 * (2 * (n_pages / 2 + 1) + n_pages); }

cudaError_t launch_pages_compact(const q4k_cache& c, void* scratch, cudaStream_t stream, const DeviceInfo& dev,
                                 int pdl) {
    const PageGeom g = geom(c);
    const int parts = parts_per_page(g);
    int32_t* plan = static_cast<int32_t*>(scratch);
    int32_t* src = plan + 64;
    int32_t* dst = src + c.n_pages / 2 + 1;
    int32_t* to = dst + c.n_pages / 2 + 1;
    cudaError_t e = launch_serve(q4k_pages_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, pdl, 1, c.n_pages,
                                 c.refs, plan, src, dst, to);
    if (e != cudaSuccess) return e;
    return launch_serve(q4k_pages_move_kernel, dim3(copy_grid(c.n_pages / 2 * g.layers * 2 * parts, dev)),
                        dim3(kCopyThreads), 0, stream, pdl, 1, g, plan, src, dst, to, c.n_pages, c.n_seqs, c.width,
                        c.page_size, c.table, c.lens, parts);
}

}  // namespace q4k
