/*
 * q4k.h -- C ABI of libq4k, a GB300 (sm_103a) library for the packed Q4_K
 * dequant-matmul: the Op::DequantMatMul that the rlx pages emit for every
 * linear layer of a GGUF K-quant model ("rlx-qwen3" crate page, packed-GGUF
 * note under "Quick start": K-quant tensors stay packed and each matmul
 * dequantises them; "rlx-llama32" crate page, section "Packed GGUF").
 *
 * Weights stay in device memory in their 144-byte Q4_K super-blocks and are
 * dequantised inside the kernels.
 *
 * ---------------------------------------------------------------- layout ---
 * W : uint8, N rows of K/256 super-blocks, row-major. Row n's super-blocks are
 *     contiguous and in k order; super-block b of row n starts at byte
 *     (n*K/256 + b)*144. A super-block encodes weights 256b .. 256b+255:
 *       bytes 0..1   d     IEEE binary16, little-endian
 *       bytes 2..3   dmin  IEEE binary16, little-endian
 *       bytes 4..15  s[12] eight 6-bit sub-block scales and eight 6-bit mins:
 *                    sub-block j<4 : sc = s[j]&63, m = s[j+4]&63
 *                    sub-block j>=4: sc = (s[j+4]&15) | ((s[j-4]>>6)<<4),
 *                                    m  = (s[j+4]>>4) | ((s[j]>>6)<<4)
 *       bytes 16..143 qs[128]: byte 32c+l holds weight 64c+l in its low
 *                    nibble and weight 64c+32+l in its high nibble; weight i
 *                    belongs to sub-block i/32.
 *     Weight value: w = d*sc*q - dmin*m. (Both products are exact in fp32, so
 *     w is the exact value rounded once to fp32.)
 * X : [M][K] row-major activations, fp32 or bfloat16.
 * Y : fp32 [M][N] row-major, Y[m][n] = sum_k X[m][k] * w(n,k). Y is
 *     overwritten, never accumulated into.
 *
 * ---------------------------------------------------------------- calls ---
 * Every call is asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 * default stream), allocates nothing, never synchronises the host, and may be
 * captured into a CUDA graph (call q4k_init() once per device before the first
 * capture so that one-time kernel attribute set-up happens outside it).
 * All pointers are device pointers owned by the caller; the library keeps no
 * reference to them after the call returns.
 *
 * ---------------------------------------------------------------- errors ---
 * Arguments are checked on the host before anything is launched; on any
 * negative status nothing was launched, except Q4K_ERR_CUDA (the launch itself
 * failed; the CUDA error is left for the caller to query). A wait inside a
 * kernel that runs out of time (a fault, never expected) sets a device error
 * word and the kernel ends early; q4k_device_error() reports it.
 */
#ifndef Q4K_H_
#define Q4K_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum q4k_status {
    Q4K_OK = 0,
    Q4K_ERR_NULL = -1,     /* a required pointer is NULL */
    Q4K_ERR_BAD_DIM = -2,  /* a size or mode out of range: needs N, M >= 1, K >= 256 and
                              K % 256 == 0, N and M below 2^31, K <= 2^24, 1 <= count <= 8
                              (grouped calls), M <= 16 (argmax calls), mode 0..2 (PDL) */
    Q4K_ERR_CUDA = -3,     /* a CUDA runtime call or kernel launch failed */
    Q4K_ERR_ALIGN = -4,    /* a pointer lacks the alignment that the call states (W, X, Y and
                              the float or bf16 arrays: 16 bytes) */
    Q4K_ERR_ARCH = -5,     /* current device is not compute capability 10.3 */
    Q4K_ERR_TIMEOUT = -6,  /* a bounded in-kernel wait ran out (device error word) */
    Q4K_ERR_SPACE = -7     /* the workspace is smaller than the call needs */
};

/* Human-readable name of a status code (static string, never NULL). */
const char* q4k_status_string(int status);

/*
 * One-time set-up for the current device: checks the architecture and sets the
 * kernels' shared-memory attributes. Called implicitly by the first call on a
 * device; call it explicitly before capturing a CUDA graph.
 */
int q4k_init(void);

/*
 * Standalone dequantisation (the CPU-F32 parity path of the rlx-llama32 page's
 * prefill modes, done on the GPU): out_f32[n*K + k] = w(n, k) for all n < N,
 * k < K. Bit-exact: every weight is the exact d*sc*q - dmin*m rounded once.
 *   W        device, N*K/256*144 bytes, 16-byte aligned
 *   out_f32  device, N*K floats, 16-byte aligned
 */
int q4k_dequant(const void* W, int64_t N, int64_t K, float* out_f32, void* stream);

/*
 * Y = X * W^T with fp32 activations X [M][K]: the packed-weight matmul that
 * each linear layer of a K-quant model emits ("rlx-qwen3" crate page, the
 * packed-GGUF note under "Quick start"; "rlx-llama32" crate page, section
 * "Packed GGUF"), with the weights dequantised inside the kernel.
 * M <= 16 (decode) runs one decode launch (M <= 2: the CUDA-core GEMV; 3..16:
 * the tensor-core kernel, fp32 accuracy kept by splitting X into bf16 hi +
 * lo); larger M runs it over 16-row slices of X, which reads W once per slice
 * (fp32 prefill costs ceil(M/16) weight sweeps; bf16 activations through
 * q4k_matmul_bf16 read W once). Accuracy: |Y - exact| <= 1e-4 * sum_k |X*w|
 * per output.
 *   W  device, N*K/256*144 bytes; X device, M*K floats; Y device, M*N floats;
 *   all 16-byte aligned.
 */
int q4k_matmul(const void* W, int64_t N, int64_t K, const float* X, int64_t M, float* Y,
               void* stream);

/*
 * Y = X * W^T with bfloat16 activations X_bf16 [M][K] (bit patterns): the same
 * packed-weight matmul ("rlx-llama32" crate page, section "Packed GGUF") for a
 * block of token rows, as the chunked prefill of the nx_f32_llm_run_v3 listing
 * issues it. M <= 16 runs the decode kernels (M <= 2 on the CUDA cores, 3..16
 * on the tensor cores with the 4-bit codes as the MMA operand; accuracy 1e-4 *
 * sum|X*w|); M >= 17 (chunked prefill) runs the tcgen05 tensor-core GEMM,
 * which rounds the dequantised weights to bfloat16 (accuracy 5e-3 * sum|X*w|).
 *   W  device, N*K/256*144 bytes; X_bf16 device, M*K uint16; Y device, M*N
 *   floats; all 16-byte aligned.
 */
int q4k_matmul_bf16(const void* W, int64_t N, int64_t K, const uint16_t* X_bf16, int64_t M,
                    float* Y, void* stream);

/*
 * Grouped decode call: Y_i = X * W_i^T for i < count (1 <= count <= 8), where
 * all W_i have the same K and take the same activations X -- e.g. the q, k and
 * v projections of a layer, or its gate and up projections. W, N and Y are
 * host arrays of length count holding device pointers / row counts; Y_i is
 * fp32 [M][N_i]. All matrices run in one launch (fp32 activations with
 * M > 16: one launch per 16-row slice of X), with the kernel and accuracy of
 * q4k_matmul / q4k_matmul_bf16 for the same M. The same checks as the single
 * calls apply to every matrix.
 */
int q4k_matmul_multi(int count, const void* const* W, const int64_t* N, int64_t K, const float* X,
                     int64_t M, float* const* Y, void* stream);
int q4k_matmul_multi_bf16(int count, const void* const* W, const int64_t* N, int64_t K,
                          const uint16_t* X_bf16, int64_t M, float* const* Y, void* stream);

/*
 * Fused lm_head + greedy pick (the device-side version of the host-greedy
 * decode of the "rlx-llama32" crate page, section "Env flags"; the in-graph
 * lm_head there is a DequantMatMul like every other matmul): out_idx[m] =
 * argmax_n Y[m][n] for Y = X * W^T, for 1 <= M <= 16 rows of activations,
 * without writing Y. Ties go to the lowest n; NaN outputs are never picked
 * unless every output of the row is NaN (then 0). Y itself is computed as by
 * q4k_matmul / q4k_matmul_bf16 (accuracy 1e-4 * sum|X*w|), so rows whose two
 * largest outputs differ by less than that may pick either. out_idx: device,
 * int64 [M], 8-byte aligned; it is overwritten (it holds intermediate keys
 * while the call runs). Three kernels on `stream`; allocates nothing.
 */
int q4k_matmul_argmax(const void* W, int64_t N, int64_t K, const float* X, int64_t M,
                      int64_t* out_idx, void* stream);
int q4k_matmul_argmax_bf16(const void* W, int64_t N, int64_t K, const uint16_t* X_bf16, int64_t M,
                           int64_t* out_idx, void* stream);

/*
 * Programmatic dependent launch for every later call in the process (a
 * decode step issues one call per weight matrix, so the gaps between
 * back-to-back kernels matter). Returns the previous mode, or
 * Q4K_ERR_BAD_DIM for an unknown mode.
 *   0  plain launches (default).
 *   1  each call's kernel may be scheduled while the preceding kernel on the
 *      stream is still running; it reads and writes no global memory until
 *      that kernel has completed. Always safe.
 *   2  as 1, and the kernel may also start reading its packed weights W
 *      before the preceding kernel has completed. Only valid when W is not
 *      written by the kernel that immediately precedes the call on the stream
 *      (true for model weights).
 */
int q4k_set_pdl(int mode);

/*
 * Reads the device error word of the current device (synchronous: waits for
 * all prior work on the device). Returns Q4K_OK or Q4K_ERR_TIMEOUT; with
 * clear != 0 the word is reset. Not capturable.
 */
int q4k_device_error(int clear);

/*
 * Exercises the failure path of the in-kernel waits without any fault: one
 * thread of a one-warp kernel waits on an mbarrier that nothing arrives at,
 * bounded by limit_ns nanoseconds (1 .. 10^9). The wait runs out, sets the
 * device error word as a timed-out wait in any libq4k kernel does, and the
 * kernel returns; no copy or tensor-core work is in flight, so the context
 * stays usable. Afterwards q4k_device_error() reports Q4K_ERR_TIMEOUT. For
 * tests of error handling; asynchronous on `stream`. (The pages describe no
 * such call: it checks this library's own timeout mechanism.)
 */
int q4k_selftest_timeout(int64_t limit_ns, void* stream);

/* ======================================================================
 * Between the products of a decode or prefill step
 * ======================================================================
 * What a served model does between two of the calls above: the q, k and v rows
 * of a step go into a paged cache (q4k_cache_append), attention reads it
 * (q4k_cache_attention), the pages are handed out, shared, given back and
 * moved together as sequences come and go (q4k_pages_*), and the logits are
 * adjusted before the greedy pick (q4k_logits_pick). The pages of the
 * reference describe these parts of the runner around Op::DequantMatMul:
 * resident K/V decode ("rlx-llama32" crate page, section "Decode"), the
 * repetition penalty over recent tokens and the pick (nx_f32_llm_run_v3
 * listing).
 *
 * The rules of the calls above hold: asynchronous on `stream`, no allocation,
 * no host synchronisation, capturable, arguments checked before any launch.
 * Device arrays are read when the call runs on the device, so their contents
 * may be produced by earlier work on the stream; contents out of range (a
 * sequence, page, length or token id) never lead outside the arrays, and what
 * they mean is said at each call.
 *
 * A cache describes the K and V pages of all layers of a model:
 *   element (layer, page, kv head, row, dim) of K is at
 *     k[layer*layer_stride + page*page_stride + (head*page_size + row)*head_dim + dim],
 *   and the same for V. Position p of sequence s lives in row p % page_size of
 *   page table[s*width + p/page_size].
 * refs[page] counts the sequences that hold the page; 0: the page is free.
 * lens[s] is the number of positions of sequence s, 0: not in use. Entries of
 * table past a sequence's pages must be -1: q4k_pages_free gives back every page
 * that a row names, the other calls follow a sequence's own pages only.
 *
 * A step's batch is n sequences with new tokens: seqs[i] (device, distinct;
 * NULL: 0..n-1) names the i-th one, and its new tokens are rows starts[i] to
 * starts[i+1]-1 of the step's arrays (starts: device, n+1 ascending values; a
 * sequence may have none). lens counts the new tokens: q4k_pages_reserve adds
 * them, so new token r of a sequence with m of them is at position
 * lens - m + r.
 */
typedef struct q4k_cache {
    uint16_t* k;           /* device, bf16 bit patterns, 16-byte aligned; K and V must not */
    uint16_t* v;           /* overlap, unless k == v: what is stored then is the values */
    int64_t layer_stride;  /* elements; multiples of 8; layers and pages must not overlap */
    int64_t page_stride;
    int32_t* refs;         /* device, [n_pages] */
    int32_t* table;        /* device, [n_seqs][width] */
    int32_t* lens;         /* device, [n_seqs] */
    int64_t n_pages;       /* 1 .. 2^30 */
    int32_t layers;        /* 1 .. 65535 */
    int32_t kv_heads;      /* 1 .. 1024 */
    int32_t page_size;     /* 16, 32, 64 or 128 */
    int32_t head_dim;      /* 64 or 128 */
    int32_t n_seqs;        /* 1 .. 2^24 */
    int32_t width;         /* pages per sequence at most; width*page_size <= 2^30 */
} q4k_cache;

/*
 * Bytes of the workspace that the calls below take (device, 256-byte aligned),
 * or a negative status. It must be zero-filled before its first use; every
 * call leaves what later calls rely on, so one workspace serves any sequence
 * of calls on one stream. Calls that may run at the same time need one each.
 * A call that ended in Q4K_ERR_TIMEOUT leaves it undefined: zero it again.
 * The size depends on n_pages, head_dim and the device only.
 */
int64_t q4k_cache_workspace(const q4k_cache* c);

/*
 * Stores a step's keys and values in one layer, from the fp32 outputs of its
 * q, k and v products (q4k_matmul_multi): for every new token
 *   K page row = bf16(rot(norm(Yk row, k_norm))),  V page row = bf16(Yv row),
 *   q_out row  = bf16(rot(norm(Yq row, q_norm))),
 * per head. norm(x, w) = x / sqrt(mean(x^2) + eps) * w where the weights are
 * given (head_dim floats, the per-head norm of Qwen3), else x. rot turns pairs
 * of elements by the angle of the token's position p: (a, b) becomes
 * (a cos - b sin, a sin + b cos), with cos = rope[p*head_dim + i] and sin =
 * rope[p*head_dim + head_dim/2 + i] for pair i; pairs = 1: elements (2i, 2i+1),
 * 2: (i, i + head_dim/2), 0: no rotation (rope may be NULL). Everything is
 * computed in fp32 and rounded once.
 *   Yq  device, [tokens][heads*head_dim] floats; Yk, Yv [tokens][kv_heads*head_dim]
 *   q_out  device, [tokens][heads][head_dim] bf16
 *   rope   device, [rope_rows][head_dim] floats, rope_rows >= width*page_size
 * heads is a multiple of kv_heads. 1 <= n <= 4096; 1 <= tokens < 2^31.
 * Rows of a sequence id, position or page out of range are not stored (their
 * q_out is still written, unrotated when there is no position).
 */
int q4k_cache_append(const q4k_cache* c, int layer, const int32_t* seqs, int n, const int32_t* starts,
                     int64_t tokens, const float* Yq, const float* Yk, const float* Yv,
                     uint16_t* q_out, int heads, const float* rope, int64_t rope_rows, int pairs,
                     const float* q_norm, const float* k_norm, float eps, void* stream);

/*
 * Attention of the step's new tokens over their sequences' pages in one layer:
 * for the token at position p of its sequence and query head h (which reads kv
 * head h / (heads/kv_heads)),
 *   out = sum_j a_j v_j / sum_j a_j,   a_j = exp(scale q.k_j - max),
 * over the positions j <= p and, with window > 0, only j > p - window or
 * j < sinks (a sliding window, and first tokens that stay visible). A token
 * that sees nothing (a position below 0, a sequence id out of range) gets
 * zeros. What no token sees (rows past a sequence's length, other sequences'
 * pages) does not enter, whatever it holds, NaN and infinities included; table
 * entries out of range read as zeros.
 *   Q, out  device, [tokens][heads][head_dim] bf16, 16-byte aligned; rows of
 *           out that belong to no sequence of the batch are left as they are
 *   max_new the largest number of new tokens of a sequence, as far as the
 *           caller knows it: it selects between kernels, and with that the
 *           rounding of the weights (below), for all tokens of the call; any
 *           value is right for any step
 *   scale   > 0, finite; window, sinks >= 0 (sinks is ignored with window 0)
 *   ws      see q4k_cache_workspace; ws_bytes its size
 * heads/kv_heads <= 128; 1 <= n <= 4096; 1 <= tokens < 2^31 / heads.
 * Accumulates in fp32; for the product with V the weights a_j are rounded to
 * bf16, or, with max_new * heads/kv_heads <= 16, to the sum of two bf16. The
 * result does not depend on timing.
 */
int q4k_cache_attention(const q4k_cache* c, int layer, const int32_t* seqs, int n,
                        const int32_t* starts, int64_t tokens, const uint16_t* Q, uint16_t* out,
                        int heads, int max_new, float scale, int window, int sinks, void* ws,
                        int64_t ws_bytes, void* stream);

/*
 * Makes room for a step's new tokens: sequence seqs[i] grows by starts[i+1] -
 * starts[i] positions, with pages from the lowest free ones, given out in the
 * order of i. status[i] (device): 0, or 1 where the pages left over (or width)
 * do not suffice, or the id is out of range; such a sequence keeps its length
 * and pages. (Pages are given while the running total of the batch's needs
 * fits the free pages; a sequence that needs none always succeeds.) Give a
 * sequence with status 1 no new tokens in the step's other calls: its length does
 * not count them, so they would be stored over its last positions, in pages
 * that other sequences may hold too.
 * 1 <= n <= 4096.
 */
int q4k_pages_reserve(const q4k_cache* c, const int32_t* seqs, int n, const int32_t* starts,
                      int32_t* status, void* stream);

/*
 * Forks: sequence children[i], which must have length 0, becomes a copy of
 * parents[i]. Full pages are shared (refs + 1); a partly filled last page is
 * copied, in every layer, to the lowest free page, in the order of i. status[i]
 * (device): 0, or 1 where no page is left, the child is in use or an id is out
 * of range (nothing changes for it). A parent may appear several times; a child
 * appears once and is no parent of the same call. 1 <= n <= 4096.
 */
int q4k_pages_fork(const q4k_cache* c, const int32_t* parents, const int32_t* children, int n,
                   int32_t* status, void* ws, int64_t ws_bytes, void* stream);

/*
 * Ends the n distinct sequences: their pages lose a reference, their lengths
 * become 0 and their table rows -1. Ids out of range are skipped.
 */
int q4k_pages_free(const q4k_cache* c, const int32_t* seqs, int n, void* stream);

/*
 * Copies page src[i] to page dst[i] in every layer, K and V (device arrays;
 * the pages of dst are distinct and none is in src; pairs with an id out of
 * range are skipped). refs and table are the caller's business. n < 2^31.
 */
int q4k_pages_copy(const q4k_cache* c, const int32_t* src, const int32_t* dst, int64_t n, void* stream);

/*
 * Moves the pages in use to the lowest ids: with L of them, the i-th free page
 * below L takes the i-th used page from L on, in every layer; refs and table
 * follow. Pages from L on are free afterwards.
 */
int q4k_pages_compact(const q4k_cache* c, void* ws, int64_t ws_bytes, void* stream);

/*
 * Adjusts M rows of V logits and picks the largest of each: for a token that
 * occurs count > 0 times in its row's history,
 *   x = x > 0 ? x / repeat : x * repeat;  x = (x - count*frequency) - presence;
 * then x = x + bias where the row has one for the token, then -inf where the
 * row's grammar forbids it. pick[m] is the lowest index with the largest x
 * among the allowed ones (NaN below every number), or -1 if none is allowed.
 * fp32, every operation rounded by itself.
 *   logits    device, [M][V] floats, 16-byte aligned
 *   out       device, [M][V] floats, 16-byte aligned, may be logits itself; NULL: not kept
 *   pick      device, [M] int64; NULL: no pick (out and pick are not both NULL)
 *   history   device, token ids of row m at hist_starts[m] .. hist_starts[m+1]-1
 *             (M+1 ascending offsets); NULL: none. Ids out of range are ignored.
 *   penalties device, [M][3]: repeat, presence, frequency; required with history
 *   bias_ids, bias, bias_starts  device, ids and values of row m likewise; NULL:
 *             none. Ids out of range are ignored; of an id given twice in a row
 *             the later entry counts.
 *   mask      device, [M][ceil(V/32)] words, bit v % 32 of word v / 32 set:
 *             token v is allowed; NULL: all are
 * 1 <= M <= 65535; 1 <= V < 2^31.
 */
int q4k_logits_pick(const float* logits, int64_t M, int64_t V, float* out, int64_t* pick,
                    const int32_t* history, const int32_t* hist_starts, const float* penalties,
                    const int32_t* bias_ids, const float* bias, const int32_t* bias_starts,
                    const uint32_t* mask, void* stream);

/* ======================================================================
 * The expert layer of a mixture-of-experts model
 * ======================================================================
 * A layer whose feed-forward part is E experts with packed Q4_K matrices, k of
 * them for each token: the norm before it (q4k_add_norm), the router's picks
 * and the order of the rows by expert (q4k_route, from the logits of the
 * router's product), the rows in that order (q4k_experts_gather), the experts'
 * products (q4k_experts_gated for gate and up, q4k_experts_matmul for down),
 * and the way back with the weights applied (q4k_experts_combine).
 *
 * The rules of the calls above hold: asynchronous on `stream`, no allocation,
 * no host synchronisation, capturable, arguments checked before any launch,
 * contents of device arrays never lead outside the arrays. Arrays and stream belong to
 * the current device. Arrays that a call writes overlap no other array of the call unless it
 * is said.
 *
 * A step has T tokens. Its pairs are (t, j), token t with its j-th pick, numbered
 * t*k + j. Sorted by expert and within an expert by number they are the rows of
 * the experts' products: row p is pair order[p], pair i is row slots[i], and
 * expert e has rows starts[e] .. starts[e+1]-1.
 */

enum q4k_type { Q4K_F32 = 0, Q4K_BF16 = 1 };

/*
 * r = x + delta; sum = r; y = r / sqrt(mean(r^2) + eps) * weight, row by row, in
 * fp32, and y as wanted: `out` in fp32 or bf16, and `codes` with `scales` in 8
 * bits: of every 32 columns the scale is the smallest power of two s >= 2^-127
 * with max|y| <= 448 s, held as the byte log2(s) + 127, and the codes are y / s
 * rounded to e4m3 (4 significant bits, to nearest even). 32 columns with an
 * infinity or a NaN have the scale byte 255 and codes of NaN. Where mean(r^2)
 * passes fp32, the row's y are 0 (those of infinities NaN).
 *   x       device, [T][C], fp32 or bf16 by x_type
 *   delta   device, [T][C] floats (what the layer before adds); NULL: 0
 *   weight  device, [C] floats
 *   sum     device, [T][C] of x's type (r rounded once; y is taken from r), may be x; NULL: not kept
 *   out     device, [T][C] by out_type; NULL: not wanted
 *   codes, scales  device, [T][C] and [T][C/32] bytes; NULL: not wanted
 * At least one of out and codes is wanted; codes and scales go together.
 * 1 <= T < 2^31; C a multiple of 32, 32 .. 32768; eps >= 0, finite. codes is 8-byte
 * aligned, the others but scales 16.
 */
int q4k_add_norm(const void* x, int x_type, const float* delta, const float* weight, float eps, int64_t T, int64_t C,
                 void* sum, void* out, int out_type, uint8_t* codes, uint8_t* scales, void* stream);

/* How the weights of a token's picks follow from its logits (each times `scale`): */
enum q4k_weighting {
    Q4K_ROUTE_SOFTMAX = 0,     /* softmax over all experts */
    Q4K_ROUTE_SOFTMAX_TOP = 1, /* softmax over the picked ones */
    Q4K_ROUTE_SIGMOID = 2,     /* 1 / (1 + exp(-logit)) */
    Q4K_ROUTE_SIGMOID_TOP = 3  /* the same divided by their sum over the picked ones (0 where no logit is -1000 or more: a mask) */
};

/*
 * The k largest logits of each token, largest first (ties: the lowest expert
 * first), their weights, and the order of the pairs by expert. A logit of -inf or
 * NaN is never picked and counts for nothing in a softmax (a mask); where fewer
 * than k are left, the last picks have id -1, weight 0 and slot -1, and are
 * among no expert's rows. starts[E] is the number of rows; order is -1 from there on.
 *   logits  device, [T][E] floats
 *   ids, weights, slots  device, [T][k] int32, floats, int32
 *   order   device, [T*k] int32;  starts  device, [E+1] int32
 *   ws      device, ws_bytes >= q4k_route_workspace(T, E), 4-byte aligned; needs no
 *           set-up and holds nothing between calls; calls that may run at the same
 *           time need one each
 * 1 <= k <= 32, k <= E <= 1024; T >= 1, T*k < 2^31; scale finite.
 */
int64_t q4k_route_workspace(int64_t T, int64_t E); /* 4 E (ceil(T / 64) + 1) */
int q4k_route(const float* logits, int64_t T, int64_t E, int k, int weighting, float scale, int32_t* ids, float* weights,
              int32_t* order, int32_t* slots, int32_t* starts, void* ws, int64_t ws_bytes, void* stream);

/*
 * Rows in the order of their experts: out[p] = X[order[p] / k] for p < T*k; rows
 * whose order is outside [0, T*k) are left as they are. X: bf16 (scales NULL), or
 * e4m3 codes with scales as q4k_add_norm writes them; a code times its scale is
 * exact in bf16 (down to 2^-126). (Codes are for rows that are kept or sent
 * in 8 bits: they have 4 significant bits, and where the norm writes bf16 rows as well,
 * gathering those is the faster and the more exact way.)
 *   X    device, [T][C] bf16 or codes;  scales  device, [T][C/32] bytes or NULL
 *   out  device, [T*k][C] bf16
 * 1 <= k <= 32, T >= 1, T*k < 2^31; C a multiple of 8 (of 32 with scales), 8 .. 32768.
 * X and out 16-byte aligned (codes 8).
 */
int q4k_experts_gather(const void* X, const uint8_t* scales, const int32_t* order, int64_t T, int k, int64_t C,
                       uint16_t* out, void* stream);

/*
 * The experts' products: Y[p] = X[p] W_e^T for the rows p of every expert e, W_e
 * the e-th of E packed matrices [N][K] that follow one another; accumulated in
 * fp32 and rounded once to bf16. q4k_experts_gated takes two of them and gives
 * Y[p] = g / (1 + exp(-g)) * u with g = X[p] gate_e^T and u = X[p] up_e^T in fp32.
 * By the sizes (never by what the arrays hold) one of two kernels runs: for few
 * rows the weights enter exactly (the sums of x beside the mins as two bf16 each,
 * off by 2^-16); for many the tcgen05 tensor cores take them as bf16: with a =
 * d sc and b = dmin m of a weight's sub-block, off by 2^-8 (|w| + |a| / 16) to
 * within 3 % where 0 <= b <= 15.96 a, by 2^-8 3 |w| elsewhere (q4k_matmul_bf16's
 * weights, for 17 rows and more, by 2^-8 |w|).
 * Rows before starts[0] and from starts[E] on are left as they are; starts is
 * taken as ascending and inside [0, pairs] (values are clamped to that).
 *   W, gate, up  device, E*N*K/256*144 bytes, 16-byte aligned
 *   X  device, [pairs][K] bf16, values below 2^64 (those below 2^-56 may count as
 *      zero);  Y  device, [pairs][N] bf16
 *   starts  device, [E+1] int32
 * X and Y 16-byte aligned. 1 <= E <= 1024, N >= 1, E*N < 2^31; K a multiple of 256, 256 .. 2^24; 1 <= pairs < 2^31.
 */
int q4k_experts_matmul(const void* W, int64_t E, int64_t N, int64_t K, const uint16_t* X, const int32_t* starts,
                       int64_t pairs, uint16_t* Y, void* stream);
int q4k_experts_gated(const void* gate, const void* up, int64_t E, int64_t N, int64_t K, const uint16_t* X,
                      const int32_t* starts, int64_t pairs, uint16_t* Y, void* stream);

/*
 * Back to the tokens: out[t] = base[t] + sum_j weights[t][j] * Y[slots[t][j]], in
 * fp32, added in the order of j. A slot outside [0, pairs) adds nothing.
 *   Y      device, [pairs][C] bf16;  slots, weights  device, [T][k]
 *   base   device, [T][C] floats (a shared expert's output, the residual stream); NULL: 0
 *   out    device, [T][C] floats, may be base
 * 1 <= k <= 32, T >= 1, T*k < 2^31, 1 <= pairs < 2^31; C a multiple of 8, 8 .. 32768. Y, base
 * and out 16-byte aligned.
 */
int q4k_experts_combine(const uint16_t* Y, int64_t pairs, const int32_t* slots, const float* weights, const float* base,
                        int64_t T, int k, int64_t C, float* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* Q4K_H_ */
