/*
 * w4a16moe.h - C ABI of the GB300 (sm_103a) W4A16 routed-expert MoE layer.
 *
 * The layer is the routed-expert block of the 125B-A6B MoE described in
 * "Running 125B MoE on Three 3090s - vLLM Optimization Edition", section 3.3
 * "MoE block (decode-05)": a BF16 router GEMV, softmax and top-k with
 * renormalised weights (norm_topk_prob), the token-to-expert alignment, and
 * the fused W4A16 expert GEMMs (gate_up, SiluAndMul, down) followed by the
 * weighted sum over the selected experts. Shapes are those of "Running 125B
 * MoE on Three 3090s - vLLM Edition", section 1 "Shape of This Model"
 * (hidden 2560, 512 experts, 10 per token, moe_intermediate 640); the weight
 * format is group A of the model card's "What is quantized" table (INT4,
 * group size 128, symmetric, compressed-tensors pack-quantized).
 *
 * Conventions for every call:
 *  - All pointers except `dims`/`bytes` outputs are DEVICE pointers of the
 *    current CUDA device, owned by the caller; the library never allocates,
 *    frees or synchronises inside moe_route / moe_w4a16_forward /
 *    moe_w4a16_forward_rms / moe_permute / moe_pack_int4.
 *  - `stream` is a cudaStream_t (NULL = legacy default stream). Work is
 *    enqueued asynchronously; results are valid once the stream reaches them.
 *  - bf16 tensors are passed as `uint16_t*` holding IEEE bfloat16 bits.
 *  - Every tensor is row-major and contiguous; every pointer is 16-byte
 *    aligned.
 *  - Supported shapes: T >= 0, H and I multiples of 128, 1 <= k <= 32,
 *    k <= E <= 1024, H <= 8064, I <= 4096, T <= 2^20 and T * H < 2^32.
 *    Others return MOE_ERR_UNSUPPORTED before anything is enqueued.
 *  - Argument errors are returned synchronously and enqueue nothing. A
 *    launch failure returns MOE_ERR_CUDA. Errors seen by a kernel (an expert
 *    id outside [0, E), an internal wait that gave up) are recorded in the
 *    workspace's error word and reported by moe_check_device_error.
 *  - Workspace: `ws` must hold at least moe_workspace_size() bytes and must
 *    be all zero before its first use (the library leaves the counters it
 *    uses at zero when a call completes, at offsets that depend on no
 *    dimension, so calls of different dims may share a workspace large
 *    enough for each). One workspace must not be used by two calls that may
 *    run concurrently. A call whose bounded wait gave up
 *    (MOE_ERR_TIMEOUT) can leave counters non-zero: moe_check_device_error
 *    then clears the whole workspace before it returns, and a caller that
 *    does not call it must clear the workspace itself before reusing it.
 */
#ifndef W4A16MOE_H
#define W4A16MOE_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MOE_API __attribute__((visibility("default")))
#else
#define MOE_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,  /* null / misaligned pointer, negative size */
    MOE_ERR_UNSUPPORTED = 2,  /* shape outside the supported set */
    MOE_ERR_WORKSPACE = 3,    /* workspace too small */
    MOE_ERR_CUDA = 4,         /* a CUDA runtime call or launch failed */
    MOE_ERR_DEVICE = 5,       /* a kernel saw an expert id, slot, page, length, token or logit out of range */
    MOE_ERR_TIMEOUT = 6       /* a kernel's bounded wait gave up */
} moe_status;

/* Layer dimensions: T tokens, hidden H, E experts, k experts per token,
 * expert intermediate I. The quantisation group is fixed at 128. */
typedef struct {
    int32_t T, H, E, k, I;
} moe_dims;

/* Static description of a status code. Never NULL. */
MOE_API const char *moe_status_str(int status);

/* Library version as major*10000 + minor*100 + patch. */
MOE_API int moe_version(void);

/* Workspace bytes needed by moe_route, moe_permute and the forward calls
 * for dims `d`. Writes *bytes; returns MOE_OK or MOE_ERR_UNSUPPORTED /
 * MOE_ERR_INVALID_ARG. */
MOE_API int moe_workspace_size(moe_dims d, size_t *bytes);

/*
 * Router + softmax + top-k + renormalisation ("vLLM Optimization Edition",
 * section 3.3 "MoE block": router GEMV, topk_softmax, norm_topk_prob, and
 * the key that sends ties to the lower expert id).
 *
 *   logits[t][e] = sum_h hidden[t][h] * router_w[e][h] (+ bias[e])
 *   topk_ids[t][0..k) = the k largest logits, in order of descending logit,
 *                       ties to the lower id; ranked in fp32
 *   topk_w[t][j]      = softmax over the k selected logits, which equals the
 *                       renormalised full softmax
 *
 * hidden   bf16 [T][H]     router_w bf16 [E][H]
 * bias     f32 [E] or NULL (added to the logits for selection and weights)
 * topk_ids int32 [T][k]    topk_w   f32 [T][k]   (outputs)
 */
MOE_API int moe_route(const uint16_t *hidden, const uint16_t *router_w, const float *bias,
              moe_dims d, int32_t *topk_ids, float *topk_w,
              void *ws, size_t ws_bytes, void *stream);

/*
 * moe_route for a layer with a shared expert ("vLLM Optimization Edition",
 * section 3.3 "MoE block (decode-05)": the router and the shared expert's gate
 * are one GEMV of 512 + 1 rows, and the layer's output is routed +
 * sigmoid(gate) x shared).
 *
 * router_w bf16 [E+1][H]: rows [0, E) route, row E is the shared expert's gate.
 * d: the routed dims (E routed experts, k of them per token); k + 1 <= 32 and
 * E + 1 <= 1024. bias f32 [E] or NULL applies to the routed logits only.
 * topk_ids int32 [T][k+1], topk_w f32 [T][k+1] (outputs): slots [0, k) as
 * moe_route; slot k = expert E with weight sigmoid(x . router_w[E]) (fp32).
 * The workspace is sized by moe_workspace_size(d).
 *
 * The shared expert is then expert E of the weight tensors (stored as a
 * routed expert, INT4 g128, intermediate I): moe_w4a16_forward with dims
 * (T, H, E+1, k+1, I) and these ids and weights computes
 *   out = sum_j topk_w[j] * expert_j(x) + sigmoid(gate) * shared(x)
 * in one pass, with one rounding to bf16. Its workspace is sized by
 * moe_workspace_size(T, H, E+1, k+1, I).
 */
MOE_API int moe_route_shared(const uint16_t *hidden, const uint16_t *router_w, const float *bias,
                     moe_dims d, int32_t *topk_ids, float *topk_w,
                     void *ws, size_t ws_bytes, void *stream);

/*
 * Routed-expert forward ("vLLM Optimization Edition", section 3.3: the fused
 * Marlin MoE gate_up, SiluAndMul, down, and moe_sum; weights as in the model
 * card's group A):
 *
 *   W1[e][n][c] = (nibble c%8 of w1_packed[e][n][c/8] - 8) * w1_scales[e][n][c/128]
 *   W2[e][n][c] likewise from w2_packed / w2_scales
 *   for each token t and slot j, e = topk_ids[t][j]:
 *     g = W1[e][0:I] . x_t,  u = W1[e][I:2I] . x_t,  h = SiLU(g) * u
 *     out[t] += topk_w[t][j] * (W2[e] . h)
 *   out is rounded to bf16 once.
 *
 * hidden    bf16 [T][H]         topk_ids int32 [T][k] in [0, E)
 * topk_w    f32 [T][k]          (taken as given; need not sum to 1)
 * w1_packed int32 [E][2I][H/8]  (rows [0,I) gate, [I,2I) up; low nibble first)
 * w1_scales bf16 [E][2I][H/128]
 * w2_packed int32 [E][H][I/8]   w2_scales bf16 [E][H][I/128]
 * out       bf16 [T][H]         (output; must not overlap any input)
 *
 * Accumulation is fp32; the SiLU(g)*u activation is rounded to bf16 where it
 * feeds the down projection. An id outside [0, E) sets MOE_ERR_DEVICE in the
 * workspace and that slot contributes nothing.
 */
MOE_API int moe_w4a16_forward(const uint16_t *hidden, const int32_t *topk_ids, const float *topk_w,
                      const int32_t *w1_packed, const uint16_t *w1_scales,
                      const int32_t *w2_packed, const uint16_t *w2_scales,
                      uint16_t *out, moe_dims d, void *ws, size_t ws_bytes, void *stream);

/*
 * Forward followed by the residual and RMS rescale used between the layers
 * of a stack (no learned weight):
 *   r = hidden + moe(hidden) (fp32),  next[t] = bf16(r / sqrt(mean(r^2) + eps))
 * Same arguments as moe_w4a16_forward; `next` bf16 [T][H] may not overlap
 * `hidden`.
 */
MOE_API int moe_w4a16_forward_rms(const uint16_t *hidden, const int32_t *topk_ids, const float *topk_w,
                          const int32_t *w1_packed, const uint16_t *w1_scales,
                          const int32_t *w2_packed, const uint16_t *w2_scales,
                          uint16_t *next, float eps, moe_dims d, void *ws, size_t ws_bytes,
                          void *stream);

/*
 * The whole MoE block in one call ("vLLM Optimization Edition", section 3.3
 * "MoE block (decode-05)": the router GEMV, topk_softmax, the fused experts and
 * moe_sum; with `shared`, the shared expert's gate as one more router row):
 *
 *   moe_route (shared = 0) or moe_route_shared (shared = 1) with dims d,
 *   then moe_w4a16_forward (out not NULL) or moe_w4a16_forward_rms (next not
 *   NULL) with dims (T, H, E + shared, k + shared, I).
 *
 * Arguments are those of the calls above: router_w bf16 [E + shared][H], bias
 * f32 [E] or NULL, the weights of E + shared experts, topk_ids int32 and
 * topk_w f32 [T][k + shared] (outputs: the selection, as the router calls
 * write it), and exactly one of out / next (the other NULL; eps is read only
 * with next). The workspace must hold max(moe_workspace_size(d),
 * moe_workspace_size(T, H, E + shared, k + shared, I)) bytes; the rules on
 * zeroing are those of every call.
 *
 * Where moe_forward_plan reports bit 512 for the forward's dims (decode
 * batches, T <= 8, whose activations the expert kernel stages in shared
 * memory), one cooperative kernel runs the block: each CTA computes a few
 * router rows with the small-batch router's own arithmetic, the CTAs meet at a
 * grid-wide barrier, every CTA selects the top-k from all logits, and the
 * experts follow in the same launch. Selection, weights and outputs are then
 * bit-identical to the separate calls. Otherwise the router's kernels run,
 * then the forward's.
 */
MOE_API int moe_layer_forward(const uint16_t *hidden, const uint16_t *router_w, const float *bias, int32_t shared,
                      const int32_t *w1_packed, const uint16_t *w1_scales,
                      const int32_t *w2_packed, const uint16_t *w2_scales,
                      uint16_t *out, uint16_t *next, float eps, int32_t *topk_ids, float *topk_w,
                      moe_dims d, void *ws, size_t ws_bytes, void *stream);

/*
 * moe_w4a16_forward for decode batches without a caller workspace. The pages
 * have no counterpart: this entry point exists for callers that cannot
 * provide or allocate a device scratch buffer where they run the layer (a
 * fully carved memory pool, a plugin signature without a workspace argument,
 * a loop where cudaMalloc's device-wide synchronisation is not acceptable).
 *
 * Same computation and arguments as moe_w4a16_forward minus ws/ws_bytes. The
 * scratch is a 1 MiB array that the library holds in device memory, one per
 * device per process; the call allocates and frees nothing.
 *  - Served shapes: those of the fused decode path (T <= 8) whose
 *    moe_workspace_size() is at most 1 MiB (T = 7 at H 2560, E 512, k 10,
 *    I 640 needs about 0.51 MiB). A larger workspace size returns
 *    MOE_ERR_WORKSPACE and T > 8 returns MOE_ERR_UNSUPPORTED, in both cases
 *    before anything is enqueued. T = 0 returns MOE_OK.
 *  - The first call on a device looks up the array's device address (which
 *    may load the module that holds it); make that call before any stream
 *    capture begins.
 *  - Each call first clears the kernel's completion counters in the array
 *    (one cudaMemsetAsync on `stream`), so nothing needs to be zero
 *    beforehand and an earlier call of another shape does not matter.
 *  - Calls on the same device that may overlap in time (other streams, other
 *    host threads) race on the array and give wrong results.
 *  - Ids outside [0, E) contribute nothing; the error word the kernel sets
 *    stays inside the array, where moe_noalloc_check_device_error reads it.
 */
MOE_API int moe_w4a16_forward_noalloc(const uint16_t *hidden, const int32_t *topk_ids, const float *topk_w,
                              const int32_t *w1_packed, const uint16_t *w1_scales,
                              const int32_t *w2_packed, const uint16_t *w2_scales,
                              uint16_t *out, moe_dims d, void *stream);

/*
 * Token-to-expert permutation ("vLLM Optimization Edition", section 3.3:
 * moe_align_block_size, here without block padding): per-expert counts,
 * their exclusive prefix sum, and the assignments a = t*k + j listed expert
 * by expert, in increasing a within an expert. Exposed for testing; the
 * forward calls run the same kernels.
 *
 * topk_ids int32 [T][k]; offsets int32 [E+1] (output); perm int32 [T*k]
 * (output). An id outside [0, E) sets MOE_ERR_DEVICE; such assignments are
 * left out, so offsets[E] counts only valid ones.
 */
MOE_API int moe_permute(const int32_t *topk_ids, moe_dims d, int32_t *offsets, int32_t *perm,
                void *ws, size_t ws_bytes, void *stream);

/*
 * Pack signed int4 values into the storage format of the weights (model
 * card "What is quantized", pack-quantized): packed[n][w] holds
 * q[n][8w..8w+7] + 8, value 8w+i in bits [4i, 4i+4).
 * q int8 [N][K] with values in [-8, 7] (others are clamped and flagged in
 * *bad_count, a device int32 that is incremented, may be NULL);
 * packed int32 [N][K/8]. K must be a multiple of 8.
 */
MOE_API int moe_pack_int4(const int8_t *q, int64_t N, int64_t K, int32_t *packed,
                  int32_t *bad_count, void *stream);

/*
 * W8A16 linear layer ("vLLM Optimization Edition", section 3.3
 * "Hyper-connection (decode-04)": INT8 GEMVs on the pack-quantized words as
 * stored, and a W8A16 GEMM for batches; model card "What is quantized",
 * groups C (INT8 gs64: hyper-connection mixers) and D (INT8 gs128: lm_head)):
 *   W[n][c] = (byte c%4 of w_packed[n][c/4] - 128) * scales[n][c/gs]
 *   y[t][n] = sum_c x[t][c] * W[n][c]   (fp32 accumulation, rounded to bf16 once)
 * x bf16 [T][K]; w_packed int32 [N][K/4] (four values per word, least
 * significant byte first, stored q + 128); scales bf16 [N][K/gs]; y bf16
 * [T][N] (output). gs is 64 or 128 and divides K (K a multiple of 64, at most
 * 65536); T <= 2^20.
 *  - 1 <= T <= 8: the decode GEMV (weights streamed from HBM, mma.sync), when
 *    T * (K + 8) * 2 <= 196608 (else MOE_ERR_UNSUPPORTED). ws may be NULL.
 *  - T > 8: the tcgen05 GEMM (tiles of 128 rows x 128 tokens; a layer with
 *    fewer tiles than SMs is split over K, and the splits are summed in a
 *    fixed order). ws: at least moe_w8a16_workspace_size() bytes, 16-byte
 *    aligned, its first 256 bytes zero before its first use: they hold the
 *    error word that moe_check_device_error reads (a bounded wait that gave
 *    up); the rest holds the splits' f32 results.
 * T = 0 or N = 0 return MOE_OK with nothing enqueued.
 */
MOE_API int moe_w8a16_linear(const uint16_t *x, const int32_t *w_packed, const uint16_t *scales, int32_t gs,
                     uint16_t *y, int32_t T, int32_t N, int32_t K, void *ws, size_t ws_bytes, void *stream);

/* Workspace bytes moe_w8a16_linear needs for these dims (256 for the GEMV and
 * for GEMMs that are not split). Returns MOE_ERR_INVALID_ARG for bad dims. */
MOE_API int moe_w8a16_workspace_size(int32_t T, int32_t N, int32_t K, int32_t gs, size_t *bytes);

/*
 * W4A16 linear layer (no counterpart on the pages, whose INT4 weights are the
 * experts' alone): y = x . W^T with a matrix in the experts' storage, as
 * moe_quantize_int4 writes it:
 *   W[n][c] = (nibble c%8 of w_packed[n][c/8] - 8) * scales[n][c/128]
 *   y[t][n] = sum_c x[t][c] * W[n][c]
 * x bf16 [T][K]; w_packed int32 [N][K/8]; scales bf16 [N][K/128]; y bf16 [T][N]
 * (output; must not overlap an input). K is a multiple of 128, at most 65536;
 * T <= 2^20; N <= 2^31 - 256. Codes enter the products exactly, sums are fp32 and each
 * group's is multiplied by its scale in fp32; y is rounded to bf16 once. (A group's sum
 * is formed before its scale: it is in range where |x| <= 2^117, and may pass to an
 * infinity above that, whatever the scale.) A scale or a value of x that is not finite
 * reaches the values of y that it belongs to, and no others.
 * Each value of y is summed in one order, whatever T and N.
 * ws: moe_w4a16_workspace_size() bytes, reserved: the call neither reads nor writes
 * them (it may be a workspace of the MoE calls).
 * T = 0 or N = 0 return MOE_OK with nothing enqueued.
 */
MOE_API int moe_w4a16_linear(const uint16_t *x, const int32_t *w_packed, const uint16_t *scales, uint16_t *y, int32_t T,
                     int32_t N, int32_t K, void *ws, size_t ws_bytes, void *stream);

/* Workspace bytes moe_w4a16_linear needs for these dims (256 at least). */
MOE_API int moe_w4a16_workspace_size(int32_t T, int32_t N, int32_t K, size_t *bytes);

/*
 * INT4 quantiser of BF16 weights into the experts' storage ("vLLM
 * Optimization Edition", section 7 "Putting MTP on the GPU", make_mtp_int4.py:
 * round to nearest, group size 128, symmetric, per-group search for the clip
 * that minimises the squared error). For each 128 consecutive values w of a
 * row, with amax = max |w| and clip c_j = (100 - j) / 100, j in [0, nclip):
 *   s_j = bf16(c_j * amax / 7)  (fp32 multiply and divide, bf16 round to nearest even)
 *   q_i = clamp(rint(w_i / s_j), -8, 7)  (fp32 divide; q = 0 when s_j = 0)
 * and the group keeps the j with the smallest sum_i (w_i - q_i s_j)^2 (the
 * lowest j on a tie; the sums are formed in fp32, in units of max|w|^2 so that
 * they neither underflow nor overflow). nclip = 1 is plain round to nearest.
 *
 * w bf16 [N][K], finite; K a multiple of 128; 1 <= nclip <= 100.
 * packed int32 [N][K/8] (outputs; q + 8, lowest nibble first), scales bf16
 * [N][K/128], choice int32 [N][K/128] (the chosen j; may be NULL).
 */
MOE_API int moe_quantize_int4(const uint16_t *w, int64_t N, int64_t K, int32_t nclip, int32_t *packed,
                      uint16_t *scales, int32_t *choice, void *stream);

/*
 * The attention block beside the MoE block (no counterpart on the pages, whose
 * attention kernels stay with the serving engine): per-head norms with the
 * rotary turn, a paged KV cache in 4 bits, and attention over it.
 *
 * Tensors of heads are [T][heads][D] with D contiguous and strides of their
 * own for tokens and heads (in elements, multiples of 8; the base 16-byte
 * aligned), so that they may be views of one projection's output.
 */
typedef struct {
    int64_t token, head;
} moe_strides;

/*
 * One layer's cache. A row is the D values (64 or 128) of one (token, KV
 * head): its codes are q + 8 with q in [-8, 7], eight to an int32 word, lowest
 * nibble first, its scale one bf16, and its values q * scale.
 *   k_codes, v_codes   int32 [n_pages][Hkv][page_size][D/8]
 *   k_scales, v_scales bf16  [n_pages][Hkv][page_size]
 * page_size is a power of two from 16 to 1024; n_pages * page_size < 2^31 and
 * n_pages * page_size * Hkv < 2^32 - 1; Hkv is at most 1024. The
 * slot of a token is page * page_size + its place in the page. A scale that is
 * not finite marks a row that held a value that was not: every query that
 * sees the row, and no other, gets NaN.
 */
typedef struct {
    int32_t *k_codes;
    uint16_t *k_scales;
    int32_t *v_codes;
    uint16_t *v_scales;
    int32_t n_pages, Hkv, page_size, D;
} moe_kv4_cache;

/*
 * RMS norm of each query and key head, then the rotary turn, in one pass:
 *   y = x * weight / sqrt(mean(x^2) + eps)            (over the head's D values)
 *   for the pair i of the first rot values, theta = positions[t] * inv_freq[i]:
 *     (a, b) -> (a cos theta - b sin theta, a sin theta + b cos theta)
 * with the pairs (i, i + rot/2), or (2i, 2i + 1) where interleaved is 1. fp32
 * inside (theta is reduced to a fraction of a turn in integers, so far
 * positions lose nothing), rounded to bf16 once.
 *
 * q, q_out bf16 [T][Hq][D], k, k_out bf16 [T][Hkv][D] (an output may be its
 * input, with the same strides); q_weight, k_weight bf16 [D] or NULL (ones);
 * positions int32 [T]; inv_freq f32 [rot/2], finite. D is 64, 128 or 256; rot a
 * multiple of 16 from 0 to D (0: norms alone; positions and inv_freq may be
 * NULL); Hq or Hkv may be 0.
 */
MOE_API int moe_qk_norm_rope(const uint16_t *q, moe_strides q_strides, const uint16_t *k, moe_strides k_strides,
                     const uint16_t *q_weight, const uint16_t *k_weight, const int32_t *positions,
                     const float *inv_freq, int32_t rot, int32_t interleaved, float eps,
                     uint16_t *q_out, moe_strides q_out_strides, uint16_t *k_out, moe_strides k_out_strides,
                     int32_t T, int32_t Hq, int32_t Hkv, int32_t D, void *stream);

/*
 * Writes token t's rows k[t], v[t] (bf16 [T][Hkv][D]) into the cache at
 * slots[t] (int32 [T]; -1: not stored), per row:
 *   s = bf16(max|x| / 7),  q = clamp(rint(x / s), -8, 7)  (fp32 divisions; q = 0 when s = 0)
 * which is moe_quantize_int4 with nclip = 1 over a row. A row with a NaN or an
 * infinity gets a NaN scale. Slots must differ. A slot outside [-1, n_pages *
 * page_size) is left out and sets MOE_ERR_DEVICE in the workspace (at least
 * 256 bytes, the first 256 zero before its first use).
 */
MOE_API int moe_kv4_append(const uint16_t *k, moe_strides k_strides, const uint16_t *v, moe_strides v_strides,
                   const int32_t *slots, int32_t T, moe_kv4_cache cache, void *ws, size_t ws_bytes, void *stream);

/*
 * The inverse: k[t], v[t] (bf16 [T][Hkv][D], contiguous; outputs) = the values
 * of the rows at slots[t], rounded to bf16; a slot of -1 reads as zero, one
 * outside the cache too and sets MOE_ERR_DEVICE.
 */
MOE_API int moe_kv4_read(const int32_t *slots, int32_t T, moe_kv4_cache cache, uint16_t *k, uint16_t *v,
                 void *ws, size_t ws_bytes, void *stream);

/* Workspace bytes moe_kv4_attention needs for these dims (256 serve
 * moe_kv4_append and moe_kv4_read). */
MOE_API int moe_kv4_workspace_size(int32_t T, int32_t Hq, int32_t Hkv, int32_t D, size_t *bytes);

/*
 * Causal attention of B sequences' new tokens over the cache. Sequence b has
 * the queries [cu_q[b], cu_q[b+1]) of q (cu_q int32 [B+1]; NULL: query b, and
 * T = B) and lens[b] keys (int32 [B]), the new tokens' own among them; key j
 * is at page page_table[b][j / page_size] (int32 [B][max_pages]). Of nq
 * queries, query i sees the first lens[b] - nq + i + 1 keys; query head h
 * reads KV head h / (Hq / Hkv):
 *   S_j = scale * q . k_j,  out = sum_j softmax(S)_j v_j,  lse = log sum_j exp(S_j)
 * A query that sees no key gets out = 0 and lse = -inf.
 *
 * q, out bf16 [T][Hq][D] (out must not overlap q or the cache); lse f32
 * [T][Hq] or NULL. Hq is a multiple of Hkv with at most 32 query heads a KV
 * head; T <= 2^20, B <= 4096. max_q is the largest number of queries of a
 * sequence: it decides which kernel runs, never the result, but for the roundings
 * that follow.
 *
 * Softmax statistics and sums are fp32. Codes and scales enter the products
 * exactly; a query's values do where they lie within 2^25 of its row's largest,
 * and are rounded at 2^-33 of that otherwise. A probability (or its product with
 * the key's V scale) is rounded to fp16 where it feeds the tensor core: by 2^-11
 * of itself, or by 2^-31 of the row's largest where it is smaller than 2^-20 of
 * that. A key counts by what it adds to a row: one that the row does not see, or
 * that has no probability in it, takes nothing from the others, whatever its
 * scales (which may lie 2^100 apart in a sequence). out is rounded to bf16 once.
 *
 * A page outside [0, n_pages), a length outside [0, max_pages * page_size] and
 * query offsets that do not rise within [0, T] set MOE_ERR_DEVICE: such a
 * page's rows read as zero, and the others are brought into their range. Rows
 * of out that no sequence covers are not written. Work is counted in units of
 * 128 keys of one KV head for up to 8, 16 or 32 query rows of a sequence (256
 * where max_q chooses the kernel for many), and 3 or 4 more for each such group
 * of rows: a call of 2^31 units or more sets MOE_ERR_DEVICE too and writes
 * nothing (a million queries behind a million keys on 128 KV heads; split it).
 *
 * The workspace holds moe_kv4_workspace_size() bytes under the rules of the
 * MoE calls (all zero before its first use); it may be one that they use.
 */
MOE_API int moe_kv4_attention(const uint16_t *q, moe_strides q_strides, moe_kv4_cache cache,
                      const int32_t *page_table, int32_t max_pages, const int32_t *lens, const int32_t *cu_q,
                      int32_t B, int32_t T, int32_t Hq, int32_t max_q, float scale,
                      uint16_t *out, moe_strides out_strides, float *lse, void *ws, size_t ws_bytes, void *stream);

/*
 * The same with a sliding window and first keys that stay visible: the query at
 * position i (the last of a sequence is at lens[b] - 1) sees the keys j <= i with
 * j > i - window (itself and the window - 1 before it) or j < sinks. window >= 1,
 * sinks >= 0; a window of at least max_pages * page_size is moe_kv4_attention.
 *
 * Only what some query of a (sequence, KV head)'s row tile sees is read, in runs of
 * 16 keys, so the pages that lie wholly before the windows of a sequence's queries
 * of this call (first keys aside) may be gone: their entries in page_table are not
 * looked at. What else holds for moe_kv4_attention holds here, hidden keys counting
 * as those that a query does not see. What lies in keys that no query of a row tile
 * sees (they share a run with keys that one does) changes no bit of the tile's rows.
 */
MOE_API int moe_kv4_attention_window(const uint16_t *q, moe_strides q_strides, moe_kv4_cache cache,
                             const int32_t *page_table, int32_t max_pages, const int32_t *lens, const int32_t *cu_q,
                             int32_t B, int32_t T, int32_t Hq, int32_t max_q, float scale, int32_t window,
                             int32_t sinks, uint16_t *out, moe_strides out_strides, float *lse, void *ws,
                             size_t ws_bytes, void *stream);

/*
 * Verification of drafted tokens against the target's probabilities (no
 * counterpart on the pages, whose drafting stays with the serving engine).
 *
 * Sequence b has the rows [cu_rows[b], cu_rows[b+1]) (cu_rows int32 [B+1]) of
 * logits: its drafts' and one more. Row i predicts the token after the sequence
 * and its first i drafts; drafts[r] (int32 [T]) is the draft that stands at row r
 * (the last row's entry is not read). With t = temperature[b] (f32 [B]; NULL: 1):
 *   p = softmax(logits / t),  q = softmax(draft_logits / t), or 1 at the draft
 *   and 0 elsewhere where draft_logits is NULL;
 *   the draft x of row r is accepted while uniform[r] * q(x) < p(x);
 *   at the first row that refuses its draft, the next token is the v with the
 *   largest max(p_v - q_v, 0) / noise[b][v] (p_v / noise[b][v] where that is zero
 *   for all), at the last row the v with the largest p_v / noise[b][v].
 * With uniform from [0, 1) and noise from Exp(1) the tokens are distributed as if
 * they had been drawn from the target alone. t = 0: a draft is accepted while it is
 * the row's largest logit, which is the next token. Ties go to the lowest v.
 *
 * tokens int32 [T]: of each sequence its accepted drafts, the next token, then -1.
 * accepted int32 [B]: the number of accepted drafts (0 for a sequence without rows).
 *
 * logits, draft_logits bf16 [T][V] with rows `stride` values apart (a multiple of
 * 8); uniform f32 [T]; noise f32 [B][V], rows noise_stride (a multiple of 4)
 * apart. V <= 2^20, T <= 65536, B <= 4096. A logit of -inf is a token of
 * probability zero (so that a row's top k or top p alone are sampled where the
 * caller writes -inf elsewhere; draft_logits are those that the drafts were drawn
 * from). noise below 2^-126 (NaN too) counts as 2^-126.
 *
 * Whatever is compared is compared in fp32 where bounds on its error leave no doubt,
 * and else in 64 bits, the rows' sums included: the result is that of the definition in
 * 64-bit arithmetic, and depends on the arguments alone. (About one draft or race in
 * 10^5 needs better sums: 0.1 ms a row of 248320 logits, one in 10^6 1.3 ms. So does,
 * always, a temperature below 1.5e-30 or above 1e36.)
 *
 * These set MOE_ERR_DEVICE, where the definition reaches them: a NaN, a +inf or
 * nothing but -inf in a row of logits or draft logits, and a temperature that is
 * negative or not finite (the next token is then -1); a draft outside [0, V) (it is
 * refused, and takes nothing from p where draft_logits is NULL); offsets that do not
 * rise within [0, T], anywhere (nothing is accepted, and there is no next token: -1).
 * Rows of tokens that no sequence has are not written.
 *
 * ws: moe_verify_workspace_size() bytes under the rules of the MoE calls; it may
 * be one that they use.
 */
MOE_API int moe_verify_drafts(const uint16_t *logits, int64_t logits_stride, const uint16_t *draft_logits,
                      int64_t draft_stride, const int32_t *drafts, const int32_t *cu_rows, const float *temperature,
                      const float *uniform, const float *noise, int64_t noise_stride, int32_t B, int32_t T, int32_t V,
                      int32_t *tokens, int32_t *accepted, void *ws, size_t ws_bytes, void *stream);

/* Workspace bytes moe_verify_drafts needs for these dims. */
MOE_API int moe_verify_workspace_size(int32_t B, int32_t T, int32_t V, size_t *bytes);

/*
 * Which kernels a forward call of dims `d` runs (a host-only query, no
 * counterpart on the pages; for tests and tuning). Writes *plan = 0 for the
 * tensor-core pipeline (permute, grouped gate_up and down GEMMs, conversion);
 * otherwise the fused decode kernel runs and *plan = s + 16 * g + 256 * y + 512 * r,
 * where s = 1 if the activations are staged in shared memory and 2 if they
 * are read from global memory, g (at most 15) is the number of 128-wide
 * groups per gate_up chunk, and y = 1 if the down outputs' block buffers have
 * a shared-memory region of their own (0: they reuse the gate_up partial-sum
 * area once the CTA's gate_up work is done), and r = 1 if moe_layer_forward
 * runs the router inside the same kernel for these (forward) dims.
 * Returns the shape checks' status.
 */
MOE_API int moe_forward_plan(moe_dims d, int32_t *plan);

/*
 * Profiling aid (no counterpart on the pages): from now on, every forward
 * call records `before_experts` on its stream just before it launches the
 * expert kernel and `after_experts` just after it, so that the caller can
 * time that kernel alone with cudaEventElapsedTime. Both are cudaEvent_t
 * handles owned by the caller (created with timing enabled); while the stream
 * is being captured into a CUDA graph they become event-record nodes. Pass
 * NULL, NULL to stop. The setting is process-wide and not thread-safe.
 */
MOE_API int moe_profile_events(void *before_experts, void *after_experts);

/*
 * Synchronises `stream`, then reads and clears the workspace's error word.
 * Returns MOE_OK, MOE_ERR_DEVICE or MOE_ERR_TIMEOUT (or MOE_ERR_CUDA if the
 * synchronisation itself failed). On MOE_ERR_TIMEOUT it also sets all
 * ws_bytes of the workspace to zero (and waits for that), so that the
 * workspace is fit for the next call.
 */
MOE_API int moe_check_device_error(void *ws, size_t ws_bytes, void *stream);

/*
 * The same check for moe_w4a16_forward_noalloc (no counterpart on the pages):
 * synchronises `stream`, then reads and clears the error word of the
 * library's static scratch on the current device. Every no-alloc call clears
 * the word before it starts, so this reports on the last call only.
 */
MOE_API int moe_noalloc_check_device_error(void *stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A16MOE_H */
