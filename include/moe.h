/*
 * libmoe -- C ABI of the MoE expert-layer forward on one GPU (sm_103a).
 *
 * The layer:  out[t] = sum_{j<k} w[t,j] * FFN_{e[t,j]}(x[t]),
 *             FFN_e(x) = (silu(x W1[e]) * (x W3[e])) W2[e],
 * computed as four steps -- top-k gating, scatter into per-expert groups,
 * per-expert SwiGLU FFN, weighted return to token order -- following
 * "MegaScale-Infer: Serving Mixture-of-Experts at Scale with Disaggregated
 * Expert Parallelism" (§3.2 Big-Picture Architecture, steps (1)-(5);
 * §3.4 Supporting Implementation Details, Fused Kernels, steps (1)-(4)),
 * "MegaFlux: Skew-Resilient MoE Megakernels via Pipelined Expert
 * Replication" (§2.1, §3.1, §A.2) and "Piper: Efficient Large-Scale MoE
 * Training via Resource Modeling and Pipelined Hybrid Parallelism"
 * (§III-A, Table III).
 *
 * Conventions shared by every entry point
 *   - Tensor pointers are DEVICE pointers owned by the caller, row-major and
 *     contiguous, 16-byte aligned.  bf16 tensors are passed as void* and
 *     hold IEEE bfloat16 (__nv_bfloat16) values.  The library never
 *     allocates, frees or keeps a reference to caller memory beyond a call.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Every
 *     call only enqueues work on `stream` and returns; nothing synchronises
 *     except moe_get_device_status.
 *   - `ws` is a caller-owned device workspace of at least
 *     moe_workspace_size(T, H, F, E, k) bytes, 256-byte aligned.  It holds
 *     the intermediates (gathered rows, expert activations and outputs),
 *     8 to 32 MiB of partial tiles for the balanced K split of FC2, the
 *     head of the grouped GEMM's tile queue, and a device status word.  Its
 *     contents need no initialisation (each layer call clears the counters).  Calls that
 *     share one workspace must not overlap in time (use one stream per
 *     workspace).
 *   - Limits: 0 <= T, T*k < 2^31; 1 <= E <= MOE_MAX_EXPERTS;
 *     1 <= k <= min(E, MOE_MAX_TOPK); H and F positive multiples of 128.
 *     Violations are reported synchronously as MOE_ERR_INVALID_ARG and
 *     nothing is enqueued.  T == 0 is a valid no-op.
 *   - Conditions only the device can see (a non-finite router logit, a
 *     pipeline wait that ran out) are written to the status word in `ws`
 *     and read back with moe_get_device_status; the kernels never trap.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_TOPK 32

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,  /* bad size, null or misaligned pointer       */
  MOE_ERR_NONFINITE = 2,    /* a router logit is NaN or +-inf, a balance bias NaN
                             or +inf, or an adapter weight or an optimizer's
                             gradient either (device)                     */
  MOE_ERR_TIMEOUT = 3,      /* a bounded device wait ran out (device)     */
  MOE_ERR_WORKSPACE = 4,    /* ws is NULL, too small or misaligned        */
  MOE_ERR_CUDA = 5,         /* a CUDA runtime call or launch failed       */
  MOE_ERR_UNSUPPORTED = 6   /* no sm_103a device is current               */
} moe_status;

/* Bytes of workspace needed for a layer of these sizes (0 on bad sizes). */
size_t moe_workspace_size(int T, int H, int F, int E, int k);

/*
 * Step 1 -- top-k gating and weight normalisation
 * ("MegaScale-Infer", §3.4 Fused Kernels, steps (1) and (3)).
 *
 *   logits   [T, E] fp32 router output.
 *   topk_idx [T, k] int32 out: slot j is the j-th largest logit of the token;
 *            equal logits (also -0.0 vs +0.0) go to the lower expert index.
 *   topk_w   [T, k] fp32 out: softmax over the k selected logits (they sum
 *            to 1).
 * A NaN or infinite logit sets MOE_ERR_NONFINITE in the device status; the
 * outputs of that token are then unspecified.
 */
moe_status moe_route_topk(const float* logits, int T, int E, int k,
                          int32_t* topk_idx, float* topk_w,
                          void* ws, size_t ws_bytes, void* stream);

/*
 * Step 1 with scores: routing by softmax or sigmoid scores, a balance bias,
 * groups of experts and optional renormalisation.  Per token t:
 *
 *   s_e = 1 / (1 + exp(-l_e))  or  exp(l_e - max l) / sum_i exp(l_i - max l);
 *   rank by r_e = s_e + bias_e, or by the logit l_e when `bias` is null;
 *   n_group > 1: the E experts form n_group groups of E / n_group consecutive
 *     ones; a group is worth its largest r (group_top 1) or the sum of the two
 *     largest s + bias in it (group_top 2); experts outside the topk_group
 *     best groups are no candidates;
 *   topk_idx[t, :] are the k best candidates in descending r; ties, of
 *     experts and of groups, go to the lower index;
 *   topk_w[t, j] = scale * s_j, or scale * s_j / sum_i s_i over the chosen
 *     experts when `renormalize`.  The bias never enters a weight.
 *
 * The choice is made in fp32, each operation rounded to nearest (the softmax's
 * sum rounded once); with softmax scores, no bias, one group and renormalize
 * it is moe_route_topk.  Weights are within 2^-24 (16 + 2 max |l_e - max l|) of
 * themselves; renormalised ones are ratios, kept where every score underflows.
 *
 *   logits [T, E] fp32, finite; bias [E] fp32 or null, finite or -inf.  -inf
 *     switches an expert off: it is chosen only where the candidates that are
 *     on do not fill the k slots, and then has weight 0 (a row with no expert
 *     on has all weights 0).
 *   topk_idx [T, k] int32, topk_w [T, k] fp32 out.  ws: 256 bytes.
 * Limits: 1 <= n_group <= MOE_MAX_GROUPS, a divisor of E; 1 <= topk_group <=
 * n_group; topk_group * (E / n_group) >= k; group_top 1, or 2 with at least two
 * experts per group; scale finite.  A logit that is not finite, or a bias that
 * is NaN or +inf, sets MOE_ERR_NONFINITE in the device status; the indices of
 * that token are then distinct and in range, its weights unspecified.
 *
 * moe_route_scored_backward: dlogits [T, E] fp32 = the gradient of the
 * weights, given dtopk_w [T, k] = dL/dtopk_w and the topk_idx, logits, bias and
 * config of the forward.  The choice is a constant: experts that were not
 * chosen get 0, but for softmax scores that are not renormalised, whose sum
 * runs over all experts.  A slot whose index is outside [0, E) is skipped and
 * sets MOE_ERR_INVALID_ARG in the device status; the indices of a token are
 * otherwise distinct, as the forward writes them.  A non-finite logit that is
 * read sets MOE_ERR_NONFINITE.  The bias has no gradient.
 */
#define MOE_MAX_GROUPS 32
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;
typedef struct {
  int32_t score;        /* moe_score                                          */
  int32_t n_group;      /* 1: no groups                                       */
  int32_t topk_group;   /* groups whose experts are candidates                */
  int32_t group_top;    /* 1: a group's best expert; 2: the sum of its two best */
  int32_t renormalize;  /* weights divided by the sum of the chosen scores    */
  float scale;          /* factor on every weight                             */
} moe_route_config;
moe_status moe_route_scored(const float* logits, const float* bias,
                            const moe_route_config* config, int T, int E, int k,
                            int32_t* topk_idx, float* topk_w,
                            void* ws, size_t ws_bytes, void* stream);
moe_status moe_route_scored_backward(const float* dtopk_w, const int32_t* topk_idx,
                                     const float* logits, const float* bias,
                                     const moe_route_config* config, int T, int E, int k,
                                     float* dlogits, void* ws, size_t ws_bytes, void* stream);

/*
 * Step 2 -- per-expert counts and the stable scatter into expert groups
 * ("MegaScale-Infer", §3.4 Fused Kernels, steps (2) and (4); order inside an
 * expert by token, then top-k position: "MegaFlux", §A.2).
 *
 * Assignment a = t*k + j.
 *   topk_idx   [T, k] int32 in, values in [0, E).
 *   counts     [E]    int32 out: assignments per expert (sum = T*k).
 *   offsets    [E+1]  int32 out: exclusive prefix sum of counts.
 *   sorted_src [T*k]  int32 out: sorted_src[p] = a, p ascending within each
 *              expert's range [offsets[e], offsets[e+1]) in ascending a.
 *   dest_of    [T*k]  int32 out: inverse map, sorted_src[dest_of[a]] == a.
 * Deterministic: bit-identical on every run.  An expert index outside
 * [0, E) sets MOE_ERR_INVALID_ARG in the device status; that assignment is
 * left out of the counts and takes no position: its dest_of is -1, and
 * sorted_src[offsets[E] .. T*k) holds -1.  The other assignments are grouped
 * as above.  moe_grouped_ffn and moe_combine skip positions and slots marked
 * -1, so a bad index never turns into a memory access.
 */
moe_status moe_permute(const int32_t* topk_idx, int T, int E, int k,
                       int32_t* counts, int32_t* offsets,
                       int32_t* sorted_src, int32_t* dest_of,
                       void* ws, size_t ws_bytes, void* stream);

/*
 * Step 3 -- per-expert SwiGLU FFN as a grouped GEMM over the expert groups
 * ("Piper", §III-A: W_gate, W_up in R^{d x dffn}, W_down in R^{dffn x d};
 * "MegaScale-Infer", §3.4 Performance Simulation Model: FFN Input and FFN
 * Output GEMMs; token blocks of at most beta rows per expert: "MegaFlux",
 * §3.1).  beta is 64, 128 or 256 rows, chosen from the mean rows per expert
 * (T*k/E at most 40, at most 80, above); an expert's rows are cut into
 * ceil(rows / beta) blocks of equal size (a multiple of 16 rows), so no block
 * is a near-empty tail.  The groups are unpadded: nothing is stored for rows
 * past offsets[E].
 *
 *   x          [T, H] bf16.
 *   sorted_src [T*k], offsets [E+1] as produced by moe_permute (positions
 *              holding -1 are skipped).  offsets that do not group T*k rows
 *              (offsets[0] != 0, a decrease, offsets[E] > T*k) set
 *              MOE_ERR_INVALID_ARG in the device status and nothing is
 *              computed.
 *   W1, W3     [E, H, F] bf16: gate (silu applied) and up projections.
 *   W2         [E, F, H] bf16: down projection.
 *   y_sorted   [T*k, H] bf16 out: y_sorted[p] = FFN_e(x[sorted_src[p]/k])
 *              for p in expert e's range.
 * bf16 operands, fp32 accumulation, SwiGLU applied to the fp32 accumulators;
 * the intermediate h = silu(g)*u is stored in bf16.
 */
moe_status moe_grouped_ffn(const void* x, const int32_t* sorted_src,
                           const int32_t* offsets,
                           const void* W1, const void* W3, const void* W2,
                           int T, int H, int F, int E, int k,
                           void* y_sorted, void* ws, size_t ws_bytes, void* stream);

/*
 * Step 4 -- weighted return to token order
 * ("MegaFlux", §2.1 final top-k sum; "MegaScale-Infer", §3.2 step (4)).
 *
 *   out[t] = sum_{j<k} topk_w[t,j] * y_sorted[dest_of[t*k+j]], summed in
 *   slot order in fp32 and rounded once to bf16.
 *   y_sorted [T*k, H] bf16, dest_of [T*k] int32, topk_w [T, k] fp32,
 *   out [T, H] bf16 out.  No workspace.  A slot whose dest_of is outside
 *   [0, T*k) (-1 from moe_permute for an out-of-range expert index) adds
 *   nothing.
 */
moe_status moe_combine(const void* y_sorted, const int32_t* dest_of,
                       const float* topk_w, int T, int H, int k,
                       void* out, void* stream);

/*
 * moe_permute for callers that cannot allocate device memory.  The pages
 * have no counterpart to this entry point; it exists for how the library is
 * called, not for what the layer computes.
 *
 * Who needs it: code whose device memory is wholly owned by another
 * allocator (a serving engine or host framework that reserves the GPU's
 * memory up front and hands out no extra buffers), and code on a hot path
 * that must not take cudaMalloc's implicit device synchronisation.  Such a
 * caller cannot provide the workspace moe_permute needs, so this variant
 * takes none and performs no allocation of any kind (no cudaMalloc, no
 * cudaFree, no allocating library routine).
 *
 * Arguments, outputs and ordering are those of moe_permute.  Its scratch
 * (per-chunk histograms, the token-block plan, a status word) is a fixed
 * device array of MOE_PERMUTE_NOALLOC_SCRATCH_BYTES inside the library;
 * every GPU on which the library's device code is loaded holds that array
 * until the process exits.  Sizes whose scratch would not fit return
 * MOE_ERR_WORKSPACE and enqueue nothing; they fit while
 *   4 * (64 + C*E + (E+1) + 64 + NB) <= MOE_PERMUTE_NOALLOC_SCRATCH_BYTES
 * (each term rounded up to 64), with C = ceil(T / floor(512 / k)) chunks
 * and NB = ceil(T*k / 128) + min(T*k, E) token blocks -- for example
 * T = 8192, k = 8, E = 256 needs about 136 KB.
 *
 * The first call in each CUDA context looks up the array's device address
 * (cudaGetSymbolAddress) with that context current, and caches it under the
 * context's ID; make that first call before any stream capture begins.  A
 * device reset (or a new context on the same device) loads the library's
 * device code afresh, at an address of its own: the next call sees a new
 * context ID and looks the address up again, so it never uses a stale one.
 * Every call shares the one array and it keeps the previous call's contents
 * (the status word is cleared by each call), so calls whose work overlaps on
 * the GPU -- on different streams, or from different threads -- race and
 * corrupt each other's results; serialise them.  Out-of-range expert indices
 * get the same -1 markers as in moe_permute (so the gather and the combine
 * skip them) but, unlike moe_permute, cannot be read back as a device status.
 */
#define MOE_PERMUTE_NOALLOC_SCRATCH_BYTES (1u << 20)
moe_status moe_permute_noalloc(const int32_t* topk_idx, int T, int E, int k,
                               int32_t* counts, int32_t* offsets,
                               int32_t* sorted_src, int32_t* dest_of,
                               void* stream);

/*
 * The whole layer: steps 1-4 on `stream`, intermediates in `ws`.
 *   x [T, H] bf16, router_logits [T, E] fp32, W1/W3 [E, H, F] bf16,
 *   W2 [E, F, H] bf16, out [T, H] bf16.
 * The device status word is cleared at the start of the call.
 */
moe_status moe_forward(const void* x, const float* router_logits,
                       const void* W1, const void* W3, const void* W2,
                       int T, int H, int F, int E, int k, void* out,
                       void* ws, size_t ws_bytes, void* stream);

/*
 * moe_forward, with moe_route_scored in the place of step 1: the same
 * arguments, workspace and status, and the router's bias (or null) and
 * configuration.
 */
moe_status moe_forward_scored(const void* x, const float* router_logits, const float* bias,
                              const moe_route_config* config,
                              const void* W1, const void* W3, const void* W2,
                              int T, int H, int F, int E, int k, void* out,
                              void* ws, size_t ws_bytes, void* stream);

/*
 * moe_forward captured once into a CUDA graph, for small batches whose
 * kernels are as short as the host's launches (measured: a 256-token,
 * 8-expert layer 42.6 -> 36.1 us per step, a 128-token decode layer 0.717 ->
 * 0.707 ms; large layers run slower from a graph, e.g. a 4096-token, 16-expert
 * prefill chunk 3.82 -> 4.08 ms).  moe_forward_graph_create records one
 * moe_forward with exactly these arguments on `stream` (a non-default
 * stream, not capturing; only the calling thread's work is recorded) and
 * instantiates it; nothing runs.
 * moe_graph_launch enqueues the whole layer on `stream`: it reads x and
 * router_logits and writes out, ws as they are at that time (same pointers,
 * same sizes, same weights), so a caller refills x and router_logits in place
 * between launches.  The graph holds no reference to the buffers: they must
 * outlive every launch.  Launches on one workspace must not overlap (order
 * them on one stream).  The handle is the caller's until moe_graph_destroy,
 * which waits for nothing: destroy only after the last launch has completed.
 * Errors: MOE_ERR_INVALID_ARG (as moe_forward; also a null stream or handle
 * pointer, a stream already capturing, T == 0), MOE_ERR_WORKSPACE,
 * MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA (capture or instantiation failed);
 * *graph is null on any error.
 */
typedef struct moe_graph_s* moe_graph;
moe_status moe_forward_graph_create(const void* x, const float* router_logits,
                                    const void* W1, const void* W3, const void* W2,
                                    int T, int H, int F, int E, int k, void* out,
                                    void* ws, size_t ws_bytes, void* stream,
                                    moe_graph* graph);
moe_status moe_graph_launch(moe_graph graph, void* stream);
moe_status moe_graph_destroy(moe_graph graph);

/*
 * moe_forward with the combine's fp32 sum left unrounded: out [T, H] fp32.
 * For a layer split over GPUs along the FFN features ("MegaScale-Infer",
 * §3.4 Performance Simulation Model: expert tensor parallelism, tpe), where
 * each GPU holds W1[:, :, Fg], W3[:, :, Fg] and W2[:, Fg, :] for its slice
 * Fg of the features, routes every token identically and computes this
 * partial output; the sum of the partials over the GPUs (one all-reduce or
 * reduce-scatter, in fp32) is the layer, since SwiGLU acts feature by
 * feature and the combine is linear.  Same arguments, workspace and status
 * as moe_forward; F is the slice's width (a multiple of 128).
 */
moe_status moe_forward_f32(const void* x, const float* router_logits,
                           const void* W1, const void* W3, const void* W2,
                           int T, int H, int F, int E, int k, float* out,
                           void* ws, size_t ws_bytes, void* stream);

/*
 * The routing a moe_forward (or moe_forward_f32 / moe_forward_host /
 * moe_forward_train) call on `ws` with these sizes computed: copies the
 * layer's own topk_idx [T, k], topk_w [T, k], counts [E], offsets [E+1],
 * sorted_src [T*k] and dest_of [T*k] (layouts as in moe_route_topk and
 * moe_permute) out of the workspace, stream-ordered after that call, for
 * inspecting and testing the fused path.
 */
moe_status moe_forward_routing(const void* ws, size_t ws_bytes, int T, int H, int F, int E,
                               int k, int32_t* topk_idx, float* topk_w, int32_t* counts,
                               int32_t* offsets, int32_t* sorted_src, int32_t* dest_of,
                               void* stream);

/* out[i] = bf16(in[i]) for i < n, round to nearest even: the layer's output
 * from the reduced fp32 partials of moe_forward_f32.  in fp32 [n], out bf16
 * [n], both 16-byte aligned device pointers; no workspace. */
moe_status moe_cast_bf16(const float* in, void* out, size_t n, void* stream);

/*
 * The whole layer with the per-step activations in HOST memory: takes
 * x_host [T, H] bf16 and logits_host [T, E] fp32, runs moe_forward and
 * returns the result in out_host [T, H] bf16.  The weights are device
 * pointers (resident model parameters).  A host buffer that is page-locked
 * and mapped into the device's address space (cudaHostAlloc, cudaHostRegister,
 * or a framework's pinned allocation) is used in place: the kernels read x and
 * the logits and write the result across the host-device link, each element
 * once, with no staging copy.  Any other host buffer is copied through a staging region of
 * `ws` (moe_workspace_size covers it) with cudaMemcpyAsync.  out_host is
 * valid once `stream` has been synchronised.
 */
moe_status moe_forward_host(const void* x_host, const float* logits_host,
                            const void* W1, const void* W3, const void* W2,
                            int T, int H, int F, int E, int k, void* out_host,
                            void* ws, size_t ws_bytes, void* stream);

/*
 * The steps either side of the routed path.
 *
 * Router projection ("MegaScale-Infer" §3.2, item 2: the gating network
 * decides each token's experts; "Piper" §II-A: a learned gating function):
 *   logits[T, E] fp32 = x[T, H] bf16 @ Wg[H, E] bf16, fp32 accumulation,
 *   no bias.  E < 64: any E; E >= 64: E a multiple of 8.  H a multiple of
 *   128.  ws: at least 512 + 4 * (ceil(T/128) + 2) bytes (256-byte aligned);
 *   moe_workspace_size_gated covers it.
 */
moe_status moe_router_logits(const void* x, const void* Wg, int T, int H, int E,
                             float* logits, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes for moe_forward_gated (Fs = 0 when there is no shared
 * expert); 0 on bad sizes. */
size_t moe_workspace_size_gated(int T, int H, int F, int Fs, int E, int k);

/*
 * The layer from hidden states: router projection, then moe_forward's four
 * steps, plus an optional always-active shared expert ("Piper", Table I:
 * "R + S" = routed + shared experts per token) applied to every token and
 * added with weight one after the routed slots:
 *   out[t] = sum_j w[t,j] FFN_{e[t,j]}(x[t]) + FFN_s(x[t]).
 *   Wg [H, E] bf16; W1/W3 [E, H, F], W2 [E, F, H] bf16;
 *   Ws1/Ws3 [H, Fs], Ws2 [Fs, H] bf16, all three NULL for no shared expert;
 *   Fs a multiple of 128 when present.  Routing is decided on the fp32
 *   router logits.  ws: moe_workspace_size_gated bytes.
 */
moe_status moe_forward_gated(const void* x, const void* Wg,
                             const void* W1, const void* W3, const void* W2,
                             const void* Ws1, const void* Ws3, const void* Ws2,
                             int T, int H, int F, int Fs, int E, int k, void* out,
                             void* ws, size_t ws_bytes, void* stream);

/*
 * Low-rank adapters of many requests at once beside a projection that all of
 * them share (either side of the layer: an attention or shared-expert
 * projection served for many fine-tuned variants).  With a = adapter_idx[t]:
 *
 *   y[t] = x[t] W + scale[a] * (x[t] A[a]^T) B[a]      (a = -1: y[t] = x[t] W)
 *
 *   x [T, H], W [H, N], y [T, N] bf16;
 *   A [n, R, H] bf16, the adapters' down projections, one row per rank;
 *   B [n, R, N] bf16, their up projections;
 *   scale [n] fp32; adapter_idx [T] int32, -1 or 0 .. n - 1 in any order.
 * A smaller rank is padded with zero rows.  bf16 operands, fp32 accumulation;
 * the scaled low-rank activation is rounded to bf16 once (it is a matrix
 * operand), y is rounded once.  Any other index in adapter_idx counts as -1
 * and sets MOE_ERR_INVALID_ARG in the device status.  T == 1 is the form for a
 * single token.
 *
 * The backward, given dy [T, N] bf16 = dL/dy and W frozen:
 *   dx [T, H] bf16 = dy W^T + dz A,   dz[t] = scale[a] * (dy[t] B[a]^T)
 *   dA [n, R, H] bf16: dA[a] = sum over its tokens of dz[t]^T x[t]
 *   dB [n, R, N] bf16: dB[a] = sum of z[t]^T dy[t], z[t] = scale[a] * (x[t] A[a]^T)
 * with exact zeros for adapters without a token.  Sums run in a fixed order.
 *
 * Requests do not see each other's infinities and NaN: a token or an adapter
 * that holds one spoils its own results only.  Where the weights enter the
 * product that a whole block of tokens shares -- B in y, A in dx -- such a
 * weight counts as zero and sets MOE_ERR_NONFINITE in the device status.
 *
 * ws: moe_adapter_workspace_size bytes (.._backward for the backward, which
 * covers both): about T * min(n, 256) * R * 2 for the low-rank activations,
 * which are kept with R columns for every adapter that a block of up to 256
 * tokens can meet, twice in the backward (8192 tokens, 1024 adapters of rank
 * 128: 0.54 and 1.07 GB).  It grows with T, so a workspace for the largest batch
 * serves smaller ones.  Limits: H and N positive multiples of 128, T < 2^30,
 * 1 <= n <= MOE_MAX_ADAPTERS, R a multiple of 8 up to MOE_MAX_RANK.
 */
#define MOE_MAX_ADAPTERS 1024
#define MOE_MAX_RANK 128
size_t moe_adapter_workspace_size(int T, int H, int N, int n, int R);
size_t moe_adapter_workspace_size_backward(int T, int H, int N, int n, int R);
moe_status moe_adapter_project(const void* x, const void* W, const void* A, const void* B,
                               const float* scale, const int32_t* adapter_idx,
                               int T, int H, int N, int n, int R, void* y,
                               void* ws, size_t ws_bytes, void* stream);
moe_status moe_adapter_project_backward(const void* dy, const void* x, const void* W,
                                        const void* A, const void* B, const float* scale,
                                        const int32_t* adapter_idx,
                                        int T, int H, int N, int n, int R,
                                        void* dx, void* dA, void* dB,
                                        void* ws, size_t ws_bytes, void* stream);

/*
 * Training: the layer's backward ("MegaFlux" §2.1 and §3.2: the backward
 * streams token blocks through DGrad and WGrad grouped GEMMs; the final
 * top-k sum's gradient gives each routing weight's gradient).
 *
 * moe_forward_train is moe_forward that also keeps, in `ws`, what the
 * backward needs (routing, gathered x rows, the gate and up pre-activations
 * g = x W1 and u = x W3 in bf16, h and the expert outputs); ws must hold
 * moe_workspace_size_train bytes.  moe_backward then takes dout = dL/dout
 * [T, H] bf16 and the same logits and weights, and writes
 *   dx      [T, H] bf16,
 *   dlogits [T, E] fp32 (softmax Jacobian over the k selected logits;
 *           zero for unselected experts),
 *   dW1, dW3 [E, H, F] bf16, dW2 [E, F, H] bf16 (fp32 accumulation; zero
 *           for experts that received no token, and so all of it when
 *           T == 0, where null pointers are left alone).
 * The two calls must use the same ws, sizes, logits and weights, with no
 * other call on that ws in between; moe_backward leaves the saved state
 * intact, so it may be repeated (e.g. for another dout).
 */
size_t moe_workspace_size_train(int T, int H, int F, int E, int k);
moe_status moe_forward_train(const void* x, const float* router_logits,
                             const void* W1, const void* W3, const void* W2,
                             int T, int H, int F, int E, int k, void* out,
                             void* ws, size_t ws_bytes, void* stream);
moe_status moe_backward(const void* dout, const float* router_logits,
                        const void* W1, const void* W3, const void* W2,
                        int T, int H, int F, int E, int k,
                        void* dx, float* dlogits, void* dW1, void* dW3, void* dW2,
                        void* ws, size_t ws_bytes, void* stream);

/*
 * moe_forward_train and moe_backward with moe_route_scored in the place of
 * step 1: bias and config as there, the same in both calls.  dlogits is
 * moe_route_scored_backward's.
 */
moe_status moe_forward_scored_train(const void* x, const float* router_logits, const float* bias,
                                    const moe_route_config* config,
                                    const void* W1, const void* W3, const void* W2,
                                    int T, int H, int F, int E, int k, void* out,
                                    void* ws, size_t ws_bytes, void* stream);
moe_status moe_backward_scored(const void* dout, const float* router_logits, const float* bias,
                               const moe_route_config* config,
                               const void* W1, const void* W3, const void* W2,
                               int T, int H, int F, int E, int k,
                               void* dx, float* dlogits, void* dW1, void* dW3, void* dW2,
                               void* ws, size_t ws_bytes, void* stream);

/*
 * What a training step runs around the layer.
 *
 * Layer norm, ahead of the router and the experts, with the residual add:
 *   h[t] = x[t] + residual[t], rounded to the tensors' type; x itself without
 *          a residual
 *   mean, rstd = 1 / sqrt(var + eps) over the H values of h[t], var their
 *          variance around the mean (divided by H)
 *   y[t] = (h[t] - mean) * rstd * weight + bias
 * x, residual, h, y [T, H] of `type`; weight, bias [H] of `weight_type`; stats
 * [T, 2] fp32 out: mean and rstd of each token.  bias, residual and stats may
 * be null; h is written where there is a residual, and null otherwise.  x or
 * residual may be h (the sum takes its place), and x may be y where there is
 * no residual.
 *
 * The backward, given dy = dL/dy and, where the sum is used past the norm too,
 * dh = dL/dh [T, H] (or null):
 *   dx[t] = rstd (w dy - mean(w dy) - xhat mean(w dy xhat)) + dh[t],
 *           xhat = (h[t] - mean) rstd: the gradient of x and of the residual
 *   dweight = sum_t dy xhat,  dbias = sum_t dy   (dbias may be null)
 * dx of `type`, dweight and dbias of `weight_type`.  dx may be dy or dh.  With
 * T == 0 dweight and dbias are zero.
 *
 * Statistics and sums are fp32 in a fixed order, which goes by the sizes and,
 * where H is no multiple of 8, by the place of a row between 16-byte boundaries;
 * every output is rounded once.  The backward sets the device status of ws.
 * A NaN or infinity spoils its own token, and what is summed over tokens.
 * type: MOE_BF16 or MOE_F32; weight_type: MOE_F32, or MOE_BF16 beside bf16
 * tensors.  eps > 0, finite.  1 <= H <= MOE_MAX_NORM_WIDTH; any H is taken,
 * multiples of 8 by wide accesses.  ws (backward):
 * moe_layer_norm_workspace_size bytes; the forward takes none.
 */
typedef enum { MOE_BF16 = 0, MOE_F32 = 1 } moe_dtype;
#define MOE_MAX_NORM_WIDTH 16384
moe_status moe_layer_norm(const void* x, const void* residual, const void* weight,
                          const void* bias, float eps, int T, int H, int type, int weight_type,
                          void* y, void* h, float* stats, void* stream);
size_t moe_layer_norm_workspace_size(int T, int H);
moe_status moe_layer_norm_backward(const void* dy, const void* h, const float* stats,
                                   const void* weight, const void* dh, int T, int H, int type,
                                   int weight_type, void* dx, void* dweight, void* dbias,
                                   void* ws, size_t ws_bytes, void* stream);

/*
 * The loss that keeps the experts' loads even, and the loads.  The batch holds
 * S sequences one after the other, tokens seq_offsets[s] .. seq_offsets[s + 1]
 * - 1 each; a token counts where its mask is not zero.  With n_s counted
 * tokens in sequence s and c_se of their choices (topk_idx) expert e:
 *
 *   p_t = softmax(l_t), or sigmoid(l_t) / sum_i sigmoid(l_ti)
 *   loss = alpha / S * sum_s sum_e (E c_se / (k n_s)) (sum_t p_te / n_s)
 *
 * (alpha where the loads are even); a sequence in which no token counts adds
 * nothing.  The choices are constants:
 *
 *   dlogits_te = dloss * alpha E / (S k n_s^2) * p_te f_te (c_se - sum_i p_ti c_si)
 *
 * with f = 1 for softmax and 1 - sigmoid(l_te) for sigmoid.  Tokens that are
 * masked, or ahead of the first or behind the last sequence, have gradient zero.
 *
 *   logits [T, E] fp32; topk_idx [T, k] int32, of any routing;
 *   score: moe_score;
 *   seq_offsets [S + 1] int32, ascending, within 0 .. T; null (then S == 1):
 *     all tokens are one sequence;
 *   mask [T] bytes, or null: every token counts;
 *   loss [1] fp32, counts [S, E] int32, tokens [S] int32 (n_s) out.
 * moe_balance_loss_backward takes counts and tokens as the forward wrote them,
 * and dloss [1] fp32 on the device (null: 1; 4-byte aligned).  `accumulate`: the gradient is
 * added onto dlogits [T, E] fp32 (onto the layer's own, say), and rows with
 * gradient zero are left as they were; otherwise all of dlogits is written.
 *
 * Sums are fp32 in a fixed order: results are the same from run to run.  Where
 * the loads are even the gradient is exactly zero.  The forward reports in the
 * device status: a logit of a counted token that is not finite
 * (MOE_ERR_NONFINITE; loss and that row's gradient are then unspecified), a
 * choice outside [0, E) or offsets that do not ascend within 0 .. T
 * (MOE_ERR_INVALID_ARG; such a choice is not counted).  Masked tokens' logits
 * and choices are not looked at.  ws (forward): moe_balance_workspace_size
 * bytes, about 8 E for each sequence and each block of up to T / 304 tokens; the
 * backward takes none.  Limits: 1 <= S <= MOE_MAX_SEQUENCES, alpha
 * and alpha E / (S k) finite in fp32.
 */
#define MOE_MAX_SEQUENCES 65536
size_t moe_balance_workspace_size(int T, int E, int S);
moe_status moe_balance_loss(const float* logits, const int32_t* topk_idx, int score, float alpha,
                            const int32_t* seq_offsets, const uint8_t* mask, int T, int E, int k,
                            int S, float* loss, int32_t* counts, int32_t* tokens,
                            void* ws, size_t ws_bytes, void* stream);
moe_status moe_balance_loss_backward(const float* dloss, const int32_t* counts,
                                     const int32_t* tokens, const float* logits, int score,
                                     float alpha, const int32_t* seq_offsets, const uint8_t* mask,
                                     int T, int E, int k, int S, int accumulate, float* dlogits,
                                     void* stream);

/*
 * One AdamW step over many tensors, in place.  For each element, at step t:
 *
 *   g' = grad_scale g
 *   m = beta1 m + (1 - beta1) g',  v = beta2 v + (1 - beta2) g'^2
 *   p = p (1 - lr weight_decay decay)
 *       - lr / (1 - beta1^t) * m / (sqrt(v / (1 - beta2^t)) + eps)
 *
 * p is the fp32 master weight where there are masters, and the parameter its
 * rounding to bf16; otherwise the parameter itself, rounded once.  Arithmetic
 * is fp32.
 *
 * The tensors (param, and grads[i] of tensor i: device pointers, each to n values
 * one after the other) are listed in host memory, which may be reused after the
 * call.  Their moments and masters lie in arrays that all of them share, tensor i at
 * elements start .. start + n - 1, start a multiple of MOE_ADAMW_BLOCK, so that
 * no block of that many elements belongs to two tensors:
 *   master         fp32, or null;
 *   exp_avg        m, fp32 or e4m3 values (state_bits 32 or 8);
 *   exp_avg_sq     v in fp32, or its square root in e4m3;
 *   exp_avg_scale, exp_avg_sq_scale   (8 bits) fp32 [one per block]: what the
 *                  block's e4m3 values are multiplied by.
 * A block's scale is its largest magnitude times fl(1 / 448) (0 where that is
 * below the normal fp32 range: the block is then zero), and a value is rounded to the
 * nearest e4m3 one; the step itself uses m and v before that rounding.  A root
 * that is held as zero (below 2^-10 scale) counts as 2^-11 scale in the next
 * step, so that an element whose gradient is zero then does not move by what is
 * left of its first moment over eps.  8-bit
 * arrays hold whole blocks, zero past a tensor's end.  State arrays that are
 * zero are those of step 0.
 *
 * step: the number t of this step (1 for the first); or step_at, device int64,
 * read when the step runs (so that a captured step can count; below 1 it counts
 * as 1), where not null.
 * lr_at: device fp32, in the place of config->lr where not null.  grad_scale:
 * device fp32, 1 where null (a clipping or unscaling factor).
 *
 * An element whose moments would not be finite (a gradient that is NaN or
 * infinite, or too large to be squared) is left as it was, and
 * MOE_ERR_NONFINITE is set in the device status.  (8 bits: its moments are held
 * in the units of its block, and rounded again where these change.)  With a
 * grad_scale that is not finite the whole step is skipped, and nothing but the
 * status is written.
 *
 * param_type, grad_type: moe_dtype, of all tensors of the call; masters only
 * beside bf16 parameters.  Tensors and scales are 16-byte aligned, the other
 * state arrays 32-byte.  No tensor may appear twice.
 * 0 <= beta < 1, eps a normal fp32 number, lr, weight_decay, decay and
 * weight_decay * decay finite in fp32, step >= 1 (with step_at it is not looked
 * at).  ws: 256 bytes.
 */
#define MOE_ADAMW_BLOCK 256
typedef struct {
  void* param;
  int64_t n;        /* elements                                             */
  int64_t start;    /* first element in the state arrays                    */
  double decay;     /* factor on the weight decay (0: none, 1: the config's) */
} moe_adamw_tensor;
typedef struct {
  double lr, beta1, beta2, eps, weight_decay;
  int32_t state_bits;   /* 32 or 8 */
} moe_adamw_config;
moe_status moe_adamw_step(const moe_adamw_tensor* tensors, const void* const* grads, int count,
                          int param_type, int grad_type, const moe_adamw_config* config, int64_t step,
                          const int64_t* step_at, const float* lr_at, const float* grad_scale,
                          float* master, void* exp_avg, void* exp_avg_sq, float* exp_avg_scale,
                          float* exp_avg_sq_scale, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_forward with timing marks: records events[0] on `stream` before the
 * first kernel and events[i] after stage i, for the MOE_FORWARD_STAGES
 * stages route, scan, scatter, gather, fc1, fc2, combine (in that order; the
 * gather stage is empty when the token blocks are small -- T*k <= 40 E -- and
 * FC1 gathers the rows of x it needs itself; the scan and scatter stages are
 * empty for small batches -- T*k <= 1024 and E <= 256 -- where one kernel
 * routes, counts, scans and scatters).
 * `events` points to MOE_FORWARD_STAGES + 1 cudaEvent_t created by the
 * caller.  Same arguments, work and results as moe_forward.
 */
#define MOE_FORWARD_STAGES 7
moe_status moe_forward_events(const void* x, const float* router_logits,
                              const void* W1, const void* W3, const void* W2,
                              int T, int H, int F, int E, int k, void* out,
                              void* ws, size_t ws_bytes, void* const* events,
                              void* stream);

/* Name of timing stage i of moe_forward_events (NULL if out of range). */
const char* moe_forward_stage_name(int i);

/*
 * Expert-replica planning for expert-parallel execution on G GPUs
 * ("MegaFlux: Skew-Resilient MoE Megakernels via Pipelined Expert
 * Replication", §3.1 Planner: replica placement and token-block assignment;
 * §A.1 Greedy placement and refinement; §A.2 Reduction-aware planning).
 * Runs on the device, from the per-expert row counts of a routing (e.g. the
 * `counts` of moe_permute), so no host round trip sits between routing and
 * the plan; it changes no routed assignment, only which GPU computes which
 * token blocks of an expert.
 *
 * GPU g owns experts [ceil(g E / G), ceil((g+1) E / G)), i.e. expert e is owned
 * by floor(e G / E).  Each expert's rows are cut into ceil(c_e / beta) blocks
 * (the last one partial); block counts are the load.  Starting from the
 * no-replica plan, four bounded greedy searches move blocks from GPUs above
 * tau = ceil(total blocks / G) to GPUs below it that hold the expert, or to a
 * new replica there (at most `budget` replicas per GPU), for at most s + 2
 * rounds (s = `rounds`, or the budget when `rounds` is -1); the plan with the
 * smallest maximum load (then fewest replicas) is refined -- redundant
 * replicas pruned, single blocks moved between holders of an expert -- and,
 * when lambda >= 0 (backward plans, lambda = 12 in the pages), pruned with a
 * penalty of lambda blocks per remote replica charged to the expert's owner,
 * falling back to the no-replica plan unless that lowers the penalised
 * maximum load.  Ties go to the lower GPU, then the lower expert: the plan is
 * a deterministic function of the counts.
 *
 *   counts         [E] int32 device in: routed rows per expert (>= 0).
 *   blocks_per_gpu [E, G] int32 out: blocks of expert e computed on GPU g
 *                  (row sums = ceil(c_e / beta)).
 *   row_ranges     [E, G, 2] int32 out: [lo, hi) of expert e's rows (offsets
 *                  inside its group, routed order) that GPU g computes; the
 *                  holders take consecutive ranges in ascending GPU order.
 *   gpu_load       [G] int32 out: blocks per GPU.
 *   info           [4] int32 out: the winning search (0-3: donor priority by
 *                  GPU load / by block count x one / several new replicas
 *                  per round; 4: the no-replica plan), tau, the number of
 *                  replicas, the maximum load.
 *   ws             moe_plan_workspace_size(E, G) bytes, 256-byte aligned.
 * Limits: 1 <= G <= min(E, MOE_PLAN_MAX_GPUS), E <= MOE_MAX_EXPERTS,
 * beta >= 1, 0 <= budget <= E, rounds >= -1, lambda >= -1; otherwise
 * MOE_ERR_INVALID_ARG with nothing enqueued.  One CTA of 128 threads; its
 * time grows with E * G and with the number of single-block moves.
 */
#define MOE_PLAN_MAX_GPUS 64
size_t moe_plan_workspace_size(int E, int G);
moe_status moe_plan_replicas(const int32_t* counts, int E, int G, int beta, int budget,
                             int rounds, int lambda, int32_t* blocks_per_gpu,
                             int32_t* row_ranges, int32_t* gpu_load, int32_t* info,
                             void* ws, size_t ws_bytes, void* stream);

/*
 * Synchronises `stream` and returns the device status word of `ws`
 * (MOE_OK, MOE_ERR_NONFINITE, MOE_ERR_TIMEOUT or MOE_ERR_INVALID_ARG), or
 * MOE_ERR_CUDA if the synchronisation itself failed.
 */
moe_status moe_get_device_status(const void* ws, void* stream);

/*
 * Diagnostic (no counterpart on the pages): runs the bounded wait that
 * every pipeline wait of the grouped GEMM uses on a barrier that nothing
 * arrives on.  After `limit_ns` (1 ms .. 2 s, else MOE_ERR_INVALID_ARG) the
 * wait gives up and MOE_ERR_TIMEOUT is written to the status word of `ws`,
 * which moe_get_device_status then returns; the CUDA context stays usable.
 * It lets a test check the timeout path without faulting or hanging a GPU.
 */
moe_status moe_diag_wait_timeout(void* ws, size_t ws_bytes, long long limit_ns,
                                 void* stream);

/*
 * Diagnostic (no counterpart on the pages): the same for the bounded counter
 * wait with which FC2 waits for a token block's FC1 tiles when the two
 * overlap, on a counter in `ws` that nothing increments.  Same arguments and
 * results as moe_diag_wait_timeout.
 */
moe_status moe_diag_count_wait_timeout(void* ws, size_t ws_bytes, long long limit_ns,
                                       void* stream);

/*
 * Diagnostic (no counterpart on the pages): for the calling thread's calls of
 * moe_balance_loss and moe_layer_norm_backward from here on, bounded waits run
 * out after `limit_ns` (1 ms .. 2 s; 0: their usual second), and a part that
 * others wait for -- the first block's sums, or its first row -- comes late by
 * as many nanoseconds as the device int64 at `hold_at` holds (2 s at most; null:
 * by none).  The word is read when the call runs, so a captured call can be late
 * once.  With both 0 calls are as usual again.
 */
moe_status moe_diag_hold(const int64_t* hold_at, long long limit_ns);

/* Static, NUL-terminated description of a status code. */
const char* moe_status_string(moe_status s);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
