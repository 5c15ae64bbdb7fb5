/*
 * spec.h -- C ABI of a B200 (sm_100a) library for the tree-verification step
 * of EAGLE-3 speculative decoding.
 *
 * What the step computes ("EAGLE-3投机解码：树验证器方法", fanquanpp.github.io,
 * sections 验证-接受语义 and 树draft vs 链draft):
 *   - the target model runs ONE forward pass over a whole draft tree, given as
 *     a token array plus parent indices, on top of the sequence's K/V cache;
 *   - every tree node attends to the cached prefix and to its own ancestors
 *     only (the tree's structure is fixed before verification);
 *   - a draft node is accepted iff its token equals the target's argmax at its
 *     parent; the walk from the root keeps the longest accepted path (lowest
 *     index child first) and emits one bonus token, the target's argmax at the
 *     last accepted node -- so each step emits accepted_len + 1 tokens, exactly
 *     what greedy autoregressive decoding would emit;
 *   - only the root's and the accepted nodes' K/V stay in the cache, moved to
 *     consecutive slots.
 *
 * Conventions for every function below:
 *   - return value: SPEC_OK (0) or a negative SPEC_ERR_* code; on error the
 *     cached state of every sequence is unchanged and spec_last_error() holds
 *     a message;
 *   - "device" pointers are CUDA device memory of the GPU that was current at
 *     spec_init; "host" pointers are ordinary CPU memory;
 *   - the library borrows every buffer it is given (weights, K/V cache,
 *     workspace) and never frees one; they must outlive the handle;
 *   - a handle is not thread-safe; all GPU work runs on the stream given to
 *     spec_init.
 */
#ifndef SPEC_H
#define SPEC_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define SPEC_API __attribute__((visibility("default")))
#else
#define SPEC_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* return codes */
#define SPEC_OK 0
#define SPEC_ERR_ARG (-1)      /* null pointer, bad dimension, misaligned buffer */
#define SPEC_ERR_TREE (-2)     /* parents[0] != -1, or some parents[i] outside [0, i) */
#define SPEC_ERR_TOKEN (-3)    /* a token outside [0, vocab) */
#define SPEC_ERR_CAPACITY (-4) /* n_nodes > max_nodes, batch > max_batch, length + n_nodes > max_seq, buffer too small */
#define SPEC_ERR_ROOT (-5)     /* tokens[0] is not the sequence's pending token */
#define SPEC_ERR_CUDA (-6)     /* a CUDA call failed; the message names the cudaError_t */
#define SPEC_ERR_TIMEOUT (-7)  /* a bounded wait inside a kernel expired */
#define SPEC_ERR_STATE (-8)    /* sequence not prefilled, or truncation beyond its length */
#define SPEC_ERR_RANGE (-9)    /* bf16 models: a q / K / V value outside the fp16 range of the cache (|v| > 65504) */

/* model dtypes */
#define SPEC_DTYPE_F32 0       /* weights, activations and K/V in fp32; plain FFMA arithmetic */
#define SPEC_DTYPE_BF16 1      /* weights bf16; GEMM activations as split bf16 (hi + lo); q, K/V cache and
                                  attention probabilities fp16; fp32 accumulation, residual and softmax.
                                  q, K and V (after the rotary embedding) must lie within the fp16 range,
                                  |v| <= 65504: a step that meets a value beyond it (or a NaN) stores it
                                  saturated, leaves every sequence's state as it was, and fails with
                                  SPEC_ERR_RANGE */
#define SPEC_DTYPE_F16 2       /* fp16 rows; only the spec_kv8_* calls take it */

/* flags of spec_verify_tree_batch */
#define SPEC_DEVICE_OUTPUTS 1  /* outputs are device pointers (or NULL); return without synchronising */
#define SPEC_DEBUG_LOGITS 2    /* also store fp32 logits [total nodes][vocab] to the buffer of spec_set_debug_logits */
#define SPEC_NO_GRAPH 4        /* launch kernel by kernel instead of replaying a captured CUDA graph */
#define SPEC_FEATURES 8        /* also write the draft-head features of the root and the accepted nodes to
                                  the buffer of spec_set_feature_out (needs cfg.feature_layers) */

typedef struct spec_config {
  int32_t n_layers;
  int32_t hidden;       /* d */
  int32_t n_q_heads;    /* Hq */
  int32_t n_kv_heads;   /* Hkv; Hq % Hkv == 0 (query head j reads kv head j / (Hq/Hkv)) */
  int32_t head_dim;     /* hd; bf16 models need 128, fp32 models <= 128 and even */
  int32_t ffn;          /* SwiGLU width */
  int32_t vocab;
  int32_t dtype;        /* SPEC_DTYPE_* */
  float rms_eps;        /* RMSNorm epsilon */
  float rope_theta;     /* rotary base (rotate-half pairing, no frequency scaling) */
  int32_t max_batch;    /* sequences held in the cache */
  int32_t max_seq;      /* cache slots per sequence */
  int32_t max_nodes;    /* tree nodes per sequence per step, root included; <= 128 */
  int32_t draft_head;   /* 1: the handle also runs the EAGLE-3 draft head (bf16 only): its weights in
                           spec_weights, its layer's K/V one more cache layer (counted by spec_kv_bytes) */
  int32_t feature_layers[3]; /* the low, mid and high features the EAGLE-3 draft head takes (its
                           draft-stage description: the target's low-, mid- and high-level hidden
                           states of every position): the residual stream after this many decoder
                           layers, each in [1, n_layers]; {0, 0, 0}: no feature tap.  The pages name
                           no layers; 2, n_layers / 2 and n_layers - 3 is one choice. */
  int32_t draft_vocab;  /* reduced draft vocabulary (VocabTrim / FR-Spec / SpecVocab in the aitangshan.cn
                           walkthrough, sections 1 and 3.2): 0 = the draft head scores the whole vocabulary;
                           2 .. vocab = its LM head is spec_weights.draft_lm_head, the target's rows of the
                           token ids draft_vocab_ids, its softmax and its drafts cover only those tokens
                           (verification is unchanged).  Needs draft_head. */
} spec_config;

/* Per-layer weights, device pointers, row-major [out][in] in the model dtype:
 * wq [Hq*hd][d], wk/wv [Hkv*hd][d], wo [d][Hq*hd], w_gate/w_up [ffn][d],
 * w_down [d][ffn]; attn_norm / mlp_norm [d]. */
typedef struct spec_layer_weights {
  const void* wq;
  const void* wk;
  const void* wv;
  const void* wo;
  const void* w_gate;
  const void* w_up;
  const void* w_down;
  const void* attn_norm;
  const void* mlp_norm;
} spec_layer_weights;

/* Model weights.  `layers` is a HOST array of n_layers entries (copied by
 * spec_init); every weight pointer in it, and embed [vocab][d], final_norm [d],
 * lm_head [vocab][d], are device pointers 16-byte aligned.  The draft-head
 * fields may be NULL when cfg.draft_head == 0: draft_fc_fuse [d][3d],
 * draft_fc_in [d][2d], draft_layer (host pointer to one entry), draft_final_norm [d]. */
typedef struct spec_weights {
  const void* embed;
  const void* final_norm;
  const void* lm_head;
  const spec_layer_weights* layers;
  const void* draft_fc_fuse;
  const void* draft_fc_in;
  const spec_layer_weights* draft_layer;
  const void* draft_final_norm;
  const void* draft_lm_head;        /* cfg.draft_vocab > 0: [draft_vocab][d], device, 16-byte aligned */
  const int32_t* draft_vocab_ids;   /* cfg.draft_vocab > 0: [draft_vocab] token ids, device, strictly
                                       increasing in [0, vocab) (checked by spec_init: SPEC_ERR_ARG) */
} spec_weights;

typedef struct spec_handle spec_handle;

/* Bytes of device memory for the K/V cache.  Layout [layer][plane][seq][kv head][slot][hd]:
 * fp32 models hold planes K, V (fp32); bf16 models hold K, V and K_lo in fp16, where
 * K_lo = fp16(k - fp16(k)) carries the rounding error of K so that the attention
 * scores see ~22 bits of each key. */
SPEC_API size_t spec_kv_bytes(const spec_config* cfg);
/* Bytes of device workspace (activations, split-K partials, per-sequence state). */
SPEC_API size_t spec_workspace_bytes(const spec_config* cfg);

/* Validate dimensions, record the borrowed device buffers, build the TMA
 * descriptors.  kv_cache and workspace are device buffers of at least the
 * sizes above; cuda_stream is a cudaStream_t (NULL: the legacy default stream,
 * on which steps are launched kernel by kernel because it cannot be captured
 * into a CUDA graph).
 * Every sequence starts empty. */
SPEC_API int spec_init(const spec_config* cfg, const spec_weights* w, void* kv_cache, size_t kv_bytes, void* workspace,
              size_t ws_bytes, void* cuda_stream, spec_handle** out);

/* Reset sequence `seq` and run the prompt (host int32[n], n >= 1) through the
 * target in causal chunks of at most max_nodes tokens, caching every position.
 * *pending_token (host) receives the argmax at the last position: the root of
 * the next tree.  Synchronises the stream. */
SPEC_API int spec_prefill(spec_handle* h, int seq, const int32_t* tokens, int n, int32_t* pending_token);
/* spec_prefill that also writes the draft-head features of every prompt position (the
 * residual stream after feature_layers[0], [1] and [2] decoder layers, rounded to bf16) to
 * feats_out: device bf16 [n][3][hidden], 16-byte aligned, owned by the caller.  These are
 * the features the EAGLE-3 draft head records during prefill (its draft-stage description).
 * SPEC_ERR_STATE when the handle has no feature layers. */
SPEC_API int spec_prefill_features(spec_handle* h, int seq, const int32_t* tokens, int n, int32_t* pending_token,
                                   void* feats_out);

/* One verification step for one sequence (host pointers, synchronises).
 * tokens[0] must be the pending token; parents[0] == -1 and 0 <= parents[i] < i.
 * accepted_tokens needs room for n_nodes - 1 entries.  Emitted tokens are
 * accepted_tokens[0 .. *accepted_len) followed by *bonus_token, which becomes
 * the next pending token. */
SPEC_API int spec_verify_tree(spec_handle* h, int seq, const int32_t* tokens, const int32_t* parents, int n_nodes,
                     int32_t* accepted_len, int32_t* accepted_tokens, int32_t* bonus_token);

/* Batched verification.  Host inputs: seq_ids[B] (distinct), node_offsets[B+1]
 * (node_offsets[0] == 0), tokens / parents concatenated per sequence, parents
 * local to their sequence.  Outputs per sequence b: accepted_len[b],
 * accepted_nodes[b * max_nodes + k] (local node indices), accepted_tokens
 * (same layout), bonus[b].  Without SPEC_DEVICE_OUTPUTS they are host pointers
 * and the call synchronises; with it they are device pointers (or NULL) and the
 * call returns once the work is queued -- errors found on the device are then
 * reported by the next spec_sync. */
SPEC_API int spec_verify_tree_batch(spec_handle* h, int B, const int32_t* seq_ids, const int32_t* tokens,
                           const int32_t* parents, const int32_t* node_offsets, int32_t* accepted_len,
                           int32_t* accepted_nodes, int32_t* accepted_tokens, int32_t* bonus, int flags);

/* The target's argmax (and top-1 / top-2 logits) at every node of a batch of
 * trees, without acceptance and without changing any cached state.  Inputs as
 * in spec_verify_tree_batch; outputs are host arrays of node_offsets[B]
 * entries.  Synchronises. */
SPEC_API int spec_score_trees(spec_handle* h, int B, const int32_t* seq_ids, const int32_t* tokens, const int32_t* parents,
                     const int32_t* node_offsets, int32_t* argmax, float* top1, float* top2, int flags);

/* ---- EAGLE-3 draft head (cfg.draft_head = 1, bf16 models) ----------------
 * The draft stage of "EAGLE-3: Scaling up Inference Acceleration of Large
 * Language Models via Training-Time Test" (summary page, draft-stage section):
 * the target's low, mid and high features l, m, h of a position (d each) are
 * concatenated and reduced by one FC layer to the fused feature g = [l|m|h].
 * W_fuse^T; g is concatenated with the embedding e of the token one step ahead
 * and reduced by a second FC layer, x = [g|e].W_in^T; one pre-norm decoder layer
 * of the target's shape (its own K/V cache) turns x into a, and the target's LM
 * head, after the draft head's final RMSNorm, scores a.  Readings where the page
 * is silent: concatenation orders [l|m|h] and [g|e]; e from the target's
 * embedding table; tree nodes attend to the draft prefix and their ancestors
 * at positions prefix + depth, as in verification.
 *
 * feats are DEVICE pointers to bf16 [rows][3][d] (l, m, h per row); tokens,
 * parents and node_offsets are host arrays as in spec_verify_tree_batch. */
#define SPEC_DRAFT_TOPK 10     /* draft candidates per node (the pages' tree top-k) */

/* Build the draft layer's K/V for positions 0 .. n-1 of `seq` from n rows of
 * features and tokens (n <= max_seq), replacing what was there.  Synchronises. */
SPEC_API int spec_draft_prefill(spec_handle* h, int seq, const void* feats, const int32_t* tokens, int n);
/* As spec_draft_prefill, but the n rows extend the draft prefix of `seq` (positions len ..
 * len + n - 1, attending to the rows before them): the rows a verification step adds.
 * SPEC_ERR_STATE when the sequence has no draft prefix; SPEC_ERR_CAPACITY past max_seq (both
 * before any work, the prefix unchanged).  An error during the work leaves the prefix marked
 * unusable: rebuild it with spec_draft_prefill.  Synchronises. */
SPEC_API int spec_draft_append(spec_handle* h, int seq, const void* feats, const int32_t* tokens, int n);
/* One draft-head step over a batch of trees on the draft prefixes: per node,
 * the SPEC_DRAFT_TOPK best vocabulary entries of the draft distribution, by
 * logit descending then index ascending, in top_idx / top_val [nodes][TOPK]
 * (selected inside the LM-head GEMM, per 128-row vocabulary tile, then merged:
 * the draft logits are not stored).
 * The draft prefixes are not extended (the trees' K/V are scratch).  Flags:
 * SPEC_DEVICE_OUTPUTS (outputs are device pointers, no synchronisation),
 * SPEC_DEBUG_LOGITS (also the fp32 draft logits to the debug buffer),
 * SPEC_NO_GRAPH.  Errors as in spec_verify_tree_batch; SPEC_ERR_STATE when a
 * sequence has no draft prefix. */
SPEC_API int spec_draft_step(spec_handle* h, int B, const int32_t* seq_ids, const void* feats, const int32_t* tokens,
                             const int32_t* parents, const int32_t* node_offsets, int32_t* top_idx, float* top_val,
                             int flags);
/* Draft prefix length of `seq` (host output). */
SPEC_API int spec_draft_len(spec_handle* h, int seq, int32_t* len);

/* Dynamic draft tree for B sequences ("EAGLE-3: Scaling up Inference Acceleration of Large
 * Language Models via Training-Time Test", draft-stage description: multi-step drafting, where
 * from the second step on the draft's own output a replaces the target feature; and its account
 * of EAGLE-2: the draft's confidence stands in for the acceptance rate and shapes the tree).
 * Reading taken where the pages leave steps open: a node's value is the sum of the draft's
 * log-probabilities (full-vocabulary softmax) along its root path; step t = 0 .. steps-1 runs
 * the draft head over the tree built so far (the root's feature is the fused target feature,
 * every other node's the output a of its parent); the nodes that joined last (the root at step
 * 0) offer their topk best tokens and the topk best offers join (ties: earlier offer); after the
 * last step the `total` best offers, joined or not (ties: lower depth, then earlier offer), form
 * the tree, which is closed under ancestors.
 * root_feats: device bf16 [B][3][hidden], 16-byte aligned, the low/mid/high target features of
 * each sequence's last verified position (as SPEC_FEATURES returns them); root_tokens: host
 * int32 [B], the pending tokens (the roots).  Each sequence needs a draft prefix (the rows up to
 * the last verified position, spec_draft_prefill), which the call leaves unchanged.  topk is 4,
 * 8, 10 or 16; 1 + (steps-1)*topk <= max_nodes, 1 + steps*topk <= 128, topk + (steps-1)*topk^2
 * <= 1024 offers, total <= that and total + 1 <= max_nodes (SPEC_ERR_CAPACITY otherwise).
 * Outputs (host): out_tokens / out_parents int32 [B][total+1], root first, nodes by depth and
 * then value, parents[i] < i (a tree spec_verify_tree_batch accepts); out_values (may be NULL)
 * float [B][total+1], each node's value (0 for the root).  Synchronises. */
SPEC_API int spec_draft_tree(spec_handle* h, int B, const int32_t* seq_ids, const void* root_feats,
                             const int32_t* root_tokens, int steps, int topk, int total, int32_t* out_tokens,
                             int32_t* out_parents, float* out_values);

/* Device buffer for SPEC_FEATURES, bf16 [B][max_nodes][3][hidden], 16-byte aligned, owned by the
 * caller.  A verification step with SPEC_FEATURES writes, for batch entry b and k = 0 ..
 * accepted_len[b], row [b][k] = the residual stream after feature_layers[0], [1] and [2] decoder
 * layers (rounded to bf16) at the k-th node of the emitted path: the root for k = 0, then the
 * accepted nodes in order, i.e. the positions P .. P + accepted_len that the step adds to the cache.
 * Rows beyond accepted_len[b] are left as they were.  bytes must cover the step's batch:
 * B * max_nodes * 3 * hidden * 2 (checked per step; SPEC_ERR_CAPACITY otherwise).  SPEC_ERR_STATE
 * when the handle has no feature layers; device_buf NULL detaches the buffer. */
SPEC_API int spec_set_feature_out(spec_handle* h, void* device_buf, size_t bytes);

/* Temperature sampling instead of greedy choices (both leave the target's output distribution
 * unchanged: "EAGLE-3投机解码：树验证器方法", section 验证-接受语义, and the sampling rule of
 * Leviathan et al., "Fast Inference from Transformers via Speculative Decoding", which that page
 * cites).  temperature = 0 (the default) restores greedy decoding.
 *
 * With temperature T > 0, every token the target chooses -- the pending token of a prefill, the
 * choice at each tree node of a verification or scoring step -- is a draw from softmax(logits / T),
 * taken as argmax_v(logit_v / T + g_v) with g_v a standard Gumbel variable.  The noise of a row
 * depends only on (seed, sequence id, the row's position, v): g_v = -ln(-ln u) with
 * u = (2 (x >> 9) + 1) 2^-24 and x word 0 of Philox4x32-10 (Salmon et al., SC 2011) at counter
 * (v, position, sequence id, 0) and key (seed & 0xffffffff, seed >> 32).  A tree node at position
 * P + depth accepts, as in the greedy walk, the first child whose token equals its draw; the bonus is
 * the draw at the last accepted node.  Each draft token thus acts as a point-mass proposal in the
 * speculative-sampling rule (accepted with probability p(x) given the earlier siblings' rejections),
 * and the emitted stream is exactly autoregressive sampling with the same noise.  spec_score_trees
 * then returns the draws as "argmax" and the perturbed scores logit / T + g as top1 / top2.  The
 * draft head's top-k is unaffected.  SPEC_ERR_ARG for a negative, infinite or NaN temperature or
 * one whose reciprocal overflows.  Takes effect for calls made after it (cached graphs are rebuilt). */
SPEC_API int spec_set_sampling(spec_handle* h, float temperature, uint64_t seed);

/* Device buffer (fp32, >= max_batch * max_nodes * vocab entries) for SPEC_DEBUG_LOGITS. */
SPEC_API int spec_set_debug_logits(spec_handle* h, float* device_buf, size_t bytes);

/* Roll sequence `seq` back to new_len cached positions (new_len < current
 * length, or equal for a no-op); the token cached at new_len becomes pending. */
SPEC_API int spec_truncate(spec_handle* h, int seq, int new_len);
/* Cached length and pending token of `seq` (host outputs; synchronises). */
SPEC_API int spec_seq_len(spec_handle* h, int seq, int32_t* len, int32_t* pending);
/* Wait for queued work; report (and clear) errors recorded on the device. */
SPEC_API int spec_sync(spec_handle* h);

/* Host-only check of one tree, usable without a GPU or a handle: 1 <= n <=
 * max_nodes (else SPEC_ERR_CAPACITY), parents[0] == -1 and 0 <= parents[i] < i
 * (else SPEC_ERR_TREE), every token in [0, vocab) (else SPEC_ERR_TOKEN); null
 * pointers give SPEC_ERR_ARG.  The verification calls apply the same checks. */
SPEC_API int spec_validate_tree(const int32_t* tokens, const int32_t* parents, int n, int vocab, int max_nodes);

/* Kernel classes timed by the profiler (index into spec_profile_read's arrays). */
#define SPEC_PROF_EMBED_META 0   /* tree metadata + embedding + first RMSNorm */
#define SPEC_PROF_GEMM_QKV 1
#define SPEC_PROF_ROPE_KV 2      /* split-K sum + rotary + K/V cache store */
#define SPEC_PROF_ATTENTION 3    /* tree attention chunks + merge */
#define SPEC_PROF_GEMM_O 4
#define SPEC_PROF_RESID_NORM 5   /* split-K sum + residual + RMSNorm */
#define SPEC_PROF_GEMM_GATE_UP 6 /* gate/up GEMM with fused SwiGLU */
#define SPEC_PROF_GEMM_DOWN 7
#define SPEC_PROF_LM_HEAD 8      /* LM-head GEMM with fused argmax */
#define SPEC_PROF_LM_REDUCE 9
#define SPEC_PROF_WALK 10        /* acceptance walk + state update */
#define SPEC_PROF_COMPACT 11     /* K/V compaction */
#define SPEC_PROF_GEMM_LAYER 12  /* one launch: O, gate/up, down, then the next QKV or the LM head */
#define SPEC_PROF_DRAFT_FC 13    /* draft head: feature split, fusion FC, input FC */
#define SPEC_PROF_TOPK 14        /* draft head: merge of the LM-head tiles' top-k candidates */
#define SPEC_PROF_FEATURES 15    /* draft-head feature tap and gather (SPEC_FEATURES) */
#define SPEC_PROF_TREE 16        /* dynamic draft tree: root features, expansion, rerank */
#define SPEC_PROF_CLASSES 17

/* enable != 0: subsequent steps launch kernel by kernel (no graph) with a CUDA
 * event pair around every launch on the handle's stream. */
SPEC_API int spec_profile(spec_handle* h, int enable);
/* Synchronise, then add the recorded device milliseconds and launch counts per
 * class into ms[SPEC_PROF_CLASSES] and launches[SPEC_PROF_CLASSES] (host
 * arrays, either may be NULL) and forget the records. */
SPEC_API int spec_profile_read(spec_handle* h, double* ms, int64_t* launches);
/* Bytes one synchronous verification step copies host->device (parameter
 * block) and device->host (outputs and error word). */
SPEC_API int spec_io_bytes(spec_handle* h, size_t* h2d, size_t* d2h);
/* Human-readable execution plan (residency, GEMM tiling and split-K, attention
 * chunking) for a batch of B trees of n_nodes nodes on prefixes of `prefix`
 * tokens, written to buf (n bytes, NUL-terminated). */
SPEC_API int spec_info(spec_handle* h, int B, int n_nodes, int prefix, char* buf, size_t n);
/* Optional timeline of decoder layer `layer` (bf16 models), in %globaltimer
 * stamps (uint64 ns); NULL turns it off.  device_buf holds 2 * SMs * 64 + 8192
 * entries: first the layer's GEMM launch, [2 * SMs CTAs][4 phases][16] (0-7:
 * producer starts the phase, may load its activations, has issued its last
 * load; epilogue starts the phase, first accumulator complete, split-K
 * rendezvous passed, units done, phase counted at the grid barrier; 8-11 for the
 * first unit: partial stored, split partials summed, finishing stores done,
 * unit done), then its attention launch and the next layer's, [2][256 CTAs][16] (start, Q landed,
 * first K/V block landed, first scores ready, output accumulated, partial
 * written, chunk rendezvous passed, merge done, first block's max found, first
 * block's P written, first scores issued, last P seen by the issuer).  Entries
 * of CTAs that did not run stay as they were. */
SPEC_API int spec_set_trace(spec_handle* h, uint64_t* device_buf, size_t bytes, int layer);
/* Number of kernels the most recent step enqueued. */
SPEC_API int spec_step_launches(spec_handle* h);

/* LM head with fused per-row argmax, for callers that cannot allocate device
 * memory.  (The pages have no counterpart: this is a deployment variant of the
 * step's last kernel.)  Some callers are not allowed to call cudaMalloc: code
 * running inside a CUDA-graph capture, runtimes that own every buffer and hand
 * out no allocation rights, plug-in hosts that forbid allocation after start-up.
 * This entry point needs no allocation and no handle: its scratch (a split-bf16
 * copy of the normalised rows and per-vocabulary-tile top-2 partials) is one
 * fixed array of about 3.5 MiB inside the library, which every GPU that loads
 * the library holds until the process exits.
 *
 * Computes, for each of M hidden rows h (device fp32 [M][d], before the final
 * norm): RMSNorm(h) * final_norm (device bf16 [d]) times lm_head^T (device bf16
 * [V][d], 16-byte aligned), and writes argmax[M] (lowest index on ties),
 * top1[M] and top2[M] (device arrays).  Limits: 1 <= M <= 64, d a multiple of
 * 128 up to 8192, V up to 262144; larger sizes return SPEC_ERR_CAPACITY before
 * any GPU work.  Work is queued on cuda_stream (NULL: legacy default stream);
 * the call does not synchronise.
 *
 * Device-side failure: every wait inside the call is bounded (2 s).  If one
 * gives up, the GPU stays usable and every row gets argmax = -1 and
 * top1 = top2 = NaN; the return code cannot say so, because the call returns
 * before the GPU runs.  After synchronising the stream, argmax[0] < 0 means
 * the outputs are void.  The error word behind this is part of the scratch and
 * is cleared at the start of each call.
 *
 * The first call on a device looks up the scratch array's device address and
 * sets kernel attributes, so make that first call before any stream capture.
 * Every call uses the same scratch and leaves its contents behind; only the
 * error word has to start at zero, and the call clears it itself (a memset on
 * cuda_stream, no allocation).  Calls that overlap on the GPU (on different
 * streams, or from different threads) race on the scratch: serialise them. */
SPEC_API int spec_lm_head_argmax_noalloc(const float* hidden, const void* final_norm, const void* lm_head, int M,
                                         int d, int V, float eps, int32_t* argmax, float* top1, float* top2,
                                         void* cuda_stream);

/* ---- 8-bit paged K/V cache -------------------------------------------------
 * A K/V cache in 8 bits, for callers that hold more or longer sequences than the
 * handle's dense fp16 cache has room for (256 bytes per token and kv head
 * instead of 768).  Three operators share it: spec_kv8_plan finds the pages and
 * slots of new rows, spec_kv8_append stores rows, spec_kv8_attention attends over
 * cached prefixes with the tree visibility of the verification step.
 *
 * Layout: pages of `page` tokens; codes[layer][K, V][page id][kv head][token][128]
 * are e4m3, and exps[layer][K, V][page id][kv head] hold one exponent byte e per
 * page and head: a stored value is code * 2^(e - 127).  The scale is a power of
 * two so that a page whose later tokens need a larger one is rescaled by a shift
 * of its codes' exponents: exact but for codes that become subnormal.  e = 255
 * stands for NaN; the codes 0x7F and 0xFF do not occur in pages without it.  e - 127 is
 * the least whole number of [-60, 120] with max |x| <= 448 * 2^(e - 127).
 *
 * Sequence s holds lengths[s] tokens; token i lies in page tables[s][i / page], at
 * place i % page; its slot is that page id * page + the place.  lengths, tables
 * and the ring of free pages are the caller's device buffers, so that no call
 * below needs the host to know a length.
 *
 * The calls take device pointers of the GPU that was current at spec_kv8_open
 * (it has to be current again at every call: SPEC_ERR_ARG otherwise), queue their
 * work on cuda_stream (NULL: the legacy default stream), do not synchronise and
 * allocate nothing; all can be captured into a CUDA graph.  Calls that touch the
 * same pages or buffers have to be ordered by the caller, outputs may overlap inputs
 * only where it is said, and a handle is not for two threads at once. */
typedef struct spec_kv8_config {
  int32_t n_layers;
  int32_t n_kv_heads;
  int32_t head_dim;   /* 128 */
  int32_t page;       /* tokens per page: 16, 32, 64 or 128 */
  int32_t n_pages;    /* n_pages * page < 2^31 */
} spec_kv8_config;

typedef struct spec_kv8 spec_kv8;

/* Bytes of the codes and of the exponents (0: configuration rejected). */
SPEC_API size_t spec_kv8_code_bytes(const spec_kv8_config* cfg);
SPEC_API size_t spec_kv8_exp_bytes(const spec_kv8_config* cfg);
/* Record the borrowed buffers (codes 128-byte aligned; neither need be
 * initialised: a page's exponent is set when its first token is stored). */
SPEC_API int spec_kv8_open(const spec_kv8_config* cfg, void* codes, size_t code_bytes, void* exps, size_t exp_bytes,
                           spec_kv8** out);
/* Message of the last error on this handle ("" if none). */
SPEC_API const char* spec_kv8_last_error(spec_kv8* h);
/* Free host-side state; never the borrowed buffers. */
SPEC_API void spec_kv8_close(spec_kv8* h);

/* bits of the device status word that spec_kv8_plan writes (0: done) */
#define SPEC_KV8_ROWS 1   /* more new rows than max_rows */
#define SPEC_KV8_PAGES 2  /* more new pages than are free */
#define SPEC_KV8_TABLE 4  /* a sequence outgrows max_blocks */
#define SPEC_KV8_INDEX 8  /* a sequence id outside [0, n_seqs) or given twice, a length outside
                             [0, max_blocks * page], or a state outside [0, n_pages) / [0, n_pages] */

/* Lengths, pages and slots of a step.  Entry b of the batch (sequence s =
 * seq_ids[b], or b) goes from lengths[s] to max(0, lengths[s] + add[b]) tokens:
 * its new blocks get pages from the head of the ring of free pages, blocks that
 * it no longer needs give theirs back at the tail (add = -2^30 ends a sequence).
 * Pages given back are free for later calls, not for this one.  state = {head,
 * count}: the free pages are ring[(head + i) % n_pages], i < count.
 * Writes offsets (the first new row of every entry), slots (of the new rows, in
 * entry order, then -1 up to max_rows), lengths_out (all n_seqs), state_out, status,
 * the new blocks' entries of tables, and the ring's tail.  Nothing else of tables
 * and ring changes, so the old lengths and state stay valid beside the new ones:
 * a caller may keep both and drop either.  When status is not 0 nothing is done:
 * tables and ring stay as they were, lengths_out and state_out repeat the input,
 * offsets are 0 and slots -1. */
typedef struct spec_kv8_plan_args {
  const int32_t* lengths;  /* [n_seqs] */
  const int32_t* add;      /* [batch] */
  const int32_t* seq_ids;  /* [batch], distinct, or NULL: entry b is sequence b */
  int32_t* tables;         /* [n_seqs][max_blocks] */
  int32_t* ring;           /* [n_pages] */
  const int32_t* state;    /* [2] */
  int32_t* offsets;        /* [batch + 1] */
  int32_t* slots;          /* [max_rows] */
  int32_t* lengths_out;    /* [n_seqs]; may be lengths */
  int32_t* state_out;      /* [2]; may be state */
  int32_t* status;         /* [1] */
  int32_t batch;           /* 1 .. 8192 */
  int32_t n_seqs;          /* 1 .. 65536 */
  int32_t max_blocks;
  int32_t max_rows;        /* 0 .. 2^30 */
} spec_kv8_plan_args;
SPEC_API int spec_kv8_plan(spec_kv8* h, const spec_kv8_plan_args* a, void* cuda_stream);

/* Store K and V of `rows` rows into layer `layer`: row i is row src_rows[i] of k
 * and v (or row i), and goes to slots[i].  A negative slot, or one outside the
 * cache, or a source row outside [0, n_src), stores nothing.  Rows of one page
 * have to follow each other with ascending slots, as spec_kv8_plan lists them; a
 * page whose rows come in separate runs loses some of them.  The run that starts
 * at place 0 opens its page (a new exponent); another one keeps the page's
 * exponent or raises it, and then rescales the tokens before it.  Infinities are
 * stored as the largest value of the page's scale.  A NaN sets the exponent of its
 * page and head to 255: all of that page and head reads as NaN until it is opened
 * anew (its codes are then unspecified). */
typedef struct spec_kv8_append_args {
  const void* k;           /* [n_src][n_kv_heads][128] with the strides below */
  const void* v;
  const int32_t* slots;    /* [rows] */
  const int32_t* src_rows; /* [rows], or NULL */
  int64_t k_row_stride, k_head_stride, v_row_stride, v_head_stride; /* in elements; rows of 16-byte alignment */
  int32_t dtype;           /* SPEC_DTYPE_F32, _BF16 or _F16 */
  int32_t rows;            /* 0 .. 2^30 */
  int32_t n_src;
} spec_kv8_append_args;
SPEC_API int spec_kv8_append(spec_kv8* h, int layer, const spec_kv8_append_args* a, void* cuda_stream);

/* Attention of the rows offsets[b] .. offsets[b + 1] - 1 of every entry b over
 * layer `layer`.  A row sees the lengths[s] cached tokens of its sequence and, with
 * k_new / v_new, those of its own step's rows that are its ancestors, itself
 * included: parents[row] is the row's parent within its entry (-1, or a value
 * outside [0, row within the entry): none); parents NULL: every earlier row.  Query
 * head h reads kv head h / (n_q_heads / n_kv_heads).
 *   out[row][h] = sum_j softmax_j(scale q.k_j) v_j,  lse[row][h] = ln sum_j exp(scale q.k_j)
 * A row that sees nothing gets out 0 and lse -inf.  Rows beyond offsets[batch] are
 * left as they were, as are those of an entry whose sequence id, length, row count
 * (1 .. max_nodes) or offsets are out of range; with `fill`, for buffers that hold
 * nothing yet, the former get what a row gets that sees nothing, the latter NaN.  A
 * page id outside the cache reads as NaN.  out may not overlap the inputs.  Infinities and NaN in q, k_new and v_new
 * reach only the rows that see them, whatever lies in the cache behind a sequence's
 * end none.  Scores are held in 32 bits: |scale q.k| up to 2^21; what a row gets that
 * sees larger ones is not specified (other rows are not touched by it).  Rows of a
 * CTA whose waits run out (see the self-test of the bounded waits) are NaN.
 * max_prefix and max_nodes decide how the work is split: for decoding a bound far
 * above the lengths means few, long shares (8 sequences of 4096 tokens, 32 / 8 heads:
 * 21 us with the bound 4096, 47 us with 131072). */
typedef struct spec_kv8_attention_args {
  const void* q;           /* [rows][n_q_heads][128] with the strides below */
  const void* k_new;       /* [rows][n_kv_heads][128], or NULL: the cached prefix only */
  const void* v_new;
  const int32_t* parents;  /* [rows], or NULL */
  const int32_t* offsets;  /* [batch + 1] */
  const int32_t* tables;   /* [n_seqs][max_blocks] */
  const int32_t* lengths;  /* [n_seqs] */
  const int32_t* seq_ids;  /* [batch], or NULL: entry b is sequence b */
  void* out;               /* [rows][n_q_heads][128], contiguous but for out_row_stride */
  float* lse;              /* [rows][n_q_heads], or NULL */
  void* workspace;         /* spec_kv8_attention_workspace() bytes, the first SPEC_KV8_WORKSPACE_ZERO of them zero
                              before its first use (not between calls, whatever their bounds); calls (or graphs)
                              that may overlap on the GPU need one each */
  size_t workspace_bytes;
  int64_t q_row_stride, q_head_stride, k_row_stride, k_head_stride, v_row_stride, v_head_stride,
      out_row_stride;      /* in elements; rows of 16-byte alignment */
  int32_t dtype;           /* of q, k_new, v_new and out: SPEC_DTYPE_BF16 or _F16 */
  int32_t batch;
  int32_t n_seqs;
  int32_t max_blocks;
  int32_t n_q_heads;       /* a multiple of n_kv_heads, at most 64 times it */
  int32_t rows;            /* rows of q, k_new, v_new, parents and out */
  int32_t max_nodes;       /* most rows of one entry: 1 .. 128 */
  int32_t max_prefix;      /* no lengths[s] is above this (entries above it are left as they were) */
  float scale;             /* > 0; 0: 1 / sqrt(128) */
  int32_t fill;            /* SPEC_KV8_FILL_*: rows of no entry, or of one out of range, are written too */
} spec_kv8_attention_args;
#define SPEC_KV8_FILL_OUT 1
#define SPEC_KV8_FILL_LSE 2
#define SPEC_KV8_WORKSPACE_ZERO 65536
/* Workspace bytes of spec_kv8_attention for these bounds and for all calls whose bounds are none of them above these:
 * a program makes one workspace for its largest batch, trees and prefixes (0: bounds rejected). */
SPEC_API size_t spec_kv8_attention_workspace(spec_kv8* h, int batch, int n_q_heads, int max_nodes, int max_prefix);
SPEC_API int spec_kv8_attention(spec_kv8* h, int layer, const spec_kv8_attention_args* a, void* cuda_stream);

/* Self-test of the bounded waits.  Every wait inside the library's kernels
 * (split-K and attention-chunk rendezvous, grid barriers between GEMM phases,
 * pipeline mbarriers) gives up after a time limit, records a timeout in the
 * step's error word and returns; the step then fails with SPEC_ERR_TIMEOUT and
 * the CUDA context stays usable.  This call runs the same two wait primitives
 * on one GPU thread against a counter that nothing increments and an mbarrier
 * that nothing arrives on, each limited to limit_us microseconds (1 .. 10^6).
 * device_scratch: 16 bytes of device memory, 4-byte aligned, owned by the
 * caller (overwritten).  On return *expired holds how many of the two waits
 * gave up (2 when the mechanism works).  Returns SPEC_ERR_TIMEOUT when the
 * device reported the timeout (the expected outcome), SPEC_OK if it did not,
 * SPEC_ERR_ARG / SPEC_ERR_CUDA on bad arguments or a CUDA error.  Runs on the
 * legacy default stream and synchronises the device. */
SPEC_API int spec_wait_selftest(void* device_scratch, uint32_t limit_us, int32_t* expired);

/* Message of the last error on this handle ("" if none). */
SPEC_API const char* spec_last_error(spec_handle* h);
/* Free host-side state (graphs, descriptors); never frees borrowed buffers. */
SPEC_API void spec_free(spec_handle* h);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_H */
