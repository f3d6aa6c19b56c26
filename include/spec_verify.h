/*
 * spec_verify.h — C ABI of the tree-speculative-decoding verification path
 * (library: libspecverify.so, sm_103a / GB300).
 *
 * Four operations, in the order a verification step runs them:
 *
 *   spec_build_tree_mask   draft tree (parent array) -> ancestor bitmasks + depths
 *   spec_tree_verify_attn  one attention pass of every tree node over the paged
 *                          prefix and the tree's own K/V, ancestors only
 *   spec_accept            longest accepted path + bonus token (greedy / stochastic)
 *   spec_kv_commit         the accepted path's K/V written into the paged cache
 *
 * spec_accept_commit runs the last two as one call (the same results, one kernel
 * boundary fewer). spec_tree_verify_attn_parents runs the first two as one call (the mask
 * built inside the attention from the parent array). spec_tree_verify_attn_kv8 and
 * spec_kv_commit_kv8 are the attention and the commit over an FP8 (E4M3) paged cache;
 * spec_tree_init / spec_tree_expand (/ spec_tree_expand_multi) build the draft tree on
 * the device;
 * spec_accept_noalloc is spec_accept without a workspace argument.
 * Around them: spec_page_table_resize grows the sequences' page-table rows for a step and
 * maps its tokens to slots; spec_qk_norm_rope norms and rotates the projected queries and
 * keys of the tree into the layouts the attention reads; spec_tree_verify_attn_kv8p and
 * spec_kv_commit_kv8p are the attention and the commit over an FP8 (E4M3) cache with a
 * scale per (page, KV head). spec_tree_verify_attn_kv4, spec_kv_commit_kv4 and
 * spec_kv_read_kv4 are the attention, the commit and the reading back over a cache held in
 * 4 bits; spec_token_logprobs gives the log probabilities of the tokens that a step emitted.
 *
 * Sources of the operations (page title, then section):
 *   "EAGLE-2 deep dive" (techknowgenie): architecture section (all tree tokens
 *     verified in one target forward with a 2-D tree mask injected into
 *     attention; target logits contrasted with draft tokens; longest accepted
 *     path; the target KV cache must not be contaminated), core-implementation
 *     section (tree mask = node + ancestors up to the root; node ids in
 *     creation order), production section (paged tree attention indexing the
 *     mask over paged KV), benchmark section (rejection sampling, lossless).
 *   "Accelerating Sonar through speculation" (Perplexity): speculative-decoding
 *     section (n drafts -> up to n+1 tokens; the extra token from the target's
 *     logits at the stop position), draft-target section (acceptance compares
 *     full draft and target distributions; KV filled for accepted tokens),
 *     EAGLE section (a custom mask over the whole sequence slows attention by
 *     up to 50% — so the prefix here is never masked), MTP-schedule section (a
 *     kernel inserts the next token after the shift, no CPU-GPU sync — so
 *     every length stays on the device here).
 *
 * Conventions shared by every call
 *   - Pointers are DEVICE pointers unless stated otherwise; the caller owns
 *     every buffer. No call allocates, frees or synchronises with the host:
 *     each enqueues its kernels on `stream` (a cudaStream_t passed as void*,
 *     NULL = legacy default stream) and returns.
 *   - Layouts are row-major, C order. Tree node ids are sequence-local:
 *     sequence b owns global rows [qo_indptr[b], qo_indptr[b+1]) of every
 *     per-node array; its node i is global row qo_indptr[b] + i.
 *   - Errors the host can see (null pointer, bad size, unsupported shape,
 *     workspace too small) return a negative spec_status at once and enqueue
 *     nothing. Errors that depend on device data (bad parent, page id outside
 *     the pool, path longer than its buffer, timeout of a bounded wait) are
 *     written to *dev_status with first-error-wins semantics (the word is
 *     only changed while it holds SPEC_OK); the kernels then skip the bad
 *     item and finish cleanly — no trap, assert or unbounded wait. dev_status
 *     may be NULL (device errors are then not reported). The caller zeroes
 *     it when it wants a fresh report.
 *   - Workspace: `ws` is scratch of at least spec_workspace_size(...) bytes,
 *     256-byte aligned. It must be zero-filled before its first use with
 *     spec_accept (it keeps arrival counters there); every call leaves the
 *     counters it uses at zero again. One workspace must not serve two calls
 *     that may run concurrently.
 *   - Early start: the kernels are launched with programmatic stream
 *     serialization, so a call may begin while the kernel enqueued before it
 *     is still running. By default every kernel waits for that predecessor
 *     before it reads or writes anything (a predecessor's writes are visible
 *     only after that wait, whether or not it signals early); the commit that
 *     spec_accept_commit launches reads what its acceptance does not write
 *     while that runs, as the acceptance has waited. A caller whose
 *     preceding kernel writes none of the inputs listed below (nor, where that
 *     is an attention, which signals before its own wait, the kernel before
 *     it) can let two kernels read them before the wait with
 *     spec_set_early_reads(1):
 *     spec_tree_verify_attn (and its _kv8, _kv8p and _parents forms) then reads q,
 *     k_pool, v_pool, k_tree, v_tree, page_table, prefix_len, qo_indptr and
 *     kv_scale (everything but the mask or parent array) before it waits, and
 *     greedy spec_accept (and spec_accept_commit), when it walks from the root
 *     (spec_accept_plan), reads parent, draft_tokens, target_logits and
 *     qo_indptr before it waits (spec_accept_commit also the commit's k_tree,
 *     v_tree, page_table and prefix_len); both still wait before their first
 *     write.
 *     (In a target model's forward pass the kernel before the attention
 *     writes q and the tree's K/V, and the one before the acceptance writes
 *     the logits: keep the switch off there, or put an event between.) Of
 *     this library's kernels, the ones that signal early write only mask and
 *     depth (spec_build_tree_mask), out, lse and the workspace (the attention
 *     and its split merge) and the acceptance results (greedy spec_accept when
 *     it streams every row); the commit kernels and the acceptance walks,
 *     which may write the pool, the page-table resize and the norm + rotation
 *     never do (the resize signals to its own second kernel alone).
 */
#ifndef SPEC_VERIFY_H
#define SPEC_VERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SPEC_OK = 0,
  SPEC_ERR_ARG = -1,         /* host: null pointer, negative or inconsistent size            */
  SPEC_ERR_PARENT = -2,      /* device: parent array is not a tree (root != -1, parent >= i) */
  SPEC_ERR_PAGE = -3,        /* device: page table entry outside [0, num_pages)              */
  SPEC_ERR_CAPACITY = -4,    /* device: a sequence needs more nodes/pages/path slots than given */
  SPEC_ERR_WORKSPACE = -5,   /* host: ws_bytes smaller than spec_workspace_size()            */
  SPEC_ERR_UNSUPPORTED = -6, /* host: dtype / head dim / group size not implemented, or a
                                batch past a launch's grid: batch x hkv > 65535 for the
                                attention calls, batch > 65535 for stochastic acceptance
                                and the draft-tree calls                                      */
  SPEC_ERR_CUDA = -7,        /* host: a CUDA runtime call or kernel launch failed            */
  SPEC_ERR_TIMEOUT = -8,     /* device: a bounded wait inside a kernel gave up               */
  SPEC_ERR_INDEX = -9        /* device: token id / path node id out of range                 */
} spec_status;

typedef enum { SPEC_F32 = 0, SPEC_BF16 = 1 } spec_dtype;
typedef enum { SPEC_GREEDY = 0, SPEC_STOCHASTIC = 1 } spec_mode;
typedef enum { SPEC_OP_MASK = 0, SPEC_OP_ATTN = 1, SPEC_OP_ACCEPT = 2, SPEC_OP_COMMIT = 3,
               SPEC_OP_TREE = 4, SPEC_OP_ATTN_KV8P = 5, SPEC_OP_ATTN_KV4 = 6 } spec_op;

/* Bytes of workspace `op` needs for these sizes (0 when it needs none).
 * For SPEC_OP_ATTN the result depends on (batch, max_nodes, hq, hkv, d,
 * max_prefix, total_nodes); for SPEC_OP_ACCEPT on (batch, total_nodes, vocab); for
 * SPEC_OP_ATTN_KV8P (the attention over a cache with page scales) and SPEC_OP_ATTN_KV4 (over
 * a 4-bit cache) on what SPEC_OP_ATTN does, with d = 128; for
 * SPEC_OP_TREE (the draft-tree state of spec_tree_init / spec_tree_expand) on
 * (batch, max_nodes).
 * Unused arguments may be 0. Returns 0 for invalid sizes. */
size_t spec_workspace_size(int op, int batch, int total_nodes, int max_nodes, int hq, int hkv,
                           int d, int max_prefix, int vocab);

/* Launch plan spec_tree_verify_attn uses for these sizes (informational; the pages
 * have no counterpart): *splits = number of key splits (> 1 adds a merge kernel),
 * *tensor_cores = 1 when the tcgen05 kernel runs (every bf16 call with d = 128), 0 for
 * the CUDA-core kernel (fp32 inputs, or d = 64). Returns SPEC_OK or SPEC_ERR_ARG /
 * SPEC_ERR_UNSUPPORTED like the call would. */
int spec_attn_plan(int dtype, int batch, int max_nodes, int hq, int hkv, int d, int page_size,
                   int max_prefix, int* splits, int* tensor_cores);

/* Read plan spec_accept uses for these sizes (informational; the pages have no
 * counterpart): *walk = 1 when the call reads only the rows of the nodes its walk visits
 * (the root and each accepted node) -- always for SPEC_STOCHASTIC; for SPEC_GREEDY when a
 * model of the two ways (a walk from the root, one 8-CTA cluster per sequence, at most
 * path_cap rows each, against streaming every row at the copy rate) finds the walk
 * cheaper, which needs many rows per sequence -- and 0 when it streams every row (logits
 * in host memory always walk, whatever this says). The results are the same either way.
 * sm_count: the GPU's SMs (0: the current device's).
 * Assumes 16-byte aligned logits rows (the walk needs them). Returns SPEC_OK,
 * SPEC_ERR_ARG, or SPEC_ERR_CUDA when sm_count is 0 and no device answers. */
int spec_accept_plan(int mode, int batch, int total_nodes, int vocab, int path_cap, int sm_count, int* walk);

/* Whether the attention and the greedy walk may read their inputs before waiting for
 * the kernel enqueued just before them (the early-start rule above). enable != 0 turns
 * it on for the whole process, 0 (the default) off; each later call reads the setting
 * when it is made (a captured CUDA graph keeps the setting it was captured with).
 * Thread-safe. Results do not depend on it. Returns the previous setting (0 or 1). */
int spec_set_early_reads(int enable);

/* Static, NUL-terminated description of a spec_status value. */
const char* spec_status_string(int status);

/* Library version as an integer (major * 10000 + minor * 100 + patch). */
int spec_version(void);

/*
 * spec_build_tree_mask — ancestor bitmask of every draft-tree node.
 *   ("EAGLE-2 deep dive", core-implementation section: a node's row of the tree
 *   mask marks the node itself and every ancestor, walking parent links to the
 *   root; nodes are numbered after their parents.)
 *
 *   parent     int32 [total_nodes]  sequence-local parent id; the root (node 0 of
 *                                   each sequence) holds -1; node i > 0 needs
 *                                   0 <= parent[i] < i.
 *   qo_indptr  int32 [batch+1]      node ranges; qo_indptr[0] = 0, non-decreasing,
 *                                   qo_indptr[batch] = total_nodes.
 *   max_nodes  >= every sequence's node count; fixes the mask row width
 *              W = ceil(max_nodes / 64) words.
 *   mask       uint64 [total_nodes][W] (out)  bit (j & 63) of word (j >> 6) of row
 *              t = node j of t's sequence is t itself or an ancestor of t. Bits of
 *              node ids >= the sequence's node count are 0.
 *   depth      int32 [total_nodes] (out, nullable)  parent links to the root (root 0).
 *   Device errors: SPEC_ERR_PARENT (that row written all-zero, depth -1),
 *   SPEC_ERR_CAPACITY (sequence longer than max_nodes: its rows written all-zero,
 *   depth -1, so no earlier call's bits remain for a later attention to read).
 */
int spec_build_tree_mask(const int32_t* parent, const int32_t* qo_indptr, int batch,
                         int total_nodes, int max_nodes, uint64_t* mask, int32_t* depth,
                         int32_t* dev_status, void* stream);

/*
 * spec_tree_verify_attn — tree-verify attention with GQA over a paged prefix.
 *   ("EAGLE-2 deep dive", architecture and production sections: one target
 *   forward over all tree tokens, 2-D tree mask inside attention, mask indexed
 *   over paged KV. "Accelerating Sonar", EAGLE section: a mask over the whole
 *   sequence costs up to 50% — here the prefix is never masked.)
 *
 *   For sequence b, node i, query head h (KV head g = h / (hq / hkv)):
 *     keys  = prefix slots 0 .. prefix_len[b]-1  (read through page_table)
 *             ++ tree nodes j of b with mask bit j of row i set
 *     out[t][h] = softmax(sm_scale * q[t][h] . K^T) V,  lse[t][h] = ln sum exp(scores)
 *
 *   dtype      SPEC_F32 or SPEC_BF16: element type of q, k_pool, v_pool, k_tree,
 *              v_tree and out (accumulation is fp32 in both cases).
 *   q          [total_nodes][hq][d]
 *   k_pool, v_pool  [num_pages][hkv][page_size][d]  the paged KV cache ("HND" pages)
 *   page_table int32 [batch][max_pages]  page id of logical page p of sequence b;
 *              entries past ceil(prefix_len[b] / page_size) are not read.
 *   prefix_len int32 [batch]   verified prefix length per sequence (>= 0).
 *   max_prefix >= every prefix_len[b]; used on the host to size the key split.
 *   k_tree, v_tree  [total_nodes][hkv][d]  K/V of the tree tokens themselves.
 *   mask       uint64 [total_nodes][ceil(max_nodes/64)]  from spec_build_tree_mask.
 *   qo_indptr  int32 [batch+1]; max_nodes >= every sequence's node count.
 *   hq % hkv == 0; d in {64, 128}; sm_scale <= 0 selects 1/sqrt(d).
 *   Kernels: bf16 with d = 128 runs on the tensor-core kernel and on nothing else. It
 *   needs page_size 16 and hq / hkv dividing 128 (else SPEC_ERR_UNSUPPORTED), q, k_pool,
 *   v_pool, k_tree, v_tree and out 16-byte aligned (else SPEC_ERR_ARG), and the driver's
 *   tensor-map encoder (else SPEC_ERR_CUDA). fp32 inputs, and d = 64, run on the
 *   CUDA-core kernel (page_size a multiple of 8).
 *   out        [total_nodes][hq][d] (out)
 *   lse        float [total_nodes][hq] (out, nullable)  natural-log log-sum-exp.
 *   ws         workspace of spec_workspace_size(SPEC_OP_ATTN, ...) bytes (key-split
 *              partial results; any contents).
 *   Device errors: SPEC_ERR_PAGE (page id outside [0, num_pages): the page is read
 *   as zeros), SPEC_ERR_CAPACITY (a tree that passes what a launch for max_nodes holds),
 *   SPEC_ERR_TIMEOUT.
 */
int spec_tree_verify_attn(int dtype, const void* q, const void* k_pool, const void* v_pool,
                          int num_pages, int page_size, const int32_t* page_table, int max_pages,
                          const int32_t* prefix_len, int max_prefix, const void* k_tree,
                          const void* v_tree, const uint64_t* mask, const int32_t* qo_indptr,
                          int batch, int total_nodes, int max_nodes, int hq, int hkv, int d,
                          float sm_scale, void* out, float* lse, void* ws, size_t ws_bytes,
                          int32_t* dev_status, void* stream);

/*
 * spec_accept — longest accepted root-to-node path of each tree + the bonus token.
 *   Greedy ("EAGLE-2 deep dive", architecture section; "Accelerating Sonar",
 *   speculative-decoding section): a[v] = argmax of target_logits[v] (lowest
 *   token id on ties); from the root, move to the first child (lowest node id)
 *   whose draft token equals a[v]; stop when none does; bonus = a[stop node].
 *   Stochastic ("EAGLE-2 deep dive", benchmark section; "Accelerating Sonar",
 *   draft-target section; rule of the speculative-sampling works they cite):
 *   p_v = softmax(target_logits[v] / T), q_v = softmax(draft_logits[v] / T);
 *   at node v, r = p_v; each child c (increasing id, token x) is accepted iff
 *   uniforms[c][0] < r(x) / q_v(x); a rejection replaces r by
 *   max(r - q_v, 0) normalised; if no child is accepted the bonus is the
 *   inverse-CDF draw from r with uniforms[v][1].
 *   Rows read: both modes need the logits of the nodes the walk visits only (the
 *   root and each accepted node). Stochastic acceptance always reads just those;
 *   greedy acceptance either streams every row (one wave of CTAs, a last-CTA walk)
 *   or walks from the root reading just those, whichever spec_accept_plan's model
 *   finds cheaper for the sizes. The results are the same either way.
 *
 *   parent, draft_tokens  int32 [total_nodes]  (root's token = last accepted token)
 *   target_logits  float [total_nodes][vocab]
 *   draft_logits   float [total_nodes][vocab]  (stochastic only; NULL for greedy)
 *                  Either may sit in device memory or in pinned host memory the
 *                  device reads at the same address (cudaHostAlloc, or
 *                  cudaHostRegister, under unified addressing). From host memory
 *                  only the visited rows cross the host link (NVLink-C2C on a
 *                  Grace-Blackwell part): greedy acceptance then always walks from
 *                  the root. Any other pointer (pageable host memory, pinned
 *                  memory mapped elsewhere) returns SPEC_ERR_ARG.
 *   uniforms       float [total_nodes][2]      (stochastic only) (u_accept, u_bonus) in [0,1)
 *   temperature    > 0 (stochastic only)
 *   path_cap       row length of path / out_tokens (>= deepest accepted path + 1; the
 *                  trees' depth + 1 always suffices). It also bounds the greedy walk's
 *                  rows per sequence in spec_accept_plan's model.
 *   accept_len int32 [batch] (out)  L = accepted draft nodes (root excluded).
 *   path       int32 [batch][path_cap] (out)  root (0) then the accepted node ids; -1 after.
 *   out_tokens int32 [batch][path_cap] (out)  the L accepted tokens, then the bonus; -1 after.
 *   flags      uint8 [batch] (out, nullable)  stochastic near-ties seen by the GPU:
 *              bit 0 a ratio test with |u - ratio| <= 1e-6, bit 1 a bonus draw within
 *              1e-8 (relative to the residual's total) of a CDF boundary. Greedy writes 0.
 *   ws         workspace of spec_workspace_size(SPEC_OP_ACCEPT, ...) bytes, zeroed
 *              before first use (see the conventions above).
 *   Device errors: SPEC_ERR_PARENT, SPEC_ERR_INDEX (draft token outside [0, vocab)),
 *   SPEC_ERR_CAPACITY (accepted path longer than path_cap - 1: truncated).
 */
int spec_accept(int mode, const int32_t* parent, const int32_t* draft_tokens,
                const float* target_logits, const float* draft_logits, const float* uniforms,
                float temperature, int vocab, const int32_t* qo_indptr, int batch,
                int total_nodes, int max_nodes, int path_cap, int32_t* accept_len, int32_t* path,
                int32_t* out_tokens, uint8_t* flags, void* ws, size_t ws_bytes,
                int32_t* dev_status, void* stream);

/*
 * spec_kv_commit — write the accepted path's K/V into each sequence's cache.
 *   ("EAGLE-2 deep dive", architecture section: verification must not
 *   contaminate the target KV cache; "Accelerating Sonar", draft-target and
 *   MTP-schedule sections: KV of accepted tokens is filled, the next token is
 *   placed after the shift on the device with no CPU sync.)
 *   For i = 0 .. accept_len[b]: tree row qo_indptr[b] + path[b][i] (all hkv heads)
 *   is copied to logical slot prefix_len[b] + i of sequence b (page
 *   page_table[b][slot / page_size], row slot % page_size). Then
 *   seq_len_out[b] = prefix_len[b] + accept_len[b] + 1. accept_len and path are
 *   read on the device (straight from spec_accept), so no host sync is needed.
 *   The tree buffers must not alias the pool.
 *
 *   dtype       element type of k_tree, v_tree, k_pool, v_pool.
 *   k_tree, v_tree  [total_nodes][hkv][d];  k_pool, v_pool  [num_pages][hkv][page_size][d] (in/out)
 *   path        int32 [batch][path_cap];  accept_len int32 [batch]
 *   seq_len_out int32 [batch] (out, nullable)
 *   Device errors: SPEC_ERR_INDEX (path node outside the sequence's tree, or
 *   accept_len outside [0, path_cap)), SPEC_ERR_CAPACITY (slot beyond max_pages),
 *   SPEC_ERR_PAGE (page id outside the pool). A sequence with an error is
 *   left unwritten.
 */
int spec_kv_commit(int dtype, const void* k_tree, const void* v_tree, const int32_t* path,
                   int path_cap, const int32_t* accept_len, const int32_t* qo_indptr,
                   const int32_t* page_table, int max_pages, int num_pages, int page_size,
                   const int32_t* prefix_len, int32_t* seq_len_out, void* k_pool, void* v_pool,
                   int batch, int total_nodes, int hkv, int d, int32_t* dev_status, void* stream);

/*
 * spec_accept_commit — spec_accept, then spec_kv_commit of the paths it accepted, in one
 *   call: the results (accept_len, path, out_tokens, flags, the written pool rows,
 *   seq_len_out, device errors) are those of the two calls made back to back on
 *   `stream`. Greedy acceptance commits inside its own kernel where it can: walking from
 *   the root (spec_accept_plan), each sequence's cluster commits that sequence after its
 *   walk; streaming every row, the last CTA commits up to 4 sequences right after its
 *   walk. More sequences when streaming, and stochastic acceptance, launch the commit
 *   kernel after the acceptance kernels.
 *   Arguments: those of spec_accept (mode ... flags, ws, ws_bytes) and of spec_kv_commit
 *   (dtype ... d); path_cap, path and accept_len serve both. The same host errors, the
 *   same layouts; ws as for spec_accept.
 *   Next-step tokens on the device ("Accelerating Sonar", MTP-schedule section: a kernel
 *   places the next token after the shift, with no CPU-GPU sync):
 *   token_buf  int32 [batch][token_stride] (in/out, nullable)  each sequence's tokens by
 *              position, the root (the last accepted token) at prefix_len[b]. With every
 *              commit of sequence b the call also writes out_tokens[b][0 .. L] (the L
 *              accepted tokens, then the bonus token, the next step's root) to
 *              token_buf[b][P + 1 .. P + L + 1], P = prefix_len[b]; nothing else of the row
 *              changes. A row without room (P + L + 1 >= token_stride) is a device error
 *              SPEC_ERR_CAPACITY, and that sequence is left unwritten (K/V and tokens).
 *   token_stride  row length of token_buf (>= 1 when token_buf is given).
 */
int spec_accept_commit(int mode, const int32_t* parent, const int32_t* draft_tokens,
                       const float* target_logits, const float* draft_logits, const float* uniforms,
                       float temperature, int vocab, const int32_t* qo_indptr, int batch,
                       int total_nodes, int max_nodes, int path_cap, int32_t* accept_len,
                       int32_t* path, int32_t* out_tokens, uint8_t* flags, int dtype,
                       const void* k_tree, const void* v_tree, const int32_t* page_table,
                       int max_pages, int num_pages, int page_size, const int32_t* prefix_len,
                       int32_t* seq_len_out, void* k_pool, void* v_pool, int hkv, int d,
                       int32_t* token_buf, int token_stride, void* ws, size_t ws_bytes,
                       int32_t* dev_status, void* stream);

/*
 * spec_tree_init / spec_tree_expand -- the EAGLE-2 dynamic draft tree, built on the device.
 *   ("EAGLE-2 deep dive", section on the dynamic draft-tree algorithm: a node's confidence
 *   is the product of the draft probabilities along its path; a priority queue pops the
 *   best candidate as the next node; a node below the depth limit is expanded into its
 *   top-k tokens, scored by the product, those at or below a threshold dropped; the tree
 *   stops at the node budget.)
 *   The draft model is the caller's: between two spec_tree_expand calls it writes the
 *   logits row of each sequence's node awaiting expansion (next_node). A call reads that
 *   row, computes p = softmax(row) and the top-k tokens (largest logit first, lower token
 *   id on ties), pushes the k candidates with score = score(node) * p(token), then pops the
 *   best candidate (largest score, the earlier push on ties) as node n_nodes (its parent and
 *   token in parent_out / tokens_out); a popped node at the depth limit is not expanded and
 *   the next best is popped, until one needs its expansion or max_nodes nodes exist. Node
 *   ids therefore grow in pop order and parent[i] < i: parent_out / tokens_out feed
 *   spec_build_tree_mask and the verification calls directly (row b = sequence b).
 *
 *   spec_tree_init: root_tokens int32 [batch] (the last accepted token of each sequence);
 *     sets node 0 (parent -1, score 1), every other entry of parent_out / tokens_out to -1,
 *     n_nodes_out = 1 and next_node = 0 (the root awaits its expansion; -1 if max_nodes = 1).
 *   spec_tree_expand:
 *     draft_logits  float; the row of sequence b for node u starts at
 *                   draft_logits + b * row_stride + u * node_stride (elements). With the
 *                   draft model writing one row per sequence: row_stride = vocab,
 *                   node_stride = 0. Sequences whose next_node is -1 are skipped.
 *     topk in [1, 16]; max_depth >= 1 (a node of that depth is not expanded);
 *     threshold    candidates with score <= threshold are dropped (<= 0: none).
 *     state        spec_workspace_size(SPEC_OP_TREE, batch, 0, max_nodes, ...) bytes,
 *                  written by spec_tree_init; one state per tree under construction.
 *     parent_out, tokens_out  int32 [batch][max_nodes] (in/out);  n_nodes_out, next_node
 *                  int32 [batch] (out);  flags uint8 [batch] (out, nullable): bit 0 set
 *                  when a pop's best two scores were within a relative 1e-6 (the
 *                  probabilities are exp in fp32: such a pop could be ordered either way).
 *   Scores: fp64 products of p(token) = exp(x - max) (fp32) / Z, Z summed in double-float.
 *   Host errors as for the other calls; no device errors.
 */
int spec_tree_init(const int32_t* root_tokens, int batch, int max_nodes, void* state, size_t state_bytes,
                   int32_t* parent_out, int32_t* tokens_out, int32_t* n_nodes_out, int32_t* next_node,
                   uint8_t* flags, void* stream);
int spec_tree_expand(const float* draft_logits, int vocab, long long row_stride, long long node_stride,
                     int batch, int max_nodes, int topk, int max_depth, double threshold, void* state,
                     size_t state_bytes, int32_t* parent_out, int32_t* tokens_out, int32_t* n_nodes_out,
                     int32_t* next_node, uint8_t* flags, int32_t* dev_status, void* stream);

/*
 * spec_tree_expand_multi -- the same construction, several draft rows per call.
 *   ("EAGLE-2 deep dive", section on the dynamic draft-tree algorithm, as above; the batching
 *   is this library's and leaves the tree unchanged.)
 *   A queued candidate's expansion (its draft row's top-k and probabilities) depends only on
 *   the candidate -- its parent node and its token -- not on when it is popped. So each call
 *   lists up to `width` requests per sequence for the next call: request 0 is the node
 *   awaiting its expansion (the last node created), requests 1.. are the best queued
 *   candidates (largest score first, earlier push on ties) that have no row yet and sit
 *   below the depth limit. The caller's draft model writes one row per request (for a
 *   candidate: the row of the node it would become, given its parent and token). The next
 *   call reduces every row, keeps each candidate's result, expands the awaiting node and
 *   pops exactly as spec_tree_expand would, expanding at once every popped node whose result
 *   it holds; it stops at the first popped node that needs a row it has not got, or when the
 *   tree is complete. The tree (parent_out, tokens_out, n_nodes_out, flags) is therefore
 *   spec_tree_expand's, node for node, for every width; width 1 is spec_tree_expand.
 *
 *   After spec_tree_init the request list is the root alone (row 0).
 *   draft_logits  float; row j of sequence b starts at draft_logits + b * row_stride +
 *                 j * req_stride (elements); rows j >= req_n[b] are not read.
 *   width         in [1, 8]: the same for every call on one state (a state listing more
 *                 requests than the call's width is refused: SPEC_ERR_ARG in *dev_status,
 *                 nothing changes). topk, max_depth and threshold as for spec_tree_expand,
 *                 also the same for every call on one state.
 *   state         as for spec_tree_expand (spec_tree_init's), driven by this call only.
 *   req_parent, req_token  int32 [batch][width] (out): the parent node id (-1 for the root)
 *                 and token of each request; -1 past req_n[b].
 *   req_n         int32 [batch] (out): requests listed; 0 once the tree is complete.
 *   next_node     int32 [batch] (out): the awaiting node (request 0), -1 once complete.
 *   A sequence whose tree is complete is skipped: its outputs keep their last values.
 *   Device errors: SPEC_ERR_ARG as above; SPEC_ERR_CAPACITY if the state's result entries
 *   ran out (they cannot: max_nodes * 8 entries, and each call takes at most width while
 *   creating at least one node), the tree then ends.
 */
int spec_tree_expand_multi(const float* draft_logits, int vocab, long long row_stride, long long req_stride,
                           int batch, int max_nodes, int width, int topk, int max_depth, double threshold,
                           void* state, size_t state_bytes, int32_t* parent_out, int32_t* tokens_out,
                           int32_t* n_nodes_out, int32_t* next_node, int32_t* req_parent, int32_t* req_token,
                           int32_t* req_n, uint8_t* flags, int32_t* dev_status, void* stream);

/*
 * spec_accept_noalloc — spec_accept for callers that cannot allocate device memory.
 *   (No counterpart on the pages: this is a deployment convenience of this library.)
 *   Some callers have no way to obtain scratch memory: a runtime that only lends out
 *   the tensors it owns, a plugin host without an allocator, a serving loop that
 *   forbids allocation once it runs. This entry point takes the same arguments as
 *   spec_accept minus the workspace and computes the same results; its scratch is a
 *   fixed 4 MiB array inside the library (a file-scope __device__ array that every GPU
 *   loading the library holds until the process exits). It allocates and frees nothing.
 *   - Limit: sizes whose workspace (spec_workspace_size(SPEC_OP_ACCEPT, ...)) exceeds
 *     4 MiB return SPEC_ERR_WORKSPACE at once (e.g. 128256-token rows: up to ~10K nodes).
 *   - Set-up: the first call on a device, with that device current, looks up the array's
 *     device address; make that first call before any stream capture. The address is
 *     kept for the life of the process: do not use this entry point on a device after
 *     cudaDeviceReset (the array is then reloaded elsewhere).
 *   - Host checks are spec_accept's (the same argument errors, the same limits).
 *   - Every call zeroes the array's counters on `stream` first, then runs the kernels.
 *   - All calls share the one array: calls that may overlap on the GPU (different
 *     streams, or different host threads) race and must be serialised by the caller.
 */
int spec_accept_noalloc(int mode, const int32_t* parent, const int32_t* draft_tokens,
                        const float* target_logits, const float* draft_logits, const float* uniforms,
                        float temperature, int vocab, const int32_t* qo_indptr, int batch,
                        int total_nodes, int max_nodes, int path_cap, int32_t* accept_len,
                        int32_t* path, int32_t* out_tokens, uint8_t* flags, int32_t* dev_status,
                        void* stream);

/*
 * spec_tree_verify_attn_parents — spec_tree_verify_attn with the tree given as its parent
 *   array instead of a mask: the mask step runs inside the attention call.
 *   ("EAGLE-2 deep dive", core-implementation section: a node's mask row is the node and
 *   every ancestor up to the root.)
 *   Arguments: those of spec_tree_verify_attn, minus dtype (bf16 only) and mask, plus
 *   parent  int32 [total_nodes]  sequence-local parents, as for spec_build_tree_mask.
 *   The result equals spec_build_tree_mask followed by spec_tree_verify_attn on the same
 *   stream: for each in-tree key block, every query row derives its ancestor bits by
 *   walking parent links (staged in shared memory), with no mask buffer in between.
 *   - Device error SPEC_ERR_PARENT for a parent array that is not a tree; the affected
 *     rows then see no tree keys.
 *   - The tensor-core path only: d = 128, page_size = 16, hq / hkv dividing 128; other
 *     shapes return SPEC_ERR_UNSUPPORTED (use the two calls).
 *   - The parent array is read after the PDL wait, so it may come from the kernel just
 *     before. No depth output.
 */
int spec_tree_verify_attn_parents(const void* q, const void* k_pool, const void* v_pool, int num_pages,
                                  int page_size, const int32_t* page_table, int max_pages,
                                  const int32_t* prefix_len, int max_prefix, const void* k_tree,
                                  const void* v_tree, const int32_t* parent, const int32_t* qo_indptr,
                                  int batch, int total_nodes, int max_nodes, int hq, int hkv, int d,
                                  float sm_scale, void* out, float* lse, void* ws, size_t ws_bytes,
                                  int32_t* dev_status, void* stream);

/*
 * FP8 KV cache: spec_tree_verify_attn_kv8 / spec_kv_commit_kv8.
 *   ("EAGLE-3 paper explainer" (0h-n0), operations section, model-optimisation list:
 *   quantisation and PagedAttention KV-cache tuning to cut GPU memory. The page names no
 *   format; this library reads it as follows.)
 *   The paged pool holds E4M3 codes, as the OCP 8-bit floating-point format defines them:
 *   1 sign, 4 exponent (bias 7) and 3 mantissa bits, subnormals at exponent 0, S.1111.111
 *   = NaN, largest magnitude 448. Code c of KV head g stands for
 *   value(c) * kv_scale[0][g] in K and value(c) * kv_scale[1][g] in V.
 *   kv_scale   float32 [2][hkv], device memory: K scales, then V scales. Each scale must
 *              be positive, finite and normal. A scale is read on the device at every
 *              call, so it may change between replays of a captured graph.
 *   k_pool, v_pool  uint8 [num_pages][hkv][page_size][d] codes, 16-byte aligned.
 *   The tree's own K/V (k_tree, v_tree), q and out stay bf16.
 *
 * spec_tree_verify_attn_kv8 — spec_tree_verify_attn (same arguments minus dtype, plus
 *   kv_scale) over an FP8 pool. The result is the attention of the definition with every
 *   prefix key and value replaced by its dequantised value; the tree keys are used as
 *   given. The tensor-core path only: d = 128, page_size = 16, hq / hkv dividing 128;
 *   other shapes return SPEC_ERR_UNSUPPORTED. The workspace is spec_workspace_size(
 *   SPEC_OP_ATTN, ...) for the same sizes. Errors as for spec_tree_verify_attn; q, k_tree,
 *   v_tree, out and (with a prefix) the pools must be 16-byte aligned (else SPEC_ERR_ARG).
 *   The pool must hold finite codes: a NaN code (S.1111.111) is read as +-480.
 */
int spec_tree_verify_attn_kv8(const void* q, const uint8_t* k_pool, const uint8_t* v_pool,
                              const float* kv_scale, int num_pages, int page_size,
                              const int32_t* page_table, int max_pages, const int32_t* prefix_len,
                              int max_prefix, const void* k_tree, const void* v_tree,
                              const uint64_t* mask, const int32_t* qo_indptr, int batch,
                              int total_nodes, int max_nodes, int hq, int hkv, int d, float sm_scale,
                              void* out, float* lse, void* ws, size_t ws_bytes, int32_t* dev_status,
                              void* stream);

/*
 * spec_kv_commit_kv8 — spec_kv_commit from bf16 tree rows into an FP8 pool.
 *   Every element x of a committed row of KV head g is written as the E4M3 code nearest to
 *   x / scale (the division in IEEE fp32, then round to nearest, ties to the even code).
 *   Finite quotients beyond +-448 saturate to +-448. scale = kv_scale[0][g] for K,
 *   kv_scale[1][g] for V. Arguments, checks and device errors are those of spec_kv_commit
 *   with dtype = SPEC_BF16 for the tree rows. d must be a multiple of 16 (else
 *   SPEC_ERR_UNSUPPORTED). kv_scale must not be NULL (SPEC_ERR_ARG).
 *   For a fused greedy acceptance + commit into an FP8 pool, call spec_accept and then
 *   this call on the same stream.
 */
int spec_kv_commit_kv8(const void* k_tree, const void* v_tree, const float* kv_scale,
                       const int32_t* path, int path_cap, const int32_t* accept_len,
                       const int32_t* qo_indptr, const int32_t* page_table, int max_pages,
                       int num_pages, int page_size, const int32_t* prefix_len, int32_t* seq_len_out,
                       uint8_t* k_pool, uint8_t* v_pool, int batch, int total_nodes, int hkv, int d,
                       int32_t* dev_status, void* stream);

/*
 * spec_tree_verify_attn_kv8p — spec_tree_verify_attn over an E4M3 paged cache whose scales
 *   belong to pages: one for K and one for V of every (page, KV head).
 *
 *   q, k_tree, v_tree, out  bf16, as spec_tree_verify_attn_kv8
 *   k_pool, v_pool  uint8 [num_pages][hkv][16][128]  OCP E4M3 codes
 *   kv_scale    float [num_pages][hkv][2]  (K scale, V scale) of a page and head; a code
 *               stands for value * scale. Any positive scale; each is read as
 *               min(max(scale, 2^-50), 2^50) (0 and NaN read as 2^-50).
 *   hq / hkv    any group size up to 128 (it need not divide 128).
 *   Everything else as spec_tree_verify_attn (d = 128, page_size 16, else
 *   SPEC_ERR_UNSUPPORTED; kv_scale 8-byte aligned, the other tensors 16, else
 *   SPEC_ERR_ARG). What a row may not see does not reach it: cache rows past prefix_len,
 *   tree nodes its mask bits leave out and nodes of other sequences may hold infinities,
 *   NaN or NaN codes. A row that does see a NaN or an infinity in k or v may be NaN in
 *   every element. A row that sees no key at all is 0 with lse = -infinity.
 *   Rows at or past qo_indptr[batch] are left as they were.
 *   Arithmetic: scores, softmax statistics, sums and lse in fp32. Fewer bits: q enters the
 *   prefix's scores as the sum of two E4M3 terms (exact for elements within 2^9 of their
 *   row's largest, else off by at most 2^-17 of that); a weight meets V in fp16 (prefix:
 *   2^-11 of it) or as two bf16 terms (tree: 2^-16), while the row sum adds it unrounded;
 *   out is rounded to bf16 once. An output element is off by about 2^-11 sum p |v| and that
 *   last rounding.
 *   ws          workspace of spec_workspace_size(SPEC_OP_ATTN_KV8P, ...) bytes (256-byte
 *               aligned; any contents).
 *   Device errors: SPEC_ERR_PAGE (the page is read as zeros), SPEC_ERR_CAPACITY (a tree
 *   past max_nodes, a prefix past max_prefix: that sequence's rows are left as they were),
 *   SPEC_ERR_TIMEOUT.
 */
int spec_tree_verify_attn_kv8p(const void* q, const uint8_t* k_pool, const uint8_t* v_pool,
                               const float* kv_scale, int num_pages, int page_size,
                               const int32_t* page_table, int max_pages, const int32_t* prefix_len,
                               int max_prefix, const void* k_tree, const void* v_tree,
                               const uint64_t* mask, const int32_t* qo_indptr, int batch,
                               int total_nodes, int max_nodes, int hq, int hkv, int d, float sm_scale,
                               void* out, float* lse, void* ws, size_t ws_bytes, int32_t* dev_status,
                               void* stream);

/*
 * spec_kv_commit_kv8p — spec_kv_commit from bf16 tree rows into a cache with page scales;
 *   it keeps the scales.
 *   For every page it writes to, every KV head, K and V apart: let t be the largest finite
 *   |x| of the rows written to the page and s0 the smallest power of two in [2^-50, 2^50]
 *   with t <= 448 s0. A page without older rows (slots below prefix_len[b]) gets the scale
 *   s = s0, whatever it held; a page with older rows s = max(s0, its scale). Written rows
 *   become the E4M3 codes nearest to x / s (ties to the even code, beyond +-448, and
 *   infinities, saturated to +-448, NaN kept); where s has grown, the older rows' codes
 *   become those nearest to value * old scale / s. (Products and quotients in fp32: exact
 *   for the powers of two that this call writes; a scale that came with a page may be any
 *   number, and then they are rounded to fp32 before the code is taken.) Rows past the
 *   written ones keep their codes (they hold nothing). So a scale never shrinks while its
 *   page holds a token.
 *   A page that receives rows must belong to one sequence of the call.
 *
 *   kv_scale    float [num_pages][hkv][2] (in/out)
 *   The other arguments, the checks and the device errors are those of spec_kv_commit with
 *   dtype = SPEC_BF16 (a path may have any length; a sequence whose node range does not lie
 *   in [0, total_nodes) is SPEC_ERR_INDEX). d a multiple of 16 and page_size * d <= 8192, else
 *   SPEC_ERR_UNSUPPORTED.
 */
int spec_kv_commit_kv8p(const void* k_tree, const void* v_tree, const int32_t* path, int path_cap,
                        const int32_t* accept_len, const int32_t* qo_indptr,
                        const int32_t* page_table, int max_pages, int num_pages, int page_size,
                        const int32_t* prefix_len, int32_t* seq_len_out, uint8_t* k_pool,
                        uint8_t* v_pool, float* kv_scale, int batch, int total_nodes, int hkv, int d,
                        int32_t* dev_status, void* stream);

/*
 * 4-bit KV cache: spec_tree_verify_attn_kv4 / spec_kv_commit_kv4 / spec_kv_read_kv4.
 *   ("EAGLE-3 paper explainer" (0h-n0), operations section, model-optimisation list:
 *   quantisation and PagedAttention KV-cache tuning to cut GPU memory. The page names no
 *   format; this library reads it as follows.)
 *   Elements are E2M1 codes (1 sign, 2 exponent, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6);
 *   every 16 consecutive elements of a token's head share a scale, an OCP E4M3 code; an element
 *   of KV head g stands for code * scale * kv_scale[0][g] in K, kv_scale[1][g] in V.
 *   kv_pool    uint8 [num_pages][hkv][2304], 16-byte aligned. The record of a page and head
 *              holds 16 tokens of 128 elements:
 *                bytes    0 .. 1023  K codes  [4 parts of 32 elements][16 tokens][16 bytes],
 *                                    the even element in a byte's low half
 *                bytes 1024 .. 2047  V codes  [128 elements][8 bytes], the even token in a
 *                                    byte's low half
 *                bytes 2048 .. 2175  K scales [16 tokens][8 groups]
 *                bytes 2176 .. 2303  V scales [8 groups][16 tokens]
 *              (4.5 bits an element: 144 bytes a token and head, K and V, for 512 in bf16.)
 *   kv_scale   float32 [2][hkv], device memory, nullable (all 1): K scales, then V scales, which
 *              place E4M3's range. Each is read at every call as
 *              min(max(scale, 2^-50), 2^50) (0 and NaN read as 2^-50).
 *   page_size 16 and d 128 only, else SPEC_ERR_UNSUPPORTED.
 *
 * spec_tree_verify_attn_kv4 — spec_tree_verify_attn over a 4-bit pool.
 *   q, k_tree, v_tree, out  bf16;  hq / hkv: any group size up to 128 (it need not divide 128).
 *   Everything else as spec_tree_verify_attn; the tensors but kv_scale, lse and the int32 arrays 16-byte
 *   aligned, else SPEC_ERR_ARG. What a row may not see does not reach it: cache rows past
 *   prefix_len, tree nodes its mask bits leave out and nodes of other sequences may hold
 *   infinities, NaN or NaN scales. A row that does see a NaN or an infinity in k or v may be
 *   NaN in every element. A row that sees no key at all is 0 with lse = -infinity. Rows at or
 *   past qo_indptr[batch] are left as they were. The call never reads ahead of its wait
 *   (spec_set_early_reads does not concern it).
 *   ws          workspace of spec_workspace_size(SPEC_OP_ATTN_KV4, ...) bytes (256-byte
 *               aligned; any contents).
 *   Arithmetic: K and V are widened exactly; q, scaled per row, is exact in fp16 for elements within 2^31 of the
 *   row's largest; weights of the prefix are rounded to fp16 beside a row's largest of 2^5 at least, those of the
 *   tree to two bf16 terms; scores, sums and outputs in fp32, the result rounded once to bf16. (Products are summed
 *   before they are divided by the row sum: tree values up to 2^100 times the head's V scale stay in fp32's range.)
 *   SPEC_ERR_UNSUPPORTED where batch * hkv * (row tiles of max_nodes) * (blocks of max_prefix and max_nodes) passes
 *   2^30 (row tiles of 16 to 128 rows, blocks of 128 keys or 32 nodes), or max_prefix 2^31 - 1025.
 *   Device errors: SPEC_ERR_PAGE (the page is read as zeros), SPEC_ERR_CAPACITY (a tree
 *   past max_nodes, a prefix past max_prefix: that sequence's rows are left as they were),
 *   SPEC_ERR_INDEX (a node range that falls or is not within [0, total_nodes]: likewise, whatever the
 *   others' ranges), SPEC_ERR_TIMEOUT.
 *
 * spec_kv_commit_kv4 — spec_kv_commit from bf16 tree rows into a 4-bit pool.
 *   Every 16 elements x of a row: with a the largest finite |x| and f the head's kv_scale,
 *   s = E4M3(a / (6 f)) rounded to nearest, within [2^-9, 448]; each element becomes the E2M1
 *   code nearest to x / (s f) (ties to the even code, beyond +-6, and infinities, saturated).
 *   Quotients and products in IEEE fp32. A group that holds a NaN gets the NaN scale code 0x7F (its
 *   NaN elements the code 0). Rows are written once: no later commit changes their
 *   codes or scales, and nothing else of a page changes. A page that receives rows must belong to
 *   one sequence of the call. The other arguments, the checks and the device errors are those of
 *   spec_kv_commit with dtype = SPEC_BF16 (a sequence whose node range does not lie in
 *   [0, total_nodes) is SPEC_ERR_INDEX).
 *
 * spec_kv_read_kv4 — rows of the cache brought back in bf16 (for a reader of bf16 rows, a move
 *   to another cache). Row i of sequence b, i < n_b = qo_indptr[b+1] - qo_indptr[b], is logical
 *   slot first[b] + i: k_out[qo_indptr[b] + i] and v_out likewise, [total_rows][hkv][128] bf16,
 *   code * scale * kv_scale rounded to fp32, then to bf16.
 *   first, qo_indptr  int32 [batch], [batch+1];  total_rows >= qo_indptr[batch].
 *   Rows at or past qo_indptr[batch] are left as they were. Device errors: SPEC_ERR_INDEX (a
 *   negative first or count, rows outside total_rows: that sequence's rows are left as they were),
 *   SPEC_ERR_CAPACITY (a slot past max_pages), SPEC_ERR_PAGE (a page id outside the pool): in both
 *   cases those rows are zeros. Each sequence is judged by its own numbers, whether or not qo_indptr rises; of
 *   rows that two ranges share it is not said whose they hold.
 */
int spec_tree_verify_attn_kv4(const void* q, const uint8_t* kv_pool, const float* kv_scale, int num_pages,
                              int page_size, const int32_t* page_table, int max_pages,
                              const int32_t* prefix_len, int max_prefix, const void* k_tree,
                              const void* v_tree, const uint64_t* mask, const int32_t* qo_indptr, int batch,
                              int total_nodes, int max_nodes, int hq, int hkv, int d, float sm_scale,
                              void* out, float* lse, void* ws, size_t ws_bytes, int32_t* dev_status,
                              void* stream);
int spec_kv_commit_kv4(const void* k_tree, const void* v_tree, const int32_t* path, int path_cap,
                       const int32_t* accept_len, const int32_t* qo_indptr, const int32_t* page_table,
                       int max_pages, int num_pages, int page_size, const int32_t* prefix_len,
                       int32_t* seq_len_out, uint8_t* kv_pool, const float* kv_scale, int batch,
                       int total_nodes, int hkv, int d, int32_t* dev_status, void* stream);
int spec_kv_read_kv4(const uint8_t* kv_pool, const float* kv_scale, int num_pages, int page_size,
                     const int32_t* page_table, int max_pages, const int32_t* first,
                     const int32_t* qo_indptr, int batch, int total_rows, int hkv, int d, void* k_out,
                     void* v_out, int32_t* dev_status, void* stream);

/*
 * spec_token_logprobs — the log probability of each given token, its rank, the entropy of its
 *   distribution and the most probable tokens, from rows of logits.
 *   ("Accelerating Sonar", draft-target section: acceptance is determined by comparing complete
 *   probability distributions; what a serving call reports beside the accepted tokens.)
 *   Entry (b, i), i < path_cap, has the row x of logits and the token t = tokens[b][i]:
 *     p = softmax(x / temperature),  logprob = ln p_t,  entropy = -sum p ln p,
 *     rank = 1 + the tokens before t in the order (larger logit first, lower id on ties),
 *     top_ids / top_logprobs = the first topk tokens of that order and their ln p.
 *   With a path (straight from spec_accept): the row is qo_indptr[b] + path[b][i] for
 *   i <= accept_len[b], tokens = out_tokens (the accepted tokens, then the bonus); entries past it get
 *   logprob, entropy and top_logprobs 0, rank and top_ids -1. Without one (path and accept_len NULL):
 *   entry (b, i) is row b * path_cap + i (a prompt's rows: batch = rows, path_cap = 1).
 *
 *   dtype      SPEC_F32 or SPEC_BF16, of logits (all sums are in fp32).
 *   logits     [total_rows] rows of vocab elements, row_stride (>= vocab) elements apart; any
 *              alignment of the rows. Device memory, or pinned host memory as for spec_accept.
 *   tokens     int32 [batch][path_cap]; NULL where neither logprob nor rank is asked for.
 *   logprob, entropy  float [batch][path_cap];  rank  int32 [batch][path_cap];
 *   top_ids    int32 [batch][path_cap][topk];  top_logprobs  float likewise. Any may be NULL.
 *   topk       in [0, 32]; vocab <= 2^24; temperature positive, at most 3e38, with a finite
 *              log2(e) / temperature in fp32 (4.25e-39 and up), else SPEC_ERR_ARG.
 *   The difference of a logit and its row's largest is taken in fp32 before it is divided: past fp32's
 *   largest number it counts as infinite, whatever the temperature.
 *   A token of probability 0 (logit -infinity) is no alternative: places that are left get id -1
 *   and -infinity. A row with a NaN or +infinity, or with nothing above -infinity, has NaN for
 *   logprob and entropy; its ids and rank mean nothing.
 *   Device errors: SPEC_ERR_INDEX (accept_len outside [0, path_cap), a path node outside the
 *   sequence's tree or the rows: that entry, or that sequence's entries, as past the path; a token
 *   outside [0, vocab): that entry's logprob is 0 and its rank -1).
 */
int spec_token_logprobs(int dtype, const void* logits, long long row_stride, int vocab, const int32_t* tokens,
                        const int32_t* path, const int32_t* accept_len, const int32_t* qo_indptr,
                        int batch, int path_cap, int total_rows, float temperature, int topk,
                        float* logprob, int32_t* rank, float* entropy, int32_t* top_ids,
                        float* top_logprobs, int32_t* dev_status, void* stream);

/*
 * spec_qk_norm_rope — queries and keys of the tree's nodes from the projection's output:
 *   normed per head, rotated to their positions, written in the layouts the attention
 *   reads (and the values copied into theirs).
 *   For node t of sequence b the position is prefix_len[b] + depth[t], the place the node
 *   takes if its path is accepted. Every query and key head x (d elements):
 *     y = x / sqrt(mean(x^2) + eps) * weight   (weight NULL: y = x), then the rot_dim / 2
 *     pairs (u, v) of its first rot_dim elements become (u c - v s, v c + u s) with the
 *     cosine c and sine s of the position's table row; later elements pass through.
 *   Pair i is (y[i], y[i + rot_dim / 2]), or (y[2i], y[2i + 1]) where interleaved != 0.
 *   fp32 arithmetic, rounded once.
 *
 *   dtype      SPEC_F32 or SPEC_BF16, of every tensor but the table.
 *   q_in       [total_nodes] rows of hq * d elements, q_stride elements apart (the heads of
 *              a fused projection can be read in place); k_in, v_in likewise with hkv * d.
 *              v_in / v_out: both or neither. Strides: multiples of 16 bytes.
 *   q_weight, k_weight  [d], either NULL.
 *   cos_sin    float [max_pos][rot_dim]: rot_dim / 2 cosines, then rot_dim / 2 sines of
 *              each position (NULL where rot_dim = 0).
 *   depth      int32 [total_nodes] from spec_build_tree_mask; NULL: node i of a sequence
 *              stands i tokens past its prefix (a chain, a prompt chunk).
 *   q_out      [total_nodes][hq][d];  k_out, v_out  [total_nodes][hkv][d]. An output may be
 *              its own input where the strides agree; no other overlap.
 *   d and rot_dim multiples of 16, d <= 512, rot_dim <= d, at most 4096 heads, else
 *   SPEC_ERR_UNSUPPORTED; every tensor 16-byte aligned, eps >= 0, else SPEC_ERR_ARG.
 *   Device errors: SPEC_ERR_INDEX (a negative depth or prefix, a position outside
 *   [0, max_pos): that node's outputs are left as they were). Rows at or past
 *   qo_indptr[batch] are left as they were.
 */
int spec_qk_norm_rope(int dtype, const void* q_in, long long q_stride, const void* k_in,
                      long long k_stride, const void* v_in, long long v_stride, const void* q_weight,
                      const void* k_weight, float eps, const float* cos_sin, int max_pos, int rot_dim,
                      int interleaved, const int32_t* prefix_len, const int32_t* depth,
                      const int32_t* qo_indptr, int batch, int total_nodes, int hq, int hkv, int d,
                      void* q_out, void* k_out, void* v_out, int32_t* dev_status, void* stream);

/*
 * spec_page_table_resize — the page-table rows a step needs, from the lengths on the
 *   device, and the slots of its tokens. (The commit leaves seq_len on the device; with
 *   this call the next step's pages are given out there too, with no host round trip.)
 *   Sequence b needs ceil((seq_len[b] + n_b) / page_size) pages, n_b = qo_indptr[b+1] -
 *   qo_indptr[b]. What its row lacks is taken off the stack of free pages; with
 *   shrink != 0 the row's entries past its need go back onto it (a finished sequence: 0
 *   tokens). Returned pages are pushed first, by rising sequence and entry; then the
 *   sequences, in order, each pop their pages while all of a sequence's fit in what is
 *   left (the first that does not fit, and every later one that asks, get none and keep
 *   their row: SPEC_ERR_CAPACITY).
 *
 *   seq_len    int32 [batch]   tokens in the cache
 *   qo_indptr  int32 [batch+1] the step's nodes (counts may be 0)
 *   held, held_out  int32 [batch]  pages of each row before and after; may be one buffer
 *   page_table int32 [batch][max_pages] (in/out)  entries held .. need-1 of a growing row are
 *              written, nothing else; entries past held_out[b] mean nothing
 *   free_pages int32 [num_pages] (in/out)  the stack: places 0 .. n_free-1 hold free pages
 *   n_free, n_free_out  int32 [1]  its height before and after; may be one buffer
 *   slot_map   int64 [total_nodes] (out, nullable)  node i of sequence b as the token at
 *              seq_len[b] + i: page * page_size + row, or -1 where the row does not reach
 *              (and for every node of a sequence with SPEC_ERR_INDEX).
 *              Rows at or past qo_indptr[batch] are left as they were.
 *   batch <= 4096 and batch * max_pages < 2^31, else SPEC_ERR_UNSUPPORTED.
 *   Device errors: SPEC_ERR_INDEX (a negative length or count, held outside
 *   [0, max_pages]), SPEC_ERR_CAPACITY (a need past max_pages: in both cases that row
 *   stays; too few free pages; a stack that would be outside [0, num_pages], then nothing
 *   moves), SPEC_ERR_PAGE (a page id outside [0, num_pages)). No page may stand twice in
 *   the rows and the stack.
 */
int spec_page_table_resize(const int32_t* seq_len, const int32_t* qo_indptr, const int32_t* held,
                           int32_t* page_table, int max_pages, int32_t* free_pages, int num_pages,
                           const int32_t* n_free, int page_size, int shrink, int batch,
                           int total_nodes, int32_t* held_out, int32_t* n_free_out,
                           long long* slot_map, int32_t* dev_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H */
