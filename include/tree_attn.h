/*
 * tree_attn.h -- C ABI of the GB300 (sm_103a) batched tree-attention library
 * (libtreeattn.so).
 *
 * The operation is the one the page "tree_attn.py"
 * (python/tvm/relax/frontend/nn/llm/tree_attn.py) generates as
 * ``batch_tree_attn`` (``tree_attn`` for GPUs, ``tree_attn_cpu`` for CPUs):
 * ragged, multi-sequence grouped-query attention in which q row r of
 * sequence b attends kv column c iff c lies in the sequence's causal prefix
 * or c's tree node is an ancestor-or-self of r's tree node, decided from the
 * DFS [enter, exit) intervals of ``_check_tree_order`` on that page.  RoPE
 * (``_rope`` on the page "_kernel_common.py",
 * python/tvm/relax/frontend/nn/llm/_kernel_common.py) is optionally applied
 * to q and k as they are loaded.  The outputs are the attention output and
 * the base-2 log-sum-exp (``m + log2(d)``, the ``lse_store`` epilogue).
 *
 * Conventions shared by every entry point:
 *   - Pointers named "device" are CUDA device pointers owned by the caller;
 *     the library never frees them and keeps no reference after returning.
 *   - ``stream`` is a ``cudaStream_t`` passed as ``void*`` (NULL = the
 *     legacy default stream).  Launching entry points are asynchronous on it
 *     and never synchronise the host.
 *   - Errors detectable from the arguments alone are returned synchronously
 *     before anything is launched.  The contents of device index arrays are
 *     not read on the host in the launching calls (see
 *     ``tree_attn_check_inputs``).
 *   - Only the current CUDA device is used.
 */
#ifndef TREE_ATTN_H_
#define TREE_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  TA_OK = 0,
  TA_ERR_INVALID_ARGUMENT = 1, /* null pointer, bad size, bad scalar         */
  TA_ERR_UNSUPPORTED = 2,      /* valid but not built: head_dim, group size  */
  TA_ERR_CUDA = 3,             /* a CUDA runtime/driver call failed          */
  TA_ERR_DEVICE_TIMEOUT = 4    /* a bounded device-side wait expired         */
} ta_status;

typedef enum { TA_FP16 = 0, TA_BF16 = 1 } ta_dtype;

/* Problem sizes.  The page's PrimFunc takes these from buffer shapes and
 * generator constants (h_kv, h_q, d, dtype); a C ABI passes them explicitly.
 *   batch_size  B, number of sequences (>= 1)
 *   total_q     rows of q / out / lse           (q_indptr[B])
 *   total_kv    rows of k / v                   (kv_indptr[B])
 *   total_tree  rows of tree_order              (mn_indptr[B])
 *   h_q, h_kv   heads; h_q % h_kv == 0, group size g = h_q / h_kv <= 128
 *   head_dim    64 or 128
 *   dtype       element type of q, k, v and out
 *   rotary_mode 0 or 1: whether the calls this workspace serves apply RoPE
 *               (it sizes the workspace; it must match their rotary_mode) */
typedef struct {
  int32_t batch_size;
  int32_t total_q;
  int32_t total_kv;
  int32_t total_tree;
  int32_t h_q;
  int32_t h_kv;
  int32_t head_dim;
  ta_dtype dtype;
  int32_t rotary_mode;
} ta_dims;

/* Bytes of device workspace ``tree_attn`` needs for these sizes (a multiple
 * of 256; 0 on invalid dims).  The workspace holds the per-launch work plan
 * (tile classes, the cost-ordered work queue), a device status word and,
 * with RoPE, the cos/sin table of the kv tokens and the rotated k
 * (total_kv * h_kv * head_dim elements, rotated once per call instead of
 * once per q tile that reads it), and when tree_attn splits the kv range
 * (tree_attn_auto_split_chunks > 1) the split-KV partial states, as
 * tree_attn_split_workspace_size(dims, that cap).  It depends on the dims and
 * the current device's SM count only, so one allocation serves every call
 * with the same dims on that kind of GPU. */
size_t tree_attn_workspace_size(const ta_dims* dims);

/* The split-KV chunk cap tree_attn uses for these dims on the current device
 * (0 on invalid dims).  1: no split.  tree_attn splits when the work units
 * (a unit is 2 q tiles of 128 / g rows of one sequence and kv head) number
 * fewer than the SMs even at their lower bound ceil(total_q / (256 / g)) x
 * h_kv, while the sequences average at least 2048 kv rows; the cap is then
 * ceil(4 x SMs / ((ceil(total_q / (256 / g)) + batch_size) x h_kv)) clamped
 * to 2..16 (about four work records per SM), and the plan picks the chunk
 * length (chunk_tiles 0 of tree_attn_split).  A split result equals the
 * unsplit one up to float32 rounding order (merge of base-2 LSE states). */
int32_t tree_attn_auto_split_chunks(const ta_dims* dims);

/* Batched tree attention.  Layouts (all row-major, contiguous, device):
 *   q               [total_q, h_q, head_dim]   dtype
 *   q_indptr        [B+1] int32, q rows of sequence b are
 *                   q_indptr[b] .. q_indptr[b+1]-1
 *   k, v            [total_kv, h_kv, head_dim] dtype
 *   kv_indptr       [B+1] int32, kv rows of sequence b
 *   q_rope_position [total_kv] int32, the RoPE position of every kv token;
 *                   q row r of sequence b takes the position of its own tree
 *                   node's kv slot.  May be NULL iff rotary_mode == 0.
 *   mn_indptr       [B+1] int32, tree nodes of sequence b are tree_order
 *                   rows mn_indptr[b] .. mn_indptr[b+1]-1
 *   tree_order      [total_tree][2] int32, (enter, exit) DFS interval of each
 *                   node, exit exclusive
 *   out             [total_q, h_q, head_dim] dtype   (written)
 *   lse             [total_q, h_q] float32, base-2 log-sum-exp (written);
 *                   natural-log LSE = lse * ln 2
 * For sequence b let qo = q rows, kv = kv rows, T = tree nodes; the last T kv
 * rows are the tree nodes in node order, the first kv - T the prefix, and the
 * q rows are the last qo tree nodes (0 <= qo <= T <= kv).  A q row none of
 * whose columns is visible gets out = 0 and lse = -inf.
 *   rotary_mode     0: no RoPE; 1: rotate-half RoPE on q and k at load time
 *                   (any other value, or one that differs from
 *                   dims->rotary_mode, is TA_ERR_INVALID_ARGUMENT)
 *   rope_scale      position multiplier (finite)
 *   rope_theta      RoPE base (finite, > 0)
 *   sm_scale        score scale (finite), typically 1/sqrt(head_dim)
 *   workspace       device buffer of >= tree_attn_workspace_size(dims) bytes,
 *                   256-byte aligned, zero-filled once before its first use
 *                   (e.g. cudaMemset); every call leaves it ready for the
 *                   next one.  Calls that may overlap on the GPU must use
 *                   distinct workspaces.
 * q, k, v and out must be 16-byte aligned.  Returns TA_OK once the work is
 * enqueued; device-side failures are reported by tree_attn_device_status.
 * When tree_attn_auto_split_chunks(dims) > 1 the call is tree_attn_split with
 * that cap and chunk_tiles 0 (plan, attention and merge kernels). */
ta_status tree_attn(const void* q, const int32_t* q_indptr, const void* k, const void* v,
                    const int32_t* kv_indptr, const int32_t* q_rope_position,
                    const int32_t* mn_indptr, const int32_t* tree_order, void* out,
                    float* lse, int32_t rotary_mode, float rope_scale, float rope_theta,
                    float sm_scale, const ta_dims* dims, void* workspace,
                    size_t workspace_bytes, void* stream);

/* The two launches of unsplit tree_attn (these never split the kv range), for
 * callers that reuse one tree layout across calls (every layer of a model
 * verifies the same draft tree):
 *   tree_attn_plan  enumerates the (sequence, q tile) work items, classifies
 *                   every (q tile, kv tile) pair as empty / partial / full
 *                   from the DFS intervals and orders the items
 *                   longest-first; it reads only the index arrays (the RoPE
 *                   arguments are validated, not used).
 *   tree_attn_run   with rotary_mode == 1 the RoPE of every kv token (its
 *                   cos/sin from q_rope_position, rope_scale and rope_theta,
 *                   and its rotated keys), then the attention kernel proper,
 *                   consuming the plan that the last tree_attn_plan (or
 *                   tree_attn) left in ``workspace``.
 * tree_attn_run must follow a plan made on the same workspace with the same
 * dims, index-array contents, positions, rotary_mode, rope_scale and
 * rope_theta; q, k, v, out, lse and sm_scale may change between runs.
 * Arguments mean what they mean for tree_attn; both are asynchronous. */
ta_status tree_attn_plan(const int32_t* q_indptr, const int32_t* kv_indptr,
                         const int32_t* q_rope_position, const int32_t* mn_indptr,
                         const int32_t* tree_order, int32_t rotary_mode, float rope_scale,
                         float rope_theta, const ta_dims* dims, void* workspace,
                         size_t workspace_bytes, void* stream);

ta_status tree_attn_run(const void* q, const void* k, const void* v, const int32_t* q_indptr,
                        const int32_t* kv_indptr, const int32_t* q_rope_position,
                        const int32_t* mn_indptr, const int32_t* tree_order, void* out,
                        float* lse, int32_t rotary_mode, float rope_scale, float rope_theta,
                        float sm_scale, const ta_dims* dims, void* workspace,
                        size_t workspace_bytes, void* stream);

/* Allocation-free variant of tree_attn (the pages have no counterpart: it is
 * a deployment convenience of this library).  Some callers cannot allocate
 * device memory: a serving engine that has handed all free HBM to its own
 * pool (typically the KV cache) and forbids further cudaMalloc, or a host
 * framework whose plugins may not call allocation routines because they
 * synchronise the device or escape the framework's memory accounting.  This
 * entry point takes the same arguments as tree_attn minus the workspace and
 * uses a static device array of 32 MiB (held by every GPU that loads the
 * library until the process exits) as its workspace; it calls no cudaMalloc,
 * cudaFree or other allocating routine.
 *   - It never splits the kv range (tree_attn_split with max_chunks 1).
 *   - Problems whose unsplit workspace (tree_attn_split_workspace_size(dims,
 *     1)) exceeds 32 MiB are rejected
 *     with TA_ERR_UNSUPPORTED before anything is enqueued.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress); make that first call before any stream capture.
 *   - Every call clears the array's work counters (two cudaMemsetAsync on
 *     ``stream``) and then runs tree_attn on it.  All calls share the one
 *     array, so calls that may overlap on the GPU (different streams without
 *     ordering between them) race and must not be issued. */
ta_status tree_attn_noalloc(const void* q, const int32_t* q_indptr, const void* k, const void* v,
                            const int32_t* kv_indptr, const int32_t* q_rope_position,
                            const int32_t* mn_indptr, const int32_t* tree_order, void* out,
                            float* lse, int32_t rotary_mode, float rope_scale, float rope_theta,
                            float sm_scale, const ta_dims* dims, void* stream);

/* Synchronises ``stream`` and reads and clears the device status word that
 * earlier tree_attn_noalloc calls on the current device left in the static
 * scratch array (the caller never sees that array's address): TA_OK,
 * TA_ERR_DEVICE_TIMEOUT if a bounded wait expired, TA_ERR_INVALID_ARGUMENT if
 * the index arrays broke the layout rules (nothing was computed), TA_ERR_CUDA
 * on a CUDA error.  Like tree_attn_device_status, but for the array. */
ta_status tree_attn_noalloc_device_status(void* stream);

/* ---- Paged KV cache ------------------------------------------------------
 * The same tree attention with K and V held in a paged cache, as the page
 * "tree_attn.py" generates it in ``tree_attn_with_paged_kv_cache`` (GPU) and
 * ``tree_attn_with_paged_kv_cache_cpu``; kv lengths follow
 * ``_get_kv_chunk_len`` of the page "_kernel_common.py" without a sliding
 * window (the pages disable it for tree attention).
 *   batch_size, total_q, total_tree, h_q, h_kv, head_dim, dtype
 *               as in ta_dims
 *   num_pages   pages in the pool (>= 1): the pages buffer is
 *               [num_pages, 2, h_kv, 16, head_dim]
 *   nnz_pages   entries of page_values (= page_indptr[B]) */
typedef struct {
  int32_t batch_size;
  int32_t total_q;
  int32_t total_tree;
  int32_t h_q;
  int32_t h_kv;
  int32_t head_dim;
  ta_dtype dtype;
  int32_t num_pages;
  int32_t nnz_pages;
} ta_paged_dims;

/* Bytes of device workspace tree_attn_paged needs (0 on invalid dims); the
 * same rules as tree_attn_workspace_size. */
size_t tree_attn_paged_workspace_size(const ta_paged_dims* dims);

/* Tree attention over a paged KV cache (one call: plan and run).  Layouts
 * (device, contiguous):
 *   q, out, lse, q_indptr, mn_indptr, tree_order   as for tree_attn
 *   pages        [num_pages, 2, h_kv, 16, head_dim] dtype: plane 0 holds K,
 *                plane 1 holds V, 16 kv slots per page
 *   page_indptr  [B+1] int32: sequence b owns page_values[page_indptr[b] ..
 *                page_indptr[b+1]-1], in kv order
 *   page_values  [nnz_pages] int32 physical page indices (an index outside
 *                [0, num_pages) reads zeros)
 *   length_info  [B] int32, the number of slots used in each sequence's last
 *                page (1..16 when the sequence owns a page); sequence b has
 *                kv = (pages - 1) * 16 + length_info[b] rows, 0 without pages
 * kv row r of sequence b is slot r % 16 of page page_values[page_indptr[b] +
 * r / 16]; the tree mask, the q rows and the outputs are those of tree_attn
 * with that kv length.  Slots past a sequence's kv length are never used (their
 * contents may be anything, NaN included).  The pages assert that this kernel
 * has no RoPE: rotary_mode must be 0 (else TA_ERR_UNSUPPORTED), and the pages'
 * position arguments (k_rope_pos_offset, q_rope_position) are therefore not
 * taken.  Inconsistent page tables (indptr not ending at nnz_pages, a
 * length_info outside 1..16) are reported by tree_attn_device_status and
 * nothing is computed.  q, pages and out must be 16-byte aligned; the
 * workspace follows tree_attn's rules.  Asynchronous on stream. */
ta_status tree_attn_paged(const void* q, const int32_t* q_indptr, const void* pages,
                          const int32_t* page_indptr, const int32_t* page_values,
                          const int32_t* length_info, const int32_t* mn_indptr,
                          const int32_t* tree_order, void* out, float* lse, int32_t rotary_mode,
                          float sm_scale, const ta_paged_dims* dims, void* workspace,
                          size_t workspace_bytes, void* stream);

/* ---- Serving a paged KV cache ----------------------------------------------
 * What a decoding loop does to the cache that tree_attn_paged reads, besides
 * verifying trees over it: append new tokens (norms and RoPE of their queries
 * and keys in the same pass), attend one new token per sequence, drop the
 * rejected nodes of a verified tree, copy pages (forking a sequence whose last
 * page is partly filled).  The pages have no counterpart; the cache layout and
 * the page table are those of tree_attn_paged:
 *   pages        [num_pages, 2, h_kv, 16, head_dim] dtype
 *   page_indptr  [B+1] int32, page_values [nnz_pages] int32,
 *   length_info  [B] int32 (1..16 when the sequence owns a page)
 * except that page_values may be longer than the table: page_indptr[B] <=
 * nnz_pages (nnz_pages is the array's capacity).
 *   batch_size   B, 1..16384
 *   h_q, h_kv, head_dim, dtype, num_pages   as in ta_paged_dims
 *   nnz_pages    entries of page_values (16 * nnz_pages <= INT32_MAX, nnz_pages *
 *                h_kv < 2^30) */
typedef struct {
  int32_t batch_size;
  int32_t h_q;
  int32_t h_kv;
  int32_t head_dim;
  ta_dtype dtype;
  int32_t num_pages;
  int32_t nnz_pages;
} ta_cache_dims;

/* Bytes of device workspace each of the calls below needs for these dims (a
 * multiple of 256; 0 on invalid or unsupported dims).  It holds the device
 * status word (tree_attn_device_status), for tree_attn_decode_paged the partial
 * states of sequences that several CTAs share, and for tree_attn_copy_pages a
 * mark per page of the pool.  tree_attn's workspace
 * rules apply: 256-byte aligned, zero-filled once before its first use, left
 * ready for the next call by every call, one workspace per set of calls that
 * may overlap on the GPU (two graphs that may replay at once are such calls).
 * It depends on the dims and the current device's SM count only; calls of this
 * section that share one may differ in any of the dims (it holds the largest). */
size_t tree_attn_cache_workspace_size(const ta_cache_dims* dims);

typedef enum {
  TA_ROPE_HALF = 1,        /* pairs (j, j + rotary_dim / 2)                   */
  TA_ROPE_INTERLEAVED = 2  /* pairs (2 j, 2 j + 1)                            */
} ta_rope_layout;

/* A rotation, filled by tree_attn_rope_init and passed to
 * tree_attn_append_paged.  Pair j of a token at position p turns by
 * p * turns[j] / 2^64 full turns (mod 1): the product of a position and a
 * 64-bit fixed-point frequency keeps its fraction of a turn exactly, so far
 * positions lose nothing. */
typedef struct {
  int32_t layout;       /* ta_rope_layout                                     */
  int32_t rotary_dim;   /* elements rotated, from the head's first            */
  float magnitude;      /* factor of cos and sin                              */
  uint64_t turns[64];
} ta_rope;

/* Fills ``rope`` on the host.  layout: ta_rope_layout.  rotary_dim: a multiple
 * of 16 in 16..128.  Pair j (of rotary_dim / 2) turns by
 *   angle = position * scale * f_j,   f_j = theta^(-2 j / rotary_dim),
 * or f_j = inv_freq[j] (a host array of rotary_dim / 2 doubles) when inv_freq
 * is not NULL, which carries any rescaling of frequencies for long contexts.
 * scale and every f_j finite, theta finite and > 0 (ignored with inv_freq),
 * magnitude finite (1 for a plain rotation). */
ta_status tree_attn_rope_init(ta_rope* rope, int32_t layout, int32_t rotary_dim, double theta,
                              double scale, float magnitude, const double* inv_freq);

/* Appends tokens to the cache.  The page table describes the cache after the
 * call: the last n_b = append_indptr[b+1] - append_indptr[b] kv rows of
 * sequence b receive its n_b new tokens, in order.
 *   q, k, v        rows of total_new tokens, [h_q, head_dim] and
 *                  [h_kv, head_dim] contiguous per token; q_stride, k_stride,
 *                  v_stride elements from one token to the next (multiples of
 *                  8, at least the row), so that views of one fused
 *                  projection need no copy
 *   append_indptr  [B+1] int32, from 0 to total_new
 *   positions      [total_new] int32, any value (may be NULL iff rope is NULL)
 *   q_weight, k_weight  [head_dim] dtype, or NULL for no norm: per head
 *                  x <- x * w / sqrt(mean(x^2) + norm_eps)
 *   norm_eps       finite, >= 0
 *   rope           a filled ta_rope (read during the call), or NULL
 *   q_out          [total_new, h_q, head_dim] contiguous (written): q after
 *                  norm and rotation.  It may be q itself (q_stride = h_q *
 *                  head_dim); otherwise it overlaps none of the inputs.
 * k after norm and rotation goes to plane 0 of its slot, v as it is to
 * plane 1.  Norm and rotation are float32, rounded once to dtype; cos and sin
 * are those of the angle itself, not of an angle rounded to float32 as in
 * tree_attn's rotary_mode 1 (the two differ by up to position * 2^-23).
 * Every other slot of the cache keeps its contents.  No two sequences may
 * share a page that receives tokens.  A token whose sequence's tables are
 * inconsistent (or whose page is outside the pool) is not written to the
 * cache, which tree_attn_device_status reports.  Pointers 16-byte aligned.
 * total_new times the steps of 512 / head_dim heads of a token's q, k and v
 * must fit an int32 (else TA_ERR_UNSUPPORTED).  Asynchronous on stream. */
ta_status tree_attn_append_paged(const void* q, int64_t q_stride, const void* k,
                                 int64_t k_stride, const void* v, int64_t v_stride,
                                 int32_t total_new, const int32_t* append_indptr,
                                 const int32_t* positions, const void* q_weight,
                                 const void* k_weight, float norm_eps, const ta_rope* rope,
                                 void* pages, const int32_t* page_indptr,
                                 const int32_t* page_values, const int32_t* length_info,
                                 void* q_out, const ta_cache_dims* dims, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* Attention of one token per sequence over the paged cache: q [B, h_q,
 * head_dim], row b attends every kv row of sequence b (its own key and value
 * were appended before).  Writes out [B, h_q, head_dim] and the base-2 lse
 * [B, h_q] (a sequence without kv rows gets out = 0 and lse = -inf).  The kv
 * rows of the whole batch are split evenly over the GPU, whatever the
 * sequences' lengths, and the parts merged through their lse; the result does
 * not depend on timing.  Weights count as positive however small: where an
 * element of a sequence's values is infinite or NaN in some rows, the element
 * of out is the sum of those, and all others are as without them.  A page
 * index outside the pool reads zeros and slots past a sequence's length are
 * never used, as in tree_attn_paged.
 * Inconsistent page tables are reported by tree_attn_device_status and
 * nothing is computed.  h_q / h_kv <= 128; q, pages and out 16-byte aligned.
 * Asynchronous on stream. */
ta_status tree_attn_decode_paged(const void* q, const void* pages, const int32_t* page_indptr,
                                 const int32_t* page_values, const int32_t* length_info,
                                 void* out, float* lse, float sm_scale,
                                 const ta_cache_dims* dims, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* Keeps the accepted nodes of verified trees and drops the others.  The last
 * T = mn_indptr[b+1] - mn_indptr[b] kv rows of sequence b are its tree's nodes
 * (as in tree_attn_paged); of those, accept_nodes[accept_indptr[b] ..
 * accept_indptr[b+1]-1] -- strictly ascending node indices, a of them -- move
 * to the first a tree rows: row kv - T + accept_nodes[j] goes to row
 * kv - T + j, keys and values of every head.  The sequence then has
 * kv - T + a rows.  Writes the new table (none of these arrays may overlap the
 * old table):
 *   new_page_indptr [B+1], new_length_info [B] (0 for a sequence left without
 *                   pages), new_page_values [nnz_pages]: each sequence's first
 *                   pages, in order (entries past new_page_indptr[B] keep
 *                   their contents)
 *   freed_pages     [nnz_pages]: the pages each sequence no longer needs, in
 *                   table order; num_freed [1] their number (entries past it
 *                   keep their contents)
 * total_accept = accept_indptr[B].  Pages that receive rows belong to one
 * sequence only.  When an indptr array, a length or a count (0 <= a <= T <= kv)
 * is inconsistent nothing is written; a sequence whose accept_nodes are not
 * ascending within [0, T), or reach a page outside the pool, keeps its rows
 * as they are; tree_attn_device_status reports either.  pages 16-byte
 * aligned.  Asynchronous on stream. */
ta_status tree_attn_compact_paged(void* pages, const int32_t* page_indptr,
                                  const int32_t* page_values, const int32_t* length_info,
                                  const int32_t* mn_indptr, const int32_t* accept_indptr,
                                  const int32_t* accept_nodes, int32_t total_accept,
                                  int32_t* new_page_indptr, int32_t* new_page_values,
                                  int32_t* new_length_info, int32_t* freed_pages,
                                  int32_t* num_freed, const ta_cache_dims* dims,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* Copies whole pages within the pool: page dst_pages[i] becomes a copy of page
 * src_pages[i], i < n (int32 device arrays).  Only the pool's dims are used
 * (num_pages, h_kv, head_dim).  A pair that names a page outside the pool, or
 * whose dst_pages[i] is also another pair's source or destination, is not
 * copied, and tree_attn_device_status reports it; the other pairs are.
 * src_pages[i] == dst_pages[i] leaves the page as it is.  pages 16-byte
 * aligned.  Asynchronous on stream. */
ta_status tree_attn_copy_pages(void* pages, const int32_t* src_pages, const int32_t* dst_pages,
                               int32_t n, const ta_cache_dims* dims, void* workspace,
                               size_t workspace_bytes, void* stream);

/* ---- Split-KV ------------------------------------------------------------
 * The same tree attention with the kv tiles of long (sequence, q tile) pairs
 * cut into chunks that run as separate work items, so that a batch of few
 * but long sequences (a long shared prefix before a small draft tree) still
 * covers every SM.  The pages have no split-KV; it rests on the base-2 LSE
 * their ``lse_store`` epilogue emits (page "tree_attn.py"), which is what
 * merges attention over disjoint kv sets: each chunk writes its float32
 * partial output O_i / l_i and lse_i to the workspace, and a merge kernel
 * forms lse = log2(sum_i 2^lse_i) and out = sum_i 2^(lse_i - lse) O_i / l_i.
 * Results equal tree_attn's up to float32 rounding order (not bit for bit).
 *
 * Bytes of device workspace tree_attn_split needs for these dims and chunk
 * cap: tree_attn_workspace_size's plus, per possible work record
 * (((total_q + R - 1) / R + batch_size) * max_chunks of them, R the q rows per
 * tile), an h_kv x 128 x head_dim float32 partial output and its lse.
 * 0 on invalid dims or max_chunks outside 1..16. */
size_t tree_attn_split_workspace_size(const ta_dims* dims, int32_t max_chunks);

/* tree_attn with split-KV (one call: plan, attention, merge).  Arguments as
 * for tree_attn, plus:
 *   max_chunks   1..16, the most chunks one (sequence, q tile) pair is cut
 *                into (1: no split, the result is then tree_attn's exactly)
 *   chunk_tiles  target chunk length in kv tiles of 128 columns (>= 0); a
 *                pair whose kv tiles up to its last row's own slot number c
 *                gets min(max_chunks, ceil(c / chunk_tiles)) chunks.  0 lets
 *                the plan choose it from the batch's total work: a quarter of
 *                one SM's share of it, at least 8.
 * The chunks of a pair split the range of its kv tiles up to its last
 * non-empty tile into equal lengths.  workspace must hold at least
 * tree_attn_split_workspace_size(dims, max_chunks) bytes, with tree_attn's
 * other rules.  Asynchronous on stream. */
ta_status tree_attn_split(const void* q, const int32_t* q_indptr, const void* k, const void* v,
                          const int32_t* kv_indptr, const int32_t* q_rope_position,
                          const int32_t* mn_indptr, const int32_t* tree_order, void* out,
                          float* lse, int32_t rotary_mode, float rope_scale, float rope_theta,
                          float sm_scale, int32_t max_chunks, int32_t chunk_tiles,
                          const ta_dims* dims, void* workspace, size_t workspace_bytes,
                          void* stream);

/* Merges n_parts attention states over disjoint kv sets of the same rows
 * into the state over their union, with the base-2 LSE rule above (parts of
 * lse = -inf contribute nothing; a row whose parts are all -inf gets out = 0
 * and lse = -inf).  Layouts (device, contiguous):
 *   parts  [n_parts, rows, head_dim] dtype, each part normalised (as
 *          tree_attn's out); rows = total_q * h_q for tree_attn outputs
 *   lses   [n_parts, rows] float32, base-2
 *   out    [rows, head_dim] dtype (written);  lse [rows] float32 (written)
 * head_dim 64 or 128 (else TA_ERR_UNSUPPORTED); parts and out 16-byte
 * aligned.  Asynchronous on stream. */
ta_status tree_attn_merge_states(const void* parts, const float* lses, int32_t n_parts,
                                 int64_t rows, int32_t head_dim, ta_dtype dtype, void* out,
                                 float* lse, void* stream);

/* Synchronises ``stream``, reads and clears the device status word that the
 * kernels of earlier calls left in ``workspace`` (TA_ERR_DEVICE_TIMEOUT if a
 * bounded wait expired, TA_ERR_CUDA on a CUDA error, else TA_OK). */
ta_status tree_attn_device_status(void* workspace, void* stream);

/* Test hooks for the failure detection of this library (the pages have no
 * counterpart; their only checks are compile-time asserts such as
 * ``check_thread_limits`` on the page "_kernel_common.py").  Every hand-off
 * between the warps of the attention kernel is an mbarrier wait bounded by a
 * wall-clock limit (2 s); when one runs out the kernel records
 * TA_ERR_DEVICE_TIMEOUT in the workspace status word, lets its in-flight
 * copies and tensor-core operations land, frees its tensor memory and
 * returns, and tree_attn_device_status reports it.  These hooks let a test
 * take that path on purpose, for the attention kernels launched by later
 * calls made on the calling host thread:
 *   wait_limit_ns  the limit of every bounded wait (0: the default 2 s)
 *   stall          1: the MMA thread of every pipeline first waits on a
 *                  barrier that nothing arrives on, so that this wait runs
 *                  out after wait_limit_ns and every other warp then gives up
 *                  its own waits; 0: normal operation
 * Returns TA_ERR_INVALID_ARGUMENT for stall outside {0, 1}.  Not for
 * production use: a stalled call computes nothing. */
ta_status tree_attn_set_wait_hooks(uint64_t wait_limit_ns, int32_t stall);

/* Work scheduling of the attention kernels launched by later calls on the
 * calling host thread (page "tile_scheduler.py", the persistent schedulers and
 * ``ClusterLaunchControlScheduler``):
 *   mode 0  one CTA per SM; CTA b takes the b-th work unit of the
 *           longest-first list, then units from an atomic counter in the
 *           workspace, one fetched ahead of use;
 *   mode 1  (default) one CTA per possible work unit; CTA b takes unit b, and when it
 *           starts a unit it asks the hardware (clusterlaunchcontrol.try_cancel)
 *           to cancel the launch of a CTA that has not started yet and then
 *           takes that CTA's unit; CTAs past the last unit are cancelled the
 *           same way so that they do not launch empty.
 * Both give the same results bit for bit; mode 1 measured equal or faster on
 * every benchmarked workload (spec-decode 31.6 -> 30.4 us).  Returns
 * TA_ERR_INVALID_ARGUMENT for any other mode. */
ta_status tree_attn_set_scheduler(int32_t mode);

/* The CUDA runtime's description of the error behind the calling thread's
 * most recent TA_ERR_CUDA ("no error" if there was none; static storage).
 * A failure that has no CUDA error of its own (no device, a tensor map the
 * driver rejects) reads as an invalid-value error. */
const char* tree_attn_last_cuda_error(void);

/* Human-readable name of a status code (static storage). */
const char* tree_attn_status_string(ta_status s);

/* Test helper: dense visibility of every (q row, kv column) pair, evaluated
 * by the same device mask code the attention kernel uses.  Writes
 * vis[total_q][max_kv] bytes (1 = visible) where column c of q row
 * q_indptr[b] + r is kv column c of sequence b; columns >= kv_len are 0.
 * Index arrays and vis are device pointers.  max_kv must be >= every
 * sequence's kv length.  Asynchronous on stream. */
ta_status tree_attn_mask_dense(const int32_t* q_indptr, const int32_t* kv_indptr,
                               const int32_t* mn_indptr, const int32_t* tree_order,
                               int32_t batch_size, int32_t total_q, int32_t max_kv,
                               uint8_t* vis, void* stream);

/* Host-side validation of HOST copies of the index arrays, for callers and
 * tests: indptr arrays start at 0, are non-decreasing and end at the dims'
 * totals; per sequence 0 <= qo <= T <= kv; every interval has
 * 0 <= enter < exit <= T and the intervals of a sequence nest (any two are
 * disjoint or one contains the other).  ``q_rope_position`` is accepted for
 * symmetry with tree_attn and not inspected (every int32 position is valid).
 * Returns TA_OK or TA_ERR_INVALID_ARGUMENT. */
ta_status tree_attn_check_inputs(const int32_t* q_indptr, const int32_t* kv_indptr,
                                 const int32_t* mn_indptr, const int32_t* tree_order,
                                 const int32_t* q_rope_position, const ta_dims* dims);

#ifdef __cplusplus
}
#endif

#endif /* TREE_ATTN_H_ */
