// ta_launch.h -- internal interface between the C-ABI host code (ta_api.cu)
// and the kernel translation units (ta_plan.cu, ta_attn.cu, ta_merge.cu,
// ta_cache.cu, ta_decode.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <utility>

#include "ta_layout.h"

namespace ta {

// Launches a kernel of this library with programmatic dependent launch: its
// CTAs may be scheduled while the previous kernel on the stream is still
// running, and every kernel here executes pdl_wait() (griddepcontrol.wait)
// before it reads or writes anything that kernel may touch, so stream order
// is kept while launch latency and prologues overlap.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// Lets a kernel use ``bytes`` of dynamic shared memory, once per device
// (``done``: a bit for each; devices past the 64th are asked every time).
inline cudaError_t allow_shared(const void* kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Key rotation: the RoPE frequency denominators fl32(theta^(2i/d)) for
// i < d/2 (``_rope``, page "_kernel_common.py"; rounded once from float64 on
// the host), the position scale and the sizes.
struct KrotParams {
  float rope_den[64];
  float rope_scale;
  int total_kv, h_kv;
};

struct PlanParams {
  const int32_t* q_indptr;
  const int32_t* kv_indptr;
  const int32_t* mn_indptr;
  const int32_t* tree_order;
  // paged KV cache (paged != 0): kv rows come from 16-slot pages; kv_indptr
  // is unused, the kv length of sequence b is (pages - 1) * 16 + length_info[b]
  int paged;
  const int32_t* page_indptr;
  const int32_t* length_info;
  int nnz_pages;
  int batch, g, R, h_kv, head_dim, total_q, total_kv, total_tree;
  int64_t max_pairs;
  // split-KV: a pair's kv tiles are cut into up to max_chunks records of
  // about chunk_tiles tiles (0: chosen from the batch's total work so that
  // the items cover the ``pipes`` pipelines of the attention grid -- one
  // per SM -- a few times); max_chunks == 1 disables it
  int max_chunks, chunk_tiles, pipes;
  int4* merge;       // per pair (split-KV): q_row0, q rows, chunks, first record
  // one-call entry points: the plan kernel also does the key rotation of the
  // run (krot_kernel's work) on the warps the plan leaves idle.  rot: 0 none,
  // else 1 + 2 * (head_dim == 128) + (dtype == bf16)
  int rot;
  const uint32_t* rot_k;
  uint32_t* rot_out;
  const int32_t* rot_pos;
  float4* rot_cs;
  KrotParams kp;
  WsHeader* hdr;
  ItemRec* sorted;   // one record per (sequence, q tile) or chunk of one, longest first
  uint8_t* classes;
};

struct AttnParams {
  const int32_t* tree_order;
  void* out;
  float* lse;
  const ItemRec* sorted;
  const uint8_t* classes;
  const float2* rope_cs;   // [total_kv][head_dim / 2] cos/sin per kv token (RoPE)
  WsHeader* hdr;
  const int32_t* page_values;   // paged KV cache: physical page of each (sequence, page)
  int num_pages;                // pages in the pool (an out-of-range page reads zeros)
  int h_q, h_kv, g, R, rotary;
  int64_t max_records;  // capacity of the record table in the workspace
  float scale_log2;     // sm_scale * log2(e)
  unsigned long long timeout_ns;
  // test hook: the MMA threads first wait on a barrier that nothing arrives
  // on, so that the bounded wait runs out and the abort path runs
  int debug_stall;
  // 0: one CTA per SM takes its first unit by CTA index and the rest from the
  // atomic work queue; 1: one CTA per possible unit, and a CTA that finishes
  // takes the unit of a CTA not yet started by cancelling its launch
  // (cluster launch control)
  int sched_clc;
  // split-KV partial states of the records with part >= 0: O / l in float32
  // [record][h_kv][128 packed rows][d] and the base-2 lse [record][h_kv][128]
  float* part_o;
  float* part_lse;
};

struct MergeParams {
  const int4* merge;           // per pair: q_row0, q rows, chunks, first record
  const float* part_o;
  const float* part_lse;
  void* out;
  float* lse;
  const WsHeader* hdr;         // num_pairs
  int64_t max_pairs, max_records;
  int h_q, h_kv, g;
};

// Page table of a paged cache: sequence b owns page_values[page_indptr[b] ..
// page_indptr[b+1]-1], its last page holding length_info[b] rows.
struct PageTable {
  const int32_t* page_indptr;
  const int32_t* page_values;
  const int32_t* length_info;
  int batch, nnz_pages, num_pages;
};

struct AppendParams {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;   // elements from token to token
  const int32_t* append_indptr;
  const int32_t* positions;
  const uint16_t *q_weight, *k_weight;    // null: no norm
  uint16_t* pages;
  uint16_t* q_out;
  PageTable tab;
  unsigned int* error;
  int total_new, h_q, h_kv;
  int steps_per_warp, steps_extra;        // warps below steps_extra have one step more
  float eps;
  int rope_layout, rotary_dim;            // layout 0: no rotation
  float magnitude;
  uint64_t turns[64];
};

// The units of one-token attention over its CTAs: CTA c < ctas has warps c * W
// and so on, warp w the units from w * per + min(w, extra) on.
struct DecodeSplit {
  int ctas, per, extra;
};

struct DecodeParams {
  const uint16_t* q;
  const uint16_t* pages;
  uint16_t* out;
  float* lse;
  PageTable tab;
  unsigned int* error;
  float* parts;             // states of the sequences that several CTAs share
  int* counters;            // per (kv head, sequence, head group): its CTAs done; 0 between calls
  int h_q, h_kv, g;
  int groups;               // head groups per kv head (one CTA handles one)
  DecodeSplit split;        // for a table of nnz_pages entries (set by launch_decode)
  float scale_log2;         // sm_scale * log2(e)
};

// Workspace of the paged-cache calls: header | launch_decode's parts |
// launch_copy_pages's marks | launch_decode's counters.  The parts have the same
// place and room whatever the dims, and only they hold anything between calls,
// so calls with any dims find their marks and counters zero.
struct CacheWorkspace {
  int groups;
  int64_t off_parts, off_marks, off_counters, total;
};
CacheWorkspace cache_workspace(int batch, int num_pages, int h_kv, int g, int nsm);

struct CompactParams {
  uint4* pages;
  PageTable tab;
  const int32_t* mn_indptr;
  const int32_t* accept_indptr;
  const int32_t* accept_nodes;
  int32_t *new_indptr, *new_values, *new_length, *freed, *num_freed;
  unsigned int* error;
  int total_accept, h_kv, row_vecs;       // row_vecs: 16-byte vectors per head row
};

struct CopyParams {
  uint4* pages;
  const int32_t *src, *dst;
  unsigned int* error;
  int n, num_pages;
  int page_lines;                         // 4 KB lines per page
  unsigned int* marks;                    // [num_pages], zero between calls
};

// Plan kernel: sequence/tile enumeration, tile classification and LPT
// ordering.  ``grid`` >= max_pairs.
cudaError_t launch_plan(const PlanParams& p, int grid, cudaStream_t stream);


// RoPE of every kv token: the cos/sin table row of token t at position
// rope_pos[t] (rope_cs[t][i] = (cos, sin) of frequency i) and the rotated
// keys krot[t, h, :] = rope(k[t, h, :]).
cudaError_t launch_krot(const void* k, void* krot, const int32_t* rope_pos, float2* rope_cs,
                        const KrotParams& kp, int head_dim, bool bf16, int grid,
                        cudaStream_t stream);

// Dense mask export (test helper).
cudaError_t launch_mask_dense(const int32_t* q_indptr, const int32_t* kv_indptr,
                              const int32_t* mn_indptr, const int32_t* tree_order, int batch,
                              int total_q, int max_kv, uint8_t* vis, cudaStream_t stream);

// Split-KV: combines the partial states of every split pair into out / lse
// (the base-2 log-sum-exp merge of attention states over disjoint kv sets).
cudaError_t launch_merge(const MergeParams& p, int head_dim, bool bf16, int grid,
                         cudaStream_t stream);

// Stand-alone merge of n_parts attention states per row: parts [n][rows][d]
// and lses [n][rows] -> out [rows][d], lse [rows].
cudaError_t launch_merge_states(const void* parts, const float* lses, int n_parts,
                                long long rows, int head_dim, bool bf16, void* out, float* lse,
                                int grid, cudaStream_t stream);

// Appends tokens to the cache (norm and rotation of q and k on the way).
cudaError_t launch_append(const AppendParams& p, int head_dim, bool bf16, int grid,
                          cudaStream_t stream);

// One token per sequence against the paged cache.
cudaError_t launch_decode(const DecodeParams& p, int head_dim, bool bf16, int nsm,
                          cudaStream_t stream);

// Accepted tree nodes moved down, new page table, freed pages.
cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream);

// pages[dst[i]] = pages[src[i]].
cudaError_t launch_copy_pages(const CopyParams& p, int nsm, cudaStream_t stream);

// Persistent tree-attention kernel.
template <int D, bool BF16, bool PAGED>
cudaError_t launch_attn(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                        const AttnParams& p, int grid, cudaStream_t stream);

}  // namespace ta
