// ta_cache.cu -- filling and tidying a paged KV cache: appending tokens (with
// the norm and rotation of their queries and keys), keeping the accepted
// nodes of verified trees, copying pages.
//
// The cache is [num_pages, 2, h_kv, 16, d] (plane 0 keys, plane 1 values), so
// one head's 16 rows of a page are contiguous, and a row moves as d / 8
// vectors of 16 bytes.
#include <cuda_runtime.h>

#include <cstdint>

#include "ta_device.cuh"
#include "ta_launch.h"

namespace ta {
namespace {

__device__ __forceinline__ void report_bad_tables(unsigned int* error) {
  atomicOr(error, DEVERR_BAD_INDPTR);
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 128;

// The largest b in [0, batch) with indptr[b] <= t, by one warp: 32 probes cut
// the range by 33 each round, so 1,000 sequences take two round trips to
// memory instead of a binary search's ten.  Any table contents end the
// search inside the range.
__device__ __forceinline__ int find_sequence(const int32_t* indptr, int batch, int t, int lane) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 32) / 33;
    const int at = lo + (lane + 1) * step;
    const bool le = at < hi && __ldg(indptr + at) <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    lo += c * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// One CTA per token.  A row (one head's d elements) belongs to d / 16 lanes;
// each holds two 16-byte chunks of it, chosen so that both elements of every
// rotated pair are in one lane.  Rows 0 .. h_q-1 are the token's queries, then
// its keys, then its values.
template <int D, bool BF16>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  constexpr int kLanes = D / 16;           // lanes per row
  constexpr int kRows = 32 / kLanes;       // rows per warp and step
  __shared__ float2 s_cs[64];              // cos, sin of each pair (times magnitude)
  __shared__ long long s_slot;             // element offset of the token's K slot, head 0
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < p.rotary_dim / 2 && p.rope_layout != 0) {
    // the fraction of a turn, exact modulo 1, then one rounding to float32
    const uint64_t ph = (uint64_t)(int64_t)p.positions[t] * p.turns[tid];
    const float half_turns = (float)(int64_t)ph * 0x1p-63f;   // in [-1, 1]
    float s, c;
    sincospif(half_turns, &s, &c);
    s_cs[tid] = make_float2(c * p.magnitude, s * p.magnitude);
  }
  if (warp == kAppendThreads / 32 - 1) {
    const int b = find_sequence(p.append_indptr, p.tab.batch, t, lane);
    const int a0 = __ldg(p.append_indptr + b), a1 = __ldg(p.append_indptr + b + 1);
    const int p0 = __ldg(p.tab.page_indptr + b), p1 = __ldg(p.tab.page_indptr + b + 1);
    const int last = __ldg(p.tab.length_info + b);
    long long slot = -1;
    if (a0 >= 0 && t >= a0 && t < a1 && a1 <= p.total_new && p0 >= 0 && p1 > p0 &&
        p1 <= p.tab.nnz_pages && last >= 1 && last <= kPageSize) {
      const long long kv = (long long)(p1 - p0 - 1) * kPageSize + last;
      const long long row = kv - (a1 - t);
      if (kv >= a1 - a0) {
        const int page = __ldg(p.tab.page_values + p0 + row / kPageSize);
        if (page >= 0 && page < p.tab.num_pages)
          slot = ((long long)page * 2 * p.h_kv * kPageSize + row % kPageSize) * D;
      }
    }
    if (lane == 0) {
      s_slot = slot;
      if (slot < 0) report_bad_tables(p.error);
    }
  }
  __syncthreads();
  const long long slot = s_slot;
  const int rd = p.rope_layout != 0 ? p.rotary_dim : 0;
  const int sub = lane % kLanes;
  const int rows = p.h_q + 2 * p.h_kv;
  // this lane's chunks of 8 elements: half layout pairs chunk i with chunk
  // i + rotary_dim / 16, interleaved pairs lie within a chunk; the part of
  // the head that is not rotated is split in adjacent chunks
  const bool rot = sub < rd / 16;
  int c0 = 2 * sub, c1 = 2 * sub + 1;
  if (p.rope_layout == 1 && rot) {
    c0 = sub;
    c1 = sub + rd / 16;
  }
  for (int r0 = warp * kRows; r0 < rows; r0 += kRows * (kAppendThreads / 32)) {
    const int r = r0 + lane / kLanes;
    const bool live = r < rows;
    const uint16_t* src = p.q;
    uint16_t* dst = nullptr;
    const uint16_t* w = nullptr;
    bool plain = false;                     // a value row: copied as it is
    if (live) {
      if (r < p.h_q) {
        src = p.q + (int64_t)t * p.q_stride + (int64_t)r * D;
        dst = p.q_out + ((int64_t)t * p.h_q + r) * D;
        w = p.q_weight;
      } else if (r < p.h_q + p.h_kv) {
        const int h = r - p.h_q;
        src = p.k + (int64_t)t * p.k_stride + (int64_t)h * D;
        if (slot >= 0) dst = p.pages + slot + (int64_t)h * kPageSize * D;
        w = p.k_weight;
      } else {
        const int h = r - p.h_q - p.h_kv;
        src = p.v + (int64_t)t * p.v_stride + (int64_t)h * D;
        if (slot >= 0) dst = p.pages + slot + (int64_t)(p.h_kv + h) * kPageSize * D;
        plain = true;
      }
    }
    uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
    if (live) {
      u0 = reinterpret_cast<const uint4*>(src)[c0];
      u1 = reinterpret_cast<const uint4*>(src)[c1];
    }
    const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w}, w1[4] = {u1.x, u1.y, u1.z, u1.w};
    float x0[8], x1[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = unpack2<BF16>(w0[i]), b = unpack2<BF16>(w1[i]);
      x0[2 * i] = a.x;
      x0[2 * i + 1] = a.y;
      x1[2 * i] = b.x;
      x1[2 * i + 1] = b.y;
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += x0[i] * x0[i] + x1[i] * x1[i];
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (w != nullptr) {
      const float inv = 1.f / sqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = unpack2<BF16>(reinterpret_cast<const uint32_t*>(w)[c0 * 4 + i]);
        const float2 b = unpack2<BF16>(reinterpret_cast<const uint32_t*>(w)[c1 * 4 + i]);
        x0[2 * i] *= inv * a.x;
        x0[2 * i + 1] *= inv * a.y;
        x1[2 * i] *= inv * b.x;
        x1[2 * i + 1] *= inv * b.y;
      }
    }
    if (rot && !plain) {
      if (p.rope_layout == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 cs = s_cs[8 * sub + i];
          const float a = x0[i], b = x1[i];
          x0[i] = a * cs.x - b * cs.y;
          x1[i] = b * cs.x + a * cs.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 ca = s_cs[8 * sub + i], cb = s_cs[8 * sub + 4 + i];
          const float a0 = x0[2 * i], a1 = x0[2 * i + 1];
          const float b0 = x1[2 * i], b1 = x1[2 * i + 1];
          x0[2 * i] = a0 * ca.x - a1 * ca.y;
          x0[2 * i + 1] = a1 * ca.x + a0 * ca.y;
          x1[2 * i] = b0 * cb.x - b1 * cb.y;
          x1[2 * i + 1] = b1 * cb.x + b0 * cb.y;
        }
      }
    }
    if (!plain) {
      u0 = make_uint4(pack2<BF16>(x0[0], x0[1]), pack2<BF16>(x0[2], x0[3]),
                      pack2<BF16>(x0[4], x0[5]), pack2<BF16>(x0[6], x0[7]));
      u1 = make_uint4(pack2<BF16>(x1[0], x1[1]), pack2<BF16>(x1[2], x1[3]),
                      pack2<BF16>(x1[4], x1[5]), pack2<BF16>(x1[6], x1[7]));
    }
    if (dst != nullptr) {
      reinterpret_cast<uint4*>(dst)[c0] = u0;
      reinterpret_cast<uint4*>(dst)[c1] = u1;
    }
  }
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------
constexpr int kCompactThreads = 256;
constexpr int kCompactBatch = 16;   // rows whose vectors one thread has in flight

// CTA (b, y): sequence b, 256 of the 16-byte columns of its cache rows (a
// column: one vector of one head of keys or values).  The moves are in place
// and a destination may be another move's source.  Node lists ascend, so
// move j reads a row at or behind row j: a thread that owns its column and
// takes the moves in order, a batch of loads before the batch's stores, never
// reads what it has overwritten.
// CTA (b, 0) also writes sequence b's part of the new table, whose place it
// finds by summing the pages the sequences before it keep.
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const CompactParams p) {
  __shared__ long long s_src[kCompactThreads], s_dst[kCompactThreads];
  __shared__ int s_sum[kCompactThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, b = blockIdx.x;
  const PageTable& tb = p.tab;
  int before = 0;          // pages kept by the sequences before b
  int bad = 0;
  if (tid == 0)
    bad = tb.page_indptr[0] != 0 || p.accept_indptr[0] != 0 ||
          tb.page_indptr[tb.batch] > tb.nnz_pages ||
          p.accept_indptr[tb.batch] != p.total_accept;
  auto rows_of = [&](int i, int& p0, int& np, int& kv, int& tree, int& a0, int& acc) {
    p0 = __ldg(tb.page_indptr + i);
    np = __ldg(tb.page_indptr + i + 1) - p0;
    const int last = __ldg(tb.length_info + i);
    tree = __ldg(p.mn_indptr + i + 1) - __ldg(p.mn_indptr + i);
    a0 = __ldg(p.accept_indptr + i);
    acc = __ldg(p.accept_indptr + i + 1) - a0;
    kv = np > 0 ? (np - 1) * kPageSize + last : 0;
    return np >= 0 && p0 >= 0 && np <= tb.nnz_pages &&
           (np == 0 || (last >= 1 && last <= kPageSize)) && acc >= 0 && acc <= tree && tree <= kv;
  };
  int p0, np, kv, tree, a0, acc;
  for (int i = tid; i < tb.batch; i += kCompactThreads) {
    bad |= !rows_of(i, p0, np, kv, tree, a0, acc);
    if (i < b) before += (kv - tree + acc + kPageSize - 1) / kPageSize;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) report_bad_tables(p.error);
    return;
  }
  rows_of(b, p0, np, kv, tree, a0, acc);
  const int start = kv - tree;
  const int keep = (start + acc + kPageSize - 1) / kPageSize;

  // the moves: every node checked before the first row moves
  const int64_t head_vecs = (int64_t)kPageSize * p.row_vecs;   // one head's plane of a page
  const int cols = 2 * p.h_kv * p.row_vecs;
  const int col = blockIdx.y * kCompactThreads + tid;
  const int64_t col_off = (int64_t)(col / p.row_vecs) * head_vecs + col % p.row_vecs;
  auto row_offset = [&](int row) -> long long {
    const int page = __ldg(tb.page_values + p0 + row / kPageSize);
    if (page < 0 || page >= tb.num_pages) return -1;
    return (long long)page * 2 * p.h_kv * head_vecs + (long long)(row % kPageSize) * p.row_vecs;
  };
  auto stage = [&](int j) {      // move j into slot tid; whether it is valid
    const int node = __ldg(p.accept_nodes + a0 + j);
    const int prev = j > 0 ? __ldg(p.accept_nodes + a0 + j - 1) : -1;
    if (node <= prev || node >= tree) return false;
    s_src[tid] = s_dst[tid] = -1;
    if (node == j) return true;  // stays where it is
    s_src[tid] = row_offset(start + node);
    s_dst[tid] = row_offset(start + j);
    return s_src[tid] >= 0 && s_dst[tid] >= 0;
  };
  bool ok = true;
  for (int j = tid; j < acc; j += kCompactThreads) ok = stage(j) && ok;
  if (__syncthreads_and(ok)) {
    for (int j0 = 0; j0 < acc; j0 += kCompactThreads) {
      if (acc > kCompactThreads) {
        __syncthreads();
        if (j0 + tid < acc) stage(j0 + tid);
        __syncthreads();
      }
      const int n = min(kCompactThreads, acc - j0);
      if (col < cols) {
        for (int k0 = 0; k0 < n; k0 += kCompactBatch) {
          uint4 v[kCompactBatch];
#pragma unroll
          for (int k = 0; k < kCompactBatch; ++k)
            if (k0 + k < n && s_src[k0 + k] >= 0) v[k] = p.pages[s_src[k0 + k] + col_off];
#pragma unroll
          for (int k = 0; k < kCompactBatch; ++k)
            if (k0 + k < n && s_src[k0 + k] >= 0) p.pages[s_dst[k0 + k] + col_off] = v[k];
        }
      }
    }
  } else if (tid == 0) {
    report_bad_tables(p.error);
  }

  // the table
  if (blockIdx.y != 0) return;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  if ((tid & 31) == 0) s_sum[tid >> 5] = before;
  __syncthreads();
  before = 0;
#pragma unroll
  for (int i = 0; i < kCompactThreads / 32; ++i) before += s_sum[i];
  for (int i = tid; i < np; i += kCompactThreads) {
    const int page = __ldg(tb.page_values + p0 + i);
    if (i < keep)
      p.new_values[before + i] = page;
    else
      p.freed[p0 - before + i - keep] = page;
  }
  if (tid == 0) {
    p.new_indptr[b] = before;
    p.new_length[b] = keep > 0 ? start + acc - (keep - 1) * kPageSize : 0;
    if (b == tb.batch - 1) {
      p.new_indptr[tb.batch] = before + keep;
      *p.num_freed = p0 + np - (before + keep);
    }
  }
}

// ---------------------------------------------------------------------------
// copies of pages
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kCopyDepth = 10;       // lines a CTA has in flight
constexpr int kCopyPairs = 256;      // pairs a CTA checks at a time
constexpr int kCopyFilter = 4096;    // bits

// A position in the list of lines: pair k of this round's, line ``line`` of its page.
struct CopyAt {
  int k, line;
  __device__ __forceinline__ void next(int page_lines) {
    if (++line == page_lines) {
      line = 0;
      ++k;
    }
  }
};

// The n pages are one list of 4 KB lines (a page is h_kv * d / 64 of them: one
// 16-byte vector per thread each), cut evenly over the CTAs.  Lines pass
// through a ring in shared memory by cp.async, each thread reading back only
// what it fetched itself, so nothing waits for anything but its own data: ten
// lines in flight in each of five CTAs keep 200 KB of loads on the way to an
// SM, which the registers could not hold.  Before its first store a CTA looks for its
// pairs' destinations among all other pairs' sources and destinations, through
// a bit filter in shared memory (a hit is then looked up exactly), while the
// first lines arrive.
__global__ void __launch_bounds__(kCopyThreads, 5) copy_pages_kernel(const CopyParams p) {
  __shared__ uint4 s_ring[kCopyDepth][kCopyThreads];
  __shared__ unsigned int s_filter[kCopyFilter / 32];
  __shared__ int s_src[kCopyPairs], s_dst[kCopyPairs];
  __shared__ int s_skip[kCopyPairs];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int64_t total = (int64_t)p.n * p.page_lines;
  const int64_t per = total / gridDim.x, extra = total % gridDim.x;
  const int64_t lo = per * blockIdx.x + min((int64_t)blockIdx.x, extra);
  const int64_t hi = lo + per + (blockIdx.x < extra);
  if (lo >= hi) return;
  const int64_t first = lo / p.page_lines, last = (hi - 1) / p.page_lines;
  const int64_t page_vecs = (int64_t)p.page_lines * kCopyThreads;
  for (int64_t base = first; base <= last; base += kCopyPairs) {
    const int m = (int)min((int64_t)kCopyPairs, last - base + 1);
    __syncthreads();
    for (int i = tid; i < kCopyFilter / 32; i += kCopyThreads) s_filter[i] = 0;
    int s = 0, d = 0;
    if (tid < m) {
      s = p.src[base + tid];
      d = p.dst[base + tid];
    }
    __syncthreads();
    if (tid < m) {
      const bool out = s < 0 || s >= p.num_pages || d < 0 || d >= p.num_pages;
      s_src[tid] = s;
      s_dst[tid] = d;
      s_skip[tid] = out || s == d;
      if (s != d) atomicOr(&s_filter[(d & (kCopyFilter - 1)) >> 5], 1u << (d & 31));
      if (out) report_bad_tables(p.error);
    }
    __syncthreads();
    const int line0 = (int)(max(lo, base * p.page_lines) - base * p.page_lines);
    const int lines = (int)(min(hi, (base + m) * p.page_lines) - base * p.page_lines) - line0;
    CopyAt get{line0 / p.page_lines, line0 % p.page_lines}, put = get;
    auto fetch = [&](int l) {
      if (l < lines) {
        if (!s_skip[get.k]) {
          const uint4* from = p.pages + s_src[get.k] * page_vecs + get.line * kCopyThreads + tid;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           smem_u32(&s_ring[l % kCopyDepth][tid])),
                       "l"(from)
                       : "memory");
        }
        get.next(p.page_lines);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int l = 0; l < kCopyDepth; ++l) fetch(l);
    __syncthreads();                   // s_skip is read above and written below
#pragma unroll 4
    for (int i = tid; i < p.n; i += kCopyThreads) {
      const int w[2] = {p.src[i], p.dst[i]};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!(s_filter[(w[x] & (kCopyFilter - 1)) >> 5] >> (w[x] & 31) & 1)) continue;
        for (int k = 0; k < m; ++k)
          if (s_dst[k] == w[x] && base + k != i && s_src[k] != s_dst[k]) {
            s_skip[k] = 1;
            report_bad_tables(p.error);
          }
      }
    }
    __syncthreads();
    for (int l = 0; l < lines; ++l) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kCopyDepth - 1) : "memory");
      if (!s_skip[put.k])
        p.pages[s_dst[put.k] * page_vecs + put.line * kCopyThreads + tid] = s_ring[l % kCopyDepth][tid];
      put.next(p.page_lines);
      fetch(l + kCopyDepth);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, int head_dim, bool bf16, cudaStream_t stream) {
  const dim3 g(p.total_new), b(kAppendThreads);
  if (head_dim == 128)
    return bf16 ? launch_pdl(append_kernel<128, true>, g, b, 0, stream, p)
                : launch_pdl(append_kernel<128, false>, g, b, 0, stream, p);
  return bf16 ? launch_pdl(append_kernel<64, true>, g, b, 0, stream, p)
              : launch_pdl(append_kernel<64, false>, g, b, 0, stream, p);
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream) {
  const int cols = 2 * p.h_kv * p.row_vecs;
  const dim3 g(p.tab.batch, (cols + kCompactThreads - 1) / kCompactThreads);
  return launch_pdl(compact_kernel, g, dim3(kCompactThreads), 0, stream, p);
}

cudaError_t launch_copy_pages(const CopyParams& p, int grid, cudaStream_t stream) {
  return launch_pdl(copy_pages_kernel, dim3(grid), dim3(kCopyThreads), 0, stream, p);
}

}  // namespace ta
