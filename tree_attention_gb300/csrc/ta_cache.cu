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
constexpr int kAppendTokens = 8;  // tokens that a warp comes by, at most
static_assert((kAppendMaxSteps - 1) / 3 + 2 <= kAppendTokens, "a token has three steps at least");
constexpr int kAppendDepth = 5;   // steps (1 KB) a warp has in flight (3: 3 % slower, 8 no faster)

// The largest b in [0, batch) with indptr[b] <= t, by one warp: 32 probes cut
// the range by 33 each round, so 1,000 sequences take two round trips to
// memory instead of a binary search's ten.  Any table contents end the
// search inside the range.
__device__ __forceinline__ int find_sequence(const int32_t* indptr, int batch, int t, int lane) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 32) / 33;
    const int at = lo + (lane + 1) * step;
    const bool le = at < hi && indptr[at] <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    lo += c * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// A step is 32 * 16 elements of one token's queries, keys or values; the steps
// of all tokens are cut evenly over the warps, a dozen steps each at most.  A
// row (one head's d elements) belongs to d / 16 lanes; each holds two 16-byte
// chunks of it, chosen so that both elements of every rotated pair are in one
// lane.
//
// Bound by memory: 4 bytes of traffic per element against the memory's rate
// leave a lane some 200 instructions for its 16 elements of a step, and the
// latencies within a step have to be hidden by few warps, as what a token's
// rows have in common is kept in registers: cos and sin, made once per token,
// and their products with the weights, made once for its queries and once for
// its keys.  Each lane fetches its own chunks kAppendDepth steps ahead into
// shared memory (cp.async; nothing else reads them, so no barrier), past the
// ends of tokens, and the arithmetic is in pairs of float32.
//
// Measured: 9,478 tokens of 64 + 8 + 8 heads of 128, with norms and interleaved
// pairs (388 MB): 61.2 us, 6.3 TB/s; without norm and rotation 59.9 us, so the
// memory, in rows of 256 bytes, is what bounds it.  2,048 tokens of 32 + 8 + 8:
// 11.0 us, bound by the look-ups and the latency of eight steps per warp.
template <int D, bool BF16, int LAYOUT>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas) append_kernel(const AppendParams p) {
  constexpr int kLanes = D / 16;           // lanes per row
  constexpr int kRows = 32 / kLanes;       // rows per step
  constexpr bool kHalves = LAYOUT == 1;
  __shared__ uint4 s_ring[kAppendThreads / 32][kAppendDepth][2][32];
  __shared__ __align__(16) float2 s_cos_sin[kAppendThreads / 32][D / 2];
  __shared__ uint64_t s_turns[64];
  __shared__ uint4 s_weight[2][D / 8];     // of queries, of keys
  __shared__ long long s_slot[kAppendThreads / 32][kAppendTokens];   // see look_up
  __shared__ int s_pos[kAppendThreads / 32][kAppendTokens];
  // lanes that index the parameters apart are served one by one: once per CTA
  static_assert(kAppendThreads >= 64 + D / 4, "a thread per frequency and per vector of weights");
  if (LAYOUT != 0 && threadIdx.x < 64) s_turns[threadIdx.x] = p.turns[threadIdx.x];
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x >= 64 && threadIdx.x < 64 + D / 4) {
    const int i = threadIdx.x - 64;
    const uint16_t* w = i < D / 8 ? p.q_weight : p.k_weight;
    if (w != nullptr) s_weight[i / (D / 8)][i % (D / 8)] = reinterpret_cast<const uint4*>(w)[i % (D / 8)];
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane % kLanes, lane_row = lane / kLanes;
  // this lane's chunks of 8 elements, such that the lanes of a row hold runs of
  // chunks: interleaved pairs lie within a chunk, half layout pairs chunk i with
  // chunk i + rotary_dim / 16; rot0, rot1: whether a chunk is rotated
  const int rd = LAYOUT != 0 ? p.rotary_dim : 0;
  int c0 = sub, c1 = sub + kLanes;
  bool rot0 = c0 < rd / 8, rot1 = c1 < rd / 8;
  if (kHalves) {
    rot0 = rot1 = sub < rd / 16;
    c0 = rot0 ? sub : sub + rd / 16;
    c1 = c0 + (rot0 ? rd / 16 : kLanes - rd / 16);
  }
  // steps of a token: its queries' (kind 0), keys' (1) and values' (2)
  const int steps_q = (p.h_q + kRows - 1) / kRows, steps_kv = (p.h_kv + kRows - 1) / kRows;
  const int all = steps_q + 2 * steps_kv;
  // this warp's share of all tokens' steps: ``left`` of them from step ``begin``
  // of token ``t`` on
  const int gw = blockIdx.x * (kAppendThreads / 32) + warp;
  const int lo = gw * p.steps_per_warp + min(gw, p.steps_extra);
  int left = p.steps_per_warp + (gw < p.steps_extra);
  int t = lo / all, begin = lo - t * all;
  auto first_step = [&](int kind) { return kind == 0 ? 0 : kind == 1 ? steps_q : steps_q + steps_kv; };

  // The fetches: their token, step, and of the step's rows this lane's.
  int f_left = left, f_t = t, f_step = begin, f_next_kind = begin;
  int f_rows = 0;                          // rows from this lane's on to the kind's last
  const uint16_t* f_src = nullptr;         // this lane's first chunk
  const int apart = 8 * (c1 - c0);         // its second, from there
  const uint32_t ring0 = smem_u32(&s_ring[warp][0][0][lane]);
  uint32_t f_to = ring0;
  auto fetch = [&]() {
    if (f_left > 0) {
      --f_left;
      if (f_step == f_next_kind) {         // the first step, or the first of another kind
        const int kind = f_step < steps_q ? 0 : f_step < steps_q + steps_kv ? 1 : 2;
        const int row = (f_step - first_step(kind)) * kRows + lane_row;
        f_rows = (kind == 0 ? p.h_q : p.h_kv) - row;
        f_src = (kind == 0 ? p.q : kind == 1 ? p.k : p.v) + row * D + 8 * c0 +
                f_t * (kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride);
        f_next_kind = kind == 2 ? 0 : first_step(kind + 1);
      }
      if (f_rows > 0) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(f_to), "l"(f_src) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(f_to + 512), "l"(f_src + apart)
                     : "memory");
      }
      f_rows -= kRows;
      f_src += kRows * D;
      f_to = f_to == ring0 + (kAppendDepth - 1) * 1024 ? ring0 : f_to + 1024;
      if (++f_step == all) {
        f_step = 0;
        ++f_t;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // Positions and cache slots of this warp's tokens, token x's at x % kAppendTokens,
  // looked up one per lane: one chain of dependent loads for all of them.  It goes
  // first: behind the rows of all warps in the memory's queues each of its loads
  // took 1,500 cycles instead of 700.
  auto look_up = [&]() {
    const int tt = t + lane;
    const bool mine = lane < kAppendTokens && tt <= (lo + left - 1) / all;
    const int pos = LAYOUT != 0 && mine ? p.positions[tt] : 0;
    // the sequence of the first token, then of the others behind it
    int b = find_sequence(p.append_indptr, p.tab.batch, t, lane);
    if (mine && tt >= p.append_indptr[b + 1]) {
      int hi = p.tab.batch;                // the largest b with append_indptr[b] <= tt
      while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (p.append_indptr[mid] <= tt)
          b = mid;
        else
          hi = mid;
      }
    }
    if (!mine) return;
    const int a0 = p.append_indptr[b], a1 = p.append_indptr[b + 1];
    const int p0 = p.tab.page_indptr[b], p1 = p.tab.page_indptr[b + 1], last = p.tab.length_info[b];
    long long slot = -1;                   // element offset of its K slot, head 0; -1: none
    if (a0 >= 0 && tt >= a0 && tt < a1 && a1 <= p.total_new && p0 >= 0 && p1 > p0 &&
        p1 <= p.tab.nnz_pages && last >= 1 && last <= kPageSize) {
      const int kv = (p1 - p0 - 1) * kPageSize + last, row = kv - (a1 - tt);
      if (kv >= a1 - a0) {
        const int page = p.tab.page_values[p0 + row / kPageSize];
        if (page >= 0 && page < p.tab.num_pages)
          slot = ((long long)page * 2 * p.h_kv * kPageSize + row % kPageSize) * D;
      }
    }
    if (slot < 0) report_bad_tables(p.error);
    s_slot[warp][tt % kAppendTokens] = slot;
    if (LAYOUT != 0) s_pos[warp][tt % kAppendTokens] = pos;
  };
  if (left > 0) look_up();
#pragma unroll 1
  for (int i = 0; i < kAppendDepth; ++i) fetch();
  __syncthreads();                         // s_turns, s_weight, s_slot, s_pos

  int ring = 0;
  for (; left > 0; ++t, begin = 0) {
    const int end = min(all, begin + left);
    left -= end - begin;
    const long long slot = s_slot[warp][t % kAppendTokens];
    if (LAYOUT != 0) {
      const int64_t pos = s_pos[warp][t % kAppendTokens];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const int j = lane + 32 * i;
        if (j < rd / 2) {
          // the fraction of a turn, exact modulo 1, then one rounding to float32
          const uint64_t ph = (uint64_t)pos * s_turns[j];
          const float half_turns = (float)(int64_t)ph * 0x1p-63f;   // in [-1, 1]
          float sn, cs;
          sincospif(half_turns, &sn, &cs);
          s_cos_sin[warp][j] = make_float2(cs * p.magnitude, sn * p.magnitude);
        }
      }
      __syncwarp();
    }
#pragma unroll 1
    for (int kind = 0; kind < 3; ++kind) {
      const int k_lo = first_step(kind), k_hi = kind == 2 ? all : first_step(kind + 1);
      const int s_lo = max(begin, k_lo), s_hi = min(end, k_hi);
      if (s_lo >= s_hi) continue;
      // where rows go: planes and heads of the cache follow one another
      int row = (s_lo - k_lo) * kRows + lane_row;
      const int rows = kind == 0 ? p.h_q : p.h_kv;
      const int64_t stride = kind == 0 ? D : kPageSize * D;
      uint16_t* dst = kind == 0 ? p.q_out + (int64_t)t * p.h_q * D
                                : p.pages + slot + (kind == 2 ? (int64_t)p.h_kv * stride : 0);
      dst += row * stride;
      if (kind != 0 && slot < 0) row = rows;           // nothing is written
      // x * own + partner * other, times 1 / rms
      float2 own0[4], own1[4], other0[4], other1[4];
      const bool norm = (kind == 0 ? p.q_weight : p.k_weight) != nullptr;
#pragma unroll
      for (int i = 0; i < 4; ++i) own0[i] = own1[i] = make_float2(1.f, 1.f);
      if (kind < 2) {
        if (norm) {
          const uint4 a = s_weight[kind][c0], b = s_weight[kind][c1];
          own0[0] = unpack2<BF16>(a.x), own0[1] = unpack2<BF16>(a.y);
          own0[2] = unpack2<BF16>(a.z), own0[3] = unpack2<BF16>(a.w);
          own1[0] = unpack2<BF16>(b.x), own1[1] = unpack2<BF16>(b.y);
          own1[2] = unpack2<BF16>(b.z), own1[3] = unpack2<BF16>(b.w);
        }
        // two pairs each: cos, sin, cos, sin
        const float4* cs = reinterpret_cast<const float4*>(s_cos_sin[warp]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          other0[i] = other1[i] = make_float2(0.f, 0.f);
          const float2 w0 = own0[i], w1 = own1[i];
          if (kHalves) {
            if (!rot0) continue;
            const float4 x = cs[4 * c0 + i];           // pairs 8 c0 + 2 i, 8 c0 + 2 i + 1
            own0[i] = make_float2(w0.x * x.x, w0.y * x.z);
            other0[i] = make_float2(-w1.x * x.y, -w1.y * x.w);
            own1[i] = make_float2(w1.x * x.x, w1.y * x.z);
            other1[i] = make_float2(w0.x * x.y, w0.y * x.w);
          } else {
            if (rot0) {
              const float4 x = cs[2 * c0 + (i >> 1)];  // pair 4 c0 + i
              const float2 a = i & 1 ? make_float2(x.z, x.w) : make_float2(x.x, x.y);
              own0[i] = make_float2(w0.x * a.x, w0.y * a.x);
              other0[i] = make_float2(-w0.y * a.y, w0.x * a.y);
            }
            if (rot1) {
              const float4 x = cs[2 * c1 + (i >> 1)];
              const float2 a = i & 1 ? make_float2(x.z, x.w) : make_float2(x.x, x.y);
              own1[i] = make_float2(w1.x * a.x, w1.y * a.x);
              other1[i] = make_float2(-w1.y * a.y, w1.x * a.y);
            }
          }
        }
      }
      // what neither norm nor rotation touches keeps its bits
      const bool plain0 = kind == 2 || !(norm || rot0), plain1 = kind == 2 || !(norm || rot1);
#pragma unroll 1
      for (int s = s_lo; s < s_hi; ++s) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAppendDepth - 1) : "memory");
        uint4 u0 = s_ring[warp][ring][0][lane], u1 = s_ring[warp][ring][1][lane];
        ring = ring + 1 == kAppendDepth ? 0 : ring + 1;
        if (kind < 2) {
          float2 x0[4] = {unpack2<BF16>(u0.x), unpack2<BF16>(u0.y), unpack2<BF16>(u0.z),
                          unpack2<BF16>(u0.w)};
          float2 x1[4] = {unpack2<BF16>(u1.x), unpack2<BF16>(u1.y), unpack2<BF16>(u1.z),
                          unpack2<BF16>(u1.w)};
          const float2 zero = make_float2(0.f, 0.f);
          if (norm) {
            float2 sa = zero, sb = zero;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              sa = ffma2(x0[i], x0[i], sa);
              sb = ffma2(x1[i], x1[i], sb);
            }
            float sum = (sa.x + sa.y) + (sb.x + sb.y);
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float inv = rsqrtf(sum * (1.f / D) + p.eps);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x0[i] = ffma2(x0[i], make_float2(inv, inv), zero);
              x1[i] = ffma2(x1[i], make_float2(inv, inv), zero);
            }
          }
          float2 y0[4], y1[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y0[i] = ffma2(x0[i], own0[i], zero);
            y1[i] = ffma2(x1[i], own1[i], zero);
            if (rot0)
              y0[i] = ffma2(kHalves ? x1[i] : make_float2(x0[i].y, x0[i].x), other0[i], y0[i]);
            if (rot1)
              y1[i] = ffma2(kHalves ? x0[i] : make_float2(x1[i].y, x1[i].x), other1[i], y1[i]);
          }
          if (!plain0)
            u0 = make_uint4(pack2<BF16>(y0[0].x, y0[0].y), pack2<BF16>(y0[1].x, y0[1].y),
                            pack2<BF16>(y0[2].x, y0[2].y), pack2<BF16>(y0[3].x, y0[3].y));
          if (!plain1)
            u1 = make_uint4(pack2<BF16>(y1[0].x, y1[0].y), pack2<BF16>(y1[1].x, y1[1].y),
                            pack2<BF16>(y1[2].x, y1[2].y), pack2<BF16>(y1[3].x, y1[3].y));
        }
        if (row < rows) {
          reinterpret_cast<uint4*>(dst)[c0] = u0;
          reinterpret_cast<uint4*>(dst)[c1] = u1;
        }
        row += kRows;
        dst += kRows * stride;
        fetch();                           // into the slot read above
      }
    }
  }
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------
constexpr int kCompactThreads = 256;
constexpr int kCompactBatch = 8;   // rows whose vectors one thread has in flight

// What the tables say of one sequence.
struct CompactSeq {
  int p0, p1, last, m0, m1, a0, a1;
  __device__ __forceinline__ int pages() const { return p1 - p0; }
  __device__ __forceinline__ int tree() const { return m1 - m0; }
  __device__ __forceinline__ int accepted() const { return a1 - a0; }
  __device__ __forceinline__ int kv() const { return p1 > p0 ? (p1 - p0 - 1) * kPageSize + last : 0; }
  // pages it keeps
  __device__ __forceinline__ int keep() const {
    return (kv() - tree() + accepted() + kPageSize - 1) / kPageSize;
  }
  __device__ __forceinline__ bool good(const CompactParams& p) const {
    return p0 >= 0 && p1 >= p0 && p1 <= p.tab.nnz_pages &&
           (p1 == p0 || (last >= 1 && last <= kPageSize)) && a0 >= 0 && a1 >= a0 &&
           a1 <= p.total_accept && m1 >= m0 && accepted() <= tree() && tree() <= kv();
  }
};
__device__ __forceinline__ CompactSeq compact_seq(const CompactParams& p, int i) {
  return CompactSeq{p.tab.page_indptr[i], p.tab.page_indptr[i + 1], p.tab.length_info[i],
                    p.mn_indptr[i],       p.mn_indptr[i + 1],       p.accept_indptr[i],
                    p.accept_indptr[i + 1]};
}

// CTA (b, y): sequence b, 256 of the 16-byte columns of its cache rows (a
// column: one vector of one head of keys or values).  The moves are in place
// and a destination may be another move's source.  Node lists ascend, so
// move j reads a row at or behind row j: a thread that owns its column and
// takes the moves in order, a batch of loads before the batch's stores, never
// reads what it has overwritten.
// CTA (b, 0) also writes sequence b's part of the new table, whose place it
// finds by summing the pages the sequences before it keep.
// Few sequences: bound by the chain of dependent loads (tables, nodes, pages,
// rows), so the independent ones are issued together.  More: by the batches of
// the longest paths, as a batch's loads wait for the stores before it (512
// sequences, clock stamps: tables and nodes 4,500 cycles, then 3,700 for paths of
// up to 6 nodes, 9,300 up to 12, 12,700 up to 18, 16,900 up to 24).  Many
// thousands: by the tables, which every CTA reads whole, work that grows with the
// square of the batch.  The registers leave room for four CTAs per SM.
// Measured: 512 sequences, paths of up to 24 nodes, 8 kv heads of 128: 12.2 us
// (16.5 with 16 rows in flight per thread and two CTAs per SM), 4.1 TB/s; 32
// sequences: 3.8 us; with trees of 8 nodes, 4,096 sequences 50 us, 16,384
// sequences 596 us.
__global__ void __launch_bounds__(kCompactThreads, 4) compact_kernel(const CompactParams p) {
  __shared__ long long s_src[kCompactThreads], s_dst[kCompactThreads];
  __shared__ int s_sum[kCompactThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, b = blockIdx.x;
  const PageTable& tb = p.tab;
  const CompactSeq me = compact_seq(p, b);
  // all sequences' tables are checked by every CTA: one that is inconsistent
  // stops them all
  int before = 0;          // pages kept by the sequences before b
  bool bad = tid == 0 && (tb.page_indptr[0] != 0 || p.accept_indptr[0] != 0 ||
                          p.accept_indptr[tb.batch] != p.total_accept);
  for (int i = tid; i < tb.batch; i += kCompactThreads) {
    const CompactSeq x = compact_seq(p, i);
    bad |= !x.good(p);
    if (i < b) before += x.keep();
  }
  const bool mine = me.good(p);
  const int acc = mine ? me.accepted() : 0, tree = mine ? me.tree() : 0;
  auto node_at = [&](int j) { return j >= 0 && j < acc ? p.accept_nodes[me.a0 + j] : -1; };
  int node = node_at(tid), prev = node_at(tid - 1);
  const int page0 = mine && tid < me.pages() ? tb.page_values[me.p0 + tid] : 0;
  if (__syncthreads_or(bad)) {
    if (tid == 0) report_bad_tables(p.error);
    return;
  }
  const int start = me.kv() - tree, keep = me.keep();

  // the moves: every node checked before the first row moves
  const int64_t head_vecs = (int64_t)kPageSize * p.row_vecs;   // one head's plane of a page
  const int cols = p.planes * p.row_vecs;
  const int col = blockIdx.y * kCompactThreads + tid;
  const int64_t col_off = (int64_t)(col / p.row_vecs) * head_vecs + col % p.row_vecs;
  auto row_offset = [&](int row) -> long long {
    const int page = tb.page_values[me.p0 + row / kPageSize];
    if (page < 0 || page >= tb.num_pages) return -1;
    return (long long)page * p.planes * head_vecs + (long long)(row % kPageSize) * p.row_vecs;
  };
  auto stage = [&](int j) {      // move j into slot tid; whether it is valid
    if (node <= prev || node >= tree) return false;
    s_src[tid] = s_dst[tid] = -1;
    if (node == j) return true;  // stays where it is
    const long long from = row_offset(start + node), to = row_offset(start + j);
    s_src[tid] = from;
    s_dst[tid] = to;
    return from >= 0 && to >= 0;
  };
  bool ok = true;
  if (tid < acc) ok = stage(tid);
  for (int j = tid + kCompactThreads; j < acc; j += kCompactThreads) {
    node = node_at(j);
    prev = node_at(j - 1);
    ok = stage(j) && ok;
  }
  if (__syncthreads_and(ok)) {
    for (int j0 = 0; j0 < acc; j0 += kCompactThreads) {
      if (acc > kCompactThreads) {
        __syncthreads();
        node = node_at(j0 + tid);
        prev = node_at(j0 + tid - 1);
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
  for (int i = tid; i < me.pages(); i += kCompactThreads) {
    const int page = i == tid ? page0 : tb.page_values[me.p0 + i];
    if (i < keep)
      p.new_values[before + i] = page;
    else
      p.freed[me.p0 - before + i - keep] = page;
  }
  if (tid == 0) {
    p.new_indptr[b] = before;
    p.new_length[b] = keep > 0 ? start + acc - (keep - 1) * kPageSize : 0;
    if (b == tb.batch - 1) {
      p.new_indptr[tb.batch] = before + keep;
      *p.num_freed = me.p1 - (before + keep);
    }
  }
}

// ---------------------------------------------------------------------------
// copies of pages
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kCopyDepth = 4;        // lines a CTA has in flight
constexpr int kCopyPairs = 256;      // pairs a CTA checks at a time
constexpr int kCopyFilter = 4096;    // bits
constexpr int kCopyMarkedLines = 32768, kCopyMarkedPairs = 2048;   // see launch_copy_pages

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

// Marks of the pages that a list of pairs names, in the workspace: how often a
// page is a destination, and whether it is a source.  They are zero between
// calls; CLEAR puts them back.
constexpr unsigned int kMarkSource = 1u << 31;
template <bool CLEAR>
__global__ void __launch_bounds__(kCopyThreads) mark_pages_kernel(const CopyParams p) {
  pdl_wait();
  pdl_trigger();
  const int stride = gridDim.x * kCopyThreads;
  for (int64_t i = blockIdx.x * kCopyThreads + threadIdx.x; i < p.n; i += stride) {
    const int s = p.src[i], d = p.dst[i];
    if (s >= 0 && s < p.num_pages) {
      if (CLEAR)
        p.marks[s] = 0;
      else
        atomicOr(p.marks + s, kMarkSource);
    }
    if (d >= 0 && d < p.num_pages && s != d) {
      if (CLEAR)
        p.marks[d] = 0;
      else
        atomicAdd(p.marks + d, 1u);
    }
  }
}

// The n pages are one list of 4 KB lines (a page is h_kv * d / 64 of them: one
// 16-byte vector per thread each), cut evenly over the CTAs.  Lines pass
// through a ring in shared memory by cp.async, each thread reading back only
// what it fetched itself, so nothing waits for anything but its own data: four
// lines in flight in each of five CTAs keep 80 KB of loads on the way to an SM
// (ten measured the same on large copies and slower on small ones).
//
// Before its first store, while the first lines arrive, a CTA finds out which
// of its pairs must not be copied.  MARKED: from the marks of the list, made by
// a kernel before this one; CTAs are short (16 lines), as SMs reach the memory
// at different speeds and equal shares of one wave end with the slowest.  Else,
// without another launch: it looks for its pairs' destinations among all other
// pairs' sources and destinations, through a bit filter in shared memory (a hit
// is then looked up exactly), work that grows with n in every CTA.
// Measured, marked / not, us: 300 pages of 64 KB 9.0 / 7.3, 1,000 26.1 / 24.3,
// 4,096 84.9 / 94.0 (6.3 TB/s; a contiguous copy of as much takes torch 86),
// 16,000 310 / 381; of 8 KB, 1,500 pages 8.1 / 6.5, 16,000 45.5 / 88.
// RAGGED: pages that are not whole lines (a latent cache's), whose last line is short.
template <bool MARKED, bool RAGGED>
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
  const int64_t page_vecs = RAGGED ? p.page_vecs : (int64_t)p.page_lines * kCopyThreads;
  auto in_page = [&](int line) { return !RAGGED || line * kCopyThreads + tid < p.page_vecs; };
  for (int64_t base = first; base <= last; base += kCopyPairs) {
    const int m = (int)min((int64_t)kCopyPairs, last - base + 1);
    __syncthreads();
    if (!MARKED)
      for (int i = tid; i < kCopyFilter / 32; i += kCopyThreads) s_filter[i] = 0;
    int s = 0, d = 0;
    bool out = false;
    if (tid < m) {
      s = p.src[base + tid];
      d = p.dst[base + tid];
    }
    __syncthreads();
    if (tid < m) {
      out = s < 0 || s >= p.num_pages || d < 0 || d >= p.num_pages;
      s_src[tid] = s;
      s_dst[tid] = d;
      s_skip[tid] = out || s == d;
      if (!MARKED && s != d) atomicOr(&s_filter[(d & (kCopyFilter - 1)) >> 5], 1u << (d & 31));
      if (out) report_bad_tables(p.error);
    }
    __syncthreads();
    const int line0 = (int)(max(lo, base * p.page_lines) - base * p.page_lines);
    const int lines = (int)(min(hi, (base + m) * p.page_lines) - base * p.page_lines) - line0;
    CopyAt get{line0 / p.page_lines, line0 % p.page_lines}, put = get;
    auto fetch = [&](int l) {
      if (l < lines) {
        if (!s_skip[get.k] && in_page(get.line)) {
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
    if (MARKED) {
      // one destination, this pair's, and no source
      if (tid < m && !out && s != d && p.marks[d] != 1) {
        s_skip[tid] = 1;
        report_bad_tables(p.error);
      }
    } else {
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
    }
    __syncthreads();
    for (int l = 0; l < lines; ++l) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kCopyDepth - 1) : "memory");
      if (!s_skip[put.k] && in_page(put.line))
        __stcs(p.pages + s_dst[put.k] * page_vecs + put.line * kCopyThreads + tid,
               s_ring[l % kCopyDepth][tid]);
      put.next(p.page_lines);
      fetch(l + kCopyDepth);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
}

template <int D, bool BF16>
cudaError_t launch_append_as(const AppendParams& p, int grid, cudaStream_t stream) {
  const auto kern = p.rope_layout == 1   ? append_kernel<D, BF16, 1>
                    : p.rope_layout == 2 ? append_kernel<D, BF16, 2>
                                         : append_kernel<D, BF16, 0>;
  return launch_pdl(kern, dim3(grid), dim3(kAppendThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, int head_dim, bool bf16, int grid,
                          cudaStream_t stream) {
  if (head_dim == 128)
    return bf16 ? launch_append_as<128, true>(p, grid, stream)
                : launch_append_as<128, false>(p, grid, stream);
  return bf16 ? launch_append_as<64, true>(p, grid, stream)
              : launch_append_as<64, false>(p, grid, stream);
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream) {
  const int cols = p.planes * p.row_vecs;
  const dim3 g(p.tab.batch, (cols + kCompactThreads - 1) / kCompactThreads);
  return launch_pdl(compact_kernel, g, dim3(kCompactThreads), 0, stream, p);
}

namespace {
template <bool RAGGED>
cudaError_t launch_copy_as(const CopyParams& p, int nsm, cudaStream_t stream) {
  const int64_t lines = (int64_t)p.n * p.page_lines;
  const dim3 threads(kCopyThreads);
  // Marking costs two more launches, about 2 us; searching the list costs every
  // CTA 1 us per 1,000 pairs and long equal shares a tenth of a large copy.
  if (lines < kCopyMarkedLines && p.n < kCopyMarkedPairs) {
    const int64_t grid = (lines + 1) / 2 < 5 * nsm ? (lines + 1) / 2 : 5 * nsm;
    return launch_pdl(copy_pages_kernel<false, RAGGED>, dim3((unsigned)grid), threads, 0, stream, p);
  }
  const int64_t blocks = ((int64_t)p.n + kCopyThreads - 1) / kCopyThreads;
  const dim3 marking((unsigned)(blocks < 4 * nsm ? blocks : 4 * nsm));
  cudaError_t e = launch_pdl(mark_pages_kernel<false>, marking, threads, 0, stream, p);
  if (e != cudaSuccess) return e;
  int64_t grid = (lines + 15) / 16;
  if (grid > INT32_MAX) grid = INT32_MAX;
  e = launch_pdl(copy_pages_kernel<true, RAGGED>, dim3((unsigned)grid), threads, 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(mark_pages_kernel<true>, marking, threads, 0, stream, p);
}
}  // namespace

cudaError_t launch_copy_pages(const CopyParams& p, int nsm, cudaStream_t stream) {
  return p.page_vecs == p.page_lines * kCopyThreads ? launch_copy_as<false>(p, nsm, stream)
                                                    : launch_copy_as<true>(p, nsm, stream);
}

}  // namespace ta
