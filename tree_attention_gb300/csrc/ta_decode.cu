// ta_decode.cu -- attention of one token per sequence over a paged KV cache.
//
//   out = sum_j 2^(s_j - lse) v_j,  s_j = log2(e) sm_scale q.k_j,
//   lse = log2 sum_j 2^s_j
//
// over the kv rows j of a sequence, for the g query heads that share a kv
// head.  Every key and value is read once and serves g heads: g flops per byte
// at 16 bits, far below the ~290 where the tensor cores would bound it, so the
// kernel is built around the loads.
//
// * The unit of work is one page of one kv head, 16 rows of K and of V, each a
//   contiguous block.  The units of the whole batch, numbered kv head by kv head
//   and within one in page-table order, are cut into equal ranges, one per
//   warp of a grid of one CTA per SM: no sequence lengths, however ragged,
//   leave an SM idle, and page_indptr is already the prefix sum this needs.
// * A warp's lanes load their operands of mma.sync straight from global memory
//   in 16-byte pieces, without shared memory: a fragment's element order is
//   free as long as both operands agree, so a lane's 8 consecutive elements
//   are two k-steps of its fragments (keys) or, paired with the neighbouring
//   token's by a byte permute, four m-tiles (values).
// * S^T = K Q^T has 16 tokens by 8 heads, O^T = V^T P^T 16 elements by 8 heads,
//   so g <= 8 heads cost one tile each and the weights pass from one product to
//   the other by a transposition within registers (movmatrix).
// * A page's keys are consumed by the first product before its softmax, and
//   the next page's are requested into the same registers right there (and so
//   the values after the second product): each warp always has a page in
//   flight with no second set of registers.
// * A range may hold parts of several sequences.  A sequence that lies in one
//   warp's range is written by it; the parts of one that spans warps are
//   merged in shared memory, and of one that spans CTAs by the last of its
//   CTAs to finish (a counter), in CTA order, so results do not depend on
//   timing.
//
// Measured (h_q 64, h_kv 8, d 128, bf16, 64 sequences of 16 to 16,384 rows,
// 880 MB): 134 us, 6.6 TB/s, the rate of a plain copy; 4 sequences of 33,000
// rows: 84.5 us, 6.4 TB/s; one of 4,096 rows (16 kv heads): 12.5 us, of which 2
// are the chain of loads before the first page and 3 the merges; 256 of about 110
// rows (h 32 / 8): 27 us, 66 % of the memory rate: 3 us before the first page, 16
// for eight pages per warp, and 3 for the merges, as nearly every warp ends with
// parts of two sequences and an SM with those of 13.  9 to 16 heads per kv head
// run at 52 to 55 % of the memory rate (two tiles of heads leave 8 warps per SM);
// above, every 16 heads' CTAs read the pages again: 32 heads 34 %, 40 heads 28 %,
// 64 heads 23 %, 128 heads 13 %.
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdint>

#include "ta_device.cuh"
#include "ta_launch.h"

namespace ta {
namespace {

// 16 bytes that are read once: not kept in L1.
__device__ __forceinline__ uint4 load_stream(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Of two packed numbers, the infinite and NaN ones (all exponent bits set).
template <bool BF16>
__device__ __forceinline__ uint32_t not_finite_of(uint32_t u) {
  constexpr uint32_t kExponent = BF16 ? 0x7f807f80u : 0x7c007c00u;
  return u & __vcmpeq2(u & kExponent, kExponent);
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// NT tiles of 8 heads per warp.  The warps per CTA follow from the registers a
// lane needs (a page of K and of V, Q, O: 32 + 32 + 16 NT + 32 NT for d = 128).
template <int D, int NT>
struct Shape {
  static constexpr int kWarps = D == 128 ? (NT == 1 ? 12 : 8) : (NT == 1 ? 16 : 12);
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kHeads = 8 * NT;
  static constexpr int kState = kHeads * D + 2 * kHeads;   // floats: O, then m, then l
  static constexpr int kPieces = 2 * kWarps;               // parts a CTA can hold
  static_assert(kPieces <= 32, "one lane per part");
  static_assert(kPieces * kState >= 12 * kThreads, "the last merge's sums of two sequences fit");
};

// U units over up to ``grid`` CTAs of W warps, a unit per warp at least.
__host__ __device__ __forceinline__ DecodeSplit decode_split(int U, int grid, int W) {
  DecodeSplit s{};
  s.ctas = (U + W - 1) / W < grid ? (U + W - 1) / W : grid;
  if (s.ctas > 0) {
    s.per = U / (s.ctas * W);
    s.extra = U % (s.ctas * W);
  }
  return s;
}

// The largest b with s_indptr[b] <= x, over batch sequences; by one warp.
__device__ __forceinline__ int find_in(const int32_t* s_indptr, int batch, int x, int lane) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 32) / 33;
    const int at = lo + (lane + 1) * step;
    const bool le = at < hi && s_indptr[at] <= x;
    lo += __popc(__ballot_sync(0xffffffffu, le)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// One thread's 4 elements of a state: O relative to m, and l.
struct Acc {
  float m, l;
  float4 o;
  // n states more, the largest m first, so that their factors are independent
  template <int n>
  __device__ __forceinline__ void add(const float (&pm)[n], const float (&pl)[n],
                                      const float4 (&y)[n]) {
    float top = m;
#pragma unroll
    for (int k = 0; k < n; ++k) top = fmaxf(top, pm[k]);
    const float f = ex2_approx(m - top);
    m = top;
    l *= f;
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const float w = ex2_approx(pm[k] - top);
      l += pl[k] * w;
      o.x += y[k].x * w;
      o.y += y[k].y * w;
      o.z += y[k].z * w;
      o.w += y[k].w * w;
    }
  }
  // Where the sum over the states ``o_of(k)``, k = from, from + step .. below to,
  // is not finite: factors are positive, but may have underflowed to zero, so it
  // is the sum of the states' infinities and NaNs, if there are any.
  template <typename F>
  __device__ __forceinline__ void keep_infinities(int from, int to, int step, F o_of) {
    if (__builtin_expect(finite((o.x + o.y) + (o.z + o.w)), 1)) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k = from; k < to; k += step) {
      const float4 y = o_of(k);
      s.x += finite(y.x) ? 0.f : y.x;
      s.y += finite(y.y) ? 0.f : y.y;
      s.z += finite(y.z) ? 0.f : y.z;
      s.w += finite(y.w) ? 0.f : y.w;
    }
    o.x = finite(s.x) ? o.x : s.x;
    o.y = finite(s.y) ? o.y : s.y;
    o.z = finite(s.z) ? o.z : s.z;
    o.w = finite(s.w) ? o.w : s.w;
  }
};

template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::kThreads, 1)
    decode_kernel(const DecodeParams p) {
  using S = Shape<D, NT>;
  constexpr int W = S::kWarps, KS = D / 32, VH = D / 64;
  // the exponent that a weight may reach over its reference, and where a moved
  // reference puts the largest: fp16 weights are held 2^7 higher than bf16
  // ones, as what lies 2^-24 below a weight of one is the type's end and long
  // sequences have mass there
  constexpr float kTop = BF16 ? 8.f : 15.f, kRef = BF16 ? 0.f : 7.f;
  extern __shared__ __align__(16) float s_state[];         // [kPieces][kState]
  int32_t* s_indptr = reinterpret_cast<int32_t*>(s_state + S::kPieces * S::kState);
  uint8_t* s_len = reinterpret_cast<uint8_t*>(s_indptr + p.tab.batch + 1);
  __shared__ int2 s_seg[S::kPieces];                       // each part's sequence (or -1) and kv head
  __shared__ int s_part[S::kPieces];                       // the parts there are, in range order
  __shared__ int4 s_group[S::kPieces];                     // runs of s_part of one sequence
  __shared__ int2 s_group_at[S::kPieces];
  __shared__ int s_groups, s_merge[2];
  __shared__ int4 s_shared[2];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3;
  const int batch = p.tab.batch;

  // the first of the table's entries that this thread checks
  int first = 0, first_next = 0, first_len = 0;
  if (tid <= batch) first = p.tab.page_indptr[tid];
  if (tid < batch) {
    first_next = p.tab.page_indptr[tid + 1];
    first_len = p.tab.length_info[tid];
  }
  // This CTA's and this warp's range of units: U = warps * per + extra units,
  // one more for each of the first ``extra`` warps.  The table is usually as
  // long as its array, for which the host has divided: its first entries are
  // on their way while its offsets arrive.
  const int group = blockIdx.y, cta = blockIdx.x;          // group: of the heads of one kv head
  int P = p.tab.nnz_pages, u = 0, u_end = 0, pv = 0;
  DecodeSplit sp = p.split;
  auto range_start = [&](int w) { return w * sp.per + min(w, sp.extra); };
  // physical pages of the 32 units from x on, one per lane
  auto pages_at = [&](int x) {
    return x + lane < u_end ? p.tab.page_values[(x + lane) % P] : 0;
  };
  auto set_range = [&]() {
    if (cta >= sp.ctas) return;
    u = range_start(cta * W + warp);
    u_end = range_start(cta * W + warp + 1);
    pv = pages_at(u);
  };
  set_range();

  // the page table's offsets and last lengths, checked as a whole
  bool bad = false;
  for (int i = tid; i <= batch; i += S::kThreads) {
    const int a = i == tid ? first : p.tab.page_indptr[i];
    s_indptr[i] = a;
    bad |= i == 0 ? a != 0 : a < 0 || a > p.tab.nnz_pages;
    if (i < batch) {
      const int e = i == tid ? first_next : p.tab.page_indptr[i + 1];
      const int len = i == tid ? first_len : p.tab.length_info[i];
      bad |= e < a || (e > a && (len < 1 || len > kPageSize));
      s_len[i] = (uint8_t)len;
    }
  }
  if (tid < S::kPieces) s_seg[tid].x = -1;
  if (tid < 2) s_shared[tid].w = 0;
  if (__syncthreads_or(bad)) {
    if (tid == 0) atomicOr(p.error, DEVERR_BAD_INDPTR);
    return;
  }
  if (s_indptr[batch] != P) {
    P = s_indptr[batch];
    sp = decode_split(P * p.h_kv, gridDim.x, W);
    u = u_end = 0;
    set_range();
  }
  // sequences without rows
  for (int b = group * gridDim.x + cta; b < batch; b += gridDim.x * gridDim.y) {
    if (s_indptr[b] != s_indptr[b + 1]) continue;
    uint4* o = reinterpret_cast<uint4*>(p.out + (size_t)b * p.h_q * D);
    for (int i = tid; i < p.h_q * (D / 8); i += S::kThreads) o[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < p.h_q; i += S::kThreads) p.lse[(size_t)b * p.h_q + i] = -INFINITY;
  }
  if (cta >= sp.ctas) return;
  const int head0 = group * S::kHeads;                     // of the kv head's g
  const int u_first = u;
  const bool work = u < u_end;
  int kvh = u / P, pg = u % P, b = 0, seg_end = 0, ahead = u, pv_next = 0;
  uint4 qf[NT][KS], kf[2][KS], vf[4][VH];
  const uint16_t* k_page = nullptr;   // the page whose values are still to be requested
  int rows = 0;                       // its rows that count; 0 for zeros
  auto load_q = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int h = head0 + n * 8 + r;
      const uint16_t* q = p.q + ((size_t)b * p.h_q + (size_t)kvh * p.g + h) * D + 8 * c;
#pragma unroll
      for (int s = 0; s < KS; ++s)
        qf[n][s] = h < p.g ? load_stream(q + 32 * s) : make_uint4(0, 0, 0, 0);
    }
  };
  auto load_k = [&]() {               // of unit u; sets k_page and rows
    const int page = __shfl_sync(0xffffffffu, pv, u - ahead);
    const bool in = page >= 0 && page < p.tab.num_pages;
    rows = in ? (pg + 1 == seg_end ? s_len[b] : kPageSize) : 0;
    k_page = p.pages + ((int64_t)page * 2 * p.h_kv + kvh) * (kPageSize * D);
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        kf[i][s] = in ? load_stream(k_page + (r + 8 * i) * D + 32 * s + 8 * c)
                      : make_uint4(0, 0, 0, 0);
  };
  auto load_v = [&]() {
    const uint16_t* v = k_page + (int64_t)p.h_kv * kPageSize * D + 8 * r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = 2 * c + (i & 1) + 8 * (i >> 1);
#pragma unroll
      for (int h = 0; h < VH; ++h)    // a slot past the last row may hold anything
        vf[i][h] = tok < rows ? load_stream(v + tok * D + 64 * h) : make_uint4(0, 0, 0, 0);
    }
  };
  float o[NT][4 * VH][4], m[NT][2], l[NT][2];
  auto reset = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -FLT_MAX;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int t = 0; t < 4 * VH; ++t) o[n][t][0] = o[n][t][1] = o[n][t][2] = o[n][t][3] = 0.f;
    }
  };
  if (work) {
    pv_next = pages_at(u + 32);
    b = find_in(s_indptr, batch, pg, lane);
    seg_end = s_indptr[b + 1];
    load_q();
    load_k();
    load_v();
    // the sequences that this range shares with others: one that began before
    // it, one that goes on behind it
    const int last = u_end - 1, kvh_last = last / P;
    const int b_last = find_in(s_indptr, batch, last % P, lane);
    if (lane == 0) {
      if (kvh * P + s_indptr[b] < u) s_seg[2 * warp] = make_int2(b, kvh);
      const int at = kvh_last * P;
      if (at + s_indptr[b_last] >= u && at + s_indptr[b_last + 1] > u_end)
        s_seg[2 * warp + 1] = make_int2(b_last, kvh_last);
    }
  }
  __syncthreads();
  // The parts that the warps will leave in shared memory, listed in range order,
  // and the runs of parts of one sequence: {first part, one past the last, slot,
  // -}, slot -1 for a sequence that lies in this CTA, else 0 where its start does
  // not, 1 where it does.  Read behind the barrier after the loop.
  const int c_lo = range_start(cta * W), c_hi = range_start(cta * W + W);
  if (warp == 0) {
    const int2 seg = lane < S::kPieces ? s_seg[lane] : make_int2(-1, 0);
    const unsigned have = __ballot_sync(0xffffffffu, seg.x >= 0);
    const unsigned below = have & ((1u << lane) - 1);
    const int before = below ? 31 - __clz(below) : lane;   // the part before this one
    const int2 prev = make_int2(__shfl_sync(0xffffffffu, seg.x, before),
                                __shfl_sync(0xffffffffu, seg.y, before));
    const bool head = seg.x >= 0 && (!below || prev.x != seg.x || prev.y != seg.y);
    const unsigned starts = __ballot_sync(0xffffffffu, head);
    if (seg.x >= 0) s_part[__popc(below)] = lane;
    if (head) {
      const unsigned after = starts & ~(0xffffffffu >> (31 - lane));
      const int next = after ? __ffs(after) - 1 : 32;
      const int lo = seg.y * P + s_indptr[seg.x], hi = seg.y * P + s_indptr[seg.x + 1];
      const int slot = lo >= c_lo && hi <= c_hi ? -1 : lo >= c_lo ? 1 : 0;
      const int at = __popc(starts & ((1u << lane) - 1));
      s_group[at] = make_int4(__popc(below), next == 32 ? __popc(have) : __popc(have & ((1u << next) - 1)),
                              slot, 0);
      s_group_at[at] = seg;
      if (slot >= 0) {
        // the CTAs that hold a part of it
        auto cta_of = [&](int x) {
          const int wide = sp.extra * (sp.per + 1);
          return (x < wide ? x / (sp.per + 1) : sp.extra + (x - wide) / sp.per) / W;
        };
        const int first = cta_of(lo);
        s_shared[slot] = make_int4(seg.x, seg.y, first, cta_of(hi - 1) - first + 1);
      }
    }
    if (lane == 0) s_groups = __popc(starts);
  }
  if (work) {
    reset();
    while (true) {
      // scores of the page's 16 tokens
      float x[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float y[4] = {0.f, 0.f, 0.f, 0.f};
        x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          mma16816<BF16>(x[n], kf[0][s].x, kf[1][s].x, kf[0][s].y, kf[1][s].y, qf[n][s].x, qf[n][s].y);
          mma16816<BF16>(y, kf[0][s].z, kf[1][s].z, kf[0][s].w, kf[1][s].w, qf[n][s].z, qf[n][s].w);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] = (x[n][i] + y[i]) * p.scale_log2;
      }
      const bool seg_done = pg + 1 == seg_end;
      const int len = seg_done ? s_len[b] : kPageSize;
      const int b_now = b, kvh_now = kvh;
      // the next unit's keys (and queries)
      ++u;
      const bool more = u < u_end;
      if (more) {
        if (++pg == P) {
          pg = 0;
          ++kvh;
          b = -1;
          seg_end = 0;
        }
        if (pg == seg_end) {
          do ++b;
          while (s_indptr[b + 1] == pg);
          seg_end = s_indptr[b + 1];
        }
        if (u - ahead == 32) {
          ahead = u;
          pv = pv_next;
          pv_next = pages_at(u + 32);
        }
        load_k();
        if (seg_done) load_q();
      }
      // weights
      if (len < kPageSize) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (r + 8 * (i >> 1) >= len) x[n][i] = -INFINITY;
      }
      bool over = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) over |= x[n][i] - m[n][i & 1] > kTop;
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float top = fmaxf(x[n][j], x[n][j + 2]);
#pragma unroll
            for (int i = 4; i <= 16; i <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
            const float moved = fmaxf(m[n][j], top - kRef);
            const float f = ex2_approx(m[n][j] - moved);
            m[n][j] = moved;
            l[n][j] *= f;
#pragma unroll
            for (int t = 0; t < 4 * VH; ++t) {
              o[n][t][j] *= f;
              o[n][t][j + 2] *= f;
            }
          }
      }
      uint32_t w0[NT][2], w1[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] = ex2_approx(x[n][i] - m[n][i & 1]);
        l[n][0] += x[n][0] + x[n][2];
        l[n][1] += x[n][1] + x[n][3];
        // the tensor cores take a weight as two 16-bit numbers, its rounding and
        // what that left (2^-16 of it or less is lost), so that the output is
        // rounded once; measured free up to 8 heads per kv head (the loads bound
        // the loop), 2 % slower for 16.  The sum l takes the weights as they are
        const uint32_t h0 = pack2<BF16>(x[n][0], x[n][1]), h1 = pack2<BF16>(x[n][2], x[n][3]);
        const float2 g0 = unpack2<BF16>(h0), g1 = unpack2<BF16>(h1);
        w0[n][0] = transpose8x8(h0);
        w1[n][0] = transpose8x8(h1);
        w0[n][1] = transpose8x8(pack2<BF16>(x[n][0] - g0.x, x[n][1] - g0.y));
        w1[n][1] = transpose8x8(pack2<BF16>(x[n][2] - g1.x, x[n][3] - g1.y));
      }
#pragma unroll
      for (int h = 0; h < VH; ++h)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t v0 = word(vf[0][h], t), v1 = word(vf[1][h], t);
          const uint32_t v2 = word(vf[2][h], t), v3 = word(vf[3][h], t);
          const uint32_t a0 = __byte_perm(v0, v1, 0x5410), a1 = __byte_perm(v0, v1, 0x7632);
          const uint32_t a2 = __byte_perm(v2, v3, 0x5410), a3 = __byte_perm(v2, v3, 0x7632);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816<BF16>(o[n][4 * h + t], a0, a1, a2, a3, w0[n][0], w1[n][0]);
            mma16816<BF16>(o[n][4 * h + t], a0, a1, a2, a3, w0[n][1], w1[n][1]);
          }
        }
      if (more) load_v();
      if (!seg_done && more) continue;

      // the end of a sequence or of the range
      const int seg_lo = kvh_now * P + s_indptr[b_now];
      const bool whole = seg_done && seg_lo >= u_first;
      const int piece = 2 * warp + (seg_lo >= u_first ? 1 : 0);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float z = l[n][j];
#pragma unroll
          for (int i = 4; i <= 16; i <<= 1) z += __shfl_xor_sync(0xffffffffu, z, i);
          l[n][j] = z;
          const int h = n * 8 + 2 * c + j;
          if (whole) {
            if (head0 + h < p.g) {
              const float inv = z > 0.f || z != z ? 1.f / z : 0.f;
              const size_t row = (size_t)b_now * p.h_q + (size_t)kvh_now * p.g + head0 + h;
#pragma unroll
              for (int v = 0; v < VH; ++v) {
                uint32_t y[4];
#pragma unroll
                for (int t = 0; t < 4; ++t)
                  y[t] = pack2<BF16>(o[n][4 * v + t][j] * inv, o[n][4 * v + t][j + 2] * inv);
                *reinterpret_cast<uint4*>(p.out + row * D + 64 * v + 8 * r) =
                    make_uint4(y[0], y[1], y[2], y[3]);
              }
              if (r == 0) p.lse[row] = m[n][j] + log2f(z);
            }
          } else {
            float* st = s_state + piece * S::kState;
#pragma unroll
            for (int v = 0; v < VH; ++v) {
              float4* y = reinterpret_cast<float4*>(st + h * D + 64 * v + 8 * r);
              y[0] = make_float4(o[n][4 * v][j], o[n][4 * v][j + 2], o[n][4 * v + 1][j],
                                 o[n][4 * v + 1][j + 2]);
              y[1] = make_float4(o[n][4 * v + 2][j], o[n][4 * v + 2][j + 2], o[n][4 * v + 3][j],
                                 o[n][4 * v + 3][j + 2]);
            }
            if (r == 0) {
              st[S::kHeads * D + h] = m[n][j];
              st[S::kHeads * D + S::kHeads + h] = z;
            }
          }
        }
      // A sum that is not finite: weights are positive, so it is the sum of its
      // column's infinities and NaNs, if there are any, but the products above
      // need not give that, as a weight's second part may be zero or negative and
      // small weights and factors round to zero.  The segment's values are read
      // again, a tile of elements at a time, with weights of one.  (To look at every
      // value before its product cost 1 to 5 %, to look at the sums here and where
      // parts are merged 0.4 us a call at most)
      float2 odd = make_float2(0.f, 0.f);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < 4 * VH; ++t) {
          odd = ffma2(make_float2(o[n][t][0], o[n][t][1]), make_float2(0.f, 0.f), odd);
          odd = ffma2(make_float2(o[n][t][2], o[n][t][3]), make_float2(0.f, 0.f), odd);
        }
      if (__builtin_expect(__any_sync(0xffffffffu, odd.x != 0.f || odd.y != 0.f), 0)) {
        constexpr uint32_t kOnes = BF16 ? 0x3f803f80u : 0x3c003c00u;
        const int at0 = max(seg_lo, u_first) - kvh_now * P, at1 = u - kvh_now * P;
#pragma unroll 1
        for (int t = 0; t < 4 * VH; ++t) {
          const int elem = 64 * (t / 4) + 8 * r + 2 * (t % 4);      // and the next one
          float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
          for (int at = at0; at < at1; ++at) {
            const int page = p.tab.page_values[at];
            const int in = page < 0 || page >= p.tab.num_pages  ? 0
                           : at + 1 == s_indptr[b_now + 1] ? s_len[b_now] : kPageSize;
            const uint16_t* v =
                p.pages + (((int64_t)page * 2 + 1) * p.h_kv + kvh_now) * (kPageSize * D) + elem;
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int tok = 2 * c + (i & 1) + 8 * (i >> 1);
              w[i] = tok < in ? not_finite_of<BF16>(*reinterpret_cast<const uint32_t*>(v + tok * D)) : 0;
            }
            mma16816<BF16>(y, __byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632),
                           __byte_perm(w[2], w[3], 0x5410), __byte_perm(w[2], w[3], 0x7632), kOnes, kOnes);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int h = n * 8 + 2 * c + j;
              if (whole) {
                // as above; a row whose sum of weights is NaN stays NaN
                uint16_t* out = p.out + ((size_t)b_now * p.h_q + (size_t)kvh_now * p.g + head0 + h) * D + elem;
                const uint32_t both = pack2<BF16>(y[j] + 0.f * l[n][j], y[j + 2] + 0.f * l[n][j]);
                if (head0 + h < p.g && !finite(y[j])) out[0] = (uint16_t)both;
                if (head0 + h < p.g && !finite(y[j + 2])) out[1] = (uint16_t)(both >> 16);
              } else {
                float* st = s_state + piece * S::kState + h * D + elem;
                if (!finite(y[j])) st[0] = y[j];
                if (!finite(y[j + 2])) st[1] = y[j + 2];
              }
            }
        }
      }
      if (!more) break;
      reset();
    }
  }
  __syncthreads();

  constexpr int V4 = D / 4;
  const int heads = min(S::kHeads, p.g - head0), items = heads * V4;
  auto finish = [&](int2 at, int h, int i, const Acc& a) {
    const float inv = a.l > 0.f || a.l != a.l ? 1.f / a.l : 0.f;
    const size_t row = (size_t)at.x * p.h_q + (size_t)at.y * p.g + head0 + h;
    reinterpret_cast<uint2*>(p.out + row * D)[i] = make_uint2(
        pack2<BF16>(a.o.x * inv, a.o.y * inv), pack2<BF16>(a.o.z * inv, a.o.w * inv));
    if (i == 0) p.lse[row] = a.m + log2f(a.l);
  };
  auto part_of = [&](int c, int slot) {    // of CTA c of this head group, in the workspace
    return p.parts + (((size_t)group * gridDim.x + c) * 2 + slot) * S::kState;
  };
  const int n_groups = s_groups;
  for (int e = tid; e < n_groups * items; e += S::kThreads) {
    const int h = e % items / V4, i = e % V4;
    const int4 grp = s_group[e / items];
    Acc a{-FLT_MAX, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    constexpr int kBatch = 4;
    for (int k0 = grp.x; k0 < grp.y; k0 += kBatch) {
      float pm[kBatch], pl[kBatch];
      float4 y[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const bool is = k0 + k < grp.y;
        const float* st = s_state + s_part[is ? k0 + k : k0] * S::kState;
        pm[k] = is ? st[S::kHeads * D + h] : -FLT_MAX;
        pl[k] = is ? st[S::kHeads * D + S::kHeads + h] : 0.f;
        y[k] = is ? reinterpret_cast<const float4*>(st + h * D)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      a.add(pm, pl, y);
    }
    a.keep_infinities(grp.x, grp.y, 1, [&](int k) {
      return reinterpret_cast<const float4*>(s_state + s_part[k] * S::kState + h * D)[i];
    });
    if (grp.z < 0) {
      finish(s_group_at[e / items], h, i, a);
    } else {
      float* st = part_of(cta, grp.z);
      __stcg(reinterpret_cast<float4*>(st + h * D) + i, a.o);
      if (i == 0) {
        __stcg(st + S::kHeads * D + h, a.m);
        __stcg(st + S::kHeads * D + S::kHeads + h, a.l);
      }
    }
  }
  if (s_shared[0].w == 0 && s_shared[1].w == 0) return;

  // sequences that several CTAs share: the last of these to come here merges
  __syncthreads();
  if (tid < 2) {
    const int4 sh = s_shared[tid];
    int merge = 0;
    if (sh.w > 0) {
      int* n = p.counters + ((size_t)sh.y * batch + sh.x) * gridDim.y + group;
      // releases the parts that this CTA's threads wrote before the barrier and
      // acquires the others' (fences around a plain atomic took 0.3 us more)
      int before;
      asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                   : "=r"(before)
                   : "l"(n)
                   : "memory");
      merge = before == sh.w - 1;
      if (merge) *n = 0;
    }
    s_merge[tid] = merge;
  }
  __syncthreads();
  if (!s_merge[0] && !s_merge[1]) return;
  // A thread has kBatch parts of an element in flight at once; more parts go to
  // more threads, as far as one sequence's elements leave any: whether this CTA
  // merges one sequence or both depends on which CTAs end last, and the order of
  // the sums must not.
  constexpr int kBatch = 8;
  const int most = max(1, S::kThreads / items);
  const int share0 = s_merge[0] ? min((s_shared[0].w + kBatch - 1) / kBatch, most) : 0;
  const int share1 = s_merge[1] ? min((s_shared[1].w + kBatch - 1) / kBatch, most) : 0;
  float* s_ml = s_state;                                                // [share][items][2]
  float4* s_o = reinterpret_cast<float4*>(s_state + 4 * S::kThreads);   // [share][items]
  for (int e = tid; e < items * (share0 + share1); e += S::kThreads) {
    const int slot = e >= items * share0;
    const int4 sh = s_shared[slot];
    const int share = slot ? share1 : share0, y0 = slot ? e - items * share0 : e;
    const int x = y0 % items, h = x / V4, i = x % V4;
    // of its CTAs the first holds the sequence's start, its second part
    auto part = [&](int k) {
      return part_of(sh.z + k, k == 0);
    };
    Acc a{-FLT_MAX, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int k0 = y0 / items; k0 < sh.w; k0 += share * kBatch) {
      float pm[kBatch], pl[kBatch];
      float4 y[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        pm[k] = -FLT_MAX;
        pl[k] = 0.f;
        y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + k * share < sh.w) {
          const float* st = part(k0 + k * share);
          y[k] = __ldcg(reinterpret_cast<const float4*>(st + h * D) + i);
          pm[k] = __ldcg(st + S::kHeads * D + h);
          pl[k] = __ldcg(st + S::kHeads * D + S::kHeads + h);
        }
      }
      a.add(pm, pl, y);
    }
    a.keep_infinities(y0 / items, sh.w, share, [&](int k) {
      return __ldcg(reinterpret_cast<const float4*>(part(k) + h * D) + i);
    });
    if (share == 1) {
      finish(make_int2(sh.x, sh.y), h, i, a);
    } else {
      s_ml[2 * e] = a.m;
      s_ml[2 * e + 1] = a.l;
      s_o[e] = a.o;
    }
  }
  if (share0 <= 1 && share1 <= 1) return;
  __syncthreads();
  for (int x = tid; x < 2 * items; x += S::kThreads) {
    const int slot = x >= items, share = slot ? share1 : share0;
    if (share <= 1) continue;
    const int e0 = (slot ? items * share0 : 0) + x - slot * items;
    Acc a{s_ml[2 * e0], s_ml[2 * e0 + 1], s_o[e0]};
    for (int k = 1; k < share; ++k) {
      const int e = e0 + k * items;
      a.add({s_ml[2 * e]}, {s_ml[2 * e + 1]}, {s_o[e]});
    }
    a.keep_infinities(0, share, 1, [&](int k) { return s_o[e0 + k * items]; });
    finish(make_int2(s_shared[slot].x, s_shared[slot].y), x % items / V4, x % V4, a);
  }
}

// CTAs that work on one head group: one CTA per SM in all.
int ctas_per_group(int nsm, int groups) {
  return nsm / groups > 0 ? nsm / groups : 1;
}

template <int D, bool BF16, int NT>
cudaError_t launch(const DecodeParams& p, int nsm, cudaStream_t stream) {
  using S = Shape<D, NT>;
  const size_t smem = (size_t)S::kPieces * S::kState * 4 + (size_t)(p.tab.batch + 1) * 4 + p.tab.batch;
  const auto kern = decode_kernel<D, BF16, NT>;
  static std::atomic<uint64_t> allowed{0};   // for the most that any batch needs
  const cudaError_t e = allow_shared(
      (const void*)kern, S::kPieces * S::kState * 4 + kMaxCacheBatch * 5 + 4, allowed);
  if (e != cudaSuccess) return e;
  const int per_group = ctas_per_group(nsm, p.groups);
  DecodeParams dp = p;
  dp.split = decode_split(p.tab.nnz_pages * p.h_kv, per_group, S::kWarps);
  return launch_pdl(kern, dim3(per_group, p.groups), dim3(S::kThreads), smem, stream, dp);
}

template <int D, bool BF16>
cudaError_t launch_heads(const DecodeParams& p, int nsm, cudaStream_t stream) {
  return p.g <= 8 ? launch<D, BF16, 1>(p, nsm, stream) : launch<D, BF16, 2>(p, nsm, stream);
}

}  // namespace

CacheWorkspace cache_workspace(int batch, int num_pages, int h_kv, int g, int nsm) {
  constexpr int kGroups = kMaxGroup / 16;   // most head groups
  CacheWorkspace w{};
  const int heads = g <= 8 ? 8 : 16;
  w.groups = (g + heads - 1) / heads;
  w.off_parts = 256;
  // room for any heads: parts of one call must not lie over another's marks or
  // counters, which have to be zero
  const int64_t ctas = nsm > kGroups ? nsm : kGroups;
  w.off_marks = w.off_parts + round_up(ctas * 2 * Shape<128, 2>::kState * 4, 256);
  w.off_counters = w.off_marks + round_up((int64_t)num_pages * 4, 256);
  w.total = w.off_counters + round_up((int64_t)batch * h_kv * w.groups * 4, 256);
  return w;
}

cudaError_t launch_decode(const DecodeParams& p, int head_dim, bool bf16, int nsm,
                          cudaStream_t stream) {
  if (head_dim == 128)
    return bf16 ? launch_heads<128, true>(p, nsm, stream) : launch_heads<128, false>(p, nsm, stream);
  return bf16 ? launch_heads<64, true>(p, nsm, stream) : launch_heads<64, false>(p, nsm, stream);
}

}  // namespace ta
