// ta_latent.cuh -- what the kernels of absorbed latent attention share: the
// tables of a sequence, and one row's attention computed row by row.
#pragma once

#include <cstdint>

#include "ta_device.cuh"
#include "ta_launch.h"

namespace ta {

// What the tables say of one sequence: its kv rows, tree nodes and q rows.
struct LatentSeq {
  int p0, kv, m0, tree, q0, qo;
  bool good;
};
__device__ __forceinline__ LatentSeq latent_seq(const LatentParams& p, int b) {
  LatentSeq s;
  const int p1 = p.tab.page_indptr[b + 1], last = p.tab.length_info[b];
  s.p0 = p.tab.page_indptr[b];
  s.good = s.p0 >= 0 && p1 >= s.p0 && p1 <= p.tab.nnz_pages &&
           (p1 == s.p0 || (last >= 1 && last <= kPageSize)) && (b > 0 || s.p0 == 0);
  s.kv = s.good && p1 > s.p0 ? (p1 - s.p0 - 1) * kPageSize + last : 0;
  s.m0 = s.tree = 0;
  s.q0 = b;
  s.qo = 1;
  if (p.q_indptr) {
    const int q1 = p.q_indptr[b + 1], m1 = p.mn_indptr[b + 1];
    s.q0 = p.q_indptr[b];
    s.m0 = p.mn_indptr[b];
    s.qo = q1 - s.q0;
    s.tree = m1 - s.m0;
    s.good = s.good && s.q0 >= 0 && s.m0 >= 0 && q1 >= s.q0 && m1 >= s.m0 && s.qo <= s.tree &&
             s.tree <= s.kv && (b > 0 || (s.q0 == 0 && s.m0 == 0)) &&
             (b < p.tab.batch - 1 || (q1 == p.total_q && m1 == p.total_tree));
  }
  return s;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& u, float2 (&x)[4]) {
  x[0] = unpack2<BF16>(u.x);
  x[1] = unpack2<BF16>(u.y);
  x[2] = unpack2<BF16>(u.z);
  x[3] = unpack2<BF16>(u.w);
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
  return make_uint4(pack2<BF16>(x[0].x, x[0].y), pack2<BF16>(x[1].x, x[1].y),
                    pack2<BF16>(x[2].x, x[2].y), pack2<BF16>(x[3].x, x[3].y));
}

// One q row and head by one warp, kv row by kv row, its out elements from e0 to
// e1.  A lane holds 8 elements of every 256 of a latent, and lanes below
// rope_dim / 8 of its rotary key.  For rows in which the matrix products met a
// value that is not finite in a row that does not count.
template <bool BF16>
__device__ __noinline__ void latent_row_exact(const LatentParams& p, int b, int r, int h, int e0,
                                              int e1) {
  const LatentSeq s = latent_seq(p, b);
  const int lane = threadIdx.x & 31;
  const int width = p.rank + p.rope_dim, parts = p.rank / 256;
  const int64_t row = (int64_t)(s.q0 + r) * p.h + h;
  float2 q[3][4], o[2][4];
  const uint4* qp = reinterpret_cast<const uint4*>(p.q + row * width);
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const bool mine = i < 2 ? i < parts : lane < p.rope_dim / 8;
    unpack8<BF16>(mine ? qp[i < 2 ? lane + 32 * i : p.rank / 8 + lane] : zero, q[i]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) o[i][k] = make_float2(0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  const int start = s.kv - s.tree;
  const int2* order = reinterpret_cast<const int2*>(p.tree_order) + s.m0;
  const int enter = s.tree ? order[s.tree - s.qo + r].x : 0;
#pragma unroll 1
  for (int j = 0; j < s.kv; ++j) {
    if (j >= start) {
      const int2 iv = order[j - start];
      if (iv.x > enter || enter >= iv.y) continue;
    }
    const int page = p.tab.page_values[s.p0 + j / kPageSize];
    const bool in = page >= 0 && page < p.tab.num_pages;
    const uint4* kp =
        reinterpret_cast<const uint4*>(p.pages + ((int64_t)page * kPageSize + j % kPageSize) * width);
    float2 x[3][4], acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const bool mine = in && (i < 2 ? i < parts : lane < p.rope_dim / 8);
      unpack8<BF16>(mine ? kp[i < 2 ? lane + 32 * i : p.rank / 8 + lane] : zero, x[i]);
#pragma unroll
      for (int k = 0; k < 4; ++k) acc = ffma2(q[i][k], x[i][k], acc);
    }
    float sc = acc.x + acc.y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sc += __shfl_xor_sync(0xffffffffu, sc, d);
    sc *= p.scale_log2;
    if (sc == -INFINITY) continue;
    if (sc > m) {
      const float f = ex2_approx(m - sc);
      m = sc;
      l *= f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] = make_float2(o[i][k].x * f, o[i][k].y * f);
    }
    const float w = ex2_approx(sc - m);
    l += w;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = ffma2(make_float2(w, w), x[i][k], o[i][k]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint4* out = reinterpret_cast<uint4*>(p.out + row * p.rank);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int v = lane + 32 * i;
    if (i >= parts || 8 * v < e0 || 8 * v >= e1) continue;
#pragma unroll
    for (int k = 0; k < 4; ++k) o[i][k] = make_float2(o[i][k].x * inv, o[i][k].y * inv);
    out[v] = pack8<BF16>(o[i]);
  }
}

}  // namespace ta
