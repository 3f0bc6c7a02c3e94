// ta_latent.cuh -- what the kernels on a latent cache share: the tables of a
// sequence, and eight 16-bit elements as float32 and back.
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

}  // namespace ta
