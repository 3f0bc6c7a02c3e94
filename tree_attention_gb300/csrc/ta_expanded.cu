// ta_expanded.cu -- causal attention in the expanded form of latent attention:
// keys and values per head, and a rotary key that the heads share.
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "ta_device.cuh"
#include "ta_launch.h"

namespace ta {
namespace {

constexpr int kRowThreads = 128;

__device__ __forceinline__ int find_sequence(const int32_t* indptr, int batch, int t, int lane) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 32) / 33;
    const int at = lo + (lane + 1) * step;
    const bool le = at < hi && indptr[at] <= t;
    lo += __popc(__ballot_sync(0xffffffffu, le)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

__device__ __forceinline__ bool good_sequence(const ExpandedParams& p, int b) {
  const int q0 = p.q_indptr[b], q1 = p.q_indptr[b + 1], k0 = p.kv_indptr[b], k1 = p.kv_indptr[b + 1];
  return q0 >= 0 && k0 >= 0 && q1 >= q0 && k1 >= k0 && q1 - q0 <= k1 - k0 &&
         (b > 0 || (q0 == 0 && k0 == 0)) &&
         (b < p.batch - 1 || (q1 == p.total_q && k1 == p.total_kv));
}

// One q row and head by one warp, kv row by kv row; a lane holds D / 32
// elements of a head's part and 2 of the rotary part (lanes below rope_dim / 2).
template <int D, bool BF16>
__device__ void attend_row(const ExpandedParams& p, int b, int row, int h, int lane) {
  constexpr int E = D / 64;
  const int k0 = p.kv_indptr[b];
  const int n = p.kv_indptr[b + 1] - k0 - (p.q_indptr[b + 1] - row) + 1;   // rows it sees
  const uint32_t* qp = reinterpret_cast<const uint32_t*>(p.q + row * p.q_ts + h * p.q_hs);
  const bool rot = lane < p.rope_dim / 2;
  float2 q[E], qr = unpack2<BF16>(rot ? qp[D / 2 + lane] : 0u), o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = unpack2<BF16>(qp[lane + 32 * i]);
    o[i] = make_float2(0.f, 0.f);
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < n; ++j) {
    const int64_t at = k0 + j;
    const uint32_t* kp = reinterpret_cast<const uint32_t*>(p.k + at * p.k_ts + h * p.k_hs);
    const uint32_t* rp = reinterpret_cast<const uint32_t*>(p.k_rope + at * p.kr_ts);
    const uint32_t* vp = reinterpret_cast<const uint32_t*>(p.v + at * p.v_ts + h * p.v_hs);
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < E; ++i) acc = ffma2(q[i], unpack2<BF16>(kp[lane + 32 * i]), acc);
    if (rot) acc = ffma2(qr, unpack2<BF16>(rp[lane]), acc);
    float s = acc.x + acc.y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= p.scale_log2;
    if (s == -INFINITY) continue;
    if (s > m) {
      const float f = ex2_approx(m - s);
      m = s;
      l *= f;
#pragma unroll
      for (int i = 0; i < E; ++i) o[i] = make_float2(o[i].x * f, o[i].y * f);
    }
    const float w = ex2_approx(s - m);
    l += w;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = ffma2(make_float2(w, w), unpack2<BF16>(vp[lane + 32 * i]), o[i]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t at = (int64_t)row * p.h + h;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out + at * D);
#pragma unroll
  for (int i = 0; i < E; ++i) out[lane + 32 * i] = pack2<BF16>(o[i].x * inv, o[i].y * inv);
  if (lane == 0) p.lse[at] = l == 0.f ? -INFINITY : m + log2f(l);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kRowThreads) expanded_rows_kernel(const ExpandedParams p) {
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  bool bad = false;
  for (int b = tid; b < p.batch; b += kRowThreads) bad |= !good_sequence(p, b);
  if (__syncthreads_or(bad)) {
    if (tid == 0) atomicOr(p.error, DEVERR_BAD_INDPTR);
    return;
  }
  const int64_t i = (int64_t)blockIdx.x * (kRowThreads / 32) + (tid >> 5);
  if (i >= (int64_t)p.total_q * p.h) return;
  const int row = (int)(i / p.h);
  attend_row<D, BF16>(p, find_sequence(p.q_indptr, p.batch, row, lane), row, (int)(i % p.h), lane);
}

}  // namespace

cudaError_t launch_expanded(const ExpandedParams& p, int head_dim, bool bf16, int nsm,
                            cudaStream_t stream) {
  (void)nsm;
  const int64_t grid = ceil_div((int64_t)p.total_q * p.h, kRowThreads / 32);
  const auto kern = head_dim == 128
                        ? (bf16 ? expanded_rows_kernel<128, true> : expanded_rows_kernel<128, false>)
                        : (bf16 ? expanded_rows_kernel<64, true> : expanded_rows_kernel<64, false>);
  return launch_pdl(kern, dim3((unsigned)grid), dim3(kRowThreads), 0, stream, p);
}

}  // namespace ta
