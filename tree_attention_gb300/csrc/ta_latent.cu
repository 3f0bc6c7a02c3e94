// ta_latent.cu -- appending tokens to a paged latent cache.
//
// The cache is [num_pages, 16, rank + rope_dim]: row j of a sequence is its
// token's latent c_j and, behind it, the rotary key k_j that all heads share.
#include <cuda_runtime.h>

#include <cstdint>

#include "ta_latent.cuh"

namespace ta {
namespace {

__device__ __forceinline__ void report_bad_tables(unsigned int* error) {
  atomicOr(error, DEVERR_BAD_INDPTR);
}

// The largest b in [0, batch) with indptr[b] <= t, by one warp: 32 probes a
// round.  Any contents end the search inside the range.
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

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 160;

// The two 16-byte vectors i and i + half_vecs of a rotary row of 16 half_vecs
// elements, turned by (cos, sin) pairs cs: with halves as layout, element e of
// the first is paired with element e of the second; interleaved, neighbours are.
template <bool BF16, int LAYOUT>
__device__ __forceinline__ void turn(uint4& u0, uint4& u1, const float2* cs, int i, int half_vecs) {
  float2 a[4], b[4];
  unpack8<BF16>(u0, a);
  unpack8<BF16>(u1, b);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = a[k], y = b[k];
    if (LAYOUT == 1) {
      const float2 c0 = cs[8 * i + 2 * k], c1 = cs[8 * i + 2 * k + 1];
      a[k] = make_float2(x.x * c0.x - y.x * c0.y, x.y * c1.x - y.y * c1.y);
      b[k] = make_float2(y.x * c0.x + x.x * c0.y, y.y * c1.x + x.y * c1.y);
    } else {
      const float2 c0 = cs[4 * i + k], c1 = cs[4 * (i + half_vecs) + k];
      a[k] = make_float2(x.x * c0.x - x.y * c0.y, x.y * c0.x + x.x * c0.y);
      b[k] = make_float2(y.x * c1.x - y.y * c1.y, y.y * c1.x + y.x * c1.y);
    }
  }
  u0 = pack8<BF16>(a);
  u1 = pack8<BF16>(b);
}

// One CTA per token.  Its last warp looks up the token's cache row and moves the
// latent and the rotary key, the others the heads' rotary queries, whose loads go
// out before the angles are known.
//
//   c = x w / sqrt(mean x^2 + eps),  (a, b) -> (a cos t - b sin t, b cos t + a sin t)
//
// Bound by the memory for long calls: a token's W + h rope_dim elements once each way,
// and its row once more where the rows are wanted.  10,406 tokens of 64 heads, rank
// 512, rotary 64, with rows: 40.0 us, 5.2 TB/s (floor 30.9 us at the measured copy
// rate).  With the row after the queries in the same warps, whose look-ups the queries
// then waited for: 46.5.  32 tokens: 3.1 us, the chain of look-ups (4.5 with the row in
// the queries' warps).
template <bool BF16, int LAYOUT>
__global__ void __launch_bounds__(kAppendThreads) latent_append_kernel(const LatentAppendParams p) {
  __shared__ float2 s_cs[32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = blockIdx.x;
  const int half_vecs = p.rope_dim / 16, width = p.rank + p.rope_dim;
  auto angles = [&](int j) {
    // the fraction of a turn, exact modulo 1, then one rounding to float32
    const uint64_t ph = (uint64_t)(int64_t)p.positions[t] * p.turns[j];
    float sn, cs;
    sincospif((float)(int64_t)ph * 0x1p-63f, &sn, &cs);
    s_cs[j] = make_float2(cs * p.magnitude, sn * p.magnitude);
  };
  if (warp == kAppendThreads / 32 - 1) {
    const int vecs = p.rank / 8;           // 32 or 64
    const uint4* src = reinterpret_cast<const uint4*>(p.latent + t * p.latent_stride);
    const uint4* k = reinterpret_cast<const uint4*>(p.k_rope + t * p.k_rope_stride);
    uint4 u[2], k0, k1;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      u[i] = lane + 32 * i < vecs ? src[lane + 32 * i] : make_uint4(0, 0, 0, 0);
    if (lane < half_vecs) {
      k0 = k[lane];
      k1 = k[lane + half_vecs];
    }
    if (LAYOUT != 0 && lane < p.rope_dim / 2) angles(lane);
    __syncthreads();
    const int b = find_sequence(p.append_indptr, p.tab.batch, t, lane);
    const int a0 = p.append_indptr[b], a1 = p.append_indptr[b + 1];
    const int p0 = p.tab.page_indptr[b], p1 = p.tab.page_indptr[b + 1], last = p.tab.length_info[b];
    int64_t slot = -1;                     // element offset of its row; -1: none
    if (a0 >= 0 && t >= a0 && t < a1 && a1 <= p.total_new && p0 >= 0 && p1 > p0 &&
        p1 <= p.tab.nnz_pages && last >= 1 && last <= kPageSize) {
      const int kv = (p1 - p0 - 1) * kPageSize + last, row = kv - (a1 - t);
      if (kv >= a1 - a0) {
        const int page = p.tab.page_values[p0 + row / kPageSize];
        if (page >= 0 && page < p.tab.num_pages)
          slot = ((int64_t)page * kPageSize + row % kPageSize) * width;
      }
    }
    if (slot < 0 && lane == 0) report_bad_tables(p.error);
    uint16_t* rows = p.rows_out ? p.rows_out + (int64_t)t * width : nullptr;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float2 x[4];
      unpack8<BF16>(u[i], x);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum += x[j].x * x[j].x + x[j].y * x[j].y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = rsqrtf(sum / (float)p.rank + p.eps);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int v = lane + 32 * i;
      if (v >= vecs) continue;
      if (p.weight) {                      // without a norm the latent keeps its bits
        float2 x[4], w[4];
        unpack8<BF16>(u[i], x);
        unpack8<BF16>(reinterpret_cast<const uint4*>(p.weight)[v], w);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[j] = make_float2(x[j].x * inv * w[j].x, x[j].y * inv * w[j].y);
        u[i] = pack8<BF16>(x);
      }
      if (slot >= 0) reinterpret_cast<uint4*>(p.pages + slot)[v] = u[i];
      if (rows) reinterpret_cast<uint4*>(rows)[v] = u[i];
    }
    if (lane < half_vecs) {
      if (LAYOUT != 0) turn<BF16, LAYOUT>(k0, k1, s_cs, lane, half_vecs);
      if (slot >= 0) {
        uint4* to = reinterpret_cast<uint4*>(p.pages + slot + p.rank);
        to[lane] = k0;
        to[lane + half_vecs] = k1;
      }
      if (rows) {
        uint4* to = reinterpret_cast<uint4*>(rows + p.rank);
        to[lane] = k0;
        to[lane + half_vecs] = k1;
      }
    }
    return;
  }
  const int items = p.q_rope != nullptr ? p.h * half_vecs : 0;
  constexpr int kBatch = 4, kStep = kAppendThreads - 32;   // 128 heads of 64 elements at most
  uint4 u0[kBatch], u1[kBatch];
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    const int e = tid + j * kStep;
    if (e < items) {
      const uint4* q = reinterpret_cast<const uint4*>(p.q_rope + t * p.q_token_stride +
                                                      (e / half_vecs) * p.q_head_stride);
      u0[j] = q[e % half_vecs];
      u1[j] = q[e % half_vecs + half_vecs];
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    const int e = tid + j * kStep;
    if (e < items) {
      if (LAYOUT != 0) turn<BF16, LAYOUT>(u0[j], u1[j], s_cs, e % half_vecs, half_vecs);
      uint4* to = reinterpret_cast<uint4*>(p.q_out + t * p.qo_token_stride +
                                           (e / half_vecs) * p.qo_head_stride);
      to[e % half_vecs] = u0[j];
      to[e % half_vecs + half_vecs] = u1[j];
    }
  }
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendParams& p, bool bf16, cudaStream_t stream) {
  auto kern = [&](auto a, auto b, auto c) {
    return p.rope_layout == 1 ? a : p.rope_layout == 2 ? b : c;
  };
  return launch_pdl(bf16 ? kern(latent_append_kernel<true, 1>, latent_append_kernel<true, 2>,
                                latent_append_kernel<true, 0>)
                         : kern(latent_append_kernel<false, 1>, latent_append_kernel<false, 2>,
                                latent_append_kernel<false, 0>),
                    dim3(p.total_new), dim3(kAppendThreads), 0, stream, p);
}

}  // namespace ta
