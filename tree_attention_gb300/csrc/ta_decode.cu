// ta_decode.cu -- attention of one token per sequence over a paged KV cache.
#include <cuda_runtime.h>

#include <cstdint>

#include "ta_device.cuh"
#include "ta_launch.h"

namespace ta {
namespace {

constexpr int kDecodeThreads = 128;

// One CTA per (q head, sequence); each warp takes every fourth kv row with a
// running maximum and sum, then the warps' states are merged.
template <int D, bool BF16>
__global__ void __launch_bounds__(kDecodeThreads) decode_kernel(const DecodeParams p) {
  constexpr int V = D / 32, W = kDecodeThreads / 32;
  __shared__ float s_o[W][D], s_m[W], s_l[W];
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.x, b = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  bool bad = false;
  for (int i = threadIdx.x; i < p.tab.batch; i += kDecodeThreads) {
    const int p0 = p.tab.page_indptr[i], p1 = p.tab.page_indptr[i + 1];
    const int last = p.tab.length_info[i];
    bad |= p0 < 0 || p1 < p0 || p1 > p.tab.nnz_pages || (i == 0 && p0 != 0) ||
           (p1 > p0 && (last < 1 || last > kPageSize));
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) atomicOr(p.error, DEVERR_BAD_INDPTR);
    return;
  }
  const int p0 = p.tab.page_indptr[b], np = p.tab.page_indptr[b + 1] - p0;
  const int kv = np > 0 ? (np - 1) * kPageSize + p.tab.length_info[b] : 0;
  const size_t row_q = (size_t)b * p.h_q + h;
  float q[V], o[V], m = -INFINITY, l = 0.f, lc = 0.f;
  for (int i = 0; i < V; ++i) {
    q[i] = unpack2<BF16>(p.q[row_q * D + lane * V + i]).x;
    o[i] = 0.f;
  }
  for (int r = warp; r < kv; r += W) {
    const int page = p.tab.page_values[p0 + r / kPageSize];
    const bool in = page >= 0 && page < p.tab.num_pages;
    const uint16_t* k = p.pages + (((size_t)page * 2 * p.h_kv + h / p.g) * kPageSize + r % kPageSize) * D;
    const uint16_t* v = k + (size_t)p.h_kv * kPageSize * D;
    float s = 0.f, x[V];
    for (int i = 0; i < V; ++i) {
      s += in ? q[i] * unpack2<BF16>(k[lane * V + i]).x : 0.f;
      x[i] = in ? unpack2<BF16>(v[lane * V + i]).x : 0.f;
    }
    for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    // compensated: thousands of small weights next to a large one must count
    const float lf = l * f, ls = lf + w;
    lc = lc * f + (lf >= w ? (lf - ls) + w : (w - ls) + lf);
    l = ls;
    for (int i = 0; i < V; ++i) o[i] = o[i] * f + w * x[i];
  }
  for (int i = 0; i < V; ++i) s_o[warp][lane * V + i] = o[i];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l + lc;
  }
  __syncthreads();
  float mm = -INFINITY, ll = 0.f;
  for (int w = 0; w < W; ++w) mm = fmaxf(mm, s_m[w]);
  for (int w = 0; w < W; ++w) ll += s_l[w] > 0.f ? s_l[w] * exp2f(s_m[w] - mm) : 0.f;
  for (int i = threadIdx.x; i < D; i += kDecodeThreads) {
    float acc = 0.f;
    for (int w = 0; w < W; ++w) acc += s_l[w] > 0.f ? s_o[w][i] * exp2f(s_m[w] - mm) : 0.f;
    p.out[row_q * D + i] = (uint16_t)pack2<BF16>(ll > 0.f ? acc / ll : 0.f, 0.f);
  }
  if (threadIdx.x == 0) p.lse[row_q] = ll > 0.f ? mm + log2f(ll) : -INFINITY;
}

}  // namespace

cudaError_t launch_decode(const DecodeParams& p, int head_dim, bool bf16, cudaStream_t stream) {
  const dim3 g(p.h_q, p.tab.batch), b(kDecodeThreads);
  if (head_dim == 128)
    return bf16 ? launch_pdl(decode_kernel<128, true>, g, b, 0, stream, p)
                : launch_pdl(decode_kernel<128, false>, g, b, 0, stream, p);
  return bf16 ? launch_pdl(decode_kernel<64, true>, g, b, 0, stream, p)
              : launch_pdl(decode_kernel<64, false>, g, b, 0, stream, p);
}

}  // namespace ta
