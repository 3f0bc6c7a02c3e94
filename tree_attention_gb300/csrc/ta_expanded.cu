// ta_expanded.cu -- causal attention in the expanded form of latent attention:
// keys and values per head, and a rotary key that the heads share.
//
//   s = log2(e) sm_scale (q[:d] . k + q[d:] . k_rope),  out = sum 2^(s - lse) v,
//   lse = log2 sum 2^s,  over the kv rows up to the q row's own
//
// 2 (2 d + rope_dim) operations per pair of q row and kv row: bound by the tensor
// cores for prompts of some hundred rows, by the memory below.
//
// * A unit of work is 256 q rows of one sequence and head, two tiles of 128 (A and
//   B) that read the same kv tiles of 128 rows; where a sequence's last rows are 128
//   at most, they are A of one head and B of the next, which read kv tiles of their
//   own in turn.  A CTA per SM takes every gridDim.x-th unit, the last rows of a
//   sequence (the most kv tiles) first.
// * The products alternate: PV_A(t-1) QK_A(t) PV_B(t-1) QK_B(t), so that one
//   tile's softmax runs beside the other tile's products.  P lies over its own S in
//   tensor memory, and products of one thread execute in order.
// * Keys (three chunks of 64 elements, the last the rotary one) and values (two
//   halves of 64 rows) pass through one ring of eight 16 KB slots, so that a tile's
//   values arrive where the tile before had its keys.
// * One softmax thread per q row.
// * Masked value rows meet weights of zero in the products.  Where that, or an
//   infinity, left a result that is not finite, the CTA goes over its units a second
//   time, carefully: values that are not finite are zeroed before the products, and
//   the softmax threads add what the rows that see them get.
//
// Measured: prompts of 16 to 512 tokens, 64 sequences, 64 heads of 128 + 64, bf16:
// 175 to 200 us by the GPU (floor 109, the memory), up to 235 right behind a load at the
// power limit; 2,000 tokens each of two prompts with 8,195 and 13,045 held, 32 heads,
// fp16: 776 to 822 us, 1,227 to 1,158 TFLOP/s (floor 489, the tensor cores).  The latter
// are 512 units of 67 to 118 kv tiles, of which the busiest of 152 SMs has 375 and the
// average one 311, and a kv tile, for both tiles of q rows, takes 3,960 cycles of the
// 2,600 that its products need: the period is one tile's softmax (some 1,850), its
// products (1,300) and the hand-overs one after the other, beside which the other
// tile's run.  Two threads per q row, which halve the softmax but have to agree on the
// maximum and get 96 registers, took 854 instead of 783 us (prompts 336 instead of 174);
// the last round's units as single tiles on two SMs each 843 instead of 815 (a tile
// alone takes as long as two).
//
// Weights are rounded to the data's type for the product (the error against 64 bits is
// 1.2 to 1.41 times that of float32 weights, as each output is rounded as well); the
// result is divided by their unrounded sum, since that of the rounded ones was measured
// to change the error by 1 % at most and the time by 2 % (prompts 10 %).
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "ta_device.cuh"
#include "ta_launch.h"

namespace ta {
namespace {

constexpr int kThreads = 384;
constexpr int kTile = 128;
constexpr int kSlots = 8;
constexpr int kSlotBytes = 16384;
constexpr int kItems = 4;            // records ahead

struct Item {
  int b, head, q0, nq;     // q rows q0 .. q0 + nq - 1 of the batch
  int first;               // the kv row of the sequence that q0 is
  int kv0, kv;             // the sequence's rows
  int na, nb;              // kv tiles of tiles A and B; na 0: no more items
  int heads;               // 1: B is the next 128 rows, 2: B is the same rows of head + 1
  // kv tiles loaded, and the place of the s-th of them in its sequence
  __device__ __forceinline__ int loads() const { return heads == 2 ? 2 * na : max(na, nb); }
  __device__ __forceinline__ int tile(int s) const { return heads == 2 ? s >> 1 : s; }
  __device__ __forceinline__ bool is_short(int s) const { return kv < (tile(s) + 1) * kTile; }
  // rows of the s-th, and of Q tile w
  __device__ __forceinline__ int rows(int s) const { return min(kTile, kv - tile(s) * kTile); }
  __device__ __forceinline__ int q_rows(int w) const { return min(kTile, nq - w * (2 - heads) * kTile); }
};

// How far a warp has come: what it counts of records, kv tiles loaded, and uses of
// barriers, kept from the first pass over the units for the second (the cleaner's
// are what others count from while it runs).
struct Counts {
  uint32_t n, it, use[4][2];
};

struct Misc {
  uint64_t q_full[2], q_empty[2], k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t v_short[2], v_clean[2];   // a sequence's last tile, which is cleaned before use
  uint64_t s_full[2], p_full[2], o_full[2], o_free[2], item_full[kItems], item_empty[kItems];
  uint64_t stall, drain;
  Item item[kItems];
  uint32_t odd_rows[2][4];           // of a kv tile: rows with values that are not finite
  Counts counts[kThreads / 32];
  uint32_t tmem, loads;              // loads: kv tiles that were asked for
  int abort;
};

template <int D>
struct Cfg {
  static constexpr int kC = D / 64;                 // chunks of a head's part
  static constexpr int kQTile = (kC + 1) * kSlotBytes;
  static constexpr int kOffQ = 0, kOffRing = 2 * kQTile;
  static constexpr int kOffMisc = kOffRing + kSlots * kSlotBytes;
  static constexpr int kPerTile = kC + 1 + 2;       // slots a kv tile takes: K, rotary K, V, V
  static constexpr int kTmemS = 0, kTmemO = 256;    // of tile A; B 128 columns on
};

struct Ctx {
  uint8_t* smem;
  Misc* m;
  unsigned int* error;
  uint64_t limit_ns;
  __device__ __forceinline__ bool expired(uint64_t& t0, uint32_t& loads) const {
    if (*(volatile int*)&m->abort) return true;
    const uint32_t now = *(volatile uint32_t*)&m->loads;
    if (now != loads) {
      loads = now;
      t0 = globaltimer_ns();
    }
    if (globaltimer_ns() - t0 <= limit_ns) return false;
    atomicOr(error, DEVERR_TIMEOUT);
    *(volatile int*)&m->abort = 1;
    return true;
  }
  // by a whole warp, with one answer for all lanes; at most limit_ns in which no
  // further kv tile is asked for (a unit may take as long as it takes), or until another
  // warp gave up
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return wait_long(bar, parity);
  }
  __device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity) const {
    uint64_t t0 = globaltimer_ns();
    uint32_t loads = *(volatile uint32_t*)&m->loads;
    for (uint32_t spins = 1;; ++spins) {
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
      if ((spins & 63u) == 0 && __any_sync(0xffffffffu, expired(t0, loads))) return false;
    }
  }
};

__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

__device__ __forceinline__ bool good_sequence(const ExpandedParams& p, int b) {
  const int q0 = p.q_indptr[b], q1 = p.q_indptr[b + 1], k0 = p.kv_indptr[b], k1 = p.kv_indptr[b + 1];
  return q0 >= 0 && k0 >= 0 && q1 >= q0 && k1 >= k0 && q1 - q0 <= k1 - k0 &&
         (b > 0 || (q0 == 0 && k0 == 0)) &&
         (b < p.batch - 1 || (q1 == p.total_q && k1 == p.total_kv));
}

// ---------------------------------------------------------------------------
// roles
// ---------------------------------------------------------------------------

// Units of the last 256 q rows of a sequence with qo > 0 of them.
__device__ __forceinline__ int last_units(int qo, int h) {
  const int rows = (qo - 1) % (2 * kTile) + 1;
  return rows <= kTile ? (h + 1) / 2 : h;
}

// Every gridDim.x-th unit, counted sequence by sequence, in one from the last 256
// rows on, head by head; 32 sequences at a time.
__device__ void run_scheduler(const Ctx& cx, const ExpandedParams& p, int lane) {
  Misc& m = *cx.m;
  long long u = blockIdx.x, base = 0;
  int b0 = -32, q0 = 0, qo = 0, k0 = 0, kv = 0;
  long long before = 0, units = 0, total = 0;
  for (uint32_t n = m.counts[11].n;; ++n) {
    while (u >= base + total && b0 + 32 < p.batch) {
      base += total;
      b0 += 32;
      const int b = b0 + lane;
      units = 0;
      if (b < p.batch) {
        q0 = p.q_indptr[b];
        qo = p.q_indptr[b + 1] - q0;
        k0 = p.kv_indptr[b];
        kv = p.kv_indptr[b + 1] - k0;
        const int pairs = (qo + 2 * kTile - 1) / (2 * kTile);
        if (pairs) units = (long long)(pairs - 1) * p.h + last_units(qo, p.h);
      }
      long long up = units;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, up, d);
        if (lane >= d) up += y;
      }
      before = up - units;
      total = __shfl_sync(0xffffffffu, up, 31);
    }
    Item x{};
    if (u < base + total) {
      const long long in = u - base - before;
      const int src = __ffs(__ballot_sync(0xffffffffu, in >= 0 && in < units)) - 1;
      if (lane == src) {
        const int pairs = (qo + 2 * kTile - 1) / (2 * kTile), last = last_units(qo, p.h);
        const int r0 = (in < last ? pairs - 1 : pairs - 2 - (int)((in - last) / p.h)) * 2 * kTile;
        x.heads = in < last && last < p.h ? 2 : 1;
        x.b = b0 + lane;
        x.head = in < last ? (int)in * x.heads : (int)((in - last) % p.h);
        x.q0 = q0 + r0;
        x.nq = min(2 * kTile, qo - r0);
        x.first = kv - qo + r0;
        x.kv0 = k0;
        x.kv = kv;
        x.na = (x.first + min(kTile, x.nq) + kTile - 1) / kTile;
        x.nb = x.nq > kTile ? (x.first + x.nq + kTile - 1) / kTile : 0;
        if (x.heads == 2) {
          if (x.head + 1 < p.h)
            x.nb = x.na;
          else
            x.heads = 1;
        }
      }
      const int slot = n % kItems;
      if (!cx.wait(&m.item_empty[slot], ((n / kItems) & 1) ^ 1)) return;
      if (lane == src) {
        m.item[slot] = x;
        mbar_arrive(&m.item_full[slot]);
      }
      __syncwarp();
      u += gridDim.x;
    } else {
      const int slot = n % kItems;
      if (!cx.wait(&m.item_empty[slot], ((n / kItems) & 1) ^ 1)) return;
      if (lane == 0) {
        m.item[slot] = x;
        mbar_arrive(&m.item_full[slot]);
        m.counts[11].n = n + 1;
      }
      return;
    }
  }
}

// The next record, for a whole warp.
__device__ __forceinline__ bool next_item(const Ctx& cx, uint32_t n, int lane, Item& x) {
  const int slot = n % kItems;
  if (!cx.wait(&cx.m->item_full[slot], (n / kItems) & 1)) return false;
  x = cx.m->item[slot];
  __syncwarp();
  if (lane == 0) mbar_arrive(&cx.m->item_empty[slot]);
  return x.na > 0;
}

template <int D, bool CAREFUL>
__device__ __forceinline__ void run_producer(const Ctx& cx, const ExpandedMaps& maps, int lane) {
  using C = Cfg<D>;
  Misc& m = *cx.m;
  Counts& kept = m.counts[8];
  uint32_t n = kept.n, it = kept.it, chunk = kept.use[0][0], units[2] = {kept.use[1][0], kept.use[1][1]};
  Item x;
  for (; next_item(cx, n, lane, x); ++n) {
    auto load_q = [&](int tile) {
      if (!cx.wait(&m.q_empty[tile], (units[tile] & 1) ^ 1)) return false;
      ++units[tile];
      if (elect_one()) {
        // 64 rows at a time, those that there are
        const int boxes = x.q_rows(tile) > 64 ? 2 : 1;
        mbar_arrive_expect_tx(&m.q_full[tile], boxes * C::kQTile / 2);
        for (int c = 0; c <= C::kC; ++c)
          for (int i = 0; i < boxes; ++i)
            tma_load_3d(cx.smem + C::kOffQ + tile * C::kQTile + c * kSlotBytes + i * 8192, &maps.q,
                        &m.q_full[tile], 64 * c, x.head + tile * (x.heads - 1),
                        x.q0 + tile * (2 - x.heads) * kTile + 64 * i);
      }
      __syncwarp();
      return true;
    };
    // the ring slot of this producer's next chunk, once what it held is used up
    auto slot = [&]() -> uint8_t* {
      if (chunk >= kSlots) {
        const uint32_t old = chunk - kSlots, t = old / C::kPerTile;
        uint64_t* bar = old % C::kPerTile <= C::kC ? &m.k_empty[t & 1] : &m.v_empty[t & 1];
        if (!cx.wait(bar, (t >> 1) & 1)) return nullptr;
      }
      return cx.smem + C::kOffRing + (chunk++ % kSlots) * kSlotBytes;
    };
    if (!load_q(0)) return;
    const int loads = x.loads();
    for (int t = 0; t < loads; ++t, ++it) {
      if (lane == 0) *(volatile uint32_t*)&m.loads = it + 1;
      const int row = x.kv0 + x.tile(t) * kTile, s = it & 1, head = x.head + (t & (x.heads - 1));
      uint64_t* v_bar = CAREFUL || x.is_short(t) ? &m.v_short[s] : &m.v_full[s];
      const int boxes = x.rows(t) > 64 ? 2 : 1;
      for (int c = 0; c <= C::kC; ++c) {
        uint8_t* to = slot();
        if (!to) return;
        if (elect_one()) {
          if (c == 0) mbar_arrive_expect_tx(&m.k_full[s], boxes * C::kQTile / 2);
          for (int i = 0; i < boxes; ++i)
            if (c < C::kC)
              tma_load_3d(to + i * 8192, &maps.k, &m.k_full[s], 64 * c, head, row + 64 * i);
            else
              tma_load_3d(to + i * 8192, &maps.rot, &m.k_full[s], 0, row + 64 * i, 0);
        }
        __syncwarp();
      }
      if (t == 0 && x.nb > 0 && !load_q(1)) return;
      for (int half = 0; half < 2; ++half) {
        uint8_t* to = slot();
        if (!to) return;
        if (elect_one()) {
          if (half == 0) mbar_arrive_expect_tx(v_bar, boxes * kTile * D);
          for (int c = 0; c < C::kC && half < boxes; ++c)
            tma_load_3d(to + c * 8192, &maps.v, v_bar, 64 * c, head, row + 64 * half);
        }
        __syncwarp();
      }
    }
  }
  if (!CAREFUL && lane == 0) kept = Counts{n + 1, it, {{chunk, 0}, {units[0], units[1]}}};
}

// sum + 0 times eight elements: NaN where one is infinite or NaN.
template <bool BF16>
__device__ __forceinline__ void add_zero_times(uint32_t& sum, const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if constexpr (BF16)
      asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(w[i]), "r"(0u));
    else
      asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(w[i]), "r"(0u));
}
__device__ __forceinline__ bool has_nan(uint32_t sum) { return (sum & 0x7fff7fffu) != 0; }

// Zeroes the value rows behind a sequence's last, up to the 16 of a product: what
// does not count must not reach the products as NaN.  CAREFUL: of every tile also the
// values that are not finite, whose rows it notes.
template <int D, bool BF16, bool CAREFUL>
__device__ __forceinline__ void run_cleaner(const Ctx& cx, int lane) {
  using C = Cfg<D>;
  constexpr uint32_t kEnd = BF16 ? 0x7f80u : 0x7c00u;   // the exponent of what is not finite
  constexpr int kVecs = C::kC * 8;                      // of a row
  Misc& m = *cx.m;
  Counts& kept = m.counts[10];
  uint32_t n = kept.n, it = kept.it, count[2] = {kept.use[0][0], kept.use[0][1]};
  Item x;
  for (; next_item(cx, n, lane, x); ++n) {
    const int loads = x.loads();
    const bool ends = x.is_short(loads - 1);
    const uint32_t it0 = it;
    it += loads;
    if (!ends && !CAREFUL) continue;
    for (uint32_t t = CAREFUL ? it0 : it - x.heads; t < it; ++t) {
      if (!cx.wait(&m.v_short[t & 1], count[t & 1]++ & 1)) return;
      auto half = [&](int h) {   // rows 64 h on
        const uint32_t chunk = t * C::kPerTile + C::kC + 1 + h;
        return cx.smem + C::kOffRing + chunk % kSlots * kSlotBytes;
      };
      const int valid = x.rows(t - it0);
      if (CAREFUL) {
        // of 32 rows, kVecs vectors per lane; a look at all of them, and at each where
        // one is not finite
        const int mine = lane / kVecs * 128 + lane / 8 % C::kC * 8192 + (lane & 7) * 16;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t rows = 0;
          if (32 * g < valid) {
            uint8_t* at = half(g >> 1) + (g & 1) * 32 * 128 + mine;
            auto vec = [&](int k) { return reinterpret_cast<uint4*>(at + k * (32 / kVecs) * 128); };
            uint4 u[kVecs];
            uint32_t sum[4] = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < kVecs; ++k) u[k] = *vec(k);
#pragma unroll
            for (int k = 0; k < kVecs; ++k) add_zero_times<BF16>(sum[k & 3], u[k]);
            if (has_nan(sum[0]) || has_nan(sum[1]) || has_nan(sum[2]) || has_nan(sum[3])) {
              auto cleared = [](uint32_t w) {
                if ((w & kEnd) == kEnd) w &= 0xffff0000u;
                if ((w >> 16 & kEnd) == kEnd) w &= 0xffffu;
                return w;
              };
#pragma unroll 1
              for (int k = 0; k < kVecs; ++k) {
                const uint4 v = *vec(k);
                uint32_t odd = 0;
                add_zero_times<BF16>(odd, v);
                if (has_nan(odd)) {
                  *vec(k) = make_uint4(cleared(v.x), cleared(v.y), cleared(v.z), cleared(v.w));
                  rows |= 1u << (k * (32 / kVecs) + lane / kVecs);
                }
              }
            }
            rows = __reduce_or_sync(0xffffffffu, rows);
            if (valid < 32 * (g + 1)) rows &= (1u << (valid - 32 * g)) - 1;
          }
          if (lane == 0) m.odd_rows[t & 1][g] = rows;
        }
      }
      for (int i = lane; i < (-valid & 15) * kVecs; i += 32) {
        const int row = valid + i / kVecs;
        *reinterpret_cast<uint4*>(half(row >> 6) + i / 8 % C::kC * 8192 + row % 64 * 128 + (i & 7) * 16) =
            make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&m.v_clean[t & 1]);
    }
  }
  if (!CAREFUL && lane == 0) kept = Counts{n + 1, it, {{count[0], count[1]}}};
}

template <int D, bool BF16, bool CAREFUL>
__device__ __forceinline__ void run_mma(const Ctx& cx, const ExpandedParams& p, uint32_t tmem, int lane) {
  using C = Cfg<D>;
  Misc& m = *cx.m;
  constexpr uint32_t idesc_qk = umma_idesc_f16(BF16, kTile, kTile, false);
  constexpr uint32_t idesc_pv = umma_idesc_f16(BF16, kTile, D, true);
  const uint64_t dq = sw128_desc(smem_u32(cx.smem + C::kOffQ), 0);
  const uint64_t dring = sw128_desc(smem_u32(cx.smem + C::kOffRing), 0);
  const uint64_t dv = sw128_desc(smem_u32(cx.smem + C::kOffRing), 8192);
  const int rot_steps = p.rope_dim / 16;
  Counts& kept = m.counts[9];
  uint32_t n = kept.n, it = kept.it, units[2] = {kept.use[0][0], kept.use[0][1]};
  uint32_t pv[2] = {kept.use[1][0], kept.use[1][1]};
  // of v_clean, v_full
  uint32_t cleaned[2] = {kept.use[2][0], kept.use[2][1]}, full[2] = {kept.use[3][0], kept.use[3][1]};
  uint32_t k_seen = ~0u, v_seen = ~0u;              // the load last waited for
  bool ok = true, issued = false;
  if (p.debug_stall) ok = cx.wait(&m.stall, 0);
  Item x;
  using A = std::integral_constant<int, 0>;
  using B = std::integral_constant<int, 1>;
  // S of tile w and load s, of its kv tiles the first or the last (done: no tile uses
  // the load after this one); both in line, with w known, as descriptors that are not
  // the warp's constants cost 40 cycles a product
  auto qk = [&](auto wc, int s, bool first, bool last, bool done) __attribute__((always_inline)) -> bool {
    constexpr int w = decltype(wc)::value;
    const uint32_t g = it + s;
    if (first && !cx.wait(&m.q_full[w], units[w] & 1)) return false;
    if (k_seen != g) {
      if (!cx.wait(&m.k_full[g & 1], (g >> 1) & 1)) return false;
      k_seen = g;
    }
    tc_fence_after();
    issued = true;
    uint64_t k[C::kC + 1];
#pragma unroll
    for (int c = 0; c <= C::kC; ++c) k[c] = dring + (((g * C::kPerTile + c) % kSlots * kSlotBytes) >> 4);
    if (elect_one()) {
#pragma unroll
      for (int c = 0; c < C::kC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          umma_f16(tmem + C::kTmemS + 128 * w, dq + ((w * C::kQTile + c * kSlotBytes + 32 * i) >> 4),
                   k[c] + 2 * i, idesc_qk, c + i > 0 ? 1u : 0u);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < rot_steps)
          umma_f16(tmem + C::kTmemS + 128 * w, dq + ((w * C::kQTile + C::kC * kSlotBytes + 32 * i) >> 4),
                   k[C::kC] + 2 * i, idesc_qk, 1u);
      umma_commit(&m.s_full[w]);
      if (last) umma_commit(&m.q_empty[w]);
      if (done) umma_commit(&m.k_empty[g & 1]);
    }
    __syncwarp();
    return true;
  };
  auto do_pv = [&](auto wc, int s, bool first, bool last, bool done) __attribute__((always_inline)) -> bool {
    constexpr int w = decltype(wc)::value;
    const uint32_t g = it + s;
    if (!cx.wait(&m.p_full[w], pv[w] & 1)) return false;
    ++pv[w];
    if (v_seen != g) {
      // the sequence's last, short tile is cleaned first
      const bool clean = CAREFUL || x.is_short(s);
      const uint32_t uses = clean ? cleaned[g & 1]++ : full[g & 1]++;
      if (!cx.wait(clean ? &m.v_clean[g & 1] : &m.v_full[g & 1], uses & 1)) return false;
      v_seen = g;
    }
    if (first) {
      if (!cx.wait(&m.o_free[w], (units[w] & 1) ^ 1)) return false;
      ++units[w];
    }
    tc_fence_after();
    uint64_t v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      v[i] = dv + (((g * C::kPerTile + C::kC + 1 + i) % kSlots * kSlotBytes) >> 4);
    const int steps = (x.rows(s) + 15) / 16;
    const uint32_t begin = first && !CAREFUL ? 0u : 1u;   // CAREFUL: the softmax cleared O
    if (elect_one()) {
#pragma unroll
      for (int i = 0; i < kTile / 16; ++i)
        if (i < steps) umma_f16_tmem_a(tmem + C::kTmemO + 128 * w, tmem + C::kTmemS + 128 * w + 8 * i,
                        v[i >> 2] + ((i & 3) * 2048 >> 4), idesc_pv, i > 0 ? 1u : begin);
      if (last) umma_commit(&m.o_full[w]);
      if (done) umma_commit(&m.v_empty[g & 1]);
    }
    __syncwarp();
    return true;
  };
  for (; ok && next_item(cx, n, lane, x); ++n) {
    const int loads = x.loads(), step = x.heads, na = x.na, nb = x.nb;
    // kv tile t is load t of both tiles, or load 2 t of A and 2 t + 1 of B
    for (int t = 0; ok; ++t) {
      const int sa = t * step, sb = sa + step - 1;
      if (t > 0 && t - 1 < na) {
        if (!(ok = do_pv(A{}, sa - step, t == 1, t == na, step == 2 || t - 1 >= nb))) break;
      }
      if (t < na) {
        if (!(ok = qk(A{}, sa, t == 0, t == na - 1, step == 2 || t >= nb))) break;
      }
      if (t > 0 && t - 1 < nb) {
        if (!(ok = do_pv(B{}, sb - step, t == 1, t == nb, true))) break;
      }
      if (t < nb) {
        if (!(ok = qk(B{}, sb, t == 0, t == nb - 1, true))) break;
      }
      if (t >= na && t >= nb) break;
    }
    it += loads;
  }
  if (*(volatile int*)&m.abort && issued) {
    if (elect_one()) umma_commit(&m.drain);
    __syncwarp();
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(&m.drain, 0) && globaltimer_ns() - t0 < 10000000ull) {}
  }
  if (!CAREFUL && lane == 0)
    kept = Counts{n + 1, it, {{units[0], units[1]}, {pv[0], pv[1]}, {cleaned[0], cleaned[1]}, {full[0], full[1]}}};
}

// The exponent that a weight may reach over its reference, and where a moved
// reference puts the largest.  fp16 weights are held high, as what lies 2^-24 below
// a weight of one is the type's end; bf16 ones are at most one, as values may be
// near the end of float32's range.
template <bool BF16>
struct Ref {
  static constexpr float kTop = BF16 ? 0.f : 15.f, kPut = BF16 ? -8.f : 7.f;
};

template <int D>
__device__ __noinline__ void rescale(uint32_t o, float f) {
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float v[32];
    tmem_ld32(o + c, v);
    tmem_wait_ld(v);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= f;
    tmem_st32(o + c, v);
  }
  tmem_wait_st();
}

// What this warp's q rows get of a kv tile's values that are not finite, which the
// products have as zeros: O += w v, of the rows of the tile that are set in ``rows``
// and that a q row sees (up to ``lim``).  O is at rest.  ``dead``: of which 32 columns
// of O all is NaN and stays so; returned as it is then.  kv_row: the tile's first.
template <int D, bool BF16>
__device__ __noinline__ uint32_t add_odd_values(const ExpandedParams& p, const uint32_t* rows,
                                                int64_t kv_row, int head, uint32_t s_at,
                                                uint32_t o_at, int lim, float ref, uint32_t dead) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int g = 0; g < 4; ++g) {
    uint32_t left = rows[g];
#pragma unroll 1
    while (left && dead != (1u << (D / 32)) - 1) {
      const int j = 32 * g + __ffs(left) - 1;
      left &= left - 1;
      const float s = tmem_ld1(s_at + j) * p.scale_log2;
      const float w = ex2_approx(s - ref);
      const bool counts = j <= lim && s != -INFINITY;
      if (!__any_sync(0xffffffffu, counts)) continue;
      const uint16_t* v = p.v + (kv_row + j) * p.v_ts + head * p.v_hs;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        if (dead >> c & 1) continue;
        const float x = unpack2<BF16>(v[32 * c + lane]).x;
        const uint32_t odd = __ballot_sync(0xffffffffu, !(fabsf(x) < INFINITY));
        if (!odd) continue;
        float o[32];
        tmem_ld32(o_at + 32 * c, o);
        tmem_wait_ld(o);
        bool all = true;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float y = __shfl_sync(0xffffffffu, x, i);
          if (counts && (odd >> i & 1)) o[i] = fmaf(w, y, o[i]);
          all = all && o[i] != o[i];
        }
        tmem_st32(o_at + 32 * c, o);
        tmem_wait_st();
        if (__all_sync(0xffffffffu, all)) dead |= 1u << c;
      }
    }
  }
  return dead;
}

// Returns whether a result of this thread's may have to be computed carefully.
template <int D, bool BF16, bool CAREFUL>
__device__ __forceinline__ bool run_softmax(const Ctx& cx, const ExpandedParams& p, uint32_t tmem, int warp,
                                            int lane) {
  using C = Cfg<D>;
  Misc& m = *cx.m;
  Counts& kept = m.counts[warp];
  const int w = warp >> 2;                       // tile A or B
  const int rr = (warp & 3) * 32 + lane;         // the tile's row
  const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t s_at = tmem + lanes + C::kTmemS + 128 * w, o_at = tmem + lanes + C::kTmemO + 128 * w;
  uint32_t n = kept.n, it = kept.it, done = kept.use[0][0], units = kept.use[0][1];
  bool odd_result = false;
  Item x;
  for (; next_item(cx, n, lane, x); ++n) {
    const int tiles = w ? x.nb : x.na;
    const uint32_t it0 = it;
    it += x.loads();
    if (tiles == 0) continue;
    const int row = w * (2 - x.heads) * kTile + rr;          // of the unit's
    const int head = x.head + w * (x.heads - 1);
    const int see = x.first + row;               // the last kv row it sees
    const int low = see - lane;                  // the warp's first row's
    const bool work = row - lane < x.nq;
    float ref = -FLT_MAX, l = 0.f;
    uint32_t dead = 0;
    for (int t = 0; t < tiles; ++t, ++done) {
      if (!cx.wait(&m.s_full[w], done & 1)) return false;
      if (!work) {                               // no row of the warp is the sequence's
        if (lane == 0) mbar_arrive(&m.p_full[w]);
        continue;
      }
      tc_fence_after();
      // The scores are read twice, 32 at a time, for their maximum and for the
      // weights (128 registers for all of them do not go with the rest).
      float s[2][32];
      const int lim = see - t * kTile, lim0 = low - t * kTile;
      float2 sum = make_float2(0.f, 0.f);
      bool ok = true;
      // CAREFUL: of the tile's values, load g, those that are not finite
      auto add_odd = [&]() {
        const uint32_t g = it0 + t * x.heads + w * (x.heads - 1);
        // the cleaner's counts at the start of this pass, in which it cleans every load
        const Counts& then = m.counts[10];
        const uint32_t uses = then.use[0][g & 1] + ((g - then.it) >> 1);
        if (!(ok = cx.wait(&m.v_clean[g & 1], uses & 1))) return;
        if (t == 0) {
          const float zero[32] = {};
          for (int c = 0; c < D; c += 32) tmem_st32(o_at + c, zero);
          tmem_wait_st();
        }
        dead = add_odd_values<D, BF16>(p, m.odd_rows[g & 1], (int64_t)x.kv0 + t * kTile, head, s_at, o_at,
                                       see - t * kTile, ref, dead);
      };
      // Moves the reference where it has to be.  (Products that no compiler joins with an
      // addition: a careful pass gives the bits of the first.)
      auto refer = [&](float most) {
        const bool move = most - ref > Ref<BF16>::kTop;
        if (!__any_sync(0xffffffffu, move)) return;
        float f = 1.f;
        if (move) {
          const float to = most - Ref<BF16>::kPut;
          f = ex2_approx(ref - to);
          ref = to;
          l = __fmul_rn(l, f);
        }
        // the product before has been waited for with these scores: O is at rest
        if (t > 0) rescale<D>(o_at, f);
      };
      float top[2] = {-INFINITY, -INFINITY};
      tmem_ld32(s_at, s[0]);
      if (lim0 >= kTile - 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_wait_ld(s[c & 1]);
          if (c < 3) tmem_ld32(s_at + 32 * (c + 1), s[(c + 1) & 1]);
          // of the scores before their scale, whose sign is known
          if (p.scale_log2 >= 0.f) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              top[0] = fmaxf(top[0], fmaxf(s[c & 1][j], s[c & 1][j + 1]));
              top[1] = fmaxf(top[1], fmaxf(s[c & 1][j + 2], s[c & 1][j + 3]));
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) top[j & 1] = fmaxf(top[j & 1], -s[c & 1][j]);
          }
        }
        refer(__fmul_rn(fmaxf(top[0], top[1]), fabsf(p.scale_log2)));
        if (CAREFUL) {
          add_odd();
          if (!ok) return false;
        }
        tmem_ld32(s_at, s[0]);
        const float2 scale = make_float2(p.scale_log2, p.scale_log2), shift = make_float2(-ref, -ref);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_wait_ld(s[c & 1]);
          if (c < 3) tmem_ld32(s_at + 32 * (c + 1), s[(c + 1) & 1]);
          uint32_t w16[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float2 e = ffma2(make_float2(s[c & 1][2 * j], s[c & 1][2 * j + 1]), scale, shift);
            e = make_float2(ex2_approx(e.x), ex2_approx(e.y));
            sum = fadd2(sum, e);
            w16[j] = pack2<BF16>(e.x, e.y);
          }
          // over scores that have been read: columns 16 c on are of chunk c / 2
          tmem_st16(s_at + 16 * c, w16);
        }
      } else {
        // The diagonal: chunks that none of the warp's rows sees are left out.
        const int last = min(3, (lim0 + 31) / 32);
#pragma unroll 1
        for (int c = 0; c <= last; ++c) {
          tmem_wait_ld(s[0]);
          if (32 * c + 31 > lim0) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              top[j & 1] = fmaxf(top[j & 1], 32 * c + j <= lim ? s[0][j] * p.scale_log2 : -INFINITY);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) top[j & 1] = fmaxf(top[j & 1], s[0][j] * p.scale_log2);
          }
          tmem_ld32(s_at + (c < last ? 32 * (c + 1) : 0), s[0]);
        }
        tmem_wait_ld(s[0]);
        refer(fmaxf(top[0], top[1]));
        if (CAREFUL) {
          add_odd();
          if (!ok) return false;
        }
        const float2 scale = make_float2(p.scale_log2, p.scale_log2), shift = make_float2(-ref, -ref);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t w16[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) w16[j] = 0;
          if (c <= last) {
            tmem_ld32(s_at + 32 * c, s[0]);
            tmem_wait_ld(s[0]);
            const int left = lim - 32 * c;       // the last column that counts, if below 31
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float2 e = ffma2(make_float2(s[0][2 * j], s[0][2 * j + 1]), scale, shift);
              e = make_float2(2 * j <= left ? ex2_approx(e.x) : 0.f, 2 * j < left ? ex2_approx(e.y) : 0.f);
              sum = fadd2(sum, e);
              w16[j] = pack2<BF16>(e.x, e.y);
            }
          }
          tmem_st16(s_at + 16 * c, w16);
        }
      }
      l += sum.x + sum.y;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&m.p_full[w]);
    }
    if (!cx.wait(&m.o_full[w], units & 1)) return false;
    ++units;
    if (!work) {
      if (lane == 0) mbar_arrive(&m.o_free[w]);
      continue;
    }
    tc_fence_after();
    const bool valid = row < x.nq;
    const int64_t at = (int64_t)(x.q0 + row) * p.h + head;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int four = lane & ~3;                  // the rows whose vectors this lane stores
    const int64_t step = (int64_t)p.h * D;       // from row to row
    uint16_t* out = p.out + (at + (four - lane) * (int64_t)p.h) * D + (lane & 3) * 8;
    const float2 zero = make_float2(0.f, 0.f), by = make_float2(inv, inv);
    float2 odd2 = zero;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float v[32];
      tmem_ld32(o_at + c, v);
      tmem_wait_ld(v);
      uint4 z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 o = make_float2(v[8 * i + 2 * k], v[8 * i + 2 * k + 1]);
          odd2 = ffma2(o, zero, odd2);
          const float2 r = ffma2(o, by, zero);
          y[k] = pack2<BF16>(r.x, r.y);
        }
        z[i] = make_uint4(y[0], y[1], y[2], y[3]);
      }
      transpose4(z, lane);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (row - lane + four + j < x.nq) *reinterpret_cast<uint4*>(out + j * step + c) = z[j];
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&m.o_free[w]);
    const float odd = odd2.x + odd2.y;
    if (valid) p.lse[at] = l == 0.f ? -INFINITY : ref + log2f(l);
    // a value that is not finite, though the weights are: it may be one not seen
    odd_result |= valid && odd != 0.f && l < INFINITY;
  }
  if (!CAREFUL && lane == 0) kept = Counts{n + 1, it, {{done, units}}};
  return odd_result;
}

// This CTA's units, once.  Returns whether a result of this thread's may have to be
// computed carefully.
template <int D, bool BF16, bool CAREFUL>
__device__ __forceinline__ bool run_pass(const Ctx& cx, const ExpandedMaps& maps, const ExpandedParams& p,
                                         int warp, int lane) {
  const uint32_t tmem = cx.m->tmem;
  if (warp < 8) return run_softmax<D, BF16, CAREFUL>(cx, p, tmem, warp, lane);
  if (warp == 8)
    run_producer<D, CAREFUL>(cx, maps, lane);
  else if (warp == 9)
    run_mma<D, BF16, CAREFUL>(cx, p, tmem, lane);
  else if (warp == 10)
    run_cleaner<D, BF16, CAREFUL>(cx, lane);
  else
    run_scheduler(cx, p, lane);
  return false;
}
template <int D, bool BF16>
__device__ __noinline__ void run_carefully(const Ctx& cx, const ExpandedMaps& maps, const ExpandedParams& p,
                                           int warp, int lane) {
  run_pass<D, BF16, true>(cx, maps, p, warp, lane);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    expanded_kernel(const __grid_constant__ ExpandedMaps maps, const ExpandedParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc& m = *reinterpret_cast<Misc*>(smem + C::kOffMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&m.q_full[i], 1);
      mbar_init(&m.q_empty[i], 1);
      mbar_init(&m.k_full[i], 1);
      mbar_init(&m.k_empty[i], 1);
      mbar_init(&m.v_full[i], 1);
      mbar_init(&m.v_empty[i], 1);
      mbar_init(&m.v_short[i], 1);
      mbar_init(&m.v_clean[i], 1);
      mbar_init(&m.s_full[i], 1);
      mbar_init(&m.p_full[i], 4);
      mbar_init(&m.o_full[i], 1);
      mbar_init(&m.o_free[i], 4);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&m.item_full[i], 1);
      mbar_init(&m.item_empty[i], 11);   // 8 softmax warps, producer, products, cleaner
    }
    mbar_init(&m.stall, 1);
    mbar_init(&m.drain, 1);
    for (int i = 0; i < kThreads / 32; ++i) m.counts[i] = Counts{};
    m.abort = 0;
    m.loads = 0;
    mbar_fence_init();
  }
  if (warp == 8) {
    if (lane == 0) {
      tma_prefetch_desc(&maps.q);
      tma_prefetch_desc(&maps.k);
      tma_prefetch_desc(&maps.rot);
      tma_prefetch_desc(&maps.v);
    }
    tmem_alloc(&m.tmem, 512);
  }
  pdl_wait();
  pdl_trigger();
  bool bad = false;
  for (int b = tid; b < p.batch; b += kThreads) bad |= !good_sequence(p, b);
  tc_fence_before();
  const bool stop = __syncthreads_or(bad);
  tc_fence_after();
  const Ctx cx{smem, &m, p.error, p.timeout_ns};
  if (stop) {
    if (tid == 0) atomicOr(p.error, DEVERR_BAD_INDPTR);
  } else {
    const bool odd = run_pass<D, BF16, false>(cx, maps, p, warp, lane);
    __syncwarp();
    tc_fence_before();
    const bool again = __syncthreads_or(odd);
    tc_fence_after();
    if (again && !m.abort) run_carefully<D, BF16>(cx, maps, p, warp, lane);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // after a wait ran out copies may still be on their way into shared memory
  if (m.abort) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(m.tmem, 512);
  }
}

template <int D, bool BF16>
cudaError_t launch(const ExpandedParams& p, const ExpandedMaps& maps, int grid, cudaStream_t stream) {
  constexpr int smem = Cfg<D>::kOffMisc + (int)sizeof(Misc);
  static_assert(smem <= 232448, "shared memory of an SM");
  const auto kern = expanded_kernel<D, BF16>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_shared((const void*)kern, smem, allowed);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(grid), dim3(kThreads), smem, stream, maps, p);
}

}  // namespace

cudaError_t launch_expanded(const ExpandedParams& p, const ExpandedMaps& maps, int head_dim, bool bf16,
                            int nsm, cudaStream_t stream) {
  const int64_t most = (ceil_div(p.total_q, 2 * kTile) + p.batch) * p.h;   // units there can be
  const int grid = (int)(most < nsm ? most : nsm);
  if (head_dim == 128)
    return bf16 ? launch<128, true>(p, maps, grid, stream) : launch<128, false>(p, maps, grid, stream);
  return bf16 ? launch<64, true>(p, maps, grid, stream) : launch<64, false>(p, maps, grid, stream);
}

}  // namespace ta
