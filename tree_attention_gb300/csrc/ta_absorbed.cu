// ta_absorbed.cu -- absorbed latent attention over a paged latent cache, of one
// token per sequence and of draft trees, and the merge of its parts.
//
//   s_j = log2(e) sm_scale q.row_j,  out = sum_j 2^(s_j - lse) c_j,
//   lse = log2 sum_j 2^s_j,  row_j = (c_j | k_j)
//
// All heads of all of a sequence's q rows read the same rows, so q row and head
// are one dimension of h qo packed rows.  A row of W = rank + rope_dim elements
// costs 2 W + 2 rank operations per packed row: with 128 of them 242 operations
// per byte read, near what the memory and the tensor cores do at once.
//
// * A tile is 128 packed rows by 128 kv rows.  Its accumulator, 128 x 512 float32,
//   is all of one SM's tensor memory, so two SMs work on a tile (cta_group::2,
//   M = 128): each holds 64 packed rows of Q and of the accumulator, half of the
//   kv rows for S = Q K^T, and half of the latent's columns, of all kv rows, for
//   O += P V.
// * Each SM's 64 x N accumulators lie in its 128 lanes, columns 0 .. N/2 - 1 in
//   lanes 0-63 and the others in lanes 64-127.
// * The tiles of all (sequence, 128 packed rows) in order are cut into equal
//   ranges, one per pair of SMs; a range's first and last item may be parts,
//   whose float32 states a second kernel merges.
// * What is not finite in a row that does not count never meets its weight of zero:
//   the rows' scores tell (see run_softmax), and such values are zeroed first.
// * Roles: 8 warps of softmax, one that loads Q and K, one that loads V, one that
//   issues the products (of the pair's first CTA), one that walks the tables ahead
//   of all others.
//
// Measured, bf16, rank 512, rotary 64 (the memory copies at 6.69 TB/s, the tensor
// cores reach 1,947 TFLOP/s; the merge included): 4 sequences of 33,000 rows with 128
// heads 49.6 us, floor 23 (memory) and 19 (tensor cores) at once; 64 sequences of 16 to
// 16,384 rows with 64 heads 73.5 to 74.9 us, floor 37; draft trees of 64 nodes with 32
// heads behind 4 x 32,768 rows 411 to 490 us, 1,420 to 1,190 TFLOP/s, by the state of
// the GPU's power limit.  A pair's products for a tile take 2,500 cycles, its rows from
// memory 3,475 when all pairs read; for trees a tile takes 2,500 to 2,900, for decode
// 2,650 with the rows at hand and some 4,700 on average over a long call.  A call of few tiles is its start (4.3 us: tables, the first page's
// look-up), the first loads (3 us), the parts' stores (3 us) and the merge (4 to 8 us).
// Joining the parts in this kernel, pair by pair, took longer for few long sequences
// (decode of one of 4,096 rows 14.5 -> 29.5 us) than the merge as a kernel of its own,
// which all SMs share.
//
// Weights are rounded to the data's type for the product, as the tensor cores take both
// operands in it: the error against 64 bits is 1.05 to 1.25 times that of float32
// weights, as each output is rounded as well.  A second product with what the rounding
// left would want 16 KB of shared memory, of which 3 KB are left, and two fifths of
// the tensor cores' time.
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdint>

#include "ta_latent.cuh"

namespace ta {
namespace {

constexpr int kTile = 128;                 // kv rows, packed rows
constexpr int kChunkBytes = 64 * 128;      // 64 rows of 64 elements
constexpr int kThreads = 384;
constexpr int kPieces = 4;                 // records ahead
constexpr int kAhead = 2;                  // tiles
constexpr int kSlotFloats = kTile * (512 + 3);   // O, reference, sums (see run_softmax)

// ---------------------------------------------------------------------------
// two-CTA forms
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// the address of the same shared variable in the pair's first CTA
__device__ __forceinline__ uint32_t in_first_cta(const void* p) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
  return a;
}
// Arrives on a barrier of the pair's first CTA, releasing this CTA's shared memory to
// the cluster, which is what the arrivals here announce (tensor memory has fences of
// its own).  (A release of all memory waits for all that its thread has under way,
// 1,000 to 4,000 cycles a time: with it a tile took 6,500 cycles.)
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// A box of a map into this CTA's shared memory, counted on a barrier of either CTA
// of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                              int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void tma_load_pair_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                                 int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
// Contiguous memory into L2: both multiples of 16 bytes.
__device__ __forceinline__ void prefetch_l2(const void* at, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(bytes) : "memory");
}
// sw128_desc with any distance between groups of 8 rows
__device__ __forceinline__ uint64_t rows_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (sw128_desc(addr, lbo) & ~((uint64_t)0x3FFF << 32)) | ((uint64_t)(sbo >> 4) << 32);
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}
// Called within ``if (elect_one())``: in code that the compiler knows to be one
// lane's by other means it moves the descriptors from the lane's registers to the
// warp's before every product, 83 cycles a product instead of 40 to 65.
__device__ __forceinline__ void umma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on ``bar`` of both CTAs once all this thread issued is done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// ---------------------------------------------------------------------------
// layout
// ---------------------------------------------------------------------------
// Pages are loaded with one box for several 64-element chunks of their rows, as a
// box costs the SM's copy unit some 50 cycles however small it is.  In K a box is 8
// rows (the others are the other CTA's), so that groups of 8 rows, one per page,
// are equally far apart, as the products want them; V's products take 16 rows, a
// page, at a time, and its boxes hold all of them.
template <int RANK>
struct Cfg {
  static constexpr int kChunks = RANK / 64 + 1;            // of a row: latent, then rotary key
  static constexpr int kHalf = RANK / 128;                 // chunks of half of the latent
  static constexpr int kPages = kTile / kPageSize;
  static constexpr int kKBox = kHalf * 8 * 128;            // {64, 8 rows, kHalf chunks, page}
  static constexpr int kVBox = kHalf * kPageSize * 128;    // {64, 16 rows, kHalf chunks, page}
  static constexpr int kOffQ = 0;                          // [chunk][64 rows][128 B]
  static constexpr int kOffK = kOffQ + kChunks * kChunkBytes;   // [half][page][chunk][8 rows]
  static constexpr int kOffRot = kOffK + 2 * kPages * kKBox;    // [page][8 rows]
  static constexpr int kOffV = kOffRot + kChunkBytes;           // [page][chunk][16 rows]
  static constexpr int kOffP = kOffV + kPages * kVBox;          // [64 kv rows][64 rows][128 B]
  static constexpr int kOffMisc = kOffP + 2 * kChunkBytes;
  static constexpr int kTmemO = 0, kTmemS = RANK / 2;      // S: two buffers of 64 columns
  static constexpr int kCols = RANK / 4;                   // O columns per thread
};

// An item's part that one pair works on: kv tiles t0 .. t1 - 1 of one
// sequence, for packed rows from m_row on (nrows of them exist).
struct Piece {
  int p0, kv, start, m0, node0;      // start: of the tree's rows; node0: the first q row's node
  int row0, m_row, nrows;            // row0: global packed row of m_row
  int t0, t1, slot;                  // t0 == t1: no more; slot -1: the whole item, else 0 or 1
};

struct Misc {
  uint64_t q_full, q_empty, k_full[3], k_empty[3], v_full[2], v_empty[2], v_ready[2];
  uint64_t s_full[2], s_empty[2], p_full, pv_done, o_empty, piece_full[kPieces],
      piece_empty[kPieces], shared_rows[2][2], stall, drain;
  float exchange[2][4][64];
  Piece piece[kPieces];
  long long scan[12];
  LatentSeq first;                   // the range's first sequence, its first tile
  int first_seq, first_unit;
  uint32_t tmem, tiles;              // tiles: whose keys were asked for
  int abort;
};

struct Ctx {
  uint8_t* smem;
  Misc* m;
  unsigned int* error;
  uint64_t limit_ns;
  // Waits for a phase, at most limit_ns in which this CTA asks for no further tile of
  // keys (a piece may take as long as it takes), or until another thread gave up.
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {   // by one thread
    if (try_wait_cluster(bar, parity)) return true;
    return wait_long(bar, parity);
  }
  // by a whole warp, with one answer for all lanes
  __device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) const {
    if (__all_sync(0xffffffffu, try_wait_cluster(bar, parity))) return true;
    return wait_warp_long(bar, parity);
  }
  __device__ __forceinline__ bool expired(uint64_t& t0, uint32_t& tiles) const {
    if (*(volatile int*)&m->abort) return true;
    const uint32_t now = *(volatile uint32_t*)&m->tiles;
    if (now != tiles) {
      tiles = now;
      t0 = globaltimer_ns();
    }
    if (globaltimer_ns() - t0 <= limit_ns) return false;
    atomicOr(error, DEVERR_TIMEOUT);
    *(volatile int*)&m->abort = 1;
    return true;
  }
  __device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity) const {
    uint64_t t0 = globaltimer_ns();
    uint32_t tiles = *(volatile uint32_t*)&m->tiles;
    for (uint32_t spins = 1;; ++spins) {
      if (try_wait_cluster(bar, parity)) return true;
      if ((spins & 63u) == 0 && expired(t0, tiles)) return false;
    }
  }
  __device__ __noinline__ bool wait_warp_long(uint64_t* bar, uint32_t parity) const {
    uint64_t t0 = globaltimer_ns();
    uint32_t tiles = *(volatile uint32_t*)&m->tiles;
    for (uint32_t spins = 1;; ++spins) {
      if (__all_sync(0xffffffffu, try_wait_cluster(bar, parity))) return true;
      if ((spins & 63u) == 0 && __any_sync(0xffffffffu, expired(t0, tiles))) return false;
    }
  }
};

// Pair i's tiles, of fewer than 2^31: from here on.
struct Split {
  int per, extra;
  __device__ int start(int i) const { return i * per + (i < extra ? i : extra); }
  __device__ int pair_of(int u) const {
    const int wide = extra * (per + 1);
    return u < wide ? u / (per + 1) : extra + (u - wide) / per;
  }
};

// Rounded up without passing 2^31: a sequence may have 2^31 - 16 rows.
__device__ __forceinline__ int tiles(int n) { return n / kTile + (n % kTile != 0); }
__device__ __forceinline__ int tiles_of(const LatentSeq& s) { return tiles(s.kv); }
__device__ __forceinline__ int items_of(const LatentSeq& s, int h) { return tiles(s.qo * h); }

// ---------------------------------------------------------------------------
// roles
// ---------------------------------------------------------------------------

// Pieces, for the other roles of this CTA; the first CTA of a pair also leaves
// the record of an item that goes on in the next pair.
__device__ void run_planner(const Ctx& cx, const LatentParams& p, const Split& split, int pair,
                            bool leader) {
  Misc& m = *cx.m;
  int u = split.start(pair);
  const int u_end = split.start(pair + 1);
  int b = m.first_seq, base = m.first_unit;
  LatentMerge merge{};
  uint32_t n = 0;
  LatentSeq s = m.first;
  bool loaded = true;
  while (true) {
    Piece x{};
    if (u < u_end) {
      if (!loaded) {
        s = latent_seq(p, b);
        loaded = true;
      }
      const int kt = tiles_of(s), items = items_of(s, p.h);
      const int off = u - base;
      if (off >= kt * items) {
        base += kt * items;
        ++b;
        loaded = false;
        continue;
      }
      const int item = off / kt;
      x.p0 = s.p0;
      x.kv = s.kv;
      x.start = s.kv - s.tree;
      x.m0 = s.m0;
      x.node0 = s.tree - s.qo;
      x.m_row = item * kTile;
      x.row0 = s.q0 * p.h + x.m_row;
      x.nrows = min(kTile, s.qo * p.h - x.m_row);
      x.t0 = off - item * kt;
      x.t1 = min(kt, x.t0 + (u_end - u));
      x.slot = x.t0 == 0 && x.t1 == kt ? -1 : x.t0 == 0;
      if (x.slot == 1) {
        const int last = base + (item + 1) * kt - 1;
        merge.row0 = x.row0;
        merge.nrows = x.nrows;
        merge.parts = split.pair_of(last) - pair + 1;
      }
      u += x.t1 - x.t0;
    }
    const int slot = n % kPieces;
    if (!cx.wait(&m.piece_empty[slot], ((n / kPieces) & 1) ^ 1)) break;
    m.piece[slot] = x;
    mbar_arrive(&m.piece_full[slot]);
    ++n;
    if (x.t0 == x.t1) break;
  }
  if (leader) p.merge[pair] = merge;
}

// The page of a tile that a lane (modulo 8) loads; what is not there reads as zeros.
__device__ __forceinline__ int page_of(const LatentParams& p, const Piece& x, int t, int lane) {
  const int i = t * (kTile / kPageSize) + (lane & 7);
  const int pg = i * kPageSize < x.kv ? p.tab.page_values[x.p0 + i] : -1;
  return pg >= 0 && pg < p.tab.num_pages ? pg : p.tab.num_pages;
}

// Q, and of every page of a tile this CTA's 8 rows: two halves of the latent and
// the rotary key (whose box ends where rows end), one lane per page.
template <int RANK>
__device__ void run_k_producer(const Ctx& cx, const LatentParams& p, const AbsorbedMaps& maps,
                               uint32_t cta, int lane) {
  using C = Cfg<RANK>;
  Misc& m = *cx.m;
  const uint32_t q_full = in_first_cta(&m.q_full);
  const uint32_t sq = smem_u32(cx.smem + C::kOffQ);
  uint32_t n = 0, it = 0;
  for (;; ++n) {
    const int slot = n % kPieces;
    if (!cx.wait_warp(&m.piece_full[slot], (n / kPieces) & 1)) return;
    const Piece x = m.piece[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&m.piece_empty[slot]);
    if (x.t0 == x.t1) return;
    int next = page_of(p, x, x.t0, lane);
    if (!cx.wait_warp(&m.q_empty, (n & 1) ^ 1)) return;
    if (cta == 0 && lane == 0) mbar_arrive_expect_tx(&m.q_full, 2 * C::kChunks * kChunkBytes);
    __syncwarp();
    if (lane < C::kChunks)
      tma_load_pair(sq + lane * kChunkBytes, &maps.q, q_full, 64 * lane, x.row0 + 64 * (int)cta, 0);
    for (int t = x.t0; t < x.t1; ++t, ++it) {
      const int page = next;
      if (t + 1 < x.t1) next = page_of(p, x, t + 1, lane);
      if (lane == 0) *(volatile uint32_t*)&m.tiles = it + 1;
#pragma unroll
      for (int g = 0; g < 3; ++g) {
        if (!cx.wait_warp(&m.k_empty[g], (it & 1) ^ 1)) return;
        if (cta == 0 && lane == 0)
          mbar_arrive_expect_tx(&m.k_full[g], 2 * (g < 2 ? C::kPages * C::kKBox : kChunkBytes));
        __syncwarp();
        const uint32_t bar = in_first_cta(&m.k_full[g]);
        if (lane < C::kPages) {
          if (g < 2)
            tma_load_pair_4d(smem_u32(cx.smem + C::kOffK + (g * C::kPages + lane) * C::kKBox), &maps.k,
                             bar, 0, 8 * (int)cta, g * C::kHalf, page);
          else
            tma_load_pair(smem_u32(cx.smem + C::kOffRot + lane * 1024), &maps.rot, bar, RANK,
                          8 * (int)cta, page);
        }
        __syncwarp();
      }
    }
  }
}

// V: this CTA's half of the latent, all of a tile's rows, in two groups of pages.
// Slots past the sequence's last row may hold anything, and what does not count
// must not reach the products as NaN, so they are zeroed once they have arrived.
template <int RANK>
__device__ void run_v_producer(const Ctx& cx, const LatentParams& p, const AbsorbedMaps& maps,
                               uint32_t cta, int lane) {
  using C = Cfg<RANK>;
  Misc& m = *cx.m;
  uint8_t* sv = cx.smem + C::kOffV;
  uint32_t n = 0, it = 0;
  auto prefetch = [&](int page) {
    if (lane < C::kPages && page < p.tab.num_pages) {
      const int elements = kPageSize * (RANK + p.rope_dim);   // of a page: the bytes of a half
      prefetch_l2(p.pages + (int64_t)page * elements + (int)cta * (elements / 2), elements);
    }
    __syncwarp();
  };
  for (;; ++n) {
    const int slot = n % kPieces;
    if (!cx.wait_warp(&m.piece_full[slot], (n / kPieces) & 1)) return;
    const Piece x = m.piece[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&m.piece_empty[slot]);
    if (x.t0 == x.t1) return;
    int next = page_of(p, x, x.t0, lane), after = x.t0 + 1 < x.t1 ? page_of(p, x, x.t0 + 1, lane) : 0;
    if (x.t0 + 1 < x.t1) prefetch(after);
    for (int t = x.t0; t < x.t1; ++t, ++it) {
      const int page = next;
      next = after;
      // K has room for one tile, so the memory's latency would be in every tile's way:
      // the tile after the next goes into L2 ahead of it, of each page half by each CTA.
      // (As boxes of columns, two per page: decode of 64 sequences 75.4 instead of 74.5
      // us.  Three, four and six tiles ahead: 76.1, 77.4 and 85.0; trees 137 to 142
      // instead of 134.)
      if (t + kAhead < x.t1) {
        after = page_of(p, x, t + kAhead, lane);
        prefetch(after);
      }
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (!cx.wait_warp(&m.v_empty[g], (it & 1) ^ 1)) return;
        if (lane == 0) mbar_arrive_expect_tx(&m.v_full[g], C::kPages / 2 * C::kVBox);
        __syncwarp();
        if (lane / (C::kPages / 2) == g)
          tma_load_pair_4d(smem_u32(sv + lane * C::kVBox), &maps.v, smem_u32(&m.v_full[g]), 0, 0,
                           (int)cta * C::kHalf, page);
        __syncwarp();
      }
      const int valid = x.kv - t * kTile;
      const int dirty = valid < kTile && valid % kPageSize ? valid / kPageSize : -1;   // page
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (!cx.wait_warp(&m.v_full[g], it & 1)) return;
        if (dirty >= 0 && dirty / (C::kPages / 2) == g) {
          const int from = valid % kPageSize;
          for (int i = lane; i < (kPageSize - from) * C::kHalf * 8; i += 32) {
            const int c = i / 8 % C::kHalf, row = from + i / (8 * C::kHalf);
            *reinterpret_cast<uint4*>(sv + dirty * C::kVBox + (c * kPageSize + row) * 128 + (i & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) arrive_remote(in_first_cta(&m.v_ready[g]));
      }
    }
  }
}

// The products: QK(t + 1) goes before PV(t), so that the softmax of one tile
// runs beside the products of another.
template <int RANK, bool BF16>
__device__ void run_mma(const Ctx& cx, const LatentParams& p, uint32_t tmem, int pair, int lane) {
  using C = Cfg<RANK>;
  Misc& m = *cx.m;
  constexpr uint32_t idesc_qk = umma_idesc_f16(BF16, 128, 128, false);
  constexpr uint32_t idesc_pv = umma_idesc_f16(BF16, 128, 256, true);
  const uint64_t dq = sw128_desc(smem_u32(cx.smem + C::kOffQ), 0);
  const uint64_t dk = rows_desc(smem_u32(cx.smem + C::kOffK), 0, C::kKBox);
  const uint64_t dr = rows_desc(smem_u32(cx.smem + C::kOffRot), 0, 1024);
  const uint64_t dv = rows_desc(smem_u32(cx.smem + C::kOffV), kPageSize * 128, 1024);
  const uint64_t dp = sw128_desc(smem_u32(cx.smem + C::kOffP), 0);
  uint32_t n = 0, it = 0, qt = 0;   // pieces, tiles whose PV, whose QK was issued
  const int rot_steps = p.rope_dim / 16;
  bool ok = true, issued = false;
  if (p.debug_stall == 1 || p.debug_stall == -1 - pair) ok = cx.wait_warp(&m.stall, 0);
  auto qk = [&]() -> bool {
    const int b = qt & 1;
    if (!cx.wait_warp(&m.s_empty[b], ((qt >> 1) & 1) ^ 1)) return false;
    const uint32_t d = tmem + C::kTmemS + 64 * b;
    issued = true;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      if (!cx.wait_warp(&m.k_full[g], qt & 1)) return false;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < C::kHalf; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_pair(d, dq + (((g * C::kHalf + c) * kChunkBytes + k * 32) >> 4),
                      dk + ((g * C::kPages * C::kKBox + c * 1024 + k * 32) >> 4), idesc_qk,
                      g + c + k > 0 ? 1u : 0u);
        commit_pair(&m.k_empty[g]);
      }
      __syncwarp();
    }
    if (!cx.wait_warp(&m.k_full[2], qt & 1)) return false;
    tc_fence_after();
    if (elect_one()) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < rot_steps)
          umma_pair(d, dq + ((2 * C::kHalf * kChunkBytes + k * 32) >> 4), dr + (k * 32 >> 4), idesc_qk, 1u);
      commit_pair(&m.k_empty[2]);
      commit_pair(&m.s_full[b]);
    }
    __syncwarp();
    ++qt;
    return true;
  };
  for (; ok; ++n) {
    const int slot = n % kPieces;
    if (!(ok = cx.wait_warp(&m.piece_full[slot], (n / kPieces) & 1))) break;
    const int t0 = m.piece[slot].t0, t1 = m.piece[slot].t1, kv = m.piece[slot].kv;
    __syncwarp();
    if (lane == 0) mbar_arrive(&m.piece_empty[slot]);
    if (t0 == t1) break;
    if (!(ok = cx.wait_warp(&m.q_full, n & 1))) break;
    if (!(ok = qk())) break;
    if (t1 - t0 == 1 && elect_one()) commit_pair(&m.q_empty);
    __syncwarp();
    for (int t = t0; t < t1; ++t, ++it) {
      if (t + 1 < t1) {
        if (!(ok = qk())) break;
        if (t + 2 == t1 && elect_one()) commit_pair(&m.q_empty);
        __syncwarp();
      }
      if (t == t0 && !(ok = cx.wait_warp(&m.o_empty, (n & 1) ^ 1))) break;
      if (!(ok = cx.wait_warp(&m.p_full, it & 1))) break;
      const int steps = min(C::kPages, (kv - t * kTile + kPageSize - 1) / kPageSize);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (!(ok = cx.wait_warp(&m.v_ready[g], it & 1))) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = g * (C::kPages / 2); k < (g + 1) * (C::kPages / 2); ++k)
            if (k < steps)
#pragma unroll
              for (int j = 0; j < C::kHalf / 2; ++j)
                umma_pair(tmem + C::kTmemO + 128 * j,
                          dp + (((k >> 2) * kChunkBytes + (k & 3) * 32) >> 4),
                          dv + ((k * C::kVBox + j * 2 * kPageSize * 128) >> 4), idesc_pv,
                          k > 0 ? 1u : (uint32_t)(t > t0));
          commit_pair(&m.v_empty[g]);
          if (g == 1) commit_pair(&m.pv_done);
        }
        __syncwarp();
      }
      if (!ok) break;
    }
  }
  if (!ok && issued) {
    if (elect_one()) commit_pair(&m.drain);
    __syncwarp();
    const uint64_t t0 = globaltimer_ns();
    while (!try_wait_cluster(&m.drain, 0) && globaltimer_ns() - t0 < 10000000ull) {}
  }
}

// The exponent that a weight may reach over its reference, and where a moved
// reference puts the largest.  fp16 weights are held high, as what lies 2^-24 below
// a weight of one is the type's end and long sequences have mass there; bf16 ones
// are at most one, as values may be near the end of float32's range.
template <bool BF16>
struct Ref {
  static constexpr float kTop = BF16 ? 0.f : 15.f, kPut = BF16 ? -8.f : 7.f;
};

// O of this thread's lane and columns times f.
template <int RANK>
__device__ __noinline__ void rescale(uint32_t o, float f) {
#pragma unroll 1
  for (int c = 0; c < Cfg<RANK>::kCols; c += 32) {
    float v[32];
    tmem_ld32(o + c, v);
    tmem_wait_ld(v);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= f;
    tmem_st32(o + c, v);
  }
  tmem_wait_st();
}

// The elements of this CTA's values that are infinite or NaN made zero, in the rows
// of a tile that are set in ``rows``: eight of each of four pages from page0 on, row0
// their first.  By a whole warp.
template <int RANK, bool BF16>
__device__ __noinline__ void clear_values(uint8_t* sv, uint32_t rows, int page0, int row0, int lane) {
  using C = Cfg<RANK>;
  constexpr uint32_t kEnd = BF16 ? 0x7f80u : 0x7c00u;   // the exponent of what is not finite
  auto cleared = [](uint32_t w) {
    if ((w & kEnd) == kEnd) w &= 0xffff0000u;
    if ((w >> 16 & kEnd) == kEnd) w &= 0xffffu;
    return w;
  };
  while (rows) {
    const int j = __ffs(rows) - 1;
    rows &= rows - 1;
    uint8_t* row = sv + (page0 + (j >> 3)) * C::kVBox + (row0 + (j & 7)) * 128;
    for (int i = lane; i < C::kHalf * 8; i += 32) {
      uint4* at = reinterpret_cast<uint4*>(row + (i >> 3) * kPageSize * 128 + (i & 7) * 16);
      const uint4 u = *at;
      *at = make_uint4(cleared(u.x), cleared(u.y), cleared(u.z), cleared(u.w));
    }
  }
  fence_proxy_async_smem();
}

template <int RANK, bool BF16>
__device__ void run_softmax(const Ctx& cx, const LatentParams& p, uint32_t tmem, uint32_t cta,
                            int pair, int warp, int lane) {
  using C = Cfg<RANK>;
  Misc& m = *cx.m;
  const int quarter = warp & 3, wg = warp >> 2;
  const int half = quarter >> 1;                 // of every page's rows, of the latent's columns
  const int rr = (quarter & 1) * 32 + lane;      // packed row of this CTA's 64
  const int part = half * 2 + wg;                // of the row's four threads
  const bool checks = (quarter & 1) == 0;        // this warp's kv rows, for both of their warps
  const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
  const uint32_t o_at = tmem + lanes + C::kTmemO + wg * C::kCols;
  uint8_t* p_row = cx.smem + C::kOffP + wg * kChunkBytes + rr * 128;
  uint32_t n = 0, it = 0, turn = 0;
  // the four threads of a row give a number each and get all four combined (an
  // mbarrier of their warps, as every wait has a limit)
  auto exchange = [&](float& x, auto combine) {
    float(*e)[64] = m.exchange[turn & 1];
    uint64_t* bar = &m.shared_rows[quarter & 1][turn & 1];
    e[part][rr] = x;
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    if (!cx.wait_warp(bar, (turn >> 1) & 1)) return false;
    ++turn;
    x = combine(combine(e[0][rr], e[1][rr]), combine(e[2][rr], e[3][rr]));
    return true;
  };
  // where the walk of the tree enters this thread's row's node
  auto enter_of = [&](const Piece& x) {
    const int row = 64 * (int)cta + rr;
    if (x.start >= x.kv || row >= x.nrows) return 0;
    return reinterpret_cast<const int2*>(p.tree_order)[x.m0 + x.node0 + (x.m_row + row) / p.h].x;
  };
  // a scale of zero goes into the scores before those that do not count are made
  // infinite, which it would make NaN
  const bool flat = p.scale_log2 == 0.f;
  const float scale = flat ? 1.f : p.scale_log2;
  const float2 scale2 = make_float2(scale, scale);
  int enter_next = 0;
  for (;; ++n) {
    const int slot = n % kPieces;
    if (!cx.wait_warp(&m.piece_full[slot], (n / kPieces) & 1)) return;
    const Piece x = m.piece[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&m.piece_empty[slot]);
    if (x.t0 == x.t1) return;
    const int row = 64 * (int)cta + rr;          // of the item's 128
    const bool work = 64 * (int)cta + (quarter & 1) * 32 < x.nrows;   // some row of the warp exists
    const int2* order = reinterpret_cast<const int2*>(p.tree_order) + x.m0;
    const int enter = n == 0 ? enter_of(x) : enter_next;
    // l: the sum of the weights, lr: as rounded for the product, which O is divided
    // by (a row that one weight dominates then keeps its value's bits)
    float ref = -FLT_MAX, l = 0.f, lr = 0.f;
    for (int t = x.t0; t < x.t1; ++t, ++it) {
      const int b = it & 1;
      // this warp's kv rows: of four pages the 8 that its half of the lanes has; the
      // j-th score is of lane j's
      const int tok = t * kTile + wg * 64 + (lane >> 3) * kPageSize + half * 8 + (lane & 7);
      const bool masked = t * kTile > x.start - kTile;
      int2 iv = make_int2(INT32_MIN, INT32_MAX);
      if (masked && work) {
        if (tok >= x.kv)
          iv = make_int2(INT32_MAX, INT32_MIN);
        else if (tok >= x.start)
          iv = order[tok - x.start];
      }
      if (!cx.wait_warp(&m.s_full[b], (it >> 1) & 1)) return;
      tc_fence_after();
      float s[32];
      if (work || checks) {
        tmem_ld32(tmem + lanes + C::kTmemS + 64 * b + 32 * wg, s);
        tmem_wait_ld(s);
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) arrive_remote(in_first_cta(&m.s_empty[b]));
      // A weight of zero times a value that is not finite is NaN.  Such a value is an
      // element of its key too, so its scores are not finite, whatever the query (an
      // infinity times zero is NaN): for a q row that sees it the score is -inf and it
      // does not count, or the result is NaN whatever the values are.  For all rows
      // the value may be zero, so where all 32 scores of a kv row are not finite, its
      // values are looked through before their product.
      if (checks) {
        const float2 zero = make_float2(0.f, 0.f);
        float2 odd2 = zero;
#pragma unroll
        for (int j = 0; j < 32; j += 2) odd2 = ffma2(make_float2(s[j], s[j + 1]), zero, odd2);
        if (__all_sync(0xffffffffu, odd2.x + odd2.y != 0.f)) {
          uint32_t rows = 0;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            rows |= (uint32_t)(__all_sync(0xffffffffu, !(fabsf(s[j]) < INFINITY)) != 0) << j;
          rows &= __ballot_sync(0xffffffffu, tok < x.kv);   // the others are zeroed already
          if (rows) {
            if (!cx.wait_warp(&m.v_full[wg], it & 1)) return;
            clear_values<RANK, BF16>(cx.smem + C::kOffV, rows, 4 * wg, 8 * half, lane);
          }
        }
      }
      if (work) {
        // the largest of the scores, times their scale afterwards, whose sign is known;
        // what does not count is made the least there is
        const float least = scale > 0.f ? -INFINITY : INFINITY;
        if (flat) {
#pragma unroll
          for (int j = 0; j < 32; ++j) s[j] *= 0.f;
        }
        if (masked) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const int a = __shfl_sync(0xffffffffu, iv.x, j), e = __shfl_sync(0xffffffffu, iv.y, j);
            s[j] = a <= enter && enter < e ? s[j] : least;
          }
        }
        float top = s[0], top2 = s[1];
        if (scale > 0.f) {
#pragma unroll
          for (int j = 2; j < 32; j += 2) {
            top = fmaxf(top, s[j]);
            top2 = fmaxf(top2, s[j + 1]);
          }
          top = fmaxf(top, top2);
        } else {
#pragma unroll
          for (int j = 1; j < 32; ++j) top = fminf(top, s[j]);
        }
        top = top == least ? -INFINITY : top * scale;
        if (!exchange(top, [](float a, float c) { return fmaxf(a, c); })) return;
        const bool move = top - ref > Ref<BF16>::kTop;
        // P's buffer is free, and O at rest, once the tile before is done
        if (it > 0 && !cx.wait_warp(&m.pv_done, (it - 1) & 1)) return;
        if (__any_sync(0xffffffffu, move)) {
          float f = 1.f;
          if (move) {
            const float to = top - Ref<BF16>::kPut;
            f = ex2_approx(ref - to);
            ref = to;
            l *= f;
            lr *= f;
          }
          if (t > x.t0) {
            tc_fence_after();
            rescale<RANK>(o_at, f);
            tc_fence_before();
          }
        }
        float2 sum = make_float2(0.f, 0.f), sum_r = sum;
        const float2 shift = make_float2(-ref, -ref);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float2 e = ffma2(make_float2(s[8 * i + 2 * k], s[8 * i + 2 * k + 1]), scale2, shift);
            e = make_float2(ex2_approx(e.x), ex2_approx(e.y));
            w[k] = pack2<BF16>(e.x, e.y);
            sum = fadd2(sum, e);
            sum_r = fadd2(sum_r, unpack2<BF16>(w[k]));
          }
          *reinterpret_cast<uint4*>(p_row + (((2 * i + half) ^ (rr & 7)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
        l += sum.x + sum.y;
        lr += sum_r.x + sum_r.y;
        fence_proxy_async_smem();
      } else if (it > 0 && !cx.wait_warp(&m.pv_done, (it - 1) & 1)) {
        return;   // no warp is a phase of p_full ahead
      }
      __syncwarp();
      if (lane == 0) arrive_remote(in_first_cta(&m.p_full));
    }
    // the next piece's rows are looked up behind this one's last product
    if (p.tree_order) {
      const int after = (n + 1) % kPieces;
      if (!cx.wait_warp(&m.piece_full[after], ((n + 1) / kPieces) & 1)) return;
      enter_next = enter_of(m.piece[after]);
    }
    // the piece's result
    if (!cx.wait_warp(&m.pv_done, (it - 1) & 1)) return;
    if (work) {
      tc_fence_after();
      const auto add = [](float a, float c) { return a + c; };
      if (!exchange(l, add) || !exchange(lr, add)) return;
      const bool valid = row < x.nrows;
      const int col0 = half * (RANK / 2) + wg * C::kCols;
      if (x.slot < 0) {
        const int64_t at = (int64_t)x.row0 + row;
        const float inv = lr == 0.f ? 0.f : 1.f / lr;
        const int four = lane & ~3;              // the rows whose vectors this lane stores
        uint16_t* out = p.out + (at - lane + four) * RANK + col0 + (lane & 3) * 8;
        const float2 zero = make_float2(0.f, 0.f), by = make_float2(inv, inv);
#pragma unroll 1
        for (int c = 0; c < C::kCols; c += 32) {
          float v[32];
          tmem_ld32(o_at + c, v);
          tmem_wait_ld(v);
          uint4 y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 z = ffma2(make_float2(v[8 * i + 2 * k], v[8 * i + 2 * k + 1]), by, zero);
              w[k] = pack2<BF16>(z.x, z.y);
            }
            y[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          transpose4(y, lane);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (row - lane + four + j < x.nrows) *reinterpret_cast<uint4*>(out + j * RANK + c) = y[j];
        }
        if (valid && part == 0) p.lse[at] = l == 0.f ? -INFINITY : ref + log2f(l);
      } else {
        float* st = p.parts + (int64_t)(2 * pair + x.slot) * kSlotFloats;
        float4* o = reinterpret_cast<float4*>(st) + (col0 / 4) * kTile + row;
#pragma unroll 1
        for (int c = 0; c < C::kCols; c += 32) {
          float v[32];
          tmem_ld32(o_at + c, v);
          tmem_wait_ld(v);
          if (valid)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              __stcg(o + (c / 4 + i) * kTile, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
        }
        if (valid && part == 0) {
          st[kTile * 512 + row] = ref;
          st[kTile * 513 + row] = l;
          st[kTile * 514 + row] = lr;
        }
      }
      tc_fence_before();
    }
    __syncwarp();
    if (lane == 0) arrive_remote(in_first_cta(&m.o_empty));
  }
}

template <int RANK, bool BF16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    absorbed_kernel(const __grid_constant__ AbsorbedMaps maps, const LatentParams p) {
  using C = Cfg<RANK>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc& m = *reinterpret_cast<Misc*>(smem + C::kOffMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t cta = cta_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (tid == 0) {
    mbar_init(&m.q_full, 1);
    mbar_init(&m.q_empty, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&m.k_full[i], 1);
      mbar_init(&m.k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&m.v_full[i], 1);
      mbar_init(&m.v_empty[i], 1);
      mbar_init(&m.v_ready[i], 2);
      mbar_init(&m.s_full[i], 1);
      mbar_init(&m.s_empty[i], 16);
    }
    mbar_init(&m.p_full, 16);
    mbar_init(&m.pv_done, 1);
    mbar_init(&m.o_empty, 16);
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(&m.piece_full[i], 1);
      mbar_init(&m.piece_empty[i], cta == 0 ? 11 : 10);   // its readers
    }
    for (int i = 0; i < 4; ++i) mbar_init(&m.shared_rows[i >> 1][i & 1], 4);
    mbar_init(&m.stall, 1);
    mbar_init(&m.drain, 1);
    m.abort = 0;
    m.tiles = 0;
    m.first_seq = 0;
    m.first_unit = 0;
    mbar_fence_init();
  }
  if (warp == 8) {
    if (lane == 0) {
      tma_prefetch_desc(&maps.q);
      tma_prefetch_desc(&maps.k);
      tma_prefetch_desc(&maps.rot);
      tma_prefetch_desc(&maps.v);
    }
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(&m.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  // this thread's sequences: checked, and their tiles counted
  const int each = (p.tab.batch + kThreads - 1) / kThreads;
  const int b_lo = min(p.tab.batch, tid * each), b_hi = min(p.tab.batch, b_lo + each);
  long long mine = 0;
  bool bad = false, empty = false;
  LatentSeq s{};
  for (int b = b_lo; b < b_hi; ++b) {
    s = latent_seq(p, b);
    bad |= !s.good;
    empty |= s.kv == 0;
    if (s.good) mine += (long long)tiles_of(s) * items_of(s, p.h);
  }
  long long sum = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += y;
  }
  if (lane == 31) m.scan[warp] = sum;
  bool stop = __syncthreads_or(bad);
  long long before = sum - mine, total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += m.scan[i];
    total += m.scan[i];
  }
  stop |= total > INT32_MAX;
  const Split split{(int)total / pairs, (int)total % pairs};
  const int u = split.start(pair);
  if (!stop && u >= before && u < before + mine) {
    int b = b_lo;
    for (; each > 1 && b < b_hi; ++b) {
      s = latent_seq(p, b);
      const int k = tiles_of(s) * items_of(s, p.h);
      if (u < before + k) break;
      before += k;
    }
    m.first_seq = b;
    m.first = s;
    m.first_unit = (int)before;
  }
  if (stop && tid == 0) {
    atomicOr(p.error, DEVERR_BAD_INDPTR);
    if (cta == 0) p.merge[pair] = LatentMerge{};
  }
  // one-token attention of sequences without rows
  if (__syncthreads_or(empty) && !stop && !p.q_indptr) {
    for (int b = blockIdx.x; b < p.tab.batch; b += gridDim.x) {
      if (p.tab.page_indptr[b] != p.tab.page_indptr[b + 1]) continue;
      uint4* o = reinterpret_cast<uint4*>(p.out + (int64_t)b * p.h * RANK);
      for (int i = tid; i < p.h * (RANK / 8); i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
      if (tid < p.h) p.lse[(int64_t)b * p.h + tid] = -INFINITY;
    }
  }
  const Ctx cx{smem, &m, p.error, p.timeout_ns};
  if (!stop) {
    if (warp < 8)
      run_softmax<RANK, BF16>(cx, p, m.tmem, cta, pair, warp, lane);
    else if (warp == 8)
      run_k_producer<RANK>(cx, p, maps, cta, lane);
    else if (warp == 9)
      run_v_producer<RANK>(cx, p, maps, cta, lane);
    else if (warp == 10) {
      if (cta == 0) run_mma<RANK, BF16>(cx, p, m.tmem, pair, lane);
    } else if (lane == 0)
      run_planner(cx, p, split, pair, cta == 0);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // after a wait ran out copies may still be on their way into shared memory
  if (m.abort) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  cluster_sync();   // neither CTA leaves while the other's products or arrivals may reach it
  if (tid == 0) p.merge[pair].gave_up[cta] = m.abort;   // behind the pair's record
  if (warp == 8) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(m.tmem) : "memory");
  }
}

// ---------------------------------------------------------------------------
// merge
// ---------------------------------------------------------------------------
constexpr int kMergeThreads = 256;   // 32 packed rows by 8 warps
constexpr int kMaxPairs = 128;

// One unit of work: 32 rows by 32 V columns of an item, V vectors of 4 columns and B
// of its parts in flight per thread.
template <int RANK, bool BF16, int V, int B>
__device__ __forceinline__ void merge_unit(const LatentParams& p, const LatentMerge& r, int pair,
                                           int row0, int slice, uint2 (*s_out)[8 * V + 1]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, row = row0 + lane;
  const bool valid = row < r.nrows;
  const int at = min(row, r.nrows - 1);
  float top = -FLT_MAX, l = 0.f, lr = 0.f;
  float4 o[V];
#pragma unroll
  for (int j = 0; j < V; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < r.parts; k0 += B) {
    float4 v[B][V];
    float pm[B], pl[B], pr[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      pm[k] = -FLT_MAX;
      pl[k] = pr[k] = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) v[k][j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + k < r.parts) {
        const float* st = p.parts + (int64_t)(2 * (pair + k0 + k) + (k0 + k == 0)) * kSlotFloats;
        pm[k] = __ldcg(st + kTile * 512 + at);
        pl[k] = __ldcg(st + kTile * 513 + at);
        pr[k] = __ldcg(st + kTile * 514 + at);
#pragma unroll
        for (int j = 0; j < V; ++j)
          v[k][j] = __ldcg(reinterpret_cast<const float4*>(st) + ((slice * 8 + warp) * V + j) * kTile + at);
      }
    }
    float to = top;
#pragma unroll
    for (int k = 0; k < B; ++k) to = fmaxf(to, pm[k]);
    const float f = ex2_approx(top - to);
    top = to;
    l *= f;
    lr *= f;
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = make_float4(o[j].x * f, o[j].y * f, o[j].z * f, o[j].w * f);
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const float w = ex2_approx(pm[k] - top);
      l += w * pl[k];
      lr += w * pr[k];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        o[j].x += w * v[k][j].x;
        o[j].y += w * v[k][j].y;
        o[j].z += w * v[k][j].z;
        o[j].w += w * v[k][j].w;
      }
    }
  }
  const float inv = lr == 0.f ? 0.f : 1.f / lr;
  __syncthreads();                             // s_out is read from the unit before
#pragma unroll
  for (int j = 0; j < V; ++j)
    s_out[lane][warp * V + j] =
        make_uint2(pack2<BF16>(o[j].x * inv, o[j].y * inv), pack2<BF16>(o[j].z * inv, o[j].w * inv));
  const int64_t first = (int64_t)r.row0 + row0;
  if (warp == 0 && slice == 0 && valid) p.lse[first + lane] = l == 0.f ? -INFINITY : top + log2f(l);
  __syncthreads();
  // 64 V contiguous bytes of every row
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = tid + j * kMergeThreads, orow = i / (8 * V), c = i % (8 * V);
    if (row0 + orow < r.nrows)
      *reinterpret_cast<uint2*>(p.out + (first + orow) * RANK + (slice * 8 * V + c) * 4) = s_out[orow][c];
  }
}

// Joins the parts of the items that several pairs share, in their order:
//   m = max m_i,  O = sum 2^(m_i - m) O_i,  l = sum 2^(m_i - m) l_i.
// Bound by latency: 4 to 8 us, of which reading the parts (at most 2 x 76 of 264 KB,
// mostly in L2) would be 3 to 6.  All items'
// units are shared out over four CTAs per SM, of which the registers let two be
// resident: large units where there are two for each of them (a unit costs its loads'
// latency once), small ones where not.  Small units have 12 parts in flight: one
// sequence of 4,096 rows in 32 parts 13.0 us, with 8 14.0; with 16, which spill, 12.8,
// but 64 sequences 78.6 instead of 75.3.
template <int RANK, bool BF16>
__global__ void __launch_bounds__(kMergeThreads, 2) absorbed_merge_kernel(const LatentParams p, int pairs) {
  __shared__ int s_at[kMaxPairs + 1];          // groups of 32 rows before each item
  __shared__ LatentMerge s_rec[kMaxPairs];
  __shared__ uint2 s_out[32][33];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < pairs) s_rec[tid] = p.merge[tid];
  // after a wait ran out, items with a part of that pair's are left as they are
  if (__syncthreads_or(tid < pairs && (s_rec[tid].gave_up[0] | s_rec[tid].gave_up[1]))) {
    bool lost = false;
    if (tid < pairs)
      for (int i = tid; i < min(pairs, tid + s_rec[tid].parts); ++i)
        lost |= s_rec[i].gave_up[0] | s_rec[i].gave_up[1];
    __syncthreads();
    if (lost) s_rec[tid].parts = 0;
    __syncthreads();
  }
  if (tid < 32) {
    int sum = 0;
    for (int base = 0; base < pairs; base += 32) {
      const int i = base + lane;
      const int n = i < pairs && s_rec[i].parts > 0 ? (s_rec[i].nrows + 31) / 32 : 0;
      int up = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, up, d);
        if (lane >= d) up += y;
      }
      if (i < pairs) s_at[i] = sum + up - n;
      sum += __shfl_sync(0xffffffffu, up, 31);
    }
    if (lane == 0) s_at[pairs] = sum;
  }
  __syncthreads();
  const int groups = s_at[pairs];
  const bool large = groups * (RANK / 128) * 2 >= (int)gridDim.x;
  const int slices = large ? RANK / 128 : RANK / 32;
  for (int u = blockIdx.x; u < groups * slices; u += gridDim.x) {
    // the last item that begins at or before u's group (those without any begin where
    // the next does)
    const int g = u / slices;
    int pair = 0;
    for (int step = kMaxPairs / 2; step > 0; step >>= 1)
      if (pair + step < pairs && s_at[pair + step] <= g) pair += step;
    const int row0 = (g - s_at[pair]) * 32;
    if (large)
      merge_unit<RANK, BF16, 4, 4>(p, s_rec[pair], pair, row0, u % slices, s_out);
    else
      merge_unit<RANK, BF16, 1, 12>(p, s_rec[pair], pair, row0, u % slices,
                                   reinterpret_cast<uint2(*)[9]>(s_out));
  }
}

template <int RANK, bool BF16>
cudaError_t launch(const LatentParams& p, const AbsorbedMaps& maps, int pairs, int nsm,
                   cudaStream_t stream) {
  using C = Cfg<RANK>;
  constexpr int smem = C::kOffMisc + (int)sizeof(Misc);
  static_assert(smem <= 232448, "shared memory of an SM");
  const auto kern = absorbed_kernel<RANK, BF16>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_shared((const void*)kern, smem, allowed);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(2 * pairs), dim3(kThreads), smem, stream, maps, p);
  if (e != cudaSuccess) return e;
  // a table of no more pages than a tile's has no item of two tiles
  if (p.tab.nnz_pages <= kTile / kPageSize) return cudaSuccess;
  return launch_pdl(absorbed_merge_kernel<RANK, BF16>, dim3(4 * nsm), dim3(kMergeThreads), 0, stream,
                    p, pairs);
}

int max_pairs(int nsm) { return nsm < 4 ? 1 : nsm / 2 < kMaxPairs ? nsm / 2 : kMaxPairs; }

}  // namespace

LatentWorkspace latent_workspace(int num_pages, int nsm) {
  LatentWorkspace w{};
  const int64_t pairs = max_pairs(nsm);
  w.off_merge = 256;
  w.off_parts = w.off_merge + round_up(pairs * (int64_t)sizeof(LatentMerge), 256);
  w.off_marks = w.off_parts + round_up(pairs * 2 * kSlotFloats * 4, 256);
  w.total = w.off_marks + round_up((int64_t)num_pages * 4, 256);
  return w;
}

cudaError_t launch_absorbed(const LatentParams& p, const AbsorbedMaps& maps, bool bf16, int nsm,
                            cudaStream_t stream) {
  // no more pairs than tiles there can be
  const int64_t kv_tiles = p.tab.nnz_pages / (kTile / kPageSize) + p.tab.batch;
  const int64_t row_tiles = p.q_indptr ? ceil_div((int64_t)p.total_q * p.h, kTile) + p.tab.batch : 1;
  int pairs = max_pairs(nsm);
  if (kv_tiles * row_tiles < pairs) pairs = (int)(kv_tiles * row_tiles);
  if (p.rank == 512)
    return bf16 ? launch<512, true>(p, maps, pairs, nsm, stream)
                : launch<512, false>(p, maps, pairs, nsm, stream);
  return bf16 ? launch<256, true>(p, maps, pairs, nsm, stream)
              : launch<256, false>(p, maps, pairs, nsm, stream);
}

}  // namespace ta
