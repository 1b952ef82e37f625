// Attention over the paged cache for many rows a key head: chunks of prompts,
// and the rows of all sequences together against a shared prefix.
//
// With 256 rows to a key head's tile the work is bound by the tensor cores,
// not by HBM, so the rows go through tcgen05 as in the square forward: one
// persistent CTA per SM, two 128-row tiles (A and B) that share the stream of
// keys and values, softmax warpgroups that own one row a thread, accumulators
// in tensor memory, and the lazy reference maximum and the correction of the
// largest rounded weight of that kernel (fwd.cu).  What differs:
//
//  - Rows.  The G * Nq rows of a key head are one row space (or B * G * Nq for
//    the prefix: the queries of every sequence side by side, which is what
//    lets its keys be read once).  A warp gathers them from q into the swizzled
//    tiles, a piece ahead; each row has its own last visible key.
//  - Keys come from pages: a tile of 128 keys is 128 / box_rows TMA boxes, one a
//    lane of the producer warp, page ids read 32 boxes ahead.  A box brings all
//    columns of its rows, in groups of 8 rows whose 64-column blocks lie one
//    behind the other: a layout that the MMA descriptors know as well as blocks
//    of all rows, and half the loads at d = 128.
//  - Division.  The first one to two units (256 rows of a key head) for every
//    CTA form a line of key tiles that is cut into equal ranges, one a CTA, as
//    in the step kernel; the others are drawn whole from a counter, heaviest
//    first within groups of heads whose keys stay in L2.  So few units fill
//    the GPU, and many end together, on their lightest.  Where units differ so
//    much that they end together anyway (prompts under the causal rule), none
//    is cut; the kernel finds that out from the lengths.  Pieces of a unit leave
//    normalised outputs and log-sum-exps that the merge kernels of paged.cu take
//    up.  One warp works out what the next pieces are and the others read it,
//    so that none of it stands between two pieces.
//  - Rows of a page behind the last key may hold anything, NaN included, and
//    0 * NaN would poison the product with V: a spare warp zeroes them in the
//    last tile before that product is issued.
//
// Measured (whole calls): a square prompt of 16 heads x 16384 tokens 1574
// TFLOP/s, 32 heads under the causal rule 1409 to 1442; two chunks of 1000
// tokens, 32 heads on 8, over 9001 and 16384 keys 290 us = 1378
// TFLOP/s; 2048 rows of 8 heads behind 32768 shared keys 193 us in this kernel.  The tensor
// pipe is 59 to 61% busy in the last two, DRAM 12 to 14%.  The smallest call, 64
// rows of 8 heads over 512 keys, is 12.8 us: 1.7 until the line is there, 1.8 until a
// piece is worked out, 1.5 until its first scores, 2 for the softmax and the second
// product, 2 for writing the rows, then the merge.  Prompts under the causal
// rule: 16 heads x 4096 tokens 68 us, 8 x 8192 121, 16 x 8192 233 with pages of 16,
// 32, 64 or 128 keys.  (With a box a 64-column block pages of 16 keys cost a sixth
// more, bound by the issue of the boxes.)
//
//   warps 0-3  softmax of tile A     warp 8   TMA producer
//   warps 4-7  softmax of tile B     warp 9   MMA issuer, owns tensor memory
//                                    warp 10  brings rows in; zeroes values behind the last key
//                                    warp 11  works out the pieces
//
// A cache in E4M3 (FP8).  A key or value is its number times the scale of its 16
// tokens and head: scores z_j = scale * sk_j (q . k_j), weights p_j = 2^z_j, O = sum p_j
// sv_j v_j / sum p_j.  The softmax takes the scales in: x_j = z_j + log2 sv_j is what the
// maximum is taken of, 2^(x_j - reference) what the product takes, that times 1 / sv_j
// what the sum takes, with three numbers for every 16 columns of a tile.
//
//  - Keys go into the product as they lie in the cache.  A query, times a power of
//    two that brings its row's largest value into [128, 256), is the sum of two E4M3
//    numbers, which a softmax thread puts in the place of its row: S = hi K^T + lo K^T
//    at twice the rate of bf16.
//  - Values become fp16, in which they are exact, and so do the weights (11
//    significand bits, 2^7 at the reference): in E4M3 those far below the largest,
//    many as they may be, would be lost.  Three more warps (12, 14, 15) convert a
//    tile's values, and zero those behind the last key.
//
// Measured: the two chunks 341 us = 1172 TFLOP/s, 256 sequences x 64 heads on 8 behind
// 32768 shared keys 254 us (221 in this kernel), 24 sequences of 4 drafted tokens
// behind 8208 keys 31.6.  A step (a key tile with both row tiles) has 2048 cycles
// of products, as in bf16, and takes 3270 to 3350 in a long piece (bf16 3060 to 3140):
// the chain score product - softmax - value product of either row tile bounds it, not
// the tensor cores (51 to 52% busy) nor DRAM (4 to 5%).  Copies that skip work (two
// chunks, 384 us at the time): without the conversion of values 376, with half the
// score products 394, without exponentials 333.  A piece begins 4700 cycles later for
// its rows' conversion.
#pragma once

#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>
#include <cfloat>
#include <climits>
#include <type_traits>

#include "internal.h"
#include "paged.cuh"
#include "ptx_e4m3.cuh"
#include "serving.h"

namespace fa {
namespace {

// registers: the split of the square forward (fwd.cu), 2*128*192 + 128*120 =
// 384*168; with four more warps 2*128*168 + 2*128*88 = 512*128
template <bool FP8>
struct Launch {
  static constexpr int kThreads = FP8 ? 512 : 384;
  static constexpr int kRegs = FP8 ? 128 : 168;
  static constexpr int kSoftmaxRegs = FP8 ? 168 : 192;
  static constexpr int kOtherRegs = FP8 ? 88 : 120;
  // warps that follow the pieces: all but the one that works them out, and with
  // E4M3 one that is idle
  static constexpr int kReaders = kThreads / 32 - 1 - FP8;
  static_assert(2 * 128 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs <= kThreads * kRegs,
                "register split exceeds the launch allocation");
};
constexpr float kTau = 8.f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoScore = -FLT_MAX;  // reference maximum before any score: finite, so that -inf less it is -inf
constexpr int kRows = 128;        // rows and keys a tile
// Key tiles before a piece's end that the next one is drawn.  (16 heads x 8192
// tokens 231 us with 2, 230 with 4, 228 with 6, 284 at the piece's beginning; 2 x
// 12 heads x 5000 tokens 169, 167, 169 and 204; 4 x 16 x 4096 262, 256, 258, 278.)
constexpr int kTellTiles = 4;
constexpr int kScales = kRows / kScaleTokens;  // scales of a tile's keys
constexpr int kScaleTiles = 16;   // tiles whose scales are kept: more than lie between a tile's loads and its weights
constexpr float kShift = 7.f;     // log2 of an fp16 weight at the reference
// Warps that convert values: 12, 14 and 15, while 13, which would share the
// issuer's scheduler, is idle.  (Two chunks of 1000 tokens, 256 sequences behind a
// prefix, us: 380 and 259 with all four, 377 and 253 so.)
constexpr int kConverters = 3;

enum TileSite : int {
  SITE_TILE_LOAD = 75,
  SITE_TILE_MMA = 76,
  SITE_TILE_S = 77,
  SITE_TILE_O = 78,
  SITE_TILE_CLEAN = 79,
  SITE_TILE_PIECE = 80,
  SITE_TILE_CONVERT = 84,
};

// A piece of a unit, as the roles read it.
struct Piece {
  int na, nb;      // key tiles that row tiles A and B take; na < 0: there is no further piece
  int tiles;       // key tiles
  int tile;        // the unit's first of them
  int limit;       // keys (from the origin) whose values are the sequence's own
  int clean;       // the piece's tile that the limit falls into, or -1
  int b, head, r0; // sequence, key head, first row
  int whole;       // all of the unit, and its result is the row's
  int slot;        // of the partial result
};

template <int D, bool DUAL, bool FP8>
struct TileLayout {
  static constexpr int kTileBytes = kRows * D * 2;
  // two tiles of rows; where both row tiles have the same rows one, and one
  // more key or value tile on its way (64 sequences x 8 heads x 64 rows x 1000
  // keys: 85 us with four, 80 with five)
  static constexpr int kQTiles = DUAL ? 1 : 2;
  // bf16: one ring, keys and values in turn.  E4M3: a ring of keys, one of values
  // (half the bytes) and one of values in fp16.
  static constexpr int kWide = D == 128 ? 1 : 2;
  static constexpr int kSlots = FP8 ? 0 : 6 * kWide - kQTiles * kWide;
  static constexpr int kKeySlots = FP8 ? (DUAL ? 3 : 2) * kWide : 0;
  static constexpr int kRawSlots = kKeySlots;
  static constexpr int kValueSlots = FP8 ? 2 * kWide : 0;
  static constexpr int kRingOff = kQTiles * kTileBytes;
  static constexpr int kKeyOff = kRingOff + (kSlots + kValueSlots) * kTileBytes;
  static constexpr int kRawOff = kKeyOff + kKeySlots * (kTileBytes / 2);
  // a warp's staging of its output rows: 32 rows of 64 bytes, so that rows
  // leave in 64-byte runs instead of a 16-byte store a row
  static constexpr int kStageOff = kRawOff + kRawSlots * (kTileBytes / 2);
  static constexpr int kBarOff = kStageOff + 8 * 2048;
  static constexpr int KV_FULL = 0;
  static constexpr int KV_EMPTY = KV_FULL + kSlots;
  static constexpr int K_FULL = KV_EMPTY + kSlots;
  static constexpr int K_EMPTY = K_FULL + kKeySlots;
  static constexpr int RAW_FULL = K_EMPTY + kKeySlots;   // values as they lie in the cache
  static constexpr int RAW_EMPTY = RAW_FULL + kRawSlots;
  static constexpr int V_FULL = RAW_EMPTY + kRawSlots;   // ... and in fp16
  static constexpr int V_EMPTY = V_FULL + kValueSlots;
  static constexpr int SCALES = V_EMPTY + kValueSlots;
  static constexpr int BEGUN = SCALES + (FP8 ? kScaleTiles : 0);  // the pieces' scales before this one are there
  static constexpr int Q_RAW = BEGUN + (FP8 ? 2 : 0);    // rows in bf16
  static constexpr int Q_FULL = Q_RAW + (FP8 ? 2 : 0);
  static constexpr int Q_IN = FP8 ? Q_RAW : Q_FULL;      // what the loads of rows arrive on
  static constexpr int Q_EMPTY = Q_FULL + 2;
  static constexpr int S_FULL = Q_EMPTY + 2;
  static constexpr int P_FULL = S_FULL + 2;
  static constexpr int O_FULL = P_FULL + 2;
  static constexpr int DIRTY = O_FULL + 2;
  static constexpr int CLEAN = DIRTY + 1;
  static constexpr int PIECE_FULL = CLEAN + 1;
  static constexpr int PIECE_EMPTY = PIECE_FULL + 2;
  static constexpr int ROWS_FULL = PIECE_EMPTY + 2;
  static constexpr int LOADED = ROWS_FULL + 2;
  static constexpr int PAIR = LOADED + 1;    // two row tiles on the same rows: warps w and w + 4 have their statistics
  static constexpr int PAIR_DONE = PAIR + 4; // ... and have read both accumulators
  static constexpr int DRAIN = PAIR_DONE + 4;
  static constexpr int kNumBars = DRAIN + 1;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kScratchOff = kMiscOff + 16;            // one word a warp
  static constexpr int kPieceOff = kScratchOff + 64;           // two pieces
  static constexpr int kRowOff = kPieceOff + 2 * 48;           // [2 pieces][256 rows] place in q and o, then last key
  static constexpr int kStatOff = kRowOff + 2 * kPairRows * 8; // [2 row tiles][maximum, sum, correction][128]
  // [tiles][groups of 16 keys][keys' scale times `scale`, log2 of values', 1 / values', -]
  static constexpr int kScaleOff = (kStatOff + 2 * 3 * kRows * 4 + 15) / 16 * 16;
  static constexpr int kGrowOff = kScaleOff + (FP8 ? kScaleTiles * kScales * 16 : 0);  // [128] rows' multipliers
  static constexpr int kLineOff = kGrowOff + (FP8 && DUAL ? kRows * 4 : 0);
  static constexpr int kSmemBytes = kLineOff + (kTileLine + 1) * 4 + 1024;
  static constexpr uint32_t kColO = 256;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");
  // Scales are written behind the wait for a key slot, which is free once the
  // scores of the tile kKeySlots before it are there, and so the weights of the
  // row tile's one before that (DUAL: two before it).  A row tile that has had no
  // keys waits until the producer has begun its piece (BEGUN).
  static_assert(!FP8 || kKeySlots + 2 <= kScaleTiles, "scales still in use");
};
static_assert(sizeof(Piece) <= 48, "a piece's room");

__device__ __forceinline__ bool tile_wait(uint32_t bar, uint32_t parity, const WaitCtl& w, int site, int unit) {
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, w, site, unit));
}

// A box of whole rows of a page, in groups of 8 rows from `group` on.
__device__ __forceinline__ void tma_load_groups(uint32_t dst, const CUtensorMap* map, uint32_t bar, int group,
                                                int outer, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %2, %2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(outer), "r"(bar), "l"(policy)
      : "memory");
}

__device__ __forceinline__ float2 ld_shared_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > limit_ns) return;
  }
}

// Keys (from the origin prefix_len) that some row of rows [r0, r0 + 128) of a
// sequence sees, at most; 0 if none of them is a valid query.
__device__ __forceinline__ int tile_keys(int r0, int rows, int nq, int lq, int lk, int origin, bool causal) {
  if (r0 >= rows || lq == 0) return 0;
  int keys = lk - origin;
  if (causal) {
    const int r1 = min(r0 + kRows, rows) - 1;
    if (r0 / nq == r1 / nq) {  // rows of one head: queries [i0, i1]
      const int i0 = r0 % nq, i1 = r1 % nq;
      if (i0 >= lq) return 0;
      keys = min(i1, lq - 1) + 1 + lk - lq - origin;
    }
  }
  return max(keys, 0);
}

// Byte offset of 16-byte chunk c of row r in a tile of rows of D bytes.
template <int D>
__device__ __forceinline__ uint32_t byte_chunk(int r, int c) {
  return D == 128 ? sw128(r, c) : sw64(r, c);
}

template <int D, bool PREFIX, bool DUAL, bool FP8>
__global__ void __launch_bounds__(Launch<FP8>::kThreads, 1)
    paged_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedTiles p) {
  using L = TileLayout<D, DUAL, FP8>;
  constexpr int kThreads = Launch<FP8>::kThreads;
  constexpr int S = FP8 ? 1 : L::kSlots;
  constexpr int KSL = FP8 ? L::kKeySlots : 1, RSL = FP8 ? L::kRawSlots : 1, VSL = FP8 ? L::kValueSlots : 1;
  constexpr int CB = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + L::kBarOff;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  int* scratch = reinterpret_cast<int*>(smem + L::kScratchOff);
  int* line = reinterpret_cast<int*>(smem + L::kLineOff);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int Hkv = p.seq.Hkv;
  const int rows = p.seq.G * p.seq.Nq;              // rows a key head of a sequence
  const int space = PREFIX ? p.seq.B * rows : rows;  // rows of an entry's row space
  const int origin = PREFIX ? 0 : p.seq.prefix_len;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kSlots; ++s) {
      mbar_init(bars + 8 * (L::KV_FULL + s), 1);
      mbar_init(bars + 8 * (L::KV_EMPTY + s), 1);
    }
    if constexpr (FP8) {
      for (int s = 0; s < KSL; ++s) {
        mbar_init(bars + 8 * (L::K_FULL + s), 1);
        mbar_init(bars + 8 * (L::K_EMPTY + s), 1);
      }
      for (int s = 0; s < RSL; ++s) {
        mbar_init(bars + 8 * (L::RAW_FULL + s), 1);
        mbar_init(bars + 8 * (L::RAW_EMPTY + s), kConverters);
      }
      for (int s = 0; s < VSL; ++s) {
        mbar_init(bars + 8 * (L::V_FULL + s), kConverters);
        mbar_init(bars + 8 * (L::V_EMPTY + s), 1);
      }
      for (int s = 0; s < kScaleTiles; ++s) mbar_init(bars + 8 * (L::SCALES + s), 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(bars + 8 * (L::BEGUN + i), 1);
        mbar_init(bars + 8 * (L::Q_RAW + i), 1);
      }
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bars + 8 * (L::Q_FULL + t), FP8 ? 4 : 1);
      mbar_init(bars + 8 * (L::Q_EMPTY + t), 1);
      mbar_init(bars + 8 * (L::S_FULL + t), 1);
      mbar_init(bars + 8 * (L::P_FULL + t), 4);
      mbar_init(bars + 8 * (L::O_FULL + t), 1);
    }
    mbar_init(bars + 8 * L::DIRTY, 1);
    mbar_init(bars + 8 * L::CLEAN, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + 8 * (L::PIECE_FULL + i), 1);
      mbar_init(bars + 8 * (L::PIECE_EMPTY + i), Launch<FP8>::kReaders);
      mbar_init(bars + 8 * (L::ROWS_FULL + i), 1);
    }
    mbar_init(bars + 8 * L::LOADED, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(bars + 8 * (L::PAIR + i), 2);
      mbar_init(bars + 8 * (L::PAIR_DONE + i), 2);
    }
    mbar_init(bars + 8 * L::DRAIN, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    if (p.boxed_rows) prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (p.wait_first) grid_wait(); else grid_overlap();
  grid_trigger();
  // the prefix's keys that some sequence reaches
  int reach = 0;
  if constexpr (PREFIX) {
    for (int b = threadIdx.x; b < p.seq.B; b += kThreads) {
      int lq, lk;
      seq_lens(p.seq, b, lq, lk);
      if (lq > 0) reach = max(reach, min(lk, p.seq.prefix_len));
    }
    reach = __reduce_max_sync(0xffffffffu, reach);
    if (lane == 0) scratch[warp] = reach;
    __syncthreads();
    for (int i = 0; i < kThreads / 32; ++i) reach = max(reach, scratch[i]);
  }
  // sequence (0 for the prefix), key head and first row of unit u: groups of
  // `group` (sequence, head)s; in a group the row pairs from the last, which
  // under the causal rule sees the most keys, each for every head
  auto unit_at = [&](int u, int& b, int& head, int& r0) {
    const int g = u / (p.part.group * p.part.pairs);
    const int in = u - g * p.part.group * p.part.pairs;
    const int hs = min(p.part.group, p.part.heads - g * p.part.group);
    const int level = in / hs;
    const int bh = g * p.part.group + in - level * hs;
    b = PREFIX ? 0 : bh / Hkv;
    head = bh - b * Hkv;
    r0 = (p.part.pairs - 1 - level) * kPairRows;
  };
  // keys (from the origin) that tiles A and B of a unit need
  auto unit_keys = [&](int b, int r0, int& ka, int& kb, int& limit) {
    if constexpr (PREFIX) {
      ka = limit = reach;
      kb = r0 + kRows < space ? reach : 0;
    } else {
      int lq, lk;
      seq_lens(p.seq, b, lq, lk);
      ka = tile_keys(r0, rows, p.seq.Nq, lq, lk, origin, p.causal);
      kb = tile_keys(r0 + kRows, rows, p.seq.Nq, lq, lk, origin, p.causal);
      limit = lk - origin;
    }
  };
  auto unit_tiles = [&](int u) {
    int b, head, r0, ka, kb, limit;
    unit_at(u, b, head, r0);
    unit_keys(b, r0, ka, kb, limit);
    return (max(ka, kb) + kRows - 1) / kRows;
  };
  const int cut = p.part.cut;  // units of the line
  auto cost = [&](int tiles) { return tiles > 0 ? tiles + p.part.piece_cost : 0; };
  if constexpr (PREFIX) {  // the same for every unit
    const int n = cost((reach + kRows - 1) / kRows);
    for (int i = threadIdx.x; i <= cut; i += kThreads) line[i] = i * n;
    __syncthreads();
  } else {
    build_line<kThreads>(line, scratch, cut, [&](int e) { return cost(unit_tiles(e)); });
  }
  const int total = line[cut];
  // Whole units instead of the line, where that ends as early or nearly so
  // (partial results and their merge are worth four tiles and an eighth): with
  // fewer than two units a CTA one from either end of their order, else all
  // drawn, if the last ones are light.  Prompts under the causal rule: 16 heads x
  // 4096 tokens 135 us on the line, 68 so; 8 heads x 8192 149 and 123; 16 heads x
  // 8192, drawn, 276 and 233.  4 chunks of 100 tokens over 1500 keys, 32 heads on 8,
  // are 27 us on the line and would be 34.
  bool whole_units = false;
  if constexpr (!PREFIX && !DUAL) {
    if (p.direct && p.part.piece_cost > 0) {  // (not with few units)
      const int ctas = gridDim.x, c = threadIdx.x;
      int last = 0;  // of one CTA: its two units, or the one that it may draw last
      if (cut == p.part.units) {
        const int u2 = 2 * ctas - 1 - c;
        if (c < ctas && c < cut) last = line[c + 1] - line[c] + (u2 < cut ? line[u2 + 1] - line[u2] : 0);
      } else if (c < ctas) {
        last = cost(unit_tiles(p.part.units - 1 - c));
      }
      last = __reduce_max_sync(0xffffffffu, last);
      __syncthreads();
      if (lane == 0) scratch[warp] = last;
      __syncthreads();
      for (int i = 0; i < kThreads / 32; ++i) last = max(last, scratch[i]);
      const int mean = total / ctas;
      whole_units = cut == p.part.units ? last <= mean + mean / 8 + 4 : last <= total / cut / 2;
    }
  }
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i <= cut; i += kThreads) p.line_out[i] = line[i];
    if (threadIdx.x == 0) {
      const Ranges ranges = make_ranges<PREFIX ? 0 : kEvenTiles>(total, gridDim.x, p.part.min_tiles);
      p.line_out[cut + 1] = whole_units ? kWholeUnits : ranges.base;
      p.line_out[cut + 2] = ranges.more;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto BAR = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  const WaitCtl wc{abort_flag, p.status, p.wait_limit_ns};
  // A row tile without keys in a piece, and the spare warps, wait while whole
  // pieces go by: their limit is longer.  The producer and the issuer notice a
  // stall within the limit itself and end all waits.
  const WaitCtl wc_idle{abort_flag, p.status, p.wait_limit_ns * 64};
  const volatile Piece* pieces = reinterpret_cast<const volatile Piece*>(smem + L::kPieceOff);
  static_assert(sizeof(Piece) == 44, "pieces lie 44 bytes apart");
  const volatile uint32_t* row_at = reinterpret_cast<const volatile uint32_t*>(smem + L::kRowOff);
  const volatile int* row_end = reinterpret_cast<const volatile int*>(smem + L::kRowOff + 2 * kPairRows * 4);
  constexpr uint32_t kNoRow = 0xffffffffu;
  // Every role but warp 11 calls this before its n-th piece, with all lanes of
  // its warp (false: none left, or a wait ran out), and piece_done behind it.
  auto next_piece = [&](uint32_t n, bool& ok) {
    ok = tile_wait(BAR(L::PIECE_FULL + (n & 1)), (n >> 1) & 1, wc_idle, SITE_TILE_PIECE, n);
    return ok && pieces[n & 1].na >= 0;
  };
  auto piece_done = [&](uint32_t n) { mbar_arrive_warp(BAR(L::PIECE_EMPTY + (n & 1))); };

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    regs_increase<Launch<FP8>::kSoftmaxRegs>();
    const int t = warp >> 2;
    const int r = ((warp & 3) << 5) + lane;  // row inside the tile == TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) << 5) << 16;
    const uint32_t tS = tmem + lane_off + static_cast<uint32_t>(t * 128);
    const uint32_t tO = tmem + lane_off + L::kColO + static_cast<uint32_t>(t * D);
    const float scale_log2 = p.scale_log2;
    uint32_t sn = 0, on = 0, on2 = 0;
    [[maybe_unused]] uint32_t qn = 0, base = 0;  // tiles of rows so far, and key tiles
    bool ok = true;
    for (uint32_t n = 0; next_piece(n, ok); ++n) {
      [[maybe_unused]] float grow = 1.f;  // what this row's scores are multiplied by
      if constexpr (FP8) {
        // this thread's row becomes two E4M3 numbers a value, in its place: at d =
        // 128 hi in the first 64 columns' block and lo in the second, at d = 64 side
        // by side
        const bool rows_in = (DUAL || t == 0 ? pieces[n & 1].na : pieces[n & 1].nb) > 0;
        float* shared_grow = reinterpret_cast<float*>(smem + L::kGrowOff);
        if (rows_in && (!DUAL || t == 0)) {
          ok = tile_wait(BAR(L::Q_RAW + t), qn & 1, wc_idle, SITE_TILE_CONVERT, n);
          if (!ok) break;
          const uint32_t qt = sbase + t * L::kTileBytes;
          const uint32_t stage = sbase + L::kStageOff + warp * 2048 + lane * 64;
          auto raw = [&](int c, uint32_t (&x)[4]) { ld_shared_v4(qt + (c >> 3) * 16384 + sw128(r, c & 7), x); };
          uint32_t top = 0;  // the largest magnitude's bits
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) {
            uint32_t x[4];
            raw(c, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max(top, max((x[i] << 16) & 0x7fffffffu, x[i] & 0x7fff0000u));
          }
          const uint32_t e = max(top >> 23, 8u);  // the exponent's field
          const float up = __uint_as_float((261u - e) << 23);
          grow = e == 255u ? CUDART_NAN_F : __uint_as_float((e - 7u) << 23);  // (an infinity or a NaN in the row)
          // 16 columns at a time: those of the first block in order and the second's
          // from behind, with the first block's lo set aside, so that nothing is
          // written where a value is still to be read
#pragma unroll 1
          for (int k = 0; k < D / 16; ++k) {
            const int c = k < 4 ? k : 11 - k;
            uint32_t x[8], hi[4], lo[4];
            raw(2 * c, *reinterpret_cast<uint32_t(*)[4]>(x));
            raw(2 * c + 1, *reinterpret_cast<uint32_t(*)[4]>(x + 4));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float v0 = __uint_as_float(x[2 * i] << 16) * up, v1 = __uint_as_float(x[2 * i] & 0xFFFF0000u) * up;
              const float v2 = __uint_as_float(x[2 * i + 1] << 16) * up;
              const float v3 = __uint_as_float(x[2 * i + 1] & 0xFFFF0000u) * up;
              hi[i] = pack_e4m3x4(v0, v1, v2, v3);
              float u[4];
              unpack_e4m3x4(hi[i], u);
              lo[i] = pack_e4m3x4(v0 - u[0], v1 - u[1], v2 - u[2], v3 - u[3]);
            }
            st_shared_v4(qt + sw128(r, c), hi[0], hi[1], hi[2], hi[3]);
            st_shared_v4(k < 4 ? stage + ((k ^ ((lane >> 1) & 3)) << 4) : qt + 16384 + sw128(r, c), lo[0], lo[1], lo[2],
                         lo[3]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t x[4];
            ld_shared_v4(stage + ((k ^ ((lane >> 1) & 3)) << 4), x);
            st_shared_v4(D == 128 ? qt + 16384 + sw128(r, k) : qt + sw128(r, 4 + k), x[0], x[1], x[2], x[3]);
          }
          if constexpr (DUAL) shared_grow[r] = grow;
          fence_proxy_async_smem();
          mbar_arrive_warp(BAR(L::Q_FULL + t));
        }
        if (DUAL && rows_in && t == 1) {
          ok = tile_wait(BAR(L::Q_FULL + 0), qn & 1, wc_idle, SITE_TILE_CONVERT, n);
          if (!ok) break;
          grow = shared_grow[r];
        }
        if (rows_in) ++qn;
      }
      ok = tile_wait(BAR(L::ROWS_FULL + (n & 1)), (n >> 1) & 1, wc_idle, SITE_TILE_PIECE, n);
      if (!ok) break;
      const int nt = t ? pieces[n & 1].nb : pieces[n & 1].na;
      // this row's visible keys from the tile's first, and how far its key
      // tiles are apart
      int lim0 = row_end[(n & 1) * kPairRows + t * kRows + r];
      constexpr int stride = DUAL ? 2 * kRows : kRows;
      // A row without a key here, or that does not exist, is computed as if it saw
      // all and dropped in the end: its masks would cost its warp more than a tenth
      // of a step, and a CTA whose piece ends in such rows would end last.  (Two
      // chunks of 1000 tokens, of 31 and a quarter row tiles, 319 us with the masks,
      // 290 so; in E4M3 377 and 341.)
      const bool sees = lim0 > 0;
      if (!sees) lim0 = INT_MAX / 2;
      float m_ref = 0.f, l = 0.f, dl = 0.f;
      if constexpr (FP8) {
        // A row tile may have no keys for many pieces' tiles and come here before the
        // scales of those tiles: their barriers, which have one bit of count, would
        // then let it through to the last ones in the same place.
        ok = tile_wait(BAR(L::BEGUN + (n & 1)), (n >> 1) & 1, wc_idle, SITE_TILE_CONVERT, n);
        if (!ok) break;
      }
      auto rescale = [&](float alpha) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(tO + 32 * c, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
          tmem_st32(tO + 32 * c, v);
        }
        tmem_st_wait();
      };
      for (int j = 0; j < nt; ++j) {
        [[maybe_unused]] const uint32_t at = base + (DUAL ? 2 * j + t : j);
        if constexpr (FP8) {  // (there before the scores are)
          ok = tile_wait(BAR(L::SCALES + at % kScaleTiles), (at / kScaleTiles) & 1, wc_idle, SITE_TILE_CONVERT, n);
          if (!ok) break;
        }
        ok = tile_wait(BAR(L::S_FULL + t), sn & 1, wc_idle, SITE_TILE_S, n);
        if (!ok) break;
        ++sn;
        tc_fence_after();
        const int lim = lim0 - j * stride;
        if constexpr (FP8) {
          const uint32_t scales = sbase + L::kScaleOff + at % kScaleTiles * kScales * 16;
          if (__any_sync(0xffffffffu, lim < kRows)) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t v[32];
              tmem_ld32(tS + 32 * c, v);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 32 * c + i < lim ? v[i] : 0xff800000u;  // -inf
              tmem_st32(tS + 32 * c, v);
            }
            tmem_st_wait();
          }
          // The scores are read twice, for the maximum and for the weights, 64 columns
          // at a time, in loops that stay rolled: with all 128 columns' instructions in
          // a row a tile's are more than the first instruction cache holds, and the
          // warps wait for them (two chunks of 1000 tokens, us: 415 with the scores in
          // registers, 377 so).
          float top = -CUDART_INF_F;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t v[64];
#pragma unroll
            for (int c = 0; c < 2; ++c) tmem_ld32(tS + 64 * h + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(v + 32 * c));
            tmem_ld_wait();
#pragma unroll
            for (int b = 0; b < kScales / 2; ++b) {
              auto x = [&](int i) { return __uint_as_float(v[kScaleTokens * b + i]); };
              const float t1 = fmax3(fmax3(x(0), x(1), x(2)), fmax3(x(3), x(4), x(5)), fmax3(x(6), x(7), x(8)));
              const float t2 = fmax3(fmax3(x(9), x(10), x(11)), fmax3(x(12), x(13), x(14)), x(15));
              const float2 k = ld_shared_f2(scales + 16 * (4 * h + b));
              top = fmaxf(top, fmaf(fmaxf(t1, t2), k.x * grow, k.y));  // (-inf * 0 is passed over)
            }
          }
          if (j == 0) {
            m_ref = fmaxf(top, kNoScore);  // (as below)
          } else {
            const bool need = top > m_ref + kTau;
            if (__any_sync(0xffffffffu, need)) {
              const float m_new = fmaxf(m_ref, top);
              const float alpha = ex2_approx(m_ref - m_new);
              m_ref = m_new;
              l *= alpha;
              rescale(alpha);
            }
          }
          const float add0 = kShift - m_ref;
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t x[64], pk[32];
            tmem_ld32(tS + 64 * c, *reinterpret_cast<uint32_t(*)[32]>(x));
            tmem_ld32(tS + 64 * c + 32, *reinterpret_cast<uint32_t(*)[32]>(x + 32));
            tmem_ld_wait();
#pragma unroll
            for (int b = 0; b < 4; ++b) {  // 16 columns of one scale each
              uint32_t k[4];
              ld_shared_v4(scales + 16 * (4 * c + b), k);
              // (not 0, for a masked score is -inf: the product underflows for a row of
              // zeros over a cell of the smallest scale; scores are below 2^26, so that
              // the least factor stands for 0 as well)
              const float mul = max_nan(__uint_as_float(k[0]) * grow, FLT_MIN), add = __uint_as_float(k[1]) + add0;
              const uint64_t c2 = f2_pack(mul, mul), n2 = f2_pack(add, add);
              uint64_t sum = f2_pack(0.f, 0.f);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float x0, x1;
                f2_unpack(ffma2(f2_pack(__uint_as_float(x[16 * b + 2 * i]), __uint_as_float(x[16 * b + 2 * i + 1])), c2,
                                n2),
                          x0, x1);
                const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                sum = fadd2(sum, f2_pack(p0, p1));
                pk[8 * b + i] = pack_f16x2(p0, p1);
              }
              float a0, a1;
              f2_unpack(sum, a0, a1);
              l = fmaf(a0 + a1, __uint_as_float(k[2]), l);
            }
            tmem_st32(tS + 32 * c, pk);
          }
        } else {
          float s[128];
          {
            uint32_t sr[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(sr + 32 * c));
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 128; ++c) s[c] = __uint_as_float(sr[c]);
          }
          if (__any_sync(0xffffffffu, lim < kRows)) {
#pragma unroll
            for (int c = 0; c < 128; ++c) s[c] = (c < lim) ? s[c] : -CUDART_INF_F;
          }
          // row maximum as a log-depth tree of 3-input max
          float t1[43];
#pragma unroll
          for (int c = 0; c < 42; ++c) t1[c] = fmax3(s[3 * c], s[3 * c + 1], s[3 * c + 2]);
          t1[42] = fmaxf(s[126], s[127]);
          float t2[15];
#pragma unroll
          for (int c = 0; c < 14; ++c) t2[c] = fmax3(t1[3 * c], t1[3 * c + 1], t1[3 * c + 2]);
          t2[14] = t1[42];
          float t3[5];
#pragma unroll
          for (int c = 0; c < 5; ++c) t3[c] = fmax3(t2[3 * c], t2[3 * c + 1], t2[3 * c + 2]);
          const float mt = fmaxf(fmax3(t3[0], t3[1], t3[2]), fmaxf(t3[3], t3[4])) * scale_log2;
          if (j == 0) {
            // -inf: the row sees a leading range of the piece's keys and so none
            // at all, or keys whose scores are -inf, behind which any other's
            // becomes the reference
            m_ref = fmaxf(mt, kNoScore);
          } else {
            const bool need = mt > m_ref + kTau;
            if (__any_sync(0xffffffffu, need)) {
              const float m_new = fmaxf(m_ref, mt);
              const float alpha = ex2_approx(m_ref - m_new);
              m_ref = m_new;
              l *= alpha;
              dl *= alpha;
              rescale(alpha);
            }
          }
          const uint64_t c2 = f2_pack(scale_log2, scale_log2);
          const uint64_t n2 = f2_pack(-m_ref, -m_ref);
          {
            // the tile's largest weight and its change by the rounding to bf16
            const float pmax = ex2_approx(mt - m_ref);
            dl += __uint_as_float(pack_bf16x2(pmax, 0.f) << 16) - pmax;
          }
          uint64_t acc0 = f2_pack(0.f, 0.f), acc1 = acc0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              float x0, x1, x2, x3;
              f2_unpack(ffma2(f2_pack(s[32 * c + 2 * i], s[32 * c + 2 * i + 1]), c2, n2), x0, x1);
              f2_unpack(ffma2(f2_pack(s[32 * c + 2 * i + 2], s[32 * c + 2 * i + 3]), c2, n2), x2, x3);
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1), p2 = ex2_approx(x2), p3 = ex2_approx(x3);
              acc0 = fadd2(acc0, f2_pack(p0, p1));
              acc1 = fadd2(acc1, f2_pack(p2, p3));
              pk[i] = pack_bf16x2(p0, p1);
              pk[i + 1] = pack_bf16x2(p2, p3);
            }
            tmem_st16(tS + 16 * c, pk);
          }
          float a0, a1, a2, a3;
          f2_unpack(acc0, a0, a1);
          f2_unpack(acc1, a2, a3);
          l += (a0 + a1) + (a2 + a3);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(BAR(L::P_FULL + t));
      }
      if (!ok) break;
      if constexpr (FP8) base += pieces[n & 1].tiles;
      if (nt > 0) {
        ok = tile_wait(BAR(L::O_FULL + t), on & 1, wc, SITE_TILE_O, n);
        if (!ok) break;
        ++on;
        tc_fence_after();
      }
      if (!sees) l = dl = 0.f;  // (dl too: +inf among what it does not see makes a NaN of it)
      // The row is acc_own * f_own + acc_other * f_other (a tile without keys
      // reads what was left in tensor memory, and drops it).  A sum is 0 only
      // where no key is seen; a NaN goes through.
      bool live = l != 0.f;
      float f_own = live ? 1.0f / (l + dl) : 0.f, f_other = 0.f;
      if constexpr (DUAL) {
        // the other row tile's warp has the same rows, in the same lanes of
        // tensor memory: each writes half of the columns of both together
        float* stat = reinterpret_cast<float*>(smem + L::kStatOff) + r;
        stat[t * 3 * kRows] = m_ref;
        stat[t * 3 * kRows + kRows] = l;
        stat[t * 3 * kRows + 2 * kRows] = dl;
        if ((t ? pieces[n & 1].na : pieces[n & 1].nb) > 0) {
          ok = tile_wait(BAR(L::O_FULL + 1 - t), on2 & 1, wc, SITE_TILE_O, n);
          if (!ok) break;
          ++on2;
        }
        mbar_arrive_warp(BAR(L::PAIR + (warp & 3)));
        ok = tile_wait(BAR(L::PAIR + (warp & 3)), n & 1, wc_idle, SITE_TILE_O, n);
        if (!ok) break;
        tc_fence_after();
        const float m2 = stat[(1 - t) * 3 * kRows], l2 = stat[(1 - t) * 3 * kRows + kRows];
        const float dl2 = stat[(1 - t) * 3 * kRows + 2 * kRows];
        const float m = l != 0.f ? (l2 != 0.f ? fmaxf(m_ref, m2) : m_ref) : m2;
        const float a = l != 0.f ? ex2_approx(m_ref - m) : 0.f, a2 = l2 != 0.f ? ex2_approx(m2 - m) : 0.f;
        live = live || l2 != 0.f;
        const float inv = live ? 1.0f / (a * (l + dl) + a2 * (l2 + dl2)) : 0.f;
        f_own = a * inv;
        f_other = a2 * inv;
        l = a * l + a2 * l2;
        m_ref = m;
      }
      // columns c0 .. c0 + N - 1 of the row
      auto columns = [&](int c0, auto& w) {
        constexpr int N = sizeof(w) / 4;
        auto fetch = [&](uint32_t from, uint32_t (&x)[N]) {
          if constexpr (N == 32)
            tmem_ld32(from + c0, x);
          else
            tmem_ld16(from + c0, x);
        };
        uint32_t x[N];
        [[maybe_unused]] uint32_t y[DUAL ? N : 1];
        fetch(tO, x);
        if constexpr (DUAL) fetch(tmem + lane_off + L::kColO + static_cast<uint32_t>((1 - t) * D), y);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < N; ++i) {
          w[i] = f_own != 0.f ? __uint_as_float(x[i]) * f_own : 0.f;
          if constexpr (DUAL) w[i] += f_other != 0.f ? __uint_as_float(y[i]) * f_other : 0.f;
        }
      };
      constexpr int kShare = DUAL ? 2 : 1;           // warps that write a row
      const int share = DUAL ? t : 0;
      const bool whole = pieces[n & 1].whole;
      const long long prow0 =
          static_cast<long long>(pieces[n & 1].slot) * kPairRows + (DUAL ? 0 : t * kRows) + (r - lane);
      const volatile uint32_t* at = row_at + (n & 1) * kPairRows + t * kRows + (r - lane);
      if (!whole) {
        // a partial result lies in runs of 16 bytes, a row group's 32 rows side
        // by side (PartRef), so a store is 512 bytes in one piece
        float4* dst = reinterpret_cast<float4*>(p.part.o + prow0 * D) + lane;
        const bool keep = at[lane] != kNoRow;
#pragma unroll 1
        for (int c = share * D / 32 / kShare; c < (share + 1) * D / 32 / kShare; ++c) {
          float w[32];
          columns(32 * c, w);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (keep) dst[(8 * c + i) * 32] = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
      } else {
        // rows leave through the warp's staging area, 64 bytes at a time: each
        // lane writes a run of its own row there, then the lanes take the runs
        // of eight rows at once
        const bool half = p.o_bf16;
        const uint32_t stage = sbase + L::kStageOff + warp * 2048;
        const uint32_t put = stage + lane * 64, put_x = (lane >> 1) & 3;
        const int from = lane >> 2, run = lane & 3;  // read: rows from, from + 8, ..., 16 bytes each
        uint8_t* dst[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t g = at[8 * k + from];
          dst[k] = g == kNoRow ? nullptr
                               : static_cast<uint8_t*>(p.o) + static_cast<size_t>(g) * D * (half ? 2 : 4) + 16 * run;
        }
        const int runs = (half ? D / 32 : D / 16) / kShare;
#pragma unroll 1
        for (int c = share * runs; c < (share + 1) * runs; ++c) {
          uint32_t w[16];
          if (half) {
            float v[32];
            columns(32 * c, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
          } else {
            float v[16];
            columns(16 * c, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[i]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            st_shared_v4(put + ((i ^ put_x) << 4), w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          __syncwarp();
          uint32_t x[4][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = 8 * k + from;
            ld_shared_v4(stage + row * 64 + ((run ^ ((row >> 1) & 3)) << 4), x[k]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (dst[k]) *reinterpret_cast<uint4*>(dst[k] + 64 * c) = make_uint4(x[k][0], x[k][1], x[k][2], x[k][3]);
          __syncwarp();
        }
      }
      const uint32_t mine = at[lane];
      if (share == 0 && mine != kNoRow) {
        const float lse2 = live ? m_ref - (FP8 ? kShift : 0.f) + log2f(l) : -CUDART_INF_F;
        if (whole)
          p.lse[mine] = live ? lse2 * kLn2 : -CUDART_INF_F;
        else
          p.part.lse[prow0 + lane] = lse2;
      }
      if constexpr (DUAL) {  // before the next product overwrites what the other warp reads
        tc_fence_before();
        mbar_arrive_warp(BAR(L::PAIR_DONE + (warp & 3)));
        ok = tile_wait(BAR(L::PAIR_DONE + (warp & 3)), n & 1, wc_idle, SITE_TILE_O, n);
        if (!ok) break;
        tc_fence_after();
      }
      piece_done(n);
    }
  } else {
    regs_decrease<Launch<FP8>::kOtherRegs>();
    if (warp == 8) {
      // -------------------------------------------------------- TMA producer
      const int boxes = kRows / p.box_rows;
      const int box = lane & (boxes - 1);  // this lane's load of a tile
      const bool loads = lane < boxes;
      const uint32_t offset = static_cast<uint32_t>(box * p.box_rows * (FP8 ? D : CB * 128));
      const uint64_t policy = l2_policy_evict_last();
      uint32_t kvpos = 0;
      [[maybe_unused]] uint32_t keys_issued = 0;
      bool ok = true;
      for (uint32_t n = 0; next_piece(n, ok); ++n) {
        const volatile Piece& x = pieces[n & 1];
        if (FP8 && lane == 0) mbar_arrive(BAR(L::BEGUN + (n & 1)));
        const int head = x.head, b = x.b, tiles = x.tiles;
        const int* pages = PREFIX ? p.prefix_table : p.table.block_table + b * p.table.table_stride;
        const int first = origin + x.tile * kRows;
        const int last = origin + x.limit;
        const int count = tiles * boxes;
        auto page_of = [&](int i) {
          const int key = first + i * p.box_rows;
          return i < count && key < last ? pages[key / p.table.page_size] : -1;
        };
        int cur = page_of(lane), next = page_of(32 + lane);
        // a lane's scale of a tile: of keys' groups of 16, then of values'; 0 for a
        // group of no page.  Loaded a tile ahead.
        const int group = lane % kScales;
        auto scale_of = [&](int j, int pages_of_32) {
          const int page = __shfl_sync(0xffffffffu, pages_of_32, (j * boxes + group * kScaleTokens / p.box_rows) % 32);
          const int key = first + j * kRows + group * kScaleTokens;
          if (lane >= 2 * kScales || j >= tiles || key >= last || page < 0 || page >= p.table.num_pages) return 0.f;
          const long long cell = (static_cast<long long>(page) * Hkv + head) * (p.table.page_size / kScaleTokens) +
                                 key % p.table.page_size / kScaleTokens;
          return (lane < kScales ? p.k_scales : p.v_scales)[cell];
        };
        [[maybe_unused]] float scale_ahead = 0.f;
        if constexpr (FP8) scale_ahead = scale_of(0, cur);
        const int tell = max(0, tiles - kTellTiles);
        for (int j = 0; j < tiles && ok; ++j) {
          if (j == tell && lane == 0) mbar_arrive(BAR(L::LOADED));
          if (j > 0 && (j * boxes) % 32 == 0) {
            cur = next;
            next = page_of(j * boxes + 32 + lane);
          }
          const int page = __shfl_sync(0xffffffffu, cur, (j * boxes + box) % 32);
          const int key = first + j * kRows + box * p.box_rows;
          int outer = p.table.num_pages * Hkv;  // past the map: zeros
          if (loads && key < last) {
            if (page >= 0 && page < p.table.num_pages)
              outer = page * Hkv + head;
            else
              record_bad_page(p.status, SITE_PAGE_READ, b, page);
          }
          const int row = key % p.table.page_size;
          if constexpr (FP8) {
            const float scale = scale_ahead;
            scale_ahead = scale_of(j + 1, (j + 1) * boxes % 32 == 0 ? next : cur);
            const bool skip = blockIdx.x == 0 && static_cast<int>(n) == p.stall_unit && j == 0;  // testing hook
            const uint32_t ks = kvpos % KSL, vs = kvpos % RSL;
            ok = tile_wait(BAR(L::K_EMPTY + ks), ((kvpos / KSL) & 1) ^ 1, wc, SITE_TILE_LOAD, n);
            if (!ok) break;
            ++keys_issued;
            if (!skip) {
              if (lane == 0) mbar_arrive_expect_tx(BAR(L::K_FULL + ks), L::kTileBytes / 2);
              __syncwarp();
              if (loads)
                tma_load_3d_hint(sbase + L::kKeyOff + ks * (L::kTileBytes / 2) + offset, &tm_k, BAR(L::K_FULL + ks), 0,
                                 row, outer, policy);
              __syncwarp();
            }
            float* scales = reinterpret_cast<float*>(smem + L::kScaleOff) + (kvpos % kScaleTiles * kScales + group) * 4;
            if (lane < kScales) {
              scales[0] = scale * p.scale_log2;
            } else if (lane < 2 * kScales) {
              // (the sum takes 2^-log2 of the same rounded logarithm, which drops out)
              const float log = scale != 0.f ? __log2f(scale) : 0.f;
              scales[1] = log;
              scales[2] = scale != 0.f ? ex2_approx(-log) : 0.f;
            }
            mbar_arrive_warp(BAR(L::SCALES + kvpos % kScaleTiles));
            ok = tile_wait(BAR(L::RAW_EMPTY + vs), ((kvpos / RSL) & 1) ^ 1, wc, SITE_TILE_LOAD, n);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(BAR(L::RAW_FULL + vs), L::kTileBytes / 2);
            __syncwarp();
            if (loads)
              tma_load_3d_hint(sbase + L::kRawOff + vs * (L::kTileBytes / 2) + offset, &tm_v, BAR(L::RAW_FULL + vs), 0,
                               row, outer, policy);
            ++kvpos;
          } else {
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {
              const uint32_t s = kvpos % S, use = kvpos / S;
              ok = tile_wait(BAR(L::KV_EMPTY + s), (use & 1) ^ 1, wc, SITE_TILE_LOAD, n);
              if (!ok) break;
              ++kvpos;
              if (blockIdx.x == 0 && static_cast<int>(n) == p.stall_unit && j == 0 && kv == 0)
                continue;  // testing hook: leave this tile unloaded
              if (lane == 0) mbar_arrive_expect_tx(BAR(L::KV_FULL + s), L::kTileBytes);
              __syncwarp();
              if (loads)
                tma_load_groups(sbase + L::kRingOff + s * L::kTileBytes + offset, kv == 0 ? &tm_k : &tm_v,
                                BAR(L::KV_FULL + s), row / 8, outer, policy);
              __syncwarp();
            }
          }
        }
        if (!ok) break;
        if (tell >= tiles && lane == 0) mbar_arrive(BAR(L::LOADED));
        piece_done(n);
      }
      if (FP8 && !ok && lane == 0) {
        auto drain = [&](int bar, uint32_t slots, uint32_t issued) {
          for (uint32_t s = 0; s < slots && s < issued; ++s)
            drain_wait(BAR(bar + s), ((issued - 1 - (issued - 1 - s) % slots) / slots) & 1, p.wait_limit_ns);
        };
        drain(L::K_FULL, KSL, keys_issued);
        drain(L::RAW_FULL, RSL, kvpos);
      } else if (!ok && lane == 0) {
        for (uint32_t s = 0; s < static_cast<uint32_t>(S); ++s) {
          if (kvpos > s) {
            const uint32_t last = kvpos - 1 - ((kvpos - 1 - s) % S);
            drain_wait(BAR(L::KV_FULL + s), (last / S) & 1, p.wait_limit_ns);
          }
        }
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------- MMA issuer
      {
        constexpr uint32_t id_s = FP8 ? idesc_e4m3_f32(128, 128) : idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t id_pv = FP8 ? idesc_f16_f32(128, D, false, true) : idesc_bf16_f32(128, D, false, true);
        const SDesc qdesc0 = sdesc_sw128(sbase, 16, 1024);
        // keys and values: groups of 8 rows, in a group its 64-column blocks; keys
        // in E4M3: rows of D bytes
        const SDesc kdesc0 = !FP8 ? sdesc_sw128(sbase + L::kRingOff, 16, CB * 1024)
                             : D == 128 ? sdesc_sw128(sbase + L::kKeyOff, 16, 1024)
                                        : sdesc_sw64(sbase + L::kKeyOff, 16, 512);
        const SDesc vdesc0 = sdesc_sw128(sbase + L::kRingOff, 1024, CB * 1024);
        constexpr uint32_t kTileUnits = L::kTileBytes >> 4;
        auto issue_s = [&](int t, uint32_t slot) {
          SDesc qd = qdesc0 + static_cast<uint32_t>(DUAL ? 0 : t) * kTileUnits;
          SDesc kd = kdesc0 + slot * (FP8 ? kTileUnits / 2 : kTileUnits);
          // (each step's own descriptors are an addition here, not registers kept
          // for all steps of both tiles, of which there are too few)
          if constexpr (FP8) asm volatile("" : "+r"(qd.lo), "+r"(kd.lo));
          if constexpr (FP8) {
#pragma unroll
            for (int part = 0; part < 2; ++part)  // hi, lo
#pragma unroll
              for (int ks = 0; ks < D / 32; ++ks)
                umma_ss_f8(tmem + static_cast<uint32_t>(t * 128),
                           qd + static_cast<uint32_t>((part * (D == 128 ? 16384 : 64) + ks * 32) >> 4),
                           kd + static_cast<uint32_t>((ks * 32) >> 4), id_s, part + ks > 0 ? 1u : 0u);
          } else {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t q_off = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
              const uint32_t k_off = ((ks >> 2) * 1024 + (ks & 3) * 32) >> 4;
              umma_ss(tmem + static_cast<uint32_t>(t * 128), qd + q_off, kd + k_off, id_s, ks > 0 ? 1u : 0u);
            }
          }
        };
        auto issue_pv = [&](int t, uint32_t slot, bool acc) {
          SDesc vd = vdesc0 + slot * kTileUnits;
          if constexpr (FP8) asm volatile("" : "+r"(vd.lo));
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            umma_ts(tmem + L::kColO + static_cast<uint32_t>(t * D), tmem + static_cast<uint32_t>(t * 128 + ks * 8),
                    vd + static_cast<uint32_t>((ks * CB * 2048) >> 4), id_pv, (acc || ks > 0) ? 1u : 0u);
          }
        };
        // Where key tile j's keys and values are: place in their rings from the
        // first tile on, and the rings' barriers.
        constexpr int kStep = FP8 ? 1 : 2, kValues = FP8 ? 0 : 1;
        constexpr uint32_t KS = FP8 ? KSL : S, VS = FP8 ? VSL : S;
        constexpr int kKeysFull = FP8 ? L::K_FULL : L::KV_FULL, kKeysEmpty = FP8 ? L::K_EMPTY : L::KV_EMPTY;
        constexpr int kValuesFull = FP8 ? L::V_FULL : L::KV_FULL, kValuesEmpty = FP8 ? L::V_EMPTY : L::KV_EMPTY;
        uint32_t qa = 0, qb = 0, kvbase = 0, pa = 0, pb = 0, cleaned = 0;
        bool ok = true;
        for (uint32_t n = 0; next_piece(n, ok); ++n) {
          const int unit = static_cast<int>(n);
          const int na = pieces[n & 1].na, nb = pieces[n & 1].nb, clean = FP8 ? -1 : pieces[n & 1].clean;
          const int tiles = pieces[n & 1].tiles;
          auto arrived = [&](int bar, uint32_t phase) {
            return wait_bounded(BAR(bar), phase & 1, wc, SITE_TILE_MMA, unit);
          };
          // all of a piece, by one thread
          auto issue_piece = [&]() -> bool {
            if constexpr (DUAL) {
              // key tile j belongs to row tile j & 1, whose chain S -> softmax ->
              // P V -> next S runs beside the other's
              auto start = [&](int t, int j) -> bool {
                const uint32_t kpos = kvbase + kStep * j;
                if (!arrived(kKeysFull + kpos % KS, kpos / KS)) return false;
                tc_fence_after();
                issue_s(t, kpos % KS);
                umma_commit(BAR(L::S_FULL + t));
                umma_commit(BAR(kKeysEmpty + kpos % KS));
                if (j + 1 == tiles) umma_commit(BAR(L::Q_EMPTY + 0));  // the piece's last use of Q
                return true;
              };
              if (na > 0) {
                if (!arrived(L::Q_FULL + 0, qa) || !start(0, 0)) return false;
                ++qa;
              }
              if (nb > 0 && !start(1, 1)) return false;
              for (int j = 0; j < tiles; ++j) {
                const int t = j & 1;
                const uint32_t vpos = kvbase + kStep * j + kValues;
                if (!arrived(kValuesFull + vpos % VS, vpos / VS)) return false;
                if (j == clean) mbar_arrive(BAR(L::DIRTY));
                if (!arrived(L::P_FULL + t, t ? pb : pa)) return false;
                if (t) ++pb; else ++pa;
                if (j == clean) {
                  if (!wait_bounded(BAR(L::CLEAN), cleaned & 1, wc, SITE_TILE_CLEAN, unit)) return false;
                  ++cleaned;
                }
                tc_fence_after();
                issue_pv(t, vpos % VS, j > 1);
                if (j + 2 >= tiles) umma_commit(BAR(L::O_FULL + t));
                umma_commit(BAR(kValuesEmpty + vpos % VS));
                if (j + 2 < tiles && !start(t, j + 2)) return false;
              }
            } else {
              if (tiles > 0) {
                if (!arrived(kKeysFull + kvbase % KS, kvbase / KS)) return false;
                if (na > 0) {
                  if (!arrived(L::Q_FULL + 0, qa)) return false;
                  ++qa;
                  tc_fence_after();
                  issue_s(0, kvbase % KS);
                  umma_commit(BAR(L::S_FULL + 0));
                  if (na == 1) umma_commit(BAR(L::Q_EMPTY + 0));  // the piece's last use of Q
                }
                if (nb > 0) {
                  if (!arrived(L::Q_FULL + 1, qb)) return false;
                  ++qb;
                  // (behind tile A's first weights, so that the two softmaxes begin
                  // half a step apart: two chunks of 1000 tokens 382 us without, 374)
                  if (FP8 && na > 0 && !arrived(L::P_FULL + 0, pa)) return false;
                  tc_fence_after();
                  issue_s(1, kvbase % KS);
                  umma_commit(BAR(L::S_FULL + 1));
                  if (nb == 1) umma_commit(BAR(L::Q_EMPTY + 1));
                }
              }
              // One key tile.  STEADY: both row tiles have it and two more, and its
              // values need no zeroing: all but the last steps of most pieces.
              // Nothing is decided in such a step, since this thread's
              // instructions are on every step's critical path.
              auto step = [&](auto steady_tag, int j) -> bool {
                constexpr bool STEADY = decltype(steady_tag)::value;
                const uint32_t kpos = kvbase + kStep * j, vpos = kpos + kValues, knext = kpos + kStep;
                const bool has_a = STEADY || j < na, next_a = STEADY || j + 1 < na;
                const bool has_b = STEADY || j < nb, next_b = STEADY || j + 1 < nb;
                const bool dirty = !STEADY && j == clean;
                umma_commit(BAR(kKeysEmpty + kpos % KS));  // K_j is free once S(j) of both tiles completes
                if (!arrived(kValuesFull + vpos % VS, vpos / VS)) return false;
                // the last keys' values: zeroed behind the last key by warp 10
                // while the softmax of this tile runs
                if (dirty) mbar_arrive(BAR(L::DIRTY));
                auto values_ready = [&]() {
                  return !dirty || wait_bounded(BAR(L::CLEAN), cleaned & 1, wc, SITE_TILE_CLEAN, unit);
                };
                if (has_a) {
                  if (!arrived(L::P_FULL + 0, pa) || !values_ready()) return false;
                  ++pa;
                  tc_fence_after();
                  issue_pv(0, vpos % VS, j > 0);
                  if (!next_a) umma_commit(BAR(L::O_FULL + 0));
                  if (next_a) {
                    if (!arrived(kKeysFull + knext % KS, knext / KS)) return false;
                    tc_fence_after();
                    issue_s(0, knext % KS);
                    umma_commit(BAR(L::S_FULL + 0));
                    if (!STEADY && j + 2 == na) umma_commit(BAR(L::Q_EMPTY + 0));
                  }
                }
                if (has_b) {
                  if (!arrived(L::P_FULL + 1, pb) || !values_ready()) return false;
                  ++pb;
                  tc_fence_after();
                  issue_pv(1, vpos % VS, j > 0);
                  if (!next_b) umma_commit(BAR(L::O_FULL + 1));
                }
                if (dirty) ++cleaned;
                umma_commit(BAR(kValuesEmpty + vpos % VS));  // V_j is free once PV(j) of both tiles completes
                if (next_b) {
                  if (!(has_a && next_a)) {  // otherwise tile A's S(j+1) already waited for K_{j+1}
                    if (!arrived(kKeysFull + knext % KS, knext / KS)) return false;
                    tc_fence_after();
                  }
                  issue_s(1, knext % KS);
                  umma_commit(BAR(L::S_FULL + 1));
                  if (!STEADY && j + 2 == nb) umma_commit(BAR(L::Q_EMPTY + 1));
                }
                return true;
              };
              const int steady = min(na, nb) - 2;
              for (int j = 0; j < tiles; ++j)
                if (!(j < steady && j != clean ? step(std::true_type{}, j) : step(std::false_type{}, j))) return false;
            }
            return true;
          };
          if (lane == 0) ok = issue_piece();
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          kvbase += kStep * tiles;
          piece_done(n);
        }
        // every MMA this thread issued completes before tensor memory is freed
        if (lane == 0) {
          umma_commit(BAR(L::DRAIN));
          drain_wait(BAR(L::DRAIN), 0, p.wait_limit_ns);
        }
      }
    } else if (warp == 10) {
      // ------------------------------ rows in, and values behind the last key
      volatile uint32_t* at_w = const_cast<volatile uint32_t*>(row_at);
      volatile int* end_w = const_cast<volatile int*>(row_end);
      uint32_t kvbase = 0, cleaned = 0, qn[2] = {0, 0};
      bool ok = true;
      for (uint32_t n = 0; next_piece(n, ok); ++n) {
        const volatile Piece& x = pieces[n & 1];
        const int r0 = x.r0, head = x.head, tile0 = x.tile * kRows, clean = FP8 ? -1 : x.clean, limit = x.limit;
        const int nt[2] = {x.na, DUAL ? 0 : x.nb};  // key tiles of what each tile of rows is for
        const int buf = (n & 1) * kPairRows;
        // a sequence's rows of a key head lie together (rows of the tile behind
        // the last are the next head's, and see no key), the prefix's rows in
        // as many runs as it has sequences: boxes where those divide 128 rows,
        // gathered row by row where not
        const bool boxed = !PREFIX || p.boxed_rows;
        if (boxed) {
          for (int t = 0; t < 2; ++t) {
            if (nt[t] == 0) continue;
            ok = tile_wait(BAR(L::Q_EMPTY + t), (qn[t] & 1) ^ 1, wc_idle, SITE_TILE_PIECE, n);
            if (!ok) break;
            ++qn[t];
            if (lane == 0) {
              mbar_arrive_expect_tx(BAR(L::Q_IN + t), L::kTileBytes);
              const int row = r0 + (DUAL ? 0 : t * kRows);
#pragma unroll
              for (int c = 0; c < CB; ++c) {
                const uint32_t dst = sbase + t * L::kTileBytes + c * 16384;
                if constexpr (PREFIX)
                  tma_load_4d(dst, &tm_q, BAR(L::Q_IN + t), c * 64, row % rows, head, row / rows);
                else
                  tma_load_3d(dst, &tm_q, BAR(L::Q_IN + t), c * 64, (x.b * Hkv + head) * rows + row, 0);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
        }
        constexpr int RL = kPairRows / 32;  // rows a lane
        auto row_of = [&](int i) { return DUAL ? i & (kRows - 1) : i; };
        int lq[RL], lk[RL], rb[RL];
        const int xb = x.b;
#pragma unroll
        for (int k = 0; k < RL; ++k) {  // all the lengths' loads in flight at once
          rb[k] = PREFIX ? min((r0 + row_of(32 * k + lane)) / rows, p.seq.B - 1) : xb;
          seq_lens(p.seq, rb[k], lq[k], lk[k]);
        }
#pragma unroll
        for (int k = 0; k < RL; ++k) {
          const int i = 32 * k + lane, row = r0 + row_of(i);
          const int rr = PREFIX ? row - rb[k] * rows : row;
          at_w[buf + i] = row < space ? (static_cast<uint32_t>(rb[k]) * Hkv + head) * rows + rr : kNoRow;
        }
        __syncwarp();
        if (PREFIX && !boxed) {
          constexpr int LPR = D / 8;     // lanes a row, 16 bytes each
          const int chunk = lane % LPR;
          for (int t = 0; t < 2; ++t) {
            if (nt[t] > 0) {
              ok = tile_wait(BAR(L::Q_EMPTY + t), (qn[t] & 1) ^ 1, wc_idle, SITE_TILE_PIECE, n);
              if (!ok) break;
              ++qn[t];
              const uint32_t qt = sbase + t * L::kTileBytes + (chunk >> 3) * 16384;
              constexpr int RPI = 32 / LPR, IN = FP8 ? 8 : 16;  // rows an instruction, instructions looked up at once
#pragma unroll 1
              for (int i0 = lane / LPR; i0 < kRows; i0 += RPI * IN) {
                uint32_t at[IN];
#pragma unroll
                for (int k = 0; k < IN; ++k) at[k] = row_at[buf + t * kRows + i0 + RPI * k];
#pragma unroll
                for (int k = 0; k < IN; ++k) {
                  const bool live = at[k] != kNoRow;
                  cp_async16(qt + sw128(i0 + RPI * k, chunk & 7),
                             p.q + (live ? static_cast<size_t>(at[k]) * D : 0) + chunk * 8, live ? 16u : 0u);
                }
              }
            }
            cp_async_commit();
          }
        }
        // the rows' last keys, while their values arrive
        if (ok) {
#pragma unroll
          for (int k = 0; k < RL; ++k) {
            const int i = 32 * k + lane, row = r0 + row_of(i);
            const int qi = (PREFIX ? row - rb[k] * rows : row) % p.seq.Nq;
            int end = 0;
            if (row < space && qi < lq[k]) end = (p.causal ? min(qi + lk[k] - lq[k] + 1, lk[k]) : lk[k]) - origin;
            if (PREFIX) end = min(end, p.seq.prefix_len);
            end_w[buf + i] = end - tile0 - (DUAL ? i & kRows : 0);  // tile B of two begins a key tile later
          }
          mbar_arrive_warp(BAR(L::ROWS_FULL + (n & 1)));
        }
        if (PREFIX && !boxed) {
          if (!ok) {
            cp_async_wait<0>();
            break;
          }
          // tile A's rows may go while tile B's arrive
          cp_async_wait<1>();
          fence_proxy_async_smem();
          if (nt[0] > 0) mbar_arrive_warp(BAR(L::Q_IN + 0));
          cp_async_wait<0>();
          fence_proxy_async_smem();
          if (nt[1] > 0) mbar_arrive_warp(BAR(L::Q_IN + 1));
        }
        if (!FP8 && clean >= 0) {
          const uint32_t vpos = kvbase + 2u * static_cast<uint32_t>(clean) + 1;
          ok = tile_wait(BAR(L::DIRTY), cleaned & 1, wc_idle, SITE_TILE_CLEAN, n);
          if (!ok) break;
          // the rest of the last key's box; whole boxes behind it were read as zeros
          const int from = limit % kRows, rest = p.box_rows - from % p.box_rows;
          const uint32_t vt = sbase + L::kRingOff + (vpos % S) * L::kTileBytes;
          for (int i = lane; i < rest * (D / 8); i += 32) {
            const int row = from + i / (D / 8), c = i % (D / 8);
            st_shared_v4(vt + ((row >> 3) * CB + (c >> 3)) * 1024 + sw128(row & 7, c & 7), 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          mbar_arrive_warp(BAR(L::CLEAN));
          ++cleaned;
        }
        kvbase += 2 * x.tiles;
        piece_done(n);
      }
      if ((!PREFIX || p.boxed_rows) && !ok && lane == 0) {
        // let the copies already issued land before the CTA can exit
        for (int t = 0; t < 2; ++t)
          if (qn[t] > 0) drain_wait(BAR(L::Q_IN + t), (qn[t] - 1) & 1, p.wait_limit_ns);
      }
    } else if (FP8 && warp >= 12) {
      // ------------------------------------------------- values become fp16
      uint32_t pos = 0;
      const int sub = warp == 12 ? 0 : warp - 13;
      bool ok = true;
      for (uint32_t n = 0; warp != 13 && next_piece(n, ok); ++n) {
        const int tiles = pieces[n & 1].tiles;
        const int limit = pieces[n & 1].limit - pieces[n & 1].tile * kRows;  // keys from the piece's first on
        for (int j = 0; j < tiles; ++j, ++pos) {
          const uint32_t rs = pos % RSL, vs = pos % VSL;
          ok = tile_wait(BAR(L::V_EMPTY + vs), ((pos / VSL) & 1) ^ 1, wc_idle, SITE_TILE_CONVERT, n) &&
               tile_wait(BAR(L::RAW_FULL + rs), (pos / RSL) & 1, wc_idle, SITE_TILE_CONVERT, n);
          if (!ok) break;
          const uint32_t src = sbase + L::kRawOff + rs * (L::kTileBytes / 2);
          const uint32_t dst = sbase + L::kRingOff + vs * L::kTileBytes;
          const int left = limit - j * kRows;  // rows behind the last key may hold anything
          constexpr int CHUNKS = D / 16;         // 16-byte chunks of a row
          constexpr int ITEMS = kRows * CHUNKS / 32, AT_ONCE = 4;
          // an item is four chunks of eight rows: eight lanes take a chunk of eight
          // rows, which lie in different banks on both sides
#pragma unroll 1
          for (int i0 = sub; i0 < ITEMS; i0 += kConverters * AT_ONCE) {
            uint32_t x[AT_ONCE][4];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
              const int item = i0 + i * kConverters;
              const int row = item / (CHUNKS / 4) * 8 + (lane & 7), c = item % (CHUNKS / 4) * 4 + (lane >> 3);
              if (item < ITEMS) ld_shared_v4(src + byte_chunk<D>(row, c), x[i]);
            }
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
              const int item = i0 + i * kConverters;
              if (item >= ITEMS) break;
              const int row = item / (CHUNKS / 4) * 8 + (lane & 7), c = (item % (CHUNKS / 4) * 4 + (lane >> 3)) * 2;
              const bool live = row < left;
              uint32_t h[8];
#pragma unroll
              for (int k = 0; k < 4; ++k) e4m3x4_to_f16(live ? x[i][k] : 0u, h[2 * k], h[2 * k + 1]);
              const uint32_t at = dst + ((row >> 3) * CB + (c >> 3)) * 1024;
              st_shared_v4(at + sw128(row & 7, c & 7), h[0], h[1], h[2], h[3]);
              st_shared_v4(at + sw128(row & 7, (c & 7) + 1), h[4], h[5], h[6], h[7]);
            }
          }
          mbar_arrive_warp(BAR(L::RAW_EMPTY + rs));
          fence_proxy_async_smem();
          mbar_arrive_warp(BAR(L::V_FULL + vs));
        }
        if (!ok) break;
        piece_done(n);
      }
    } else {
      // ------------------------------------------------------------- pieces
      const Ranges ranges = make_ranges<PREFIX ? 0 : kEvenTiles>(total, gridDim.x, p.part.min_tiles);
      const int at0 = range_start(ranges, blockIdx.x), stop = range_start(ranges, blockIdx.x + 1);
      int at = at0;  // on the line; then units are drawn
      for (uint32_t n = 0;; ++n) {
        if (!tile_wait(BAR(L::PIECE_EMPTY + (n & 1)), ((n >> 1) & 1) ^ 1, wc_idle, SITE_TILE_PIECE, n)) break;
        int u = -1, len = 0;
        Piece x{};
        x.na = -1;
        while (!whole_units && at < stop && len == 0) {
          // the last unit that starts at or before this place (one with tiles:
          // an empty one starts where its successor does)
          int lo = 0, hi = cut - 1;
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (line[mid] <= at) lo = mid; else hi = mid - 1;
          }
          u = lo;
          const int in = at - line[lo], out = min(line[lo + 1], stop) - line[lo];
          const int tiles = line[lo + 1] - line[lo] - p.part.piece_cost;
          x.tile = min(in, tiles);
          len = min(out, tiles) - x.tile;  // 0: the range begins behind the unit's last tile
          x.whole = p.direct && len == tiles;
          x.slot = p.part.two_a_cta ? 2 * blockIdx.x + (x.tile > 0 ? 0 : 1) : u + blockIdx.x;
          at += out - in;
        }
        if (len == 0) {
          u = -1;
          if (whole_units && cut == p.part.units) {
            if (n < 2) u = n == 0 ? blockIdx.x : 2 * gridDim.x - 1 - blockIdx.x;
          } else if (cut < p.part.units) {
            // as late as the next piece can be begun without a pause: when the
            // last one's tiles are on their way
            if (n > 0 && !tile_wait(BAR(L::LOADED), (n - 1) & 1, wc_idle, SITE_TILE_PIECE, n)) break;
            if (lane == 0) u = (whole_units ? 0 : cut) + atomicAdd(p.counter, 1);
            u = __shfl_sync(0xffffffffu, u, 0);
          }
          if (u >= p.part.units) u = -1;
          if (u >= 0) {
            len = unit_tiles(u);
            x.tile = 0;
            x.whole = p.direct;
            x.slot = u + gridDim.x;
          }
        }
        if (u >= 0) {
          int ka, kb;
          unit_at(u, x.b, x.head, x.r0);
          unit_keys(x.b, x.r0, ka, kb, x.limit);
          x.na = max(0, min((ka + kRows - 1) / kRows - x.tile, len));
          x.nb = max(0, min((kb + kRows - 1) / kRows - x.tile, len));
          x.tiles = max(x.na, x.nb);
          if constexpr (DUAL) {
            x.nb = x.tiles / 2;
            x.na = x.tiles - x.nb;
          }
          const int at_tile = x.limit / kRows - x.tile;
          x.clean = x.limit % p.box_rows != 0 && at_tile >= 0 && at_tile < x.tiles ? at_tile : -1;
        }
        if (lane == 0) *reinterpret_cast<Piece*>(smem + L::kPieceOff + (n & 1) * sizeof(Piece)) = x;
        mbar_arrive_warp(BAR(L::PIECE_FULL + (n & 1)));
        if (u < 0) break;
      }
    }
  }

  if (!p.wait_first && threadIdx.x == 0) grid_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool PREFIX, bool DUAL, bool FP8>
cudaError_t launch_t(const PagedTiles& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                     int ctas, cudaStream_t stream) {
  using L = TileLayout<D, DUAL, FP8>;
  auto kern = paged_tiles_kernel<D, PREFIX, DUAL, FP8>;
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = setup_kernel_once(kern, L::kSmemBytes, Launch<FP8>::kRegs, ready);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kern, dim3(ctas), Launch<FP8>::kThreads, L::kSmemBytes, stream, tm_q, tm_k, tm_v, p);
}

template <bool FP8>
cudaError_t launch_any(const PagedTiles& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                       int d, int ctas, cudaStream_t stream) {
  auto launch = [&](auto prefix, auto dual) {
    return d == 64 ? launch_t<64, prefix.value, dual.value, FP8>(p, tm_q, tm_k, tm_v, ctas, stream)
                   : launch_t<128, prefix.value, dual.value, FP8>(p, tm_q, tm_k, tm_v, ctas, stream);
  };
  const std::true_type yes;
  const std::false_type no;
  if (p.prefix_table) return p.part.dual ? launch(yes, yes) : launch(yes, no);
  return p.part.dual ? launch(no, yes) : launch(no, no);
}

}  // namespace
}  // namespace fa
