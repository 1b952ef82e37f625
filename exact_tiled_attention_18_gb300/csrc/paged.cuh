// What the kernels of attention over the paged cache share: the sequences'
// lengths on the device, the line of key tiles, the partial results.
#pragma once

#include <cuda_runtime.h>

#include "serving.h"

namespace fa {

// Rows a key head that the step kernel takes; more are the tile kernel's, which
// takes 128 whether they are there or not.  (8 heads; here and there, us.  8
// sequences x 8192 keys: 24 rows 55 and 57, 32 rows 62 and 57; 64 x 1000 keys: 57
// and 77, 65 and 77; 38 x 512 keys: 18 and 29, 21 and 30.  64 rows are 58, 79
// and 29 there.)
constexpr int kStepRows = 32;
constexpr int kLineSequences = 256;    // sequences a launch of the step kernel: the line's table is in shared memory
constexpr int kLineWords = 528;        // 4-byte words of a line in the workspace, a multiple of 4
constexpr int kMaxCtas = 512;
// Key tiles a CTA takes at least.  Step kernel (64 keys): 1000 keys of 8 key
// heads 6.9 us with 1, 7.3 with 2, 8.5 with 4.  Tile kernel (128 keys): 64 rows
// of 8 heads on 8, 512 keys 15.0 / 15.5 / 16.8 us with 1 / 2 / 4, 4096 keys
// 18.1 / 17.4 / 19.0, 64 sequences behind a prefix of 1024 keys 30.3 / 27.2 / 29.8.
constexpr int kMinSteps = 1, kMinTiles = 2;
constexpr int kEvenSteps = 2, kEvenTiles = 8;  // (make_ranges)
// A piece's beginning and end in the tile kernel, in key tiles, where there are
// units enough for a CTA to have several.
constexpr int kTilePieceCost = 2;
constexpr int kWholeUnits = -1;     // in the place of the ranges' base: no unit has been cut
constexpr int kMaxTileCtas = 160;
constexpr int kTileLine = 2 * kMaxTileCtas;  // units of the tile kernel's line
constexpr int kPairRows = 256;         // query rows a unit of the tile kernel: two 128-row tiles
static_assert(kLineWords >= kLineSequences + 3 && kLineWords >= kTileLine + 4, "the line's room");
static_assert(kLineWords % 4 == 0, "what lies behind it is read 16 bytes at a time");

struct PagedSeq {
  const int *seqlens_q, *seqlens_k;
  int B, Hkv, G, Nq;
  int capacity;     // positions that the table reaches
  int prefix_len;   // keys that are not these tiles' work
};

// Partial results of units (the step kernel: a sequence's keys of one key
// head; the tile kernel: 256 rows of one) that CTAs cut out of a line of key
// tiles.  Unit u's piece of CTA c is in slot u + c, which no other piece has
// (units from `cut` on are whole and in slot u + ctas); with two_a_cta, where
// only a CTA's first and last pieces of the line are partial, in slot 2 c (one
// that goes on from the CTA before) or 2 c + 1.
//
// A unit of the tile kernel ends on the line with piece_cost places that hold
// no tile: what the beginning and the end of a piece cost.
//
// A row of the step kernel's is d floats in one run.  The tile kernel writes a
// row a lane, so its 32 rows of a warp lie as [d / 4][32 rows][4]: every store
// is then 512 bytes in one piece, and so is every load of a merge that takes a
// row a lane.
struct PartRef {
  const int* line;     // first tile of every unit before `cut` (the step kernel: of its `cut` sequences, a head),
                       // their sum, then the ranges' base and more
  int ctas, min_tiles;
  int cut;
  int two_a_cta;
  int piece_cost;
  int slot_rows;
  // 1: a unit of the tile kernel has at most 128 rows, so that its tile B would
  // be empty: tile B takes the same rows and every other key tile, and the two
  // are put together in the CTA.  (64 rows of 8 heads: 8 sequences x 8192 keys
  // 58 us, 63 with tile A alone, at d = 64 42 and 56; 64 sequences x 1000 keys 79
  // and 98.)
  int dual;
  int units;
  int heads, pairs, group;  // the tile kernel: (sequence, head)s, row pairs of each, heads dealt out together
  float *o, *lse;      // [slot] of slot_rows rows of d; [slot][slot_rows] (log2 units)
};

struct PagedStep {
  PagedSeq seq;
  PageTable table;
  const uint16_t* q;
  void* o;
  int o_bf16;
  float* lse;
  int* line_out;     // the line's table, for the merge
  PartRef part;
  int direct;        // 1: a piece that is a whole unit's writes o and lse
  int wait_first;    // 1: wait for the kernels before this one at the start; 0: before the end
  int box_rows;
  int b0;            // first sequence of this launch, for error reports
  int causal;
  float scale_log2;
  int* status;
  unsigned long long wait_limit_ns;
  int stall_unit;
};

// The tile kernel: units are 256 rows of a key head, of one sequence or (the
// shared prefix) of all sequences' rows together.
struct PagedTiles {
  PagedSeq seq;
  PageTable table;
  const int* prefix_table;
  const uint16_t* q;
  void* o;
  int o_bf16;
  float* lse;
  int* line_out;     // the line's table, for the merge
  PartRef part;
  int direct;
  int boxed_rows;    // tiles of rows come by TMA (always but for some prefixes)
  int* counter;      // draws units from part.cut on; zero at the start
  int wait_first;    // as PagedStep's
  int box_rows;
  int causal;
  float scale_log2;
  int* status;
  unsigned long long wait_limit_ns;
  int stall_unit;
};

struct PagedCombine {
  PagedSeq seq;
  PartRef part;      // the sequences' own keys
  PartRef prefix;    // the shared prefix (o null: none)
  int direct;
  int units;         // units to merge: those behind them are written already
  int b0;            // sequences before this launch's first (rows of the prefix)
  void* o;
  int o_bf16;
  float* lse;
};

cudaError_t launch_tiles(const PagedTiles& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                         const CUtensorMap& tm_v, int d, int ctas, cudaStream_t stream);

#if defined(__CUDACC__)
// 4-D form of tma_load_3d (ptx.cuh).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                            int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// 16 bytes global -> shared without registers; `bytes` 0 writes zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Until at most N of this thread's committed groups are in flight.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// The larger of two, NaN if either is: row statistics of partial results carry
// a NaN score into the row, whichever of its pieces met it.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ void seq_lens(const PagedSeq& s, int b, int& lq, int& lk) {
  paged_lens(s.seqlens_q, s.seqlens_k, b, s.Nq, s.capacity, lq, lk);
}

// Byte offset of 16-byte chunk c of row r inside a 128-byte-swizzled box
// (the chunk index is XORed with the row index modulo 8).
__device__ __forceinline__ uint32_t sw128(int r, int c) {
  return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
}

// The line's tiles in equal ranges, one a CTA (the first `more` CTAs have one
// tile more than `base`), for no more CTAs than leave each `least` tiles and,
// where the longest range has at most EVEN tiles, for no more than ranges of
// that length need: as quick, with fewer partial results, and units more often
// cut into equal parts.  (One sequence of 30000 keys, one key head, 469 tiles
// for 456 CTAs: 14.6 us without, 10.4 with it; 4 chunks of 100 tokens over 1500
// keys, 32 heads on 8: 33.4 and 28.1 us.  The shared prefix's tiles do
// without, for CTAs that end early make room for the step kernel's: 24 sequences
// of 4 drafted tokens behind 8208 keys 30.0 us, 30.5 with it; single tokens of 16
// behind 4096 21.3 and 21.7, of 64 behind 8192 45 and 47, of 128 behind 16384 107
// either way.)
struct Ranges {
  int base, more, total;
};

template <int EVEN>
__device__ __forceinline__ Ranges make_ranges(int total, int ctas, int least) {
  int n = max(1, min(ctas, total / least));
  if constexpr (EVEN == 2) {  // (without a division, which a step of few keys would notice)
    if (total > n && total <= 2 * n) n = (total + 1) >> 1;
  } else if constexpr (EVEN > 2) {
    const int longest = (total + n - 1) / n;
    if (longest > 0 && longest <= EVEN) n = (total + longest - 1) / longest;
  }
  const int base = total / n;
  return Ranges{base, total - base * n, total};
}

__device__ __forceinline__ int range_start(const Ranges& r, int c) {
  // (in 64 bits: c * base passes 2^31 for CTAs behind the last that has work)
  return static_cast<int>(min(static_cast<long long>(c) * r.base + min(c, r.more), static_cast<long long>(r.total)));
}

// The CTA whose range holds a tile.
__device__ __forceinline__ int range_of(const Ranges& r, int tile) {
  const int longer = r.more * (r.base + 1);
  return tile < longer ? tile / (r.base + 1) : r.more + (tile - longer) / r.base;
}

// line[e] = tiles of one key head of all entries before e, for e in
// [0, entries]; tiles_of(e) counts an entry's; `scratch` holds one word a
// warp.  Ends with a CTA-wide barrier.
template <int THREADS, typename F>
__device__ __forceinline__ void build_line(int* line, int* scratch, int entries, F tiles_of) {
  constexpr int WARPS = THREADS / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int base = 0;
  for (int e0 = 0; e0 < entries; e0 += THREADS) {
    const int e = e0 + static_cast<int>(threadIdx.x);
    const int n = e < entries ? tiles_of(e) : 0;
    int x = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    __syncthreads();  // the scratch words of the last round have been read
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    int before = base;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
      if (i < warp) before += scratch[i];
      base += scratch[i];
    }
    if (e < entries) line[e] = before + x - n;
  }
  if (threadIdx.x == 0) line[entries] = base;
  __syncthreads();
}

// A walk over the pieces of units that a CTA's range [at, stop) of the line
// holds.  starts(e) is the first tile of entry e in tiles of one key head.
struct Walk {
  int e, head;      // entry and key head of the piece
  int tile, end;    // its tiles within the unit: [tile, end)
  int tiles;        // tiles of the unit
};

template <typename F>
__device__ __forceinline__ bool walk_begin(Walk& w, F starts, int entries, int Hkv, int at, int stop) {
  if (at >= stop) return false;
  // the last entry that starts at or before `at` (one with tiles: an empty
  // one starts where its successor does)
  int lo = 0, hi = entries - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (starts(mid) * Hkv <= at) lo = mid; else hi = mid - 1;
  }
  w.e = lo;
  w.tiles = starts(lo + 1) - starts(lo);
  const int in = at - starts(lo) * Hkv;
  w.head = in / w.tiles;
  w.tile = in - w.head * w.tiles;
  w.end = min(w.tiles, w.tile + stop - at);
  return true;
}

template <typename F>
__device__ __forceinline__ bool walk_next(Walk& w, F starts, int Hkv, int& at, int stop) {
  at += w.end - w.tile;
  if (at >= stop) return false;
  if (++w.head == Hkv) {
    w.head = 0;
    do {
      ++w.e;
      w.tiles = starts(w.e + 1) - starts(w.e);
    } while (w.tiles == 0);
  }
  w.tile = 0;
  w.end = min(w.tiles, stop - at);
  return true;
}
#endif

}  // namespace fa
