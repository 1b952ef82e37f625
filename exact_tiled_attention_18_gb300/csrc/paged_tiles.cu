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
//    lets its keys be read once).  Rows are gathered from q by the softmax
//    warps themselves with plain loads into the swizzled tile; each row has
//    its own last visible key.
//  - Keys come from pages: a tile of 128 keys is 128 / box_rows TMA boxes a
//    64-column block, issued by the lanes of the producer warp, page ids read
//    32 boxes ahead.
//  - Division.  The first one to two units (256 rows of a key head) for every
//    CTA form a line of key tiles that is cut into equal ranges, one a CTA, as
//    in the step kernel; the others are drawn whole from a counter, heaviest
//    first within groups of heads whose keys stay in L2.  So few units fill
//    the GPU, and many end together, on their lightest.  Pieces of a unit leave normalised outputs
//    and log-sum-exps that paged_combine_kernel merges.
//  - Rows of a page behind the last key may hold anything, NaN included, and
//    0 * NaN would poison the product with V: a spare warp zeroes them in the
//    last tile before that product is issued.
//
//   warps 0-3  softmax of tile A     warp 8   TMA producer
//   warps 4-7  softmax of tile B     warp 9   MMA issuer, owns tensor memory
//                                    warp 10  zeroes the values behind the last key
//                                    warp 11  draws the whole units
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "serving.h"

namespace fa {
namespace {

constexpr int kThreads = 384;
// registers: the split of the square forward (fwd.cu), 2*128*192 + 128*120 =
// 384*168
constexpr int kLaunchRegs = 168;
constexpr int kSoftmaxRegs = 192;
constexpr int kOtherRegs = 120;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr float kTau = 8.f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRows = 128;        // rows and keys a tile
constexpr int kUnitReaders = 11;  // warps that follow the drawn units: softmax, producer, issuer, cleaner

enum TileSite : int {
  SITE_TILE_LOAD = 75,
  SITE_TILE_MMA = 76,
  SITE_TILE_S = 77,
  SITE_TILE_O = 78,
  SITE_TILE_CLEAN = 79,
  SITE_TILE_UNIT = 80,
};

template <int D>
struct TileLayout {
  static constexpr int kTileBytes = kRows * D * 2;
  static constexpr int kSlots = (D == 128) ? 4 : 8;
  static constexpr int kRingOff = 2 * kTileBytes;
  static constexpr int kBarOff = kRingOff + kSlots * kTileBytes;
  static constexpr int KV_FULL = 0;
  static constexpr int KV_EMPTY = KV_FULL + kSlots;
  static constexpr int Q_FULL = KV_EMPTY + kSlots;
  static constexpr int S_FULL = Q_FULL + 2;
  static constexpr int P_FULL = S_FULL + 2;
  static constexpr int O_FULL = P_FULL + 2;
  static constexpr int DIRTY = O_FULL + 2;
  static constexpr int CLEAN = DIRTY + 1;
  static constexpr int UNIT_FULL = CLEAN + 1;
  static constexpr int UNIT_EMPTY = UNIT_FULL + 2;
  static constexpr int DRAIN = UNIT_EMPTY + 2;
  static constexpr int kNumBars = DRAIN + 1;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kScratchOff = kMiscOff + 16;  // one word a warp, then the two drawn units
  static constexpr int kLineOff = kScratchOff + 64;
  static constexpr int kSmemBytes = kLineOff + (kTileLine + 1) * 4 + 1024;
  static constexpr uint32_t kColO = 256;
};

// One piece of a unit: how many key tiles of it each row tile needs.
struct Piece {
  int na, nb;     // key tiles from w.tile on
  int nmax;
  int limit;      // first key (from the origin) whose values may be anything
  int clean;      // piece tile that holds it, or -1
};

// Row space of a unit: rows [256 pair, 256 pair + 256) of `total`.
__device__ __forceinline__ bool tile_wait(uint32_t bar, uint32_t parity, const WaitCtl& w, int site, int unit) {
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, w, site, unit));
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

template <int D, bool PREFIX>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tiles_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ PagedTiles p) {
  using L = TileLayout<D>;
  constexpr int S = L::kSlots;
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
    for (int s = 0; s < S; ++s) {
      mbar_init(bars + 8 * (L::KV_FULL + s), 1);
      mbar_init(bars + 8 * (L::KV_EMPTY + s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bars + 8 * (L::Q_FULL + t), 4);
      mbar_init(bars + 8 * (L::S_FULL + t), 1);
      mbar_init(bars + 8 * (L::P_FULL + t), 4);
      mbar_init(bars + 8 * (L::O_FULL + t), 1);
    }
    mbar_init(bars + 8 * L::DIRTY, 1);
    mbar_init(bars + 8 * L::CLEAN, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + 8 * (L::UNIT_FULL + i), 1);
      mbar_init(bars + 8 * (L::UNIT_EMPTY + i), kUnitReaders);
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
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (p.wait_first) grid_wait();
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
  if constexpr (PREFIX) {  // the same for every unit
    const int n = (reach + kRows - 1) / kRows;
    for (int i = threadIdx.x; i <= cut; i += kThreads) line[i] = i * n;
    __syncthreads();
  } else {
    build_line<kThreads>(line, scratch, cut, [&](int e) { return unit_tiles(e); });
  }
  const int total = line[cut];
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= cut; i += kThreads) p.line_out[i] = line[i];
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto BAR = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  // A CTA's work: its range of the line (place x: from tile x on), then the
  // units it draws (place -1 - n: the n-th).
  volatile int* drawn = scratch + 14;
  const Ranges ranges = make_ranges(total, gridDim.x, p.part.min_tiles);
  const int at0 = range_start(ranges, blockIdx.x);
  const int stop = range_start(ranges, blockIdx.x + 1);
  int at = at0;
  struct Place {
    int u;           // unit
    int tile, end;   // its tiles in this piece: [tile, end)
    bool whole;      // all of the unit's
  };
  auto locate = [&](int place) {
    Place w;
    if (place < 0) {
      w.u = drawn[(-1 - place) & 1];
      w.tile = 0;
      w.end = unit_tiles(w.u);
      w.whole = true;
      return w;
    }
    // the last unit that starts at or before the tile (one with tiles: an
    // empty one starts where its successor does)
    int lo = 0, hi = cut - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (line[mid] <= place) lo = mid; else hi = mid - 1;
    }
    w.u = lo;
    w.tile = place - line[lo];
    const int tiles = line[lo + 1] - line[lo];
    w.end = min(tiles, w.tile + stop - place);
    w.whole = w.tile == 0 && w.end == tiles;
    return w;
  };
  const WaitCtl wc{abort_flag, p.status, p.wait_limit_ns};
  // A row tile without keys in a piece, and the cleaner, wait while the other
  // tile's whole pieces go by: their limit grows with the range.  The producer
  // and the issuer notice a stall within the limit itself and end all waits.
  const WaitCtl wc_idle{abort_flag, p.status, p.wait_limit_ns * 64};

  // Every role that follows the work calls this before a piece, with all lanes
  // of its warp (`true`: there is one), and done() behind it.
  auto another = [&](bool& ok) {
    if (at >= 0) {
      if (at < stop) return true;
      if (cut == p.part.units) return false;
      at = -1;
    }
    const int n = -1 - at;
    ok = tile_wait(BAR(L::UNIT_FULL + (n & 1)), (n >> 1) & 1, wc_idle, SITE_TILE_UNIT, at);
    return ok && drawn[n & 1] < p.part.units;
  };
  auto done = [&](int tiles) {
    if (at < 0) {
      mbar_arrive_warp(BAR(L::UNIT_EMPTY + ((-1 - at) & 1)));
      --at;
    } else {
      at += tiles;
    }
  };

  auto piece_of = [&](const Place& w, int& b, int& head, int& r0) {
    Piece x;
    unit_at(w.u, b, head, r0);
    int ka, kb;
    unit_keys(b, r0, ka, kb, x.limit);
    const int len = w.end - w.tile;
    x.na = max(0, min((ka + kRows - 1) / kRows - w.tile, len));
    x.nb = max(0, min((kb + kRows - 1) / kRows - w.tile, len));
    x.nmax = max(x.na, x.nb);
    const int at_tile = x.limit / kRows - w.tile;
    x.clean = x.limit % p.box_rows != 0 && at_tile >= 0 && at_tile < x.nmax ? at_tile : -1;
    return x;
  };

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    regs_increase<kSoftmaxRegs>();
    const int t = warp >> 2;
    const int r = ((warp & 3) << 5) + lane;  // row inside the tile == TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) << 5) << 16;
    const uint32_t tS = tmem + lane_off + static_cast<uint32_t>(t * 128);
    const uint32_t tO = tmem + lane_off + L::kColO + static_cast<uint32_t>(t * D);
    const float scale_log2 = p.scale_log2;
    // A row's whole register budget is its 128 scores, so a piece is described
    // by its place `at` on the line alone; the rest is worked out again from
    // shared memory before and after the sweep.
    auto row_of = [&](int b, int r0, int& rb, int& rr) {  // sequence and row of this thread's row; false: none
      const int row = r0 + t * kRows + r;
      rb = PREFIX ? row / rows : b;
      rr = PREFIX ? row - rb * rows : row;
      return row < space;
    };
    uint32_t sn = 0, on = 0;
    bool ok = true;
    while (another(ok)) {
      int nt, lim0 = 0;  // key tiles; this row's visible keys from the piece's first
      {
        int b, head, r0, rb, rr;
        const Place w = locate(at);
        const Piece x = piece_of(w, b, head, r0);
        nt = t ? x.nb : x.na;
        unsigned long long grow = 0;
        const bool valid = row_of(b, r0, rb, rr);
        if (valid) {
          const int i = rr % p.seq.Nq;
          int lq, lk;
          seq_lens(p.seq, rb, lq, lk);
          if (i < lq) lim0 = (p.causal ? min(i + lk - lq + 1, lk) : lk) - origin;
          if (PREFIX) lim0 = min(lim0, p.seq.prefix_len);
          lim0 -= w.tile * kRows;
          grow = (static_cast<unsigned long long>(rb) * Hkv + head) * rows + rr;
        }
        if (nt > 0) {
          // gather the tile's 128 rows: a warp its 32, whole rows at a time.
          // The tile is free: its last product completed before O was read.
          constexpr int LPR = D / 8;            // lanes a row, 16 bytes each
          constexpr int RPI = 32 / LPR;         // rows an iteration
          const int chunk = lane % LPR;
          const uint32_t qt = sbase + t * L::kTileBytes + (chunk >> 3) * 16384;
          uint4 v[32 / RPI];
#pragma unroll
          for (int k = 0; k < 32 / RPI; ++k) {
            const int src = k * RPI + lane / LPR;   // lane of the warp that owns the row
            const unsigned long long g = __shfl_sync(0xffffffffu, grow, src);
            const int live = __shfl_sync(0xffffffffu, static_cast<int>(valid), src);
            v[k] = live ? __ldg(reinterpret_cast<const uint4*>(p.q + g * D) + chunk) : make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
          for (int k = 0; k < 32 / RPI; ++k) {
            const int rr2 = ((warp & 3) << 5) + k * RPI + lane / LPR;
            st_shared_v4(qt + sw128(rr2, chunk & 7), v[k].x, v[k].y, v[k].z, v[k].w);
          }
          fence_proxy_async_smem();
          mbar_arrive_warp(BAR(L::Q_FULL + t));
        }
      }
      float m_ref = 0.f, l = 0.f, dl = 0.f;
      for (int j = 0; j < nt; ++j) {
        ok = tile_wait(BAR(L::S_FULL + t), sn & 1, wc_idle, SITE_TILE_S, at);
        if (!ok) break;
        ++sn;
        tc_fence_after();
        float s[128];
        {
          uint32_t sr[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(sr + 32 * c));
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 128; ++c) s[c] = __uint_as_float(sr[c]);
        }
        const int lim = lim0 - j * kRows;
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
          // a row sees a leading range of the piece's keys: if it sees none of
          // the first tile it sees none at all
          m_ref = mt == -CUDART_INF_F ? 0.f : mt;
        } else {
          const bool need = mt > m_ref + kTau;
          if (__any_sync(0xffffffffu, need)) {
            const float m_new = fmaxf(m_ref, mt);
            const float alpha = ex2_approx(m_ref - m_new);
            m_ref = m_new;
            l *= alpha;
            dl *= alpha;
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
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(BAR(L::P_FULL + t));
      }
      if (!ok) break;
      if (nt > 0) {
        ok = tile_wait(BAR(L::O_FULL + t), on & 1, wc, SITE_TILE_O, at);
        if (!ok) break;
        ++on;
        tc_fence_after();
      }
      const bool live = l > 0.f;
      const float inv = live ? 1.0f / (l + dl) : 0.f;
      int b, head, r0, rb, rr;
      const Place w = locate(at);
      unit_at(w.u, b, head, r0);
      const bool valid = row_of(b, r0, rb, rr);
      const bool whole = p.direct && w.whole;
      const size_t grow = (static_cast<size_t>(rb) * Hkv + head) * rows + rr;
      const long long slot = p.part.two_a_cta ? 2LL * blockIdx.x + (at == at0 ? 0 : 1)
                                              : static_cast<long long>(w.u) + (at < 0 ? gridDim.x : blockIdx.x);
      const long long prow = slot * kPairRows + t * kRows + r;
      float* dst = whole ? static_cast<float*>(p.o) + grow * D : p.part.o + prow * D;
      const bool half = whole && p.o_bf16;
      uint16_t* dst_h = static_cast<uint16_t*>(p.o) + grow * D;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        // (a tile without keys reads what was left there, and drops it)
        tmem_ld32(tO + 32 * c, v);
        tmem_ld_wait();
        if (!live) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;
        }
        if (valid && half) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 h;
            h.x = pack_bf16x2(__uint_as_float(v[8 * i + 0]) * inv, __uint_as_float(v[8 * i + 1]) * inv);
            h.y = pack_bf16x2(__uint_as_float(v[8 * i + 2]) * inv, __uint_as_float(v[8 * i + 3]) * inv);
            h.z = pack_bf16x2(__uint_as_float(v[8 * i + 4]) * inv, __uint_as_float(v[8 * i + 5]) * inv);
            h.w = pack_bf16x2(__uint_as_float(v[8 * i + 6]) * inv, __uint_as_float(v[8 * i + 7]) * inv);
            *reinterpret_cast<uint4*>(dst_h + 32 * c + 8 * i) = h;
          }
        } else if (valid) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float4 f;
            f.x = __uint_as_float(v[4 * i + 0]) * inv;
            f.y = __uint_as_float(v[4 * i + 1]) * inv;
            f.z = __uint_as_float(v[4 * i + 2]) * inv;
            f.w = __uint_as_float(v[4 * i + 3]) * inv;
            *reinterpret_cast<float4*>(dst + 32 * c + 4 * i) = f;
          }
        }
      }
      if (valid) {
        const float lse2 = live ? m_ref + log2f(l) : -CUDART_INF_F;
        if (whole)
          p.lse[grow] = live ? lse2 * kLn2 : -CUDART_INF_F;
        else
          p.part.lse[prow] = lse2;
      }
      done(w.end - w.tile);
    }
  } else {
    regs_decrease<kOtherRegs>();
    if (warp == 8) {
      // -------------------------------------------------------- TMA producer
      const int boxes = kRows / p.box_rows;
      const int block = lane / boxes, box = lane - block * boxes;  // this lane's load of a tile
      const bool loads = block < CB;
      const uint32_t offset = static_cast<uint32_t>(block * 16384 + box * p.box_rows * 128);
      const uint64_t policy = l2_policy_evict_last();
      uint32_t kvpos = 0;
      int piece = 0;
      bool ok = true;
      while (another(ok)) {
        int b, head, r0;
        const Place w = locate(at);
        const Piece x = piece_of(w, b, head, r0);
        const int* pages = PREFIX ? p.prefix_table : p.table.block_table + b * p.table.table_stride;
        const int first = origin + w.tile * kRows;
        const int last = origin + x.limit;
        const int count = x.nmax * boxes;
        auto page_of = [&](int i) {
          const int key = first + i * p.box_rows;
          return i < count && key < last ? __ldg(pages + key / p.table.page_size) : -1;
        };
        int cur = page_of(lane), next = page_of(32 + lane);
        for (int j = 0; j < x.nmax && ok; ++j) {
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
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t s = kvpos % S, use = kvpos / S;
            ok = tile_wait(BAR(L::KV_EMPTY + s), (use & 1) ^ 1, wc, SITE_TILE_LOAD, at);
            if (!ok) break;
            ++kvpos;
            if (blockIdx.x == 0 && piece == p.stall_unit && j == 0 && kv == 0)
              continue;  // testing hook: leave this tile unloaded
            if (lane == 0) mbar_arrive_expect_tx(BAR(L::KV_FULL + s), L::kTileBytes);
            __syncwarp();
            if (loads)
              tma_load_3d_hint(sbase + L::kRingOff + s * L::kTileBytes + offset, kv == 0 ? &tm_k : &tm_v,
                               BAR(L::KV_FULL + s), block * 64, row, outer, policy);
            __syncwarp();
          }
        }
        if (!ok) break;
        ++piece;
        done(w.end - w.tile);
      }
      if (!ok && lane == 0) {
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
        constexpr uint32_t id_s = idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t id_pv = idesc_bf16_f32(128, D, false, true);
        const SDesc qdesc0 = sdesc_sw128(sbase, 16, 1024);
        const SDesc kdesc0 = sdesc_sw128(sbase + L::kRingOff, 16, 1024);
        const SDesc vdesc0 = sdesc_sw128(sbase + L::kRingOff, kRows * 128, 1024);
        constexpr uint32_t kTileUnits = L::kTileBytes >> 4;
        auto issue_s = [&](int t, uint32_t slot) {
          const SDesc qd = qdesc0 + static_cast<uint32_t>(t) * kTileUnits;
          const SDesc kd = kdesc0 + slot * kTileUnits;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
            umma_ss(tmem + static_cast<uint32_t>(t * 128), qd + off, kd + off, id_s, ks > 0 ? 1u : 0u);
          }
        };
        auto issue_pv = [&](int t, uint32_t slot, bool acc) {
          const SDesc vd = vdesc0 + slot * kTileUnits;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            umma_ts(tmem + L::kColO + static_cast<uint32_t>(t * D), tmem + static_cast<uint32_t>(t * 128 + ks * 8),
                    vd + static_cast<uint32_t>((ks * 2048) >> 4), id_pv, (acc || ks > 0) ? 1u : 0u);
          }
        };
        uint32_t qa = 0, qb = 0, kvbase = 0, pa = 0, pb = 0, cleaned = 0;
        bool ok = true;
        while (another(ok)) {
          int b, head, r0;
          const Place w = locate(at);
          const Piece x = piece_of(w, b, head, r0);
          const int unit = at;
          const int na = x.na, nb = x.nb;
          if (lane == 0) {
          do {
          if (x.nmax > 0) {
            ok = wait_bounded(BAR(L::KV_FULL + kvbase % S), (kvbase / S) & 1, wc, SITE_TILE_MMA, unit);
            if (!ok) break;
            if (na > 0) {
              ok = wait_bounded(BAR(L::Q_FULL + 0), qa & 1, wc, SITE_TILE_MMA, unit);
              if (!ok) break;
              ++qa;
              tc_fence_after();
              issue_s(0, kvbase % S);
              umma_commit(BAR(L::S_FULL + 0));
            }
            if (nb > 0) {
              ok = wait_bounded(BAR(L::Q_FULL + 1), qb & 1, wc, SITE_TILE_MMA, unit);
              if (!ok) break;
              ++qb;
              tc_fence_after();
              issue_s(1, kvbase % S);
              umma_commit(BAR(L::S_FULL + 1));
            }
          }
          // One key tile.  STEADY: both row tiles have it and the next one, and
          // its values need no zeroing -- all but the last steps of most
          // pieces, with nothing to decide in them: this thread's instructions
          // are on every step's critical path.
          auto step = [&](auto steady_tag, int j) -> bool {
            constexpr bool STEADY = decltype(steady_tag)::value;
            const uint32_t kpos = kvbase + 2 * j, vpos = kpos + 1, knext = kpos + 2;
            const bool has_a = STEADY || j < na, next_a = STEADY || j + 1 < na;
            const bool has_b = STEADY || j < nb, next_b = STEADY || j + 1 < nb;
            const bool dirty = !STEADY && j == x.clean;
            umma_commit(BAR(L::KV_EMPTY + kpos % S));  // K_j is free once S(j) of both tiles completes
            if (!wait_bounded(BAR(L::KV_FULL + vpos % S), (vpos / S) & 1, wc, SITE_TILE_MMA, unit)) return false;
            // the last keys' values: zeroed behind the last key by warp 10
            // while the softmax of this tile runs
            if (dirty) mbar_arrive(BAR(L::DIRTY));
            auto values_ready = [&]() {
              return !dirty || wait_bounded(BAR(L::CLEAN), cleaned & 1, wc, SITE_TILE_CLEAN, unit);
            };
            if (has_a) {
              if (!wait_bounded(BAR(L::P_FULL + 0), pa & 1, wc, SITE_TILE_MMA, unit) || !values_ready()) return false;
              ++pa;
              tc_fence_after();
              issue_pv(0, vpos % S, j > 0);
              if (!next_a) umma_commit(BAR(L::O_FULL + 0));
              if (next_a) {
                if (!wait_bounded(BAR(L::KV_FULL + knext % S), (knext / S) & 1, wc, SITE_TILE_MMA, unit)) return false;
                tc_fence_after();
                issue_s(0, knext % S);
                umma_commit(BAR(L::S_FULL + 0));
              }
            }
            if (has_b) {
              if (!wait_bounded(BAR(L::P_FULL + 1), pb & 1, wc, SITE_TILE_MMA, unit) || !values_ready()) return false;
              ++pb;
              tc_fence_after();
              issue_pv(1, vpos % S, j > 0);
              if (!next_b) umma_commit(BAR(L::O_FULL + 1));
            }
            if (dirty) ++cleaned;
            umma_commit(BAR(L::KV_EMPTY + vpos % S));  // V_j is free once PV(j) of both tiles completes
            if (next_b) {
              if (!(has_a && next_a)) {  // otherwise tile A's S(j+1) already waited for K_{j+1}
                if (!wait_bounded(BAR(L::KV_FULL + knext % S), (knext / S) & 1, wc, SITE_TILE_MMA, unit)) return false;
                tc_fence_after();
              }
              issue_s(1, knext % S);
              umma_commit(BAR(L::S_FULL + 1));
            }
            return true;
          };
          const int both = min(na, nb) - 1;
          for (int j = 0; j < x.nmax && ok; ++j)
            ok = j < both && j != x.clean ? step(std::true_type{}, j) : step(std::false_type{}, j);
          } while (false);
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          kvbase += 2 * x.nmax;
          done(w.end - w.tile);
        }
        // every MMA this thread issued completes before tensor memory is freed
        if (lane == 0) {
          umma_commit(BAR(L::DRAIN));
          drain_wait(BAR(L::DRAIN), 0, p.wait_limit_ns);
        }
      }
    } else if (warp == 10) {
      // ------------------------------------------- values behind the last key
      uint32_t kvbase = 0, cleaned = 0;
      bool ok = true;
      while (another(ok)) {
        int b, head, r0;
        const Place w = locate(at);
        const Piece x = piece_of(w, b, head, r0);
        const int unit = at;
        if (x.clean >= 0) {
          const uint32_t vpos = kvbase + 2 * x.clean + 1;
          ok = tile_wait(BAR(L::DIRTY), cleaned & 1, wc_idle, SITE_TILE_CLEAN, unit);
          if (!ok) break;
          // the rest of the last key's box; whole boxes behind it were read as zeros
          const int from = x.limit % kRows, rest = p.box_rows - from % p.box_rows;
          const uint32_t vt = sbase + L::kRingOff + (vpos % S) * L::kTileBytes;
          for (int i = lane; i < rest * (D / 8); i += 32) {
            const int row = from + i / (D / 8), c = i % (D / 8);
            st_shared_v4(vt + (c >> 3) * 16384 + sw128(row, c & 7), 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          mbar_arrive_warp(BAR(L::CLEAN));
          ++cleaned;
        }
        kvbase += 2 * x.nmax;
        done(w.end - w.tile);
      }
    } else if (lane == 0 && cut < p.part.units) {
      // ------------------------------------------------------ whole units
      // drawn two ahead: the draw's latency passes behind the work before
      for (int n = 0;; ++n) {
        if (!wait_bounded(BAR(L::UNIT_EMPTY + (n & 1)), ((n >> 1) & 1) ^ 1, wc_idle, SITE_TILE_UNIT, n)) break;
        const int u = cut + atomicAdd(p.counter, 1);
        drawn[n & 1] = u;
        mbar_arrive(BAR(L::UNIT_FULL + (n & 1)));
        if (u >= p.part.units) break;
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

template <int D, bool PREFIX>
cudaError_t launch_t(const PagedTiles& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, int ctas,
                     cudaStream_t stream) {
  using L = TileLayout<D>;
  auto kern = paged_tiles_kernel<D, PREFIX>;
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = setup_kernel_once(kern, L::kSmemBytes, kLaunchRegs, ready);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kern, dim3(ctas), kThreads, L::kSmemBytes, stream, tm_k, tm_v, p);
}

}  // namespace

cudaError_t launch_tiles(const PagedTiles& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, int d, int ctas,
                         cudaStream_t stream) {
  if (d == 64)
    return p.prefix_table ? launch_t<64, true>(p, tm_k, tm_v, ctas, stream)
                          : launch_t<64, false>(p, tm_k, tm_v, ctas, stream);
  return p.prefix_table ? launch_t<128, true>(p, tm_k, tm_v, ctas, stream)
                        : launch_t<128, false>(p, tm_k, tm_v, ctas, stream);
}

}  // namespace fa
