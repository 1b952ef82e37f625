// Attention over the paged cache for few rows a key head: single tokens and
// drafted ones of every query head of its group.
//
// A step reads the keys and values of every sequence once, for G * Nq rows of
// queries a key head: 2 G Nq FLOPs per byte, so it is bound by HBM as long as
// the products run on the tensor cores (on the CUDA cores 8 heads a group
// already cost more than the reading).  A tcgen05 tile would be 128 rows high
// and its result would have to come back through tensor memory before a row
// maximum can be taken, so these use warp-wide mma with the fragments in
// registers, fed by ldmatrix from the swizzled TMA tiles.  Keys and value
// columns are the 16-high side of each mma, query rows the 8-wide side
// (S^T = K Q^T, O^T = V^T P^T): up to 8 rows cost half of what they would as
// rows of a 16-high tile, and the mma rate is what comes next after HBM.
//
//   paged_steps_kernel    persistent CTAs of four compute warps and a TMA warp,
//                         two or three an SM.  The key tiles (64 keys of one
//                         key head) of all sequences form one line, cut into
//                         equal ranges, one a CTA: the lengths stay on the
//                         device, and a batch of very different lengths is
//                         balanced to one tile.  Where a sequence's tiles fall
//                         into more than one range each leaves a partial
//                         result.
//   merge_rows_kernel     merges a row's partial results by their log-sum-exp
//                         (merge_lanes_kernel: with a prefix, or the tile kernel's).
//
// Within a tile each warp multiplies the rows with its 16 keys, the warps
// agree on the row maxima through shared memory, exchange the probabilities
// the same way, and each multiplies all 64 keys with its quarter of the value
// columns: one accumulator and one set of statistics per CTA, so a CTA moves
// from one sequence to the next without merging warps.
//
// Up to 16 rows the probabilities go into the product as a pair of bf16 (the
// value and what its rounding left), 16 significand bits: the second product
// costs tensor time that the kernel has to spare, and O is as exact as with
// fp32 products.  From 17 rows on they are one bf16, as in the other kernels,
// and O is divided by the sum of the rounded weights, so that their rounding
// does not scale a row; the queries then stay in shared memory instead of
// registers (8 sequences x 8 heads x 8192 keys: 24 rows 86 us with fragments
// and pairs, 55 us so; 32 rows 87 and 62).
//
// Measured (whole calls; HBM read rate of keys and values): 8 sequences x 32
// heads x 32768 keys, one row a head, 604 to 619 us = 6.9 to 7.1 TB/s; 32
// sequences of 100 to 16384 keys, 32 heads on 4, 42 us = 5.3 TB/s, of which 6 us
// pass before the first tiles are there; 8 sequences x 8 heads x 8192 keys 48 us =
// 5.6 TB/s with 1 to 8 rows a head, 50 with 9 to 16, 55 with 24, 62 with 32; one
// sequence of 1000 keys 6.9 to 7.2 us in a graph.  A pass
// over a quarter of the first keeps DRAM 85% of its peak busy, the tensor pipe
// 13%.
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

constexpr int kStepKeys = 64;         // keys a tile
constexpr int kStepWarps = 4;         // compute warps, 16 keys of a tile each
constexpr int kStepThreads = 32 * (kStepWarps + 1);
constexpr float kTau = 8.f;           // the reference maximum moves when a row's grows by more than 2^8
constexpr float kLn2 = 0.6931471805599453f;

enum StepSite : int { SITE_STEP_EMPTY = 73, SITE_STEP_FULL = 74 };

// CTAs an SM: three with up to 8 rows, whose registers and rings (two tiles of
// 32 KB at d = 128) leave room for it; two with more (three tiles).  The
// bytes in flight an SM are the same; a third CTA fills the gaps that the
// others leave between sequences.  (256 sequences of 1 to 1024 keys behind a
// prefix: 262 us with three, 267 with two; 64 sequences of 300 keys 13.8 and
// 15.1; one of 4000 keys, where there is less to share, 8.4 and 8.7.)
template <int RB>
constexpr int step_ctas_per_sm() { return RB <= 1 ? 3 : 2; }

// RB: blocks of 8 query rows.
template <int D, int RB>
struct StepLayout {
  // K (or V) of a tile: box by box, in a box its 64-column blocks, in a block
  // one 128-byte row a key, swizzled
  static constexpr int kHalf = (D / 64) * kStepKeys * 128;
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = (step_ctas_per_sm<RB>() == 3 ? 2 : 3) * (128 / D);
  static constexpr bool kMany = RB > 2;   // 17 rows or more
  // probabilities: hi, then lo (up to 16 rows), [RB][64 keys][8 rows] bf16, so
  // that eight keys of a block are 128 contiguous bytes
  static constexpr int kPOff = kStages * kStage;
  static constexpr int kPBlock = kStepKeys * 16;
  // queries (17 rows or more): 64-column blocks of 32 rows of 128 bytes, swizzled
  static constexpr int kQOff = kPOff + (kMany ? 1 : 2) * RB * kPBlock;
  static constexpr int kQBytes = kMany ? 32 * D * 2 : 0;
  static constexpr int kBarOff = kQOff + kQBytes;            // FULL[s] then EMPTY[s]
  // [warps][8 RB] row maxima, row sums, and (17 rows or more) sums of rounded weights
  static constexpr int kMaxOff = kBarOff + 2 * kStages * 8;
  static constexpr int kMiscOff = kMaxOff + (kMany ? 3 : 2) * kStepWarps * 8 * RB * 4;
  // first tile of every sequence, then lk, then lq (a byte: at most 32 here)
  static constexpr int kLineOff = kMiscOff + 16;
  static constexpr int kSmemBytes = kLineOff + (2 * kLineSequences + 1) * 4 + kLineSequences + 1024;
  static_assert(step_ctas_per_sm<RB>() * (kSmemBytes + 1024) <= 228 * 1024, "resident CTAs an SM");
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// c (16 x 8, fp32) += a (16 x 16) b (16 x 8), bf16
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void store_pair(float* p, float x, float y) {
  *reinterpret_cast<float2*>(p) = make_float2(x, y);
}

__device__ __forceinline__ void store_pair(uint16_t* p, float x, float y) {
  *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(x, y);
}

// All four compute warps; true if every one of them passed true.
__device__ __forceinline__ bool warps_agree(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u), "n"(32 * kStepWarps)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void warps_sync() {
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(32 * kStepWarps) : "memory");
}

template <int D, int RB>
__global__ void __launch_bounds__(kStepThreads, step_ctas_per_sm<RB>())
    paged_steps_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_k16, const __grid_constant__ CUtensorMap tm_v16,
                       const __grid_constant__ PagedStep p) {
  using L = StepLayout<D, RB>;
  constexpr int S = L::kStages;
  constexpr int CB = D / 64;       // 64-column blocks of a head
  constexpr int KS = D / 16;       // steps of the score product
  constexpr int MT = D / 64;       // 16-column tiles of a warp's quarter of the values
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + L::kBarOff;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff);
  int* line = reinterpret_cast<int*>(smem + L::kLineOff);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(bars + 8 * s, 1);
      mbar_init(bars + 8 * (S + s), kStepWarps);
    }
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == kStepWarps && lane == 0) {
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
    prefetch_tensormap(&tm_k16);
    prefetch_tensormap(&tm_v16);
  }
  if (p.wait_first) grid_wait(); else grid_overlap();
  grid_trigger();
  // the scratch of the scan is the row-maxima area, unused so far
  int* len_k = line + kLineSequences + 1;
  uint8_t* len_q = reinterpret_cast<uint8_t*>(len_k + kLineSequences);
  build_line<kStepThreads>(line, reinterpret_cast<int*>(smem + L::kMaxOff), p.seq.B, [&](int b) {
    int lq, lk;
    seq_lens(p.seq, b, lq, lk);
    len_q[b] = static_cast<uint8_t>(lq);
    len_k[b] = lk;
    return lq > 0 && lk > p.seq.prefix_len ? (lk - p.seq.prefix_len + kStepKeys - 1) / kStepKeys : 0;
  });
  auto starts = [&](int b) { return line[b]; };
  const int total = line[p.seq.B] * p.seq.Hkv;
  const Ranges ranges = make_ranges<kEvenSteps>(total, gridDim.x, p.part.min_tiles);
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i <= p.seq.B; i += kStepThreads) p.line_out[i] = line[i];
    if (threadIdx.x == 0) {
      p.line_out[p.seq.B + 1] = ranges.base;
      p.line_out[p.seq.B + 2] = ranges.more;
    }
  }
  int at = range_start(ranges, blockIdx.x);
  const int stop = range_start(ranges, blockIdx.x + 1);
  const WaitCtl wc{abort_flag, p.status, p.wait_limit_ns};
  const int unit = static_cast<int>(blockIdx.x);
  Walk w;
  bool more = walk_begin(w, starts, p.seq.B, p.seq.Hkv, at, stop);

  if (warp == kStepWarps) {
    // ------------------------------------------------------------ TMA producer
    // lane i of a tile's loads: operand and box of rows
    const int boxes = kStepKeys / p.box_rows;
    int issued = 0;
    bool ok = true;
    // page of box i of a piece; -1 behind the sequence's end
    auto page_of = [&](const Walk& x, int i) {
      const int key = p.seq.prefix_len + x.tile * kStepKeys + i * p.box_rows;
      return i < (x.end - x.tile) * boxes && key < len_k[x.e]
                 ? p.table.block_table[x.e * p.table.table_stride + key / p.table.page_size]
                 : -1;
    };
    // pages are looked up 32 boxes ahead: the next ones of this piece, and the
    // first of the piece after it
    int ahead = more ? page_of(w, lane) : -1;
    while (more && ok) {
      const int lk = len_k[w.e];
      const int first = p.seq.prefix_len + w.tile * kStepKeys;
      int cur = ahead, next = page_of(w, 32 + lane);
      Walk after = w;
      int after_at = at;
      if (walk_next(after, starts, p.seq.Hkv, after_at, stop)) ahead = page_of(after, lane);
      for (int t = 0; t < w.end - w.tile; ++t, ++issued) {
        if (t > 0 && (t * boxes) % 32 == 0) {
          cur = next;
          next = page_of(w, t * boxes + 32 + lane);
        }
        const int s = issued % S;
        ok = __all_sync(0xffffffffu,
                        wait_bounded(bars + 8 * (S + s), ((issued / S) & 1) ^ 1, wc, SITE_STEP_EMPTY, unit));
        if (!ok) break;
        // a sequence's last tile comes in boxes of 16 rows, so that at most 15
        // rows behind its last key are read
        const bool tail = first + (t + 1) * kStepKeys > lk;
        const int rows_box = tail ? 16 : p.box_rows;
        const int count = kStepKeys / rows_box;          // boxes an operand; one lane loads each
        const int value = lane >= count;
        const int row = (lane - value * count) * rows_box;
        const int page = __shfl_sync(0xffffffffu, cur, (t * boxes + row / p.box_rows) % 32);
        if (unit == p.stall_unit && issued == 0) continue;  // testing hook: leave this tile unloaded
        const uint32_t full = bars + 8 * s;
        if (lane == 0) mbar_arrive_expect_tx(full, L::kStage);
        __syncwarp();
        if (lane < 2 * count) {
          const int key = first + t * kStepKeys + row;
          // rows of no page: a coordinate past the map, which reads zeros
          int outer = p.table.num_pages * p.seq.Hkv;
          if (key < lk) {
            if (page >= 0 && page < p.table.num_pages)
              outer = page * p.seq.Hkv + w.head;
            else
              record_bad_page(p.status, SITE_PAGE_READ, p.b0 + w.e, page);
          }
          const CUtensorMap* tm = value ? (tail ? &tm_v16 : &tm_v) : (tail ? &tm_k16 : &tm_k);
          tma_load_4d(sbase + s * L::kStage + value * L::kHalf + row * (CB * 128), tm, full, 0,
                      key % p.table.page_size, 0, outer);
        }
        __syncwarp();
      }
      if (ok) more = walk_next(w, starts, p.seq.Hkv, at, stop);
    }
    if (!p.wait_first && lane == 0) grid_wait();
    if (!ok && lane == 0) {
      // let the copies already issued land before the CTA can exit
      for (int s = 0; s < S; ++s) {
        if (issued > s) {
          const int last = issued - 1 - ((issued - 1 - s) % S);
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(bars + 8 * s, (last / S) & 1)) {
            if (globaltimer_ns() - t0 > p.wait_limit_ns) break;
          }
        }
      }
    }
    return;
  }

  // ---------------------------------------------------------------- compute
  float* maxima = reinterpret_cast<float*>(smem + L::kMaxOff);   // [warp][8 RB]
  float* sums = maxima + kStepWarps * 8 * RB;
  const int fr = lane >> 2;        // fragment line: key (or value column) fr and fr + 8
  const int fc = (lane & 3) * 2;   // fragment columns: query rows fc, fc + 1 of a block
  const int rows = p.seq.G * p.seq.Nq;
  // ldmatrix lane addresses: K (16 keys x 16 columns), V and P transposed
  const int k_row = lane & 15, k_half = lane >> 4;
  const int v_row = ((lane >> 4) << 3) + (lane & 7), v_half = (lane >> 3) & 1;
  const int v_col = warp * (D / 4);  // first value column of this warp
  const uint32_t p_hi = sbase + L::kPOff, p_lo = p_hi + RB * L::kPBlock;
  constexpr bool MANY = L::kMany;
  constexpr int QC = 32 * D / 8 / (32 * kStepWarps);  // 16-byte chunks of 32 rows of queries, a thread
  uint32_t qf[MANY ? 1 : RB][MANY ? 1 : KS][2];
  uint4 qs[MANY ? QC : 1];
  // the rows of a piece (rows of the group lie together): as fragments, or on
  // their way to shared memory
  auto load_q = [&](const Walk& x) {
    const uint16_t* base = p.q + (static_cast<size_t>(x.e) * p.seq.Hkv + x.head) * rows * D;
    if constexpr (MANY) {
#pragma unroll
      for (int i = 0; i < QC; ++i) {
        const int at = static_cast<int>(threadIdx.x) + i * 32 * kStepWarps;
        const int r = min(at / (D / 8), rows - 1);  // rows behind the last see no key
        qs[i] = *reinterpret_cast<const uint4*>(base + r * D + at % (D / 8) * 8);
      }
      return;
    }
    base += fc;
#pragma unroll
    for (int m = 0; m < (MANY ? 0 : RB); ++m) {
      const uint16_t* src = base + min(8 * m + fr, rows - 1) * D;  // rows of the block behind the last see no key
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qf[m][ks][0] = *reinterpret_cast<const uint32_t*>(src + 16 * ks);
        qf[m][ks][1] = *reinterpret_cast<const uint32_t*>(src + 16 * ks + 8);
      }
    }
  };
  int query[RB];  // query index of rows fc (low half) and fc + 1 of each block; past lq where there is no row
#pragma unroll
  for (int m = 0; m < RB; ++m) {
    const int r = 8 * m + fc;
    query[m] = (r < rows ? r % p.seq.Nq : 0x7fff) | (r + 1 < rows ? (r + 1) % p.seq.Nq : 0x7fff) << 16;
  }
  // ... and from there into it, when every warp is through with the last ones
  auto place_q = [&]() {
    if constexpr (MANY) {
#pragma unroll
      for (int i = 0; i < QC; ++i) {
        const int at = static_cast<int>(threadIdx.x) + i * 32 * kStepWarps;
        const int c = at % (D / 8);
        st_shared_v4(sbase + L::kQOff + (c >> 3) * 4096 + sw128(at / (D / 8), c & 7), qs[i].x, qs[i].y, qs[i].z,
                     qs[i].w);
      }
    }
  };
  if (more) load_q(w);
  if (more) place_q();
  int done = 0;
  bool ok = true;
  while (more && ok) {
    const int lq = len_q[w.e], lk = len_k[w.e];
    int kend[RB][2];               // last visible key + 1 of rows fc, fc + 1
    float m_ref[RB][2], l[RB][2], acc[RB][MT][4];
    float lr[MANY ? RB : 1][2];    // sums of the rounded weights
    if constexpr (MANY) {
#pragma unroll
      for (int m = 0; m < RB; ++m) lr[m][0] = lr[m][1] = 0.f;
      warps_sync();                // the queries are in place
    }
#pragma unroll
    for (int m = 0; m < RB; ++m) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = (query[m] >> (16 * e)) & 0x7fff;
        kend[m][e] = i < lq ? (p.causal ? min(i + lk - lq + 1, lk) : lk) : 0;
        m_ref[m][e] = -CUDART_INF_F;
        l[m][e] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < MT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][n][e] = 0.f;
    }
    Walk after = w;
    int after_at = at;
    const bool another = walk_next(after, starts, p.seq.Hkv, after_at, stop);
    for (int t = w.tile; t < w.end; ++t, ++done) {
      const int s = done % S;
      const bool full = wait_bounded(bars + 8 * s, (done / S) & 1, wc, SITE_STEP_FULL, unit);
      const uint32_t kb = sbase + s * L::kStage;
      const uint32_t vb = kb + L::kHalf;
      const int key0 = p.seq.prefix_len + t * kStepKeys;
      // bytes of a 64-column block of a box; the 16 keys from 16 g on start at
      // box (16 g / its rows), row (16 g modulo them)
      const uint32_t block = (key0 + kStepKeys > lk ? 16 : p.box_rows) * 128;
      auto keys_at = [&](int g) { return (g * 2048 & ~(block - 1)) * CB + (g * 2048 & (block - 1)); };
      // scores of this warp's 16 keys: keys fr (elements 0, 1) and fr + 8 (2, 3)
      float sc[RB][4];
#pragma unroll
      for (int m = 0; m < RB; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[m][e] = 0.f;
      if (__all_sync(0xffffffffu, full)) {
        const uint32_t k16 = kb + keys_at(warp);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t kf[4];
          ldmatrix4(kf, k16 + (ks >> 2) * block + sw128(k_row, 2 * (ks & 3) + k_half));
          if constexpr (MANY) {
#pragma unroll
            for (int m = 0; m < RB; m += 2) {  // 16 rows a load (of 24 the last eight are not used)
              uint32_t qv[4];
              ldmatrix4(qv, sbase + L::kQOff + (ks >> 2) * 4096 +
                                sw128(8 * m + ((lane >> 4) << 3) + (lane & 7), 2 * (ks & 3) + ((lane >> 3) & 1)));
              mma_bf16(sc[m], kf, qv[0], qv[1]);
              if (m + 1 < RB) mma_bf16(sc[m + 1 < RB ? m + 1 : m], kf, qv[2], qv[3]);
            }
          } else {
#pragma unroll
            for (int m = 0; m < RB; ++m) mma_bf16(sc[m], kf, qf[m][ks][0], qf[m][ks][1]);
          }
        }
        if (key0 + kStepKeys > lk) {
          // rows behind the last key may hold anything: their weights are 0,
          // so their values must be finite
          // (whole boxes behind it were read as zeros)
          if ((lk - key0) / 16 == warp) {
            for (int i = lane; i < 16 * 8 * CB; i += 32) {
              const int r = i & 15;
              if (key0 + 16 * warp + r >= lk)
                st_shared_v4(vb + keys_at(warp) + (i >> 7) * block + sw128(r, (i >> 4) & 7), 0u, 0u, 0u, 0u);
            }
          }
          fence_proxy_async_smem();  // before the slot's next TMA load
        }
      }
      const int j = key0 + 16 * warp + fr;
#pragma unroll
      for (int m = 0; m < RB; ++m) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (j >= kend[m][e]) sc[m][e] = -CUDART_INF_F;
          if (j + 8 >= kend[m][e]) sc[m][2 + e] = -CUDART_INF_F;
          float x = fmaxf(sc[m][e], sc[m][2 + e]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          if (lane < 4) maxima[warp * 8 * RB + 8 * m + fc + e] = x;
        }
      }
      ok = warps_agree(full);
      if (!ok) break;
#pragma unroll
      for (int m = 0; m < RB; ++m) {
        float2 x = *reinterpret_cast<const float2*>(maxima + 8 * m + fc);
#pragma unroll
        for (int o = 1; o < kStepWarps; ++o) {
          const float2 y = *reinterpret_cast<const float2*>(maxima + o * 8 * RB + 8 * m + fc);
          x.x = fmaxf(x.x, y.x);
          x.y = fmaxf(x.y, y.y);
        }
        const float top[2] = {x.x * p.scale_log2, x.y * p.scale_log2};
        float pr[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (top[e] > m_ref[m][e] + kTau) {  // the same in every warp
            const float alpha = ex2_approx(m_ref[m][e] - top[e]);  // 0 on the first visible key
            m_ref[m][e] = top[e];
            l[m][e] *= alpha;
            if constexpr (MANY) lr[m][e] *= alpha;
#pragma unroll
            for (int n = 0; n < MT; ++n) {
              acc[m][n][e] *= alpha;
              acc[m][n][2 + e] *= alpha;
            }
          }
          const float mu = m_ref[m][e] == -CUDART_INF_F ? 0.f : m_ref[m][e];
          pr[e] = ex2_approx(fmaf(sc[m][e], p.scale_log2, -mu));
          pr[2 + e] = ex2_approx(fmaf(sc[m][2 + e], p.scale_log2, -mu));
          l[m][e] += pr[e] + pr[2 + e];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // keys fr and fr + 8
          const uint32_t hi = pack_bf16x2(pr[2 * h], pr[2 * h + 1]);
          const float h0 = __uint_as_float(hi << 16), h1 = __uint_as_float(hi & 0xFFFF0000u);
          const uint32_t off = m * L::kPBlock + (16 * warp + 8 * h + fr) * 16 + fc * 2;
          st_shared_u32(p_hi + off, hi);
          if constexpr (MANY) {
            lr[m][0] += h0;
            lr[m][1] += h1;
          } else {
            st_shared_u32(p_lo + off, pack_bf16x2(pr[2 * h] - h0, pr[2 * h + 1] - h1));
          }
        }
      }
      warps_sync();
      // O^T += V^T P^T: all 64 keys, this warp's quarter of the columns
#pragma unroll
      for (int kk = 0; kk < kStepKeys / 16; kk += 2) {
        uint32_t vf[2][MT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < MT; ++n) {
            const int chunk = v_col / 8 + 2 * n + v_half;  // 16-byte chunk of the head's row
            ldmatrix4_t(vf[h][n], vb + keys_at(kk + h) + (chunk >> 3) * block + sw128(v_row, chunk & 7));
          }
#pragma unroll
        for (int m = 0; m < RB; ++m) {
          uint32_t ph[4], pl[4];  // keys 16 kk .. + 32, eight a matrix
          const uint32_t off = m * L::kPBlock + (16 * kk + lane) * 16;
          ldmatrix4_t(ph, p_hi + off);
          if constexpr (!MANY) ldmatrix4_t(pl, p_lo + off);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < MT; ++n) {
              mma_bf16(acc[m][n], vf[h][n], ph[2 * h], ph[2 * h + 1]);
              if constexpr (!MANY) mma_bf16(acc[m][n], vf[h][n], pl[2 * h], pl[2 * h + 1]);
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (S + s));
    }
    if (!ok) break;
    if (another) load_q(after);  // in flight while this piece's results are written
    const size_t row0 = (static_cast<size_t>(w.e) * p.seq.Hkv + w.head) * rows;
    // the row sums of all warps
#pragma unroll
    for (int m = 0; m < RB; ++m) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[m][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (lane < 4) sums[warp * 8 * RB + 8 * m + fc + e] = x;
        if constexpr (MANY) {
          float y = lr[m][e];
          y += __shfl_xor_sync(0xffffffffu, y, 4);
          y += __shfl_xor_sync(0xffffffffu, y, 8);
          y += __shfl_xor_sync(0xffffffffu, y, 16);
          if (lane < 4) sums[(kStepWarps + warp) * 8 * RB + 8 * m + fc + e] = y;
        }
      }
    }
    warps_sync();
    if (another) place_q();
    const bool whole = p.direct && w.tile == 0 && w.end == w.tiles;
    const size_t slot = static_cast<size_t>(w.e) * p.seq.Hkv + w.head + blockIdx.x;
    const int odd = fr & 1;
    auto write = [&](auto* dst, float* lse, const float unit) {  // rows of d outputs; log-sum-exps in units of ln 2
#pragma unroll
      for (int m = 0; m < RB; ++m) {
        float2 sum = *reinterpret_cast<const float2*>(sums + 8 * m + fc);
#pragma unroll
        for (int o = 1; o < kStepWarps; ++o) {
          const float2 y = *reinterpret_cast<const float2*>(sums + o * 8 * RB + 8 * m + fc);
          sum.x += y.x;
          sum.y += y.y;
        }
        float2 weights = sum;  // what O is divided by
        if constexpr (MANY) {
          weights = make_float2(0.f, 0.f);
#pragma unroll
          for (int o = 0; o < kStepWarps; ++o) {
            const float2 y = *reinterpret_cast<const float2*>(sums + (kStepWarps + o) * 8 * RB + 8 * m + fc);
            weights.x += y.x;
            weights.y += y.y;
          }
        }
        // (sums are 0 only where no key is seen; a NaN goes through)
        const float s0 = weights.x != 0.f ? __fdividef(1.f, weights.x) : 0.f;
        const float s1 = weights.y != 0.f ? __fdividef(1.f, weights.y) : 0.f;
        // neighbours in the column exchange rows: a lane then holds two
        // adjacent columns of row fc (even columns' lanes) or fc + 1 (odd ones')
        const int r = 8 * m + fc + odd;
        const bool valid = r < rows;
#pragma unroll
        for (int n = 0; n < MT; ++n) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float a = acc[m][n][2 * h] * s0, b = acc[m][n][2 * h + 1] * s1;
            const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 4);
            const float x = odd ? got : a, y = odd ? b : got;
            if (valid) store_pair(dst + r * D + v_col + 16 * n + 8 * h + (fr & ~1), x, y);
          }
        }
        if (warp == 0 && fr < 2 && valid) {
          const float total = odd ? sum.y : sum.x;
          lse[r] = total != 0.f ? ((odd ? m_ref[m][1] : m_ref[m][0]) + __log2f(total)) * unit : -CUDART_INF_F;
        }
      }
    };
    if (!whole)
      write(p.part.o + slot * rows * D, p.part.lse + slot * rows, 1.f);
    else if (p.o_bf16)
      write(static_cast<uint16_t*>(p.o) + row0 * D, p.lse + row0, kLn2);
    else
      write(static_cast<float*>(p.o) + row0 * D, p.lse + row0, kLn2);
    w = after;
    at = after_at;
    more = another;
  }
}

// Where a unit has its partial results.
struct Pieces {
  int n;              // pieces
  int c0;             // first CTA
  int slot;           // slot of a piece of CTA 0
};

// `tile`: the unit's first tile on the line; nt: its tiles.
__device__ __forceinline__ Pieces pieces_on_line(const Ranges& ranges, int unit, int tile, int nt) {
  Pieces x{0, 0, unit};
  if (nt > 0) {
    x.c0 = range_of(ranges, tile);
    x.n = range_of(ranges, tile + nt - 1) - x.c0 + 1;
  }
  return x;
}

// The ranges stand behind the line's table of `entries` entries.
__device__ __forceinline__ Ranges line_ranges(const int* line, int entries) {
  return Ranges{line[entries + 1], line[entries + 2], line[entries]};
}

// Unit (entry, head) of the step kernel.
__device__ __forceinline__ Pieces step_pieces(const PartRef& r, int entry, int head, int Hkv) {
  const int t0 = r.line[entry], nt = r.line[entry + 1] - t0;
  Ranges ranges = line_ranges(r.line, r.cut);
  ranges.total *= Hkv;
  return pieces_on_line(ranges, entry * Hkv + head, t0 * Hkv + head * nt, nt);
}

// Unit u of the tile kernel.
__device__ __forceinline__ Pieces tile_pieces(const PartRef& r, int u) {
  if (u >= r.cut) return Pieces{1, 0, u + r.ctas};
  const int t0 = r.line[u], nt = r.line[u + 1] - t0 - r.piece_cost;
  const Ranges ranges = line_ranges(r.line, r.cut);
  if (ranges.base == kWholeUnits) return Pieces{1, 0, 0};
  return pieces_on_line(ranges, u, t0, nt);
}

// The tile kernel's unit of (sequence, head) bh and row pair `pair`.
__device__ __forceinline__ int tile_unit(const PartRef& r, int bh, int pair) {
  const int g = bh / r.group;
  const int hs = min(r.group, r.heads - g * r.group);
  return g * r.group * r.pairs + (r.pairs - 1 - pair) * hs + bh - g * r.group;
}

// Rows of a unit.
__host__ __device__ __forceinline__ int rows_of_unit(const PartRef& r) { return r.dual ? kTileRows : r.slot_rows; }

// Where column `col` (a multiple of 4) of row `row` of the tile kernel's lies.
__device__ __forceinline__ long long tile_part(long long row, int col, int d) {
  return (row & ~31LL) * d + (col >> 2) * 128 + (row & 31) * 4;
}

__device__ __forceinline__ long long piece_row(const PartRef& r, const Pieces& x, int k, int in) {
  const int slot = r.two_a_cta ? 2 * (x.c0 + k) + (k > 0 ? 0 : 1) : x.slot + x.c0 + k;
  return static_cast<long long>(slot) * r.slot_rows + in;
}

// The running merge of partial results: maximum, sum (0: no key seen so far)
// and C columns.
template <int C>
struct Merged {
  float top, sum, acc[C];

  __device__ __forceinline__ void clear() {
    top = -CUDART_INF_F;
    sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
  }

  // `lse` (U of them, -inf: none) and their columns
  template <int U>
  __device__ __forceinline__ void add(const float (&lse)[U], const float (&v)[U][C]) {
    float m = top;
#pragma unroll
    for (int u = 0; u < U; ++u) m = max_nan(m, lse[u]);
    if (m == -CUDART_INF_F) return;
    const float g = ex2_approx(top - m);
    top = m;
    sum *= g;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] *= g;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (lse[u] == -CUDART_INF_F) continue;
      const float f = ex2_approx(lse[u] - m);
      sum += f;
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] = fmaf(f, v[u][c], acc[c]);
    }
  }

  __device__ __forceinline__ float lse() const { return sum != 0.f ? (top + __log2f(sum)) * kLn2 : -CUDART_INF_F; }
  __device__ __forceinline__ float scale() const { return sum != 0.f ? __fdividef(1.f, sum) : 0.f; }
};

// Merges the rows of the step kernel's units where there is no prefix.  A warp
// takes RPW neighbouring rows of one unit (their pieces are the same) or, where
// rows are few and pieces many, WARPS warps share one row; a lane takes D / 32
// columns.  Bound by instructions and by the latency of two rounds of loads
// (where the pieces are, the pieces).
template <int D, int WARPS, int RPW>
__global__ void __launch_bounds__(256) merge_rows_kernel(const __grid_constant__ PagedCombine p) {
  static_assert(WARPS == 1 || RPW == 1, "one or the other");
  constexpr int CW = D / 32;
  constexpr int U = WARPS > 1 ? 4 : 2;  // pieces in flight
  __shared__ float s_max[8], s_sum[8], s_acc[WARPS > 1 ? 8 : 1][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp % WARPS;
  const int rows = p.seq.G * p.seq.Nq;
  const unsigned groups = (rows + RPW - 1) / RPW;  // of rows, in a unit
  const unsigned item = blockIdx.x * (8 / WARPS) + warp / WARPS;
  const int unit = static_cast<int>(min(item / groups, static_cast<unsigned>(p.units - 1)));
  const int r0 = static_cast<int>(item % groups) * RPW;
  const bool in = item < p.units * groups;
  const int b = unit / p.seq.Hkv, head = unit - b * p.seq.Hkv;
  grid_wait();
  const Pieces own = step_pieces(p.part, b, head, p.seq.Hkv);
  const bool skip = !in || (p.direct && own.n == 1);  // written by the only CTA that had it
  const int count = skip ? 0 : min(RPW, rows - r0);
  Merged<CW> m[RPW];
#pragma unroll
  for (int q = 0; q < RPW; ++q) m[q].clear();
  auto load = [&](const float* src, float (&v)[CW]) {
    if constexpr (CW == 4)
      *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src);
    else
      *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src);
  };
  const int n = count > 0 ? own.n : 0;
  for (int i = sub; i < n; i += WARPS * U) {
    float lse[RPW][U], v[RPW][U][CW];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = i + u * WARPS;
      const long long at = piece_row(p.part, own, k, r0);
#pragma unroll
      for (int q = 0; q < RPW; ++q) {
        lse[q][u] = -CUDART_INF_F;
        if (k < n && q < count) {
          lse[q][u] = p.part.lse[at + q];
          load(p.part.o + (at + q) * D + CW * lane, v[q][u]);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < RPW; ++q) m[q].add(lse[q], v[q]);
  }
  if constexpr (WARPS > 1) {
#pragma unroll
    for (int c = 0; c < CW; ++c) s_acc[warp][CW * lane + c] = m[0].acc[c];
    if (lane == 0) {
      s_max[warp] = m[0].top;
      s_sum[warp] = m[0].sum;
    }
    __syncthreads();
    if (sub != 0) return;
#pragma unroll
    for (int o = 1; o < WARPS; ++o) {
      const float m2 = s_max[warp + o];
      if (m2 == -CUDART_INF_F) continue;
      const float top = max_nan(m[0].top, m2);
      const float f = ex2_approx(m2 - top), g = ex2_approx(m[0].top - top);
      m[0].top = top;
      m[0].sum = m[0].sum * g + s_sum[warp + o] * f;
#pragma unroll
      for (int c = 0; c < CW; ++c) m[0].acc[c] = m[0].acc[c] * g + s_acc[warp + o][CW * lane + c] * f;
    }
  }
#pragma unroll
  for (int q = 0; q < RPW; ++q) {
    if (q >= count) break;
    const float inv = m[q].scale();
    const size_t row = static_cast<size_t>(unit) * rows + r0 + q;
    const size_t at = row * D + CW * lane;
#pragma unroll
    for (int c = 0; c < CW; c += 2) {
      const float x = m[q].acc[c] * inv, y = m[q].acc[c + 1] * inv;
      if (p.o_bf16)
        store_pair(static_cast<uint16_t*>(p.o) + at + c, x, y);
      else
        store_pair(static_cast<float*>(p.o) + at + c, x, y);
    }
    if (lane == 0) p.lse[row] = m[q].lse();
  }
}

// Merges the rows of the tile kernel's units (STEPS = false) or of the step
// kernel's, and those of the shared prefix.  A lane takes one of 32 rows that
// lie together, and 16 of its columns; a CTA's warps take the row group's other
// columns (WARPS = 1) or, where rows are few and pieces many, every WARPS-th
// piece each.
template <int D, int WARPS, bool STEPS>
__global__ void __launch_bounds__(256) merge_lanes_kernel(const __grid_constant__ PagedCombine p) {
  constexpr int C = 16;                          // columns a warp
  constexpr int BLOCKS = D / C * WARPS / 8;      // CTAs a row group; 0: a CTA takes several
  constexpr int PER = BLOCKS ? 1 : 8 * C / D;    // row groups a CTA
  constexpr int COLS = D / C;                    // column parts of a row group
  __shared__ float s_max[WARPS > 1 ? 8 : 1][32], s_sum[WARPS > 1 ? 8 : 1][32], s_acc[WARPS > 1 ? 8 : 1][C][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = p.seq.G * p.seq.Nq;
  // row groups of a unit, or (STEPS) of all sequences' rows of a key head
  const int groups = STEPS ? (p.seq.B * rows + 31) / 32 : rows_of_unit(p.part) / 32;
  const int part = WARPS > 1 ? static_cast<int>(blockIdx.x % BLOCKS) : warp % COLS;
  const int sub = WARPS > 1 ? warp : 0;
  const unsigned item = WARPS > 1 ? blockIdx.x / BLOCKS : blockIdx.x * PER + warp / COLS;
  const int units = STEPS ? p.seq.Hkv : p.units;
  const int unit = static_cast<int>(min(item / groups, static_cast<unsigned>(units - 1)));
  const int in_unit = static_cast<int>(item % groups) * 32 + lane;
  int b, head, row_in;  // sequence, key head, row of its rows
  bool live = item < static_cast<unsigned>(units) * groups;
  if constexpr (STEPS) {
    head = unit;
    live = live && in_unit < p.seq.B * rows;
    b = live ? in_unit / rows : 0;
    row_in = live ? in_unit - b * rows : 0;
  } else {
    // paged_tiles_kernel's order of units
    const int g = unit / (p.part.group * p.part.pairs);
    const int i = unit - g * p.part.group * p.part.pairs;
    const int hs = min(p.part.group, p.part.heads - g * p.part.group);
    const int level = i / hs;
    const int bh = g * p.part.group + i - level * hs;
    b = bh / p.seq.Hkv;
    head = bh - b * p.seq.Hkv;
    row_in = (p.part.pairs - 1 - level) * kPairRows + in_unit;
    live = live && row_in < rows;
  }
  grid_wait();
  Pieces own;
  if constexpr (STEPS)
    own = step_pieces(p.part, b, head, p.seq.Hkv);
  else
    own = tile_pieces(p.part, unit);
  if (p.direct && own.n == 1) live = false;  // written by the only CTA that had it
  Merged<C> m;
  m.clear();
  auto gather = [&](auto steps_tag, const PartRef& ref, const Pieces& x, int row) {
    constexpr bool ROWS = decltype(steps_tag)::value;  // the step kernel's layout
    constexpr int U = 2;  // pieces in flight
    const int n = live ? x.n : 0;
    for (int k0 = sub; k0 < n; k0 += WARPS * U) {
      float lse[U], v[U][C];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * WARPS;
        lse[u] = -CUDART_INF_F;
        if (k < n) {
          const long long at = piece_row(ref, x, k, row);
          lse[u] = ref.lse[at];
          const float* src = ref.o + (ROWS ? at * D + C * part : tile_part(at, C * part, D));
#pragma unroll
          for (int c = 0; c < C; c += 4)
            *reinterpret_cast<float4*>(v[u] + c) = *reinterpret_cast<const float4*>(src + (ROWS ? c : c * 32));
        }
      }
      m.add(lse, v);
    }
  };
  gather(std::bool_constant<STEPS>{}, p.part, own, STEPS ? row_in : in_unit);
  if (STEPS || p.prefix.o) {
    const int all = (p.b0 + b) * rows + row_in;  // row among all sequences'
    const int pair = min(all / kPairRows, p.prefix.pairs - 1);
    gather(std::false_type{}, p.prefix, tile_pieces(p.prefix, tile_unit(p.prefix, head, pair)), all % kPairRows);
  }
  if constexpr (WARPS > 1) {
    s_max[warp][lane] = m.top;
    s_sum[warp][lane] = m.sum;
#pragma unroll
    for (int c = 0; c < C; ++c) s_acc[warp][c][lane] = m.acc[c];
    __syncthreads();
    if (warp != 0) return;
#pragma unroll 1
    for (int o = 1; o < WARPS; ++o) {
      const float m2 = s_max[o][lane];
      const float top = max_nan(m.top, m2);
      if (top == -CUDART_INF_F) continue;
      const float f = ex2_approx(m2 - top), g2 = ex2_approx(m.top - top);
      m.top = top;
      m.sum = m.sum * g2 + s_sum[o][lane] * f;
#pragma unroll
      for (int c = 0; c < C; ++c) m.acc[c] = m.acc[c] * g2 + s_acc[o][c][lane] * f;
    }
  }
  if (!live) return;
  const float inv = m.scale();
  const size_t row = (static_cast<size_t>(b) * p.seq.Hkv + head) * rows + row_in;
  const size_t at = row * D + C * part;
  if (p.o_bf16) {
    uint32_t w[C / 2];
#pragma unroll
    for (int c = 0; c < C; c += 2) w[c / 2] = pack_bf16x2(m.acc[c] * inv, m.acc[c + 1] * inv);
#pragma unroll
    for (int c = 0; c < C / 2; c += 4)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + at + 2 * c) =
          make_uint4(w[c], w[c + 1], w[c + 2], w[c + 3]);
  } else {
#pragma unroll
    for (int c = 0; c < C; c += 4)
      *reinterpret_cast<float4*>(static_cast<float*>(p.o) + at + c) =
          make_float4(m.acc[c] * inv, m.acc[c + 1] * inv, m.acc[c + 2] * inv, m.acc[c + 3] * inv);
  }
  if (part == 0) p.lse[row] = m.lse();
}

template <int D, int RB>
cudaError_t launch_steps(const PagedArgs& a, const PagedStep& p, int ctas, cudaStream_t stream) {
  using L = StepLayout<D, RB>;
  auto kern = paged_steps_kernel<D, RB>;
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = setup_kernel_once(kern, L::kSmemBytes, 0, ready);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kern, dim3(ctas), kStepThreads, L::kSmemBytes, stream, a.st_k, a.st_v, a.st_k16, a.st_v16,
                           p);
}

// Warps a row: as many as the rows leave room for on the GPU at once, for the
// rows with the most partial results are those of the smallest batches.  (Whole
// calls with 8 / 4 / 1 warps: one sequence of 16384 keys, one key head, 10.1 /
// 13.2 / 54.7 us; one of 4000 keys, 8 key heads, 8.3 / 8.6 / 14.9; 64 of 300 keys 17.0
// / 15.1 / 14.1.)
template <int D>
cudaError_t launch_merge_rows(const PagedCombine& p, int sms, cudaStream_t stream) {
  constexpr int RPW = 2;
  const long long rows = static_cast<long long>(p.units) * p.part.slot_rows;
  const long long groups = static_cast<long long>(p.units) * ((p.part.slot_rows + RPW - 1) / RPW);
  const long long room = 4LL * sms;
  auto launch = [&](auto kern, long long items, int per_block) {
    return launch_overlapped(kern, dim3(static_cast<unsigned>((items + per_block - 1) / per_block)), 256, 0, stream, p);
  };
  if (rows <= room) return launch(merge_rows_kernel<D, 8, 1>, rows, 1);
  if (rows <= 2 * room) return launch(merge_rows_kernel<D, 4, 1>, rows, 2);
  return launch(merge_rows_kernel<D, 1, RPW>, groups, 8);
}

// Eight warps to a row group's 16 columns while that leaves every CTA its own
// room on the GPU.  (Whole calls with 8 / 1: 64 rows of 8 heads, 4096 keys, 15.5 and
// 27.2 us; 16 sequences behind a prefix of 2048 keys 16.4 and 21.5; the long
// chunk 388 and 323, 256 sequences behind a prefix 270 and 247.)
template <int D, bool STEPS>
cudaError_t launch_merge_lanes(const PagedCombine& p, int sms, cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.seq.B) * p.seq.G * p.seq.Nq;
  const long long groups = STEPS ? p.seq.Hkv * ((rows + 31) / 32)
                                 : static_cast<long long>(p.units) * (rows_of_unit(p.part) / 32);
  auto launch = [&](auto kern, long long blocks) {
    return launch_overlapped(kern, dim3(static_cast<unsigned>(blocks)), 256, 0, stream, p);
  };
  if (groups * (D / 16) <= 4LL * sms) return launch(merge_lanes_kernel<D, 8, STEPS>, groups * (D / 16));
  constexpr int PER = 128 / D;  // row groups a CTA
  return launch(merge_lanes_kernel<D, 1, STEPS>, (groups + PER - 1) / PER);
}

// How a call is divided, and where its partial results lie in the workspace
// (offsets in 4-byte words).
struct Plan {
  int rows, pairs;            // rows a key head of a sequence, and its row pairs
  bool steps;                 // the sequences' own keys: the step kernel, else the tile kernel
  int chunk;                  // sequences a launch of the step kernel
  int prefix_pairs;           // row pairs of all sequences' rows
  size_t own_slots, prefix_slots;
  size_t own, prefix, words;
};

Plan make_plan(int B, int Hkv, int G, int Nq, int d, bool with_prefix) {
  Plan x;
  x.rows = G * Nq;
  x.pairs = (x.rows + kPairRows - 1) / kPairRows;
  x.steps = paged_uses_steps(G, Nq);
  x.chunk = B < kLineSequences ? B : kLineSequences;
  if (x.steps)
    x.own_slots = static_cast<size_t>(x.chunk) * Hkv + kMaxCtas;
  else if (with_prefix)
    x.own_slots = static_cast<size_t>(B) * Hkv * x.pairs + kMaxTileCtas;
  else
    x.own_slots = 2 * kMaxTileCtas;
  const size_t own_words = x.own_slots * (x.steps ? x.rows : kPairRows) * (d + 1);
  x.prefix_pairs = static_cast<int>((static_cast<long long>(B) * x.rows + kPairRows - 1) / kPairRows);
  x.prefix_slots = with_prefix ? static_cast<size_t>(x.prefix_pairs) * Hkv + kMaxTileCtas : 0;
  x.own = 2 * kLineWords;     // the lines' tables
  x.prefix = x.own + (own_words + 3) / 4 * 4;
  x.words = x.prefix + x.prefix_slots * kPairRows * (d + 1);
  return x;
}

// Heads whose units are dealt out together: as many as keep their keys and
// values (of at most `keys` keys a head) within 32 MB of L2, and at least one
// round's.
int head_group(long long heads, int pairs, long long keys, int d, int ctas) {
  long long g = (32LL << 20) / (keys * d * 4);
  const long long round = (ctas + pairs - 1) / pairs;
  if (g < round) g = round;
  return static_cast<int>(g > heads ? heads : g);
}

template <int D>
cudaError_t launch_paged_d(const PagedArgs& a, cudaStream_t stream) {
  const int G = a.Hq / a.Hkv;
  const bool with_prefix = a.prefix_len > 0;
  const Plan x = make_plan(a.B, a.Hkv, G, a.Nq, D, with_prefix);
  const int per_sm = x.rows <= 8 ? step_ctas_per_sm<1>() : step_ctas_per_sm<4>();
  const int step_ctas = per_sm * a.sms < kMaxCtas ? per_sm * a.sms : kMaxCtas;
  const int tile_ctas = a.sms < kMaxTileCtas ? a.sms : kMaxTileCtas;
  int* line = reinterpret_cast<int*>(a.part);
  const int capacity = a.table.max_pages * a.table.page_size;
  const PagedSeq all{a.seqlens_q, a.seqlens_k, a.B, a.Hkv, G, a.Nq, capacity, a.prefix_len};
  // the tile kernel on `heads` row spaces of `pairs` row pairs; the workspace
  // from `at` on holds `slots` slots
  auto tiles = [&](PagedTiles& t, bool prefix, int heads, int pairs, int keys, bool direct, bool dual, size_t at,
                   size_t slots, int* table) -> cudaError_t {
    t.seq = all;
    t.table = a.table;
    t.q = a.q;
    t.o = a.o;
    t.o_bf16 = a.o_bf16;
    t.lse = a.lse;
    const int units = heads * pairs;
    const int cut = units < 2 * tile_ctas ? units : tile_ctas + units % tile_ctas;
    t.line_out = table;
    t.counter = table + kTileLine + 3;
    const int piece_cost = !prefix && !dual && 2 * units >= tile_ctas ? kTilePieceCost : 0;
    t.part = PartRef{table, tile_ctas, kMinTiles, cut, direct, piece_cost, kPairRows, dual, units, heads,
                     pairs, head_group(heads, pairs, keys, D, tile_ctas), a.part + at,
                     a.part + at + slots * kPairRows * D};
    t.box_rows = a.box_rows;
    t.causal = a.causal;
    t.scale_log2 = a.scale_log2;
    t.status = a.status;
    t.wait_limit_ns = a.wait_limit_ns;
    t.stall_unit = a.stall_unit;
    return cut < units ? cudaMemsetAsync(t.counter, 0, sizeof(int), stream) : cudaSuccess;
  };
  PagedCombine c{};
  c.direct = !with_prefix;
  c.o_bf16 = a.o_bf16;
  cudaError_t e;
  if (with_prefix) {
    PagedTiles t{};
    e = tiles(t, true, a.Hkv, x.prefix_pairs, a.prefix_len, false, static_cast<long long>(a.B) * x.rows <= kTileRows,
              x.prefix, x.prefix_slots, line + kLineWords);
    if (e != cudaSuccess) return e;
    t.prefix_table = a.prefix_table;
    t.boxed_rows = a.boxed_rows;
    t.wait_first = 1;
    e = launch_tiles(t, a.tm_qp, a.tm_k, a.tm_v, D, tile_ctas, stream);
    if (e != cudaSuccess) return e;
    c.prefix = t.part;
  }
  if (!x.steps) {
    PagedTiles t{};
    e = tiles(t, false, a.B * a.Hkv, x.pairs, capacity, !with_prefix, x.rows <= kTileRows, x.own, x.own_slots, line);
    if (e != cudaSuccess) return e;
    t.direct = c.direct;
    t.boxed_rows = 1;
    // (behind a memset the launch does not overlap with the prefix's)
    t.wait_first = !with_prefix || t.part.cut < t.part.units;
    e = launch_tiles(t, a.tm_q, a.tm_k, a.tm_v, D, tile_ctas, stream);
    if (e != cudaSuccess) return e;
    c.seq = all;
    c.part = t.part;
    c.units = c.direct ? t.part.cut : t.part.units;
    c.o = a.o;
    c.lse = a.lse;
    return launch_merge_lanes<D, false>(c, a.sms, stream);
  }
  for (int b0 = 0; b0 < a.B; b0 += x.chunk) {
    const int n = a.B - b0 < x.chunk ? a.B - b0 : x.chunk;
    const size_t first = static_cast<size_t>(b0) * a.Hq * a.Nq;
    PagedStep p;
    p.seq = all;
    p.seq.B = n;
    if (p.seq.seqlens_q) p.seq.seqlens_q += b0;
    if (p.seq.seqlens_k) p.seq.seqlens_k += b0;
    p.table = a.table;
    p.table.block_table += b0 * a.table.table_stride;
    p.q = a.q + first * D;
    p.o = static_cast<uint8_t*>(a.o) + first * D * (a.o_bf16 ? 2 : 4);
    p.o_bf16 = a.o_bf16;
    p.lse = a.lse + first;
    p.line_out = line;
    p.part = PartRef{line,        step_ctas, kMinSteps, n, 0, 0, x.rows, 0, n * a.Hkv, 0, 0, 0, a.part + x.own,
                     a.part + x.own + x.own_slots * x.rows * D};
    p.direct = c.direct;
    p.wait_first = !with_prefix || b0 > 0;
    p.box_rows = a.box_rows;
    p.b0 = b0;
    p.causal = a.causal;
    p.scale_log2 = a.scale_log2;
    p.status = a.status;
    p.wait_limit_ns = a.wait_limit_ns;
    p.stall_unit = a.stall_unit;
    e = x.rows <= 8    ? launch_steps<D, 1>(a, p, step_ctas, stream)
        : x.rows <= 16 ? launch_steps<D, 2>(a, p, step_ctas, stream)
        : x.rows <= 24 ? launch_steps<D, 3>(a, p, step_ctas, stream)
                       : launch_steps<D, 4>(a, p, step_ctas, stream);
    if (e != cudaSuccess) return e;
    c.seq = p.seq;
    c.part = p.part;
    c.units = p.part.units;
    c.b0 = b0;
    c.o = p.o;
    c.lse = p.lse;
    e = with_prefix ? launch_merge_lanes<D, true>(c, a.sms, stream) : launch_merge_rows<D>(c, a.sms, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

bool paged_uses_steps(int G, int Nq) { return static_cast<long long>(G) * Nq <= kStepRows; }

size_t paged_workspace_floats(int B, int Hkv, int G, int Nq, int d, bool with_prefix) {
  return make_plan(B, Hkv, G, Nq, d, with_prefix).words;
}

cudaError_t launch_paged(const PagedArgs& a, cudaStream_t stream) {
  return a.d == 64 ? launch_paged_d<64>(a, stream) : launch_paged_d<128>(a, stream);
}

}  // namespace fa
