// Attention over the paged cache in E4M3 for few rows a key head: single tokens
// and drafted ones of every query head of its group.
//
// A stored key or value is its E4M3 number times the scale of its 16 tokens
// and head.  With scores z_j = scale * sk_j (q . k_j) and weights p_j = 2^z_j the
// row is O = sum p_j sv_j v_j / sum p_j.  Both products run on fp16 (mma with fp32
// sums), in which every E4M3 number is exact, with the scales outside:
//
//  - A query row is taken times a power of two that brings its largest value into
//    [2^14, 2^15): exact but for elements below 2^-28 of it.
//  - The exponent of a weight takes the values' scale in: x_j = z_j + log2 sv_j, and
//    w_j = 2^(x_j - max x + 14) with the maximum over the tile's 128 keys, in 11
//    significand bits, and 2^-39 of the tile's largest at the least.  The row's
//    accumulator follows: it is in units of 2^(the last tile's maximum), or of 2^-60
//    times the largest so far where that is more (what a tile adds below that is
//    nothing).  The sum of the p_j takes w_j / sv_j.
//
// (With mma on E4M3 operands for the score product instead 8 sequences x 8 heads x
// 8192 keys were 35 us with up to 8 rows and 61 with 16, the long case below 351.)
//
// paged_steps_fp8_kernel: the work is divided as in paged_steps_kernel (paged.cu),
// with tiles of 128 keys, the same number of bytes.  Each compute warp multiplies
// the rows with its 32 keys, the warps agree on the tile's row maxima, exchange
// the weights through shared memory, and each multiplies all 128 keys with its
// quarter of the value columns.  The transposed value fragments come by ldmatrix
// of 16 x 16 bytes.  Fragments are converted where they are: a word holds four
// numbers in a row, which become two pairs, so an mma's 16 columns are taken in the
// order 0 1 4 5 8 9 12 13 2 3 6 7 10 11 14 15 on both sides.  A lane's four keys of
// the score product are those of one word of the value fragments: key 8 j + (i ^
// 2 j), j < 4, of a warp's 32 for line i of the fragments, an order in which the
// rows that one ldmatrix phase reads lie in different banks for keys and values
// both.
//
// Bound by HBM where there are keys enough: 8 sequences x 32 heads x 32768 keys, one
// row a head, 308 to 313 us = 6.9 to 7.0 TB/s of keys and values (a step reads only, the copy that
// peaks are taken from writes too).  32 sequences of 100 to 16384 keys, 32 heads on 4,
// 23.6 to 25.1 us, of which about 9 are the start (lengths, page ids, first tiles) and the
// merge; one sequence of 1000 keys 8.5 us in a graph, all latency.  8 sequences x 8
// heads x 8192 keys 29.4 us with 1 to 8 rows a head, 35.5 with 16, 42 with 24 and 57
// with 32 (bf16 48, 50, 55, 62): with more rows the warps' instructions bound it, and
// registers, of which a thread has 168 (100 to 300 bytes spill from 9 rows on).  Tensor pipe 18%, issue
// slots 35% in the long case.
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "paged.cuh"
#include "ptx_e4m3.cuh"
#include "serving.h"

namespace fa {
namespace {

constexpr int kKeys = 128;            // keys a tile
constexpr int kWarpKeys = kKeys / kStepWarps;
constexpr int kTileScales = kKeys / kScaleTokens;
constexpr float kLn2 = 0.6931471805599453f;

enum StepSite : int { SITE_STEP8_EMPTY = 82, SITE_STEP8_FULL = 83 };

// RB: blocks of 8 query rows.
template <int D, int RB>
struct StepLayout {
  // keys (or values) of a tile: a row of D bytes a key, swizzled
  static constexpr int kHalf = kKeys * D;
  static constexpr int kStage = 2 * kHalf;
  static constexpr bool kMany = RB > 2;   // 17 rows or more
  static constexpr int kStages = (RB == 2 ? 3 : 2) * (128 / D);
  // weights: [8 RB rows][128 keys] fp16 and 16 bytes more a row, so that rows
  // begin in different banks
  static constexpr int kPRow = 2 * kKeys + 16;
  static constexpr int kPOff = kStages * kStage;
  // queries (17 rows or more): [8 RB rows][d] fp16 and 16 bytes more a row, then the
  // rows' multipliers
  static constexpr int kQRow = 2 * D + 16;
  static constexpr int kQOff = kPOff + 8 * RB * kPRow;
  static constexpr int kCqOff = kQOff + (kMany ? 8 * RB * kQRow : 0);
  // a stage's scales: of the keys' groups of 16, then of the values'
  static constexpr int kScaleOff = kCqOff + (kMany ? 8 * RB * 4 : 0);
  static constexpr int kBarOff = kScaleOff + kStages * 2 * kTileScales * 4;  // FULL[s] then EMPTY[s]
  static constexpr int kMaxOff = kBarOff + 2 * kStages * 8;                  // [warps][8 RB] row maxima, row sums
  static constexpr int kMiscOff = kMaxOff + 2 * kStepWarps * 8 * RB * 4;
  // first tile of every sequence, then lk, then lq (a byte: at most 32 here)
  static constexpr int kLineOff = kMiscOff + 16;
  static constexpr int kSmemBytes = kLineOff + (2 * kLineSequences + 1) * 4 + kLineSequences + 1024;
  static_assert(step_ctas_per_sm<RB>() * (kSmemBytes + 1024) <= 228 * 1024, "resident CTAs an SM");
};

// Byte offset of 16-byte chunk c of key r in a tile.  Chunk c's is chunk 0's XOR
// 16 c, also behind the tile's 1024-byte aligned address.
template <int D>
__device__ __forceinline__ uint32_t row_chunk(int r, int c) {
  return D == 128 ? sw128(r, c) : sw64(r, c);
}

// Two 16 x 16 matrices of bytes, transposed: words 0 and 1 of lane 4 c + i are
// bytes c and c + 8 of rows 4 i to 4 i + 3 of the first, 2 and 3 of the second.
template <int OFF>
__device__ __forceinline__ void ldmatrix2_t8(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4+%5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(OFF)
               : "memory");
}

// c (16 x 8, fp32) += a (16 x 16) b (16 x 8), fp16
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The fp16 fragment of 16 columns from words of lines fr and fr + 8.
__device__ __forceinline__ void widen(uint32_t (&a)[4], uint32_t upper, uint32_t lower) {
  e4m3x4_to_f16(upper, a[0], a[2]);
  e4m3x4_to_f16(lower, a[1], a[3]);
}

// 4 bytes global -> shared without registers; `bytes` 0 writes zeros.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// This thread's arrival on the barrier when its copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <int D, int RB>
__global__ void __launch_bounds__(kStepThreads, step_ctas_per_sm<RB>())
    paged_steps_fp8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ CUtensorMap tm_k16, const __grid_constant__ CUtensorMap tm_v16,
                           const __grid_constant__ PagedStep p) {
  using L = StepLayout<D, RB>;
  constexpr int S = L::kStages;
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
      mbar_init(bars + 8 * s, 1 + 32);  // the tile's bytes, and every lane's scale
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
    return lq > 0 && lk > p.seq.prefix_len ? (lk - p.seq.prefix_len + kKeys - 1) / kKeys : 0;
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
    // lane i of a tile's loads: operand and box of rows, and operand and group of
    // 16 keys whose scale it fetches
    const int boxes = kKeys / p.box_rows;
    const int groups = p.table.page_size / kScaleTokens;  // of a page
    const int group = lane % kTileScales;
    const float* scales = lane < kTileScales ? p.k_scales : p.v_scales;
    int issued = 0;
    bool ok = true;
    // page of box i of a piece; -1 behind the sequence's end
    auto page_of = [&](const Walk& x, int i) {
      const int key = p.seq.prefix_len + x.tile * kKeys + i * p.box_rows;
      return i < (x.end - x.tile) * boxes && key < len_k[x.e]
                 ? p.table.block_table[x.e * p.table.table_stride + key / p.table.page_size]
                 : -1;
    };
    // pages are looked up 32 boxes ahead: the next ones of this piece, and the
    // first of the piece after it
    int ahead = more ? page_of(w, lane) : -1;
    while (more && ok) {
      const int lk = len_k[w.e];
      const int first = p.seq.prefix_len + w.tile * kKeys;
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
                        wait_bounded(bars + 8 * (S + s), ((issued / S) & 1) ^ 1, wc, SITE_STEP8_EMPTY, unit));
        if (!ok) break;
        // a sequence's last tile comes in boxes of 16 rows, so that at most 15
        // rows behind its last key are read
        const int key0 = first + t * kKeys;
        const bool tail = key0 + kKeys > lk;
        const int rows_box = tail ? 16 : p.box_rows;
        const int count = kKeys / rows_box;              // boxes an operand; one lane loads each
        const int value = lane >= count;
        const int row = (lane - value * count) * rows_box;
        const int page = __shfl_sync(0xffffffffu, cur, (t * boxes + row / p.box_rows) % 32);
        const int scale_key = key0 + group * kScaleTokens;
        const int scale_page = __shfl_sync(0xffffffffu, cur, (t * boxes + group * kScaleTokens / p.box_rows) % 32);
        if (unit == p.stall_unit && issued == 0) continue;  // testing hook: leave this tile unloaded
        const uint32_t full = bars + 8 * s;
        if (lane == 0) mbar_arrive_expect_tx(full, L::kStage);
        __syncwarp();
        if (lane < 2 * count) {
          const int key = key0 + row;
          // rows of no page: a coordinate past the map, which reads zeros
          int outer = p.table.num_pages * p.seq.Hkv;
          if (key < lk) {
            if (page >= 0 && page < p.table.num_pages)
              outer = page * p.seq.Hkv + w.head;
            else
              record_bad_page(p.status, SITE_PAGE_READ, p.b0 + w.e, page);
          }
          const CUtensorMap* tm = value ? (tail ? &tm_v16 : &tm_v) : (tail ? &tm_k16 : &tm_k);
          tma_load_3d(sbase + s * L::kStage + value * L::kHalf + row * D, tm, full, 0, key % p.table.page_size,
                      outer);
        }
        if (lane < 2 * kTileScales) {
          const bool live = scale_key < lk && scale_page >= 0 && scale_page < p.table.num_pages;
          const long long cell = (static_cast<long long>(scale_page) * p.seq.Hkv + w.head) * groups +
                                 scale_key % p.table.page_size / kScaleTokens;
          cp_async4(sbase + L::kScaleOff + (s * 2 * kTileScales + lane) * 4, live ? scales + cell : scales,
                    live ? 4u : 0u);
        }
        cp_async_arrive(full);
        __syncwarp();
      }
      if (ok) more = walk_next(w, starts, p.seq.Hkv, at, stop);
    }
    if (!p.wait_first && lane == 0) grid_wait();
    cp_async_commit();
    cp_async_wait<0>();
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
  const int fr = lane >> 2;        // fragment line
  const int fc = (lane & 3) * 2;   // fragment columns: query rows fc, fc + 1 of a block
  const int rows = p.seq.G * p.seq.Nq;
  auto key_at = [](int i, int j) { return 8 * j + (i ^ (2 * j)); };  // of a warp's 32
  // ldmatrix lane addresses: keys (two groups of 16 rows), values
  uint32_t k_off[2];
#pragma unroll
  for (int g = 0; g < 2; ++g)
    k_off[g] = row_chunk<D>(kWarpKeys * warp + key_at(lane & 7, 2 * g + ((lane >> 3) & 1)), lane >> 4);
  const int v_col = warp * (D / 4);  // first value column of this warp
  const uint32_t v_off = row_chunk<D>(key_at(lane >> 2, lane & 3), v_col / 16);
  // weights: where the lane's four keys of row fc go, and 8 keys of a row for the
  // product
  const uint32_t p_store = sbase + L::kPOff + fc * L::kPRow + 2 * kWarpKeys * warp + 32 * (fr >> 2) + 4 * (fr & 3);
  const uint32_t p_load = sbase + L::kPOff + (lane & 7) * L::kPRow + 16 * (lane >> 3);
  constexpr bool MANY = L::kMany;
  constexpr int QB = MANY ? 1 : RB;  // blocks of rows whose queries a warp loads: one, for all warps, or all
  uint32_t qf[QB][KS][2];
  uint2 raw[QB][KS];
  float cq[QB][2];                 // what a score of rows fc, fc + 1 is multiplied by
  float* cq_shared = reinterpret_cast<float*>(smem + L::kCqOff);
  [[maybe_unused]] const uint32_t q_load = sbase + L::kQOff + (lane & 7) * L::kQRow + 16 * (lane >> 3);
  auto load_q = [&](const Walk& x) {
    const uint16_t* base = p.q + (static_cast<size_t>(x.e) * p.seq.Hkv + x.head) * rows * D + 2 * fc;
#pragma unroll
    for (int m = 0; m < QB; ++m) {
      const int row = 8 * (MANY ? warp : m) + fr;
      const uint16_t* src = base + min(row, rows - 1) * D;  // rows of the block behind the last are not kept
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) raw[m][ks] = *reinterpret_cast<const uint2*>(src + 16 * ks);
    }
  };
  // the rows in fp16, and their multipliers; an infinity or a NaN in a row makes
  // its multiplier a NaN.  17 rows or more: into shared memory, when every warp is
  // through with the last ones.
  auto scale_q = [&]() {
#pragma unroll
    for (int m = 0; m < QB; ++m) {
      uint32_t top = 0;            // the largest magnitude's bits
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint2 x = raw[m][ks];
        top = max(top, max(max((x.x << 16) & 0x7fffffffu, x.x & 0x7fff0000u),
                           max((x.y << 16) & 0x7fffffffu, x.y & 0x7fff0000u)));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t e = max(top >> 23, 15u);  // the exponent's field
      const float up = __uint_as_float((268u - e) << 23);
      const float mine = e == 255u ? CUDART_NAN_F : __uint_as_float((e - 14u) << 23) * p.scale_log2;
#pragma unroll
      for (int i = 0; i < 2; ++i) cq[m][i] = __shfl_sync(0xffffffffu, mine, 4 * (fc + i));
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint2 x = raw[m][ks];
        qf[m][ks][0] = pack_f16x2(__uint_as_float(x.x << 16) * up, __uint_as_float(x.x & 0xFFFF0000u) * up);
        qf[m][ks][1] = pack_f16x2(__uint_as_float(x.y << 16) * up, __uint_as_float(x.y & 0xFFFF0000u) * up);
      }
      if constexpr (MANY) {
        if (warp < RB) {
          const uint32_t dst = sbase + L::kQOff + (8 * warp + fr) * L::kQRow + 2 * fc;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            st_shared_u32(dst + 32 * ks, qf[m][ks][0]);
            st_shared_u32(dst + 32 * ks + 16, qf[m][ks][1]);
          }
          if ((lane & 3) == 0) cq_shared[8 * warp + fr] = mine;
        }
        warps_sync();
      }
    }
  };
  int query[RB];  // query index of rows fc (low half) and fc + 1 of each block; past lq where there is no row
#pragma unroll
  for (int m = 0; m < RB; ++m) {
    const int r = 8 * m + fc;
    query[m] = (r < rows ? r % p.seq.Nq : 0x7fff) | (r + 1 < rows ? (r + 1) % p.seq.Nq : 0x7fff) << 16;
  }
  if (more) load_q(w);
  int done = 0;
  bool ok = true;
  while (more && ok) {
    const int lq = len_q[w.e], lk = len_k[w.e];
    int kend[RB][2];               // last visible key + 1 of rows fc, fc + 1
    // the largest x so far; the sum of the p_j and the accumulators, in units of 2^(ref - 14)
    float top[RB][2], ref[RB][2], l[RB][2], acc[RB][MT][4];
    scale_q();
#pragma unroll
    for (int m = 0; m < RB; ++m) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = (query[m] >> (16 * e)) & 0x7fff;
        kend[m][e] = i < lq ? (p.causal ? min(i + lk - lq + 1, lk) : lk) : 0;
        top[m][e] = ref[m][e] = -CUDART_INF_F;
        l[m][e] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < MT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][n][e] = 0.f;
    }
    // keys that every query of the sequence sees (rows behind the last may see any)
    const int all_see = lq < p.seq.Nq ? 0 : p.causal ? lk - lq + 1 : lk;
    Walk after = w;
    int after_at = at;
    const bool another = walk_next(after, starts, p.seq.Hkv, after_at, stop);
    for (int t = w.tile; t < w.end; ++t, ++done) {
      const int s = done % S;
      const bool full = wait_bounded(bars + 8 * s, (done / S) & 1, wc, SITE_STEP8_FULL, unit);
      const uint32_t kb = sbase + s * L::kStage;
      const uint32_t vb = kb + L::kHalf;
      const int key0 = p.seq.prefix_len + t * kKeys;
      const bool edge = key0 + kKeys > all_see;
      // x of this warp's 32 keys: [group][row block][key line fr of its first (0, 1) and second 8 keys]
      float x[2][RB][4], isv[2];
      if (__all_sync(0xffffffffu, full)) {
        const float* sc = reinterpret_cast<const float*>(smem + L::kScaleOff) + s * 2 * kTileScales + 2 * warp;
        const float2 sk = *reinterpret_cast<const float2*>(sc);
        const float2 sv = *reinterpret_cast<const float2*>(sc + kTileScales);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float sc[RB][4];
#pragma unroll
          for (int m = 0; m < RB; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[m][e] = 0.f;
#pragma unroll
          for (int ks = 0; ks < KS; ks += 2) {
            uint32_t w8[4], kf[2][4];
            ldmatrix4(w8, (kb + k_off[g]) ^ (16 * ks));
            widen(kf[0], w8[0], w8[1]);
            widen(kf[1], w8[2], w8[3]);
#pragma unroll
            for (int m = 0; m < RB; ++m) {
              if constexpr (MANY) {
                uint32_t qv[4];
                ldmatrix4(qv, q_load + (8 * m * L::kQRow + 32 * ks));
                mma_f16(sc[m], kf[0], qv[0], qv[1]);
                mma_f16(sc[m], kf[1], qv[2], qv[3]);
              } else {
                mma_f16(sc[m], kf[0], qf[m][ks][0], qf[m][ks][1]);
                mma_f16(sc[m], kf[1], qf[m][ks + 1][0], qf[m][ks + 1][1]);
              }
            }
          }
          // 2^log2 sv and its inverse come from the same rounded logarithm, so
          // that it drops out of the sum of the p_j
          const float kscale = g ? sk.y : sk.x, lsv = __log2f(g ? sv.y : sv.x);
          isv[g] = lsv == -CUDART_INF_F ? 0.f : ex2_approx(-lsv);  // (a group behind the last key)
#pragma unroll
          for (int m = 0; m < RB; ++m) {
            float2 c;
            if constexpr (MANY)
              c = *reinterpret_cast<const float2*>(cq_shared + 8 * m + fc);
            else
              c = make_float2(cq[m][0], cq[m][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[g][m][e] = fmaf(sc[m][e], (e & 1 ? c.y : c.x) * kscale, lsv);
              if (edge) {
                const int j = key0 + kWarpKeys * warp + key_at(fr, 2 * g + (e >> 1));
                if (j >= kend[m][e & 1]) x[g][m][e] = -CUDART_INF_F;
              }
            }
          }
        }
        if (key0 + kKeys > lk) {
          // rows behind the last key may hold anything: their weights are 0,
          // so their values must be finite
          // (whole boxes behind it were read as zeros)
          const int from = lk - key0, rest = -from & 15;
          if (from / kWarpKeys == warp) {
            for (int i = lane; i < rest * (D / 16); i += 32)
              st_shared_v4(vb + row_chunk<D>(from + i / (D / 16), i % (D / 16)), 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();  // before the slot's next TMA load
        }
#pragma unroll
        for (int m = 0; m < RB; ++m) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y = fmaxf(fmaxf(x[0][m][e], x[0][m][2 + e]), fmaxf(x[1][m][e], x[1][m][2 + e]));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
            if (lane < 4) maxima[warp * 8 * RB + 8 * m + fc + e] = y;
          }
        }
      }
      ok = warps_agree(full);
      if (!ok) break;
#pragma unroll
      for (int m = 0; m < RB; ++m) {
        float2 y = *reinterpret_cast<const float2*>(maxima + 8 * m + fc);
#pragma unroll
        for (int o = 1; o < kStepWarps; ++o) {
          const float2 z = *reinterpret_cast<const float2*>(maxima + o * 8 * RB + 8 * m + fc);
          y.x = fmaxf(y.x, z.x);
          y.y = fmaxf(y.y, z.y);
        }
        float wt[2][4];            // weights of the lane's four keys: rows fc, fc + 1
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mine = e ? y.y : y.x;
          top[m][e] = fmaxf(top[m][e], mine);
          const float next = fmaxf(mine, top[m][e] - 60.f);
          const float base = next == -CUDART_INF_F ? 0.f : next;
          const float f = ex2_approx(ref[m][e] - base);  // 0 before the first visible key
          ref[m][e] = next;
          float sum = 0.f;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            wt[e][2 * g] = ex2_approx(x[g][m][e] - base + 14.f);
            wt[e][2 * g + 1] = ex2_approx(x[g][m][2 + e] - base + 14.f);
            sum = fmaf(wt[e][2 * g] + wt[e][2 * g + 1], isv[g], sum);
          }
          l[m][e] = fmaf(l[m][e], f, sum);
#pragma unroll
          for (int n = 0; n < MT; ++n) {
            acc[m][n][e] *= f;
            acc[m][n][2 + e] *= f;
          }
          const uint32_t at = p_store + (8 * m + e) * L::kPRow;
          st_shared_u32(at, pack_f16x2(wt[e][0], wt[e][1]));
          st_shared_u32(at + 16, pack_f16x2(wt[e][2], wt[e][3]));
        }
      }
      warps_sync();
      // O^T += V^T W^T: all 128 keys, this warp's quarter of the columns
      auto keys32 = [&](auto tag) {
        constexpr int KK = decltype(tag)::value;
        uint32_t vf[MT][2][4];
#pragma unroll
        for (int n = 0; n < MT; ++n) {
          uint32_t w8[4];
          ldmatrix2_t8<32 * KK * D>(w8, (vb + v_off) ^ (16 * n));
          widen(vf[n][0], w8[0], w8[1]);
          widen(vf[n][1], w8[2], w8[3]);
        }
#pragma unroll
        for (int m = 0; m < RB; ++m) {
          uint32_t pf[4];  // 32 keys of eight rows
          ldmatrix4(pf, p_load + (8 * m * L::kPRow + 64 * KK));
#pragma unroll
          for (int n = 0; n < MT; ++n) {
            mma_f16(acc[m][n], vf[n][0], pf[0], pf[1]);
            mma_f16(acc[m][n], vf[n][1], pf[2], pf[3]);
          }
        }
      };
      keys32(std::integral_constant<int, 0>{});
      keys32(std::integral_constant<int, 1>{});
      keys32(std::integral_constant<int, 2>{});
      keys32(std::integral_constant<int, 3>{});
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
        float y = l[m][e];
        y += __shfl_xor_sync(0xffffffffu, y, 4);
        y += __shfl_xor_sync(0xffffffffu, y, 8);
        y += __shfl_xor_sync(0xffffffffu, y, 16);
        if (lane < 4) sums[warp * 8 * RB + 8 * m + fc + e] = y;
      }
    }
    warps_sync();
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
        // (sums are 0 only where no key is seen; a NaN goes through)
        const float s0 = sum.x != 0.f ? 1.f / sum.x : 0.f;
        const float s1 = sum.y != 0.f ? 1.f / sum.y : 0.f;
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
            const float u = odd ? got : a, v = odd ? b : got;
            if (valid) store_pair(dst + r * D + v_col + 16 * n + 8 * h + (fr & ~1), u, v);
          }
        }
        if (warp == 0 && fr < 2 && valid) {
          const float all = odd ? sum.y : sum.x;
          lse[r] = all != 0.f ? ((odd ? ref[m][1] : ref[m][0]) - 14.f + __log2f(all)) * unit : -CUDART_INF_F;
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

template <int D, int RB>
cudaError_t launch_t(const PagedArgs& a, const PagedStep& p, int ctas, cudaStream_t stream) {
  using L = StepLayout<D, RB>;
  auto kern = paged_steps_fp8_kernel<D, RB>;
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = setup_kernel_once(kern, L::kSmemBytes, 0, ready);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kern, dim3(ctas), kStepThreads, L::kSmemBytes, stream, a.st_k, a.st_v, a.st_k16, a.st_v16,
                           p);
}

template <int D>
cudaError_t launch_d(const PagedArgs& a, const PagedStep& p, int rows, int ctas, cudaStream_t stream) {
  return rows <= 8    ? launch_t<D, 1>(a, p, ctas, stream)
         : rows <= 16 ? launch_t<D, 2>(a, p, ctas, stream)
         : rows <= 24 ? launch_t<D, 3>(a, p, ctas, stream)
                      : launch_t<D, 4>(a, p, ctas, stream);
}

}  // namespace

cudaError_t launch_steps_fp8(const PagedArgs& a, const PagedStep& p, int rows, int ctas, cudaStream_t stream) {
  return a.d == 64 ? launch_d<64>(a, p, rows, ctas, stream) : launch_d<128>(a, p, rows, ctas, stream);
}

}  // namespace fa
