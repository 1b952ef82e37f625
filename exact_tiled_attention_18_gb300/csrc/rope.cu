// Rotary positions, and the append to the paged cache that applies them.
//
// A pair (a, b) of a head's values at position p becomes
//     a' = g (a cos t - b sin t),   b' = g (b cos t + a sin t),   t = p f_i,
// with one frequency f_i per pair and an amplitude g; the backward pass is
// the same with -t (the rotation is orthogonal, its transpose its inverse).
//
// The angle.  p reaches 10^6 and f_0 = 1 radian, so p * f in 32 bits would be
// wrong by 0.06 radians; in 64 bits it costs fp64 arithmetic, which this GPU
// has little of.  Only the angle modulo one turn matters, and multiplication
// modulo 2^64 gives exactly that: the frequency is held as turns * 2^-64 of a
// full turn, p * turns wraps around by itself, and the top 32 bits are the
// phase in [-1/2, 1/2) turns to 2^-32.  That phase as an fp32 number of half
// turns is off by at most 2^-26 turns (24 of its 31 bits, near half a turn),
// which is the largest part of the angle's error and no more than the sine's
// own.  The word's rounding leaves p * 2^-65 turns, the doubles that it is
// computed from about p * 2^-53: 2^-33 at p = 10^6.
//
// Both kernels are copies with a little arithmetic: bound by HBM bandwidth
// (two bytes in and two out per bf16 value) when large and by launch latency
// when small.  A thread owns 16 values of a token's head (8 pairs), computes
// their 8 sines and cosines once, and walks over heads with them, several
// heads' loads in flight at a time.
//
// Measured: 4 x 16 heads x 8192 tokens, d = 128, bf16, out of a fused projection
// 45.2 us = 5.9 TB/s, contiguous from bf16 to fp32 63 us = 6.4 TB/s, fp32 to
// fp32 81 us = 6.6 TB/s; 32 heads x 16384 tokens from fp32 to bf16, interleaved,
// 61.8 us = 6.5 TB/s; the append of four prompts of 2048 to 8192 tokens, 16 + 16
// + 16 heads, 75.9 us = 6.0 TB/s; a step of 8 sequences 2.1 us (rotation) and 2.5
// us (append) a call in a graph.  128 threads a block: 45.2, 61.7 and 79.8 us; half the heads in
// flight 47.3, 63.2, 76.0; twice as many 45.3, 61.9, 75.9; an append of three
// blocks an SM 86.5.
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <type_traits>

#include "internal.h"
#include "ptx_e4m3.cuh"
#include "serving.h"

namespace fa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kLowestScale = -32;  // a scale of the append's is at least 2^-32
constexpr int kAppendStages = 6;   // heads whose values are on their way or in use, in the append into E4M3
constexpr int kAppendStageBytes = 2 * kRopeThreads * 16;

// A lane's 16 values of a head are RUNS runs of as many bytes as one load
// takes, spread over the rotated part (or the part behind it) so that
// neighbouring lanes' runs are neighbours: run k of lane c is elements
//     base + k * span / RUNS + c * PER, ...      (PER = 16 / RUNS).
// Pairs never leave a lane: with the half layout element i of the first half
// of the runs belongs to element i of the second half, span / 2 further on;
// interleaved pairs are neighbours inside a run.  Eight values a run (16 bytes
// of bf16), four where fp32 is read or written.
template <int RUNS>
struct Lane {
  int at;           // first element of run 0
  int step;         // from run to run
  bool turns;       // false: the values behind rot_dim, copied
  float cs[8], sn[8];  // of pair i of the lane
};

template <int RUNS>
__device__ __forceinline__ Lane<RUNS> make_lane(const RopeRef& r, int d, int c, bool rotate) {
  constexpr int PER = 16 / RUNS;
  Lane<RUNS> l;
  const int turned = rotate ? r.rot_dim : 0;
  l.turns = 16 * c < turned;
  const int span = l.turns ? turned : d - turned;
  l.at = l.turns ? PER * c : turned + PER * (c - turned / 16);
  l.step = span / RUNS;
  return l;
}

// REST: with what the phase's rounding to fp32 leaves, to first order, so that
// sine and cosine are as near as fp32 holds them.  For keys that are rounded to
// E4M3 at once, of whose values next to the middle of two numbers fewer go to the
// farther one (of 30 batches' 96 without, 59 so, 54 with angles in 64 bits).
template <bool REST = false, int RUNS>
__device__ __forceinline__ void set_angles(Lane<RUNS>& l, const RopeRef& r, int position, float sign) {
  if (!l.turns) return;
  constexpr int PER = 16 / RUNS;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // pair i: element i of the lane's first eight (half), or elements 2i, 2i+1
    const int e = r.interleaved ? 2 * i : i;
    const int element = l.at + (e / PER) * l.step + e % PER;
    const unsigned long long f = static_cast<unsigned long long>(__ldg(r.turns + (r.interleaved ? element / 2 : element)));
    const unsigned long long phase = static_cast<unsigned long long>(static_cast<long long>(position)) * f;
    const int word = static_cast<int>(phase >> 32);
    const float rounded = static_cast<float>(word);
    const float half_turns = rounded * 4.656612873077393e-10f;  // 2^-31
    float s, co;
    sincospif(half_turns, &s, &co);
    if constexpr (REST) {
      const float rest = static_cast<float>(word - __float2int_rn(rounded)) * 1.4629180792671596e-9f;  // pi 2^-31
      const float t = s;
      s = fmaf(co, rest, s);
      co = fmaf(-t, rest, co);
    }
    l.cs[i] = co * r.amplitude;
    l.sn[i] = s * (r.amplitude * sign);
  }
}

template <int RUNS>
__device__ __forceinline__ void turn(const Lane<RUNS>& l, bool interleaved, float (&v)[16]) {
  if (!l.turns) return;
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = v[2 * i], b = v[2 * i + 1];
      v[2 * i] = a * l.cs[i] - b * l.sn[i];
      v[2 * i + 1] = b * l.cs[i] + a * l.sn[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = v[i], b = v[8 + i];
      v[i] = a * l.cs[i] - b * l.sn[i];
      v[8 + i] = b * l.cs[i] + a * l.sn[i];
    }
  }
}

// A lane's values as they lie in memory: 8 words of bf16, 16 of fp32.
template <bool BF16>
struct Raw {
  uint32_t w[BF16 ? 8 : 16];
};

template <bool BF16, int RUNS>
__device__ __forceinline__ Raw<BF16> load(const void* base, long long row, const Lane<RUNS>& l) {
  constexpr int PER = 16 / RUNS;
  Raw<BF16> x;
#pragma unroll
  for (int k = 0; k < RUNS; ++k) {
    const long long i = row + l.at + k * l.step;
    if constexpr (!BF16) {
      static_assert(BF16 || PER == 4, "fp32 comes in runs of four");
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const float*>(base) + i);
      x.w[4 * k] = v.x, x.w[4 * k + 1] = v.y, x.w[4 * k + 2] = v.z, x.w[4 * k + 3] = v.w;
    } else if constexpr (PER == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
      x.w[4 * k] = v.x, x.w[4 * k + 1] = v.y, x.w[4 * k + 2] = v.z, x.w[4 * k + 3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
      x.w[2 * k] = v.x, x.w[2 * k + 1] = v.y;
    }
  }
  return x;
}

template <bool BF16>
__device__ __forceinline__ void unpack(const Raw<BF16>& x, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if constexpr (BF16)
      v[i] = __uint_as_float(i & 1 ? x.w[i / 2] & 0xFFFF0000u : x.w[i / 2] << 16);
    else
      v[i] = __uint_as_float(x.w[i]);
  }
}

// The values rounded once when the output is bf16.
template <bool BF16>
__device__ __forceinline__ Raw<BF16> pack(const float (&v)[16]) {
  Raw<BF16> x;
#pragma unroll
  for (int i = 0; i < (BF16 ? 8 : 16); ++i) {
    if constexpr (BF16)
      x.w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    else
      x.w[i] = __float_as_uint(v[i]);
  }
  return x;
}

// Four E4M3 numbers times r, rounded to E4M3.
__device__ __forceinline__ uint32_t scale_e4m3x4(uint32_t packed, float r) {
  float v[4];
  unpack_e4m3x4(packed, v);
  return pack_e4m3x4(v[0] * r, v[1] * r, v[2] * r, v[3] * r);
}

template <bool BF16, int RUNS>
__device__ __forceinline__ void store(void* base, long long row, const Lane<RUNS>& l, const Raw<BF16>& x) {
  constexpr int PER = 16 / RUNS;
#pragma unroll
  for (int k = 0; k < RUNS; ++k) {
    const long long i = row + l.at + k * l.step;
    if constexpr (!BF16)
      *reinterpret_cast<uint4*>(static_cast<float*>(base) + i) =
          make_uint4(x.w[4 * k], x.w[4 * k + 1], x.w[4 * k + 2], x.w[4 * k + 3]);
    else if constexpr (PER == 8)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) =
          make_uint4(x.w[4 * k], x.w[4 * k + 1], x.w[4 * k + 2], x.w[4 * k + 3]);
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + i) = make_uint2(x.w[2 * k], x.w[2 * k + 1]);
  }
}

template <int D, bool XBF, bool YBF>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_kernel(const RopeArgs a, const int heads_per_thread) {
  constexpr int LANES = D / 16;
  constexpr int RUNS = XBF && YBF ? 2 : 4;
  constexpr int HEADS = XBF ? 4 : 2;  // heads in flight: 128 bytes a thread
  grid_trigger();
  const long long item = static_cast<long long>(blockIdx.x) * (kRopeThreads / LANES) + threadIdx.x / LANES;
  if (item >= static_cast<long long>(a.B) * a.N) return;
  const int c = threadIdx.x % LANES;
  const int b = static_cast<int>(item / a.N);
  const int n = static_cast<int>(item - static_cast<long long>(b) * a.N);
  const int h0 = blockIdx.y * heads_per_thread;
  const int h1 = min(h0 + heads_per_thread, a.H);
  const int position = a.rope.positions ? __ldg(a.rope.positions + b * a.rope.positions_sb + n) : n;
  Lane<RUNS> l = make_lane<RUNS>(a.rope, D, c, true);
  set_angles(l, a.rope, position, a.inverse ? -1.f : 1.f);
  const long long xo = b * a.xs.b + n * a.xs.n;
  const long long yo = b * a.ys.b + n * a.ys.n;
  for (int h = h0; h < h1; h += HEADS) {
    Raw<XBF> raw[HEADS];
#pragma unroll
    for (int u = 0; u < HEADS; ++u)
      if (h + u < h1) raw[u] = load<XBF>(a.x, xo + (h + u) * a.xs.h, l);
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
      if (h + u < h1) {
        float v[16];
        unpack<XBF>(raw[u], v);
        turn(l, a.rope.interleaved, v);
        store<YBF>(a.y, yo + (h + u) * a.ys.h, l, pack<YBF>(v));
      }
    }
  }
}

// Heads of the append in one line: Hq of q (none without q), Hkv of k, Hkv
// of v.
template <int D>
__global__ void __launch_bounds__(kRopeThreads) append_kernel(const AppendArgs a, const int heads_per_thread) {
  constexpr int LANES = D / 16;
  constexpr int RUNS = 2, HEADS = 4;
  grid_trigger();
  const long long item = static_cast<long long>(blockIdx.x) * (kRopeThreads / LANES) + threadIdx.x / LANES;
  if (item >= static_cast<long long>(a.B) * a.N) return;
  const int c = threadIdx.x % LANES;
  const int b = static_cast<int>(item / a.N);
  const int t = static_cast<int>(item - static_cast<long long>(b) * a.N);
  // (the keys' number as it is given, not cut to what the table holds: a token
  // past the table's end must not come to lie on an earlier one's row)
  int lq, lk;
  paged_lens(a.seqlens_q, a.seqlens_k, b, a.N, INT_MAX, lq, lk);
  if (t >= lq) return;  // padding: nothing of it is written
  const int place = lk - lq + t;
  const int hq = a.q ? a.Hq : 0;
  const int heads = hq + 2 * a.Hkv;
  const int h0 = blockIdx.y * heads_per_thread;
  const int h1 = min(h0 + heads_per_thread, heads);
  // the row of the cache; a token before position 0 or past the table's end,
  // or one whose page does not exist, has none
  long long row = -1;
  if (h1 > hq && place >= a.table.max_pages * a.table.page_size) {
    if (c == 0) record_bad_page(a.status, SITE_PAGE_PAST_TABLE, b, place);
  } else if (h1 > hq && place >= 0) {
    const int page = __ldg(a.table.block_table + b * a.table.table_stride + place / a.table.page_size);
    if (page >= 0 && page < a.table.num_pages)
      row = (static_cast<long long>(page) * a.Hkv) * a.table.page_size + place % a.table.page_size;
    else if (c == 0)
      record_bad_page(a.status, SITE_PAGE_APPEND, b, page);
  }
  Lane<RUNS> l = make_lane<RUNS>(a.rope, D, c, a.rope.rot_dim > 0);
  if (h0 < hq + a.Hkv) {
    const int position = a.rope.positions ? __ldg(a.rope.positions + b * a.rope.positions_sb + t) : place;
    set_angles(l, a.rope, position, 1.f);
  }
  for (int h = h0; h < h1; h += HEADS) {
    Raw<true> raw[HEADS];
    uint16_t* dst[HEADS];  // null: no such head, or no row of the cache
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
      const int g = h + u;
      dst[u] = nullptr;
      if (g < h1) {
        const uint16_t* src;
        if (g < hq) {
          src = a.q + b * a.qs.b + g * a.qs.h + t * a.qs.n;
          dst[u] = a.q_out + ((static_cast<long long>(b) * a.Hq + g) * a.N + t) * D;
        } else {
          const bool value = g >= hq + a.Hkv;
          const int kh = g - hq - (value ? a.Hkv : 0);
          src = value ? a.v + b * a.vs.b + kh * a.vs.h + t * a.vs.n : a.k + b * a.ks.b + kh * a.ks.h + t * a.ks.n;
          if (row >= 0)
            dst[u] = (value ? a.v_pages : a.k_pages) + (row + static_cast<long long>(kh) * a.table.page_size) * D;
        }
        raw[u] = load<true>(src, 0, l);
      }
    }
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
      if (dst[u]) {
        if (h + u < hq + a.Hkv && l.turns) {
          float v[16];
          unpack<true>(raw[u], v);
          turn(l, a.rope.interleaved, v);
          raw[u] = pack<true>(v);
        }
        store<true>(dst[u], 0, l, raw[u]);
      }
    }
  }
}

// The same into a cache in E4M3, whose cells (16 tokens of a page, one head, keys
// or values) have one scale: the smallest power of two that brings the new tokens'
// largest magnitude to at most 448, or the one that the cell has if it holds older
// tokens and that is larger.  A power of two is as exact as any scale here (E4M3
// numbers keep four bits wherever they lie), and raising it leaves what is stored
// as it was but for the numbers that become subnormal.  The largest magnitude is
// taken before the rotation, times sqrt(2) |amplitude|, which is as far as a pair's
// values can go: the scale then does not depend on the position.
//
// Measured: four prompts of 2048 to 8192 tokens, 16 + 16 + 16 heads, d = 128, queries
// rotated too, 66 us = 5.8 TB/s of what has to be read and written (0.86 of the copy
// rate; issue slots and DRAM both 68% busy), a step of 8 sequences 4.2 us a call in a graph.
// Loads through registers, two heads at a time, 99 us; one after the other 128.
//
// A group of d threads takes a cell of the tokens' heads one after the other, a
// thread 16 values of a token as in append_kernel; the group's maximum goes
// through shared memory, once for HEADS heads.
template <int D>
__global__ void __launch_bounds__(kRopeThreads, 3) append_fp8_kernel(const AppendArgs a, const int heads_per_thread) {
  constexpr int LANES = D / 16;
  constexpr int RUNS = 2;
  constexpr int WARPS = D / 32;                  // of a cell's group
  constexpr int CELLS = kRopeThreads / D;        // a block
  constexpr uint32_t kFinite = 0x7f800000u;      // a finite number's magnitude is below it
  __shared__ uint32_t s_max[2][kRopeThreads / 32];
  extern __shared__ __align__(16) uint8_t s_raw[];
  grid_trigger();
  const int group = threadIdx.x / D;
  const int row_in = threadIdx.x % D / LANES, c = threadIdx.x % LANES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_sequence = (a.N + kScaleTokens - 2) / kScaleTokens + 1;
  const long long item = static_cast<long long>(blockIdx.x) * CELLS + group;
  const bool exists = item < static_cast<long long>(a.B) * per_sequence;
  const int b = exists ? static_cast<int>(item / per_sequence) : 0;
  int lq, lk;
  paged_lens(a.seqlens_q, a.seqlens_k, b, a.N, INT_MAX, lq, lk);
  const int first = lk - lq;                     // the first new token's position; may be negative
  const long long cell0 = (static_cast<long long>(first >> 4) + (item - static_cast<long long>(b) * per_sequence)) * 16;
  const bool active = exists && lq > 0 && cell0 < lk;
  if (!active) return;                           // the whole group: a cell behind its sequence's end
  const long long place = cell0 + row_in;
  const bool fresh = place >= first && place < lk;
  const int t = static_cast<int>(place - first);
  const int hq = a.q ? a.Hq : 0;
  const int heads = hq + 2 * a.Hkv;
  const int h0 = blockIdx.y * heads_per_thread;
  const int h1 = min(h0 + heads_per_thread, heads);
  // the cell's first row in its page, or -1: before position 0, past the table's
  // end or in a page that does not exist
  long long row = -1, scale_at = 0;
  if (h1 > hq && cell0 >= 0) {
    if (cell0 >= static_cast<long long>(a.table.max_pages) * a.table.page_size) {
      if (fresh && c == 0) record_bad_page(a.status, SITE_PAGE_PAST_TABLE, b, static_cast<int>(place));
    } else {
      const int page = __ldg(a.table.block_table + b * a.table.table_stride + cell0 / a.table.page_size);
      if (page >= 0 && page < a.table.num_pages) {
        const int in = static_cast<int>(cell0 % a.table.page_size);
        row = static_cast<long long>(page) * a.Hkv * a.table.page_size + in;
        scale_at = static_cast<long long>(page) * a.Hkv * (a.table.page_size / kScaleTokens) + in / kScaleTokens;
      } else if (fresh && c == 0) {
        record_bad_page(a.status, SITE_PAGE_APPEND, b, page);
      }
    }
  }
  const bool has_old = row >= 0 && cell0 < first;
  const bool old = has_old && place < first;
  const bool counts = fresh && place >= 0;       // a token with a place
  Lane<RUNS> l = make_lane<RUNS>(a.rope, D, c, a.rope.rot_dim > 0);
  const int position = fresh && a.rope.positions ? __ldg(a.rope.positions + b * a.rope.positions_sb + t)
                                                 : static_cast<int>(place);
  if (fresh && h0 < hq) set_angles(l, a.rope, position, 1.f);  // (queries: to the bit as fa_rope has them)
  // A thread's values of the heads to come are on their way to its own places in
  // shared memory, up to kAppendStages heads' ahead.  Addresses go from head to
  // head by additions: this kernel is bound by its instructions.
  const uint32_t place_at = smem_u32(s_raw) + threadIdx.x * 16;
  constexpr uint32_t kRing = kAppendStages * kAppendStageBytes;
  const uint16_t* k0 = a.k + b * a.ks.b + t * a.ks.n + l.at;
  const uint16_t* v0 = a.v + b * a.vs.b + t * a.vs.n + l.at;
  const uint16_t* from = nullptr;                // of head f
  long long from_step = 0;
  int f = h0;
  uint32_t in_at = 0;
  auto begin_fetch = [&](int g) {                // g: the line's head that comes next
    if (g < hq) {
      from = a.q + b * a.qs.b + t * a.qs.n + l.at + g * a.qs.h;
      from_step = a.qs.h;
    } else if (g < hq + a.Hkv) {
      from = k0 + (g - hq) * a.ks.h;
      from_step = a.ks.h;
    } else {
      from = v0 + (g - hq - a.Hkv) * a.vs.h;
      from_step = a.vs.h;
    }
  };
  auto fetch = [&]() {
    if (fresh && f < h1) {
#pragma unroll
      for (int k = 0; k < RUNS; ++k)
        cp_async16(place_at + in_at + k * kRopeThreads * 16, from + k * l.step, 16u);
    }
    cp_async_commit();
    ++f;
    from += from_step;
    if (f == hq || f == hq + a.Hkv) begin_fetch(f);
    in_at = in_at + kAppendStageBytes == kRing ? 0 : in_at + kAppendStageBytes;
  };
  begin_fetch(h0);
#pragma unroll 1
  for (int s = 0; s < kAppendStages - 1; ++s) fetch();
  uint32_t out_at = 0;
  Raw<true> raw;
  auto next = [&]() {                            // this thread's values of the next head
    fetch();
    cp_async_wait<kAppendStages - 1>();
#pragma unroll
    for (int k = 0; k < RUNS; ++k)
      ld_shared_v4(place_at + out_at + k * kRopeThreads * 16, reinterpret_cast<uint32_t(&)[4]>(raw.w[4 * k]));
    out_at = out_at + kAppendStageBytes == kRing ? 0 : out_at + kAppendStageBytes;
  };
  if (h0 < hq) {
    uint16_t* to = a.q_out + ((static_cast<long long>(b) * a.Hq + h0) * a.N + t) * D;
#pragma unroll 1
    for (int h = h0; h < min(h1, hq); ++h, to += static_cast<long long>(a.N) * D) {
      next();
      if (!fresh) continue;
      float v[16];
      unpack<true>(raw, v);
      turn(l, a.rope.interleaved, v);
      store<true>(to, 0, l, pack<true>(v));
    }
  }
  const int cells_of_page = a.table.page_size / kScaleTokens;
  int round = 0;
  // heads [begin, end) of keys or values
  auto cells = [&](auto value_tag, int begin, int end) {
    constexpr bool VALUE = decltype(value_tag)::value;
    float* scale_to = (VALUE ? a.v_scales : a.k_scales) +
                      (row >= 0 ? scale_at + static_cast<long long>(begin) * cells_of_page : 0);
    uint8_t* to0 = (VALUE ? a.v_bytes : a.k_bytes) + (row >= 0 ? (row + row_in) * D : 0);  // of head 0
    const uint32_t* found = s_max[0] + group * WARPS;
#pragma unroll 1
    for (int h = begin; h < end; ++h, round ^= 1, scale_to += cells_of_page) {
      const float before = has_old ? *scale_to : 0.f;
      next();
      uint32_t top = 0;                          // the largest magnitudes' bits, two side by side
#pragma unroll
      for (int i = 0; i < 8; ++i) top = __vmaxu2(top, raw.w[i] & 0x7fff7fffu);
      top = max(top & 0xffff0000u, top << 16);
      const bool odd = top >= kFinite;           // an infinity or a NaN among this thread's values
      if (odd) {                                 // the largest finite one
        top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t x = (raw.w[i] << 16) & 0x7fffffffu, y = raw.w[i] & 0x7fff0000u;
          if (x < kFinite) top = max(top, x);
          if (y < kFinite) top = max(top, y);
        }
      }
      top = __reduce_max_sync(0xffffffffu, counts ? top : 0u);
      if (lane == 0) s_max[round][warp] = top;
      // the group's threads
      asm volatile("barrier.cta.sync %0, %1;" ::"r"(group + 1), "n"(D) : "memory");
      if (row < 0) continue;
      top = 0;
#pragma unroll
      for (int i = 0; i < WARPS; ++i) top = max(top, found[round * (kRopeThreads / 32) + i]);
      float largest = __uint_as_float(top);
      if constexpr (!VALUE) largest = fminf(largest * a.key_growth, 3.4028235e38f);
      const uint32_t bits = __float_as_uint(largest);
      // 448 = 1.75 * 2^8: the exponent's field, one more above 1.75
      const int e = max(static_cast<int>((bits + 0x1fffffu) >> 23) - 8, kLowestScale + 127);
      float scale = __uint_as_float(static_cast<uint32_t>(e) << 23);
      float inverse = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
      const bool raised = has_old && scale > before;
      if (has_old && !raised) {
        scale = before;
        inverse = __frcp_rn(before);
      }
      // (a head of a page may be 2^37 bytes; an addition a head in 64 bits spills)
      uint8_t* to = to0 + static_cast<unsigned long long>(static_cast<unsigned>(h)) *
                              static_cast<unsigned>(a.table.page_size) * D;
      if (fresh) {
        float v[16];
        unpack<true>(raw, v);
        if constexpr (!VALUE) turn(l, a.rope.interleaved, v);
        if (odd) {                               // E4M3 has no infinity
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if ((__float_as_uint(v[i]) & 0x7fffffffu) >= kFinite) v[i] = __uint_as_float(0x7fc00000u);
        }
#pragma unroll
        for (int k = 0; k < RUNS; ++k) {
          const float* x = v + 8 * k;
          *reinterpret_cast<uint2*>(to + l.at + k * l.step) =
              make_uint2(pack_e4m3x4(x[0] * inverse, x[1] * inverse, x[2] * inverse, x[3] * inverse),
                         pack_e4m3x4(x[4] * inverse, x[5] * inverse, x[6] * inverse, x[7] * inverse));
        }
      } else if (old && raised) {
        const float ratio = before * inverse;
        uint4 x = *reinterpret_cast<const uint4*>(to + 16 * c);
        x.x = scale_e4m3x4(x.x, ratio);
        x.y = scale_e4m3x4(x.y, ratio);
        x.z = scale_e4m3x4(x.z, ratio);
        x.w = scale_e4m3x4(x.w, ratio);
        *reinterpret_cast<uint4*>(to + 16 * c) = x;
      }
      if (threadIdx.x % D == 0 && (!has_old || raised)) *scale_to = scale;
    }
  };
  const int kv = hq + a.Hkv;
  if (fresh && h0 < kv && h1 > hq) set_angles<true>(l, a.rope, position, 1.f);
  cells(std::false_type{}, max(h0, hq) - hq, min(h1, kv) - hq);
  cells(std::true_type{}, max(h0, kv) - kv, h1 - kv);
  cp_async_wait<0>();
}

// Heads per thread: as many as leave about a thousand threads for every SM,
// so that a large call computes each angle for many heads and a call of few
// tokens spreads its heads over the GPU; at most `most`: eight for the rotation,
// all for the append, which looks its lengths and page up once a thread, sixteen
// for the one into E4M3, whose longer waits want more blocks.  (d =
// 128, bf16, at most 4 / 8 / 16 heads a thread: rotation of 16 heads x 32768
// tokens 42.8 / 43.5 / 44.7 us in a graph and 46.6 / 45.7 / 47.2 in eager calls, 8 x
// 64 heads x 2048 82.0 / 82.6 / 84.0, smaller ones alike.  At most 8 / 16 / all: four
// prompts of 2048 to 8192 tokens, 48 heads, 82 / - / 76; 4 x 48 heads x 8192
// 132.9 / 127.1 / 128.5, 2 x 80 heads x 8192 111.1 / 107.3 / 108.3, 24 heads x 16384
// 37.9 / 39.4 / 39.3, 48 heads x 4096 18.1 / 18.4 / 18.4.  Into E4M3 the four
// prompts 71 with 12 or all, 66 with 16.)
int heads_per_thread(long long tokens, int lanes, int heads, int sms, int most) {
  long long n = tokens * lanes * heads / (static_cast<long long>(sms) * 1024);
  if (n < 1) n = 1;
  if (n > most) n = most;
  if (n < (heads + 65534) / 65535) n = (heads + 65534) / 65535;  // the grid's second axis
  if (n > heads) n = heads;
  const int groups = static_cast<int>((heads + n - 1) / n);
  return (heads + groups - 1) / groups;
}

template <int D>
cudaError_t launch_rope_d(const RopeArgs& a, cudaStream_t stream) {
  constexpr int ITEMS = kRopeThreads / (D / 16);
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const int per = heads_per_thread(tokens, D / 16, a.H, a.sms, 8);
  const dim3 grid(static_cast<unsigned>((tokens + ITEMS - 1) / ITEMS), (a.H + per - 1) / per);
  if (a.x_bf16 && a.y_bf16)
    rope_kernel<D, true, true><<<grid, kRopeThreads, 0, stream>>>(a, per);
  else if (a.x_bf16)
    rope_kernel<D, true, false><<<grid, kRopeThreads, 0, stream>>>(a, per);
  else if (a.y_bf16)
    rope_kernel<D, false, true><<<grid, kRopeThreads, 0, stream>>>(a, per);
  else
    rope_kernel<D, false, false><<<grid, kRopeThreads, 0, stream>>>(a, per);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_append_d(const AppendArgs& a, cudaStream_t stream) {
  constexpr int ITEMS = kRopeThreads / (D / 16);
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const int heads = (a.q ? a.Hq : 0) + 2 * a.Hkv;
  const int per = heads_per_thread(tokens, D / 16, heads, a.sms, heads);
  const dim3 grid(static_cast<unsigned>((tokens + ITEMS - 1) / ITEMS), (heads + per - 1) / per);
  append_kernel<D><<<grid, kRopeThreads, 0, stream>>>(a, per);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_append_fp8_d(const AppendArgs& a, cudaStream_t stream) {
  constexpr int CELLS = kRopeThreads / D;
  const long long cells = static_cast<long long>(a.B) * ((a.N + kScaleTokens - 2) / kScaleTokens + 1);
  const int heads = (a.q ? a.Hq : 0) + 2 * a.Hkv;
  const int per = heads_per_thread(cells * kScaleTokens, D / 16, heads, a.sms, 16);
  const dim3 grid(static_cast<unsigned>((cells + CELLS - 1) / CELLS), (heads + per - 1) / per);
  auto kern = append_fp8_kernel<D>;
  static std::atomic<unsigned long long> ready{0};
  const cudaError_t e = setup_kernel_once(kern, kAppendStages * kAppendStageBytes, 0, ready);
  if (e != cudaSuccess) return e;
  kern<<<grid, kRopeThreads, kAppendStages * kAppendStageBytes, stream>>>(a, per);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream) {
  return a.d == 64 ? launch_rope_d<64>(a, stream) : launch_rope_d<128>(a, stream);
}

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream) {
  if (a.k_scales) return a.d == 64 ? launch_append_fp8_d<64>(a, stream) : launch_append_fp8_d<128>(a, stream);
  return a.d == 64 ? launch_append_d<64>(a, stream) : launch_append_d<128>(a, stream);
}

}  // namespace fa
