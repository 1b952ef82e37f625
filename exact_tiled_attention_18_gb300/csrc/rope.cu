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

#include <climits>

#include "ptx.cuh"
#include "serving.h"

namespace fa {
namespace {

constexpr int kRopeThreads = 256;

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

template <int RUNS>
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
    const float half_turns = static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f;  // 2^-31
    float s, co;
    sincospif(half_turns, &s, &co);
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

// Heads per thread: as many as leave about a thousand threads for every SM,
// so that a large call computes each angle for many heads and a call of few
// tokens spreads its heads over the GPU; at most `most`: eight for the rotation,
// all for the append, which looks its lengths and page up once a thread.  (d =
// 128, bf16, at most 4 / 8 / 16 heads a thread: rotation of 16 heads x 32768
// tokens 42.8 / 43.5 / 44.7 us in a graph and 46.6 / 45.7 / 47.2 in eager calls, 8 x
// 64 heads x 2048 82.0 / 82.6 / 84.0, smaller ones alike.  At most 8 / 16 / all: four
// prompts of 2048 to 8192 tokens, 48 heads, 82 / - / 76; 4 x 48 heads x 8192
// 132.9 / 127.1 / 128.5, 2 x 80 heads x 8192 111.1 / 107.3 / 108.3, 24 heads x 16384
// 37.9 / 39.4 / 39.3, 48 heads x 4096 18.1 / 18.4 / 18.4.)
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

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream) {
  return a.d == 64 ? launch_rope_d<64>(a, stream) : launch_rope_d<128>(a, stream);
}

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream) {
  return a.d == 64 ? launch_append_d<64>(a, stream) : launch_append_d<128>(a, stream);
}

}  // namespace fa
