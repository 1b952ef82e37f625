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
// phase in [-1/2, 1/2) turns to 2^-32.  The frequency's own rounding leaves
// p * 2^-65 turns, below 10^-13 at p = 10^6.
//
// Both kernels are copies with a little arithmetic: bound by HBM bandwidth
// (two bytes in and two out per bf16 value) when large and by launch latency
// when small.  A thread owns 16 values of a token's head (8 pairs) in 16-byte
// loads, computes their 8 sines and cosines once, and walks over heads with
// them, four heads' loads in flight at a time.
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "serving.h"

namespace fa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kHeadsInFlight = 4;

// Eight consecutive values as fp32.
template <bool BF16>
struct Eight {
  uint4 w[BF16 ? 1 : 2];
};

template <bool BF16>
__device__ __forceinline__ Eight<BF16> load8(const void* base, long long i) {
  Eight<BF16> e;
  if constexpr (BF16) {
    e.w[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + i);
    e.w[0] = p[0];
    e.w[1] = p[1];
  }
  return e;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const Eight<BF16>& e, float (&f)[8]) {
  if constexpr (BF16) {
    const uint32_t w[4] = {e.w[0].x, e.w[0].y, e.w[0].z, e.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[4 * i] = __uint_as_float(e.w[i].x);
      f[4 * i + 1] = __uint_as_float(e.w[i].y);
      f[4 * i + 2] = __uint_as_float(e.w[i].z);
      f[4 * i + 3] = __uint_as_float(e.w[i].w);
    }
  }
}

// Eight fp32 values, rounded once when the output is bf16.
template <bool BF16>
__device__ __forceinline__ void store8(void* base, long long i, const float (&f)[8]) {
  if constexpr (BF16) {
    uint4 w;
    w.x = pack_bf16x2(f[0], f[1]);
    w.y = pack_bf16x2(f[2], f[3]);
    w.z = pack_bf16x2(f[4], f[5]);
    w.w = pack_bf16x2(f[6], f[7]);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) = w;
  } else {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    p[0] = make_float4(f[0], f[1], f[2], f[3]);
    p[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// The 16 values of a head that lane c of its d / 16 lanes owns, as two runs of
// eight, and the pairs it turns.
struct Lane {
  int lo, hi;       // first element of either run
  bool turns;       // false: the values behind rot_dim, copied
  float cs[8], sn[8];
};

__device__ __forceinline__ Lane make_lane(const RopeRef& r, int c, bool turn) {
  Lane l;
  l.turns = turn && 16 * c < r.rot_dim;
  if (l.turns && !r.interleaved) {
    l.lo = 8 * c;
    l.hi = r.rot_dim / 2 + 8 * c;
  } else {
    l.lo = 16 * c;
    l.hi = 16 * c + 8;
  }
  return l;
}

__device__ __forceinline__ void set_angles(Lane& l, const RopeRef& r, int c, int position, float sign) {
  if (!l.turns) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const unsigned long long f = static_cast<unsigned long long>(__ldg(r.turns + 8 * c + i));
    const unsigned long long phase = static_cast<unsigned long long>(static_cast<long long>(position)) * f;
    const float half_turns = static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f;  // 2^-31
    float s, co;
    sincospif(half_turns, &s, &co);
    l.cs[i] = co * r.amplitude;
    l.sn[i] = s * (r.amplitude * sign);
  }
}

// Turns the lane's pairs: interleaved pairs are neighbours inside a run,
// otherwise pair i is (lo[i], hi[i]).
__device__ __forceinline__ void turn(const Lane& l, bool interleaved, float (&lo)[8], float (&hi)[8]) {
  if (!l.turns) return;
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = lo[2 * i], b = lo[2 * i + 1];
      lo[2 * i] = a * l.cs[i] - b * l.sn[i];
      lo[2 * i + 1] = b * l.cs[i] + a * l.sn[i];
      const float e = hi[2 * i], f = hi[2 * i + 1];
      hi[2 * i] = e * l.cs[4 + i] - f * l.sn[4 + i];
      hi[2 * i + 1] = f * l.cs[4 + i] + e * l.sn[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = lo[i], b = hi[i];
      lo[i] = a * l.cs[i] - b * l.sn[i];
      hi[i] = b * l.cs[i] + a * l.sn[i];
    }
  }
}

template <int D, bool XBF, bool YBF>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a, const int heads_per_thread) {
  constexpr int LANES = D / 16;
  grid_trigger();
  const long long item = static_cast<long long>(blockIdx.x) * (kRopeThreads / LANES) + threadIdx.x / LANES;
  if (item >= static_cast<long long>(a.B) * a.N) return;
  const int c = threadIdx.x % LANES;
  const int b = static_cast<int>(item / a.N);
  const int n = static_cast<int>(item - static_cast<long long>(b) * a.N);
  const int h0 = blockIdx.y * heads_per_thread;
  const int h1 = min(h0 + heads_per_thread, a.H);
  const int position = a.rope.positions ? __ldg(a.rope.positions + b * a.rope.positions_sb + n) : n;
  Lane l = make_lane(a.rope, c, true);
  set_angles(l, a.rope, c, position, a.inverse ? -1.f : 1.f);
  const long long xo = b * a.xs.b + n * a.xs.n;
  const long long yo = b * a.ys.b + n * a.ys.n;
  for (int h = h0; h < h1; h += kHeadsInFlight) {
    Eight<XBF> lo[kHeadsInFlight], hi[kHeadsInFlight];
#pragma unroll
    for (int u = 0; u < kHeadsInFlight; ++u) {
      if (h + u < h1) {
        lo[u] = load8<XBF>(a.x, xo + (h + u) * a.xs.h + l.lo);
        hi[u] = load8<XBF>(a.x, xo + (h + u) * a.xs.h + l.hi);
      }
    }
#pragma unroll
    for (int u = 0; u < kHeadsInFlight; ++u) {
      if (h + u < h1) {
        float p[8], q[8];
        unpack8<XBF>(lo[u], p);
        unpack8<XBF>(hi[u], q);
        turn(l, a.rope.interleaved, p, q);
        store8<YBF>(a.y, yo + (h + u) * a.ys.h + l.lo, p);
        store8<YBF>(a.y, yo + (h + u) * a.ys.h + l.hi, q);
      }
    }
  }
}

// Heads of the append in one line: Hq of q (none without q), Hkv of k, Hkv
// of v.
template <int D>
__global__ void __launch_bounds__(kRopeThreads) append_kernel(const AppendArgs a, const int heads_per_thread) {
  constexpr int LANES = D / 16;
  grid_trigger();
  const long long item = static_cast<long long>(blockIdx.x) * (kRopeThreads / LANES) + threadIdx.x / LANES;
  if (item >= static_cast<long long>(a.B) * a.N) return;
  const int c = threadIdx.x % LANES;
  const int b = static_cast<int>(item / a.N);
  const int t = static_cast<int>(item - static_cast<long long>(b) * a.N);
  const int capacity = a.table.max_pages * a.table.page_size;
  int lq, lk;
  paged_lens(a.seqlens_q, a.seqlens_k, b, a.N, capacity, lq, lk);
  if (t >= lq) return;  // padding: nothing of it is written
  const int place = lk - lq + t;
  const int hq = a.q ? a.Hq : 0;
  const int heads = hq + 2 * a.Hkv;
  const int h0 = blockIdx.y * heads_per_thread;
  const int h1 = min(h0 + heads_per_thread, heads);
  // the row of the cache; a token before position 0, or one whose page does
  // not exist, has none
  long long row = -1;
  if (h1 > hq && place >= 0) {
    const int page = __ldg(a.table.block_table + b * a.table.table_stride + place / a.table.page_size);
    if (page >= 0 && page < a.table.num_pages)
      row = (static_cast<long long>(page) * a.Hkv) * a.table.page_size + place % a.table.page_size;
    else if (c == 0)
      record_bad_page(a.status, SITE_PAGE_APPEND, b, page);
  }
  const bool rotate = a.rope.rot_dim > 0;
  Lane l = make_lane(a.rope, c, rotate);
  if (h0 < hq + a.Hkv) {
    const int position = a.rope.positions ? __ldg(a.rope.positions + b * a.rope.positions_sb + t) : place;
    set_angles(l, a.rope, c, position, 1.f);
  }
  for (int h = h0; h < h1; h += kHeadsInFlight) {
    Eight<true> lo[kHeadsInFlight], hi[kHeadsInFlight];
    uint16_t* dst[kHeadsInFlight];
#pragma unroll
    for (int u = 0; u < kHeadsInFlight; ++u) {
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
        lo[u] = load8<true>(src, l.lo);
        hi[u] = load8<true>(src, l.hi);
      }
    }
#pragma unroll
    for (int u = 0; u < kHeadsInFlight; ++u) {
      if (dst[u]) {
        if (h + u < hq + a.Hkv && l.turns) {
          float p[8], q[8];
          unpack8<true>(lo[u], p);
          unpack8<true>(hi[u], q);
          turn(l, a.rope.interleaved, p, q);
          store8<true>(dst[u], l.lo, p);
          store8<true>(dst[u], l.hi, q);
        } else {
          *reinterpret_cast<uint4*>(dst[u] + l.lo) = lo[u].w[0];
          *reinterpret_cast<uint4*>(dst[u] + l.hi) = hi[u].w[0];
        }
      }
    }
  }
}

// Heads per thread: as many as leave about a thousand threads for every SM,
// so that a large call computes each angle once for all heads and a call of
// few tokens spreads its heads over the GPU.
int heads_per_thread(long long tokens, int lanes, int heads, int sms) {
  long long n = tokens * lanes * heads / (static_cast<long long>(sms) * 1024);
  if (n < 1) n = 1;
  if (n > heads) n = heads;
  const int groups = static_cast<int>((heads + n - 1) / n);
  return (heads + groups - 1) / groups;
}

template <int D>
cudaError_t launch_rope_d(const RopeArgs& a, cudaStream_t stream) {
  constexpr int ITEMS = kRopeThreads / (D / 16);
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const int per = heads_per_thread(tokens, D / 16, a.H, a.sms);
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
  const int per = heads_per_thread(tokens, D / 16, heads, a.sms);
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
