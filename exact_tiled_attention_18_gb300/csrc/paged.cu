// Attention over the paged cache: one warp per query row, plain loops.
#include <cuda_runtime.h>
#include <math_constants.h>

#include "ptx.cuh"
#include "serving.h"

namespace fa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float bf16_at(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
}

template <int D>
__global__ void __launch_bounds__(128) paged_rows_kernel(const PagedArgs a) {
  constexpr int CW = D / 32;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(a.B) * a.Hq * a.Nq) return;
  const int lane = threadIdx.x & 31;
  const int i = static_cast<int>(row % a.Nq);
  const int hq = static_cast<int>(row / a.Nq % a.Hq);
  const int b = static_cast<int>(row / a.Nq / a.Hq);
  const int kh = hq / (a.Hq / a.Hkv);
  const int ps = a.table.page_size;
  int lq, lk;
  paged_lens(a.seqlens_q, a.seqlens_k, b, a.Nq, a.table.max_pages * ps, lq, lk);
  const int end = i < lq ? (a.causal ? min(i + lk - lq + 1, lk) : lk) : 0;
  float qv[CW], acc[CW];
  for (int c = 0; c < CW; ++c) {
    qv[c] = bf16_at(a.q + row * D + lane * CW + c) * a.scale_log2;
    acc[c] = 0.f;
  }
  float m = -CUDART_INF_F, l = 0.f;
  for (int j = 0; j < end; ++j) {
    const int page = j < a.prefix_len ? __ldg(a.prefix_table + j / ps)
                                      : __ldg(a.table.block_table + b * a.table.table_stride + j / ps);
    if (page < 0 || page >= a.table.num_pages) {
      if (lane == 0) record_bad_page(a.status, SITE_PAGE_READ, b, page);
      continue;
    }
    const long long at = ((static_cast<long long>(page) * a.Hkv + kh) * ps + j % ps) * D + lane * CW;
    float s = 0.f;
    for (int c = 0; c < CW; ++c) s = fmaf(qv[c], bf16_at(a.k_pages + at + c), s);
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const float mn = fmaxf(m, s);
    const float alpha = exp2f(m - mn), p = exp2f(s - mn);
    l = l * alpha + p;
    for (int c = 0; c < CW; ++c) acc[c] = acc[c] * alpha + p * bf16_at(a.v_pages + at + c);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int c = 0; c < CW; ++c) {
    const float o = acc[c] * inv;
    if (a.o_bf16)
      static_cast<uint16_t*>(a.o)[row * D + lane * CW + c] = static_cast<uint16_t>(pack_bf16x2(o, 0.f));
    else
      static_cast<float*>(a.o)[row * D + lane * CW + c] = o;
  }
  if (lane == 0) a.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : -CUDART_INF_F;
}

}  // namespace

cudaError_t launch_paged(const PagedArgs& a, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.B) * a.Hq * a.Nq;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  if (a.d == 64)
    paged_rows_kernel<64><<<grid, 128, 0, stream>>>(a);
  else
    paged_rows_kernel<128><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
