// What the kernels of attention over the paged cache share: the sequences'
// lengths on the device, the line of key tiles, the partial results.
#pragma once

#include <cuda_runtime.h>

#include "serving.h"

namespace fa {

constexpr int kStepRows = 32;          // rows a key head that the step kernel takes
constexpr int kLineSequences = 1024;   // sequences a launch: the line's table is in shared memory
constexpr int kLineWords = 1040;       // 4-byte words of the line in the workspace, a multiple of 4
constexpr int kMaxCtas = 512;
constexpr int kMinTiles = 4;           // key tiles a CTA takes at least
static_assert(kLineWords >= kLineSequences + 1 && kLineWords % 4 == 0, "the line's room");

struct PagedSeq {
  const int *seqlens_q, *seqlens_k;
  int B, Hkv, G, Nq;
  int capacity;     // positions that the table reaches
  int prefix_len;   // keys that are not these tiles' work
};

struct PagedStep {
  PagedSeq seq;
  PageTable table;
  const uint16_t* q;
  void* o;
  int o_bf16;
  float* lse;
  int* line_out;     // the line's table, for the combine
  float *part, *part_lse;  // [slot][G * Nq][d] outputs and [slot][G * Nq] log2-sum-exp
  int direct;        // 1: a piece that is a whole sequence's writes o and lse
  int box_rows;
  int b0;            // first sequence of this launch, for error reports
  int causal;
  float scale_log2;
  int* status;
  unsigned long long wait_limit_ns;
  int stall_unit;
};

struct PagedCombine {
  PagedSeq seq;
  const int* line;
  int ctas;
  const float *part, *part_lse;
  int direct;
  void* o;
  int o_bf16;
  float* lse;
};

#if defined(__CUDACC__)
__device__ __forceinline__ void seq_lens(const PagedSeq& s, int b, int& lq, int& lk) {
  paged_lens(s.seqlens_q, s.seqlens_k, b, s.Nq, s.capacity, lq, lk);
}

// Tiles of the line that each CTA takes.
__device__ __forceinline__ int tiles_per_cta(int total, int ctas) {
  return max((total + ctas - 1) / ctas, kMinTiles);
}

// line[b] = tiles of one key head of all sequences before b, for b in
// [0, B]; `scratch` holds one word a warp.  Ends with a CTA-wide barrier.
template <int THREADS>
__device__ __forceinline__ void build_line(int* line, int* scratch, const PagedSeq& s, int tile_keys) {
  constexpr int WARPS = THREADS / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int base = 0;
  for (int b0 = 0; b0 < s.B; b0 += THREADS) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    int n = 0;
    if (b < s.B) {
      int lq, lk;
      seq_lens(s, b, lq, lk);
      if (lq > 0 && lk > s.prefix_len) n = (lk - s.prefix_len + tile_keys - 1) / tile_keys;
    }
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
    if (b < s.B) line[b] = before + x - n;
  }
  if (threadIdx.x == 0) line[s.B] = base;
  __syncthreads();
}
#endif

}  // namespace fa
