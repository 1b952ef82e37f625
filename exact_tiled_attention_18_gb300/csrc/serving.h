// Interface between the C-ABI translation unit and the kernels of rotary
// positions, the paged key/value cache and the attention that reads it.  Not
// part of the public boundary (that is include/fa.h).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace fa {

// Status codes these kernels leave in the device status word, besides the
// timeout of ptx.cuh.
constexpr int FA_DEV_BAD_PAGE = 7;

// Sites recorded with FA_DEV_BAD_PAGE.
enum PageSite : int { SITE_PAGE_APPEND = 71, SITE_PAGE_READ = 72, SITE_PAGE_PAST_TABLE = 81 };

// A [B][H][N][d] tensor with contiguous d: element strides of the others.
struct Strides {
  long long b, h, n;
};

// Where position p of sequence b lives: page block_table[b * table_stride +
// p / page_size], row p % page_size, of pages [num_pages][Hkv][page_size][d].
struct PageTable {
  const int* block_table;
  long long table_stride;
  int max_pages;   // entries per sequence that may be read
  int page_size;   // a multiple of 16
  int num_pages;   // page ids are valid in [0, num_pages)
};

// The rotation of a token at position p: pair i turns by p * turns[i] / 2^64
// of a full turn, and the pair's values are multiplied by `amplitude`.
struct RopeRef {
  const long long* turns;  // [rot_dim / 2]; null: no rotation
  const int* positions;    // [B][N] (stride positions_sb between sequences), or null
  long long positions_sb;
  int rot_dim;             // a multiple of 16, at most d; 0: no rotation
  int interleaved;         // 0: pairs (i, i + rot_dim / 2), 1: pairs (2i, 2i + 1)
  float amplitude;
};

struct RopeArgs {
  const void* x;
  void* y;
  int x_bf16, y_bf16;
  Strides xs, ys;
  RopeRef rope;
  int inverse;
  int B, H, N, d;
  int sms;
};

struct AppendArgs {
  const uint16_t *q, *k, *v;  // q may be null
  Strides qs, ks, vs;
  uint16_t* q_out;            // [B][Hq][N][d]
  uint16_t *k_pages, *v_pages;
  PageTable table;
  RopeRef rope;               // positions null: the cache position
  const int *seqlens_q, *seqlens_k;
  int B, Hq, Hkv, N, d;
  int sms;
  int* status;
};

struct PagedArgs {
  CUtensorMap tm_k, tm_v;     // tile kernel: maps of [num_pages * Hkv][page_size][d], boxes of box_rows rows, 8 at a time
  CUtensorMap tm_q;           // and over q's rows [B * Hq * Nq][d], boxes 64 x 128 (chunks only)
  CUtensorMap tm_qp;          // and over [B][Hkv][G * Nq][d], boxes of 128 rows (prefix, where boxed_rows)
  CUtensorMap st_k, st_v;     // step kernel: blocked maps of the same, boxes of box_rows whole rows
  CUtensorMap st_k16, st_v16; // and of 16
  const uint16_t *q;          // [B][Hq][Nq][d]
  PageTable table;
  const int* prefix_table;    // pages of the shared prefix
  int prefix_len;             // keys of the shared prefix, a multiple of page_size; 0: none
  int boxed_rows;             // the prefix's row tiles come in boxes of tm_qp, else row by row
  void* o;                    // [B][Hq][Nq][d] fp32, or bf16 when o_bf16
  int o_bf16;
  float* lse;                 // [B][Hq][Nq]
  float* part;                // workspace
  const int *seqlens_q, *seqlens_k;
  int B, Hq, Hkv, Nq, d;
  int causal;
  float scale_log2;
  int box_rows;               // rows of a TMA box: the largest power of two up to 64 that divides page_size
  int sms;
  int* status;
  unsigned long long wait_limit_ns;
  int stall_unit;
};

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream);
cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_paged(const PagedArgs& a, cudaStream_t stream);

// Whether the sequences' own keys are the step kernel's work (few rows a key
// head) or the tile kernel's.
bool paged_uses_steps(int G, int Nq);

// Workspace of launch_paged in 4-byte words.
size_t paged_workspace_floats(int B, int Hkv, int G, int Nq, int d, bool with_prefix);

// Launches a kernel that may start while the one before it in the stream
// still runs, provided that one has let its dependents go (grid_trigger); it
// waits for it itself (grid_wait).
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kern)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                              Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
}

#if defined(__CUDACC__)
// The kernel behind this one in the stream may start its CTAs from here on
// (once every CTA of this grid has said so or ended).
__device__ __forceinline__ void grid_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Until the kernels before this one have ended and their writes are visible.
// What they wrote is read behind it with ordinary loads, never with __ldg,
// which the compiler may move before it.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Records an entry of a block table that names no page, or a position behind
// the table's last one (first failure wins).
__device__ __forceinline__ void record_bad_page(int* status, int site, int sequence, int what) {
  if (atomicCAS(status, 0, FA_DEV_BAD_PAGE) == 0) {
    volatile int* s = status;
    s[1] = site;
    s[2] = sequence;
    s[3] = what;
    __threadfence();
  }
}

// For a kernel that does not wait for the one before it at its start, because
// that one has nothing for it: what it reads was written by kernels further
// back, which that one has waited for before it let this one start; a fence
// keeps this SM's L1 from answering with what it held before.
__device__ __forceinline__ void grid_overlap() { __threadfence(); }

// Valid lengths of sequence b: new tokens and keys in the cache.
__device__ __forceinline__ void paged_lens(const int* seqlens_q, const int* seqlens_k, int b, int nq, int capacity,
                                           int& lq, int& lk) {
  lq = seqlens_q ? min(max(seqlens_q[b], 0), nq) : nq;
  lk = seqlens_k ? min(max(seqlens_k[b], 0), capacity) : capacity;
}
#endif

}  // namespace fa
