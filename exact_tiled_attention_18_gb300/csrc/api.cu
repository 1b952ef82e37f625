// C ABI of the library: argument checks, TMA descriptors, launches and the
// device status word.  The operation each entry point computes is stated in
// include/fa.h.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "../../include/fa.h"
#include "internal.h"
#include "serving.h"

// Device status word written by the kernels when a bounded wait gives up:
// [0] code, [1] wait site, [2] block, [3] work unit.  First failure wins.
__device__ int g_fa_status[4];

namespace {

constexpr long long kDefaultL2Budget = 32LL << 20;  // K+V bytes of one L2 head group
constexpr int kMaxDevices = 64;

struct DeviceInfo {
  bool ready = false;
  int sms = 0;
  int* status = nullptr;
};

std::mutex g_mu;
DeviceInfo g_dev[kMaxDevices];
int g_last_failure[4];

fa_status device_info(DeviceInfo& out) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_LAUNCH;
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.ready) {
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return FA_ERR_LAUNCH;
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_fa_status) != cudaSuccess) return FA_ERR_LAUNCH;
    d.status = static_cast<int*>(p);
    d.ready = true;
  }
  out = d;
  return FA_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// Encoded tensor maps, cached by everything that goes into them (base
// address, element type, extents, box), so that repeated calls on the same
// tensors skip the driver's encoder.  A map depends on nothing else: reusing
// one for a buffer freed and allocated again at the same address with the
// same shape is still exact.  The paged calls use four to seven maps for every
// layer's own cache, so there is room for some hundred layers' (4096 maps, in
// sets of eight that a hash of the key picks, each replaced round robin).
// (Host time of a forward_paged over 32 layers' caches in turn: 22.3 us a call
// with one list of 64 maps, 20.8 to 21.7 so; of one cache 21.6 to 21.8 and 21.6.)
constexpr int kMapSetBits = 9, kMapWays = 8;

struct MapKey {
  const void* base = nullptr;
  int elem_bytes = 0, heads = 0, rows = 0, inner = 0, box_inner = 0, box_rows = 0;
  int blocked = 0;       // 1, 4-D: a box takes all the 64-column blocks of its rows; 2, 5-D: of 8 rows at a time
  int batch = 0;         // > 0, 4-D: over [batch][heads][rows][inner], a box takes box_batch sequences' rows
  int box_batch = 0;
  bool operator==(const MapKey& o) const {
    return base == o.base && elem_bytes == o.elem_bytes && heads == o.heads && rows == o.rows && inner == o.inner &&
           box_inner == o.box_inner && box_rows == o.box_rows && blocked == o.blocked && batch == o.batch &&
           box_batch == o.box_batch;
  }
  // set of the cache: the top bits of the fields multiplied together
  unsigned set() const {
    unsigned long long h = reinterpret_cast<uintptr_t>(base);
    for (int v : {elem_bytes, heads, rows, inner, box_inner, box_rows, blocked, batch, box_batch})
      h = (h ^ (h >> 29) ^ static_cast<unsigned>(v)) * 0x9E3779B97F4A7C15ULL;  // 2^64 / golden ratio, odd
    return static_cast<unsigned>(h >> (64 - kMapSetBits));
  }
};

struct MapSet {
  MapKey keys[kMapWays];  // base null: free
  CUtensorMap maps[kMapWays];
  unsigned next;          // way that the next map goes to
};

std::mutex g_map_mu;
MapSet g_map_sets[1 << kMapSetBits];
long long g_map_encodes = 0;

bool remember_map(const MapKey& key, const CUtensorMap& m) {
  std::lock_guard<std::mutex> lock(g_map_mu);
  ++g_map_encodes;
  MapSet& set = g_map_sets[key.set()];
  const unsigned way = set.next++ % kMapWays;
  set.keys[way] = key;
  set.maps[way] = m;
  return true;
}

// 3-D map over [heads][rows][inner] elements of `elem_bytes` (2: bf16, 1:
// E4M3 bytes), box = box_inner x box_rows x 1 with the 128-byte swizzle (the
// layout the MMA descriptors expect).  Rows past `rows` read as zeros.
// Blocked (bf16): a 4-D map over [heads][inner / 64][rows][64] of the same
// memory, box = 64 x box_rows x (inner / 64) x 1, so that one load brings the
// box's rows block by block (blocked = 1), or a 5-D map over
// [heads][rows / 8][inner / 64][8][64], box = 64 x 8 x (inner / 64) x box_rows / 8
// x 1, so that it brings them 8 rows at a time, block by block (blocked = 2; rows
// a multiple of 8).  With a batch (bf16): a 4-D map over
// [batch][heads][rows][inner], box = 64 x box_rows x 1 x box_batch, for the
// rows of several sequences' same head one behind the other.
bool encode_map(CUtensorMap* m, const MapKey& key) {
  {
    std::lock_guard<std::mutex> lock(g_map_mu);
    const MapSet& set = g_map_sets[key.set()];
    for (int i = 0; i < kMapWays; ++i) {
      if (set.keys[i] == key) {
        *m = set.maps[i];
        return true;
      }
    }
  }
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t eb = static_cast<cuuint64_t>(key.elem_bytes);
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(key.inner), static_cast<cuuint64_t>(key.rows),
                        static_cast<cuuint64_t>(key.heads)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(key.inner) * eb,
                           static_cast<cuuint64_t>(key.rows) * key.inner * eb};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(key.box_inner), static_cast<cuuint32_t>(key.box_rows), 1};
  cuuint32_t estride[5] = {1, 1, 1, 1, 1};
  if (key.blocked == 2) {
    const cuuint64_t blocks = static_cast<cuuint64_t>(key.inner / 64);
    cuuint64_t dims5[5] = {64, 8, blocks, dims[1] / 8, dims[2]};
    cuuint64_t strides5[4] = {strides[0], 128, 8 * strides[0], strides[1]};
    cuuint32_t box5[5] = {64, 8, static_cast<cuuint32_t>(blocks), box[1] / 8, 1};
    if (fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(key.base), dims5, strides5, box5, estride,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
    return remember_map(key, *m);
  }
  if (key.blocked || key.batch > 0) {
    cuuint64_t dims4[4] = {64, dims[1], static_cast<cuuint64_t>(key.inner / 64), dims[2]};
    cuuint64_t strides4[3] = {strides[0], 128, strides[1]};
    cuuint32_t box4[4] = {64, box[1], static_cast<cuuint32_t>(key.inner / 64), 1};
    if (key.batch > 0) {
      dims4[0] = dims[0];
      dims4[2] = dims[2];
      dims4[3] = static_cast<cuuint64_t>(key.batch);
      strides4[1] = strides[1];
      strides4[2] = strides[1] * key.heads;
      box4[2] = 1;
      box4[3] = static_cast<cuuint32_t>(key.box_batch);
    }
    if (fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(key.base), dims4, strides4, box4, estride,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
    return remember_map(key, *m);
  }
  CUresult r = fn(m, key.elem_bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
                  const_cast<void*>(key.base), dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return false;
  return remember_map(key, *m);
}

// bf16 [heads][n][d], boxes of 64 columns x box_rows rows.
bool encode_bf16_map(CUtensorMap* m, const void* base, int heads, int n, int d, int box_rows = fa::kTileRows) {
  return encode_map(m, MapKey{base, 2, heads, n, d, 64, box_rows});
}

// one-byte elements [heads][rows][inner], 128 x 128 boxes (one 128-byte row
// of the box per matrix row).
bool encode_u8_map(CUtensorMap* m, const void* base, int heads, int rows, int inner) {
  return encode_map(m, MapKey{base, 1, heads, rows, inner, 128, fa::kTileRows});
}

unsigned long long wait_limit_ns() {
  static unsigned long long v = []() -> unsigned long long {
    const char* s = std::getenv("FA_WAIT_LIMIT_MS");
    long long ms = s ? std::atoll(s) : 0;
    if (ms <= 0) ms = 4000;
    return static_cast<unsigned long long>(ms) * 1000000ULL;
  }();
  return v;
}

// Testing only: a unit index n >= 0 makes CTA 0 of the next launches skip one
// tile load of the n-th work unit it processes (the decode kernel: CTA n
// skips its first stage), so that a pipeline wait runs out and the timeout
// path can be exercised without faulting anything.  -1 (the default) means
// never.  Its first value comes from FA_TEST_STALL_UNIT, read once per
// process; fa_test_set_stall changes it.
std::atomic<int>& stall_unit_cell() {
  static std::atomic<int> cell([]() {
    const char* s = std::getenv("FA_TEST_STALL_UNIT");
    return (s && *s) ? std::atoi(s) : -1;
  }());
  return cell;
}

int test_stall_unit() { return stall_unit_cell().load(std::memory_order_relaxed); }

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

fa_status check_sizes(int B, int H, int N, int d, int causal) {
  if (B < 1 || H < 1 || N < 1) return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * H * N >= (1LL << 31)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED_D;
  return FA_OK;
}

// n: rows the units tile (query rows for the forward and dQ, keys for dK/dV);
// n_stream: rows every unit of a head streams through (sizes the L2 groups).
fa::SchedParams make_sched(int heads, int n, int d, int causal, int grid_cap, long long budget,
                           int unit_rows = fa::kUnitRows, int cost_grows = 1, int n_stream = 0) {
  fa::SchedParams sp;
  sp.heads = heads;
  sp.units_per_head = (n + unit_rows - 1) / unit_rows;
  sp.cost_grows = cost_grows;
  sp.group_heads =
      fa::sched_group_heads(heads, n_stream > 0 ? n_stream : n, d, budget > 0 ? budget : kDefaultL2Budget);
  const long long units = static_cast<long long>(heads) * sp.units_per_head;
  sp.grid = static_cast<int>(units < grid_cap ? units : grid_cap);
  sp.causal = causal;
  return sp;
}

// Strides in elements; a query stride of 0 broadcasts one row of key
// biases over the queries, otherwise rows hold Nk keys.
fa_status check_bias(const void* bias, long long sb, long long sh, long long sq, int Nk) {
  if (!bias) return FA_ERR_INVALID_ARG;
  if (sb < 0 || sh < 0 || sq < 0 || (sq != 0 && sq < Nk)) return FA_ERR_INVALID_ARG;
  if (!aligned(bias, 2)) return FA_ERR_MISALIGNED;
  return FA_OK;
}

fa_status fwd_common(const void* q, const void* k, const void* v, void* o, int o_dtype, float* lse,
                     const int* seqlens_q, const int* seqlens_k, int B, int H, int Nq, int Nk, int d, float scale,
                     int causal, fa_stream_t stream, const void* bias = nullptr, long long bias_sb = 0,
                     long long bias_sh = 0, long long bias_sq = 0) {
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (bias) {
    const fa_status bs = check_bias(bias, bias_sb, bias_sh, bias_sq, Nk);
    if (bs != FA_OK) return bs;
  }
  if (o_dtype != FA_DTYPE_F32 && o_dtype != FA_DTYPE_BF16) return FA_ERR_INVALID_ARG;
  fa_status st = check_sizes(B, H, Nq, d, causal);
  if (st != FA_OK) return st;
  st = check_sizes(B, H, Nk, d, causal);
  if (st != FA_OK) return st;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
      (seqlens_q && !aligned(seqlens_q, 4)) || (seqlens_k && !aligned(seqlens_k, 4)))
    return FA_ERR_MISALIGNED;
  DeviceInfo di;
  if (device_info(di) != FA_OK) return FA_ERR_LAUNCH;
  const int heads = B * H;
  fa::FwdArgs a;
  std::memset(&a, 0, sizeof(a));
  if (!encode_bf16_map(&a.tm_q, q, heads, Nq, d) || !encode_bf16_map(&a.tm_k, k, heads, Nk, d) ||
      !encode_bf16_map(&a.tm_v, v, heads, Nk, d))
    return FA_ERR_LAUNCH;
  a.o = o;
  a.o_bf16 = o_dtype == FA_DTYPE_BF16;
  a.lse = lse;
  a.geom.nq = Nq;
  a.geom.nk = Nk;
  a.geom.seqlens_q = seqlens_q;
  a.geom.seqlens_k = seqlens_k;
  a.geom.heads_per_batch = H;
  a.d = d;
  a.causal = causal;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.sched = make_sched(heads, Nq, d, causal, di.sms, 0, fa::kUnitRows, 1, Nk);
  a.status = di.status;
  a.wait_limit_ns = wait_limit_ns();
  a.stall_unit = test_stall_unit();
  a.bias = static_cast<const uint16_t*>(bias);
  a.bias_sb = bias_sb;
  a.bias_sh = bias_sh;
  a.bias_sq = bias_sq;
  return fa::launch_fwd(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

// Key splits of the split-key forward: at most kMaxKeySplits, at least two
// key tiles each, and only as many as it takes to fill the SMs once.
constexpr int kMaxKeySplits = 16;

int key_split_cap(int N) {
  const int nkt = (N + fa::kTileRows - 1) / fa::kTileRows;
  const int cap = nkt / 2;
  return cap < 1 ? 1 : (cap > kMaxKeySplits ? kMaxKeySplits : cap);
}

void key_splits(int heads, int N, int sms, int& splits, int& chunk) {
  const int nkt = (N + fa::kTileRows - 1) / fa::kTileRows;
  const long long units = static_cast<long long>(heads) * ((N + fa::kUnitRows - 1) / fa::kUnitRows);
  long long s = units >= sms ? 1 : (sms + units - 1) / units;
  const int cap = key_split_cap(N);
  if (s > cap) s = cap;
  if (s < 1) s = 1;
  chunk = static_cast<int>((nkt + s - 1) / s);
  splits = (nkt + chunk - 1) / chunk;
}

// Checks the arguments of a backward call (the workspace only for alignment;
// it may be null) and fills every field of `a` but the row-term buffer.  q, dO, o, lse, dq: [B*H][Nq] rows; k, v, dk, dv:
// [B*H][Nk] rows.
// need_o = false (the single-pass backward, which forms D without O): o is
// ignored and may be null.
fa_status bwd_prepare(fa::BwdArgs& a, const void* q, const void* k, const void* v, const void* o, int o_dtype,
                      const float* lse, const void* dO, float* dq, float* dk, float* dv, const float* workspace,
                      const int* seqlens_q, const int* seqlens_k, int B, int H, int Nq, int Nk, int d, float scale,
                      int causal, bool need_o = true) {
  if (!need_o) {
    o = q;  // never read
    o_dtype = FA_DTYPE_F32;
  }
  if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
  if (o_dtype != FA_DTYPE_F32 && o_dtype != FA_DTYPE_BF16) return FA_ERR_INVALID_ARG;
  fa_status st = check_sizes(B, H, Nq, d, causal);
  if (st != FA_OK) return st;
  st = check_sizes(B, H, Nk, d, causal);
  if (st != FA_OK) return st;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(dO, 16) ||
      !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(lse, 4) ||
      (workspace && !aligned(workspace, 4)) || (seqlens_q && !aligned(seqlens_q, 4)) ||
      (seqlens_k && !aligned(seqlens_k, 4)))
    return FA_ERR_MISALIGNED;
  DeviceInfo di;
  if (device_info(di) != FA_OK) return FA_ERR_LAUNCH;
  const int heads = B * H;
  std::memset(&a, 0, sizeof(a));
  if (!encode_bf16_map(&a.tm_q, q, heads, Nq, d) || !encode_bf16_map(&a.tm_k, k, heads, Nk, d) ||
      !encode_bf16_map(&a.tm_v, v, heads, Nk, d) || !encode_bf16_map(&a.tm_do, dO, heads, Nq, d))
    return FA_ERR_LAUNCH;
  a.o = o;
  a.o_bf16 = o_dtype == FA_DTYPE_BF16;
  a.lse = lse;
  a.dout = static_cast<const uint16_t*>(dO);
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.heads = heads;
  a.geom.nq = Nq;
  a.geom.nk = Nk;
  a.geom.seqlens_q = seqlens_q;
  a.geom.seqlens_k = seqlens_k;
  a.geom.heads_per_batch = H;
  a.d = d;
  a.causal = causal;
  a.scale = scale;
  a.scale_log2 = scale * 1.4426950408889634f;
  // dK/dV: one unit per 128-key tile, heaviest at the start of the sequence,
  // streaming the head's queries; dQ: one unit per 128-query tile, heaviest
  // at the end, streaming the head's keys.
  a.sched_kv = make_sched(heads, Nk, d, causal, di.sms, 0, fa::kTileRows, 0, Nq);
  a.sched_q = make_sched(heads, Nq, d, causal, di.sms, 0, fa::kTileRows, 1, Nk);
  a.grid_kv = a.sched_kv.grid;
  a.grid_q = a.sched_q.grid;
  a.status = di.status;
  a.wait_limit_ns = wait_limit_ns();
  a.stall_unit = test_stall_unit();
  return FA_OK;
}

// Key splits of the decode kernel.  Each split is at least kDecodeMinChunk
// keys; the count aims at a few waves of two resident CTAs per SM over all
// heads, and is capped so that the workspace bound below holds.
constexpr int kDecodeMinChunk = 512;
constexpr int kDecodeMaxSplits = 256;

int decode_max_splits(int Nk) {
  const int s = (Nk + kDecodeMinChunk - 1) / kDecodeMinChunk;
  return s < 1 ? 1 : (s > kDecodeMaxSplits ? kDecodeMaxSplits : s);
}

void decode_splits(int heads, int Nk, int sms, int& splits, int& chunk) {
  const long long target = 4LL * 2 * sms;  // four waves of two CTAs per SM
  long long s = (target + heads - 1) / heads;
  const int cap = decode_max_splits(Nk);
  if (s > cap) s = cap;
  if (s < 1) s = 1;
  chunk = static_cast<int>(((Nk + s - 1) / s + 63) / 64 * 64);
  splits = (Nk + chunk - 1) / chunk;
}

// Both backward kernels on prepared arguments; without a workspace the row
// term lives in a stream-ordered allocation freed behind the kernels.
fa_status bwd_launch(fa::BwdArgs& a, float* workspace, int B, int H, int Nq, fa_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  float* delta = workspace;
  if (!delta) {
    if (cudaMallocAsync(reinterpret_cast<void**>(&delta), fa_bwd_workspace_bytes(B, H, Nq), s) != cudaSuccess)
      return FA_ERR_LAUNCH;
  }
  a.delta = delta;
  cudaError_t e = fa::launch_bwd(a, s);
  if (!workspace) {
    cudaError_t e2 = cudaFreeAsync(delta, s);
    if (e == cudaSuccess) e = e2;
  }
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

// ------------------------------------------- rotary positions, paged cache

// Pool of the paged calls' own workspaces on the current device.  The
// device's default pool gives freed memory back at the next synchronisation,
// and taking it anew then costs a small call more than its kernels; this one
// keeps what the calls have used, up to kPoolKeep bytes.  (One sequence of
// 1000 keys, 32 heads: 6.8 to 7.2 us of host time a call with it, 6.0 to 6.1
// with a workspace given.)
constexpr unsigned long long kPoolKeep = 256ULL << 20;

cudaMemPool_t workspace_pool() {
  static std::mutex mu;
  static cudaMemPool_t pools[kMaxDevices];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!pools[dev]) {
    cudaMemPoolProps props{};
    props.allocType = cudaMemAllocationTypePinned;
    props.location.type = cudaMemLocationTypeDevice;
    props.location.id = dev;
    cudaMemPool_t pool;
    if (cudaMemPoolCreate(&pool, &props) != cudaSuccess) return nullptr;
    unsigned long long keep = kPoolKeep;
    if (cudaMemPoolSetAttribute(pool, cudaMemPoolAttrReleaseThreshold, &keep) != cudaSuccess) return nullptr;
    pools[dev] = pool;
  }
  return pools[dev];
}

// Strides of the dimensions that are walked; the stride of a dimension of
// size one means nothing and is dropped.
fa::Strides used_strides(long long sb, long long sh, long long sn, int B, int H, int N) {
  return fa::Strides{B > 1 ? sb : 0, H > 1 ? sh : 0, N > 1 ? sn : 0};
}

// Whether rows of d elements at b * s.b + h * s.h + n * s.n fall on one
// another.  Strides that nest, each at least what the smaller ones span, never
// do; others are looked at difference by difference, the dimension with the
// most rows solved for (at most 2^22 steps for 2^31 rows).
bool rows_overlap(const fa::Strides& s, int B, int H, int N, int d) {
  struct Dim {
    long long stride, rows;
  } x[3] = {{s.b, B}, {s.h, H}, {s.n, N}};
  std::sort(x, x + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  long long span = d;
  bool nested = true;
  for (const Dim& i : x) {
    if (i.rows == 1) continue;
    nested = nested && i.stride >= span;
    span += i.stride * (i.rows - 1);
  }
  if (nested) return false;
  std::sort(x, x + 3, [](const Dim& a, const Dim& b) { return a.rows < b.rows; });
  for (long long i = 0; i < x[0].rows; ++i) {
    for (long long j = 1 - x[1].rows; j < x[1].rows; ++j) {
      const long long off = i * x[0].stride + j * x[1].stride, most = x[2].rows - 1;
      const long long near = x[2].stride > 0 ? -off / x[2].stride : 0;
      for (long long k = near - 1; k <= near + 1; ++k) {
        const long long in = std::min(std::max(k, -most), most);
        if ((i || j || in) && std::llabs(off + in * x[2].stride) < d) return true;
      }
    }
  }
  return false;
}

fa_status check_strides(const fa::Strides& s, int elem_bytes) {
  if (s.b < 0 || s.h < 0 || s.n < 0) return FA_ERR_INVALID_ARG;
  const long long unit = 16 / elem_bytes;  // rows start on 16-byte boundaries
  return s.b % unit || s.h % unit || s.n % unit ? FA_ERR_MISALIGNED : FA_OK;
}

fa_status check_rope(const long long* turns, int rot_dim, int layout, float amplitude, const int* positions,
                     long long positions_sb, int d) {
  if (rot_dim < 16 || rot_dim > d || rot_dim % 16 != 0 || !turns) return FA_ERR_INVALID_ARG;
  if (layout != FA_ROPE_HALF && layout != FA_ROPE_INTERLEAVED) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(amplitude) || positions_sb < 0) return FA_ERR_INVALID_ARG;
  if (!aligned(turns, 8) || (positions && !aligned(positions, 4))) return FA_ERR_MISALIGNED;
  return FA_OK;
}

// The cache's own sizes: pages of whole 16-key groups, positions and head
// rows of pages that fit 32 bits.
fa_status check_pages(const void* k_pages, const void* v_pages, int num_pages, int page_size, const int* block_table,
                      long long table_stride, int max_pages, int Hkv) {
  if (!k_pages || !v_pages || !block_table) return FA_ERR_INVALID_ARG;
  if (num_pages < 1 || max_pages < 1 || page_size < 16 || page_size % 16 != 0 || table_stride < 0)
    return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(max_pages) * page_size > 1LL << 30) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(num_pages) * Hkv >= 1LL << 31) return FA_ERR_INVALID_ARG;
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(block_table, 4)) return FA_ERR_MISALIGNED;
  return FA_OK;
}

fa_status paged_common(const void* q, const void* k_pages, const void* v_pages, int num_pages, int page_size,
                       const int* prefix_table, int prefix_len, const int* block_table, long long table_stride,
                       int max_pages, void* o, int o_dtype, float* lse, const int* seqlens_q, const int* seqlens_k,
                       float* workspace, int B, int Hq, int Hkv, int Nq, int d, float scale, int causal,
                       fa_stream_t stream) {
  if (!q || !o || !lse) return FA_ERR_INVALID_ARG;
  if (o_dtype != FA_DTYPE_F32 && o_dtype != FA_DTYPE_BF16) return FA_ERR_INVALID_ARG;
  fa_status st = check_sizes(B, Hq, Nq, d, causal);
  if (st != FA_OK) return st;
  if (Hkv < 1 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  st = check_pages(k_pages, v_pages, num_pages, page_size, block_table, table_stride, max_pages, Hkv);
  if (st != FA_OK) return st;
  // key tiles of all rows, in 32 bits
  const double key_tiles = (static_cast<double>(max_pages) * page_size + 63) / 64;
  const double row_tiles = static_cast<double>(B) * Hkv * (static_cast<double>(Hq / Hkv) * Nq / 256 + 1);
  if (key_tiles * row_tiles >= 2147483648.0) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || (workspace && !aligned(workspace, 16)) ||
      (seqlens_q && !aligned(seqlens_q, 4)) || (seqlens_k && !aligned(seqlens_k, 4)) ||
      (prefix_table && !aligned(prefix_table, 4)))
    return FA_ERR_MISALIGNED;
  DeviceInfo di;
  if (device_info(di) != FA_OK) return FA_ERR_LAUNCH;
  fa::PagedArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = static_cast<const uint16_t*>(q);
  a.table = fa::PageTable{block_table, table_stride, max_pages, page_size, num_pages};
  a.prefix_table = prefix_table;
  a.prefix_len = prefix_len;
  a.o = o;
  a.o_bf16 = o_dtype == FA_DTYPE_BF16;
  a.lse = lse;
  a.part = workspace;
  a.seqlens_q = seqlens_q;
  a.seqlens_k = seqlens_k;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.Nq = Nq;
  a.d = d;
  a.causal = causal;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.sms = di.sms;
  a.status = di.status;
  a.wait_limit_ns = wait_limit_ns();
  a.stall_unit = test_stall_unit();
  a.box_rows = page_size % 64 == 0 ? 64 : (page_size % 32 == 0 ? 32 : 16);
  const int page_heads = num_pages * Hkv;
  const bool steps = fa::paged_uses_steps(Hq / Hkv, Nq);
  auto page_map = [&](CUtensorMap* m, const void* pages, int box_rows, int blocked) {
    return encode_map(m, MapKey{pages, 2, page_heads, page_size, d, 64, box_rows, blocked});
  };
  if ((!steps || prefix_len > 0) &&
      (!page_map(&a.tm_k, k_pages, a.box_rows, 2) || !page_map(&a.tm_v, v_pages, a.box_rows, 2)))
    return FA_ERR_LAUNCH;
  const int rows = Hq / Hkv * Nq;  // below 2^31: checked above
  if (!steps && !encode_bf16_map(&a.tm_q, q, 1, B * Hq * Nq, d)) return FA_ERR_LAUNCH;
  // the prefix's row tiles in boxes, where 128 rows are whole sequences' rows
  // or a part of one's
  a.boxed_rows = prefix_len > 0 && (fa::kTileRows % rows == 0 || rows % fa::kTileRows == 0);
  if (a.boxed_rows) {
    MapKey key{q, 2, Hkv, rows, d, 64, rows < fa::kTileRows ? rows : fa::kTileRows};
    key.batch = B;
    key.box_batch = rows < fa::kTileRows ? fa::kTileRows / rows : 1;
    if (!encode_map(&a.tm_qp, key)) return FA_ERR_LAUNCH;
  }
  if (steps && (!page_map(&a.st_k, k_pages, a.box_rows, 1) || !page_map(&a.st_v, v_pages, a.box_rows, 1) ||
                !page_map(&a.st_k16, k_pages, 16, 1) || !page_map(&a.st_v16, v_pages, 16, 1)))
    return FA_ERR_LAUNCH;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!workspace) {
    // (a graph's allocations are its own, not the pool's)
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &capture) != cudaSuccess) return FA_ERR_LAUNCH;
    cudaMemPool_t pool = capture == cudaStreamCaptureStatusNone ? workspace_pool() : nullptr;
    const size_t bytes = sizeof(float) * fa::paged_workspace_floats(B, Hkv, Hq / Hkv, Nq, d, prefix_len > 0);
    const cudaError_t e = pool ? cudaMallocFromPoolAsync(reinterpret_cast<void**>(&a.part), bytes, pool, s)
                               : cudaMallocAsync(reinterpret_cast<void**>(&a.part), bytes, s);
    if (e != cudaSuccess) return FA_ERR_LAUNCH;
  }
  cudaError_t e = fa::launch_paged(a, s);
  if (!workspace) {
    cudaError_t e2 = cudaFreeAsync(a.part, s);
    if (e == cudaSuccess) e = e2;
  }
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // namespace

extern "C" {

fa_status fa_fwd(const void* q, const void* k, const void* v, float* o, float* lse, int B, int H, int N, int d,
                 float scale, int causal, fa_stream_t stream) {
  return fwd_common(q, k, v, o, FA_DTYPE_F32, lse, nullptr, nullptr, B, H, N, N, d, scale, causal, stream);
}

fa_status fa_fwd_varlen(const void* q, const void* k, const void* v, float* o, float* lse, const int* seqlens_q,
                        const int* seqlens_k, int B, int H, int Nq, int Nk, int d, float scale, int causal,
                        fa_stream_t stream) {
  return fwd_common(q, k, v, o, FA_DTYPE_F32, lse, seqlens_q, seqlens_k, B, H, Nq, Nk, d, scale, causal, stream);
}

fa_status fa_fwd_ex(const void* q, const void* k, const void* v, void* o, int o_dtype, float* lse,
                    const int* seqlens_q, const int* seqlens_k, int B, int H, int Nq, int Nk, int d, float scale,
                    int causal, fa_stream_t stream) {
  return fwd_common(q, k, v, o, o_dtype, lse, seqlens_q, seqlens_k, B, H, Nq, Nk, d, scale, causal, stream);
}

fa_status fa_fwd_bias(const void* q, const void* k, const void* v, void* o, int o_dtype, float* lse,
                      const void* bias, long long bias_stride_b, long long bias_stride_h, long long bias_stride_q,
                      const int* seqlens_q, const int* seqlens_k, int B, int H, int Nq, int Nk, int d, float scale,
                      int causal, fa_stream_t stream) {
  if (!bias) return FA_ERR_INVALID_ARG;  // fwd_common treats null as no mask
  return fwd_common(q, k, v, o, o_dtype, lse, seqlens_q, seqlens_k, B, H, Nq, Nk, d, scale, causal, stream, bias,
                    bias_stride_b, bias_stride_h, bias_stride_q);
}

size_t fa_fwd_splitkv_workspace_bytes(int B, int H, int N, int d) {
  if (B < 1 || H < 1 || N < 1 || (d != 64 && d != 128)) return 0;
  if (static_cast<long long>(B) * H * N >= (1LL << 31)) return 0;
  return static_cast<size_t>(B) * H * key_split_cap(N) * N * (d + 1) * sizeof(float);
}

fa_status fa_fwd_splitkv(const void* q, const void* k, const void* v, float* o, float* lse, float* workspace, int B,
                         int H, int N, int d, float scale, int causal, fa_stream_t stream) {
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  fa_status st = check_sizes(B, H, N, d, causal);
  if (st != FA_OK) return st;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
      (workspace && !aligned(workspace, 16)))
    return FA_ERR_MISALIGNED;
  DeviceInfo di;
  if (device_info(di) != FA_OK) return FA_ERR_LAUNCH;
  const int heads = B * H;
  int splits = 1, chunk = 1;
  key_splits(heads, N, di.sms, splits, chunk);
  if (splits == 1) return fwd_common(q, k, v, o, FA_DTYPE_F32, lse, nullptr, nullptr, B, H, N, N, d, scale, causal,
                                     stream);
  fa::FwdArgs a;
  std::memset(&a, 0, sizeof(a));
  if (!encode_bf16_map(&a.tm_q, q, heads, N, d) || !encode_bf16_map(&a.tm_k, k, heads, N, d) ||
      !encode_bf16_map(&a.tm_v, v, heads, N, d))
    return FA_ERR_LAUNCH;
  a.o = o;
  a.lse = lse;
  a.geom.nq = N;
  a.geom.nk = N;
  a.geom.heads_per_batch = H;
  a.d = d;
  a.causal = causal;
  a.scale_log2 = scale * 1.4426950408889634f;
  // units: (head, query pair, key split), heaviest pairs first under the
  // causal mask; splits of one pair are consecutive units
  a.sched = make_sched(heads, N, d, causal, di.sms, 0, fa::kUnitRows, 1, N);
  a.sched.units_per_head *= splits;
  const long long units = static_cast<long long>(heads) * a.sched.units_per_head;
  a.sched.grid = static_cast<int>(units < di.sms ? units : di.sms);
  a.splits = splits;
  a.chunk = chunk;
  a.status = di.status;
  a.wait_limit_ns = wait_limit_ns();
  a.stall_unit = test_stall_unit();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  float* part = workspace;
  if (!part) {
    if (cudaMallocAsync(reinterpret_cast<void**>(&part), fa_fwd_splitkv_workspace_bytes(B, H, N, d), s) !=
        cudaSuccess)
      return FA_ERR_LAUNCH;
  }
  a.part = part;
  cudaError_t e = fa::launch_fwd(a, s);
  if (!workspace) {
    cudaError_t e2 = cudaFreeAsync(part, s);
    if (e == cudaSuccess) e = e2;
  }
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

size_t fa_fwd_decode_workspace_bytes(int B, int H, int Nq, int Nk, int d) {
  if (B < 1 || H < 1 || Nq < 1 || Nq > FA_DECODE_MAX_Q || Nk < 1 || (d != 64 && d != 128)) return 0;
  if (static_cast<long long>(B) * H * Nk >= (1LL << 31)) return 0;
  return static_cast<size_t>(B) * H * decode_max_splits(Nk) * Nq * (d + 1) * sizeof(float);
}

fa_status fa_fwd_fp8(const void* q8, const void* k8, const void* vt8, float* o, float* lse, int B, int H, int N,
                     int d, float scale, int causal, fa_stream_t stream) {
  if (!q8 || !k8 || !vt8 || !o || !lse) return FA_ERR_INVALID_ARG;
  fa_status st = check_sizes(B, H, N, d, causal);
  if (st != FA_OK) return st;
  if (d != 128) return FA_ERR_UNSUPPORTED_D;
  if (N % 16 != 0) return FA_ERR_INVALID_ARG;  // rows of v^T: whole 16-byte groups
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (!aligned(q8, 16) || !aligned(k8, 16) || !aligned(vt8, 16) || !aligned(o, 16) || !aligned(lse, 4))
    return FA_ERR_MISALIGNED;
  DeviceInfo di;
  if (device_info(di) != FA_OK) return FA_ERR_LAUNCH;
  const int heads = B * H;
  fa::FwdArgs a;
  std::memset(&a, 0, sizeof(a));
  if (!encode_u8_map(&a.tm_q, q8, heads, N, d) || !encode_u8_map(&a.tm_k, k8, heads, N, d) ||
      !encode_u8_map(&a.tm_v, vt8, heads, d, N))
    return FA_ERR_LAUNCH;
  a.o = o;
  a.lse = lse;
  a.geom.nq = N;
  a.geom.nk = N;
  a.geom.heads_per_batch = H;
  a.d = d;
  a.causal = causal;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.sched = make_sched(heads, N, d, causal, di.sms, 0, fa::kUnitRows, 1, N);
  a.status = di.status;
  a.wait_limit_ns = wait_limit_ns();
  a.stall_unit = test_stall_unit();
  return fa::launch_fwd_fp8(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

fa_status fa_fwd_decode(const void* q, const void* k, const void* v, float* o, float* lse, const int* seqlens_q,
                        const int* seqlens_k, float* workspace, int B, int H, int Nq, int Nk, int d, float scale,
                        int causal, fa_stream_t stream) {
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  fa_status st = check_sizes(B, H, Nk, d, causal);
  if (st != FA_OK) return st;
  if (Nq < 1 || Nq > FA_DECODE_MAX_Q) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
      (workspace && !aligned(workspace, 16)) || (seqlens_q && !aligned(seqlens_q, 4)) ||
      (seqlens_k && !aligned(seqlens_k, 4)))
    return FA_ERR_MISALIGNED;
  DeviceInfo di;
  if (device_info(di) != FA_OK) return FA_ERR_LAUNCH;
  const int heads = B * H;
  fa::DecArgs a;
  std::memset(&a, 0, sizeof(a));
  if (!encode_bf16_map(&a.tm_k, k, heads, Nk, d, 64) || !encode_bf16_map(&a.tm_v, v, heads, Nk, d, 64))
    return FA_ERR_LAUNCH;
  a.q = static_cast<const uint16_t*>(q);
  a.o = o;
  a.lse = lse;
  a.geom.nq = Nq;
  a.geom.nk = Nk;
  a.geom.seqlens_q = seqlens_q;
  a.geom.seqlens_k = seqlens_k;
  a.geom.heads_per_batch = H;
  a.heads = heads;
  a.d = d;
  a.causal = causal;
  a.scale_log2 = scale * 1.4426950408889634f;
  decode_splits(heads, Nk, di.sms, a.splits, a.chunk);
  a.status = di.status;
  a.wait_limit_ns = wait_limit_ns();
  a.stall_unit = test_stall_unit();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  float* part = workspace;
  if (a.splits > 1 && !part) {
    if (cudaMallocAsync(reinterpret_cast<void**>(&part), fa_fwd_decode_workspace_bytes(B, H, Nq, Nk, d), s) !=
        cudaSuccess)
      return FA_ERR_LAUNCH;
  }
  a.part = part;
  cudaError_t e = fa::launch_decode(a, s);
  if (part && !workspace) {
    cudaError_t e2 = cudaFreeAsync(part, s);
    if (e == cudaSuccess) e = e2;
  }
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

size_t fa_bwd_workspace_bytes(int B, int H, int N) {
  if (B < 1 || H < 1 || N < 1) return 0;
  if (static_cast<long long>(B) * H * N >= (1LL << 31)) return 0;
  return static_cast<size_t>(B) * H * N * sizeof(float);
}

fa_status fa_bwd_ex(const void* q, const void* k, const void* v, const void* o, int o_dtype, const float* lse,
                    const void* dO, float* dq, float* dk, float* dv, float* workspace, const int* seqlens_q,
                    const int* seqlens_k, int B, int H, int Nq, int Nk, int d, float scale, int causal,
                    fa_stream_t stream) {
  fa::BwdArgs a;
  fa_status st = bwd_prepare(a, q, k, v, o, o_dtype, lse, dO, dq, dk, dv, workspace, seqlens_q, seqlens_k, B, H, Nq,
                             Nk, d, scale, causal);
  if (st != FA_OK) return st;
  return bwd_launch(a, workspace, B, H, Nq, stream);
}

fa_status fa_bwd_bias(const void* q, const void* k, const void* v, const void* o, int o_dtype, const float* lse,
                      const void* dO, const void* bias, long long bias_stride_b, long long bias_stride_h,
                      long long bias_stride_q, float* dq, float* dk, float* dv, float* workspace,
                      const int* seqlens_q, const int* seqlens_k, int B, int H, int Nq, int Nk, int d, float scale,
                      int causal, fa_stream_t stream) {
  fa_status st = check_bias(bias, bias_stride_b, bias_stride_h, bias_stride_q, Nk);
  if (st != FA_OK) return st;
  fa::BwdArgs a;
  st = bwd_prepare(a, q, k, v, o, o_dtype, lse, dO, dq, dk, dv, workspace, seqlens_q, seqlens_k, B, H, Nq, Nk, d,
                   scale, causal);
  if (st != FA_OK) return st;
  a.bias = fa::BiasRef{static_cast<const uint16_t*>(bias), bias_stride_b, bias_stride_h, bias_stride_q};
  return bwd_launch(a, workspace, B, H, Nq, stream);
}

fa_status fa_bwd_varlen(const void* q, const void* k, const void* v, const float* o, const float* lse,
                        const void* dO, float* dq, float* dk, float* dv, float* workspace, const int* seqlens_q,
                        const int* seqlens_k, int B, int H, int Nq, int Nk, int d, float scale, int causal,
                        fa_stream_t stream) {
  return fa_bwd_ex(q, k, v, o, FA_DTYPE_F32, lse, dO, dq, dk, dv, workspace, seqlens_q, seqlens_k, B, H, Nq, Nk, d,
                   scale, causal, stream);
}

fa_status fa_bwd(const void* q, const void* k, const void* v, const float* o, const float* lse, const void* dO,
                 float* dq, float* dk, float* dv, float* workspace, int B, int H, int N, int d, float scale,
                 int causal, fa_stream_t stream) {
  return fa_bwd_ex(q, k, v, o, FA_DTYPE_F32, lse, dO, dq, dk, dv, workspace, nullptr, nullptr, B, H, N, N, d, scale,
                   causal, stream);
}

// Scratch of fa_bwd_noalloc: the backward row term D for up to
// FA_NOALLOC_MAX_ROWS rows, resident on every device that loads the library.
// Host code must not hand this name to a kernel (on the host it is only a
// stand-in for the symbol); the device address comes from
// cudaGetSymbolAddress, looked up once per device.
static __device__ __align__(256) float g_fa_noalloc_delta[FA_NOALLOC_MAX_ROWS];

static std::mutex g_noalloc_mu;
static float* g_noalloc_ptr[kMaxDevices];

fa_status fa_bwd_noalloc(const void* q, const void* k, const void* v, const float* o, const float* lse,
                         const void* dO, float* dq, float* dk, float* dv, int B, int H, int N, int d, float scale,
                         int causal, fa_stream_t stream) {
  // the scratch bound first, before any descriptor is built
  if (B < 1 || H < 1 || N < 1 || static_cast<long long>(B) * H * N > FA_NOALLOC_MAX_ROWS) return FA_ERR_INVALID_ARG;
  fa::BwdArgs a;
  fa_status st =
      bwd_prepare(a, q, k, v, o, FA_DTYPE_F32, lse, dO, dq, dk, dv, nullptr, nullptr, nullptr, B, H, N, N, d, scale,
                  causal);
  if (st != FA_OK) return st;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_LAUNCH;
  {
    std::lock_guard<std::mutex> lock(g_noalloc_mu);
    if (!g_noalloc_ptr[dev]) {
      void* p = nullptr;
      if (cudaGetSymbolAddress(&p, g_fa_noalloc_delta) != cudaSuccess || !p) return FA_ERR_LAUNCH;
      g_noalloc_ptr[dev] = static_cast<float*>(p);
    }
    a.delta = g_noalloc_ptr[dev];  // every row is written by the dQ kernel before dK/dV reads it
  }
  return fa::launch_bwd(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

fa_status fa_bwd_single_pass(const void* q, const void* k, const void* v, const float* lse, const void* dO,
                             const void* bias, long long bias_stride_b, long long bias_stride_h,
                             long long bias_stride_q, float* dq, float* dk, float* dv, float* workspace,
                             const int* seqlens_q, const int* seqlens_k, int B, int H, int Nq, int Nk, int d,
                             float scale, int causal, fa_stream_t stream) {
  if (bias) {
    const fa_status bs = check_bias(bias, bias_stride_b, bias_stride_h, bias_stride_q, Nk);
    if (bs != FA_OK) return bs;
  }
  fa::BwdArgs a;
  fa_status st = bwd_prepare(a, q, k, v, nullptr, FA_DTYPE_F32, lse, dO, dq, dk, dv, workspace, seqlens_q, seqlens_k,
                             B, H, Nq, Nk, d, scale, causal, false);
  if (st != FA_OK) return st;
  if (bias) a.bias = fa::BiasRef{static_cast<const uint16_t*>(bias), bias_stride_b, bias_stride_h, bias_stride_q};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  float* delta = workspace;
  if (!delta) {
    if (cudaMallocAsync(reinterpret_cast<void**>(&delta), fa_bwd_workspace_bytes(B, H, Nq), s) != cudaSuccess)
      return FA_ERR_LAUNCH;
  }
  a.delta = delta;
  cudaError_t e = fa::launch_bwd_single_pass(a, s);
  if (!workspace) {
    cudaError_t e2 = cudaFreeAsync(delta, s);
    if (e == cudaSuccess) e = e2;
  }
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

fa_status fa_bwd_stage(int stage, const void* q, const void* k, const void* v, const float* o, const float* lse,
                       const void* dO, float* dq, float* dk, float* dv, float* workspace, int B, int H, int N, int d,
                       float scale, int causal, fa_stream_t stream) {
  if (stage < 0 || stage > 3 || !workspace) return FA_ERR_INVALID_ARG;
  fa::BwdArgs a;
  fa_status st =
      bwd_prepare(a, q, k, v, o, FA_DTYPE_F32, lse, dO, dq, dk, dv, workspace, nullptr, nullptr, B, H, N, N, d, scale,
                  causal, stage < 2);
  if (st != FA_OK) return st;
  a.delta = workspace;
  return fa::launch_bwd_stage(a, stage, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK
                                                                                              : FA_ERR_LAUNCH;
}

fa_status fa_rope_turns(long long* turns, int rot_dim, double base, int scaling, double factor, double original_len,
                        double low, double high) {
  if (!turns || rot_dim < 16 || rot_dim % 16 != 0 || !std::isfinite(base) || !(base > 1.0)) return FA_ERR_INVALID_ARG;
  if (scaling < FA_ROPE_SCALE_NONE || scaling > FA_ROPE_SCALE_PARTS) return FA_ERR_INVALID_ARG;
  if (scaling != FA_ROPE_SCALE_NONE && (!std::isfinite(factor) || !(factor >= 1.0))) return FA_ERR_INVALID_ARG;
  if (scaling == FA_ROPE_SCALE_PARTS &&
      (!std::isfinite(original_len) || !(original_len > 0.0) || !std::isfinite(low) || !std::isfinite(high) ||
       !(low >= 0.0) || !(high > low)))
    return FA_ERR_INVALID_ARG;
  constexpr double kTwoPi = 6.283185307179586;
  if (scaling == FA_ROPE_SCALE_NTK) base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
  if (!std::isfinite(base)) return FA_ERR_INVALID_ARG;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);  // radians per position
    if (scaling == FA_ROPE_SCALE_LINEAR) f /= factor;
    if (scaling == FA_ROPE_SCALE_PARTS) {
      double keep = (f * original_len / kTwoPi - low) / (high - low);
      keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
      f = f * keep + f / factor * (1.0 - keep);
    }
    turns[i] = std::llround(std::ldexp(f / kTwoPi, 64));  // f <= 1: below 2^62
  }
  return FA_OK;
}

fa_status fa_rope(const void* x, int x_dtype, long long x_stride_b, long long x_stride_h, long long x_stride_n,
                  void* y, int y_dtype, long long y_stride_b, long long y_stride_h, long long y_stride_n,
                  const int* positions, long long positions_stride_b, const long long* turns, int rot_dim, int layout,
                  float amplitude, int inverse, int B, int H, int N, int d, fa_stream_t stream) {
  if (!x || !y || (inverse != 0 && inverse != 1)) return FA_ERR_INVALID_ARG;
  if ((x_dtype != FA_DTYPE_F32 && x_dtype != FA_DTYPE_BF16) || (y_dtype != FA_DTYPE_F32 && y_dtype != FA_DTYPE_BF16))
    return FA_ERR_INVALID_ARG;
  fa_status st = check_sizes(B, H, N, d, 0);
  if (st != FA_OK) return st;
  st = check_rope(turns, rot_dim, layout, amplitude, positions, positions_stride_b, d);
  if (st != FA_OK) return st;
  const int xe = x_dtype == FA_DTYPE_BF16 ? 2 : 4, ye = y_dtype == FA_DTYPE_BF16 ? 2 : 4;
  const fa::Strides xs = used_strides(x_stride_b, x_stride_h, x_stride_n, B, H, N);
  const fa::Strides ys = used_strides(y_stride_b, y_stride_h, y_stride_n, B, H, N);
  // in place only element for element
  if (x == y && (x_dtype != y_dtype || xs.b != ys.b || xs.h != ys.h || xs.n != ys.n)) return FA_ERR_INVALID_ARG;
  if ((st = check_strides(xs, xe)) != FA_OK || (st = check_strides(ys, ye)) != FA_OK) return st;
  if (rows_overlap(ys, B, H, N, d)) return FA_ERR_INVALID_ARG;  // they would race
  if (!aligned(x, 16) || !aligned(y, 16)) return FA_ERR_MISALIGNED;
  DeviceInfo di;
  if (device_info(di) != FA_OK) return FA_ERR_LAUNCH;
  fa::RopeArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x;
  a.y = y;
  a.x_bf16 = x_dtype == FA_DTYPE_BF16;
  a.y_bf16 = y_dtype == FA_DTYPE_BF16;
  a.xs = xs;
  a.ys = ys;
  a.rope = fa::RopeRef{turns, positions, positions_stride_b, rot_dim, layout == FA_ROPE_INTERLEAVED, amplitude};
  a.inverse = inverse;
  a.B = B;
  a.H = H;
  a.N = N;
  a.d = d;
  a.sms = di.sms;
  return fa::launch_rope(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

fa_status fa_kv_append(const void* k, long long k_stride_b, long long k_stride_h, long long k_stride_n, const void* v,
                       long long v_stride_b, long long v_stride_h, long long v_stride_n, const void* q,
                       long long q_stride_b, long long q_stride_h, long long q_stride_n, void* q_out, void* k_pages,
                       void* v_pages, int num_pages, int page_size, const int* block_table, long long table_stride,
                       int max_pages, const int* seqlens_q, const int* seqlens_k, const int* positions,
                       long long positions_stride_b, const long long* turns, int rot_dim, int layout, float amplitude,
                       int B, int Hq, int Hkv, int N, int d, fa_stream_t stream) {
  if (!k || !v || !seqlens_k || (q != nullptr) != (q_out != nullptr)) return FA_ERR_INVALID_ARG;
  fa_status st = check_sizes(B, Hkv, N, d, 0);
  if (st != FA_OK) return st;
  if (q) {
    st = check_sizes(B, Hq, N, d, 0);
    if (st != FA_OK) return st;
  }
  if (turns) {
    st = check_rope(turns, rot_dim, layout, amplitude, positions, positions_stride_b, d);
    if (st != FA_OK) return st;
  } else if (positions) {
    return FA_ERR_INVALID_ARG;  // positions of a rotation that is not asked for
  }
  st = check_pages(k_pages, v_pages, num_pages, page_size, block_table, table_stride, max_pages, Hkv);
  if (st != FA_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(seqlens_k, 4) || (seqlens_q && !aligned(seqlens_q, 4)))
    return FA_ERR_MISALIGNED;
  const fa::Strides ks = used_strides(k_stride_b, k_stride_h, k_stride_n, B, Hkv, N);
  const fa::Strides vs = used_strides(v_stride_b, v_stride_h, v_stride_n, B, Hkv, N);
  if ((st = check_strides(ks, 2)) != FA_OK || (st = check_strides(vs, 2)) != FA_OK) return st;
  fa::Strides qs{0, 0, 0};
  if (q) {
    if (!aligned(q, 16) || !aligned(q_out, 16)) return FA_ERR_MISALIGNED;
    qs = used_strides(q_stride_b, q_stride_h, q_stride_n, B, Hq, N);
    if ((st = check_strides(qs, 2)) != FA_OK) return st;
    // q_out is contiguous: in place only for a contiguous q
    const fa::Strides cs = used_strides(static_cast<long long>(Hq) * N * d, static_cast<long long>(N) * d, d, B, Hq, N);
    if (q == q_out && (qs.b != cs.b || qs.h != cs.h || qs.n != cs.n)) return FA_ERR_INVALID_ARG;
  }
  DeviceInfo di;
  if (device_info(di) != FA_OK) return FA_ERR_LAUNCH;
  fa::AppendArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.qs = qs;
  a.ks = ks;
  a.vs = vs;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_pages = static_cast<uint16_t*>(k_pages);
  a.v_pages = static_cast<uint16_t*>(v_pages);
  a.table = fa::PageTable{block_table, table_stride, max_pages, page_size, num_pages};
  if (turns)
    a.rope = fa::RopeRef{turns, positions, positions_stride_b, rot_dim, layout == FA_ROPE_INTERLEAVED, amplitude};
  a.seqlens_q = seqlens_q;
  a.seqlens_k = seqlens_k;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.N = N;
  a.d = d;
  a.sms = di.sms;
  a.status = di.status;
  return fa::launch_kv_append(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

static size_t paged_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d, bool with_prefix) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Nq < 1 || Hq % Hkv != 0 || (d != 64 && d != 128)) return 0;
  if (static_cast<long long>(B) * Hq * Nq >= (1LL << 31)) return 0;
  return sizeof(float) * fa::paged_workspace_floats(B, Hkv, Hq / Hkv, Nq, d, with_prefix);
}

size_t fa_fwd_paged_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d) {
  return paged_workspace_bytes(B, Hq, Hkv, Nq, d, false);
}

fa_status fa_fwd_paged(const void* q, const void* k_pages, const void* v_pages, int num_pages, int page_size,
                       const int* block_table, long long table_stride, int max_pages, void* o, int o_dtype,
                       float* lse, const int* seqlens_q, const int* seqlens_k, float* workspace, int B, int Hq,
                       int Hkv, int Nq, int d, float scale, int causal, fa_stream_t stream) {
  return paged_common(q, k_pages, v_pages, num_pages, page_size, nullptr, 0, block_table, table_stride, max_pages, o,
                      o_dtype, lse, seqlens_q, seqlens_k, workspace, B, Hq, Hkv, Nq, d, scale, causal, stream);
}

size_t fa_fwd_shared_prefix_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d) {
  return paged_workspace_bytes(B, Hq, Hkv, Nq, d, true);
}

fa_status fa_fwd_shared_prefix(const void* q, const void* k_pages, const void* v_pages, int num_pages, int page_size,
                               const int* prefix_table, int prefix_len, const int* block_table,
                               long long table_stride, int max_pages, void* o, int o_dtype, float* lse,
                               const int* seqlens_q, const int* seqlens_k, float* workspace, int B, int Hq, int Hkv,
                               int Nq, int d, float scale, int causal, fa_stream_t stream) {
  if (!prefix_table || page_size < 16 || prefix_len < page_size || prefix_len % page_size != 0)
    return FA_ERR_INVALID_ARG;
  if (prefix_len / page_size > max_pages) return FA_ERR_INVALID_ARG;
  return paged_common(q, k_pages, v_pages, num_pages, page_size, prefix_table, prefix_len, block_table, table_stride,
                      max_pages, o, o_dtype, lse, seqlens_q, seqlens_k, workspace, B, Hq, Hkv, Nq, d, scale, causal,
                      stream);
}

fa_status fa_sync_status(fa_stream_t stream) {
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return FA_ERR_DEVICE_FAULT;
  int h[4] = {0, 0, 0, 0};
  if (cudaMemcpyFromSymbol(h, g_fa_status, sizeof(h)) != cudaSuccess) return FA_ERR_DEVICE_FAULT;
  if (h[0] != 0) {
    {
      std::lock_guard<std::mutex> lock(g_mu);
      std::memcpy(g_last_failure, h, sizeof(h));
    }
    const int zero[4] = {0, 0, 0, 0};
    if (cudaMemcpyToSymbol(g_fa_status, zero, sizeof(zero)) != cudaSuccess) return FA_ERR_DEVICE_FAULT;
    return h[0] == FA_ERR_TIMEOUT || h[0] == FA_ERR_BAD_PAGE ? static_cast<fa_status>(h[0]) : FA_ERR_DEVICE_FAULT;
  }
  return FA_OK;
}

fa_status fa_test_set_stall(int unit) {
  if (unit < -1) return FA_ERR_INVALID_ARG;
  stall_unit_cell().store(unit, std::memory_order_relaxed);
  return FA_OK;
}

long long fa_test_map_encodes(void) {
  std::lock_guard<std::mutex> lock(g_map_mu);
  return g_map_encodes;
}

fa_status fa_last_failure(int out[4]) {
  if (!out) return FA_ERR_INVALID_ARG;
  std::lock_guard<std::mutex> lock(g_mu);
  std::memcpy(out, g_last_failure, sizeof(g_last_failure));
  return FA_OK;
}

const char* fa_status_string(fa_status s) {
  switch (s) {
    case FA_OK: return "FA_OK: success";
    case FA_ERR_INVALID_ARG: return "FA_ERR_INVALID_ARG: null pointer or size/flag out of range";
    case FA_ERR_UNSUPPORTED_D: return "FA_ERR_UNSUPPORTED_D: head dimension must be 64 or 128";
    case FA_ERR_MISALIGNED: return "FA_ERR_MISALIGNED: tensor pointer breaks the 16-byte (4-byte) alignment rule";
    case FA_ERR_LAUNCH: return "FA_ERR_LAUNCH: the CUDA runtime refused a launch or an allocation";
    case FA_ERR_TIMEOUT: return "FA_ERR_TIMEOUT: a kernel pipeline wait ran past its limit";
    case FA_ERR_DEVICE_FAULT: return "FA_ERR_DEVICE_FAULT: the stream reported a CUDA error";
    case FA_ERR_BAD_PAGE:
      return "FA_ERR_BAD_PAGE: a block table names a page outside the cache, or ends before an appended token";
  }
  return "unknown fa_status";
}

long long fa_sched_enumerate(int heads, int N, int d, int causal, int grid, long long l2_budget_bytes,
                             int* out_cta, int* out_head, int* out_pair, long long capacity) {
  if (heads < 1 || N < 1 || grid < 1 || (d != 64 && d != 128) || (causal != 0 && causal != 1)) return -1;
  if (static_cast<long long>(heads) * N >= (1LL << 31)) return -1;
  fa::SchedParams sp = make_sched(heads, N, d, causal, grid, l2_budget_bytes);
  long long w = 0;
  for (int c = 0; c < sp.grid; ++c) {
    fa::SchedIter it = fa::sched_begin(sp);
    int head, pair;
    while (fa::sched_next(it, sp, c, head, pair)) {
      if (w < capacity && out_cta && out_head && out_pair) {
        out_cta[w] = c;
        out_head[w] = head;
        out_pair[w] = pair;
      }
      ++w;
    }
  }
  return w;
}

}  // extern "C"
