// Pages of the cache between sequences: forks, which share, copy and free pages,
// and compaction.
//
// What happens to the tables and counts is a chain of a few short passes over
// them, each of which needs the one before it whole, and the data are small (a
// count a page, an entry a page of a sequence): one cluster of eight CTAs does
// it, with the cluster's barrier between passes, so that a call is this launch
// and the copy's.  Everything is decided by ids and orders (the first row that
// continues a sequence, the free pages of the lowest ids), never by which thread
// comes first: additions to a count are atomic and commute.
//
// The copy of whole pages is bound by HBM (a byte read and a byte written).  Where many
// rows copy one page it comes from L2, half the bytes go to DRAM, and the instructions
// bound it (128 samples: issue slots 74% busy, DRAM 46%); a few tokens of a few
// sequences are launch latency.  It reads the list of pages and its length on the
// device.
//
// Measured, in a graph: 128 samples of two prompts of 1001 and 4000 tokens, each with
// a page of its own in the tensors of 8 layers, 72 to 75 us; about 300 of 1200 pages moved
// (in E4M3, 8 layers) 106 to 112 us = 5.6 to 5.9 TB/s; a beam search's reordering of 16 rows 12.2 us
// and a small cache's compaction 10.5, of which the tables' passes are about 8 and 7:
// chains of loads and atomics, a microsecond or more each.  One after the other in
// every thread where they now run side by side, and one more, 13.7; one, two and four
// CTAs 13.4, 13.2 and 13.1 (128 samples 77.1, 75.7, 75.4).
#include <cuda_runtime.h>

#include <climits>

#include "serving.h"

namespace fa {
namespace {

constexpr int kPlanCtas = 8;          // the largest portable cluster
constexpr int kPlanThreads = 1024;
constexpr int kPerThread = 4;         // pages a thread looks at in a step of a scan
constexpr int kCopyThreads = 256;
constexpr int kInFlight = 4;          // 16-byte loads of a thread's
constexpr long long kSliceBytes = 32 << 10;  // of a page and tensor that one CTA copies at a time

// The workspace in 4-byte words: what the passes hand on.
struct PlanSpace {
  int* pairs;      // pages to copy
  int* counts;     // [kPlanCtas][2] of each CTA's part of the pages
  int* list_a;     // fork: free pages by rank; compaction: holes
  int* list_b;     // fork: ranks of the rows that need a page, else -1; compaction: pages that move
  int* first;      // fork: the first row that continues each sequence
  PageCopy* copies;
};

constexpr size_t kPlanHead = 4 + 2 * kPlanCtas;  // words before the lists

// `lists`: words of either list; `copies`: most pages to copy.
__host__ __device__ inline PlanSpace plan_space(int* base, long long list_a, long long list_b, long long first) {
  PlanSpace s;
  s.pairs = base;
  s.counts = base + 4;
  s.list_a = base + kPlanHead;
  s.list_b = s.list_a + list_a;
  s.first = s.list_b + list_b;
  s.copies = reinterpret_cast<PageCopy*>(s.first + first);
  return s;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive prefix sums of the block's v, and their total.
__device__ __forceinline__ int block_scan(int v, int* scratch, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();  // the scratch words of the last scan have been read
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  const int mine = lane < kPlanThreads / 32 ? scratch[lane] : 0;
  int sum = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, sum, off);
    if (lane >= off) sum += y;
  }
  total = __shfl_sync(0xffffffffu, sum, 31);
  return __shfl_sync(0xffffffffu, sum - mine, warp) + x - v;
}

// Walks over pages [begin, end) in order: found(page, rank) for those of which
// is(page), ranks counted from `rank` on; returns the rank behind the last.
template <typename Is, typename Found>
__device__ __forceinline__ int scan_pages(int begin, int end, int rank, int* scratch, Is is, Found found) {
  constexpr int STEP = kPlanThreads * kPerThread;
  for (long long base = begin; base < end; base += STEP) {
    const int p0 = static_cast<int>(base) + static_cast<int>(threadIdx.x) * kPerThread;
    bool flag[kPerThread];
    int n = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      flag[i] = p0 < end - i && is(p0 + i);
      n += flag[i];
    }
    int total, at = rank + block_scan(n, scratch, total);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
      if (flag[i]) found(p0 + i, at++);
    rank += total;
  }
  return rank;
}

// How many pages of [begin, end) are; the same in every thread.
template <typename Is>
__device__ __forceinline__ int count_pages(int begin, int end, int* scratch, Is is) {
  int n = 0;
  for (long long p = begin + static_cast<int>(threadIdx.x); p < end; p += kPlanThreads) n += is(static_cast<int>(p));
  int total;
  block_scan(n, scratch, total);
  return total;
}

__device__ __forceinline__ int used_pages(int len, int page_size) {
  return static_cast<int>((static_cast<unsigned>(len) + page_size - 1) / page_size);
}

__global__ void __cluster_dims__(kPlanCtas) __launch_bounds__(kPlanThreads, 1) fork_kernel(const ForkArgs a) {
  __shared__ int scratch[32];
  grid_trigger();
  const int cta = blockIdx.x;
  const unsigned tid = blockIdx.x * kPlanThreads + threadIdx.x;
  constexpr unsigned ALL = kPlanCtas * kPlanThreads;
  const PlanSpace w = plan_space(a.workspace, a.rows, a.rows, a.B);
  const int page_size = a.table.page_size, width = a.table.max_pages;
  auto length = [&](int b) { return min(max(a.seqlens[b], 0), width * page_size); };
  auto source = [&](int i) {
    const int s = a.sources[i];
    return s >= 0 && s < a.B ? s : -1;
  };
  // the table's entry, reported (as `row`'s) if it names no page
  auto entry = [&](int b, int i, int row) {
    const int p = a.table.block_table[b * a.table.table_stride + i];
    const bool good = p >= 0 && p < a.table.num_pages;
    if (!good && row >= 0) record_bad_page(a.status, SITE_PAGE_FORK, row, p);
    return good ? p : -1;
  };
  for (unsigned p = tid; p < static_cast<unsigned>(a.table.num_pages); p += ALL) a.out_refs[p] = a.refs[p];
  for (unsigned b = tid; b < static_cast<unsigned>(a.B); b += ALL) w.first[b] = INT_MAX;
  cluster_sync();
  // the old rows let go of their pages, the new ones take the full ones
  // (one walk over all three, so that a small call's threads have one chain of
  // loads each instead of three)
  const long long new_from = static_cast<long long>(a.B) * width;
  const long long rows_from = new_from + static_cast<long long>(a.rows) * width;
  for (long long x = tid; x < rows_from + a.rows; x += ALL) {
    if (x < new_from) {
      const int b = static_cast<int>(x / width), i = static_cast<int>(x - static_cast<long long>(b) * width);
      if (i >= used_pages(length(b), page_size)) continue;
      const int p = entry(b, i, b);
      if (p >= 0) atomicAdd(a.out_refs + p, -1);
    } else if (x < rows_from) {
      const long long y = x - new_from;
      const int row = static_cast<int>(y / width), i = static_cast<int>(y - static_cast<long long>(row) * width);
      const int s = source(row), len = s >= 0 ? length(s) : 0;
      int out = -1;
      if (i < used_pages(len, page_size)) {
        const int p = entry(s, i, -1);
        out = a.table.block_table[s * a.table.table_stride + i];
        if (p >= 0 && i < len / page_size) atomicAdd(a.out_refs + p, 1);
      }
      a.out_table[row * a.out_stride + i] = out;
    } else {
      const int row = static_cast<int>(x - rows_from);
      const int s = source(row), len = s >= 0 ? length(s) : 0;
      a.out_seqlens[row] = len;
      // a page that is being filled stays with the sequence's first row: one row
      // counts it, whichever finds that none has been here
      if (s >= 0 && atomicMin(w.first + s, row) == INT_MAX && len % page_size) {
        const int p = entry(s, len / page_size, -1);
        if (p >= 0) atomicAdd(a.out_refs + p, 1);
      }
    }
  }
  cluster_sync();
  // whether a row that is not the first needs a page in its place
  auto needs = [&](int row) {
    const int s = source(row), len = s >= 0 ? length(s) : 0;
    return len % page_size && __ldcg(w.first + s) != row && entry(s, len / page_size, -1) >= 0;
  };
  // the free pages of the lowest ids, by rank, and the rows' ranks
  constexpr int COUNTING = kPlanCtas - 1;  // CTAs; the last one ranks the rows meanwhile
  const int part = (a.table.num_pages + COUNTING - 1) / COUNTING;
  const long long all = a.table.num_pages;
  const int begin = static_cast<int>(min(static_cast<long long>(cta) * part, all));
  const int end = static_cast<int>(min(static_cast<long long>(begin) + part, all));
  auto is_free = [&](int p) { return __ldcg(a.out_refs + p) == 0; };
  if (cta < COUNTING) {
    const int mine = count_pages(begin, end, scratch, is_free);
    if (threadIdx.x == 0) w.counts[cta] = mine;
  } else {
    int needed = 0;
    for (int base = 0; base < a.rows; base += kPlanThreads) {
      const int row = base + static_cast<int>(threadIdx.x);
      const int need = row < a.rows && needs(row);
      int total;
      const int rank = needed + block_scan(need, scratch, total);
      if (row < a.rows) w.list_b[row] = need ? rank : -1;
      needed += total;
    }
    if (threadIdx.x == 0) w.pairs[0] = needed;
  }
  cluster_sync();
  int before = 0, found = 0;
  for (int c = 0; c < COUNTING; ++c) {
    const int n = __ldcg(w.counts + c);
    if (c < cta) before += n;
    found += n;
  }
  const int needed = __ldcg(w.pairs);
  if (cta < COUNTING && before < needed)
    scan_pages(begin, end, before, scratch, is_free, [&](int p, int rank) {
      if (rank < needed) w.list_a[rank] = p;
    });
  cluster_sync();
  for (unsigned row = tid; row < static_cast<unsigned>(a.rows); row += ALL) {
    const int rank = __ldcg(w.list_b + row);
    if (rank < 0) continue;
    const int s = source(row), len = length(s), i = len / page_size;
    int page = -1;
    if (rank < found) {
      page = __ldcg(w.list_a + rank);
      a.out_refs[page] = 1;
      w.copies[rank] = PageCopy{a.table.block_table[s * a.table.table_stride + i], page, len % page_size};
    } else if (rank == found) {
      record_failure_at(a.status, FA_DEV_NO_PAGES, SITE_NO_PAGES, static_cast<int>(row), needed - found);
    }
    a.out_table[row * a.out_stride + i] = page;
  }
  if (tid == 0) w.pairs[1] = min(needed, found);
}

__global__ void __cluster_dims__(kPlanCtas) __launch_bounds__(kPlanThreads, 1) compact_kernel(const CompactArgs a) {
  __shared__ int scratch[32];
  grid_trigger();
  const int cta = blockIdx.x;
  const unsigned tid = blockIdx.x * kPlanThreads + threadIdx.x;
  constexpr unsigned ALL = kPlanCtas * kPlanThreads;
  const int pages = a.table.num_pages;
  const PlanSpace w = plan_space(a.workspace, pages / 2, pages / 2, 0);
  const int part = (pages + kPlanCtas - 1) / kPlanCtas;
  const int begin = static_cast<int>(min(static_cast<long long>(cta) * part, static_cast<long long>(pages)));
  const int end = static_cast<int>(min(static_cast<long long>(begin) + part, static_cast<long long>(pages)));
  const int mine = count_pages(begin, end, scratch, [&](int p) { return a.refs[p] > 0; });
  if (threadIdx.x == 0) w.counts[cta] = mine;
  cluster_sync();
  int live = 0, used_before = 0;  // pages in use, and those before this CTA's part
  for (int c = 0; c < kPlanCtas; ++c) {
    const int n = __ldcg(w.counts + c);
    if (c < cta) used_before += n;
    live += n;
  }
  // Holes are the free pages below `live`, as many as pages in use lie at or
  // behind it: a part's ranks follow from the pages in use before it.
  auto holes_before = [&](int p, int used) { return min(p, live) - used; };  // for p <= live
  const int split = min(max(live, begin), end);
  if (begin < split)
    scan_pages(begin, split, holes_before(begin, used_before), scratch, [&](int p) { return a.refs[p] <= 0; },
               [&](int p, int rank) { w.list_a[rank] = p; });
  int used_low = 0;  // pages in use below `live`
  {
    // of the parts wholly below it all, of the one that it falls into those of
    // [its begin, live): counted by every CTA alike
    const int whole = live / part;
    for (int c = 0; c < whole && c < kPlanCtas; ++c) used_low += __ldcg(w.counts + c);
    if (whole < kPlanCtas)
      used_low += count_pages(static_cast<int>(min(static_cast<long long>(whole) * part, static_cast<long long>(live))),
                              live, scratch, [&](int p) { return a.refs[p] > 0; });
  }
  const int moves = live - used_low;
  if (split < end) {
    // pages in use at or behind `live`, before this part's
    const int from = begin <= live ? 0 : used_before - used_low;
    scan_pages(split, end, from, scratch, [&](int p) { return a.refs[p] > 0; },
               [&](int p, int rank) { w.list_b[rank] = p; });
  }
  for (unsigned p = tid; p < static_cast<unsigned>(pages); p += ALL) {
    const int r = a.refs[p];
    const bool stays = static_cast<int>(p) < live && r > 0;
    if (stays || r <= 0) a.new_ids[p] = r > 0 ? static_cast<int>(p) : -1;
    if (stays || static_cast<int>(p) >= live) a.out_refs[p] = stays ? r : 0;
  }
  cluster_sync();
  for (unsigned j = tid; j < static_cast<unsigned>(moves); j += ALL) {
    const int to = __ldcg(w.list_a + j), from = __ldcg(w.list_b + j);
    a.new_ids[from] = to;
    a.out_refs[to] = a.refs[from];
    w.copies[j] = PageCopy{from, to, a.table.page_size};
  }
  if (tid == 0) w.pairs[1] = moves;
  cluster_sync();
  const int width = a.table.max_pages, page_size = a.table.page_size;
  for (long long x = tid; x < static_cast<long long>(a.B) * width; x += ALL) {
    const int b = static_cast<int>(x / width), i = static_cast<int>(x - static_cast<long long>(b) * width);
    const int len = min(max(a.seqlens[b], 0), width * page_size);
    const int p = a.table.block_table[b * a.table.table_stride + i];
    int out = p;
    if (i < used_pages(len, page_size)) {
      const int to = p >= 0 && p < pages ? __ldcg(a.new_ids + p) : -1;
      if (to >= 0)
        out = to;
      else
        record_bad_page(a.status, SITE_PAGE_COMPACT, b, p);
    }
    a.out_table[b * a.out_stride + i] = out;
  }
}

// Copies the first tokens' rows of every head, for the list's pages and the
// tensors of this launch; a CTA takes a slice of a page of a tensor at a time.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyArgs a) {
  grid_wait();
  const PlanSpace w = plan_space(a.workspace, a.list_a, a.list_b, a.first);
  const long long items = static_cast<long long>(__ldcg(w.pairs + 1)) * a.slices;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const int j = static_cast<int>(item / a.slices);
    const int slice = static_cast<int>(item - static_cast<long long>(j) * a.slices);
    // the tensor that the slice belongs to: the first that ends behind it
    int t = 0;
    for (int last = a.count - 1; t < last;) {
      const int mid = (t + last) >> 1;
      if (slice >= a.t[mid].slice_end) t = mid + 1; else last = mid;
    }
    const PageTensor& x = a.t[t];
    const int before = t > 0 ? a.t[t - 1].slice_end : 0;
    const int of = x.slice_end - before, in = slice - before;
    const PageCopy c = w.copies[j];
    const int unit = a.page_size / x.rows;                 // tokens of a row
    const int rows = (c.tokens + unit - 1) / unit;
    const long long page_bytes = static_cast<long long>(x.heads) * x.rows * x.row_bytes;
    const uint8_t* src = x.base + c.src * page_bytes;
    uint8_t* dst = x.base + c.dst * page_bytes;
    auto copy = [&](auto word) {
      using W = decltype(word);
      constexpr unsigned SIZE = sizeof(W);
      // words of a head (a page's: below 2^31)
      const unsigned head = static_cast<unsigned>(x.rows) * x.row_bytes / SIZE;
      const unsigned have = static_cast<unsigned>(rows) * x.row_bytes / SIZE;    // to copy of one
      const unsigned all = have * x.heads;
      const unsigned from = static_cast<unsigned>(static_cast<unsigned long long>(all) * in / of);
      const unsigned to = static_cast<unsigned>(static_cast<unsigned long long>(all) * (in + 1) / of);
      const bool whole = have == head;
      for (unsigned i0 = from + threadIdx.x; i0 < to; i0 += kCopyThreads * kInFlight) {
        W v[kInFlight];
        unsigned at[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
          const unsigned i = i0 + u * kCopyThreads;
          if (i < to) {
            const unsigned h = whole ? 0 : i / have;
            at[u] = h * head + (i - h * have);
            v[u] = __ldcs(reinterpret_cast<const W*>(src) + at[u]);
          }
        }
#pragma unroll
        for (int u = 0; u < kInFlight; ++u)
          if (i0 + u * kCopyThreads < to) __stcs(reinterpret_cast<W*>(dst) + at[u], v[u]);
      }
    };
    if (x.wide) copy(uint4{}); else copy(0u);
  }
}

// Copies for all tensors, at most kCopyTensors a launch.
cudaError_t launch_copies(CopyArgs& c, const PageTensor* tensors, int count, long long most, int sms,
                          cudaStream_t stream) {
  for (int t0 = 0; t0 < count; t0 += kCopyTensors) {
    const int n = count - t0 < kCopyTensors ? count - t0 : kCopyTensors;
    int slices = 0;
    for (int i = 0; i < n; ++i) {
      c.t[i] = tensors[t0 + i];
      const long long bytes = static_cast<long long>(c.t[i].heads) * c.t[i].rows * c.t[i].row_bytes;
      slices += static_cast<int>((bytes + kSliceBytes - 1) / kSliceBytes);
      c.t[i].slice_end = slices;
    }
    c.slices = slices;
    c.count = n;
    // (128 samples of two prompts of 1001 and 4000 tokens, and about 300 of 1200 pages
    // moved, us, with 8 / 16 / 32 CTAs an SM: 83 / 77 / 75 and 114 / 110 / 106; slices of
    // 16 KB 105 and 108; eight loads in flight a thread 89 and 107.)
    const long long items = most * slices, room = 32LL * sms;
    const cudaError_t e = launch_overlapped(copy_pages_kernel, dim3(static_cast<unsigned>(items < room ? items : room)),
                                            kCopyThreads, 0, stream, c);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t fork_workspace_words(int B, int rows) {
  return kPlanHead + 2LL * rows + B + static_cast<size_t>(rows) * sizeof(PageCopy) / 4;
}

size_t compact_workspace_words(int num_pages) {
  const size_t moves = static_cast<size_t>(num_pages) / 2;
  return kPlanHead + 2 * moves + moves * sizeof(PageCopy) / 4;
}

cudaError_t launch_fork(const ForkArgs& a, const PageTensor* tensors, int count, int sms, cudaStream_t stream) {
  fork_kernel<<<kPlanCtas, kPlanThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  CopyArgs c;
  c.workspace = a.workspace;
  c.list_a = c.list_b = a.rows;
  c.first = a.B;
  c.page_size = a.table.page_size;
  return launch_copies(c, tensors, count, a.rows, sms, stream);
}

cudaError_t launch_compact(const CompactArgs& a, const PageTensor* tensors, int count, int sms, cudaStream_t stream) {
  compact_kernel<<<kPlanCtas, kPlanThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  CopyArgs c;
  c.workspace = a.workspace;
  c.list_a = c.list_b = a.table.num_pages / 2;
  c.first = 0;
  c.page_size = a.table.page_size;
  if (a.table.num_pages < 2) return cudaSuccess;  // no page can move
  return launch_copies(c, tensors, count, a.table.num_pages / 2, sms, stream);
}

}  // namespace fa
