// page_kernels.hip -- gfx950 kernels of the life of a cache's pages: requests forked from others
// (full pages shared, the partly filled one copied), tokens kept and moved together, pages given
// back. shares[p] counts the requests that hold page p beyond the first.
#include <algorithm>

#include "prompt_common.h"

namespace damp {
namespace {

// ---- forked tables -----------------------------------------------------------------------------
// One workgroup a fork: it counts the forks before it that need a page (their index into the free
// list), copies the parent's table row and adds one to the shares of its full pages (integer
// atomics: the sums do not depend on their order). Bound by the launch and by the two dependent
// loads of a parent's length; the outputs are 4 bytes a page and 12 a fork.
constexpr int kForkThreads = 256;

struct Fork {
  int src, dst, full, part;   // src < 0: skipped; full pages, tokens in the page behind them
};

__device__ __forceinline__ Fork fork_of(const ForkArgs& a, int i) {
  const int src = a.src[i], dst = a.dst[i];
  if (src < 0 || src >= a.B || dst < 0 || dst >= a.B) return Fork{-1, -1, 0, 0};
  const int len = max(a.seq_lens[src], 0), full = len >> a.page_log2;
  if (full >= a.max_blocks) return Fork{src, dst, a.max_blocks, 0};
  return Fork{src, dst, full, len & ((1 << a.page_log2) - 1)};
}

__global__ __launch_bounds__(kForkThreads) void kv_fork_kernel(const ForkArgs a) {
  __shared__ int wave_sum[kForkThreads / 64];
  const int tid = __builtin_amdgcn_workitem_id_x(), i = __builtin_amdgcn_workgroup_id_x();
  int n = 0;
  for (int j = tid; j < min(i, a.n); j += kForkThreads) n += fork_of(a, j).part > 0;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o);
  if ((tid & 63) == 0) wave_sum[tid >> 6] = n;
  __syncthreads();
  const int before = (wave_sum[0] + wave_sum[1]) + (wave_sum[2] + wave_sum[3]);
  if (i >= a.n) {            // (a call without forks)
    if (tid == 0) a.used[0] = before;
    return;
  }
  const Fork f = fork_of(a, i);
  const int fresh = f.part > 0 && before < a.num_free ? a.free_pages[before] : -1;
  if (tid == 0) {
    if (i == a.n - 1) a.used[0] = before + (f.part > 0);
    int last = -1;
    if (f.part > 0) {
      last = a.table[int64_t(f.src) * a.max_blocks + f.full];
      a.table[int64_t(f.dst) * a.max_blocks + f.full] = fresh;
    }
    if (f.src >= 0) a.seq_lens[f.dst] = a.seq_lens[f.src];
    const bool copies = f.part > 0 && last >= 0 && last < a.num_pages && fresh >= 0 && fresh < a.num_pages;
    a.copy_src[i] = copies ? last : -1;
    a.copy_dst[i] = copies ? fresh : -1;
    a.copy_rows[i] = copies ? f.part : 0;
  }
  for (int j = tid; j < f.full; j += kForkThreads) {
    const int id = a.table[int64_t(f.src) * a.max_blocks + j];
    a.table[int64_t(f.dst) * a.max_blocks + j] = id;
    if (id >= 0 && id < a.num_pages) atomicAdd(a.shares + id, 1);
  }
}

// ---- copies of pages ---------------------------------------------------------------------------
// A workgroup takes one run of up to kCopyRun bytes of one (copy, head, keys or values), 16 bytes a
// thread and load, four of them on their way at once. Bound by the stream.
constexpr int kCopyRun = 16384;

__global__ __launch_bounds__(256) void kv_copy_kernel(const CopyArgs a, int runs, int arrays) {
  const int tid = __builtin_amdgcn_workitem_id_x();
  const int64_t items = int64_t(a.n) * a.Hkv * arrays * runs;
  for (int64_t x = __builtin_amdgcn_workgroup_id_x(); x < items; x += __builtin_amdgcn_grid_size_x() / 256) {
    const int run = static_cast<int>(x % runs);
    const int64_t y = x / runs;
    const int which = static_cast<int>(y % arrays), h = static_cast<int>(y / arrays % a.Hkv), i = static_cast<int>(y / arrays / a.Hkv);
    const int src = a.src[i], dst = a.dst[i];
    if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages || src == dst) continue;
    const int page = 1 << a.page_log2, rows = a.rows ? min(max(a.rows[i], 0), page) : page;
    const int64_t pieces = int64_t(rows) * (a.d / 8);
    const int64_t first = int64_t(run) * (kCopyRun / 16), stop = min(first + kCopyRun / 16, pieces);
    uint4* base = reinterpret_cast<uint4*>(which ? a.v_pages : a.k_pages);
    const int64_t whole = int64_t(page) * (a.d / 8);
    const uint4* from = base + (int64_t(src) * a.Hkv + h) * whole;
    uint4* to = base + (int64_t(dst) * a.Hkv + h) * whole;
    int64_t p = first + tid;
    for (; p + 768 < stop; p += 1024) {
      uint4 w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = from[p + 256 * k];
#pragma unroll
      for (int k = 0; k < 4; ++k) to[p + 256 * k] = w[k];
    }
    for (; p < stop; p += 256) to[p] = from[p];
  }
}

// ---- kept tokens moved together ------------------------------------------------------------------
// One workgroup per (request, head, keys or values) takes the kept tokens in order, as many at a time
// as its threads hold in registers. A token never moves up (its place in the list is at most its
// number), so a batch's stores cannot reach a later batch's tokens; within a batch every load has
// returned before the first store. Bound by the stream for long lists, by latency for short ones.
constexpr int kKeepUnroll = 4;

__global__ __launch_bounds__(256) void kv_compact_kernel(const CompactArgs a, int arrays) {
  const int tid = __builtin_amdgcn_workitem_id_x();
  const int64_t x = __builtin_amdgcn_workgroup_id_x();
  const int which = static_cast<int>(x % arrays), h = static_cast<int>(x / arrays % a.Hkv), b = static_cast<int>(x / arrays / a.Hkv);
  const int lo = min(max(a.cu[b], 0), a.K), hi = min(max(a.cu[b + 1], lo), a.K);
  const int len = max(a.seq_lens[b], 0), fresh = min(max(a.new_lens[b], 0), len), base = len - fresh;
  const int n = min(hi - lo, fresh);
  if (which == 0 && h == 0 && tid == 0) a.out_lens[b] = base + n;
  const int per_row = a.d / 8, page = 1 << a.page_log2;             // (at most 256 pieces a row)
  const int rows = 256 / per_row, row = tid / per_row, piece = tid % per_row;   // rows a pass
  uint4* pages = reinterpret_cast<uint4*>(which ? a.v_pages : a.k_pages);
  const auto at = [&](int pos) -> int64_t {   // of a position's row, in pieces; -1 where there is none
    const int j = pos >> a.page_log2;
    if (j >= a.max_blocks) return -1;
    const int id = a.table[int64_t(b) * a.max_blocks + j];
    if (id < 0 || id >= a.num_pages) return -1;
    return ((((int64_t(id) * a.Hkv + h) << a.page_log2) + (pos & (page - 1))) * per_row);
  };
  for (int j0 = 0; j0 < n; j0 += rows * kKeepUnroll) {
    int64_t from[kKeepUnroll], to[kKeepUnroll];
#pragma unroll
    for (int u = 0; u < kKeepUnroll; ++u) {
      const int j = j0 + u * rows + row;
      from[u] = to[u] = -1;
      if (row < rows && j < n) {
        const int idx = a.kept[lo + j];
        if (idx > j && idx < fresh) {
          from[u] = at(base + idx);
          to[u] = from[u] < 0 ? -1 : at(base + j);
        }
      }
    }
    uint4 w[kKeepUnroll] = {};
#pragma unroll
    for (int u = 0; u < kKeepUnroll; ++u)
      if (to[u] >= 0) w[u] = pages[from[u] + piece];
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kKeepUnroll; ++u)
      if (to[u] >= 0) pages[to[u] + piece] = w[u];
  }
}

// ---- pages given back ------------------------------------------------------------------------------
// Two steps: every page behind a request's kept tokens loses one share, the one that had none left
// is marked; then the marked pages are listed by ascending id and the marks taken off. A mark is -1
// in shares, so a page that two requests give back in one call is listed once, whoever comes first.
constexpr int kMark = -1;

__global__ __launch_bounds__(256) void kv_drop_kernel(const FreeArgs a) {
  const int b = __builtin_amdgcn_workgroup_id_x();
  const auto pages = [&](int n) { return min((n >> a.page_log2) + ((n & ((1 << a.page_log2) - 1)) != 0), a.max_blocks); };
  const int stop = pages(max(a.seq_lens[b], 0)), first = a.keep_lens ? pages(max(a.keep_lens[b], 0)) : 0;
  for (int j = first + static_cast<int>(__builtin_amdgcn_workitem_id_x()); j < stop; j += 256) {
    const int id = a.table[int64_t(b) * a.max_blocks + j];
    if (id < 0 || id >= a.num_pages) continue;
    int have = a.shares[id];
    while (have >= 0) {                       // (each failed exchange means that another one took a share)
      const int seen = atomicCAS(a.shares + id, have, have > 0 ? have - 1 : kMark);
      if (seen == have) break;
      have = seen;
    }
  }
}

constexpr int kListThreads = 1024;
constexpr int kListPages = 4 * kListThreads;      // pages a workgroup lists at a time

// Marks among pages [p, p + 4) as bits.
__device__ __forceinline__ int marks_of(const FreeArgs& a, int64_t p) {
  int bits = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (p + k < a.num_pages && a.shares[p + k] == kMark) bits |= 1 << k;
  return bits;
}

__global__ __launch_bounds__(kListThreads) void kv_count_kernel(const FreeArgs a) {
  __shared__ int wave_sum[kListThreads / 64];
  const int tid = __builtin_amdgcn_workitem_id_x();
  const int64_t p = int64_t(__builtin_amdgcn_workgroup_id_x()) * kListPages + 4 * tid;
  int n = __builtin_popcount(marks_of(a, p));
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o);
  if ((tid & 63) == 0) wave_sum[tid >> 6] = n;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kListThreads / 64; ++i) n += wave_sum[i];
    a.ws[__builtin_amdgcn_workgroup_id_x()] = n;
  }
}

// per_group: runs of kListPages that each workgroup lists (all of them where there is one workgroup).
__global__ __launch_bounds__(kListThreads) void kv_list_kernel(const FreeArgs a, int per_group) {
  __shared__ int wave_sum[kListThreads / 64];
  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63, wv = tid >> 6;
  const int g = __builtin_amdgcn_workgroup_id_x();
  int before = 0;
  if (g > 0) {
    for (int i = tid; i < g; i += kListThreads) before += a.ws[i];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) before += __shfl_xor(before, o);
    if (lane == 0) wave_sum[wv] = before;
    __syncthreads();
    before = 0;
#pragma unroll
    for (int i = 0; i < kListThreads / 64; ++i) before += wave_sum[i];
    __syncthreads();
  }
  for (int run = 0; run < per_group; ++run) {
    const int64_t p = (int64_t(g) * per_group + run) * kListPages + 4 * tid;
    const int bits = marks_of(a, p), n = __builtin_popcount(bits);
    int incl = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int y = __shfl_up(incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 63) wave_sum[wv] = incl;
    __syncthreads();
    int to = before + incl - n;
#pragma unroll
    for (int i = 0; i < kListThreads / 64; ++i) {
      if (i < wv) to += wave_sum[i];
      before += wave_sum[i];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (bits >> k & 1) {
        a.freed[to++] = static_cast<int>(p + k);
        a.shares[p + k] = 0;
      }
  }
  if (g == static_cast<int>(__builtin_amdgcn_grid_size_x() / kListThreads) - 1 && tid == 0) a.num_freed[0] = before;
}

// Up to this many pages one workgroup lists alone, without the launch that counts.
constexpr int32_t kListAlone = 16 * kListPages;

int64_t list_groups(int32_t num_pages) { return num_pages <= kListAlone ? 1 : (int64_t(num_pages) + kListPages - 1) / kListPages; }

}  // namespace

hipError_t launch_kv_fork(const ForkArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(kv_fork_kernel, dim3(std::max(a.n, 1)), dim3(kForkThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_kv_copy(const CopyArgs& a, hipStream_t s) {
  const int64_t bytes = (int64_t(a.d) * 2) << a.page_log2;
  const int runs = static_cast<int>((bytes + kCopyRun - 1) / kCopyRun), arrays = a.v_pages ? 2 : 1;
  const int64_t items = int64_t(a.n) * a.Hkv * arrays * runs;
  hipLaunchKernelGGL(kv_copy_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(items, 65536))), dim3(256), 0, s, a, runs, arrays);
  return hipGetLastError();
}

hipError_t launch_kv_compact(const CompactArgs& a, hipStream_t s) {
  const int arrays = a.v_pages ? 2 : 1;
  hipLaunchKernelGGL(kv_compact_kernel, dim3(static_cast<unsigned>(a.B) * a.Hkv * arrays), dim3(256), 0, s, a, arrays);
  return hipGetLastError();
}

size_t kv_free_ws_bytes(int32_t num_pages) {
  const int64_t groups = list_groups(num_pages);
  return groups > 1 ? static_cast<size_t>(groups) * 4 : 0;
}

hipError_t launch_kv_free(const FreeArgs& a, hipStream_t s) {
  const unsigned groups = static_cast<unsigned>(list_groups(a.num_pages));
  if (a.B > 0) hipLaunchKernelGGL(kv_drop_kernel, dim3(a.B), dim3(256), 0, s, a);
  if (groups > 1) hipLaunchKernelGGL(kv_count_kernel, dim3(groups), dim3(kListThreads), 0, s, a);
  const int per_group = groups > 1 ? 1 : static_cast<int>((a.num_pages + kListPages - 1) / kListPages);
  hipLaunchKernelGGL(kv_list_kernel, dim3(groups), dim3(kListThreads), 0, s, a, per_group);
  return hipGetLastError();
}

}  // namespace damp
