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
// loads of a parent's length (18 forks 4.0 us, 576 forks 5.2); the outputs are 4 bytes a page and 12 a fork.
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
// thread and load, eight of them on their way at once. Bound by the stream: 275 MB read and written in
// 47 us, 5.8 TB/s.
constexpr int kCopyRun = 65536, kCopyUnroll = 8;
using u32x4 = __attribute__((ext_vector_type(4))) uint32_t;

__global__ __launch_bounds__(256) void kv_copy_kernel(const CopyArgs a, unsigned runs, unsigned arrays, unsigned groups) {
  const int tid = __builtin_amdgcn_workitem_id_x();
  const unsigned items = a.n * static_cast<unsigned>(a.Hkv) * arrays * runs;
  for (unsigned x = __builtin_amdgcn_workgroup_id_x(); x < items; x += groups) {
    const unsigned run = x % runs, y = x / runs, which = y % arrays, z = y / arrays, h = z % a.Hkv, i = z / a.Hkv;
    const int src = a.src[i], dst = a.dst[i];
    if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages || src == dst) continue;
    const int page = 1 << a.page_log2, rows = a.rows ? min(max(a.rows[i], 0), page) : page;
    const int per_row = a.d / 8, first = run * (kCopyRun / 16), stop = min(first + kCopyRun / 16, rows * per_row);
    u32x4* base = reinterpret_cast<u32x4*>(which ? a.v_pages : a.k_pages);
    const int64_t whole = int64_t(page) * per_row;
    const u32x4* from = base + (int64_t(src) * a.Hkv + h) * whole;
    u32x4* to = base + (int64_t(dst) * a.Hkv + h) * whole;
    for (int p = first + tid; p < stop; p += 256 * kCopyUnroll) {
      u32x4 w[kCopyUnroll];
#pragma unroll
      for (int k = 0; k < kCopyUnroll; ++k) w[k] = __builtin_nontemporal_load(from + min(p + 256 * k, stop - 1));
#pragma unroll
      for (int k = 0; k < kCopyUnroll; ++k)
        if (p + 256 * k < stop) __builtin_nontemporal_store(w[k], to + p + 256 * k);
    }
  }
}

// ---- kept tokens moved together ------------------------------------------------------------------
// One workgroup per (request, head, keys or values) takes the kept tokens in order, as many at a time
// as its threads hold in registers. A token never moves up (its place in the list is at most its
// number), so a batch's stores cannot reach a later batch's tokens: the next batch is loaded before
// this one is stored, its pages looked up a batch ahead, and the list read one more ahead. Within a
// batch every load has returned before the first store. Long lists are bound by
// the stream of rows of 256 bytes from here and there, and by the longest of them: a workgroup's batches follow each other,
// and all 512 workgroups of 32 requests of up to 8,192 tokens halved (the longest has 32 batches, the mean is 16.5)
// start at once, so that in the end few are at work. That takes 134 us for 553 MB, as many bytes in 32 even lists 118, 4.7
// TB/s. Splitting rows over workgroups did not help; stores past the caches take 135 and 119, and where the same arrays are
// moved again and again 125 instead of 118. Short lists are bound by latency (6 us). Latents have one
// head and no values, so a request is one workgroup's: 32 of up to 16,384 tokens halved take 780 us, 0.4 TB/s.
constexpr int kKeepUnroll = 8;

__global__ __launch_bounds__(256) void kv_compact_kernel(const CompactArgs a, int arrays) {
  constexpr int U = kKeepUnroll;
  const int tid = __builtin_amdgcn_workitem_id_x();
  const unsigned x = __builtin_amdgcn_workgroup_id_x();
  const int which = static_cast<int>(x % arrays), h = static_cast<int>(x / arrays % a.Hkv), b = static_cast<int>(x / arrays / a.Hkv);
  const int lo = min(max(a.cu[b], 0), a.K), hi = min(max(a.cu[b + 1], lo), a.K);
  const int len = max(a.seq_lens[b], 0), fresh = min(max(a.new_lens[b], 0), len), base = len - fresh;
  const int n = min(hi - lo, fresh);
  if (which == 0 && h == 0 && tid == 0) a.out_lens[b] = base + n;
  if (n == 0 || a.max_blocks == 0) return;
  const int per_row = a.d / 8, in_page = (1 << a.page_log2) - 1;             // (at most 256 pieces a row)
  const int rows = 256 / per_row, row = tid / per_row, piece = tid % per_row;   // rows a pass
  u32x4* pages = reinterpret_cast<u32x4*>(which ? a.v_pages : a.k_pages);
  const int* table = a.table + int64_t(b) * a.max_blocks;
  struct Batch {                // a batch on its way: places in the list, then their pages, then their values
    int idx[U], po[U], pt[U];
  };
  // (every load is unconditional and waits are for older ones than a batch's values: the loads come back in
  // order, and the values are the last of an iteration)
  const auto list = [&](int j0, Batch& m) {
#pragma unroll
    for (int u = 0; u < U; ++u) m.idx[u] = a.kept[lo + min(j0 + u * rows + row, n - 1)];
  };
  const auto look_up = [&](int j0, Batch& m) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = min(j0 + u * rows + row, n - 1);
      m.po[u] = table[min((base + min(max(m.idx[u], 0), fresh - 1)) >> a.page_log2, a.max_blocks - 1)];
      m.pt[u] = table[min((base + j) >> a.page_log2, a.max_blocks - 1)];
    }
  };
  const auto moves = [&](int j0, const Batch& m, int u) -> bool {
    const int j = j0 + u * rows + row;
    return row < rows && j < n && m.idx[u] > j && m.idx[u] < fresh && (base + m.idx[u]) >> a.page_log2 < a.max_blocks && m.po[u] >= 0 &&
           m.po[u] < a.num_pages && m.pt[u] >= 0 && m.pt[u] < a.num_pages;
  };
  const auto load = [&](int j0, const Batch& m, u32x4 (&w)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t from = moves(j0, m, u) ? ((static_cast<uint32_t>(m.po[u]) * a.Hkv + h) << a.page_log2) + ((base + m.idx[u]) & in_page) : 0;
      w[u] = pages[int64_t(from) * per_row + piece];
    }
  };
  const int batch = rows * U;
  Batch now, next, after;
  u32x4 w[U];
  list(0, now);
  list(batch, next);
  list(2 * batch, after);
  look_up(0, now);
  look_up(batch, next);
  load(0, now, w);
  for (int j0 = 0; j0 < n; j0 += batch) {
    u32x4 ahead[U];
    Batch last;
    look_up(j0 + 2 * batch, after);
    list(j0 + 3 * batch, last);
    load(j0 + batch, next, ahead);
#pragma unroll
    for (int u = 0; u < U; ++u) asm volatile("" ::"v"(w[u]) : "memory");   // (has returned)
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (moves(j0, now, u)) {
        const uint32_t to = ((static_cast<uint32_t>(now.pt[u]) * a.Hkv + h) << a.page_log2) + ((base + j0 + u * rows + row) & in_page);
        pages[int64_t(to) * per_row + piece] = w[u];
      }
      w[u] = ahead[u];
    }
    now = next;
    next = after;
#pragma unroll
    for (int u = 0; u < U; ++u) after.idx[u] = last.idx[u];
  }
}

// ---- pages given back ------------------------------------------------------------------------------
// Two steps: every page behind a request's kept tokens loses one share, the one that had none left
// is marked; then the marked pages are listed by ascending id and the marks taken off. A mark is -1
// in shares, so a page that two requests give back in one call is listed once, whoever comes first.
// Bound by the launches (2 to 5 us each).
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
__global__ __launch_bounds__(kListThreads) void kv_list_kernel(const FreeArgs a, int per_group, int groups) {
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
  if (g == groups - 1 && tid == 0) a.num_freed[0] = before;
}

// Up to this many pages one workgroup lists alone, without the launch that counts (8,192 pages 9.5 us and
// 10.0 with it, 32,768 19.9 and 9.6, launches in a graph).
constexpr int32_t kListAlone = 2 * kListPages;

int64_t list_groups(int32_t num_pages) { return num_pages <= kListAlone ? 1 : (int64_t(num_pages) + kListPages - 1) / kListPages; }

}  // namespace

hipError_t launch_kv_fork(const ForkArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(kv_fork_kernel, dim3(std::max(a.n, 1)), dim3(kForkThreads), 0, s, a);
  return hipGetLastError();
}

int64_t kv_copy_items(const CopyArgs& a) {
  const int64_t bytes = (int64_t(a.d) * 2) << a.page_log2;
  return int64_t(a.n) * a.Hkv * (a.v_pages ? 2 : 1) * ((bytes + kCopyRun - 1) / kCopyRun);
}

hipError_t launch_kv_copy(const CopyArgs& a, hipStream_t s) {
  const int64_t items = kv_copy_items(a);
  const unsigned arrays = a.v_pages ? 2 : 1, runs = static_cast<unsigned>(items / (int64_t(a.n) * a.Hkv * arrays));
  const unsigned groups = static_cast<unsigned>(std::min<int64_t>(items, 65536));
  hipLaunchKernelGGL(kv_copy_kernel, dim3(groups), dim3(256), 0, s, a, runs, arrays, groups);
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
  hipLaunchKernelGGL(kv_list_kernel, dim3(groups), dim3(kListThreads), 0, s, a, per_group, static_cast<int>(groups));
  return hipGetLastError();
}

}  // namespace damp
