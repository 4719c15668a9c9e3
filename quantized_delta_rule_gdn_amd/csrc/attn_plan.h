// attn_plan.h -- how the attention kernels over the paged cache share out their work: a request's
// tokens are cut into items by the lengths that lie on the device.
#pragma once

#include "prompt_common.h"

namespace damp {
namespace {

constexpr int kAttnTile = 32;

// The work is shared out on the device, by the requests' actual lengths: with `per_unit` workgroups
// for each (key-value head, 16 query heads), an item is a run of at most
// chunk = max(256, total tokens / per_unit) tokens of one request, so there are at most per_unit + B
// items whatever the lengths, they are of much the same length, and those of full length fill the
// chip once. (Cut by the longest length the host knows of instead, 64 requests of 128 to 8,192
// tokens took 244-260 us against 186-197 us of as many bytes in even lengths.)
struct AttnPlan {
  int tiles;      // groups of 16 query heads per key-value head
  int heads;      // query heads of a full group
  int per_unit;
  int items;      // per_unit + B, or B where no request is cut
};

constexpr int kAttnLeast = 8 * kAttnTile;    // tokens: no chunk is shorter

// Tokens of request b that are read.
__device__ __forceinline__ int length_of(const AttnArgs& a, int b) {
  const int64_t cap = int64_t(a.max_blocks) << a.page_log2;
  return static_cast<int>(min(int64_t(min(max(a.seq_lens[b], 0), a.max_len)), cap));
}

__device__ __forceinline__ int items_of(int len, int chunk) { return max((len + chunk - 1) / chunk, 1); }

// What a workgroup adds up over the requests: up to 64 of them each wave takes for itself, one per lane;
// more are taken by all 256 threads, and the waves meet in LDS. (One request of 700 tokens 10.6 us
// against 11.3 with the waves meeting; 1,000 of 100 to 1,500 tokens 133 against 153 us without.)
__device__ __forceinline__ int requests_step(const AttnArgs& a) { return a.B <= 64 ? 64 : 256; }

__device__ __forceinline__ int64_t requests_sum(const AttnArgs& a, int64_t x, int64_t* sh) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o);
  if (a.B <= 64) return x;
  __syncthreads();
  if ((__builtin_amdgcn_workitem_id_x() & 63) == 0) sh[__builtin_amdgcn_workitem_id_x() >> 6] = x;
  __syncthreads();
  return (sh[0] + sh[1]) + (sh[2] + sh[3]);
}

__device__ __forceinline__ int chunk_of(const AttnArgs& a, const AttnPlan& plan, int64_t* sh) {
  const int step = requests_step(a);
  int64_t total = 0;
  for (int b = __builtin_amdgcn_workitem_id_x() & (step - 1); b < a.B; b += step) total += length_of(a, b);
  total = requests_sum(a, total, sh);
  const int64_t chunk = (total + plan.per_unit - 1) / plan.per_unit;
  // (no request is longer than 2^30: a longer chunk would be the same)
  return static_cast<int>(min(max((chunk + kAttnLeast - 1) / kAttnLeast * kAttnLeast, int64_t(kAttnLeast)), int64_t(1) << 30));
}

struct Item {   // part `split` of `splits` of request b; b < 0: none
  int b, split, splits;
};

__device__ __forceinline__ Item item_of(const AttnArgs& a, const AttnPlan& plan, int item, int64_t* sh) {
  if (plan.items == a.B) return Item{item, 0, 1};   // none is cut (4,000 requests of 60 tokens: 30 us, 95 with the search)
  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63, wv = tid >> 6;
  const int chunk = chunk_of(a, plan, sh), step = requests_step(a);
  int* wave_items = reinterpret_cast<int*>(sh + 4);
  int* found = wave_items + 4;
  if (step > 64 && tid == 0) found[0] = -1;
  for (int b0 = 0, before = 0; b0 < a.B && before <= item; b0 += step) {
    const int b = b0 + (tid & (step - 1));
    const int n = b < a.B ? items_of(length_of(a, b), chunk) : 0;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int y = __shfl_up(incl, o);
      if (lane >= o) incl += y;
    }
    int first = before + incl - n;
    if (step > 64) {
      if (lane == 63) wave_items[wv] = incl;
      __syncthreads();
      for (int i = 0; i < wv; ++i) first += wave_items[i];
      if (item >= first && item < first + n) {
        found[0] = b;
        found[1] = item - first;
        found[2] = n;
      }
      before += (wave_items[0] + wave_items[1]) + (wave_items[2] + wave_items[3]);
      __syncthreads();
    } else if (const uint64_t mine = __ballot(item >= first && item < first + n); mine != 0) {
      const int l = __builtin_ctzll(mine);
      return Item{l, item - __builtin_amdgcn_readlane(first, l), __builtin_amdgcn_readlane(n, l)};
    }
  }
  if (step == 64) return Item{-1, 0, 1};
  return Item{__builtin_amdgcn_readfirstlane(found[0]), __builtin_amdgcn_readfirstlane(found[1]), __builtin_amdgcn_readfirstlane(found[2])};
}

}  // namespace
}  // namespace damp
