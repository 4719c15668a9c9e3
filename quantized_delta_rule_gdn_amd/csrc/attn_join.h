// attn_join.h -- the second launch of the attention kernels of several tokens: requests that were cut
// into items are joined.
#pragma once

#include <algorithm>

#include "attn_mask.h"
#include "attn_plan.h"

namespace damp {
namespace {

// The items of a (request, row) joined: sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s, four channels a
// thread, 1,024 / D rows a workgroup. Bound by the stream of the items.
template <int D, int GRAIN>
__global__ __launch_bounds__(256) void attn_join_kernel(const TreeArgs a, const AttnPlan plan, int groups) {
  constexpr int LPR = D / 4, RPG = 256 / LPR;      // threads a row, rows a workgroup
  __shared__ int64_t sh[8];
  const int tid = __builtin_amdgcn_workitem_id_x();
  const int64_t id = __builtin_amdgcn_workgroup_id_x();
  const int units = a.Hkv * plan.tiles;
  const int group = static_cast<int>(id % groups), unit = static_cast<int>(id / groups % units), b = static_cast<int>(id / groups / units);
  const int tile = unit % plan.tiles, kvh = unit / plan.tiles, G = a.Hq / a.Hkv;
  const Drafts dr = drafts_of(a, b);
  const int64_t rows = int64_t(min(dr.n, a.max_new)) * G, tile0 = int64_t(tile) * plan.rows;
  if (tile0 + group * RPG >= rows) return;
  const int chunk = chunk_of<GRAIN>(a, plan, sh), n = items_of(length_of(a, b), chunk);
  if (n == 1) return;                              // it has its readout already
  int64_t before = 0;
  const int apart = requests_step(a);
  for (int x = tid & (apart - 1); x < b; x += apart) before += items_of(length_of(a, x), chunk);
  before = requests_sum(a, before, sh);
  const int in_tile = group * RPG + tid / LPR;
  const int64_t row = tile0 + in_tile;
  if (in_tile >= plan.heads || row >= rows) return;
  const int64_t step = int64_t(units) * plan.heads;      // between a unit's items
  const int64_t first = (before * units + unit) * plan.heads + in_tile;
  const float4* po = reinterpret_cast<const float4*>(a.ws + first * D) + tid % LPR;
  const float2* ml = reinterpret_cast<const float2*>(a.ws + int64_t(plan.items) * step * D) + first;
  float m = -INFINITY;
  for (int s = 0; s < n; ++s) m = fmaxf(m, ml[s * step].x);
  const float base = m == -INFINITY ? 0.0f : m;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float l = 0.0f;
#pragma unroll 4
  for (int s = 0; s < n; ++s) {
    const float2 x = ml[s * step];
    const float4 v = po[s * step * LPR];
    const float f = pow2(x.x - base);
    l = fmaf(f, x.y, l);
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
  }
  const float back = l == 0.0f ? 0.0f : 1.0f / l;
  const int64_t at = (int64_t(dr.first + static_cast<int>(row / G)) * a.Hq + kvh * G + row % G) * LPR + tid % LPR;
  reinterpret_cast<uint2*>(a.out)[at] = make_uint2(pack_bf16(acc.x * back, acc.y * back), pack_bf16(acc.z * back, acc.w * back));
}

// Workgroups that a (request, row tile) takes.
inline int64_t join_groups(const AttnPlan& p, int d) { return (p.heads + 1024 / d - 1) / (1024 / d); }

template <int D, int GRAIN>
void launch_join(const TreeArgs& a, const AttnPlan& p, hipStream_t s) {
  const int64_t groups = join_groups(p, D);
  hipLaunchKernelGGL((attn_join_kernel<D, GRAIN>), dim3(static_cast<unsigned>(int64_t(a.B) * a.Hkv * p.tiles * groups)), dim3(256), 0, s, a, p,
                     static_cast<int>(groups));
}

}  // namespace
}  // namespace damp
