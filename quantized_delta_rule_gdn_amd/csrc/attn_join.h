// attn_join.h -- how the attention kernels of several tokens share out their work, and their second
// launch, which joins the parts of requests that were cut.
#pragma once

#include <algorithm>

#include "attn_mask.h"
#include "attn_plan.h"

namespace damp {
namespace {

// ---- how the work is shared out --------------------------------------------------------------------
// A request's query rows (its new tokens' heads of one key-value head) are taken in tiles of `rows`, and
// its cached tokens in runs; a workgroup takes one (run, key-value head, tile). The runs are cut on the
// device, where the lengths are. Where the (request, head, row tile) units are few, by the least chunk with
// which the workgroups are no more than the chip holds at once: one round of runs of at most that length. (A request is cut
// into a whole number of runs, so they are not alike: 48 requests of 85 to 4,096 tokens, 384 units on 512, get runs of up to 43 tiles
// of 64 tokens where the mean is 25, 24 of latents, 138 units on 256, of up to 48 of 32 where it is 35.) Where
// they are many, only what is longer than a workgroup's fair share, as others fill the chip meanwhile. (Cutting
// costs the parts, a write and a read of 4 bytes a row and channel: 48 requests of 2,000 tokens with 128 rows,
// 384 units, take 118 us in two rounds of runs and 90 whole. 256 requests of 1,500 tokens of which one has 100,000,
// 2,048 units, take 1,450 us with none cut, 356 so.)
struct TokenPlan {
  int rows_log2;  // query rows of a tile
  int heads;      // rows of the largest tile there is
  int tiles;      // row tiles of a request with the most new tokens
  int slots;      // workgroups that the chip holds at once
  int groups;     // of the launch: whole rounds of the dies, at least what runs_of gives
  int whole;      // no request is cut
};

// Runs that units are cut into, at most. Few are up to three quarters of the workgroups that the chip holds: so much room
// is left to cut the longest. 32 drafted tokens, 8 heads of d = 128, 512 workgroups at once, as few and as many (us): requests of 1/B
// to all of 4,000 tokens, 272 units 75 and 98, 320 96 and 117, 384 117 and 131, 448 128 and 139, 480 138 and 147; one of 60,000 tokens
// among others of 1,200, 272 units 84 and 102, 320 92 and 101, 352 97 and 99, 384 170 and 100, 448 239 and 110, 512 1,260 and 121.
// Latents of 128 heads, 256 at once: 224 units of even steps 119 and 129; one long one among 160 99 and 112, 176 108 and 110, 192 211
// and 114.
__host__ __device__ inline bool few_units(int64_t units, int slots) { return 4 * units <= 3 * int64_t(slots); }
__host__ __device__ inline int64_t runs_of(int64_t units, int slots) { return few_units(units, slots) ? slots : units + slots / 2; }

// Neighbouring parts that a die takes at a time.
__host__ __device__ inline int dealt(int tiles) { return tiles < 16 ? tiles : 16; }

// One workgroup's part. b < 0: none.
struct Spot {
  int b, kvh, tile;
  int split, splits;     // its part of the request's tokens
  int at;                // its place in the list of parts; of one that is cut, in the workspace too
  Drafts dr;
  int len;               // tokens of the request
};

struct Share {           // of a request
  Drafts dr;
  int len, tiles;        // tokens, row tiles
};

__device__ __forceinline__ Share share_of(const TreeArgs& a, const TokenPlan& plan, int b) {
  Share s;
  s.dr = drafts_of(a, b);
  s.len = length_of(a, b);
  s.tiles = (min(s.dr.n, a.max_new) * (a.Hq / a.Hkv) + (1 << plan.rows_log2) - 1) >> plan.rows_log2;      // (rows stay below 2^30)
  return s;
}

// What the workgroups leave in the workspace: a tile's partial readouts, {maximum, sum} of its rows, and
// each request's {first place, runs}. Only parts of requests that are cut are written, and they lie in the first
// `slots` places however many units there are: a list of no more parts than that needs no more, and in a longer
// one requests that are cut come first. That list has units + slots / 2 parts at most, so units that are cut into
// r >= 2 runs each add r - 1 >= r / 2 parts to it, slots / 2 in all, and have slots at most.
template <int D>
struct Parts {
  float* o;
  float2* ml;
  int2* info;
  __device__ Parts(const TreeArgs& a, const TokenPlan& plan) {
    const int64_t n = int64_t(plan.slots) * plan.heads;
    o = a.ws;
    ml = reinterpret_cast<float2*>(a.ws + n * D);
    info = reinterpret_cast<int2*>(ml + n);
  }
};

inline size_t parts_bytes(const TokenPlan& p, const TreeSizes& z, int32_t d) {
  return p.whole ? 0 : static_cast<size_t>(p.slots) * p.heads * (static_cast<size_t>(d) + 2) * 4 + static_cast<size_t>(z.B) * 8;
}

// Every wave finds its workgroup's part for itself, its lanes taking a request each. Workgroups go round the 8
// dies, which have an L2 each: a die takes as many neighbouring parts of the list (request, run, head, tile) at
// a time as there may be row tiles (up to 16), so that those that read the same keys meet in one L2. Where the list is
// longer than a round, requests that are cut come first: the last ones to start are then short.
template <int GRAIN, int D>
__device__ __forceinline__ Spot spot_of(const TreeArgs& a, const TokenPlan& plan) {
  const unsigned id = __builtin_amdgcn_workgroup_id_x();
  if (plan.whole) {
    const int per = plan.tiles * a.Hkv;
    const int at = per == 1 ? static_cast<int>(id) : static_cast<int>(id % 8 * (plan.groups / 8) + id / 8);   // (rounded up to 8)
    const int b = at / per, unit = at % per;
    if (b >= a.B) return Spot{-1};
    return Spot{b, unit / plan.tiles, unit % plan.tiles, 0, 1, 0, drafts_of(a, b), length_of(a, b)};
  }
  const int lane = __builtin_amdgcn_workitem_id_x() & 63;
  const auto share = [&](int b) -> Share {           // none behind the last request
    Share s = share_of(a, plan, min(b, a.B - 1));
    if (b >= a.B) s.tiles = 0;
    return s;
  };
  const Share own = share(lane);
  const auto each_request = [&](auto&& f) {          // (four at a time: their loads wait for each other's no longer)
    f(own);
    for (int b = 64; b < a.B; b += 256) {
      const Share s[4] = {share(b + lane), share(b + 64 + lane), share(b + 128 + lane), share(b + 192 + lane)};
#pragma unroll
      for (int k = 0; k < 4; ++k) f(s[k]);
    }
  };
  int least = 0;
  float work = 0.0f;                                 // (a first guess in binary32, the same in every wave; the count that it is held to is exact)
  each_request([&](const Share& s) {
    least += s.tiles;
    work += static_cast<float>(s.tiles) * static_cast<float>(s.len);
  });
  least = last_lane(scan64(least)) * a.Hkv;
  work = last_lane(scan64(work)) * a.Hkv;
  const int budget = static_cast<int>(runs_of(least, plan.slots));   // at most plan.groups
  constexpr float kMost = 0x1p30f;
  float guess = work / plan.slots;
  int chunk, n, cut;
  for (int round = 0;; ++round) {
    chunk = (static_cast<int>(fminf(guess, kMost - GRAIN)) / GRAIN + 1) * GRAIN;
    n = cut = 0;
    each_request([&](const Share& s) {
      const int runs = items_of(s.len, chunk);
      n += s.tiles * runs;
      cut += runs > 1 ? s.tiles * runs : 0;
    });
    n = last_lane(scan64(n)) * a.Hkv;
    if (n <= budget || guess >= kMost) break;
    // as much longer as there are too many (twice, where that has not done for a while)
    guess = fmaxf(round < 6 ? chunk * (static_cast<float>(n) / budget) : 2.0f * chunk, chunk + GRAIN * 0.5f);
  }
  const unsigned deal = dealt(plan.tiles), turn = id / 8;
  const int at = static_cast<int>((turn / deal * 8 + id % 8) * deal + turn % deal);
  if (at >= n) return Spot{-1};
  const bool cut_first = n > plan.slots;
  cut = cut_first ? last_lane(scan64(cut)) * a.Hkv : 0;
  Share next = own;
  for (int b0 = 0, before[2] = {cut, 0}; b0 < a.B; b0 += 64) {
    const Share s = next;
    if (b0 + 64 < a.B) next = share(b0 + 64 + lane);
    const int runs = items_of(s.len, chunk), mine = s.tiles * runs * a.Hkv;
    const bool early = cut_first && runs > 1;
    const int early_to = before[1] + scan64(early ? mine : 0), to = before[0] + scan64(early ? 0 : mine);
    const int first = (early ? early_to : to) - mine;
    if (const uint64_t here = __ballot(at >= first && at < first + mine); here != 0) {
      const int l = __builtin_ctzll(here);
      const auto of = [&](int x) { return __builtin_amdgcn_readlane(x, l); };
      const int tiles = of(s.tiles), first_l = of(first), local = at - first_l, splits = of(runs), unit = local / tiles;
      if (local == 0 && __builtin_amdgcn_workitem_id_x() == 0) Parts<D>(a, plan).info[b0 + l] = make_int2(first_l, splits);
      return Spot{b0 + l, unit % a.Hkv, local % tiles, unit / a.Hkv, splits, at, Drafts{of(s.dr.first), of(s.dr.n), of(s.dr.base)}, of(s.len)};
    }
    before[0] = last_lane(to);
    before[1] = last_lane(early_to);
  }
  return Spot{-1};
}

// What is left of readouts that weigh nothing (see add_part).
__device__ __forceinline__ float4 infinite_only(float4 x) {
  return make_float4(add_part(0.0f, x.x, 0.0f), add_part(0.0f, x.y, 0.0f), add_part(0.0f, x.z, 0.0f), add_part(0.0f, x.w, 0.0f));
}

// The runs of a (request, row) joined: sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s, four channels of K rows a
// thread, U runs at a time; S threads share out the runs of a row, and meet in LDS. K 1,024 / (D S) rows a
// workgroup. Bound by the launch and by dependent loads.
template <int D, int K, int U, int S>
__device__ __forceinline__ void join_piece(const TreeArgs& a, const TokenPlan& plan, int groups, unsigned id) {
  constexpr int LPR = D / 4, RPG = 256 / LPR / S;  // threads for a row's channels, rows at once
  static_assert(S == 1 || K == 1);
  const int tid = __builtin_amdgcn_workitem_id_x(), seg = tid / (256 / S), lane = tid % (256 / S);
  const int units = a.Hkv * plan.tiles;
  const int group = static_cast<int>(id % groups), unit = static_cast<int>(id / groups % units), b = static_cast<int>(id / groups / units);
  const int tile = unit % plan.tiles, kvh = unit / plan.tiles, G = a.Hq / a.Hkv;
  const Parts<D> parts(a, plan);
  const int2 info = parts.info[b];                 // (not written where a request has no rows: not used either)
  const Drafts dr = drafts_of(a, b);
  const int rows = min(min(dr.n, a.max_new) * G - (tile << plan.rows_log2), plan.heads);    // of this tile
  if (group * (K * RPG) >= rows || info.y == 1) return;     // (one run: it has its readout already)
  const int tiles = (min(dr.n, a.max_new) * G + (1 << plan.rows_log2) - 1) >> plan.rows_log2;
  const int64_t step = int64_t(a.Hkv) * tiles * plan.heads;      // between a tile's runs
  const int64_t first = (int64_t(info.x) + kvh * tiles + tile) * plan.heads;
  int in_tile[K];
  float4 acc[K];
  float m[K], l[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    in_tile[k] = group * (K * RPG) + k * RPG + lane / LPR;
    acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    m[k] = -INFINITY;
    l[k] = 0.0f;
  }
  for (int s0 = seg; s0 < info.y; s0 += U * S) {
    float2 x[K][U];
    float4 v[K][U];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t at = first + min(in_tile[k], rows - 1) + min(s0 + i * S, info.y - 1) * step;
        x[k][i] = parts.ml[at];
        v[k][i] = reinterpret_cast<const float4*>(parts.o + at * D)[lane % LPR];
      }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float top = m[k];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (s0 + i * S >= info.y) x[k][i] = make_float2(-INFINITY, 0.0f);
        top = fmaxf(top, x[k][i].x);
      }
      const float base = top == -INFINITY ? 0.0f : top;
      float shrink = m[k] == -INFINITY ? 1.0f : pow2(m[k] - base), f[U], least = shrink;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        f[i] = s0 + i * S < info.y ? pow2(x[k][i].x - base) : 1.0f;
        least = fminf(least, f[i]);
      }
      m[k] = top;
      l[k] *= shrink;
#pragma unroll
      for (int i = 0; i < U; ++i) l[k] = fmaf(f[i], x[k][i].y, l[k]);
      if (__any(least == 0.0f)) {
        if (shrink == 0.0f) acc[k] = infinite_only(acc[k]), shrink = 1.0f;
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (f[i] == 0.0f) v[k][i] = infinite_only(v[k][i]), f[i] = 1.0f;
      }
      acc[k].x *= shrink; acc[k].y *= shrink; acc[k].z *= shrink; acc[k].w *= shrink;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (s0 + i * S >= info.y) break;               // (its values stand in for none)
        acc[k].x = fmaf(f[i], v[k][i].x, acc[k].x);
        acc[k].y = fmaf(f[i], v[k][i].y, acc[k].y);
        acc[k].z = fmaf(f[i], v[k][i].z, acc[k].z);
        acc[k].w = fmaf(f[i], v[k][i].w, acc[k].w);
      }
    }
  }
  if constexpr (S > 1) {
    __shared__ float4 part_o[S][256 / S];
    __shared__ float2 part_ml[S][256 / S];
    part_o[seg][lane] = acc[0];
    part_ml[seg][lane] = make_float2(m[0], l[0]);
    __syncthreads();
    if (seg > 0) return;
    float top = m[0];
#pragma unroll
    for (int i = 1; i < S; ++i) top = fmaxf(top, part_ml[i][lane].x);
    const float base = top == -INFINITY ? 0.0f : top;
    acc[0] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    l[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const float f = pow2(part_ml[i][lane].x - base);
      const float4 v = part_o[i][lane];
      l[0] = fmaf(f, part_ml[i][lane].y, l[0]);
      acc[0] = make_float4(add_part(f, v.x, acc[0].x), add_part(f, v.y, acc[0].y), add_part(f, v.z, acc[0].z), add_part(f, v.w, acc[0].w));
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (in_tile[k] >= rows) continue;
    const int row = (tile << plan.rows_log2) + in_tile[k];
    const float back = l[k] == 0.0f ? 0.0f : 1.0f / l[k];
    const int64_t at = (int64_t(dr.first + row / G) * a.Hq + kvh * G + row % G) * LPR + lane % LPR;
    reinterpret_cast<uint2*>(a.out)[at] = make_uint2(pack_bf16(acc[k].x * back, acc[k].y * back), pack_bf16(acc[k].z * back, acc[k].w * back));
  }
}

// Each workgroup takes every step-th of `pieces` (with one row a thread there is a workgroup for each).
template <int D, int K, int U, int S>
__global__ __launch_bounds__(256) void attn_join_kernel(const TreeArgs a, const TokenPlan plan, int groups, unsigned pieces, unsigned step) {
  const unsigned first = __builtin_amdgcn_workgroup_id_x();
  if constexpr (K == 1) {
    join_piece<D, K, U, S>(a, plan, groups, first);
  } else {
    for (unsigned id = first; id < pieces; id += step) join_piece<D, K, U, S>(a, plan, groups, id);
  }
}

// Rows and slots are the kernel's. Requests of up to `whole` tokens are not cut, nor are any where there are more
// than kManyRequests, which alone fill the chip four times over: each workgroup finding its part among 1,024 of 1,100
// tokens, 8 heads of d = 64, takes 449 us, whole ones 385; but 756 and 1,000 where one of them has 60,000. Among 512
// it costs nothing.
constexpr int kManyRequests = 512;

inline TokenPlan token_plan(const TreeSizes& z, int rows_log2, int slots, int whole) {
  const int64_t all = int64_t(z.max_new) * (z.Hq / z.Hkv), rows = int64_t(1) << rows_log2;
  TokenPlan p;
  p.rows_log2 = rows_log2;
  p.tiles = static_cast<int>((all + rows - 1) / rows);
  p.heads = static_cast<int>(std::min<int64_t>(all, rows));
  p.slots = slots;
  const int64_t most = int64_t(z.B) * z.Hkv * p.tiles;
  p.whole = z.max_len <= whole || (most >= 4 * slots && z.B > kManyRequests);
  const int64_t deal = 8 * dealt(p.tiles), groups = !p.whole ? (runs_of(most, slots) + deal - 1) / deal * deal : p.tiles * z.Hkv == 1 ? most : (most + 7) / 8 * 8;
  p.groups = static_cast<int>(std::min<int64_t>(groups, 0x7fffffff));
  return p;
}

// The launch that joins. Two rows a thread where one each would not fit the chip at once (6,144 workgroups, most
// without work: 14 us with one, 7.5 with two), else the runs shared out (48 runs of 512 rows: 11.7 us by one thread
// a piece, 8.0 by four; 13 runs of 64 rows 7.1 and 4.6).
constexpr int join_shares(int d) { return d == 512 ? 2 : 4; }   // (a workgroup holds a row of each share)

struct JoinPlan {
  bool many;
  int per_unit;          // pieces of a (request, head, row tile)
  int64_t pieces;
};

// Workgroups that the launch has at most, so that its size bounds no call; a call's units may have 16 pieces each.
constexpr int64_t kJoinGroups = 65536;

inline JoinPlan join_plan(const TokenPlan& p, int64_t B, int64_t Hkv, int d) {
  const int few_rows = 1024 / d / join_shares(d), many_rows = 2 * 1024 / d;
  const int64_t units = B * Hkv * p.tiles, few = (p.heads + few_rows - 1) / few_rows, many = (p.heads + many_rows - 1) / many_rows;
  const bool is_many = units * few > 2048;
  return JoinPlan{is_many, static_cast<int>(is_many ? many : few), units * (is_many ? many : few)};
}

template <int D>
void launch_join(const TreeArgs& a, const TokenPlan& p, hipStream_t s) {
  if (p.whole) return;
  const JoinPlan j = join_plan(p, a.B, a.Hkv, D);
  const unsigned pieces = static_cast<unsigned>(j.pieces), groups = static_cast<unsigned>(std::min(j.pieces, kJoinGroups));
  if (j.many) hipLaunchKernelGGL((attn_join_kernel<D, 2, 4, 1>), dim3(groups), dim3(256), 0, s, a, p, j.per_unit, pieces, groups);
  else hipLaunchKernelGGL((attn_join_kernel<D, 1, 8, join_shares(D)>), dim3(groups), dim3(256), 0, s, a, p, j.per_unit, pieces, groups);
}

}  // namespace
}  // namespace damp
