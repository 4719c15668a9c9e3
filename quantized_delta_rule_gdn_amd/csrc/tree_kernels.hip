// tree_kernels.hip -- gfx950 kernels of attention of a request's drafted tokens (a tree, or a run in
// order) over its paged key-value cache.
#include <algorithm>

#include "attn_join.h"

namespace damp {
namespace {

// ---- attention of drafted tokens -------------------------------------------------------------------
// For drafted token i of a request's n, o_i = sum_t p_it v_t / sum_t p_it over the positions t that it
// sees: all before the drafted ones, and of those the ones in its mask. As in the attention of one
// token, a request's tokens are cut into items, each of the 4 waves of a workgroup takes every fourth
// tile of 32 tokens straight from the pages into registers as operands, and the waves meet in LDS
// at the end. The rows of a product are the (drafted token, query head) pairs of one key-value head,
// 16 a workgroup. Bound by the stream of the cache: 64 requests of 8,000 tokens, 8 heads of d = 128, 354 us with 4
// rows a head and with 16, or 5.9 TB/s (reading alone reaches 7.1; waves wait 64% of their time, matrix cores are busy 6%); short
// ones by latency (one request of 500 tokens 10 us, call included). The weights' second piece costs nothing there.
template <int D, bool P16>
__global__ __launch_bounds__(256, 3) void kv_tree_kernel(const TreeArgs a, const TokenPlan plan) {
  constexpr int KS = D / 32;       // k steps of the score product
  constexpr int DPL = D / 16;      // value channels per lane
  constexpr int VW = DPL / 2;      // dwords of them
  constexpr uint32_t kNone = 0xffffffffu;
  constexpr int kAttnPages = 1024;                    // page addresses held in LDS at a time
  __shared__ uint32_t first_row[kAttnPages];          // of a page, in rows of this key-value head
  __shared__ int any_odd;                             // values that are not finite have been taken out
  __shared__ float part_m[4][16], part_l[4][16];
  __shared__ __align__(16) float part_o[4][16][D + 4];

  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const Spot spot = spot_of<4 * kAttnTile, D>(a, plan);
  const int b = spot.b, kvh = spot.kvh, split = spot.split, splits = spot.splits;
  if (b < 0) return;
  const int G = a.Hq / a.Hkv;
  const Drafts dr = spot.dr;
  const int64_t rows = int64_t(min(dr.n, a.max_new)) * G, row0 = int64_t(spot.tile) * 16;
  if (row0 >= rows) return;
  const Parts<D> parts(a, plan);
  const int len = spot.len;
  // its tokens: an even share of the request's, in whole tiles
  const int share = ((len + splits - 1) / splits + kAttnTile - 1) / kAttnTile * kAttnTile;
  const int begin = min(split * share, len), end = min(begin + share, len);
  const int in_page = (1 << a.page_log2) - 1;

  const int live_rows = static_cast<int>(min(rows - row0, int64_t(16)));
  const unsigned my_row = static_cast<unsigned>(row0) + min(r, live_rows - 1);
  const int token = my_row / G;
  Frag qf[KS];
  {
    const int64_t at = int64_t(dr.first + token) * a.Hq + kvh * G + my_row % G;
#pragma unroll
    for (int x = 0; x < KS; ++x) qf[x] = load_frag(a.q + (at * D + g * 8 + x * 32) * 2);
  }

  f32x4 o[DPL];
  float mx = -INFINITY, sum = 0.0f;
  bool taken_out = false;
#pragma unroll
  for (int m = 0; m < DPL; ++m) o[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const uint32_t k_off = r * (D * 2) + g * 16;                  // a half tile's K rows as operands
  const uint32_t v_off = 4 * g * (D * 2) + r * (DPL * 2);       // and its V rows
  constexpr int kRun = P16 ? kAttnPages * 16 : kAttnPages;
  if (tid == 0) any_odd = 0;
  for (int from = begin; from < end; from += kRun) {
    const int to = min(from + kRun, end);
    const int p0 = from >> a.page_log2, np = ((to - 1) >> a.page_log2) - p0 + 1;
    if (from > begin) __syncthreads();       // the last addresses are no longer read
    for (int i = tid; i < np; i += 256) {
      const int pid = a.table[int64_t(b) * a.max_blocks + p0 + i];
      const bool fine = pid >= 0 && pid < a.num_pages;
      first_row[i] = fine ? (static_cast<uint32_t>(pid) * a.Hkv + kvh) << a.page_log2 : kNone;
    }
    __syncthreads();
    for (int t0 = from + wv * kAttnTile; t0 < to; t0 += 4 * kAttnTile) {
      // (rows past the end lie in the last page or repeat its last row; what they give is masked)
      Frag kf[2][KS];
      uint32_t vr[8][VW];
      uint32_t dead = 0;   // bit i: this lane's value row i is not part of the request
      const auto load_v = [&](const uint8_t* vp, int i) {
        if constexpr (VW == 4) {
          const uint4 w = *reinterpret_cast<const uint4*>(vp);
          vr[i][0] = w.x; vr[i][1] = w.y; vr[i][2] = w.z; vr[i][3] = w.w;
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(vp);
          vr[i][0] = w.x; vr[i][1] = w.y;
        }
      };
      if constexpr (P16) {
        int64_t base[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int pos = t0 + 16 * h;
          const uint32_t page = __builtin_amdgcn_readfirstlane(first_row[min((pos >> a.page_log2) - p0, np - 1)]);
          if (page == kNone) dead |= 0xfu << (4 * h);
          base[h] = int64_t(page == kNone ? 0 : page + (pos & in_page)) * (D * 2);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int x = 0; x < KS; ++x) kf[h][x] = load_frag(a.k_pages + base[h] + k_off + x * 64);
#pragma unroll
        for (int i = 0; i < 8; ++i) load_v(a.v_pages + base[i >> 2] + v_off + (i & 3) * (D * 2), i);
      } else {
        const auto row_of = [&](int pos) -> uint32_t {   // cache row of a position, kNone where there is none
          const uint32_t page = first_row[(pos >> a.page_log2) - p0];
          return page == kNone ? kNone : page + (pos & in_page);
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t row = row_of(min(t0 + 16 * h + r, to - 1));
          const uint8_t* kp = a.k_pages + int64_t(row == kNone ? 0 : row) * (D * 2) + g * 16;
#pragma unroll
          for (int x = 0; x < KS; ++x) kf[h][x] = load_frag(kp + x * 64);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t row = row_of(min(t0 + 16 * (i >> 2) + 4 * g + (i & 3), to - 1));
          if (row == kNone) dead |= 1u << i;
          load_v(a.v_pages + int64_t(row == kNone ? 0 : row) * (D * 2) + r * (DPL * 2), i);
        }
      }
      float p[8];
      {
        f32x4 s[2] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
        for (int x = 0; x < KS; ++x)
#pragma unroll
          for (int h = 0; h < 2; ++h) s[h] = mfma(kf[h][x], qf[x], s[h]);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = s[i >> 2][i & 3] * a.scale_log2;
      }
      if (__any(dead != 0) || t0 + kAttnTile > to) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (t0 + 16 * (i >> 2) + 4 * g + (i & 3) >= to) dead |= 1u << i;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (dead >> i & 1) {
            p[i] = -INFINITY;
#pragma unroll
            for (int w = 0; w < VW; ++w) vr[i][w] = 0;   // whatever lies there: 0 * NaN is NaN
          }
      }
      if (t0 + kAttnTile > dr.base) {
        uint32_t odd = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int w = 0; w < VW; ++w) odd |= not_finite(vr[i][w]);
        if (__any(odd != 0)) {
          taken_out = true;
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int w = 0; w < VW; ++w) vr[i][w] = finite_only(vr[i][w]);
        }
        const uint32_t seen = seen_window(a, dr, token, t0 - dr.base) >> (4 * g);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!(seen >> (16 * (i >> 2) + (i & 3)) & 1)) p[i] = -INFINITY;
      }
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, p[i]);
      if (__any(top > mx + kSlack)) {
        top = fmaxf(max_row_slots(top), mx);
        const float shrink = top == -INFINITY ? 1.0f : pow2(mx - top);
        mx = top;
        sum *= shrink;
#pragma unroll
        for (int m = 0; m < DPL; ++m) o[m] *= shrink;
      }
      const float base = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = pow2(p[i] - base);
      Frag pf[2];
      pack_weights(p, pf, sum);
#pragma unroll
      for (int m = 0; m < DPL; m += 2) {   // (each sum's products apart)
        Frag vf[2];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          vf[0].w[w] = __builtin_amdgcn_perm(vr[2 * w + 1][m / 2], vr[2 * w][m / 2], 0x05040100u);
          vf[1].w[w] = __builtin_amdgcn_perm(vr[2 * w + 1][m / 2], vr[2 * w][m / 2], 0x07060302u);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          o[m] = mfma(vf[0], pf[x], o[m]);
          o[m + 1] = mfma(vf[1], pf[x], o[m + 1]);
        }
      }
    }
  }
  __syncthreads();
  if (taken_out && lane == 0) any_odd = 1;
  __syncthreads();
  if (any_odd && wv == 0) {
    // (from the first tile with a drafted token on; what an earlier tile has already is added again, to no effect)
    for (int t = max(dr.base - kAttnTile, begin); t < end; ++t) {
      const int page = a.table[int64_t(b) * a.max_blocks + (t >> a.page_log2)];
      if (page < 0 || page >= a.num_pages) continue;
      const int64_t row = (((int64_t(page) * a.Hkv + kvh) << a.page_log2) + (t & in_page)) * (D * 2);
      const bool seen = t < dr.base || (seen_window(a, dr, token, t - dr.base) & 1);
#pragma unroll
      for (int i = 0; i < 4; ++i)          // channel DPL (4 g + i) + m
#pragma unroll
        for (int m = 0; m < DPL; m += 4) {
          const uint2 v = *reinterpret_cast<const uint2*>(a.v_pages + row + (DPL * (4 * g + i) + m) * 2);
          const f32x4 x = add_odd(f32x4{o[m][i], o[m + 1][i], o[m + 2][i], o[m + 3][i]}, v, seen);
#pragma unroll
          for (int k = 0; k < 4; ++k) o[m + k][i] = x[k];
        }
    }
  }

  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  if (g == 0) {
    part_m[wv][r] = mx;
    part_l[wv][r] = sum;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int m = 0; m < DPL; ++m) part_o[wv][r][DPL * (4 * g + i) + m] = o[m][i];
  __syncthreads();
  for (int x = tid; x < live_rows * D; x += 256) {
    const int h = x / D, c = x % D;
    const float m0 = fmaxf(fmaxf(part_m[0][h], part_m[1][h]), fmaxf(part_m[2][h], part_m[3][h]));
    const float base = m0 == -INFINITY ? 0.0f : m0;
    float acc = 0.0f, l = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = pow2(part_m[w][h] - base);
      acc = add_part(f, part_o[w][h][c], acc);
      l = fmaf(f, part_l[w][h], l);
    }
    if (splits == 1) {
      const unsigned row = static_cast<unsigned>(row0) + h;
      const int64_t at = (int64_t(dr.first + row / G) * a.Hq + kvh * G + row % G) * D + c;
      reinterpret_cast<uint16_t*>(a.out)[at] = float_to_bf16_bits(l == 0.0f ? 0.0f : acc / l);
    } else {
      const int64_t at = int64_t(spot.at) * plan.heads + h;
      parts.o[at * D + c] = acc;
      if (c == 0) parts.ml[at] = make_float2(m0, l);
    }
  }
}

// Many rows: the 16 R rows of each wave are its own, and tiles of 64 tokens are loaded into LDS for all four,
// the next one among this one's products, with one barrier a tile (read by every wave for itself, 64 rows
// would draw 64 KB a tile from the L1, as long as their products take). The weights are rounded once: a
// second piece took 15 to 20% more time (48 requests 127 -> 142 us, 4 long ones 166 -> 203, before the tiles were
// loaded ahead). 48 requests of up to 4,096 tokens, 128 rows, 8 heads of d = 128: 97 to 104 us and 9 for the
// join, which is 4.1 to 4.4 TB/s; the matrix cores are busy for a fifth of the time, the waves wait for the stream, of
// which the longest run has 43 tiles and the mean 25 (a third tile on its way did not help: 119 us with it, 114
// without). 4 requests of up to 65,536 tokens, 512 rows
// of d = 64: 85 us and 8, 660 TFLOP/s; matrix cores busy 37%, vector unit 55%: for 16 x 16 scores the products take
// 72 cycles, the exponentials alone 64 and the rest of the softmax 40.
constexpr int kWideTile = 64;

template <int D, int R, bool P16>
__global__ __launch_bounds__(256, D == 64 ? 3 : 2) void kv_tree_wide_kernel(const TreeArgs a, const TokenPlan plan) {
  constexpr int KS = D / 32, MB = D / 16, TB = kWideTile / 16;
  constexpr int PW = D / 8, RL = 64 / PW, NL = 16 / RL;   // 16-byte pieces of a row, rows of a load, loads for a wave's 16 rows
  // (each buffer is an array of its own, so that reads of one need not keep their order with loads into another)
  __shared__ __align__(1024) uint8_t k0[kWideTile * D * 2], k1[kWideTile * D * 2], v0[kWideTile * D * 2], v1[kWideTile * D * 2];
  __shared__ uint32_t tile_live[2][4];
  __shared__ int any_odd;                               // values that are not finite have been taken out

  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const Spot spot = spot_of<kWideTile, D>(a, plan);
  const int b = spot.b, kvh = spot.kvh, split = spot.split, splits = spot.splits;
  if (b < 0) return;
  const int G = a.Hq / a.Hkv;
  const Drafts dr = spot.dr;
  const int64_t rows = int64_t(min(dr.n, a.max_new)) * G, row0 = int64_t(spot.tile) * (64 * R);
  if (row0 >= rows) return;
  const Parts<D> parts(a, plan);
  const int len = spot.len;
  const int share = ((len + splits - 1) / splits + kWideTile - 1) / kWideTile * kWideTile;
  const int begin = min(split * share, len), end = min(begin + share, len);
  const int in_page = (1 << a.page_log2) - 1;
  const int live_rows = static_cast<int>(min(rows - row0, int64_t(64 * R)));
  const bool idle = wv * 16 * R >= live_rows;           // none of the rows is this wave's
  // (a negative scale goes into the queries' signs; one of 0 becomes the least one, as 0 times -infinity is NaN)
  const float scale = fabsf(a.scale_log2) < 0x1p-126f ? 0x1p-126f : fabsf(a.scale_log2);     // (NaN stays NaN)
  const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0;
  const float slack = fminf(kSlack / scale, 0x1p100f);

  int token[R];
  Frag qf[R][KS];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const unsigned row = static_cast<unsigned>(row0) + min(16 * (wv * R + j) + r, live_rows - 1);
    token[j] = row / G;
    const int64_t at = int64_t(dr.first + token[j]) * a.Hq + kvh * G + row % G;
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      qf[j][x] = load_frag(a.q + (at * D + g * 8 + x * 32) * 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) qf[j][x].w[i] ^= flip;
    }
  }
  f32x4 o[R][MB];
  float mx[R];
  f32x4 sum[R];                      // the same in all four
#pragma unroll
  for (int j = 0; j < R; ++j) {
    mx[j] = -INFINITY;
    sum[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int m = 0; m < MB; ++m) o[j][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  uint32_t odd = 0;

  // Each wave loads 16 rows of a tile's keys and values. Their pages are looked up one tile ahead.
  const int row_l = lane / PW, piece_l = lane % PW;
  uint32_t k_off[NL], v_off[NL];
#pragma unroll
  for (int n = 0; n < NL; ++n) {
    const int t = 16 * wv + n * RL + row_l;
    k_off[n] = (n * RL + row_l) * (P16 ? D * 2 : 0) + (piece_l ^ row_turn<PW>(t)) * 16;
    v_off[n] = (n * RL + row_l) * (P16 ? D * 2 : 0) + (piece_l ^ column_turn<PW>(t)) * 16;
  }
  const auto page_of = [&](int t0) -> int {
    const int pos = min(t0 + 16 * wv + (P16 ? 0 : r), end - 1);
    return a.table[int64_t(b) * a.max_blocks + (pos >> a.page_log2)];
  };
  struct Tile {
    int64_t at[P16 ? 1 : NL];      // bytes to the wave's rows, or to each load's
    uint32_t live;                 // which rows exist
  };
  const auto tile_at = [&](int t0, int pid) -> Tile {
    const int left = min(max(end - (t0 + 16 * wv), 0), 16);
    Tile from;
    if constexpr (P16) {
      const int id0 = __builtin_amdgcn_readfirstlane(pid);
      const bool fine = id0 >= 0 && id0 < a.num_pages && left > 0;
      from.live = fine ? (1u << left) - 1 : 0;
      // (rows past the end lie in the same page; where there is no page, the first one's rows stand in)
      from.at[0] = (fine ? ((int64_t(id0) * a.Hkv + kvh) << a.page_log2) + ((t0 + 16 * wv) & in_page) : 0) * (D * 2);
    } else {
      const bool fine = pid >= 0 && pid < a.num_pages && r < left;
      from.live = static_cast<uint32_t>(__ballot(fine)) & 0xffffu;
      const uint32_t mine = fine ? ((static_cast<uint32_t>(pid) * a.Hkv + kvh) << a.page_log2) + ((t0 + 16 * wv + r) & in_page) : 0;
#pragma unroll
      for (int n = 0; n < NL; ++n) from.at[n] = int64_t(static_cast<uint32_t>(__shfl(static_cast<int>(mine), n * RL + row_l))) * (D * 2);
    }
    return from;
  };
  constexpr int kLoads = 2 * NL;
  const auto load = [&](int n, const Tile& from, uint8_t* tile_k, uint8_t* tile_v) {
    const int i = n % NL, to = 16 * wv * (D * 2) + i * 1024;
    const int64_t at = from.at[P16 ? 0 : i];
    if (n < NL) load_to_lds(a.k_pages + at + k_off[i], tile_k + to);
    else load_to_lds(a.v_pages + at + v_off[i], tile_v + to);
  };
  int pid = 0;
  if (tid == 0) any_odd = 0;
  if (begin < end) {
    const Tile from = tile_at(begin, page_of(begin));
    pid = page_of(begin + kWideTile);
#pragma unroll
    for (int n = 0; n < kLoads; ++n) load(n, from, k0, v0);
    if (lane == 0) tile_live[0][wv] = from.live;
  } else {
    __syncthreads();
  }
  // The tile at t0, which lies in the first two buffers, while the next is loaded into the others.
  const auto step = [&](int t0, int buf, uint8_t* tile_k, uint8_t* tile_v, uint8_t* next_k, uint8_t* next_v) {
    landed();
    __syncthreads();                 // (the tile before is no longer read, either)
    uint32_t live_w[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) live_w[w] = __builtin_amdgcn_readfirstlane(tile_live[buf][w]);
    const bool drafted = t0 + kWideTile > dr.base;
    if ((live_w[0] & live_w[1] & live_w[2] & live_w[3]) != 0xffffu || drafted) {
      // rows that do not exist become 0, and values that are not finite, where some token may not see them, are taken out
#pragma unroll
      for (int n = 0; n < NL; ++n) {
        u32x4* at = reinterpret_cast<u32x4*>(tile_v + 16 * wv * (D * 2) + n * 1024 + lane * 16);
        u32x4 w = *at;
        w &= tile_live[buf][wv] >> (n * RL + row_l) & 1 ? ~0u : 0u;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (!drafted) continue;
          odd |= not_finite(w[x]);
          w[x] = finite_only(w[x]);
        }
        *at = w;
      }
      __syncthreads();
    }
    // (after the last tile rows that exist are loaded again: no branch among the products)
    const Tile from = tile_at(t0 + kWideTile, pid);
    pid = page_of(t0 + 2 * kWideTile);
    if (lane == 0) tile_live[buf ^ 1][wv] = from.live;
    if (idle) {
#pragma unroll
      for (int n = 0; n < kLoads; ++n) load(n, from, next_k, next_v);
      return;
    }

    // Operands are read four steps ahead (a read from LDS takes as long as some ten products), and the next tile's
    // loads go out one by one among the products (each takes the address unit 16 cycles).
    const auto operand = [&](int n) -> Frag {
      const int t = 16 * (n / KS) + r;
      return load_frag(tile_k + t * (D * 2) + ((4 * (n % KS) + g) ^ row_turn<PW>(t)) * 16);
    };
    f32x4 s[R][TB];
    Frag kf[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) kf[n] = operand(n);
#pragma unroll
    for (int n = 0; n < TB * KS; ++n) {
#pragma unroll
      for (int j = 0; j < R; ++j) s[j][n / KS] = mfma(kf[n % 4], qf[j][n % KS], n % KS == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : s[j][n / KS]);
      if (n + 4 < TB * KS) kf[n % 4] = operand(n + 4);
      if (n % 2 == 0 && n / 2 < kLoads) load(n / 2, from, next_k, next_v);
      __builtin_amdgcn_sched_barrier(0);
    }
    const uint32_t live[2] = {live_w[0] | live_w[1] << 16, live_w[2] | live_w[3] << 16};
    if ((live[0] & live[1]) != ~0u || drafted) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const int rel = t0 + 32 * h - dr.base;
          const uint32_t seen = rarely((rel > -32 ? live[h] & seen_window(a, dr, token[j], rel) : live[h]) >> (4 * g));
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (!(seen >> (16 * (i >> 2) + (i & 3)) & 1)) s[j][2 * h + (i >> 2)][i & 3] = -INFINITY;
        }
    }
    Frag pf[R][TB / 2];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float top = -INFINITY;
#pragma unroll
      for (int tb = 0; tb < TB; ++tb)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, s[j][tb][i]);
      if (__any(top > mx[j] + slack)) {
        top = fmaxf(max_row_slots(top), mx[j]);
        const float shrink = top == -INFINITY ? 1.0f : pow2((mx[j] - top) * scale);
        mx[j] = top;
        sum[j] *= shrink;
#pragma unroll
        for (int m = 0; m < MB; ++m) o[j][m] *= shrink;
      }
      const float base = mx[j] == -INFINITY ? 0.0f : -mx[j] * scale;
#pragma unroll
      for (int st = 0; st < TB / 2; ++st) {
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = pow2(fmaf(s[j][2 * st + (i >> 2)][i & 3], scale, base));
        pf[j][st] = round_weights(p);
        sum[j] = mfma(ones(), pf[j][st], sum[j]);
      }
    }
#pragma unroll
    for (int st = 0; st < TB / 2; ++st) {
      const int t = 32 * st + 4 * g + (r >> 2), turn = column_turn<PW>(t);    // (the row 16 further has the same turn)
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const uint8_t* v = tile_v + t * (D * 2) + ((2 * m + (r >> 1 & 1)) ^ turn) * 16 + (r & 1) * 8;
        const Frag vf = load_frag_t(reinterpret_cast<const uint16_t*>(v), reinterpret_cast<const uint16_t*>(v + 16 * D * 2));
#pragma unroll
        for (int j = 0; j < R; ++j) o[j][m] = mfma(vf, pf[j][st], o[j][m]);
      }
    }
    __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);
#pragma unroll
    for (int x = 0; x < MB * TB / 2; ++x) {
      __builtin_amdgcn_sched_group_barrier(0x008, R, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
  };
  for (int t0 = begin; t0 < end; t0 += 2 * kWideTile) {
    step(t0, 0, k0, v0, k1, v1);
    if (t0 + kWideTile < end) step(t0 + kWideTile, 1, k1, v1, k0, v0);
  }
  landed();                          // (nothing may be on its way into LDS that the workgroup no longer holds)

  if (__any(odd != 0)) any_odd = 1;
  __syncthreads();
  if (any_odd) {
    // (from the first tile with a drafted token on; what an earlier tile has already is added again, to no effect)
#pragma unroll 1
    for (int t = max(dr.base - kWideTile, begin); t < end; ++t) {
      const int page = a.table[int64_t(b) * a.max_blocks + (t >> a.page_log2)];
      if (page < 0 || page >= a.num_pages) continue;
      const uint8_t* v = a.v_pages + (((int64_t(page) * a.Hkv + kvh) << a.page_log2) + (t & in_page)) * (D * 2) + g * 8;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const bool seen = t < dr.base || (seen_window(a, dr, token[j], t - dr.base) & 1);
#pragma unroll
        for (int m = 0; m < MB; ++m) o[j][m] = add_odd(o[j][m], *reinterpret_cast<const uint2*>(v + 32 * m), seen);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int in_tile = 16 * (wv * R + j) + r;
    if (in_tile >= live_rows) continue;
    if (splits == 1) {
      const unsigned row = static_cast<unsigned>(row0) + in_tile;
      const float back = sum[j][0] == 0.0f ? 0.0f : 1.0f / sum[j][0];
      uint8_t* to = a.out + ((int64_t(dr.first + token[j]) * a.Hq + kvh * G + row % G) * D + 4 * g) * 2;
#pragma unroll
      for (int m = 0; m < MB; ++m)
        *reinterpret_cast<uint2*>(to + 32 * m) = make_uint2(pack_bf16(o[j][m][0] * back, o[j][m][1] * back), pack_bf16(o[j][m][2] * back, o[j][m][3] * back));
    } else {
      const int64_t at = int64_t(spot.at) * plan.heads + in_tile;
#pragma unroll
      for (int m = 0; m < MB; ++m) *reinterpret_cast<f32x4*>(parts.o + at * D + 16 * m + 4 * g) = o[j][m];
      if (g == 0) parts.ml[at] = make_float2(mx[j] * scale, sum[j][0]);
    }
  }
}

// How a call's rows are taken (us, call included).
// - Up to 16 rows a key-value head: by kv_tree_kernel. A request of 500 tokens takes 10 and by the wide one 13;
//   48 of 2,000, 8 heads of d = 128, take 80 and 84. With 32 rows these take 86 and 73.
// - Else in tiles of 64 rows through LDS, or of 128 where there are enough of them: one request of 300 tokens with
//   128 rows and 2 heads takes 10.1 in tiles of 64 and 13.3 in one of 128, 4 of 20,000 with 4 heads 33 and
//   38; 8 of 30,000 with 4 heads 64 and 59, 48 of 2,000 with 8 heads 126 and 119.
// - Workgroups at once: with 3 a CU instead of 2, 20 requests of 5,000 tokens with 16 rows take 86 instead of 81
//   (with 1.5, 91); the wide ones of d = 64, which hold the least LDS, 97 with 3 and 100 with 2.
// - Not cut up to 1,024 tokens (16 rows; 900 of d = 64 take 10.2 whole and 13.5 cut, of d = 128 14.4 and 13.5) or
//   512 (500 take 12.6 whole and 13.4 cut, of d = 64 10.5 and 13.4; 700 with 128 rows 20.5 and 15).
TokenPlan tree_plan(const TreeSizes& z, int d) {
  const int64_t rows = int64_t(z.max_new) * (z.Hq / z.Hkv), units = int64_t(z.B) * z.Hkv * ((rows + 127) / 128);
  const int log2 = rows <= 16 ? 4 : rows <= 64 || units < 24 ? 6 : 7;
  // workgroups that registers and LDS leave room for on the 256 CUs: 2 each, 3 of the wide ones with d = 64
  return token_plan(z, log2, d == 64 && log2 > 4 ? 768 : 512, log2 == 4 ? 1024 : 512);
}

template <int D, bool P16>
void tree_dp(const TreeArgs& a, const TokenPlan& p, hipStream_t s) {
  if (p.rows_log2 == 4) hipLaunchKernelGGL((kv_tree_kernel<D, P16>), dim3(p.groups), dim3(256), 0, s, a, p);
  else if (p.rows_log2 == 6) hipLaunchKernelGGL((kv_tree_wide_kernel<D, 1, P16>), dim3(p.groups), dim3(256), 0, s, a, p);
  else hipLaunchKernelGGL((kv_tree_wide_kernel<D, 2, P16>), dim3(p.groups), dim3(256), 0, s, a, p);
}

template <int D>
hipError_t tree_d(const TreeArgs& a, const TreeSizes& z, hipStream_t s) {
  const TokenPlan p = tree_plan(z, D);
  if (a.page_log2 >= 4) tree_dp<D, true>(a, p, s);
  else tree_dp<D, false>(a, p, s);
  launch_join<D>(a, p, s);
  return hipGetLastError();
}

}  // namespace

int64_t kv_tree_grid(const TreeSizes& z, int32_t d) { return tree_plan(z, d).groups; }

size_t kv_tree_ws_bytes(const TreeSizes& z, int32_t d) { return parts_bytes(tree_plan(z, d), z, d); }

hipError_t launch_kv_tree(int d, const TreeArgs& a, hipStream_t s) {
  const TreeSizes z{a.B, a.Hq, a.Hkv, a.max_new, a.max_len};
  switch (d) {
    case 64: return tree_d<64>(a, z, s);
    case 128: return tree_d<128>(a, z, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace damp
