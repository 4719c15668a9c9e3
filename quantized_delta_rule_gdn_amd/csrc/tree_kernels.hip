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
// 16 R a workgroup: a tile's keys and values serve R operand groups once they are in registers.
template <int D, int R, bool P16, int PIECES>
__global__ __launch_bounds__(256, R == 4 ? 1 : 2) void kv_tree_kernel(const TreeArgs a, const AttnPlan plan) {
  constexpr int KS = D / 32;       // k steps of the score product
  constexpr int DPL = D / 16;      // value channels per lane
  constexpr int VW = DPL / 2;      // dwords of them
  constexpr uint32_t kNone = 0xffffffffu;
  constexpr int kAttnPages = 1024;                    // page addresses held in LDS at a time
  __shared__ uint32_t first_row[kAttnPages];          // of a page, in rows of this key-value head
  __shared__ int64_t sh[8];
  __shared__ int any_odd;                             // values that are not finite have been taken out
  __shared__ float part_m[4][16], part_l[4][16];
  __shared__ __align__(16) float part_o[4][16][D + 4];

  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const unsigned id = __builtin_amdgcn_workgroup_id_x();
  const int units = a.Hkv * plan.tiles;
  const int item = id / units, unit = id % units, tile = unit % plan.tiles, kvh = unit / plan.tiles;
  const int G = a.Hq / a.Hkv;

  // the request this item belongs to, and its drafted tokens
  const Item it = item_of(a, plan, item, sh);
  const int b = it.b, split = it.split, splits = it.splits;
  if (b < 0) return;
  const Drafts dr = drafts_of(a, b);
  const int64_t rows = int64_t(min(dr.n, a.max_new)) * G, row0 = int64_t(tile) * (16 * R);
  if (row0 >= rows) return;
  const int len = length_of(a, b);
  // its tokens: an even share of the request's, in whole tiles
  const int share = ((len + splits - 1) / splits + kAttnTile - 1) / kAttnTile * kAttnTile;
  const int begin = min(split * share, len), end = min(begin + share, len);
  const int in_page = (1 << a.page_log2) - 1;

  const int live_rows = static_cast<int>(min(rows - row0, int64_t(16 * R)));
  int token[R];                    // of this lane's rows
  Frag qf[R][KS];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const unsigned row = static_cast<unsigned>(row0) + min(16 * j + r, live_rows - 1);
    token[j] = row / G;
    const int64_t at = int64_t(dr.first + token[j]) * a.Hq + kvh * G + row % G;
#pragma unroll
    for (int x = 0; x < KS; ++x) qf[j][x] = load_frag(a.q + (at * D + g * 8 + x * 32) * 2);
  }

  f32x4 o[R][DPL];
  float mx[R], sum[R];
  bool taken_out = false;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    mx[j] = -INFINITY;
    sum[j] = 0.0f;
#pragma unroll
    for (int m = 0; m < DPL; ++m) o[j][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
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
      float p[R][8];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        f32x4 s[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) s[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int x = 0; x < KS; ++x)
#pragma unroll
          for (int h = 0; h < 2; ++h) s[h] = mfma(kf[h][x], qf[j][x], s[h]);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[j][i] = s[i >> 2][i & 3] * a.scale_log2;
      }
      if (__any(dead != 0) || t0 + kAttnTile > to) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (t0 + 16 * (i >> 2) + 4 * g + (i & 3) >= to) dead |= 1u << i;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (dead >> i & 1) {
#pragma unroll
            for (int j = 0; j < R; ++j) p[j][i] = -INFINITY;
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
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const uint32_t seen = seen_window(a, dr, token[j], t0 - dr.base) >> (4 * g);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (!(seen >> (16 * (i >> 2) + (i & 3)) & 1)) p[j][i] = -INFINITY;
        }
      }
      Frag pf[R][PIECES];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        float top = mx[j];
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, p[j][i]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        if (__any(top > mx[j])) {               // (the maximum settles after a few tiles)
          const float shrink = top == -INFINITY ? 1.0f : pow2(mx[j] - top);
          mx[j] = top;
          sum[j] *= shrink;
#pragma unroll
          for (int m = 0; m < DPL; ++m) o[j][m] *= shrink;
        }
        const float base = mx[j] == -INFINITY ? 0.0f : mx[j];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          p[j][i] = pow2(p[j][i] - base);
        }
        pack_weights<PIECES>(p[j], pf[j], sum[j]);
      }
#pragma unroll
      for (int m = 0; m < DPL; m += 2) {   // (each sum's products apart)
        Frag vf[2];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          vf[0].w[w] = __builtin_amdgcn_perm(vr[2 * w + 1][m / 2], vr[2 * w][m / 2], 0x05040100u);
          vf[1].w[w] = __builtin_amdgcn_perm(vr[2 * w + 1][m / 2], vr[2 * w][m / 2], 0x07060302u);
        }
#pragma unroll
        for (int x = 0; x < PIECES; ++x)
#pragma unroll
          for (int j = 0; j < R; ++j) {
            o[j][m] = mfma(vf[0], pf[j][x], o[j][m]);
            o[j][m + 1] = mfma(vf[1], pf[j][x], o[j][m + 1]);
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
      bool seen[R];
#pragma unroll
      for (int j = 0; j < R; ++j) seen[j] = t < dr.base || (seen_window(a, dr, token[j], t - dr.base) & 1);
#pragma unroll
      for (int i = 0; i < 4; ++i)          // channel DPL (4 g + i) + m
#pragma unroll
        for (int m = 0; m < DPL; m += 4) {
          const uint2 v = *reinterpret_cast<const uint2*>(a.v_pages + row + (DPL * (4 * g + i) + m) * 2);
#pragma unroll
          for (int j = 0; j < R; ++j) {
            const f32x4 x = add_odd(f32x4{o[j][m][i], o[j][m + 1][i], o[j][m + 2][i], o[j][m + 3][i]}, v, seen[j]);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[j][m + k][i] = x[k];
          }
        }
    }
  }

#pragma unroll
  for (int j = 0; j < R; ++j) {
    if (16 * j >= live_rows) break;          // (the same for all threads)
    sum[j] += __shfl_xor(sum[j], 16);
    sum[j] += __shfl_xor(sum[j], 32);
    if (j > 0) __syncthreads();
    if (g == 0) {
      part_m[wv][r] = mx[j];
      part_l[wv][r] = sum[j];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < DPL; ++m) part_o[wv][r][DPL * (4 * g + i) + m] = o[j][m][i];
    __syncthreads();
    const int live = min(live_rows - 16 * j, 16);
    for (int x = tid; x < live * D; x += 256) {
      const int h = x / D, c = x % D;
      const float m0 = fmaxf(fmaxf(part_m[0][h], part_m[1][h]), fmaxf(part_m[2][h], part_m[3][h]));
      const float base = m0 == -INFINITY ? 0.0f : m0;
      float acc = 0.0f, l = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = pow2(part_m[w][h] - base);
        acc = fmaf(f, part_o[w][h][c], acc);
        l = fmaf(f, part_l[w][h], l);
      }
      if (splits == 1) {
        const unsigned row = static_cast<unsigned>(row0) + 16 * j + h;
        const int64_t at = (int64_t(dr.first + row / G) * a.Hq + kvh * G + row % G) * D + c;
        reinterpret_cast<uint16_t*>(a.out)[at] = float_to_bf16_bits(l == 0.0f ? 0.0f : acc / l);
      } else {
        const int64_t at = int64_t(id) * plan.heads + 16 * j + h;
        a.ws[at * D + c] = acc;
        if (c == 0) reinterpret_cast<float2*>(a.ws + int64_t(plan.items) * units * plan.heads * D)[at] = make_float2(m0, l);
      }
    }
  }
}

// Rows a workgroup: as many as there are, up to 64.
int tree_groups(int64_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

AttnPlan tree_plan(const TreeSizes& z) {
  const int64_t rows = int64_t(z.max_new) * (z.Hq / z.Hkv);
  AttnPlan p;
  p.rows = 16 * tree_groups(rows);
  p.tiles = static_cast<int>((rows + p.rows - 1) / p.rows);
  p.heads = static_cast<int>(std::min<int64_t>(rows, p.rows));
  const int64_t units = int64_t(z.Hkv) * p.tiles, wanted = p.rows == 64 ? 512 : 1024;
  const int64_t most = (int64_t(z.max_len) + kAttnLeast - 1) / kAttnLeast * z.B;   // no more are ever cut
  p.per_unit = static_cast<int>(std::min<int64_t>(std::max<int64_t>(wanted / units, 1), std::max<int64_t>(most, 1)));
  const bool whole = z.max_len <= 1024 || (z.max_len <= 2048 && units * z.B >= 512);
  p.items = whole ? z.B : p.per_unit + z.B;
  return p;
}

template <int D, int R>
void tree_dr(const TreeArgs& a, const AttnPlan& p, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.items) * a.Hkv * p.tiles);
  if (a.page_log2 >= 4) hipLaunchKernelGGL((kv_tree_kernel<D, R, true, 2>), grid, dim3(256), 0, s, a, p);
  else hipLaunchKernelGGL((kv_tree_kernel<D, R, false, 2>), grid, dim3(256), 0, s, a, p);
}

template <int D>
hipError_t tree_d(const TreeArgs& a, const TreeSizes& z, hipStream_t s) {
  const AttnPlan p = tree_plan(z);
  if (p.rows == 16) tree_dr<D, 1>(a, p, s);
  else if (p.rows == 32) tree_dr<D, 2>(a, p, s);
  else tree_dr<D, 4>(a, p, s);
  if (p.items > a.B) launch_join<D, kAttnLeast>(a, p, s);
  return hipGetLastError();
}

}  // namespace

int64_t kv_tree_grid(const TreeSizes& z, int32_t d) {
  const AttnPlan p = tree_plan(z);
  const int64_t units = int64_t(z.Hkv) * p.tiles;
  return std::max((int64_t(p.per_unit) + z.B) * units, z.B * units * join_groups(p, d));
}

size_t kv_tree_ws_bytes(const TreeSizes& z, int32_t d) {
  const AttnPlan p = tree_plan(z);
  if (p.items == z.B) return 0;
  return static_cast<size_t>(p.items) * z.Hkv * p.tiles * p.heads * (static_cast<size_t>(d) + 2) * 4;
}

hipError_t launch_kv_tree(int d, const TreeArgs& a, hipStream_t s) {
  const TreeSizes z{a.B, a.Hq, a.Hkv, a.max_new, a.max_len};
  switch (d) {
    case 64: return tree_d<64>(a, z, s);
    case 128: return tree_d<128>(a, z, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace damp
