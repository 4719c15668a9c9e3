// latent_kernels.hip -- gfx950 kernels of latent attention over a paged cache of latents: one row
// c | k_rope of DC + DC / 8 channels a token, shared by all heads. Absorbed form: the row is the key and
// its first DC channels are the value.
#include <algorithm>

#include "attn_join.h"

namespace damp {
namespace {

// ---- the store of new latents --------------------------------------------------------------------
// A copy by slot map, 16 bytes a thread.
__global__ __launch_bounds__(256) void latent_append_kernel(const LatentAppendArgs a) {
  const int pc = a.dc / 8, per_row = pc + a.dr / 8;
  const int64_t n = int64_t(a.T) * per_row;
  const int64_t first = int64_t(__builtin_amdgcn_workgroup_id_x()) * 256 + __builtin_amdgcn_workitem_id_x();
  const int64_t step = __builtin_amdgcn_grid_size_x();
  for (int64_t x = first; x < n; x += step) {
    const int64_t t = x / per_row;
    const int c = static_cast<int>(x - t * per_row);
    const int64_t slot = a.slot_map[t];
    if (slot < 0 || slot >= a.num_slots) continue;
    const uint4 w = c < pc ? reinterpret_cast<const uint4*>(a.c)[t * pc + c] : reinterpret_cast<const uint4*>(a.k_rope)[t * (per_row - pc) + c - pc];
    reinterpret_cast<uint4*>(a.pages)[slot * per_row + c] = w;
  }
}

// ---- attention, absorbed form ----------------------------------------------------------------------
// o = sum_t p_t c_t / sum_t p_t, p_t = exp(scale q.(c_t | k_t) - m): all heads of a token read the same
// rows, so the rows of a product are (token, head) pairs and the tile of 64 cached tokens that a
// workgroup holds in LDS serves both products of all its 16 R rows. The 4 waves share out the scores by
// tokens (and for 64 rows by two halves of the rows), meet for the maximum of each row, hand the
// weights over through LDS, and share out the readout by channels, so that a tile is read from LDS once
// (scores: as rows; readout: transposed on the way). The next tile is on its way in registers meanwhile.
// Few heads are bound by the stream of the cache, many by the products.
constexpr int kLatTile = 64;

template <int DC>
struct LatGeo {
  static constexpr int DR = DC / 8, W = DC + DR;     // channels of a row
  static constexpr int CH = W / 8;                   // 16-byte pieces of a row
  static constexpr int ST = 16 * CH / 64;            // pieces that a lane carries: 16 rows a wave,
  static constexpr int PW = CH % 8 == 0 ? 8 : 4;     // of which a load takes PW neighbouring ones
  static constexpr int RL = 64 / PW, NR = 16 / RL;   // of RL rows; NR loads for all rows
  static constexpr int LD = W * 2 + 32;              // bytes between rows in LDS: an odd number of 32-byte units
};

template <int DC, int R, bool P16, int PIECES>
__global__ __launch_bounds__(256, R * DC > 512 ? 1 : 2) void latent_kernel(const TreeArgs a, const AttnPlan plan) {
  using Geo = LatGeo<DC>;
  constexpr int W = Geo::W, KS = W / 32, CB = DC / 64;   // k steps; 16-channel blocks of a wave's share
  constexpr int RW = R == 4 ? 2 : R, TB = R == 4 ? 2 : 1, TG = 4 / TB;   // row groups and token blocks a wave scores; token groups
  constexpr int LDP = kLatTile * 2 + 16;
  __shared__ __align__(16) uint8_t tile_k[kLatTile * Geo::LD];
  __shared__ __align__(16) uint8_t tile_p[PIECES][16 * R][LDP];
  __shared__ float part[TG][16 * R];
  __shared__ uint32_t tile_live[4], tile_odd[4];
  __shared__ int64_t sh[8];

  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const unsigned id = __builtin_amdgcn_workgroup_id_x();
  const int item = id / plan.tiles, tile = id % plan.tiles, H = a.Hq;

  const Item it = item_of<kLatTile>(a, plan, item, sh);
  const int b = it.b, split = it.split, splits = it.splits;
  if (b < 0) return;
  const Drafts dr = drafts_of(a, b);
  const int64_t rows = int64_t(min(dr.n, a.max_new)) * H, row0 = int64_t(tile) * (16 * R);
  if (row0 >= rows) return;
  const int len = length_of(a, b);
  const int share = ((len + splits - 1) / splits + kLatTile - 1) / kLatTile * kLatTile;
  const int begin = min(split * share, len), end = min(begin + share, len);
  const int in_page = (1 << a.page_log2) - 1;
  const int live_rows = static_cast<int>(min(rows - row0, int64_t(16 * R)));
  const int wr = R == 4 ? wv >> 1 : 0, wt = R == 4 ? wv & 1 : wv;   // this wave's row groups and token blocks

  int token[RW];
  Frag qf[RW][KS];
#pragma unroll
  for (int j = 0; j < RW; ++j) {
    const unsigned row = static_cast<unsigned>(row0) + min(16 * (wr * RW + j) + r, live_rows - 1);
    token[j] = row / H;
    const int64_t at = int64_t(dr.first + token[j]) * H + row % H;
#pragma unroll
    for (int x = 0; x < KS; ++x) qf[j][x] = load_frag(a.q + (at * W + g * 8 + x * 32) * 2);
  }
  f32x4 o[R][CB];
  float mx[R], sum[RW];
  bool taken_out = false;            // values that are not finite (the same for all waves)
#pragma unroll
  for (int j = 0; j < R; ++j) {
    mx[j] = -INFINITY;
#pragma unroll
    for (int m = 0; m < CB; ++m) o[j][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
#pragma unroll
  for (int j = 0; j < RW; ++j) sum[j] = 0.0f;

  // Each wave carries 16 rows of a tile. Their pages are looked up one tile ahead of their loads.
  uint4 st[Geo::ST];
  uint32_t carried = 0;              // which of the rows in st exist
  const int row_l = lane / Geo::PW, piece_l = lane % Geo::PW;
  const auto page_of = [&](int t0) -> int {
    const int pos = min(t0 + 16 * wv + (P16 ? 0 : r), end - 1);
    return a.table[int64_t(b) * a.max_blocks + (pos >> a.page_log2)];
  };
  const auto issue = [&](int t0, int pid) {
    const int left = min(max(end - (t0 + 16 * wv), 0), 16);
    const uint4* pages = reinterpret_cast<const uint4*>(a.k_pages) + piece_l;
    if constexpr (P16) {
      const int id0 = __builtin_amdgcn_readfirstlane(pid);
      const bool fine = id0 >= 0 && id0 < a.num_pages && left > 0;
      carried = fine ? (1u << left) - 1 : 0;
      // (rows past the end lie in the same page; where there is no page, the first one's rows stand in)
      const int64_t row = fine ? (int64_t(id0) << a.page_log2) + ((t0 + 16 * wv) & in_page) : 0;
#pragma unroll
      for (int n = 0; n < Geo::NR; ++n) {
        const uint4* src = pages + (row + n * Geo::RL + row_l) * Geo::CH;
#pragma unroll
        for (int k = 0; k < Geo::ST / Geo::NR; ++k) st[n * (Geo::ST / Geo::NR) + k] = src[k * Geo::PW];
      }
    } else {
      const bool fine = pid >= 0 && pid < a.num_pages && r < left;
      carried = static_cast<uint32_t>(__ballot(fine)) & 0xffffu;
      const uint32_t row = fine ? (static_cast<uint32_t>(pid) << a.page_log2) + ((t0 + 16 * wv + r) & in_page) : 0;
#pragma unroll
      for (int n = 0; n < Geo::NR; ++n) {
        const uint4* src = pages + int64_t(static_cast<uint32_t>(__shfl(static_cast<int>(row), n * Geo::RL + row_l))) * Geo::CH;
#pragma unroll
        for (int k = 0; k < Geo::ST / Geo::NR; ++k) st[n * (Geo::ST / Geo::NR) + k] = src[k * Geo::PW];
      }
    }
  };
  int pid = 0;
  if (begin < end) {
    pid = page_of(begin);
    issue(begin, pid);
    if (begin + kLatTile < end) pid = page_of(begin + kLatTile);
  }
  for (int t0 = begin; t0 < end; t0 += kLatTile) {
    __syncthreads();                 // the tile before is no longer read
    {
      uint32_t odd = 0;
#pragma unroll
      for (int n = 0; n < Geo::NR; ++n) {
        const int row = n * Geo::RL + row_l;
        const uint32_t keep = carried >> row & 1 ? ~0u : 0u;
#pragma unroll
        for (int k = 0; k < Geo::ST / Geo::NR; ++k) {
          uint4 w = st[n * (Geo::ST / Geo::NR) + k];
          if (carried != 0xffffu) w = make_uint4(w.x & keep, w.y & keep, w.z & keep, w.w & keep);
          if (t0 + kLatTile > dr.base) odd |= not_finite(w.x) | not_finite(w.y) | not_finite(w.z) | not_finite(w.w);
          *reinterpret_cast<uint4*>(tile_k + (16 * wv + row) * Geo::LD + (k * Geo::PW + piece_l) * 16) = w;
        }
      }
      odd = __any(odd != 0);
      if (lane == 0) {
        tile_live[wv] = carried;
        tile_odd[wv] = odd;
      }
    }
    __syncthreads();
    if (t0 + kLatTile < end) {
      issue(t0 + kLatTile, pid);
      if (t0 + 2 * kLatTile < end) pid = page_of(t0 + 2 * kLatTile);
    }
    const bool odd_tile = (tile_odd[0] | tile_odd[1] | tile_odd[2] | tile_odd[3]) != 0;
    // scores^T [token][row]: lane column = row, tokens 4 g .. + 3 of each block
    float p[RW][TB][4];
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) {
      const int block = wt * TB + tb;
      f32x4 s[RW];
#pragma unroll
      for (int j = 0; j < RW; ++j) s[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        const Frag kf = load_frag(tile_k + (16 * block + r) * Geo::LD + g * 16 + x * 64);
#pragma unroll
        for (int j = 0; j < RW; ++j) s[j] = mfma(kf, qf[j][x], s[j]);
        if (x % 6 == 5) __builtin_amdgcn_sched_barrier(0);   // (all operands loaded ahead would not fit the registers)
      }
      const uint32_t live = __builtin_amdgcn_readfirstlane(tile_live[block]);
      const int first = t0 + 16 * block;
#pragma unroll
      for (int j = 0; j < RW; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[j][tb][i] = s[j][i] * a.scale_log2;
        if (live != 0xffffu || first + 16 > dr.base) {
          uint32_t seen = live;
          if (first + 16 > dr.base) seen &= seen_window(a, dr, token[j], first - dr.base);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!(seen >> (4 * g + i) & 1)) p[j][tb][i] = -INFINITY;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      float top = -INFINITY;
#pragma unroll
      for (int tb = 0; tb < TB; ++tb)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, p[j][tb][i]);
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      if (g == 0) part[wt][16 * (wr * RW + j) + r] = top;
    }
    __syncthreads();
    if (odd_tile) {                  // (the scores have been taken)
      taken_out = true;
#pragma unroll 1
      for (int x = lane; x < 16 * Geo::CH; x += 64) {
        uint4* at = reinterpret_cast<uint4*>(tile_k + (16 * wv + x / Geo::CH) * Geo::LD + x % Geo::CH * 16);
        const uint4 w = *at;
        *at = make_uint4(finite_only(w.x), finite_only(w.y), finite_only(w.z), finite_only(w.w));
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float top = mx[j];
#pragma unroll
      for (int t = 0; t < TG; ++t) top = fmaxf(top, part[t][16 * j + r]);
      if (__any(top > mx[j])) {
        const float shrink = top == -INFINITY ? 1.0f : pow2(mx[j] - top);
        mx[j] = top;
        if (j / RW == wr) {
          // (the same for the whole wave; RW == R but for 64 rows)
#pragma unroll
          for (int x = 0; x < RW; ++x)
            if (x == j % RW) sum[x] *= shrink;
        }
#pragma unroll
        for (int m = 0; m < CB; ++m) o[j][m] *= shrink;
      }
    }
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      float m0 = mx[0];
#pragma unroll
      for (int x = 1; x < R; ++x)
        if (x == wr * RW + j) m0 = mx[x];
      const float base = m0 == -INFINITY ? 0.0f : m0;
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[j][tb][i] = pow2(p[j][tb][i] - base);
        uint32_t w[PIECES][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) pack_pair<PIECES>(p[j][tb][2 * i], p[j][tb][2 * i + 1], i, w, sum[j]);
        const int row = 16 * (wr * RW + j) + r, at = (16 * (wt * TB + tb) + 4 * g) * 2;
#pragma unroll
        for (int x = 0; x < PIECES; ++x) *reinterpret_cast<uint2*>(&tile_p[x][row][at]) = make_uint2(w[x][0], w[x][1]);
      }
    }
    __syncthreads();
    // readout^T [channel][row] += V^T P^T, this wave's channels
#pragma unroll
    for (int step = 0; step < kLatTile / 32; ++step) {
      Frag pf[R][PIECES];
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int x = 0; x < PIECES; ++x) pf[j][x] = load_frag(&tile_p[x][16 * j + r][(32 * step + 8 * g) * 2]);
      const uint8_t* v = tile_k + (32 * step + 8 * g + (r >> 2)) * Geo::LD + (wv * (DC / 4) + 4 * (r & 3)) * 2;
#pragma unroll
      for (int m = 0; m < CB; ++m) {
        const Frag vf = load_frag_t(reinterpret_cast<const uint16_t*>(v + 32 * m), reinterpret_cast<const uint16_t*>(v + 32 * m + 4 * Geo::LD));
#pragma unroll
        for (int x = 0; x < PIECES; ++x)
#pragma unroll
          for (int j = 0; j < R; ++j) o[j][m] = mfma(vf, pf[j][x], o[j][m]);
      }
    }
  }
  if (taken_out) {
    // (from the first tile with a drafted token on; what an earlier tile has already is added again, to no effect)
#pragma unroll 1
    for (int t = max(dr.base - kLatTile, begin); t < end; ++t) {
      const int page = a.table[int64_t(b) * a.max_blocks + (t >> a.page_log2)];
      if (page < 0 || page >= a.num_pages) continue;
      const uint8_t* v = a.k_pages + ((int64_t(page) << a.page_log2) + (t & in_page)) * (W * 2) + (wv * (DC / 4) + 4 * g) * 2;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const unsigned row = static_cast<unsigned>(row0) + min(16 * j + r, live_rows - 1);
        const bool seen = t < dr.base || (seen_window(a, dr, row / H, t - dr.base) & 1);
#pragma unroll
        for (int m = 0; m < CB; ++m) o[j][m] = add_odd(o[j][m], *reinterpret_cast<const uint2*>(v + 32 * m), seen);
      }
    }
  }

  // the rows' sums over all tokens
  __syncthreads();
#pragma unroll
  for (int j = 0; j < RW; ++j) {
    sum[j] += __shfl_xor(sum[j], 16);
    sum[j] += __shfl_xor(sum[j], 32);
    if (g == 0) part[wt][16 * (wr * RW + j) + r] = sum[j];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < R; ++j) {
    float l = 0.0f;
#pragma unroll
    for (int t = 0; t < TG; ++t) l += part[t][16 * j + r];
    if (16 * j + r >= live_rows) continue;
    const int ch = wv * (DC / 4) + 4 * g;
    if (splits == 1) {
      const unsigned row = static_cast<unsigned>(row0) + 16 * j + r;
      const int64_t at = (int64_t(dr.first + row / H) * H + row % H) * DC + ch;
      const float back = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
      for (int m = 0; m < CB; ++m)
        *reinterpret_cast<uint2*>(a.out + (at + 16 * m) * 2) =
            make_uint2(pack_bf16(o[j][m][0] * back, o[j][m][1] * back), pack_bf16(o[j][m][2] * back, o[j][m][3] * back));
    } else {
      const int64_t at = int64_t(id) * plan.heads + 16 * j + r;
#pragma unroll
      for (int m = 0; m < CB; ++m) *reinterpret_cast<f32x4*>(a.ws + at * DC + ch + 16 * m) = o[j][m];
      if (wv == 0 && g == 0)
        reinterpret_cast<float2*>(a.ws + int64_t(plan.items) * plan.tiles * plan.heads * DC)[at] = make_float2(mx[j], l);
    }
  }
}

AttnPlan latent_plan(const TreeSizes& z) {
  const int64_t rows = int64_t(z.max_new) * z.Hq;
  AttnPlan p;
  p.rows = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  p.tiles = static_cast<int>((rows + p.rows - 1) / p.rows);
  p.heads = static_cast<int>(std::min<int64_t>(rows, p.rows));
  const int64_t slots = p.rows == 64 ? 256 : 512;      // workgroups that are resident at once
  // items of full length fill the chip once, the requests' last ones included
  const int64_t each = std::max<int64_t>(slots / p.tiles, 1), wanted = each > 2 * int64_t(z.B) ? each - z.B : each;
  const int64_t most = (int64_t(z.max_len) + kLatTile - 1) / kLatTile * z.B;
  p.per_unit = static_cast<int>(std::min<int64_t>(wanted, std::max<int64_t>(most, 1)));
  const bool whole = z.max_len <= 256 || int64_t(p.tiles) * z.B >= 4 * slots;
  p.items = whole ? z.B : p.per_unit + z.B;
  return p;
}

template <int DC, int R>
void latent_dr(const TreeArgs& a, const AttnPlan& p, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.items) * p.tiles);
  if (a.page_log2 >= 4) hipLaunchKernelGGL((latent_kernel<DC, R, true, 1>), grid, dim3(256), 0, s, a, p);
  else hipLaunchKernelGGL((latent_kernel<DC, R, false, 1>), grid, dim3(256), 0, s, a, p);
}

template <int DC>
hipError_t latent_d(const TreeArgs& a, const TreeSizes& z, hipStream_t s) {
  const AttnPlan p = latent_plan(z);
  if (p.rows == 16) latent_dr<DC, 1>(a, p, s);
  else if (p.rows == 32) latent_dr<DC, 2>(a, p, s);
  else latent_dr<DC, 4>(a, p, s);
  if (p.items > a.B) launch_join<DC, kLatTile>(a, p, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_latent_append(const LatentAppendArgs& a, hipStream_t s) {
  const int64_t n = int64_t(a.T) * ((a.dc + a.dr) / 8);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((n + 255) / 256, 16384));
  hipLaunchKernelGGL(latent_append_kernel, dim3(grid), dim3(256), 0, s, a);
  return hipGetLastError();
}

int64_t latent_grid(const TreeSizes& z, int32_t dc) {
  const AttnPlan p = latent_plan(z);
  return std::max((int64_t(p.per_unit) + z.B) * p.tiles, join_groups(p, dc) * z.B * p.tiles);
}

size_t latent_ws_bytes(const TreeSizes& z, int32_t dc) {
  const AttnPlan p = latent_plan(z);
  if (p.items == z.B) return 0;
  return static_cast<size_t>(p.items) * p.tiles * p.heads * (static_cast<size_t>(dc) + 2) * 4;
}

hipError_t launch_latent(int dc, const TreeArgs& a, hipStream_t s) {
  const TreeSizes z{a.B, a.Hq, 1, a.max_new, a.max_len};
  switch (dc) {
    case 256: return latent_d<256>(a, z, s);
    case 512: return latent_d<512>(a, z, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace damp
