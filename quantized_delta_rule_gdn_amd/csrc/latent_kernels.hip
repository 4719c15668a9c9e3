// latent_kernels.hip -- gfx950 kernels of latent attention over a paged cache of latents: one row
// c | k_rope of DC + DC / 8 channels a token, shared by all heads. Absorbed form: the row is the key and
// its first DC channels are the value.
#include <algorithm>

#include "attn_join.h"

namespace damp {
namespace {

// ---- the store of new latents --------------------------------------------------------------------
// A copy by slot map, 16 bytes a thread.
__global__ __launch_bounds__(256) void latent_append_kernel(const LatentAppendArgs a, int64_t step) {
  const int pc = a.dc / 8, per_row = pc + a.dr / 8;
  const int64_t n = int64_t(a.T) * per_row;
  const int64_t first = int64_t(__builtin_amdgcn_workgroup_id_x()) * 256 + __builtin_amdgcn_workitem_id_x();
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

template <int DC, int NW>
struct LatGeo {
  static constexpr int DR = DC / 8, W = DC + DR;     // channels of a row
  static constexpr int CH = W / 8;                   // 16-byte pieces of a row
  static constexpr int ROWS = kLatTile / NW;         // rows of a tile that a wave carries
  static constexpr int NR = ROWS / 8, PK = (CH + 7) / 8;   // by loads of 8 neighbouring pieces of 8 rows
  static constexpr int LD = W * 2 + 32;              // bytes between rows in LDS: an odd number of 32-byte units
};

template <int DC, int R, int NW, bool P16, int PIECES>
__global__ __launch_bounds__(64 * NW, 2) void latent_kernel(const TreeArgs a, const TokenPlan plan) {
  using Geo = LatGeo<DC, NW>;
  constexpr int W = Geo::W, KS = W / 32, CB = DC / (16 * NW);   // k steps; 16-channel blocks of a wave's share
  constexpr int TG = NW / R, TB = 4 / TG;            // the waves that share 16 rows' scores; blocks of 16 tokens each takes
  constexpr int LDP = kLatTile * 2 + 16;
  __shared__ __align__(16) uint8_t tile_k[kLatTile * Geo::LD];
  __shared__ __align__(16) uint8_t tile_p[PIECES][16 * R][LDP];
  __shared__ float part[TG][16 * R];
  __shared__ uint32_t tile_live[NW], tile_odd[NW];

  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const Spot spot = spot_of<kLatTile, DC>(a, plan);
  const int b = spot.b, split = spot.split, splits = spot.splits, H = a.Hq;
  if (b < 0) return;
  const Drafts dr = spot.dr;
  const int64_t rows = int64_t(min(dr.n, a.max_new)) * H, row0 = int64_t(spot.tile) * (16 * R);
  if (row0 >= rows) return;
  const Parts<DC> parts(a, plan);
  const int len = spot.len;
  const int share = ((len + splits - 1) / splits + kLatTile - 1) / kLatTile * kLatTile;
  const int begin = min(split * share, len), end = min(begin + share, len);
  const int in_page = (1 << a.page_log2) - 1;
  const int live_rows = static_cast<int>(min(rows - row0, int64_t(16 * R)));
  const int wr = wv / TG, wt = wv % TG;              // this wave's rows and tokens

  const unsigned my_row = static_cast<unsigned>(row0) + min(16 * wr + r, live_rows - 1);
  const int token = my_row / H;
  Frag qf[KS];
  {
    const int64_t at = int64_t(dr.first + token) * H + my_row % H;
#pragma unroll
    for (int x = 0; x < KS; ++x) qf[x] = load_frag(a.q + (at * W + g * 8 + x * 32) * 2);
  }
  f32x4 o[R][CB];
  float mx[R], sum = 0.0f;
  bool taken_out = false;            // values that are not finite (the same for all waves)
#pragma unroll
  for (int j = 0; j < R; ++j) {
    mx[j] = -INFINITY;
#pragma unroll
    for (int m = 0; m < CB; ++m) o[j][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // Each wave carries its rows of a tile. Their pages are looked up one tile ahead of their loads.
  constexpr uint32_t kAll = (1u << Geo::ROWS) - 1;
  u32x4 st[Geo::NR][Geo::PK];
  uint32_t carried = 0;              // which of the rows in st exist
  const int row_l = lane / 8, piece_l = lane % 8;
  const auto page_of = [&](int t0) -> int {
    const int pos = min(t0 + Geo::ROWS * wv + (P16 ? 0 : lane % Geo::ROWS), end - 1);
    return a.table[int64_t(b) * a.max_blocks + (pos >> a.page_log2)];
  };
  const auto issue = [&](int t0, int pid) {
    const int first = t0 + Geo::ROWS * wv, left = min(max(end - first, 0), Geo::ROWS);
    int64_t row[Geo::NR];
    if constexpr (P16) {
      const int id0 = __builtin_amdgcn_readfirstlane(pid);
      const bool fine = id0 >= 0 && id0 < a.num_pages && left > 0;
      carried = fine ? (1u << left) - 1 : 0;
      // (rows past the end lie in the same page; where there is no page, the first one's rows stand in)
      const int64_t at = fine ? (int64_t(id0) << a.page_log2) + (first & in_page) : 0;
#pragma unroll
      for (int n = 0; n < Geo::NR; ++n) row[n] = at + 8 * n + row_l;
    } else {
      const bool fine = pid >= 0 && pid < a.num_pages && lane % Geo::ROWS < left;
      carried = static_cast<uint32_t>(__ballot(fine)) & kAll;
      const uint32_t mine = fine ? (static_cast<uint32_t>(pid) << a.page_log2) + ((first + lane % Geo::ROWS) & in_page) : 0;
#pragma unroll
      for (int n = 0; n < Geo::NR; ++n) row[n] = static_cast<uint32_t>(__shfl(static_cast<int>(mine), 8 * n + row_l));
    }
#pragma unroll
    for (int n = 0; n < Geo::NR; ++n) {
      const u32x4* src = reinterpret_cast<const u32x4*>(a.k_pages) + row[n] * Geo::CH;
#pragma unroll
      for (int k = 0; k < Geo::PK; ++k) st[n][k] = src[8 * k + (8 * k + 7 < Geo::CH ? piece_l : min(piece_l, Geo::CH - 1 - 8 * k))];
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
        const int row = 8 * n + row_l;
        const uint32_t keep = carried >> row & 1 ? ~0u : 0u;
#pragma unroll
        for (int k = 0; k < Geo::PK; ++k) {
          u32x4 w = st[n][k];
          if (carried != kAll) w &= rarely(keep);
          if (t0 + kLatTile > dr.base) {
            w = rarely(w);
            odd |= not_finite(w[0]) | not_finite(w[1]) | not_finite(w[2]) | not_finite(w[3]);
          }
          if (8 * k + 7 < Geo::CH || 8 * k + piece_l < Geo::CH)
            *reinterpret_cast<u32x4*>(tile_k + (Geo::ROWS * wv + row) * Geo::LD + (8 * k + piece_l) * 16) = w;
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
    uint32_t odd_tile = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) odd_tile |= tile_odd[w];
    // scores^T [token][row]: lane column = row, tokens 4 g .. + 3 of each block
    float p[TB][4];
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) {
      const int block = wt * TB + tb;
      f32x4 s[2] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};   // (two sums: each product waits for the one before it)
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        const Frag kf = load_frag(tile_k + (16 * block + r) * Geo::LD + g * 16 + x * 64);
        s[x & 1] = mfma(kf, qf[x], s[x & 1]);
        if (x % 6 == 5) __builtin_amdgcn_sched_barrier(0);   // (all operands loaded ahead would not fit the registers)
      }
      uint32_t live = NW == 8 ? tile_live[2 * block % NW] | tile_live[(2 * block + 1) % NW] << 8 : tile_live[block % NW];
      live = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(live)));
      const int first = t0 + 16 * block;
#pragma unroll
      for (int i = 0; i < 4; ++i) p[tb][i] = (s[0][i] + s[1][i]) * a.scale_log2;
      if (live != 0xffffu || first + 16 > dr.base) {
        uint32_t seen = live;
        if (first + 16 > dr.base) seen &= seen_window(a, dr, token, first - dr.base);
        seen = rarely(seen);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!(seen >> (4 * g + i) & 1)) p[tb][i] = -INFINITY;
      }
    }
    {
      float top = -INFINITY;
#pragma unroll
      for (int tb = 0; tb < TB; ++tb)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, p[tb][i]);
      top = max_row_slots(top);
      if (g == 0) part[wt][16 * wr + r] = top;
    }
    __syncthreads();
    if (odd_tile) {                  // (the scores have been taken)
      taken_out = true;
#pragma unroll 1
      for (int x = lane; x < Geo::ROWS * Geo::CH; x += 64) {
        u32x4* at = reinterpret_cast<u32x4*>(tile_k + (Geo::ROWS * wv + x / Geo::CH) * Geo::LD + x % Geo::CH * 16);
        u32x4 w = *at;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = finite_only(w[i]);
        *at = w;
      }
    }
    float base = 0.0f;               // of this wave's rows
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float top = mx[j];
#pragma unroll
      for (int t = 0; t < TG; ++t) top = fmaxf(top, part[t][16 * j + r]);
      if (__any(top > mx[j])) {
        const float shrink = top == -INFINITY ? 1.0f : pow2(mx[j] - top);
        mx[j] = top;
        if (j == wr) sum *= shrink;
#pragma unroll
        for (int m = 0; m < CB; ++m) o[j][m] *= shrink;
      }
      if (j == wr) base = mx[j] == -INFINITY ? 0.0f : mx[j];
    }
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) {
#pragma unroll
      for (int i = 0; i < 4; ++i) p[tb][i] = pow2(p[tb][i] - base);
      uint32_t w[PIECES][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) pack_pair<PIECES>(p[tb][2 * i], p[tb][2 * i + 1], i, w, sum);
#pragma unroll
      for (int x = 0; x < PIECES; ++x) *reinterpret_cast<uint2*>(&tile_p[x][16 * wr + r][(16 * (wt * TB + tb) + 4 * g) * 2]) = make_uint2(w[x][0], w[x][1]);
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
      const uint8_t* v = tile_k + (32 * step + 8 * g + (r >> 2)) * Geo::LD + (wv * (DC / NW) + 4 * (r & 3)) * 2;
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
      const uint8_t* v = a.k_pages + ((int64_t(page) << a.page_log2) + (t & in_page)) * (W * 2) + (wv * (DC / NW) + 4 * g) * 2;
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
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  if (g == 0) part[wt][16 * wr + r] = sum;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < R; ++j) {
    float l = 0.0f;
#pragma unroll
    for (int t = 0; t < TG; ++t) l += part[t][16 * j + r];
    if (16 * j + r >= live_rows) continue;
    const int ch = wv * (DC / NW) + 4 * g;
    if (splits == 1) {
      const unsigned row = static_cast<unsigned>(row0) + 16 * j + r;
      const int64_t at = (int64_t(dr.first + row / H) * H + row % H) * DC + ch;
      const float back = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
      for (int m = 0; m < CB; ++m)
        *reinterpret_cast<uint2*>(a.out + (at + 16 * m) * 2) =
            make_uint2(pack_bf16(o[j][m][0] * back, o[j][m][1] * back), pack_bf16(o[j][m][2] * back, o[j][m][3] * back));
    } else {
      const int64_t at = int64_t(spot.at) * plan.heads + 16 * j + r;
#pragma unroll
      for (int m = 0; m < CB; ++m) *reinterpret_cast<f32x4*>(parts.o + at * DC + ch + 16 * m) = o[j][m];
      if (wv == 0 && g == 0) parts.ml[at] = make_float2(mx[j], l);
    }
  }
}

// More than 16 rows: the products take longer than the stream, so the two are given to different waves and
// run at the same time. Four waves score a tile, 16 rows each and all 64 tokens (so a row's maximum is its
// wave's own), while the other four weigh the tile before it, a quarter of the channels each and all rows:
// every SIMD holds one of either kind, and two barriers a tile are left. Two tiles lie in LDS, the third
// is on its way in the registers of all eight.
template <int DC, int R, bool P16>
__global__ __launch_bounds__(512, 2) void latent_wide_kernel(const TreeArgs a, const TokenPlan plan) {
  using Geo = LatGeo<DC, 8>;
  constexpr int W = Geo::W, KS = W / 32, CB = DC / 64, TB = kLatTile / 16;
  constexpr int LD = W * 2 + 16, LDP = kLatTile * 2 + 16;
  __shared__ __align__(16) uint8_t tile_k[2][kLatTile * LD];
  __shared__ __align__(16) uint8_t tile_p[16 * R][LDP];
  __shared__ float row_m[16 * R], row_l[16 * R];     // by what the sums shrink; in the end maximum and sum
  __shared__ uint32_t tile_live[2][8], tile_odd[2][8];

  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const Spot spot = spot_of<kLatTile, DC>(a, plan);
  const int b = spot.b, split = spot.split, splits = spot.splits, H = a.Hq;
  if (b < 0) return;
  const Drafts dr = spot.dr;
  const int64_t rows = int64_t(min(dr.n, a.max_new)) * H, row0 = int64_t(spot.tile) * (16 * R);
  if (row0 >= rows) return;
  const int len = spot.len;
  const int share = ((len + splits - 1) / splits + kLatTile - 1) / kLatTile * kLatTile;
  const int begin = min(split * share, len), end = min(begin + share, len);
  const int in_page = (1 << a.page_log2) - 1;
  const int live_rows = static_cast<int>(min(rows - row0, int64_t(16 * R)));

  // Each wave carries 8 rows of a tile. Their pages are looked up one tile ahead of their loads.
  u32x4 st[Geo::PK];
  uint32_t carried = 0;              // which of the rows in st exist
  const int row_l8 = lane / 8, piece_l = lane % 8;
  const auto page_of = [&](int t0) -> int {
    const int pos = min(t0 + 8 * wv + (P16 ? 0 : row_l8), end - 1);
    return a.table[int64_t(b) * a.max_blocks + (pos >> a.page_log2)];
  };
  const auto issue = [&](int t0, int pid) {
    const int first = t0 + 8 * wv, left = min(max(end - first, 0), 8);
    int64_t row;
    if constexpr (P16) {
      const int id0 = __builtin_amdgcn_readfirstlane(pid);
      const bool fine = id0 >= 0 && id0 < a.num_pages && left > 0;
      carried = fine ? (1u << left) - 1 : 0;
      // (rows past the end lie in the same page; where there is no page, the first one's rows stand in)
      row = (fine ? (int64_t(id0) << a.page_log2) + (first & in_page) : 0) + row_l8;
    } else {
      const bool fine = pid >= 0 && pid < a.num_pages && row_l8 < left;
      const uint64_t all = __ballot(fine);           // (8 lanes a row)
      carried = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) carried |= static_cast<uint32_t>(all >> (8 * i) & 1) << i;
      row = fine ? (int64_t(pid) << a.page_log2) + ((first + row_l8) & in_page) : 0;
    }
    const u32x4* src = reinterpret_cast<const u32x4*>(a.k_pages) + row * Geo::CH;
#pragma unroll
    for (int k = 0; k < Geo::PK; ++k) st[k] = src[8 * k + (8 * k + 7 < Geo::CH ? piece_l : min(piece_l, Geo::CH - 1 - 8 * k))];
  };
  const auto store = [&](int t0, int buf) {
    uint32_t odd = 0;
    const uint32_t keep = carried >> row_l8 & 1 ? ~0u : 0u;
#pragma unroll
    for (int k = 0; k < Geo::PK; ++k) {
      u32x4 w = st[k];
      if (carried != 0xffu) w &= rarely(keep);
      if (t0 + kLatTile > dr.base) {
        w = rarely(w);
        odd |= not_finite(w[0]) | not_finite(w[1]) | not_finite(w[2]) | not_finite(w[3]);
      }
      if (8 * k + 7 < Geo::CH || 8 * k + piece_l < Geo::CH)
        *reinterpret_cast<u32x4*>(tile_k[buf] + (8 * wv + row_l8) * LD + (8 * k + piece_l) * 16) = w;
    }
    odd = __any(odd != 0);
    if (lane == 0) {
      tile_live[buf][wv] = carried;
      tile_odd[buf][wv] = odd;
    }
  };
  int pid = 0;
  // The tile after t0 into LDS, and values of t0's that are not finite out of it (its scores have been taken).
  // True where there were any.
  const auto advance = [&](int t0, int buf) -> bool {
    if (t0 + kLatTile < end) store(t0 + kLatTile, buf ^ 1);
    if (t0 + kLatTile <= dr.base) return false;
    uint32_t odd = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) odd |= tile_odd[buf][w];
    if (odd == 0) return false;
#pragma unroll 1
    for (int x = lane; x < 8 * Geo::CH; x += 64) {
      u32x4* at = reinterpret_cast<u32x4*>(tile_k[buf] + (8 * wv + x / Geo::CH) * LD + x % Geo::CH * 16);
      u32x4 w = *at;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = finite_only(w[i]);
      *at = w;
    }
    return true;
  };
  // The loads of the tile two after t0 (past the end they repeat rows that exist), with a page looked up before.
  const auto fetch = [&](int t0) {
    issue(t0 + 2 * kLatTile, pid);
    pid = page_of(t0 + 3 * kLatTile);
  };
  if (begin < end) {
    issue(begin, page_of(begin));
    pid = page_of(begin + kLatTile);
  }

  if (wv < 4) {
    const bool mine = 16 * wv < live_rows;           // (with R == 2, and in the last row tile, some waves only carry rows)
    const unsigned my_row = static_cast<unsigned>(row0) + min(16 * wv + r, live_rows - 1);
    const int token = my_row / H;
    Frag qf[KS];
    const int64_t at = int64_t(dr.first + token) * H + my_row % H;
#pragma unroll
    for (int x = 0; x < KS; ++x) qf[x] = load_frag(a.q + (at * W + g * 8 + x * 32) * 2);
    if (begin < end) store(begin, 0);
    __syncthreads();
    float mx = -INFINITY, shrink = 1.0f, sum = 0.0f;
    uint32_t w[TB][1][2];                            // the weights: tokens 16 tb + 4 g .. + 3
    const auto score = [&](int t0, int buf) {
      f32x4 s[TB];
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) s[tb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = 0; x < KS; ++x)
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) s[tb] = mfma(load_frag(tile_k[buf] + (16 * tb + r) * LD + g * 16 + x * 64), qf[x], s[tb]);
      // operands two steps ahead, and a load of the next tile every other step
      __builtin_amdgcn_sched_group_barrier(0x100, 2 * TB, 0);
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        __builtin_amdgcn_sched_group_barrier(0x008, TB, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, TB, 0);
        if (x % 2 == 1) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      }
      float p[TB][4];
#pragma unroll
      for (int tb = 0; tb < TB; ++tb)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[tb][i] = s[tb][i] * a.scale_log2;
      uint32_t live = 0xffu;
#pragma unroll
      for (int x = 0; x < 8; ++x) live &= tile_live[buf][x];
      if (live != 0xffu || t0 + kLatTile > dr.base) {
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
          uint32_t seen = tile_live[buf][2 * tb] | tile_live[buf][2 * tb + 1] << 8;
          const int rel = t0 + 16 * tb - dr.base;
          if (rel > -16) seen &= seen_window(a, dr, token, rel);
          seen = rarely(seen >> (4 * g));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!(seen >> i & 1)) p[tb][i] = -INFINITY;
        }
      }
      float top = mx;
#pragma unroll
      for (int tb = 0; tb < TB; ++tb)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, p[tb][i]);
      top = max_row_slots(top);
      shrink = top == -INFINITY ? 1.0f : pow2(mx - top);
      mx = top;
      sum *= shrink;
      const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int tb = 0; tb < TB; ++tb)
#pragma unroll
        for (int i = 0; i < 2; ++i) pack_pair<1>(pow2(p[tb][2 * i] - base), pow2(p[tb][2 * i + 1] - base), i, w[tb], sum);
    };
    if (begin < end) {
      fetch(begin - kLatTile);
      if (mine) score(begin, 0);
    }
    if (!mine && wv < R && g == 0) row_m[16 * wv + r] = 1.0f;
    __syncthreads();
    int buf = 0;
    for (int t0 = begin; t0 < end; t0 += kLatTile, buf ^= 1) {
      if (mine) {
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) *reinterpret_cast<uint2*>(&tile_p[16 * wv + r][(16 * tb + 4 * g) * 2]) = make_uint2(w[tb][0][0], w[tb][0][1]);
        if (g == 0) row_m[16 * wv + r] = shrink;
      }
      advance(t0, buf);
      __syncthreads();
      fetch(t0);
      if (mine && t0 + kLatTile < end) score(t0 + kLatTile, buf ^ 1);
      __syncthreads();
    }
    if (wv < R) {
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (g == 0) {
        row_m[16 * wv + r] = mx;
        row_l[16 * wv + r] = sum;
      }
    }
    __syncthreads();
    return;
  }

  const int first_ch = (wv - 4) * (DC / 4);
  f32x4 o[R][CB];
  bool taken_out = false;            // values that are not finite
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int m = 0; m < CB; ++m) o[j][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (begin < end) store(begin, 0);
  __syncthreads();
  if (begin < end) fetch(begin - kLatTile);
  __syncthreads();                   // the first tile's scores
  int buf = 0;
  for (int t0 = begin; t0 < end; t0 += kLatTile, buf ^= 1) {
    taken_out |= advance(t0, buf);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const float shrink = row_m[16 * j + r];
      if (__any(shrink != 1.0f)) {     // (the maximum settles after a few tiles)
#pragma unroll
        for (int m = 0; m < CB; ++m) o[j][m] *= shrink;
      }
    }
    fetch(t0);
#pragma unroll
    for (int step = 0; step < kLatTile / 32; ++step) {
      Frag pf[R];
#pragma unroll
      for (int j = 0; j < R; ++j) pf[j] = load_frag(&tile_p[16 * j + r][(32 * step + 8 * g) * 2]);
      const uint8_t* v = tile_k[buf] + (32 * step + 8 * g + (r >> 2)) * LD + (first_ch + 4 * (r & 3)) * 2;
#pragma unroll
      for (int m = 0; m < CB; ++m) {
        const Frag vf = load_frag_t(reinterpret_cast<const uint16_t*>(v + 32 * m), reinterpret_cast<const uint16_t*>(v + 32 * m + 4 * LD));
#pragma unroll
        for (int j = 0; j < R; ++j) o[j][m] = mfma(vf, pf[j], o[j][m]);
      }
    }
    // operands three blocks ahead, and a load of the next tile every other block
    __builtin_amdgcn_sched_group_barrier(0x100, R + 6, 0);
#pragma unroll
    for (int step = 0; step < kLatTile / 32; ++step) {
#pragma unroll
      for (int m = 0; m < CB; ++m) {
        __builtin_amdgcn_sched_group_barrier(0x008, R, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        if (m % 2 == 1) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x100, R, 0);
    }
    __syncthreads();
  }
  __syncthreads();                   // maxima and sums
  if (taken_out) {
    // (from the first tile with a drafted token on; what an earlier tile has already is added again, to no effect)
#pragma unroll 1
    for (int t = max(dr.base - kLatTile, begin); t < end; ++t) {
      const int page = a.table[int64_t(b) * a.max_blocks + (t >> a.page_log2)];
      if (page < 0 || page >= a.num_pages) continue;
      const uint8_t* v = a.k_pages + ((int64_t(page) << a.page_log2) + (t & in_page)) * (W * 2) + (first_ch + 4 * g) * 2;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const unsigned row = static_cast<unsigned>(row0) + min(16 * j + r, live_rows - 1);
        const bool seen = t < dr.base || (seen_window(a, dr, row / H, t - dr.base) & 1);
#pragma unroll
        for (int m = 0; m < CB; ++m) o[j][m] = add_odd(o[j][m], *reinterpret_cast<const uint2*>(v + 32 * m), seen);
      }
    }
  }
  const Parts<DC> parts(a, plan);
#pragma unroll
  for (int j = 0; j < R; ++j) {
    if (16 * j + r >= live_rows) continue;
    const float l = row_l[16 * j + r];
    const int ch = first_ch + 4 * g;
    if (splits == 1) {
      const unsigned row = static_cast<unsigned>(row0) + 16 * j + r;
      const int64_t at = (int64_t(dr.first + row / H) * H + row % H) * DC + ch;
      const float back = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
      for (int m = 0; m < CB; ++m)
        *reinterpret_cast<uint2*>(a.out + (at + 16 * m) * 2) =
            make_uint2(pack_bf16(o[j][m][0] * back, o[j][m][1] * back), pack_bf16(o[j][m][2] * back, o[j][m][3] * back));
    } else {
      const int64_t at = int64_t(spot.at) * plan.heads + 16 * j + r;
#pragma unroll
      for (int m = 0; m < CB; ++m) *reinterpret_cast<f32x4*>(parts.o + at * DC + ch + 16 * m) = o[j][m];
      if (wv == 4 && g == 0) parts.ml[at] = make_float2(row_m[16 * j + r], l);
    }
  }
}

TokenPlan latent_plan(const TreeSizes& z) {
  const int64_t rows = int64_t(z.max_new) * z.Hq;
  const int log2 = rows <= 16 ? 4 : rows <= 32 ? 5 : 6;
  // workgroups that LDS leaves room for on the 256 CUs: two of four waves each, or one of eight
  return token_plan(z, log2, log2 == 4 ? 512 : 256, 256);
}

template <int DC, bool P16>
void latent_dp(const TreeArgs& a, const TokenPlan& p, hipStream_t s) {
  const dim3 grid(p.groups);
  if (p.rows_log2 == 4) hipLaunchKernelGGL((latent_kernel<DC, 1, 4, P16, 1>), grid, dim3(256), 0, s, a, p);
  else if (p.rows_log2 == 5) hipLaunchKernelGGL((latent_wide_kernel<DC, 2, P16>), grid, dim3(512), 0, s, a, p);
  else hipLaunchKernelGGL((latent_wide_kernel<DC, 4, P16>), grid, dim3(512), 0, s, a, p);
}

template <int DC>
hipError_t latent_d(const TreeArgs& a, const TreeSizes& z, hipStream_t s) {
  const TokenPlan p = latent_plan(z);
  if (a.page_log2 >= 4) latent_dp<DC, true>(a, p, s);
  else latent_dp<DC, false>(a, p, s);
  launch_join<DC>(a, p, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_latent_append(const LatentAppendArgs& a, hipStream_t s) {
  const int64_t n = int64_t(a.T) * ((a.dc + a.dr) / 8);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((n + 255) / 256, 16384));
  hipLaunchKernelGGL(latent_append_kernel, dim3(grid), dim3(256), 0, s, a, int64_t(grid) * 256);
  return hipGetLastError();
}

int64_t latent_grid(const TreeSizes& z, int32_t dc) { return token_groups(latent_plan(z), z, dc); }

size_t latent_ws_bytes(const TreeSizes& z, int32_t dc) { return parts_bytes(latent_plan(z), z, dc); }

hipError_t launch_latent(int dc, const TreeArgs& a, hipStream_t s) {
  const TreeSizes z{a.B, a.Hq, 1, a.max_new, a.max_len};
  switch (dc) {
    case 256: return latent_d<256>(a, z, s);
    case 512: return latent_d<512>(a, z, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace damp
