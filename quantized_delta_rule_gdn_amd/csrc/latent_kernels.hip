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
// workgroup holds in LDS serves both products of all its rows.
constexpr int kLatTile = 64;

// Up to 16 rows: the stream of the cache is what takes longest (64 requests, 266,000 tokens, 16 heads: 63 to 68 us and 6
// for the join; 5.2 TB/s behind the first 8 us, in which lengths, pages and the first tiles are on their way;
// the eight waves below take the same, and 17 instead of 16 us for one request of 700 tokens). The 4 waves
// share out the scores by tokens, meet for the maximum of each row, hand the weights over through LDS, and
// share out the readout by channels, so that a tile is read from LDS once (scores: as rows; readout:
// transposed on the way). The next tile is on its way in registers meanwhile. The weights go in two pieces, as for
// few rows of the other caches: that takes 1 to 4% of the call (these requests 68.4 -> 69.9 us, 250 of 200 tokens
// 20.6 -> 21.4), and without it values that cancel are off by 2^-8 of their size, not 2^-15.
template <int DC>
struct LatGeo {
  static constexpr int DR = DC / 8, W = DC + DR;     // channels of a row
  static constexpr int CH = W / 8;                   // 16-byte pieces of a row
  static constexpr int ROWS = kLatTile / 4;          // rows of a tile that a wave carries
  static constexpr int NR = ROWS / 8, PK = (CH + 7) / 8;   // by loads of 8 neighbouring pieces of 8 rows
  static constexpr int LD = W * 2 + 32;              // bytes between rows in LDS: an odd number of 32-byte units
};

template <int DC, bool P16>
__global__ __launch_bounds__(256, 2) void latent_kernel(const TreeArgs a, const TokenPlan plan) {
  using Geo = LatGeo<DC>;
  constexpr int W = Geo::W, KS = W / 32, CB = DC / 64;          // k steps; 16-channel blocks of a wave's share
  constexpr int LDP = kLatTile * 2 + 16;
  __shared__ __align__(16) uint8_t tile_k[kLatTile * Geo::LD];
  __shared__ __align__(16) uint8_t tile_p[2][16][LDP];              // the weights' two pieces
  __shared__ float part[4][16];
  __shared__ uint32_t tile_live[4], tile_odd[4];

  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const Spot spot = spot_of<kLatTile, DC>(a, plan);
  const int b = spot.b, split = spot.split, splits = spot.splits, H = a.Hq;
  if (b < 0) return;
  const Drafts dr = spot.dr;
  const int64_t rows = int64_t(min(dr.n, a.max_new)) * H, row0 = int64_t(spot.tile) * 16;
  if (row0 >= rows) return;
  const Parts<DC> parts(a, plan);
  const int len = spot.len;
  const int share = ((len + splits - 1) / splits + kLatTile - 1) / kLatTile * kLatTile;
  const int begin = min(split * share, len), end = min(begin + share, len);
  const int in_page = (1 << a.page_log2) - 1;
  const int live_rows = static_cast<int>(min(rows - row0, int64_t(16)));

  const unsigned my_row = static_cast<unsigned>(row0) + min(r, live_rows - 1);
  const int token = my_row / H;
  Frag qf[KS];
  {
    const int64_t at = int64_t(dr.first + token) * H + my_row % H;
#pragma unroll
    for (int x = 0; x < KS; ++x) qf[x] = load_frag(a.q + (at * W + g * 8 + x * 32) * 2);
  }
  f32x4 o[CB];
  float mx = -INFINITY, sum = 0.0f;
  bool taken_out = false;            // values that are not finite (the same for all waves)
#pragma unroll
  for (int m = 0; m < CB; ++m) o[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

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
    for (int w = 0; w < 4; ++w) odd_tile |= tile_odd[w];
    // scores^T [token][row] of 16 tokens: lane column = row, tokens 4 g .. + 3
    float p[4];
    {
      f32x4 s[2] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};   // (two sums: each product waits for the one before it)
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        const Frag kf = load_frag(tile_k + (16 * wv + r) * Geo::LD + g * 16 + x * 64);
        s[x & 1] = mfma(kf, qf[x], s[x & 1]);
        if (x % 6 == 5) __builtin_amdgcn_sched_barrier(0);   // (all operands loaded ahead would not fit the registers)
      }
      const uint32_t live = __builtin_amdgcn_readfirstlane(tile_live[wv]);
      const int first = t0 + 16 * wv;
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = (s[0][i] + s[1][i]) * a.scale_log2;
      if (live != 0xffffu || first + 16 > dr.base) {
        uint32_t seen = live;
        if (first + 16 > dr.base) seen &= seen_window(a, dr, token, first - dr.base);
        seen = rarely(seen);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!(seen >> (4 * g + i) & 1)) p[i] = -INFINITY;
      }
    }
    {
      const float top = max_row_slots(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])));
      if (g == 0) part[wv][r] = top;
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
    {
      const float top = fmaxf(fmaxf(fmaxf(mx, part[0][r]), fmaxf(part[1][r], part[2][r])), part[3][r]);
      if (__any(top > mx)) {
        const float shrink = top == -INFINITY ? 1.0f : pow2(mx - top);
        mx = top;
        sum *= shrink;
#pragma unroll
        for (int m = 0; m < CB; ++m) o[m] *= shrink;
      }
      const float base = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = pow2(p[i] - base);
      uint2 upper, rest;
      split_pair(p[0], p[1], upper.x, rest.x, sum);
      split_pair(p[2], p[3], upper.y, rest.y, sum);
      *reinterpret_cast<uint2*>(&tile_p[0][r][(16 * wv + 4 * g) * 2]) = upper;
      *reinterpret_cast<uint2*>(&tile_p[1][r][(16 * wv + 4 * g) * 2]) = rest;
    }
    __syncthreads();
    // readout^T [channel][row] += V^T P^T, this wave's channels
#pragma unroll
    for (int step = 0; step < kLatTile / 32; ++step) {
      const Frag pf[2] = {load_frag(&tile_p[0][r][(32 * step + 8 * g) * 2]), load_frag(&tile_p[1][r][(32 * step + 8 * g) * 2])};
      const uint8_t* v = tile_k + (32 * step + 8 * g + (r >> 2)) * Geo::LD + (wv * (DC / 4) + 4 * (r & 3)) * 2;
#pragma unroll
      for (int m = 0; m < CB; ++m) {
        const Frag vf = load_frag_t(reinterpret_cast<const uint16_t*>(v + 32 * m), reinterpret_cast<const uint16_t*>(v + 32 * m + 4 * Geo::LD));
#pragma unroll
        for (int x = 0; x < 2; ++x) o[m] = mfma(vf, pf[x], o[m]);
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
      const bool seen = t < dr.base || (seen_window(a, dr, token, t - dr.base) & 1);
#pragma unroll
      for (int m = 0; m < CB; ++m) o[m] = add_odd(o[m], *reinterpret_cast<const uint2*>(v + 32 * m), seen);
    }
  }

  // the rows' sums over all tokens
  __syncthreads();
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  if (g == 0) part[wv][r] = sum;
  __syncthreads();
  if (r >= live_rows) return;
  const float l = (part[0][r] + part[1][r]) + (part[2][r] + part[3][r]);
  const int ch = wv * (DC / 4) + 4 * g;
  if (splits == 1) {
    const int64_t at = (int64_t(dr.first + token) * H + my_row % H) * DC + ch;
    const float back = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int m = 0; m < CB; ++m)
      *reinterpret_cast<uint2*>(a.out + (at + 16 * m) * 2) = make_uint2(pack_bf16(o[m][0] * back, o[m][1] * back), pack_bf16(o[m][2] * back, o[m][3] * back));
  } else {
    const int64_t at = int64_t(spot.at) * plan.heads + r;
#pragma unroll
    for (int m = 0; m < CB; ++m) *reinterpret_cast<f32x4*>(parts.o + at * DC + ch + 16 * m) = o[m];
    if (wv == 0 && g == 0) parts.ml[at] = make_float2(mx, l);
  }
}

// More than 16 rows: the products take longer than the stream, so the two are given to different waves and
// run at the same time. Four waves score a tile, half of its tokens and half of the rows each, while the
// other four weigh the tile before it, a quarter of the channels each and all rows: every SIMD holds one of
// either kind. Tiles of 32 tokens are loaded into four buffers in LDS by the weighing waves, two tiles ahead;
// one barrier a tile. The rows' references (what their weights are relative to) stay as they are until a
// score passes one by 2^kSlack, as it does in a run's first tile: then, two more barriers are met, in which
// the scoring waves agree on new ones.
// 24 requests of up to 4,096 tokens with up to 4 drafted and 128 heads: 66 to 69 us and 9 for the join (85 with tiles
// carried through registers, stored to LDS between two barriers), 520 TFLOP/s. A tile of 32 tokens takes some 2,400
// cycles: 1,088 of products on each SIMD, 850 for its loads to go out (36 KB through a path of 64 bytes a cycle),
// the rest exponentials, looking what is rare and the barrier; the loads among the products slowed both (72 us),
// behind them too (83).
template <int DC, int R>
struct LatWide {
  static constexpr int DR = DC / 8, W = DC + DR, CH = W / 8;     // channels of a row, its 16-byte pieces
  static constexpr int TILE = 32, LD = W * 2, KS = W / 32, CB = DC / 64;
  static constexpr int NL = (8 * CH + 63) / 64;      // loads of 8 rows
  static constexpr int LDP = TILE * 2 + 16;
  static constexpr int RW = R / 2;                   // blocks of 16 rows that a wave scores
  // Rows are a multiple of 64 (128) bytes and half of that: piece p of row t lies at p ^ turn(t), with which
  // neither reads of whole rows nor transposed ones conflict (see row_turn for what they touch at once).
  __device__ static int turn(int t) { return DC == 512 ? (t & 6) ^ (t >> 3 & 1) * 5 : (t >> 1 & 2) ^ (t >> 3 & 1) * 3; }
};

template <int DC, int R, bool P16>
__global__ __launch_bounds__(512, 2) void latent_wide_kernel(const TreeArgs a, const TokenPlan plan) {
  using L = LatWide<DC, R>;
  constexpr int W = L::W, KS = L::KS, CB = L::CB, TILE = L::TILE, LD = L::LD, NL = L::NL, RW = L::RW;
  // (each buffer is an array of its own, so that reads of one need not keep their order with loads into another)
  __shared__ __align__(1024) uint8_t t0_[TILE * LD], t1_[TILE * LD], t2_[TILE * LD], t3_[TILE * LD];
  __shared__ __align__(16) uint8_t tile_p[2][16 * R][L::LDP];    // token 16 x + 4 y + z of the tile at 8 y + 4 x + z
  __shared__ float want[2][16 * R];                  // references that the waves would take; in the end their sums
  __shared__ float row_m[16 * R];                    // by what the readouts shrink; in the end the references
  __shared__ __align__(16) uint32_t tile_live[4][4];               // which rows exist: of a buffer, 8 for each wave that loads
  __shared__ int raised[2];                          // the tile (of every other one) for which references were raised
  __shared__ int any_odd;                            // values that are not finite have been taken out

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
  const int tiles = (end - begin + TILE - 1) / TILE;
  const int in_page = (1 << a.page_log2) - 1;
  const int live_rows = static_cast<int>(min(rows - row0, int64_t(16 * R)));
  if (tid == 0) {
    raised[0] = raised[1] = -1;
    any_odd = 0;
  }
  // What is rare before tile i is weighed: rows that do not exist become 0, values that are not finite, which some
  // token may not see, are taken out (the scores have been taken), and the references are raised. `agree` is
  // the scoring waves' part of that.
  struct Rare {
    int last;
    uint32_t live;
  };
  const auto look = [&](int i, int buf) -> Rare {
    const uint4 lives = *reinterpret_cast<const uint4*>(tile_live[buf]);
    return Rare{raised[i & 1], lives.x & lives.y & lives.z & lives.w};
  };
  const auto before_weighing = [&](int i, Rare rare, int buf, uint8_t* tile, auto&& publish, auto&& agree) -> bool {
    const int last = rare.last;
    const uint32_t live = rare.live;
    const bool up = __builtin_amdgcn_readfirstlane(last) == i;
    const bool drafted = begin + (i + 1) * TILE > dr.base;
    const bool clean = drafted || __builtin_amdgcn_readfirstlane(live) != 0xffu;
    if (!up && !clean) return false;
    if (up) publish();
    if (clean) {
      uint32_t odd = 0;
#pragma unroll 1
      for (int x = tid; x < TILE * L::CH; x += 512) {
        const int row = x / L::CH;
        u32x4* at = reinterpret_cast<u32x4*>(tile + x * 16);
        u32x4 v = *at;
        v &= tile_live[buf][row >> 3] >> (row & 7) & 1 ? ~0u : 0u;
        if (drafted) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            odd |= not_finite(v[k]);
            v[k] = finite_only(v[k]);
          }
        }
        *at = v;
      }
      if (__any(odd != 0) && lane == 0) any_odd = 1;
    }
    __syncthreads();
    if (up) {
      agree();
      __syncthreads();
    }
    return up;
  };

  if (wv < 4) {
    const int wt = wv & 1, row_w = (wv >> 1) * 16 * RW;          // this wave's tokens and rows
    const bool mine = row_w < live_rows;             // (in the last row tile some waves have none)
    int token[RW];
    Frag qf[RW][KS];
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      const unsigned my_row = static_cast<unsigned>(row0) + min(row_w + 16 * j + r, live_rows - 1);
      token[j] = my_row / H;
      const int64_t at = int64_t(dr.first + token[j]) * H + my_row % H;
#pragma unroll
      for (int x = 0; x < KS; ++x) qf[j][x] = load_frag(a.q + (at * W + g * 8 + x * 32) * 2);
    }
    float ref[RW], sum[RW], fresh[RW], top[RW];
    uint32_t w[RW][2];                               // weights of the tile scored last, tokens 16 wt + 4 g .. + 3
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      ref[j] = top[j] = -INFINITY;
      sum[j] = fresh[j] = 0.0f;
      w[j][0] = w[j][1] = 0;
    }
    const int row_at = (16 * wt + r) * LD, turn = L::turn(r);
    const auto put = [&](int i) {
#pragma unroll
      for (int j = 0; j < RW; ++j) *reinterpret_cast<uint2*>(&tile_p[i & 1][row_w + 16 * j + r][(8 * g + 4 * wt) * 2]) = make_uint2(w[j][0], w[j][1]);
    };
    const auto score = [&](int i, int buf, const uint8_t* tile) {
      constexpr int CHAINS = RW == 1 ? 2 : 1;        // (each product waits for the one before it)
      f32x4 s[RW][CHAINS];
#pragma unroll
      for (int j = 0; j < RW; ++j)
#pragma unroll
        for (int c = 0; c < CHAINS; ++c) s[j][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        const Frag kf = load_frag(tile + row_at + ((4 * x + g) ^ turn) * 16);
#pragma unroll
        for (int j = 0; j < RW; ++j) s[j][x % CHAINS] = mfma(kf, qf[j][x], s[j][x % CHAINS]);
      }
      // operands five steps ahead
      __builtin_amdgcn_sched_group_barrier(0x100, 5, 0);
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        __builtin_amdgcn_sched_group_barrier(0x008, RW, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
      const int first = begin + i * TILE + 16 * wt;
      const uint32_t live = __builtin_amdgcn_readfirstlane(tile_live[buf][2 * wt] | tile_live[buf][2 * wt + 1] << 8);
      float p[RW][4];
      bool over = false;
#pragma unroll
      for (int j = 0; j < RW; ++j) {
#pragma unroll
        for (int k = 0; k < 4; ++k) p[j][k] = (CHAINS == 2 ? s[j][0][k] + s[j][CHAINS - 1][k] : s[j][0][k]) * a.scale_log2;
        if (live != 0xffffu || first + 16 > dr.base) {
          uint32_t seen = live;
          if (first + 16 > dr.base) seen &= seen_window(a, dr, token[j], first - dr.base);
          seen = rarely(seen >> (4 * g));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (!(seen >> k & 1)) p[j][k] = -INFINITY;
        }
        top[j] = fmaxf(fmaxf(p[j][0], p[j][1]), fmaxf(p[j][2], p[j][3]));
        over |= top[j] > ref[j] + kSlack;
      }
      if (__any(over)) {
        // (whole numbers: what references differ by scales a weight exactly)
#pragma unroll
        for (int j = 0; j < RW; ++j) {
          top[j] = max_row_slots(top[j]);
          top[j] = top[j] > ref[j] + kSlack ? ceilf(top[j]) : ref[j];
        }
        if (lane == 0) raised[i & 1] = i;
      } else {
#pragma unroll
        for (int j = 0; j < RW; ++j) top[j] = ref[j];
      }
#pragma unroll
      for (int j = 0; j < RW; ++j) {
        const float base = top[j] == -INFINITY ? 0.0f : top[j];
        fresh[j] = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k) w[j][k] = round_pair(pow2(p[j][2 * k] - base), pow2(p[j][2 * k + 1] - base), fresh[j]);
      }
      put(i);
    };
    const auto publish = [&]() {
      if (g == 0) {
#pragma unroll
        for (int j = 0; j < RW; ++j) want[wt][row_w + 16 * j + r] = top[j];
      }
    };
    const auto step = [&](int i, int buf, uint8_t* tile, const uint8_t* next) {
      if (i >= tiles) return;
      before_weighing(i, look(i, buf), buf, tile, publish, [&]() {
#pragma unroll
        for (int j = 0; j < RW; ++j) {
          const int row = row_w + 16 * j + r;
          const float both = fmaxf(want[0][row], want[1][row]);
          const float f = top[j] == -INFINITY ? 1.0f : pow2(top[j] - both);
          fresh[j] *= f;
#pragma unroll
          for (int k = 0; k < 2; ++k) w[j][k] = pack_bf16(bf16_lo(w[j][k]) * f, bf16_hi(w[j][k]) * f);
          const float shrink = both == -INFINITY ? 1.0f : pow2(ref[j] - both);
          ref[j] = both;
          sum[j] *= shrink;
          if (wt == 0 && g == 0) row_m[row] = shrink;
        }
        put(i);
      });
#pragma unroll
      for (int j = 0; j < RW; ++j) sum[j] += fresh[j];
      if (mine && i + 1 < tiles) score(i + 1, (buf + 1) & 3, next);
      __syncthreads();
    };
    __syncthreads();                   // the first tile
    if (mine && tiles > 0) score(0, 0, t0_);
    __syncthreads();
    for (int i = 0; i < tiles; i += 4) {
      step(i, 0, t0_, t1_);
      step(i + 1, 1, t1_, t2_);
      step(i + 2, 2, t2_, t3_);
      step(i + 3, 3, t3_, t0_);
    }
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      sum[j] += __shfl_xor(sum[j], 16);
      sum[j] += __shfl_xor(sum[j], 32);
      if (g == 0) {
        want[wt][row_w + 16 * j + r] = sum[j];
        if (wt == 0) row_m[row_w + 16 * j + r] = ref[j];
      }
    }
    __syncthreads();
    return;
  }

  // Each weighing wave loads 8 rows of a tile. Their pages are looked up one tile ahead of their loads.
  const int wl = wv - 4, first_ch = wl * (DC / 4);
  uint32_t off[NL];
  int row_of[NL];
#pragma unroll
  for (int n = 0; n < NL; ++n) {
    const int x = min(64 * n + lane, 8 * L::CH - 1), row = x / L::CH;
    row_of[n] = row;
    off[n] = (P16 ? row * LD : 0) + ((x % L::CH) ^ L::turn(8 * wl + row)) * 16;
  }
  const int* table = a.table + int64_t(b) * a.max_blocks;
  const auto page_of = [&](int i) -> int {
    const int pos = min(begin + i * TILE + 8 * wl + (P16 ? 0 : lane & 7), end - 1);
    return table[pos >> a.page_log2];
  };
  const auto load = [&](int i, int pid, int buf, uint8_t* tile) {
    const int first = begin + i * TILE + 8 * wl, left = min(max(end - first, 0), 8);
    uint32_t live;
    int64_t at = 0;
    uint32_t own = 0;
    if constexpr (P16) {
      const int id = __builtin_amdgcn_readfirstlane(pid);
      const bool fine = id >= 0 && id < a.num_pages && left > 0;
      live = fine ? (1u << left) - 1 : 0;
      // (rows past the end lie in the same page; where there is no page, the first one's rows stand in)
      at = fine ? (int64_t(id) << a.page_log2) + (first & in_page) : 0;
    } else {
      const bool fine = pid >= 0 && pid < a.num_pages && (lane & 7) < left;
      live = static_cast<uint32_t>(__ballot(fine)) & 0xffu;
      own = fine ? (static_cast<uint32_t>(pid) << a.page_log2) + ((first + (lane & 7)) & in_page) : 0;
    }
#pragma unroll
    for (int n = 0; n < NL; ++n) {
      if constexpr (!P16) at = static_cast<uint32_t>(__shfl(static_cast<int>(own), row_of[n]));
      const uint8_t* src = a.k_pages + at * LD + off[n];
      uint8_t* to = tile + 8 * wl * LD + n * 1024;
      if (64 * n + 63 < 8 * L::CH || 64 * n + lane < 8 * L::CH) load_to_lds(src, to);
    }
    if (lane == 0) tile_live[buf][wl] = live;
  };
  f32x4 o[R][CB];
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int m = 0; m < CB; ++m) o[j][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  int pid = 0;
  // (tiles past the end load rows that exist: as many loads are on their way as landed() counts)
  if (tiles > 0) {
    const int p0 = page_of(0), p1 = page_of(1), p2 = page_of(2);
    pid = page_of(3);
    load(0, p0, 0, t0_);
    load(1, p1, 1, t1_);
    load(2, p2, 2, t2_);
    landed<2 * NL>();
  }
  __syncthreads();
  landed<NL>();
  __syncthreads();
  const auto step = [&](int i, int buf, uint8_t* tile, uint8_t* free) {
    if (i >= tiles) return;
    const Rare rare = look(i, buf);
    const int now = pid;
    pid = page_of(i + 4);
    load(i + 3, now, (buf + 3) & 3, free);
    if (before_weighing(i, rare, buf, tile, []() {}, []() {})) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const float shrink = row_m[16 * j + r];
#pragma unroll
        for (int m = 0; m < CB; ++m) o[j][m] *= shrink;
      }
    }
    Frag pf[R];
#pragma unroll
    for (int j = 0; j < R; ++j) pf[j] = load_frag(&tile_p[i & 1][16 * j + r][8 * g * 2]);
    // (rows 4 g .. + 3 and 16 more, four by four lanes each; 16 channels of 32 bytes)
    const int row = 4 * g + (r >> 2), turn = L::turn(row), ch = first_ch / 8 + (r >> 1 & 1);
#pragma unroll
    for (int m = 0; m < CB; ++m) {
      const uint8_t* v = tile + row * LD + ((ch + 2 * m) ^ turn) * 16 + (r & 1) * 8;
      const Frag vf = load_frag_t(reinterpret_cast<const uint16_t*>(v), reinterpret_cast<const uint16_t*>(v + 16 * LD));
#pragma unroll
      for (int j = 0; j < R; ++j) o[j][m] = mfma(vf, pf[j], o[j][m]);
    }
    // operands three blocks ahead
    __builtin_amdgcn_sched_group_barrier(0x100, R + 6, 0);
#pragma unroll
    for (int m = 0; m < CB; ++m) {
      __builtin_amdgcn_sched_group_barrier(0x008, R, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
    landed<NL>();
    __syncthreads();
  };
  for (int i = 0; i < tiles; i += 4) {
    step(i, 0, t0_, t3_);
    step(i + 1, 1, t1_, t0_);
    step(i + 2, 2, t2_, t1_);
    step(i + 3, 3, t3_, t2_);
  }
  landed();                          // (nothing may be on its way into LDS that the next workgroup has)
  __syncthreads();                   // references and sums
  if (any_odd) {
    // (from the first tile with a drafted token on; what an earlier tile has already is added again, to no effect)
#pragma unroll 1
    for (int t = max(dr.base - TILE, begin); t < end; ++t) {
      const int page = table[t >> a.page_log2];
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
    const float l = want[0][16 * j + r] + want[1][16 * j + r];
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
      if (wl == 0 && g == 0) parts.ml[at] = make_float2(row_m[16 * j + r], l);
    }
  }
}

TokenPlan latent_plan(const TreeSizes& z) {
  const int64_t rows = int64_t(z.max_new) * z.Hq;
  const int log2 = rows <= 16 ? 4 : rows <= 32 ? 5 : 6;
  // Workgroups that LDS leaves room for on the 256 CUs: two of four waves each, or one of eight. 32 rows in tiles
  // of 64 take 73 us instead of 69 (64 requests of 4,000 tokens, 32 heads). Requests of up to 256 tokens are not cut:
  // 250 with 16 heads take 15.5 us whole and 13.7 cut, with d_latent = 256 10.3 and 13.3, 16 of them with 128 heads
  // 22 and 29; 400 take 22.5 whole and 14.2 cut.
  return token_plan(z, log2, log2 == 4 ? 512 : 256, 256);
}

template <int DC, bool P16>
void latent_dp(const TreeArgs& a, const TokenPlan& p, hipStream_t s) {
  const dim3 grid(p.groups);
  if (p.rows_log2 == 4) hipLaunchKernelGGL((latent_kernel<DC, P16>), grid, dim3(256), 0, s, a, p);
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

// (in workgroups of 256 threads: those of more than 16 rows have twice as many)
int64_t latent_grid(const TreeSizes& z) {
  const TokenPlan p = latent_plan(z);
  return p.rows_log2 > 4 ? int64_t(2) * p.groups : p.groups;
}

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
