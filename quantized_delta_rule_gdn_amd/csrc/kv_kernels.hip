// kv_kernels.hip -- gfx950 kernels of the paged key-value cache that a hybrid model's
// full-attention layers keep beside the recurrent states: block tables and slot maps from the
// requests' lengths, the store of new keys and values, and attention of one new token per request.
#include <algorithm>

#include "attn_plan.h"

namespace damp {
namespace {

// ---- block tables and slot maps --------------------------------------------------------------
// One launch and no workspace: every workgroup scans the B lengths for itself (they are a few KB,
// in L2 after the first) and then fills its share of the tokens and of the new table entries,
// finding a token's request by bisection in LDS. What bounds it is the launch and the scan's
// latency; the outputs are 12 bytes a token. 48 requests of one token 4.7 us, 300 of 32,000 in all 9.1 us.
constexpr int kTabThreads = 512;
constexpr int kTabMaxB = 8000;   // two sums of 4 bytes each in LDS

struct Request {
  int old, have, need;   // tokens before this call, pages they fill, pages to add
  int fresh;             // tokens of this call
};

__device__ __forceinline__ Request request_of(const TableArgs& a, int b) {
  const int page = 1 << a.page_log2;
  const int len = max(a.seq_lens[b], 0), fresh = min(max(a.new_lens[b], 0), len);
  const int old = len - fresh;
  const auto pages = [&](int n) { return min((n >> a.page_log2) + ((n & (page - 1)) != 0), a.max_blocks); };
  const int have = pages(old);
  return Request{old, have, pages(len) - have, fresh};
}

// The last b with first[b] <= x (first is ascending and first[0] = 0).
__device__ __forceinline__ int owner_of(const int* first, int B, int x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(kTabThreads) void kv_tables_kernel(const TableArgs a) {
  extern __shared__ int lds[];               // tok[B], pg[B]: exclusive sums of new tokens and pages
  __shared__ int2 wave_sum[kTabThreads / 64];
  __shared__ int2 carry;
  int* tok = lds;
  int* pg = lds + a.B;
  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63, wv = tid >> 6;
  if (tid == 0) carry = make_int2(0, 0);
  for (int b0 = 0; b0 < a.B; b0 += kTabThreads) {
    const int b = b0 + tid;
    int2 own = make_int2(0, 0);
    if (b < a.B) {
      const Request r = request_of(a, b);
      own = make_int2(r.fresh, r.need);
    }
    int2 incl = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int x = __shfl_up(incl.x, o), y = __shfl_up(incl.y, o);
      if (lane >= o) incl = make_int2(incl.x + x, incl.y + y);
    }
    if (lane == 63) wave_sum[wv] = incl;
    __syncthreads();
    int2 base = carry;
    for (int i = 0; i < wv; ++i) base = make_int2(base.x + wave_sum[i].x, base.y + wave_sum[i].y);
    if (b < a.B) {
      tok[b] = base.x + incl.x - own.x;
      pg[b] = base.y + incl.y - own.y;
    }
    __syncthreads();
    if (tid == kTabThreads - 1) carry = make_int2(base.x + incl.x, base.y + incl.y);
  }
  __syncthreads();
  const int tokens = carry.x, pages = carry.y;
  const int first = __builtin_amdgcn_workgroup_id_x() * kTabThreads + tid, step = __builtin_amdgcn_grid_size_x();
  for (int b = first; b <= a.B; b += step) a.cu_new[b] = b < a.B ? tok[b] : tokens;
  if (first == 0) a.used[0] = pages;
  for (int64_t p = first; p < pages; p += step) {
    const int b = owner_of(pg, a.B, static_cast<int>(p));
    const int j = request_of(a, b).have + static_cast<int>(p) - pg[b];
    if (j >= 0 && j < a.max_blocks) a.table[int64_t(b) * a.max_blocks + j] = p < a.num_free ? a.free_pages[p] : -1;
  }
  // a token's page comes from the table where the request had it before and from the free list
  // where this call adds it, so no entry that another thread writes is read
  for (int64_t t = first; t < a.T; t += step) {
    int64_t slot = -1;
    int pos = -1;
    if (t < tokens) {
      const int b = owner_of(tok, a.B, static_cast<int>(t));
      const Request r = request_of(a, b);
      pos = r.old + static_cast<int>(t) - tok[b];
      const int j = pos >> a.page_log2;
      int id = -1;
      if (j >= 0 && j < r.have) id = a.table[int64_t(b) * a.max_blocks + j];
      else if (j >= r.have && j < r.have + r.need) {
        const int p = pg[b] + j - r.have;
        if (p >= 0 && p < a.num_free) id = a.free_pages[p];
      }
      if (id >= 0) slot = (int64_t(id) << a.page_log2) + (pos & ((1 << a.page_log2) - 1));
    }
    a.slot_map[t] = slot;
    if (a.positions) a.positions[t] = pos;
  }
}

// ---- the store of new keys and values ----------------------------------------------------------
// A copy by slot map, 16 bytes a thread: bound by the stream of 8 Hkv d bytes per token. 32,000 tokens
// of 8 heads, d = 128: 51 us for 262 MB, 5.2 TB/s.
__global__ __launch_bounds__(256) void kv_append_kernel(const AppendArgs a) {
  const int per_row = a.d / 8, per_tok = a.Hkv * per_row;
  const int64_t n = int64_t(a.T) * per_tok;
  const int64_t first = int64_t(__builtin_amdgcn_workgroup_id_x()) * 256 + __builtin_amdgcn_workitem_id_x();
  const int64_t step = __builtin_amdgcn_grid_size_x();
  for (int64_t x = first; x < n; x += step) {
    const int64_t t = x / per_tok;
    const int c = static_cast<int>(x - t * per_tok);
    const int64_t slot = a.slot_map[t];
    if (slot < 0 || slot >= a.num_slots) continue;
    const int h = c / per_row, piece = c - h * per_row;
    const int64_t row = (((slot >> a.page_log2) * a.Hkv + h) << a.page_log2) + (slot & ((1 << a.page_log2) - 1));
    const int64_t dst = row * per_row + piece;
    reinterpret_cast<uint4*>(a.k_pages)[dst] = reinterpret_cast<const uint4*>(a.k)[x];
    reinterpret_cast<uint4*>(a.v_pages)[dst] = reinterpret_cast<const uint4*>(a.v)[x];
  }
}

// ---- attention of one new token ------------------------------------------------------------------
// o = sum_t p_t v_t / sum_t p_t, p_t = exp(scale q.k_t - m), in one pass over the cache with a
// running maximum m and sum. A request's tokens are cut into items, one workgroup per (item,
// key-value head, 16 query heads), joined by a second kernel; each of the 4 waves takes every
// fourth tile of 32 tokens and the waves meet in LDS at the end. It is bound by the stream
// of the cache's bytes (4 Hkv d per token): the matrix instructions serve up to 16 query heads of
// one key-value head for the same bytes. Nothing is staged in LDS on the way:
//   scores^T [token][head] = K Q^T: a lane's operand is 16 bytes of one token's key as stored;
//   the scores' C tile is the B operand of out^T [d][head] = V^T P^T as it stands (k permuted:
//   lane group g holds tokens 4 g .. + 3 of both 16-token halves), so V^T's operand takes those
//   tokens: each lane loads D / 16 neighbouring channels of 8 tokens (whole rows per 16 lanes)
//   and transposes them with byte permutes; output channel D / 16 * row + m is tile m's row.
// A weight p enters the second product as two bf16 pieces, the upper 16 bits of p (1 - 2^-12) and the rest
// rounded, good to 2^-15 + 2^-20 of p. (One rounded piece is off by up to 2^-8, and tokens of equal
// scores all the same way: a few tokens at the maximum and all others at p = 0.50195 over a V of ones gave
// 0.996. Nor does it average below the readout's own rounding: 8,192 random scores gave an error
// 7% above that rounding's. The second piece takes no time where the stream is long, 208.5 us for the batch
// below with either, and 0.3 of 10.7 us for one request of 700 tokens: the matrix instructions are 5% busy.)
// Scores, m, the sum and the accumulators are binary32.
// 64 requests of up to 8,192 tokens (266,000 in all), 32 query heads on 8, d = 128: 200 us for 1.09 GB,
// 5.4 TB/s (reading alone reaches 7.1); 5 of up to 65,536, 32 on 4, d = 64: 36 us for 201 MB, 5.6 TB/s.
// Short requests are not cut at all: the join's launch, and an item's way in and out, cost more than
// the cutting saves. One MI355X, d = 128, 32 query heads on 8, on the device: 64 requests of up to 512
// tokens 16 us whole, 27 us cut; of up to 1,024 23 against 30; of up to 2,048 32 against 38. One of 704
// 9.7 against 10.6, of 1,024 12.1 against 10.1 (but 12 against 15 with the call), of 1,536 17 against
// 11: past 1,024 only where the requests fill the chip twice over.
bool uncut(int64_t groups, int32_t max_len) { return max_len <= 1024 || (max_len <= 2048 && groups >= 512); }

AttnPlan attn_plan(int32_t B, int32_t Hq, int32_t Hkv, int32_t max_len) {
  AttnPlan p;
  p.tiles = (Hq / Hkv + 15) / 16;
  p.heads = std::min(Hq / Hkv, 16);
  // 4 workgroups a CU, though 3 are resident at d = 128 (by registers) and 5 at 64: the load evens out.
  // 64 ragged requests from HBM, d = 128, 32 query heads on 8: 232-237 us against 237-244 with 2 a CU,
  // both after 1 GB of other traffic. (Where the pages lie in the on-chip caches fewer, longer items
  // win: 5 requests of 40,000 tokens, d = 64, 43 us against 37.)
  const int64_t units = int64_t(Hkv) * p.tiles, wanted = 256 * 4;
  const int64_t most = (int64_t(max_len) + kAttnLeast - 1) / kAttnLeast * B;   // no more are ever cut
  p.per_unit = static_cast<int>(std::min<int64_t>(std::max<int64_t>(wanted / units, 1), std::max<int64_t>(most, 1)));
  p.items = uncut(units * B, max_len) ? B : p.per_unit + B;
  return p;
}

constexpr int kAttnPages = 1024;   // page addresses held in LDS at a time

// P16: pages of 16 tokens or more, so that a half tile lies in one page and its address is the same
// for the whole wave; smaller pages are looked up for every row.
template <int D, bool P16>
__global__ __launch_bounds__(256, 2) void kv_attention_kernel(const AttnArgs a, const AttnPlan plan) {
  constexpr int KS = D / 32;       // k steps of the score product
  constexpr int DPL = D / 16;      // value channels per lane
  constexpr int VW = DPL / 2;      // dwords of them
  constexpr uint32_t kNone = 0xffffffffu;
  __shared__ uint32_t first_row[kAttnPages];          // of a page, in rows of this key-value head
  __shared__ int64_t sh[8];
  __shared__ float part_m[4][16], part_l[4][16];
  __shared__ __align__(16) float part_o[4][16][D + 4];

  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const unsigned id = __builtin_amdgcn_workgroup_id_x();
  const int units = a.Hkv * plan.tiles;
  const int item = id / units, unit = id % units, tile = unit % plan.tiles, kvh = unit / plan.tiles;
  const int G = a.Hq / a.Hkv;

  // the request this item belongs to
  const Item it = item_of(a, plan, item, sh);
  const int b = it.b, split = it.split, splits = it.splits;
  if (b < 0) return;
  const int whole = a.seq_lens[b], len = length_of(a, b);
  // its tokens: an even share of the request's, in whole tiles
  const int share = ((len + splits - 1) / splits + kAttnTile - 1) / kAttnTile * kAttnTile;
  const int begin = min(split * share, len), end = min(begin + share, len);
  const int in_page = (1 << a.page_log2) - 1;

  const int head0 = tile * 16, heads = min(16, G - head0);
  Frag qf[KS];
  {
    const uint8_t* qp = a.q + ((int64_t(b) * a.Hq + kvh * G + head0 + min(r, heads - 1)) * D + g * 8) * 2;
#pragma unroll
    for (int x = 0; x < KS; ++x) qf[x] = load_frag(qp + x * 64);
  }

  f32x4 o[DPL];
#pragma unroll
  for (int m = 0; m < DPL; ++m) o[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float mx = -INFINITY, sum = 0.0f;
  const uint32_t k_off = r * (D * 2) + g * 16;                  // a half tile's K rows as operands
  const uint32_t v_off = 4 * g * (D * 2) + r * (DPL * 2);       // and its V rows
  // page addresses for as many tokens at a time as LDS holds (4 tiles at least)
  constexpr int kRun = P16 ? kAttnPages * 16 : kAttnPages;
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
    // this call's key and value go into the cache first; the workgroup then reads them from there
    if (a.k_new && whole == len && to == len) {
      const int pos = len - 1;
      const uint32_t page = first_row[(pos >> a.page_log2) - p0];
      if (page != kNone && tid < D / 4) {
        const int64_t row = int64_t(page) + (pos & in_page);
        const int64_t src = int64_t(b) * a.Hkv + kvh;
        const int piece = tid % (D / 8);
        if (tid < D / 8) reinterpret_cast<uint4*>(a.k_pages)[row * (D / 8) + piece] = reinterpret_cast<const uint4*>(a.k_new)[src * (D / 8) + piece];
        else reinterpret_cast<uint4*>(a.v_pages)[row * (D / 8) + piece] = reinterpret_cast<const uint4*>(a.v_new)[src * (D / 8) + piece];
      }
      __syncthreads();
    }
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
      f32x4 s[2];
  #pragma unroll
      for (int h = 0; h < 2; ++h) s[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  #pragma unroll
      for (int x = 0; x < KS; ++x)
  #pragma unroll
        for (int h = 0; h < 2; ++h) s[h] = mfma(kf[h][x], qf[x], s[h]);
      float p[8];
  #pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = s[i >> 2][i & 3] * a.scale_log2;
      if (__any(dead != 0) || t0 + kAttnTile > to) {
  #pragma unroll
        for (int i = 0; i < 8; ++i) {
          if ((dead >> i & 1) || t0 + 16 * (i >> 2) + 4 * g + (i & 3) >= to) {
            p[i] = -INFINITY;
  #pragma unroll
            for (int w = 0; w < VW; ++w) vr[i][w] = 0;   // whatever lies there: 0 * NaN is NaN
          }
        }
      }
      float top = mx;
  #pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, p[i]);
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      if (__any(top > mx)) {               // (the maximum settles after a few tiles)
        const float shrink = top == -INFINITY ? 1.0f : pow2(mx - top);
        mx = top;
        sum *= shrink;
  #pragma unroll
        for (int m = 0; m < DPL; ++m) o[m] *= shrink;
      }
      const float base = mx == -INFINITY ? 0.0f : mx;
      Frag pf[2];
  #pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = pow2(p[i] - base);
        sum += p[i];
      }
  #pragma unroll
      for (int j = 0; j < 4; ++j) {
        // (of a little less than x, so that the rest is never 0: times an infinite value that would be NaN)
        const float x0 = p[2 * j], x1 = p[2 * j + 1];
        const uint32_t w0 = __float_as_uint(x0 * 0x1.ffep-1f), w1 = __float_as_uint(x1 * 0x1.ffep-1f);
        pf[0].w[j] = __builtin_amdgcn_perm(w1, w0, 0x07060302u);
        pf[1].w[j] = pack_bf16(x0 - __uint_as_float(w0 & 0xffff0000u), x1 - __uint_as_float(w1 & 0xffff0000u));
      }
  #pragma unroll
      for (int m = 0; m < DPL; m += 2) {   // (each sum's two products apart)
        Frag vf[2];
  #pragma unroll
        for (int j = 0; j < 4; ++j) {
          vf[0].w[j] = __builtin_amdgcn_perm(vr[2 * j + 1][m / 2], vr[2 * j][m / 2], 0x05040100u);
          vf[1].w[j] = __builtin_amdgcn_perm(vr[2 * j + 1][m / 2], vr[2 * j][m / 2], 0x07060302u);
        }
  #pragma unroll
        for (int x = 0; x < 2; ++x) {
          o[m] = mfma(vf[0], pf[x], o[m]);
          o[m + 1] = mfma(vf[1], pf[x], o[m + 1]);
        }
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

  for (int x = tid; x < heads * D; x += 256) {
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
      const int64_t at = (int64_t(b) * a.Hq + kvh * G + head0 + h) * D + c;
      reinterpret_cast<uint16_t*>(a.out)[at] = float_to_bf16_bits(l == 0.0f ? 0.0f : acc / l);
    } else {
      const int64_t at = int64_t(id) * plan.heads + h;
      a.ws[at * D + c] = acc;
      if (c == 0) reinterpret_cast<float2*>(a.ws + int64_t(plan.items) * units * plan.heads * D)[at] = make_float2(m0, l);
    }
  }
}

// The items of one (request, query head) joined: sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s, 256
// items at a time: a thread takes one item's weight, then every channel's sum runs over the items
// in 256 / D interleaved parts (each in order, joined in order). What bounds it is the latency of its
// few loads: 5 to 9 us. A request that was not cut has its readout already.
template <int D>
__global__ __launch_bounds__(256) void kv_join_kernel(const AttnArgs a, const AttnPlan plan) {
  constexpr int P = 256 / D;
  __shared__ float f[256], part[P][D], top[4], low[4];
  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63, wv = tid >> 6;
  const int c = tid % D, part0 = tid / D;
  const int64_t unit = __builtin_amdgcn_workgroup_id_x();
  const int b = static_cast<int>(unit / a.Hq), hq = static_cast<int>(unit - int64_t(b) * a.Hq);
  __shared__ int64_t sh[4];
  const int chunk = chunk_of(a, plan, sh);
  const int n = items_of(length_of(a, b), chunk);
  if (n == 1) return;
  int64_t before = 0;
  const int apart = requests_step(a);
  for (int x = tid & (apart - 1); x < b; x += apart) before += items_of(length_of(a, x), chunk);
  before = requests_sum(a, before, sh);
  const int G = a.Hq / a.Hkv, units = a.Hkv * plan.tiles;
  const int64_t step = int64_t(units) * plan.heads;      // between a unit's items
  const int64_t first = (before * units + hq / G * plan.tiles + hq % G / 16) * plan.heads + hq % G % 16;
  const float* po = a.ws + first * D + c;
  const float2* ml = reinterpret_cast<const float2*>(a.ws + int64_t(plan.items) * step * D) + first;
  float m = -INFINITY, acc = 0.0f, l = 0.0f;
  for (int s0 = 0; s0 < n; s0 += 256) {
    const float2 x = s0 + tid < n ? ml[(s0 + tid) * step] : make_float2(-INFINITY, 0.0f);
    float t = x.x;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) t = fmaxf(t, __shfl_xor(t, o));
    __syncthreads();                     // the last round's reads are over
    if (lane == 0) top[wv] = t;
    __syncthreads();
    const float m0 = fmaxf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), m);
    const float base = m0 == -INFINITY ? 0.0f : m0;
    const float shrink = pow2(m - base), w = pow2(x.x - base);
    f[tid] = w;
    float sum = w * x.y;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o);
    if (lane == 0) low[wv] = sum;
    __syncthreads();
    l = fmaf(l, shrink, (low[0] + low[1]) + (low[2] + low[3]));
    acc *= shrink;
    m = m0;
    const int stop = min(256, n - s0);
    float more[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int s = part0;
    for (; s + 3 * P < stop; s += 4 * P)
#pragma unroll
      for (int i = 0; i < 4; ++i) more[i] = fmaf(f[s + i * P], po[(s0 + s + i * P) * step * D], more[i]);
    for (; s < stop; s += P) more[0] = fmaf(f[s], po[(s0 + s) * step * D], more[0]);
    acc += (more[0] + more[1]) + (more[2] + more[3]);
  }
  part[part0][c] = acc;
  __syncthreads();
  if (tid < D) {
    float o = part[0][c];
#pragma unroll
    for (int i = 1; i < P; ++i) o += part[i][c];
    reinterpret_cast<uint16_t*>(a.out)[unit * D + c] = float_to_bf16_bits(l == 0.0f ? 0.0f : o / l);
  }
}

template <int D>
hipError_t attention_d(const AttnArgs& a, hipStream_t s) {
  const AttnPlan p = attn_plan(a.B, a.Hq, a.Hkv, a.max_len);
  const dim3 grid(static_cast<unsigned>(p.items) * a.Hkv * p.tiles);
  if (a.page_log2 >= 4) hipLaunchKernelGGL((kv_attention_kernel<D, true>), grid, dim3(256), 0, s, a, p);
  else hipLaunchKernelGGL((kv_attention_kernel<D, false>), grid, dim3(256), 0, s, a, p);
  if (p.items > a.B)
    hipLaunchKernelGGL((kv_join_kernel<D>), dim3(static_cast<unsigned>(a.B) * static_cast<unsigned>(a.Hq)), dim3(256), 0, s, a, p);
  return hipGetLastError();
}

}  // namespace

int kv_tables_max_requests() { return kTabMaxB; }

hipError_t launch_kv_tables(const TableArgs& a, hipStream_t s) {
  const int64_t most = std::max<int64_t>(a.T, a.B);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(std::max<int64_t>((most + kTabThreads - 1) / kTabThreads, 1), 256));
  hipLaunchKernelGGL(kv_tables_kernel, dim3(grid), dim3(kTabThreads), static_cast<size_t>(a.B) * 8, s, a);
  return hipGetLastError();
}

hipError_t launch_kv_append(const AppendArgs& a, hipStream_t s) {
  const int64_t n = int64_t(a.T) * a.Hkv * (a.d / 8);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((n + 255) / 256, 16384));
  hipLaunchKernelGGL(kv_append_kernel, dim3(grid), dim3(256), 0, s, a);
  return hipGetLastError();
}

int64_t kv_attention_grid(int32_t B, int32_t Hq, int32_t Hkv, int32_t max_len) {
  const AttnPlan p = attn_plan(B, Hq, Hkv, max_len);
  return (int64_t(p.per_unit) + B) * Hkv * p.tiles;
}

size_t kv_attention_ws_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int32_t max_len) {
  const AttnPlan p = attn_plan(B, Hq, Hkv, max_len);
  if (p.items == B) return 0;
  return static_cast<size_t>(p.items) * Hkv * p.tiles * p.heads * (static_cast<size_t>(d) + 2) * 4;
}

hipError_t launch_kv_attention(int d, const AttnArgs& a, hipStream_t s) {
  switch (d) {
    case 64: return attention_d<64>(a, s);
    case 128: return attention_d<128>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace damp
