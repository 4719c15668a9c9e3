// kv_kernels.hip -- gfx950 kernels of the paged key-value cache that a hybrid model's
// full-attention layers keep beside the recurrent states: block tables and slot maps from the
// requests' lengths, the store of new keys and values, and attention of one new token per request.
#include <algorithm>

#include "prompt_common.h"

namespace damp {
namespace {

// ---- block tables and slot maps --------------------------------------------------------------
// One launch and no workspace: every workgroup scans the B lengths for itself (they are a few KB,
// in L2 after the first) and then fills its share of the tokens and of the new table entries,
// finding a token's request by bisection in LDS. What bounds it is the launch and the scan's
// latency; the outputs are 12 bytes a token.
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
  for (int p = first; p < pages; p += step) {
    const int b = owner_of(pg, a.B, p);
    const int j = request_of(a, b).have + p - pg[b];
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
      else if (j >= r.have && j < r.have + r.need && pg[b] + j - r.have < a.num_free) id = a.free_pages[pg[b] + j - r.have];
      if (id >= 0) slot = (int64_t(id) << a.page_log2) + (pos & ((1 << a.page_log2) - 1));
    }
    a.slot_map[t] = slot;
    if (a.positions) a.positions[t] = pos;
  }
}

// ---- the store of new keys and values ----------------------------------------------------------
// A copy by slot map, 16 bytes a thread: bound by the stream of 8 Hkv d bytes per token.
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
// running maximum m and sum. A request's tokens are cut into chunks, one workgroup per (request,
// key-value head, 16 query heads, chunk), joined by a second kernel; each of the 4 waves takes
// every fourth tile of 32 tokens and the waves meet in LDS at the end. It is bound by the stream
// of the cache's bytes (4 Hkv d per token): the matrix instructions serve up to 16 query heads of
// one key-value head for the same bytes. Nothing is staged in LDS on the way:
//   scores^T [token][head] = K Q^T: a lane's operand is 16 bytes of one token's key as stored;
//   the scores' C tile is the B operand of out^T [d][head] = V^T P^T as it stands (k permuted:
//   lane group g holds tokens 4 g .. + 3 of both 16-token halves), so V^T's operand takes those
//   tokens: each lane loads D / 16 neighbouring channels of 8 tokens (whole rows per 16 lanes)
//   and transposes them with byte permutes; output channel D / 16 * row + m is tile m's row.
// The weights p are rounded to bf16 for the second product (the relative error of 2^-9 each
// averages over the tokens and stays below the rounding of the bf16 output); scores, m, the sum
// and the accumulators are binary32.
constexpr int kAttnTile = 32;

struct AttnPlan {
  int tiles;    // groups of 16 query heads per key-value head
  int chunk;    // tokens per workgroup
  int splits;   // chunks of the longest request
};

AttnPlan attn_plan(int32_t B, int32_t Hq, int32_t Hkv, int32_t max_len) {
  AttnPlan p;
  p.tiles = (Hq / Hkv + 15) / 16;
  const int64_t units = int64_t(B) * Hkv * p.tiles;
  p.chunk = 128;
  while (p.chunk < 1024 && units * ((max_len + p.chunk - 1) / p.chunk) > 4096) p.chunk *= 2;
  p.splits = (max_len + p.chunk - 1) / p.chunk;
  if (p.splits < 1) p.splits = 1;
  return p;
}

constexpr int kAttnMaxChunk = 1024;

template <int D>
__global__ __launch_bounds__(256) void kv_attention_kernel(const AttnArgs a, const AttnPlan plan) {
  constexpr int KS = D / 32;       // k steps of the score product
  constexpr int DPL = D / 16;      // value channels per lane
  constexpr int VW = DPL / 2;      // dwords of them
  __shared__ int pages[kAttnMaxChunk + 1];
  __shared__ int bad;
  __shared__ float part_m[4][16], part_l[4][16];
  __shared__ __align__(16) float part_o[4][16][D + 4];

  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  unsigned id = __builtin_amdgcn_workgroup_id_x();
  const int split = id % plan.splits; id /= plan.splits;
  const int tile = id % plan.tiles; id /= plan.tiles;
  const int kvh = id % a.Hkv;
  const int b = id / a.Hkv;
  const int G = a.Hq / a.Hkv;
  const int whole = a.seq_lens[b];
  const int64_t cap = int64_t(a.max_blocks) << a.page_log2;
  const int len = static_cast<int>(min(int64_t(min(max(whole, 0), a.max_len)), cap));
  const int begin = split * plan.chunk;
  if (begin >= len && !(split == 0 && plan.splits == 1)) return;
  const int end = min(begin + plan.chunk, len);
  const int64_t page_rows = int64_t(1) << a.page_log2;

  const int p0 = begin >> a.page_log2;
  const int np = end > begin ? ((end - 1) >> a.page_log2) - p0 + 1 : 0;
  if (tid == 0) bad = 0;
  __syncthreads();
  for (int i = tid; i < np; i += 256) {
    const int pid = a.table[int64_t(b) * a.max_blocks + p0 + i];
    const bool fine = pid >= 0 && pid < a.num_pages;
    pages[i] = fine ? pid : -1;
    if (!fine) bad = 1;
  }
  __syncthreads();
  // this call's key and value go into the cache first; the workgroup then reads them from there
  if (a.k_new && whole > 0 && whole == len && end == len && end > begin) {
    const int pos = len - 1, pid = pages[(pos >> a.page_log2) - p0];
    if (pid >= 0 && tid < D / 4) {
      const int64_t row = (int64_t(pid) * a.Hkv + kvh) * page_rows + (pos & (page_rows - 1));
      const int64_t from = int64_t(b) * a.Hkv + kvh;
      const int piece = tid % (D / 8);
      if (tid < D / 8) reinterpret_cast<uint4*>(a.k_pages)[row * (D / 8) + piece] = reinterpret_cast<const uint4*>(a.k_new)[from * (D / 8) + piece];
      else reinterpret_cast<uint4*>(a.v_pages)[row * (D / 8) + piece] = reinterpret_cast<const uint4*>(a.v_new)[from * (D / 8) + piece];
    }
    __syncthreads();
  }
  const bool clean = bad == 0;

  const int head0 = tile * 16, heads = min(16, G - head0);
  Frag qf[KS];
  {
    const uint8_t* qp = a.q + ((int64_t(b) * a.Hq + kvh * G + head0 + min(r, heads - 1)) * D + g * 8) * 2;
#pragma unroll
    for (int x = 0; x < KS; ++x) qf[x] = load_frag(qp + x * 64);
  }
  const auto row_of = [&](int pos) -> int64_t {   // cache row of a position, -1 where there is none
    const int pid = pages[(pos >> a.page_log2) - p0];
    return pid < 0 ? -1 : (int64_t(pid) * a.Hkv + kvh) * page_rows + (pos & (page_rows - 1));
  };

  f32x4 o[DPL];
#pragma unroll
  for (int m = 0; m < DPL; ++m) o[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float mx = -INFINITY, sum = 0.0f;
  for (int t0 = begin + wv * kAttnTile; t0 < end; t0 += 4 * kAttnTile) {
    // (positions past the end read the last row; what they give is masked)
    Frag kf[2][KS];
    uint32_t vr[8][VW];
    uint32_t dead = 0;   // bit i: this lane's value row i is not part of the request
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t row = max(row_of(min(t0 + 16 * h + r, end - 1)), int64_t(0));
#pragma unroll
      for (int x = 0; x < KS; ++x) kf[h][x] = load_frag(a.k_pages + row * (D * 2) + x * 64 + g * 16);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pos = t0 + 16 * (i >> 2) + 4 * g + (i & 3);
      const int64_t row = row_of(min(pos, end - 1));
      if (pos >= end || row < 0) dead |= 1u << i;
      const uint8_t* vp = a.v_pages + max(row, int64_t(0)) * (D * 2) + r * (DPL * 2);
      if constexpr (VW == 4) {
        const uint4 w = *reinterpret_cast<const uint4*>(vp);
        vr[i][0] = w.x; vr[i][1] = w.y; vr[i][2] = w.z; vr[i][3] = w.w;
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(vp);
        vr[i][0] = w.x; vr[i][1] = w.y;
      }
    }
    f32x4 s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = 0; x < KS; ++x) s[h] = mfma(kf[h][x], qf[x], s[h]);
    }
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = s[i >> 2][i & 3] * a.scale_log2;
    if (!clean || t0 + kAttnTile > end) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (dead >> i & 1) {
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
    const float base = top == -INFINITY ? 0.0f : top;
    const float shrink = pow2(mx - base);
    mx = top;
    sum *= shrink;
#pragma unroll
    for (int m = 0; m < DPL; ++m) o[m] *= shrink;
    Frag pf;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = pow2(p[i] - base);
      sum += p[i];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) pf.w[j] = pack_bf16(p[2 * j], p[2 * j + 1]);
#pragma unroll
    for (int m = 0; m < DPL; ++m) {
      Frag vf;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        vf.w[j] = __builtin_amdgcn_perm(vr[2 * j + 1][m / 2], vr[2 * j][m / 2], m % 2 ? 0x07060302u : 0x05040100u);
      o[m] = mfma(vf, pf, o[m]);
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

  const int64_t units = int64_t(a.B) * a.Hq;
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
    const int64_t unit = int64_t(b) * a.Hq + kvh * G + head0 + h;
    if (plan.splits == 1) {
      reinterpret_cast<uint16_t*>(a.out)[unit * D + c] = float_to_bf16_bits(l == 0.0f ? 0.0f : acc / l);
    } else {
      a.ws[(unit * plan.splits + split) * D + c] = acc;
      if (c == 0) reinterpret_cast<float2*>(a.ws + units * plan.splits * D)[unit * plan.splits + split] = make_float2(m0, l);
    }
  }
}

// The chunks of one (request, query head) joined: sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s,
// in the order of the chunks. A request of no tokens gets zeros.
template <int D>
__global__ __launch_bounds__(D) void kv_join_kernel(const AttnArgs a, const AttnPlan plan) {
  const int c = __builtin_amdgcn_workitem_id_x();
  const int64_t unit = __builtin_amdgcn_workgroup_id_x();
  const int b = static_cast<int>(unit / a.Hq);
  const int64_t cap = int64_t(a.max_blocks) << a.page_log2;
  const int len = static_cast<int>(min(int64_t(min(max(a.seq_lens[b], 0), a.max_len)), cap));
  const int n = (len + plan.chunk - 1) / plan.chunk;
  const float* po = a.ws + unit * plan.splits * D + c;
  const float2* ml = reinterpret_cast<const float2*>(a.ws + int64_t(a.B) * a.Hq * plan.splits * D) + unit * plan.splits;
  float m = -INFINITY;
  for (int s = 0; s < n; ++s) m = fmaxf(m, ml[s].x);
  const float base = m == -INFINITY ? 0.0f : m;
  float acc = 0.0f, l = 0.0f;
  for (int s = 0; s < n; ++s) {
    const float2 x = ml[s];
    const float f = pow2(x.x - base);
    acc = fmaf(f, po[int64_t(s) * D], acc);
    l = fmaf(f, x.y, l);
  }
  reinterpret_cast<uint16_t*>(a.out)[unit * D + c] = float_to_bf16_bits(l == 0.0f ? 0.0f : acc / l);
}

template <int D>
hipError_t attention_d(const AttnArgs& a, hipStream_t s) {
  const AttnPlan p = attn_plan(a.B, a.Hq, a.Hkv, a.max_len);
  const unsigned grid = static_cast<unsigned>(kv_attention_grid(a.B, a.Hq, a.Hkv, a.max_len));
  hipLaunchKernelGGL((kv_attention_kernel<D>), dim3(grid), dim3(256), 0, s, a, p);
  if (p.splits > 1)
    hipLaunchKernelGGL((kv_join_kernel<D>), dim3(static_cast<unsigned>(a.B) * static_cast<unsigned>(a.Hq)), dim3(D), 0, s, a, p);
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
  return int64_t(B) * Hkv * p.tiles * p.splits;
}

size_t kv_attention_ws_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int32_t max_len) {
  const AttnPlan p = attn_plan(B, Hq, Hkv, max_len);
  if (p.splits == 1) return 0;
  return static_cast<size_t>(B) * Hq * p.splits * (static_cast<size_t>(d) + 2) * 4;
}

hipError_t launch_kv_attention(int d, const AttnArgs& a, hipStream_t s) {
  switch (d) {
    case 64: return attention_d<64>(a, s);
    case 128: return attention_d<128>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace damp
