// latent_prompt_kernels.hip -- gfx950 kernel of latent attention over prompts, expanded form: keys and
// values of each head as the up-projection gives them, and one rotary key a token for all heads.
#include <algorithm>

#include "attn_mask.h"

namespace damp {
namespace {

// o_i = sum_t p_it v_t / sum_t p_it over the keys t <= before + i of the query's request, p_it =
// exp(scale (q_i.(k_t | kr_t)) - m_i) with a running maximum and sum, one pass over the keys. A
// workgroup takes 64 R queries of one head, 16 R a wave; tiles of 64 keys and values are loaded into LDS,
// the next one while this one is worked on, with one barrier a tile. Scores^T = K Q^T, so that a query is a lane's column: its
// maximum takes two exchanges, and the scores' C tiles are the B operand of out^T = V^T P^T as they
// stand (lane group g holds keys 4 g .. + 3 of both halves of 32; V^T is read transposed from LDS in the
// same order). Bound by the products and by the exponentials between them: 8 prompts, 12,288 tokens, 16 heads of
// d = 128, 200 to 210 us or 900 TFLOP/s (1,358 for a large product alone; matrix cores are busy 48% of the SIMDs' cycles; the
// clock falls under this load, and medians of 215 to 240 us are seen too).
constexpr int kKeyTile = 64;

struct Request {
  int q, nq, k, nk;        // first query and key, and how many
};

// (kept inside the arrays whatever the lists hold)
__device__ __forceinline__ Request request_of(const LatentPromptArgs& a, int b) {
  Request x;
  x.q = min(max(a.cu_q[b], 0), a.Tq);
  x.nq = min(max(a.cu_q[b + 1], x.q), a.Tq) - x.q;
  x.k = min(max(a.cu_k[b], 0), a.Tk);
  x.nk = min(max(a.cu_k[b + 1], x.k), a.Tk) - x.k;
  return x;
}

struct Part {              // row tile `tile` of request b; b < 0: none
  int b, tile;
  Request own;
};

// The row tiles by falling number of key tiles, so that the longest start first (their order is what the end of the
// launch depends on: in the requests' order a call's last row tiles, of whichever lengths, run alone). A
// request's row tiles see more keys from one to the next, so how many see at least L key tiles is a
// formula, and place `item` of the list is found by bisection over L; for more than 64 requests, which even
// out by themselves, in the requests' order.
template <int ROWS>
__device__ __forceinline__ Part part_of(const LatentPromptArgs& a, int item) {
  const int lane = __builtin_amdgcn_workitem_id_x() & 63;
  Request own{0, 0, 0, 0};
  if (lane < a.B) own = request_of(a, lane);
  const auto pick = [&](int b0, const Request& x, int first, int n, int skip) -> Part {
    const uint64_t mine = __ballot(item >= first && item < first + n);
    if (mine == 0) return Part{-1, 0, x};
    const int l = __builtin_ctzll(mine);
    const auto of = [&](int y) { return __builtin_amdgcn_readlane(y, l); };
    return Part{b0 + l, of(skip) + item - of(first), Request{of(x.q), of(x.nq), of(x.k), of(x.nk)}};
  };
  if (a.B > 64) {
    for (int b0 = 0, before = 0; b0 < a.B; b0 += 64) {
      const Request x = b0 == 0 ? own : b0 + lane < a.B ? request_of(a, b0 + lane) : Request{0, 0, 0, 0};
      const int n = (x.nq + ROWS - 1) / ROWS, incl = scan64(n);
      const Part p = pick(b0, x, before + incl - n, n, 0);
      if (p.b >= 0) return p;
      before += last_lane(incl);
    }
    return Part{-1, 0, own};
  }
  const int tiles = (own.nq + ROWS - 1) / ROWS;
  const auto at_least = [&](int L) -> int {          // this lane's row tiles that see L key tiles or more
    if (L <= 0) return tiles;
    const int key = (L - 1) * kKeyTile + 1, past = key - (own.nk - own.nq);     // a tile whose queries end at `past` or later
    return own.nk < key ? 0 : tiles - max((past + ROWS - 1) / ROWS - 1, 0);
  };
  const auto sum = [&](int x) { return last_lane(scan64(x)); };
  if (item >= sum(tiles)) return Part{-1, 0, own};
  int lo = 0, hi = (a.Tk + kKeyTile - 1) / kKeyTile + 1;   // sum(at_least(lo)) > item >= sum(at_least(hi))
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sum(at_least(mid)) > item) lo = mid; else hi = mid;
  }
  const int level = at_least(lo), more = at_least(hi), n = level - more, incl = scan64(n);
  return pick(0, own, sum(more) + incl - n, n, tiles - level);
}

template <int D, int R>
__global__ __launch_bounds__(256, D == 64 ? 3 : 2) void latent_prompt_kernel(const LatentPromptArgs a) {
  constexpr int DR = D / 2, DQ = D + DR, KS = DQ / 32, MB = D / 16, TB = kKeyTile / 16;
  constexpr int PN = D / 8, PR = DR / 8;                // 16-byte pieces of a row
  constexpr int NN = kKeyTile * PN / 256, NR = kKeyTile * PR / 256;
  constexpr int ROWS = 64 * R;
  // (two workgroups of d = 128 take a CU's 160 KB to the byte)
  // (and each buffer is an array of its own, so that reads of one need not keep their order with loads into the other)
  __shared__ __align__(1024) uint8_t n0[kKeyTile * D * 2], n1[kKeyTile * D * 2], v0[kKeyTile * D * 2], v1[kKeyTile * D * 2];
  __shared__ __align__(1024) uint8_t r0[kKeyTile * DR * 2], r1[kKeyTile * DR * 2];

  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const unsigned id = __builtin_amdgcn_workgroup_id_x();
  const int h = id % a.H;
  const Part part = part_of<ROWS>(a, static_cast<int>(id / a.H));
  const int b = part.b, local = part.tile;
  if (b < 0) return;
  const int q_lo = part.own.q, k_lo = part.own.k;
  const int nq = part.own.nq, nk = part.own.nk, before = nk - nq;
  const int row0 = local * ROWS, wave0 = row0 + wv * 16 * R;      // queries of the workgroup, of the wave
  const int stop = min(nk, before + min(row0 + ROWS, nq));        // keys that some query sees: [0, stop)
  const int full = before + row0 + 1;                             // keys that all see: [0, full)

  Frag qf[R][KS];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int64_t row = q_lo + min(wave0 + 16 * j + r, nq - 1);
    const uint8_t* qp = a.q + ((row * a.H + h) * DQ + g * 8) * 2;
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      qf[j][x] = load_frag(qp + x * 64);
      // (a negative scale goes into the queries' signs)
#pragma unroll
      for (int i = 0; i < 4; ++i) qf[j][x].w[i] ^= a.flip;
    }
  }
  f32x4 o[R][MB];
  float mx[R];
  f32x4 sum[R];                // the same in all four
#pragma unroll
  for (int j = 0; j < R; ++j) {
    mx[j] = -INFINITY;
    sum[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int m = 0; m < MB; ++m) o[j][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  const float slack = fminf(kSlack / a.scale_log2, 0x1p100f);
  uint32_t odd = 0;            // values that are not finite have been taken out

  // (offsets inside a tile fit 32 bits: a token stride is at most 2^24 elements)
  const uint32_t k_step = static_cast<uint32_t>(a.k_token) * 2, v_step = static_cast<uint32_t>(a.v_token) * 2;
  uint32_t k_off[NN], v_off[NN], r_off[NR];
  const auto offsets = [&](int last) {      // rows past the end repeat the last; masked
#pragma unroll
    for (int i = 0; i < NN; ++i) {
      const int t = tid / PN + 256 / PN * i;
      k_off[i] = min(t, last) * k_step + (tid % PN ^ row_turn<PN>(t)) * 16;
      v_off[i] = min(t, last) * v_step + (tid % PN ^ column_turn<PN>(t)) * 16;
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int t = tid / PR + 256 / PR * i;
      r_off[i] = min(t, last) * (DR * 2) + (tid % PR ^ row_turn<PR>(t)) * 16;
    }
  };
  offsets(kKeyTile);
  // Load `n` of a tile's 2 NN + NR.
  struct Tile {
    const uint8_t *n, *r, *v;
  };
  const auto tile_at = [&](int t0) -> Tile {
    const int64_t t = int64_t(k_lo) + t0;
    return Tile{a.k + (t * a.k_token + h * a.k_head) * 2, a.k_rope + t * (DR * 2), a.v + (t * a.v_token + h * a.v_head) * 2};
  };
  constexpr int kLoads = 2 * NN + NR;
  const auto load = [&](int n, const Tile& from, uint8_t* tile_n, uint8_t* tile_r, uint8_t* tile_v) {
    const int i = n % NN, at = wv * 1024;
    if (n < NN) load_to_lds(from.n + k_off[i], tile_n + i * 4096 + at);
    else if (n < 2 * NN) load_to_lds(from.v + v_off[i], tile_v + i * 4096 + at);
    else load_to_lds(from.r + r_off[i], tile_r + i * 4096 + at);
  };
  if (nk < kKeyTile) offsets(nk - 1);
  if (stop > 0) {
    const Tile from = tile_at(0);
#pragma unroll
    for (int n = 0; n < kLoads; ++n) load(n, from, n0, r0, v0);
  }
  const int last_t0 = (stop - 1) / kKeyTile * kKeyTile;
  // The tile at t0, which lies in the first three buffers, while the next is loaded into the others.
  const auto step = [&](int t0, uint8_t* tile_n, uint8_t* tile_r, uint8_t* tile_v, uint8_t* next_n, uint8_t* next_r, uint8_t* next_v) {
    landed();
    __syncthreads();                 // (the tile before is no longer read, either)
    if (t0 + kKeyTile > min(full, nk)) {
      // some query does not see some key: values that are not finite are taken out
#pragma unroll
      for (int i = 0; i < NN; ++i) {
        u32x4* at = reinterpret_cast<u32x4*>(tile_v + (i * 256 + tid) * 16);
        u32x4 w = *at;
        uint32_t here = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          here |= not_finite(w[x]);
          w[x] = finite_only(w[x]);
        }
        if (here) *at = w;
        odd |= here;
      }
      __syncthreads();
    }
    const int next = min(t0 + kKeyTile, last_t0);       // (after the last tile that one again: no branch among the products)
    if (next + kKeyTile > nk) offsets(rarely(nk - 1 - next));
    const Tile from = tile_at(next);
    if (t0 > before + wave0 + 16 * R - 1 || wave0 >= nq) {           // none of the wave's queries sees a key of the tile
#pragma unroll
      for (int n = 0; n < kLoads; ++n) load(n, from, next_n, next_r, next_v);
      return;
    }

    // Operands are read four steps ahead (a read from LDS takes as long as some ten products), and the next tile's
    // loads go out one by one among the products (each takes the address unit 16 cycles).
    const auto operand = [&](int n) -> Frag {
      const int t = 16 * (n / KS) + r, p = 4 * (n % KS) + g;
      return load_frag(n % KS < PN / 4 ? tile_n + t * (D * 2) + (p ^ row_turn<PN>(t)) * 16 : tile_r + t * (DR * 2) + ((p - PN) ^ row_turn<PR>(t)) * 16);
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
      if (n % 2 == 0 && n / 2 < kLoads) load(n / 2, from, next_n, next_r, next_v);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (t0 + kKeyTile > min(before + wave0 + 1, nk)) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int last = rarely(min(before + wave0 + 16 * j + r, nk - 1) - t0 - 4 * g);   // the last key that this query sees
#pragma unroll
        for (int tb = 0; tb < TB; ++tb)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (16 * tb + i > last) s[j][tb][i] = -INFINITY;
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
        const float shrink = top == -INFINITY ? 1.0f : pow2((mx[j] - top) * a.scale_log2);
        mx[j] = top;
        sum[j] *= shrink;
#pragma unroll
        for (int m = 0; m < MB; ++m) o[j][m] *= shrink;
      }
      const float base = mx[j] == -INFINITY ? 0.0f : -mx[j] * a.scale_log2;
#pragma unroll
      for (int st = 0; st < TB / 2; ++st) {
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = pow2(fmaf(s[j][2 * st + (i >> 2)][i & 3], a.scale_log2, base));
        pf[j][st] = round_weights(p);
        sum[j] = mfma(ones(), pf[j][st], sum[j]);
      }
    }
#pragma unroll
    for (int st = 0; st < TB / 2; ++st) {
      const int t = 32 * st + 4 * g + (r >> 2), turn = column_turn<PN>(t);    // (the row 16 further has the same turn)
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
  for (int t0 = 0; t0 < stop; t0 += 2 * kKeyTile) {
    step(t0, n0, r0, v0, n1, r1, v1);
    if (t0 + kKeyTile < stop) step(t0 + kKeyTile, n1, r1, v1, n0, r0, v0);
  }

  int* any_odd = reinterpret_cast<int*>(r0);
  landed();                        // (nothing may be on its way into the flag's place, or into LDS that the workgroup no longer holds)
  __syncthreads();
  if (tid == 0) *any_odd = 0;
  __syncthreads();
  if (__any(odd != 0)) *any_odd = 1;
  __syncthreads();
  if (*any_odd) {
#pragma unroll 1
    for (int t = max(min(full, nk) - kKeyTile, 0); t < stop; ++t) {
      const uint8_t* v = a.v + ((int64_t(k_lo) + t) * a.v_token + int64_t(h) * a.v_head) * 2 + g * 8;
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int m = 0; m < MB; ++m) o[j][m] = add_odd(o[j][m], *reinterpret_cast<const uint2*>(v + 32 * m), t <= before + wave0 + 16 * j + r);
    }
  }
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int row = wave0 + 16 * j + r;
    if (row >= nq) continue;
    const float back = sum[j][0] == 0.0f ? 0.0f : 1.0f / sum[j][0];
    uint8_t* to = a.out + ((int64_t(q_lo) + row) * a.H + h) * (D * 2) + g * 8;
#pragma unroll
    for (int m = 0; m < MB; ++m)
      *reinterpret_cast<uint2*>(to + 32 * m) = make_uint2(pack_bf16(o[j][m][0] * back, o[j][m][1] * back), pack_bf16(o[j][m][2] * back, o[j][m][3] * back));
  }
}

// Row tiles there may be, whatever the lists hold. 64 rows while full tiles of 64 are no more than the workgroups that the chip
// holds at once (2 a CU with d = 128, 3 with d = 64), else 128. With 64 and 128 rows (us; in parentheses the tiles of 64): d =
// 128, one prompt of 4,096 tokens and 8 heads (512) 74 and 95, 8 of 300 and 10 (375) 12.0 and 14.8, 16 of 100 behind 4,000 and 16
// (400) 126 and 137; 8 of 300 and 14 (525) 16.6 and 16.7, 16 of 300 and 8 (600) 19.6 and 17.7, 2 of 1,000 behind 4,000 and
// 24 (750) 174 and 157, 4 of 512 behind 8,000 and 24 (768) 404 and 287, 8 of 1,536 and 16 270 and 210; d = 64, 2 of 2,048 and 8
// (512) 27 and 36, 16 of 100 behind 4,000 and 24 (600) 120 and 111, one of 8,192 and 16 (2,048) 212 and 190. Where a prompt's tiles
// differ much in how many keys they see, more rounds of the shorter ones do as well: one of 4,096 and 12 (768) 85 and 103.
int64_t prompt_items(int64_t B, int64_t Tq, int rows) { return std::min(Tq, Tq / rows + B); }

template <int D>
hipError_t prompt_d(const LatentPromptArgs& a, hipStream_t s) {
  if (int64_t(a.Tq) * a.H > 64 * (D == 64 ? 768 : 512)) {
    const int64_t wide = prompt_items(a.B, a.Tq, 128);
    hipLaunchKernelGGL((latent_prompt_kernel<D, 2>), dim3(static_cast<unsigned>(wide * a.H)), dim3(256), 0, s, a);
  } else {
    const int64_t n = prompt_items(a.B, a.Tq, 64);
    hipLaunchKernelGGL((latent_prompt_kernel<D, 1>), dim3(static_cast<unsigned>(n * a.H)), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

int64_t latent_prompt_grid(int32_t B, int32_t Tq, int32_t H) { return prompt_items(B, Tq, 64) * H; }

hipError_t launch_latent_prompt(int d, const LatentPromptArgs& a, hipStream_t s) {
  switch (d) {
    case 64: return prompt_d<64>(a, s);
    case 128: return prompt_d<128>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace damp
