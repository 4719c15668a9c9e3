// latent_prompt_kernels.hip -- gfx950 kernel of latent attention over prompts, expanded form: keys and
// values of each head as the up-projection gives them, and one rotary key a token for all heads.
#include <algorithm>

#include "attn_mask.h"

namespace damp {
namespace {

// o_i = sum_t p_it v_t / sum_t p_it over the keys t <= before + i of the query's request, p_it =
// exp(scale (q_i.(k_t | kr_t)) - m_i) with a running maximum and sum, one pass over the keys. A
// workgroup takes 64 R queries of one head, 16 R a wave; tiles of 64 keys and values go through LDS,
// the next one on its way in registers. Scores^T = K Q^T, so that a query is a lane's column: its
// maximum takes two exchanges, and the scores' C tiles are the B operand of out^T = V^T P^T as they
// stand (lane group g holds keys 4 g .. + 3 of both halves of 32; V^T is read transposed from LDS in the
// same order). Bound by the products and by the exponentials between them.
constexpr int kKeyTile = 64;

template <int D, int R>
__global__ __launch_bounds__(256, 2) void latent_prompt_kernel(const LatentPromptArgs a, int items) {
  constexpr int DR = D / 2, DQ = D + DR, KS = DQ / 32, MB = D / 16, TB = kKeyTile / 16;
  constexpr int LK = DQ * 2 + 32, LV = D * 2 + 32;      // bytes between rows in LDS: an odd number of 32-byte units
  constexpr int PN = D / 8, PR = DR / 8;                // 16-byte pieces of a row
  constexpr int NN = kKeyTile * PN / 256, NR = kKeyTile * PR / 256;
  constexpr int ROWS = 64 * R;
  __shared__ __align__(16) uint8_t tile_k[kKeyTile * LK];
  __shared__ __align__(16) uint8_t tile_v[kKeyTile * LV];
  __shared__ int any_odd;

  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const unsigned id = __builtin_amdgcn_workgroup_id_x();
  const int h = id % a.H;
  const int item = items - 1 - static_cast<int>(id / a.H);   // the last queries of a request, which have most keys, start first

  // the request of this item: requests of n queries hold ceil(n / ROWS) items
  int b = -1, local = 0;
  for (int b0 = 0, before = 0; b0 < a.B && before <= item; b0 += 64) {
    int n = 0;
    if (b0 + lane < a.B) {
      const int lo = min(max(a.cu_q[b0 + lane], 0), a.Tq), hi = min(max(a.cu_q[b0 + lane + 1], lo), a.Tq);
      n = (hi - lo + ROWS - 1) / ROWS;
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int y = __shfl_up(incl, o);
      if (lane >= o) incl += y;
    }
    const int first = before + incl - n;
    if (const uint64_t mine = __ballot(item >= first && item < first + n); mine != 0) {
      const int l = __builtin_ctzll(mine);
      b = b0 + l;
      local = item - __builtin_amdgcn_readlane(first, l);
      break;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  if (b < 0) return;
  const int q_lo = min(max(a.cu_q[b], 0), a.Tq), q_hi = min(max(a.cu_q[b + 1], q_lo), a.Tq);
  const int k_lo = min(max(a.cu_k[b], 0), a.Tk), k_hi = min(max(a.cu_k[b + 1], k_lo), a.Tk);
  const int nq = q_hi - q_lo, nk = k_hi - k_lo, before = nk - nq;
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

  u32x4 sn[NN], sr[NR], sv[NN];
  // (offsets inside a tile fit 32 bits: a token stride is at most 2^24 elements)
  const uint32_t k_step = static_cast<uint32_t>(a.k_token) * 2, v_step = static_cast<uint32_t>(a.v_token) * 2;
  uint32_t k_off[NN], v_off[NN], r_off[NR];
  const auto offsets = [&](int last) {      // rows past the end repeat the last; masked
#pragma unroll
    for (int i = 0; i < NN; ++i) {
      const uint32_t t = min(tid / PN + 256 / PN * i, last);
      k_off[i] = t * k_step + tid % PN * 16;
      v_off[i] = t * v_step + tid % PN * 16;
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) r_off[i] = min(tid / PR + 256 / PR * i, last) * (DR * 2) + tid % PR * 16;
  };
  offsets(kKeyTile);
  const auto issue = [&](int t0) {
    if (t0 + kKeyTile > nk) {
      offsets(rarely(nk - 1 - t0));
    }
    const int64_t t = int64_t(k_lo) + t0;
    const uint8_t* kb = a.k + (t * a.k_token + h * a.k_head) * 2;
    const uint8_t* vb = a.v + (t * a.v_token + h * a.v_head) * 2;
    const uint8_t* rb = a.k_rope + t * (DR * 2);
#pragma unroll
    for (int i = 0; i < NN; ++i) {
      sn[i] = *reinterpret_cast<const u32x4*>(kb + k_off[i]);
      sv[i] = *reinterpret_cast<const u32x4*>(vb + v_off[i]);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) sr[i] = *reinterpret_cast<const u32x4*>(rb + r_off[i]);
  };
  if (tid == 0) any_odd = 0;
  if (stop > 0) issue(0);
  else __syncthreads();
  for (int t0 = 0; t0 < stop; t0 += kKeyTile) {
    const bool masked = t0 + kKeyTile > min(full, nk);
    __syncthreads();                 // the tile before is no longer read
#pragma unroll
    for (int i = 0; i < NN; ++i) {
      const int t = tid / PN + 256 / PN * i;
      *reinterpret_cast<u32x4*>(tile_k + t * LK + tid % PN * 16) = sn[i];
      u32x4 w = sv[i];
      if (masked) {
        w = rarely(w);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          odd |= not_finite(w[x]);
          w[x] = finite_only(w[x]);
        }
      }
      *reinterpret_cast<u32x4*>(tile_v + t * LV + tid % PN * 16) = w;
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) *reinterpret_cast<u32x4*>(tile_k + (tid / PR + 256 / PR * i) * LK + D * 2 + tid % PR * 16) = sr[i];
    __syncthreads();
    if (t0 + kKeyTile < stop) issue(t0 + kKeyTile);
    if (t0 > before + wave0 + 16 * R - 1 || wave0 >= nq) continue;   // none of the wave's queries sees a key of the tile

    f32x4 s[R][TB];
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) {
#pragma unroll
      for (int j = 0; j < R; ++j) s[j][tb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        const Frag kf = load_frag(tile_k + (16 * tb + r) * LK + g * 16 + x * 64);
#pragma unroll
        for (int j = 0; j < R; ++j) s[j][tb] = mfma(kf, qf[j][x], s[j][tb]);
      }
    }
    // (operands four steps ahead: a read from LDS takes as long as some ten products)
    __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
    for (int x = 0; x < TB * KS; ++x) {
      __builtin_amdgcn_sched_group_barrier(0x008, R, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
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
      const uint8_t* v = tile_v + (32 * st + 4 * g + (r >> 2)) * LV + 8 * (r & 3);
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const Frag vf = load_frag_t(reinterpret_cast<const uint16_t*>(v + 32 * m), reinterpret_cast<const uint16_t*>(v + 32 * m + 16 * LV));
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
  }

  if (__any(odd != 0)) any_odd = 1;
  __syncthreads();
  if (any_odd) {
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

int64_t prompt_items(int64_t B, int64_t Tq, int rows) { return std::min(Tq, Tq / rows + B); }

template <int D>
hipError_t prompt_d(const LatentPromptArgs& a, hipStream_t s) {
  const int64_t wide = prompt_items(a.B, a.Tq, 128);
  if (wide * a.H >= 256) {
    hipLaunchKernelGGL((latent_prompt_kernel<D, 2>), dim3(static_cast<unsigned>(wide * a.H)), dim3(256), 0, s, a, static_cast<int>(wide));
  } else {
    const int64_t n = prompt_items(a.B, a.Tq, 64);
    hipLaunchKernelGGL((latent_prompt_kernel<D, 1>), dim3(static_cast<unsigned>(n * a.H)), dim3(256), 0, s, a, static_cast<int>(n));
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
