// linear_kernels.hip -- gfx950 kernels of linear attention with a decay (S <- a S + k v^T,
// o = S^T q) on an fp32 state pool: the single-token step, and the token-by-token prompt form
// that also takes the gated delta rule (e = beta (v - S'^T k) in place of v). The chunked prompt
// form is in prompt_kernels.hip.
#include "prompt_common.h"

namespace damp {
namespace {

// ---- the single-token step -----------------------------------------------------------------
// One workgroup per unit; the state crosses HBM once in and once out, and nothing else of its
// size moves, so the kernel is bound by that stream (2 * 4 d^2 bytes per unit against 5 d^2
// flops). A row of the state is D / 4 lanes of 16 bytes; the whole unit is in flight at once
// (64 fp32 values per lane at d = 128). The readout is taken from the updated row while it is in
// registers; the partial column sums of the row groups meet in LDS, added in a fixed order.
// 1,024 requests x 32 heads, d = 128: 792 us for 4.34 GB, 5.5 TB/s (a copy reaches 5.6); 3 x 32: 4.5 us.
constexpr int lin_threads(int d) { return d >= 64 ? 256 : 64; }

template <int D>
struct LinGeo {
  static constexpr int LPR = D / 4;                         // lanes per row
  static constexpr int NT = lin_threads(D);                 // threads per workgroup
  static constexpr int RPS = NT / LPR;                      // rows per row step
  static constexpr int RPL = D / RPS;                       // rows per lane
  static_assert(RPL >= 1 && RPL * RPS == D, "unsupported d");
};

template <int D, int DECAY, int BF16>
__global__ __launch_bounds__(LinGeo<D>::NT) void linear_step_kernel(const StepArgs a) {
  using G = LinGeo<D>;
  __shared__ float sk[D], sq[D], sa[D];
  __shared__ float4 red[G::RPS][G::LPR];
  const int tid = __builtin_amdgcn_workitem_id_x();
  const int bh = __builtin_amdgcn_workgroup_id_x();
  const int b = bh / a.H, head = bh - b * a.H;
  const int64_t slot = a.slot_idx[b];
  if (!slot_in_pool(slot, a.st.num_slots)) return;
  const int rg = tid / G::LPR, cg = tid % G::LPR;
  using f4 = __attribute__((ext_vector_type(4))) float;
  f4* base = reinterpret_cast<f4*>(a.st.hbase + (slot * a.H + head) * a.st.hstride) + rg * G::LPR + cg;
  f4 S[G::RPL];
#pragma unroll
  for (int t = 0; t < G::RPL; ++t) S[t] = __builtin_nontemporal_load(base + t * G::RPS * G::LPR);
  const int64_t at = int64_t(bh) * D;
  for (int i = tid; i < D; i += G::NT) {
    sk[i] = load_in<BF16>(a.k, at + i);
    sq[i] = load_in<BF16>(a.q, at + i);
    if constexpr (DECAY == DECAY_KEY) sa[i] = a.alpha[at + i];
  }
  float v[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) v[c] = load_in<BF16>(a.v, at + cg * 4 + c);
  const float decay = DECAY == DECAY_KEY ? 0.0f : a.alpha[DECAY == DECAY_HEAD ? head : bh];
  __syncthreads();
  float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int t = 0; t < G::RPL; ++t) {
    const int i = t * G::RPS + rg;
    const float k = sk[i], q = sq[i], al = DECAY == DECAY_KEY ? sa[i] : decay;
    f4 x = S[t];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      x[c] = fmaf(k, v[c], al * S[t][c]);
      p[c] = fmaf(q, x[c], p[c]);
    }
    __builtin_nontemporal_store(x, base + t * G::RPS * G::LPR);
  }
  red[rg][cg] = make_float4(p[0], p[1], p[2], p[3]);
  __syncthreads();
  if (tid < D) {
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < G::RPS; ++r) s += reinterpret_cast<const float*>(red[r])[tid];
    a.out[at + tid] = s;
  }
}

// ---- prompts, token by token -----------------------------------------------------------------
// One workgroup per (request, head, 16 value columns): column j of the state only needs column j of
// v, so workgroups are independent and the state stays in registers for the whole prompt. D / 8
// neighbouring lanes share a column, 8 rows of it each (4 lanes at d = 16), and add up by DPP; the
// tokens' keys, queries and gates are staged in LDS for all the waves. Every operation is binary32, in
// token order. It serves what the chunked form is not built for: fp32 inputs, a decay per key channel,
// d below 64. It is bound by the latency of the token chain: each token's instructions depend on the
// last's. With a decay per key channel, bf16, 32 heads, d = 128: a prompt of 4,096 tokens takes 1.17 ms
// by the delta rule (0.29 us a token) and 0.90 ms without it, 32 prompts of 256 tokens 780 and 610 us.
// (4 lanes a column, one wave a workgroup: 2.23 and 1.87 ms, 911 and 781 us; it is faster where a
// prompt is a few tokens and the state's way in and out is all, 277 against 338 us for 256 prompts of
// 4 tokens, as its lanes read 64 bytes of a row and not 16. 16 lanes a column in workgroups of one wave
// stage the same rows four times as often: 1.77 ms for the 32 prompts.)
constexpr int kTokBlock = 16;   // tokens staged in LDS at a time

// Sum over RG neighbouring lanes, the same in each of them (DPP: quad_perm, then mirrored halves).
template <int RG>
__device__ __forceinline__ float sum_lanes(float x) {
  static_assert(RG == 4 || RG == 8 || RG == 16, "4, 8 or 16 lanes");
  x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0xB1, 0xF, 0xF, true));
  x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x4E, 0xF, 0xF, true));
  if constexpr (RG >= 8) x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x141, 0xF, 0xF, true));
  if constexpr (RG == 16) x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x140, 0xF, 0xF, true));
  return x;
}

template <int D>
struct TokGeo {
  static constexpr int RG = D >= 32 ? D / 8 : 4;   // lanes that share a column
  static constexpr int QR = D / (4 * RG);          // quads of rows of a lane
  static constexpr int NT = 16 * RG;               // threads: 16 columns
};

template <int D, bool DELTA, int DECAY, int BF16>
__global__ __launch_bounds__(TokGeo<D>::NT) void prompt_token_kernel(const PromptArgs a) {
  constexpr int RG = TokGeo<D>::RG, QR = TokGeo<D>::QR, NT = TokGeo<D>::NT;
  __shared__ __align__(16) float sk[kTokBlock][D], sq[kTokBlock][D];
  __shared__ __align__(16) float sa[DECAY == DECAY_KEY ? kTokBlock : 1][DECAY == DECAY_KEY ? D : 4];
  __shared__ float sg[kTokBlock], sb[kTokBlock];
  __shared__ __align__(16) float sv[kTokBlock][16];
  const int tid = __builtin_amdgcn_workitem_id_x();
  const int unit = __builtin_amdgcn_workgroup_id_x() / (D / 16), c0 = (__builtin_amdgcn_workgroup_id_x() % (D / 16)) * 16;
  const int b = unit / a.H, head = unit - b * a.H;
  const int64_t slot = a.slot_idx[b];
  if (!slot_in_pool(slot, a.num_slots)) return;
  const Span sp = span_of(a, b);
  if (sp.end <= sp.begin || (a.few && sp.end - sp.begin > a.few)) return;
  const int rg = tid % RG, c = tid / RG;
  float* pool = a.pool + ((slot * a.H + head) * D + 4 * rg) * int64_t(D) + c0 + c;
  f32x4 S[QR];   // S[j][i]: row 4 (rg + RG j) + i
  const bool resume = a.resume && a.resume[b] != 0;
#pragma unroll
  for (int j = 0; j < QR; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) S[j][i] = resume ? pool[(4 * RG * j + i) * D] : 0.0f;

  // A block of tokens is on its way in registers while the one before is computed: 16-byte pieces of k
  // and q (and of per-key gates), through resources that end with the request's last row.
  constexpr int E = BF16 ? 2 : 4, PR = D * E / 16, NP = (kTokBlock * PR + NT - 1) / NT;   // pieces per row, per thread
  constexpr int PA = D / 4, NA = DECAY == DECAY_KEY ? (kTokBlock * PA + NT - 1) / NT : 0;
  const uint32_t ostep = static_cast<uint32_t>(a.H) * D * E;
  struct Block {
    uint4 k[NP], q[NP], al[NA ? NA : 1];
    uint32_t v[4];
    float gate, beta;
  } in;
  const auto load = [&](int t0) {
    const int rows = min(kTokBlock, sp.end - t0);
    const int64_t at = (int64_t(t0) * a.H + head) * D;
    const auto region = [&](const void* p, int e) {
      return make_rsrc(static_cast<const uint8_t*>(p) + at * e, (rows - 1) * (a.H * D * e) + D * e);
    };
    const rsrc_t kr = region(a.k, E), qr = region(a.q, E), vr = region(a.v, E);
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int x = tid + NT * j;
      const uint32_t off = x / PR * ostep + x % PR * 16;
      const auto kk = __builtin_amdgcn_raw_buffer_load_b128(kr, off, 0, 0), qq = __builtin_amdgcn_raw_buffer_load_b128(qr, off, 0, 0);
      in.k[j] = make_uint4(kk[0], kk[1], kk[2], kk[3]);
      in.q[j] = make_uint4(qq[0], qq[1], qq[2], qq[3]);
    }
    if constexpr (NA > 0) {
      const rsrc_t ar = region(a.alpha, 4);
#pragma unroll
      for (int j = 0; j < NA; ++j) {
        const int x = tid + NT * j;
        const auto aa = __builtin_amdgcn_raw_buffer_load_b128(ar, x / PA * (a.H * D * 4) + x % PA * 16, 0, 0);
        in.al[j] = make_uint4(aa[0], aa[1], aa[2], aa[3]);
      }
    }
    // 4 value columns of token tid / 4 (those past the block load past the rows: 0)
    const uint32_t voff = tid / 4 * ostep + (c0 + tid % 4 * 4) * E;
    if constexpr (BF16) {
      const auto vv = __builtin_amdgcn_raw_buffer_load_b64(vr, voff, 0, 0);
      in.v[0] = vv[0] << 16; in.v[1] = vv[0] & 0xffff0000u; in.v[2] = vv[1] << 16; in.v[3] = vv[1] & 0xffff0000u;
    } else {
      const auto vv = __builtin_amdgcn_raw_buffer_load_b128(vr, voff, 0, 0);
      in.v[0] = vv[0]; in.v[1] = vv[1]; in.v[2] = vv[2]; in.v[3] = vv[3];
    }
    const int64_t tok = int64_t(t0 + min(tid, rows - 1)) * a.H + head;
    if constexpr (DECAY != DECAY_KEY) in.gate = a.alpha[DECAY == DECAY_HEAD ? head : tok];
    if constexpr (DELTA) in.beta = a.beta[tok];
  };
  const auto spread = [](float* to, uint4 v) {   // 16 bytes of k or q as binary32
    if constexpr (BF16) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int h = 0; h < 2; ++h)
        reinterpret_cast<float4*>(to)[h] = make_float4(bf16_lo(w[2 * h]), bf16_hi(w[2 * h]), bf16_lo(w[2 * h + 1]), bf16_hi(w[2 * h + 1]));
    } else {
      *reinterpret_cast<uint4*>(to) = v;
    }
  };
  load(sp.begin);
  for (int t0 = sp.begin; t0 < sp.end; t0 += kTokBlock) {
    const int n = min(kTokBlock, sp.end - t0);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int x = tid + NT * j;
      if (NP * NT == kTokBlock * PR || x < kTokBlock * PR) {
        spread(&sk[x / PR][x % PR * (16 / E)], in.k[j]);
        spread(&sq[x / PR][x % PR * (16 / E)], in.q[j]);
      }
    }
    if constexpr (NA > 0) {
#pragma unroll
      for (int j = 0; j < NA; ++j) {
        const int x = tid + NT * j;
        if (NA * NT == kTokBlock * PA || x < kTokBlock * PA) *reinterpret_cast<uint4*>(&sa[x / PA][x % PA * 4]) = in.al[j];
      }
    }
    if (tid < 4 * kTokBlock) *reinterpret_cast<uint4*>(&sv[tid / 4][tid % 4 * 4]) = make_uint4(in.v[0], in.v[1], in.v[2], in.v[3]);
    if (tid < kTokBlock) {
      if constexpr (DECAY != DECAY_KEY) sg[tid] = in.gate;
      if constexpr (DELTA) sb[tid] = in.beta;
    }
    __syncthreads();
    if (sp.end - t0 > kTokBlock) load(t0 + kTokBlock);
    for (int t = 0; t < n; ++t) {
      f32x4 u{0.0f, 0.0f, 0.0f, 0.0f}, p{0.0f, 0.0f, 0.0f, 0.0f}, k[QR];
      float e = sv[t][c];
#pragma unroll
      for (int j = 0; j < QR; ++j) {
        const int row = 4 * (rg + RG * j);
        k[j] = *reinterpret_cast<const f32x4*>(&sk[t][row]);
        if constexpr (DECAY == DECAY_KEY) S[j] *= *reinterpret_cast<const f32x4*>(&sa[t][row]);
        else S[j] *= sg[t];
        if constexpr (DELTA) {
#pragma unroll
          for (int i = 0; i < 4; ++i) u[i] = fmaf(k[j][i], S[j][i], u[i]);
        }
      }
      if constexpr (DELTA) e = sb[t] * (e - sum_lanes<RG>((u[0] + u[1]) + (u[2] + u[3])));
#pragma unroll
      for (int j = 0; j < QR; ++j) {
        const f32x4 q = *reinterpret_cast<const f32x4*>(&sq[t][4 * (rg + RG * j)]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          S[j][i] = fmaf(k[j][i], e, S[j][i]);
          p[i] = fmaf(q[i], S[j][i], p[i]);
        }
      }
      const float o = sum_lanes<RG>((p[0] + p[1]) + (p[2] + p[3]));
      if (rg == 0) {
        const int64_t at = (int64_t(t0 + t) * a.H + head) * D + c0 + c;
        if constexpr (BF16) reinterpret_cast<uint16_t*>(a.out)[at] = float_to_bf16_bits(o);
        else reinterpret_cast<float*>(a.out)[at] = o;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < QR; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) pool[(4 * RG * j + i) * D] = S[j][i];
}

template <int D>
hipError_t linear_step_d(int decay, int bf16, const StepArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.B) * static_cast<unsigned>(a.H)), block(LinGeo<D>::NT);
  with_decay(decay, [&]<int DECAY>() {
    if (bf16) hipLaunchKernelGGL((linear_step_kernel<D, DECAY, 1>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((linear_step_kernel<D, DECAY, 0>), grid, block, 0, s, a);
  });
  return hipGetLastError();
}

template <int D>
hipError_t prompt_token_d(bool delta, int decay, int bf16, const PromptArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.B) * static_cast<unsigned>(a.H) * (D / 16)), block(TokGeo<D>::NT);
  with_decay(decay, [&]<int DECAY>() {
    if (delta) {
      if constexpr (DECAY != DECAY_HEAD) {   // the delta rule takes no fixed decays
        if (bf16) hipLaunchKernelGGL((prompt_token_kernel<D, true, DECAY, 1>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((prompt_token_kernel<D, true, DECAY, 0>), grid, block, 0, s, a);
      }
    } else {
      if (bf16) hipLaunchKernelGGL((prompt_token_kernel<D, false, DECAY, 1>), grid, block, 0, s, a);
      else hipLaunchKernelGGL((prompt_token_kernel<D, false, DECAY, 0>), grid, block, 0, s, a);
    }
  });
  return hipGetLastError();
}

}  // namespace

int linear_step_threads(int d) { return lin_threads(d); }

hipError_t launch_linear_step(int d, int decay, int bf16, const StepArgs& a, hipStream_t s) {
  switch (d) {
    case 16: return linear_step_d<16>(decay, bf16, a, s);
    case 32: return linear_step_d<32>(decay, bf16, a, s);
    case 64: return linear_step_d<64>(decay, bf16, a, s);
    case 128: return linear_step_d<128>(decay, bf16, a, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_prompt_token(int d, bool delta, int decay, int bf16, const PromptArgs& a, hipStream_t s) {
  switch (d) {
    case 16: return prompt_token_d<16>(delta, decay, bf16, a, s);
    case 32: return prompt_token_d<32>(delta, decay, bf16, a, s);
    case 64: return prompt_token_d<64>(delta, decay, bf16, a, s);
    case 128: return prompt_token_d<128>(delta, decay, bf16, a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace damp
