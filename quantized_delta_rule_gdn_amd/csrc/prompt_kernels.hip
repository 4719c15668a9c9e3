// prompt_kernels.hip -- gfx950 kernels of the chunked prompt forms on the matrix cores: linear
// attention with a decay per head, and the gated delta rule, for bf16 inputs and d in {64, 128}.
//
// With G_t the running sum of log2 a over a chunk of 64 tokens and S the state before it,
//   o_t   = 2^G_t S^T q_t + sum_{s <= t} 2^(G_t - G_s) (q_t . k_s) e_s        (P = the weights)
//   S_out = 2^G_C S + sum_s 2^(G_C - G_s) k_s e_s^T
// with e = v for linear attention. For the delta rule e solves (I + A) E = diag(b) (V - 2^G K S),
// A_ts = b_t 2^(G_t - G_s) (k_t . k_s) for s < t: X = (I + A)^-1 only depends on the chunk's keys and
// gates, so every chunk's X diag(b) and P are formed at once, in parallel over the prompt, and the
// chain from chunk to chunk is left with products of the state.
//
// Numerics. All exponents are differences of the same running sums, held as two binary32 numbers
// each (a binary64 sum, split), so every decay is good to about 2^-23 whatever the sums reach. Keys,
// queries and values are exact bf16 operands; the state, E and X enter a product as bf16 pieces
// (prompt_common.h): three where the result feeds the state (2^-24), two where it is a readout that
// bf16 rounds at 2^-9. The state itself and all sums are binary32.
#include <algorithm>

#include "prompt_common.h"

namespace damp {
namespace {

constexpr int kC = 64;         // tokens per chunk
constexpr int kLd = kC + 8;    // LDS row of a chunk-wide bf16 array: 144 bytes, 16-byte aligned

// Chunks (or segments of `len` tokens) are numbered without a table: those of request b start at
// begin_b / len + b, which leaves room for each request's last, short one; some numbers are unused.
struct Piece {
  int b, t0, n;   // n = 0: none
};

__device__ __forceinline__ Piece piece_of(const PromptArgs& a, int i, int len) {
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (span_of(a, mid).begin / len + mid <= i) lo = mid; else hi = mid;
  }
  const Span sp = span_of(a, lo);
  const int j = i - (sp.begin / len + lo);
  const int64_t t0 = sp.begin + int64_t(j) * len;
  if (j < 0 || t0 >= sp.end) return Piece{lo, 0, 0};
  return Piece{lo, static_cast<int>(t0), min(len, static_cast<int>(sp.end - t0))};
}

// One lane's running sum of log2 decays over a chunk (lane = token; tokens past n add nothing).
template <int DECAY>
__device__ __forceinline__ double chunk_logs(const PromptArgs& a, int t0, int n, int head, int lane) {
  float l = 0.0f;
  if (lane < n) l = log2_decay(a.alpha[DECAY == DECAY_HEAD ? head : (int64_t(t0 + lane) * a.H + head)]);
  return wave_scan(static_cast<double>(l), lane);
}

struct Logs {   // G = hi + lo
  float hi, lo;
};

__device__ __forceinline__ Logs split_logs(double g) {
  const float hi = static_cast<float>(g);
  return Logs{hi, static_cast<float>(g - hi)};
}

__device__ __forceinline__ float decay_between(Logs t, Logs s) { return pow2((t.hi - s.hi) + (t.lo - s.lo)); }

// ---- the delta rule: what a chunk's keys and gates give -------------------------------------
// Workspace of one chunk and head: X diag(b) in three bf16 pieces and P in two, [64][64] each, then
// 2^G_t and 2^(G_C - G_t).
constexpr int kPlane = kC * kC * 2;
constexpr int kDeltaUnit = 5 * kPlane + 2 * kC * 4;

__device__ __forceinline__ f32x4 mul16(const float* A, const float* B, int ld, f32x4 c, int r, int g) {
#pragma unroll
  for (int x = 0; x < 4; ++x) c = mfma_f32(A[r * ld + 4 * x + g], B[(4 * x + g) * ld + r], c);
  return c;
}

// A (16 x 16 in LDS) times a C tile still in registers: k step i pairs column 4 g + i with row 4 g + i.
__device__ __forceinline__ f32x4 mul16_tile(const float* A, f32x4 m, int ld, f32x4 c, int r, int g) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = mfma_f32(A[r * ld + 4 * g + i], m[i], c);
  return c;
}

// One workgroup per (chunk, head); wave w takes token rows 16 w .. + 15. X comes from the blocks of
// 16: each wave inverts its diagonal block by forward substitution (a column per lane), then
// blocks are joined two by two, [[X, 0], [Y, Z]]^-1 = [[X', 0], [-Z' Y X', Z']], with binary32
// matrix instructions: no power of A is formed, so the result is as good as forward substitution.
template <int D>
__global__ __launch_bounds__(256) void delta_chunk_kernel(const PromptArgs a) {
  constexpr int KS = D / 32, LK = D + 8, LF = kC + 4;
  __shared__ __align__(16) float pf[kC][LF];   // the keys (bf16 rows of LK), later P
  __shared__ __align__(16) float af[kC][LF], xf[kC][LF];
  __shared__ Logs logs[kC];
  __shared__ float beta[kC];
  static_assert(LK * 2 <= LF * 4, "the keys fit P's rows");
  uint16_t* ks = reinterpret_cast<uint16_t*>(pf);
  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int unit = __builtin_amdgcn_workgroup_id_x();
  const int head = unit % a.H;
  const Piece pc = piece_of(a, unit / a.H, kC);
  if (pc.n <= 0) return;
  uint8_t* ws = a.ws + int64_t(unit) * kDeltaUnit;
  const int64_t row0 = (int64_t(pc.t0) * a.H + head) * D, rstep = int64_t(a.H) * D;
  const uint16_t* kp = static_cast<const uint16_t*>(a.k);
  const uint16_t* qp = static_cast<const uint16_t*>(a.q);

  // rows past the chunk's end repeat its last: beta = 0 there, so nothing comes of them
  for (int x = tid; x < kC * (D / 8); x += 256) {
    const int t = x / (D / 8), c = x % (D / 8);
    *reinterpret_cast<uint4*>(ks + t * LK + c * 8) = *reinterpret_cast<const uint4*>(kp + row0 + min(t, pc.n - 1) * rstep + c * 8);
  }
  Frag qf[KS];
#pragma unroll
  for (int x = 0; x < KS; ++x) qf[x] = load_frag(qp + row0 + min(16 * w + r, pc.n - 1) * rstep + x * 32 + g * 8);
  if (w == 0) {
    const double gs = chunk_logs<DECAY_SCALAR>(a, pc.t0, pc.n, head, lane);
    const double end = __shfl(gs, 63);
    logs[lane] = split_logs(gs);
    beta[lane] = lane < pc.n ? a.beta[int64_t(pc.t0 + lane) * a.H + head] : 0.0f;
    float* sc = reinterpret_cast<float*>(ws + 5 * kPlane);
    sc[lane] = pow2(static_cast<float>(gs));
    sc[kC + lane] = pow2(static_cast<float>(end - gs));
  }
  __syncthreads();

  f32x4 kk[4], qk[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    kk[c] = qk[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (c > w) continue;   // above the diagonal
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      const Frag b = load_frag(ks + (16 * c + r) * LK + x * 32 + g * 8);
      kk[c] = mfma(load_frag(ks + (16 * w + r) * LK + x * 32 + g * 8), b, kk[c]);
      qk[c] = mfma(qf[x], b, qk[c]);
    }
    const int s = 16 * c + r;
    const Logs ls = logs[s];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * w + 4 * g + i;
      const float f = decay_between(logs[t], ls);
      kk[c][i] = s < t ? beta[t] * f * kk[c][i] : 0.0f;
      qk[c][i] = s <= t ? f * qk[c][i] : 0.0f;
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      af[16 * w + 4 * g + i][16 * c + r] = kk[c][i];
      xf[16 * w + 4 * g + i][16 * c + r] = 0.0f;
    }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) pf[16 * w + 4 * g + i][16 * c + r] = qk[c][i];

  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float acc = i == r ? 1.0f : 0.0f;
#pragma unroll
    for (int j = 0; j < i; ++j) acc = fmaf(-af[16 * w + i][16 * w + j], x[j], acc);
    x[i] = acc;
  }
  if (g == 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) xf[16 * w + i][16 * w + r] = x[i];
  }
  __syncthreads();
  const f32x4 zero{0.0f, 0.0f, 0.0f, 0.0f};
  if (w < 2) {
    const int lo = 32 * w, hi = lo + 16;
    const f32x4 m = mul16(&af[hi][lo], &xf[lo][lo], LF, zero, r, g);
    const f32x4 o = mul16_tile(&xf[hi][hi], m, LF, zero, r, g);
#pragma unroll
    for (int i = 0; i < 4; ++i) xf[hi + 4 * g + i][lo + r] = -o[i];
  }
  __syncthreads();
  if (w < 2) {
    const int c = 16 * w;
    f32x4 m0 = zero, m1 = zero;
    for (int k = c; k < 32; k += 16) {
      m0 = mul16(&af[32][k], &xf[k][c], LF, m0, r, g);
      m1 = mul16(&af[48][k], &xf[k][c], LF, m1, r, g);
    }
    const f32x4 o0 = mul16_tile(&xf[32][32], m0, LF, zero, r, g);
    const f32x4 o1 = mul16_tile(&xf[48][48], m1, LF, mul16_tile(&xf[48][32], m0, LF, zero, r, g), r, g);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      xf[32 + 4 * g + i][c + r] = -o0[i];
      xf[48 + 4 * g + i][c + r] = -o1[i];
    }
  }
  __syncthreads();
  // 16 values of one row per thread: X's columns scaled by beta, in three pieces; P in two
  const int t = tid >> 2, c0 = (tid & 3) * 16;
  uint32_t px[3][8], pp[2][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t u[3];
    split_bf16<3>(xf[t][c0 + 2 * j] * beta[c0 + 2 * j], xf[t][c0 + 2 * j + 1] * beta[c0 + 2 * j + 1], u);
    px[0][j] = u[0]; px[1][j] = u[1]; px[2][j] = u[2];
    split_bf16<2>(pf[t][c0 + 2 * j], pf[t][c0 + 2 * j + 1], u);
    pp[0][j] = u[0]; pp[1][j] = u[1];
  }
  uint4* dst = reinterpret_cast<uint4*>(ws + (t * kC + c0) * 2);
#pragma unroll
  for (int p = 0; p < 3; ++p)
#pragma unroll
    for (int h = 0; h < 2; ++h) dst[p * (kPlane / 16) + h] = make_uint4(px[p][4 * h], px[p][4 * h + 1], px[p][4 * h + 2], px[p][4 * h + 3]);
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int h = 0; h < 2; ++h) dst[(3 + p) * (kPlane / 16) + h] = make_uint4(pp[p][4 * h], pp[p][4 * h + 1], pp[p][4 * h + 2], pp[p][4 * h + 3]);
}

// ---- the delta rule: the chain over the chunks ---------------------------------------------
// One workgroup of 4 waves per (request, head, 16 NT value columns): a chunk's work is split over
// token rows (16 per wave) and, for the state's update, key channels (D / 4 per wave), so a wave
// loads only its own rows of K, Q, X and P, straight into operand registers, one chunk ahead; the
// state, R and E change hands in LDS as [column][k] arrays of bf16 pieces. Three barriers a chunk.
// What bounds it is the chain's latency: about 50 NT dependent-by-stages matrix instructions a wave.
template <int D>
struct DeltaRows {   // one wave's operands of a chunk
  Frag k[D / 32], q[D / 32];
  Frag x[3][2], p[2][2];
  uint32_t kt[2][8];     // keys of tokens 32 x + 8 g + j, this lane's D / 64 channels
  float4 eg, wc;         // 2^G and 2^(G_C - G) of rows 16 w + 4 g .. + 3
  float last;            // 2^G_C
};

template <int D, int NT>
__global__ __launch_bounds__(256) void delta_chain_kernel(const PromptArgs a) {
  constexpr int KS = D / 32, MD = D / 64, LS = D + 8, NC = 16 * NT;
  __shared__ __align__(16) uint16_t sp[3][NC][LS];
  __shared__ __align__(16) uint16_t rp[3][NC][kLd], ep[2][NC][kLd], wp[3][NC][kLd];
  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  constexpr int slices = D / NC;
  unsigned id = __builtin_amdgcn_workgroup_id_x();
  const int c0 = (id % slices) * NC;
  id /= slices;
  const int head = id % a.H, b = id / a.H;
  const int64_t slot = a.slot_idx[b];
  if (!slot_in_pool(slot, a.num_slots)) return;
  const Span sp_b = span_of(a, b);
  if (sp_b.end <= sp_b.begin) return;
  const int64_t rstep = int64_t(a.H) * D;
  const uint16_t* kp = static_cast<const uint16_t*>(a.k) + int64_t(head) * D;
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + int64_t(head) * D;
  const uint16_t* vp = static_cast<const uint16_t*>(a.v) + int64_t(head) * D + c0;
  uint16_t* op = static_cast<uint16_t*>(a.out) + int64_t(head) * D + c0;
  const int own = (D / 4) * w;                      // this wave's first key channel of the state
  float* pool = a.pool + ((slot * a.H + head) * D + own + MD * 4 * g) * int64_t(D) + c0 + r;

  f32x4 S[MD][NT];   // S[m][nt][i]: key channel own + MD (4 g + i) + m, column c0 + 16 nt + r
  const bool resume = a.resume && a.resume[b] != 0;
#pragma unroll
  for (int m = 0; m < MD; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[m][nt][i] = resume ? pool[(MD * i + m) * D + 16 * nt] : 0.0f;

  const auto share_state = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t u[2 * MD][3];
#pragma unroll
      for (int j = 0; j < 2 * MD; ++j) {
        if constexpr (MD == 2) split_bf16<3>(S[0][nt][j], S[1][nt][j], u[j]);
        else split_bf16<3>(S[0][nt][2 * j], S[0][nt][2 * j + 1], u[j]);
      }
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        uint16_t* dst = &sp[p][16 * nt + r][own + MD * 4 * g];
        if constexpr (MD == 2) *reinterpret_cast<uint4*>(dst) = make_uint4(u[0][p], u[1][p], u[2][p], u[3][p]);
        else *reinterpret_cast<uint2*>(dst) = make_uint2(u[0][p], u[1][p]);
      }
    }
  };
  DeltaRows<D> f;
  uint16_t vv[NT][4];
  // rows past the last token repeat it: their beta is 0, so E is 0 there
  const auto load_kqv = [&](int t0) {
    const int64_t at = min(t0 + 16 * w + r, sp_b.end - 1) * rstep + g * 8;
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      f.k[x] = load_frag(kp + at + x * 32);
      f.q[x] = load_frag(qp + at + x * 32);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) vv[nt][i] = vp[min(t0 + 16 * w + 4 * g + i, sp_b.end - 1) * rstep + 16 * nt + r];
  };
  const auto unit_ws = [&](int t0) {
    const int64_t i = sp_b.begin / kC + b + (t0 - sp_b.begin) / kC;
    return a.ws + (i * a.H + head) * kDeltaUnit;
  };
  const auto load_x = [&](int t0) {
    const uint8_t* ws = unit_ws(t0) + ((16 * w + r) * kC + g * 8) * 2;
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (x == 0 || w >= 2) f.x[p][x] = load_frag(ws + p * kPlane + x * 64);
  };
  const auto load_rest = [&](int t0) {
    const uint8_t* ws = unit_ws(t0) + ((16 * w + r) * kC + g * 8) * 2 + 3 * kPlane;
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (x == 0 || w >= 2) f.p[p][x] = load_frag(ws + p * kPlane + x * 64);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint16_t* p = kp + min(t0 + 32 * x + 8 * g + j, sp_b.end - 1) * rstep + own + MD * r;
        f.kt[x][j] = MD == 2 ? *reinterpret_cast<const uint32_t*>(p) : *p;
      }
  };
  const auto load_gates = [&](int t0) {
    const float* sc = reinterpret_cast<const float*>(unit_ws(t0) + 5 * kPlane);
    f.eg = *reinterpret_cast<const float4*>(sc + 16 * w + 4 * g);
    f.wc = *reinterpret_cast<const float4*>(sc + kC + 16 * w + 4 * g);
    f.last = sc[kC - 1];
  };

  load_kqv(sp_b.begin);
  load_x(sp_b.begin);
  load_rest(sp_b.begin);
  load_gates(sp_b.begin);
  share_state();
  __syncthreads();
  for (int t0 = sp_b.begin; t0 < sp_b.end; t0 += kC) {
    const bool more = sp_b.end - t0 > kC;
    const float eg[4] = {f.eg.x, f.eg.y, f.eg.z, f.eg.w}, wc[4] = {f.wc.x, f.wc.y, f.wc.z, f.wc.w};
    const float last = f.last;
    // K S and Q S; R = V - 2^G K S
    f32x4 ks[NT], o[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      ks[nt] = o[nt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = 0; x < KS; ++x)
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          const Frag s = load_frag(&sp[p][16 * nt + r][x * 32 + g * 8]);
          ks[nt] = mfma(f.k[x], s, ks[nt]);
          if (p < 2) o[nt] = mfma(f.q[x], s, o[nt]);
        }
      float rr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        rr[i] = fmaf(-eg[i], ks[nt][i], __uint_as_float(uint32_t(vv[nt][i]) << 16));
        o[nt][i] *= eg[i];
      }
      uint32_t u0[3], u1[3];
      split_bf16<3>(rr[0], rr[1], u0);
      split_bf16<3>(rr[2], rr[3], u1);
#pragma unroll
      for (int p = 0; p < 3; ++p) *reinterpret_cast<uint2*>(&rp[p][16 * nt + r][16 * w + 4 * g]) = make_uint2(u0[p], u1[p]);
    }
    if (more) load_kqv(t0 + kC);
    __syncthreads();
    // E = X diag(b) R
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4 e{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (x == 1 && w < 2) continue;   // X is lower triangular
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          const Frag rf = load_frag(&rp[j][16 * nt + r][x * 32 + g * 8]);
#pragma unroll
          for (int i = 0; i + j < 3; ++i) e = mfma(f.x[i][x], rf, e);
        }
      }
      uint32_t u0[3], u1[3];
      split_bf16<2>(e[0], e[1], u0);
      split_bf16<2>(e[2], e[3], u1);
#pragma unroll
      for (int p = 0; p < 2; ++p) *reinterpret_cast<uint2*>(&ep[p][16 * nt + r][16 * w + 4 * g]) = make_uint2(u0[p], u1[p]);
      split_bf16<3>(e[0] * wc[0], e[1] * wc[1], u0);
      split_bf16<3>(e[2] * wc[2], e[3] * wc[3], u1);
#pragma unroll
      for (int p = 0; p < 3; ++p) *reinterpret_cast<uint2*>(&wp[p][16 * nt + r][16 * w + 4 * g]) = make_uint2(u0[p], u1[p]);
    }
    if (more) load_x(t0 + kC);
    __syncthreads();
    // S = 2^G_C S + K^T (2^(G_C - G) E) first: the next chunk waits for it
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int m = 0; m < MD; ++m) S[m][nt] *= last;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        Frag kt[MD];
#pragma unroll
        for (int m = 0; m < MD; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            kt[m].w[j] = __builtin_amdgcn_perm(f.kt[x][2 * j + 1], f.kt[x][2 * j], m ? 0x07060302u : 0x05040100u);
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          const Frag ef = load_frag(&wp[p][16 * nt + r][x * 32 + g * 8]);
#pragma unroll
          for (int m = 0; m < MD; ++m) S[m][nt] = mfma(kt[m], ef, S[m][nt]);
        }
      }
    }
    share_state();
    // O = 2^G Q S + P E
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (x == 1 && w < 2) continue;
        const Frag e0 = load_frag(&ep[0][16 * nt + r][x * 32 + g * 8]), e1 = load_frag(&ep[1][16 * nt + r][x * 32 + g * 8]);
        o[nt] = mfma(f.p[0][x], e0, o[nt]);
        o[nt] = mfma(f.p[1][x], e0, o[nt]);
        o[nt] = mfma(f.p[0][x], e1, o[nt]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = t0 + 16 * w + 4 * g + i;
        if (t < sp_b.end) op[t * rstep + 16 * nt + r] = float_to_bf16_bits(o[nt][i]);
      }
    }
    if (more) {
      load_rest(t0 + kC);
      load_gates(t0 + kC);
    }
    __syncthreads();
  }
#pragma unroll
  for (int m = 0; m < MD; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) pool[(MD * i + m) * D + 16 * nt] = S[m][nt][i];
}

// ---- linear attention ------------------------------------------------------------------------
// One workgroup of 4 waves per (segment of a prompt, head); wave w owns the value columns D / 4 * w
// .. of the state, the values and the readouts, so between the chunks nothing of the state leaves
// its registers: as the B operand of Q S it is the accumulator tiles as they stand (k permuted:
// mfma), and Q is read to match. K, Q and K^T are staged in LDS once per chunk for all waves, P is
// formed by 16 rows per wave. Long prompts of few heads are cut into segments: a first launch
// (STATES) sums every segment's own state, a scan turns them into the states before each segment,
// and the readouts of all segments run at once.
enum LinearMode : int { LIN_WHOLE = 0, LIN_STATES = 1, LIN_SEGMENTS = 2 };

struct Segments {
  int len;          // tokens per segment, a multiple of 64; whole prompts: larger than any
  float* states;    // [segment number][H][D][D]: own states, then the states before
  float* decays;    // [segment number][H]: log2 of a segment's decay
};

template <int D, int DECAY, int MODE>
__global__ __launch_bounds__(256) void linear_chunk_kernel(const PromptArgs a, const Segments sg) {
  constexpr int KS = D / 32, MD = D / 64, XT = D / 16, LK = D + 8;
  constexpr bool kReadout = MODE != LIN_STATES;
  __shared__ __align__(16) uint16_t qs[kReadout ? kC : 1][LK], ks[kReadout ? kC : 1][LK];
  __shared__ __align__(16) uint16_t kt[D][kLd];
  __shared__ __align__(16) uint16_t pp[2][kReadout ? kC : 1][kLd];
  __shared__ Logs logs[2][kC];
  __shared__ __align__(16) float eg[2][kC], wc[2][kC];
  __shared__ double ends[2];
  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int unit = __builtin_amdgcn_workgroup_id_x();
  const int head = unit % a.H, seg = unit / a.H;
  int b = seg, t_begin, t_end;
  if constexpr (MODE == LIN_WHOLE) {
    const Span sp = span_of(a, b);
    t_begin = sp.begin;
    t_end = sp.end;
  } else {
    const Piece pc = piece_of(a, seg, sg.len);
    b = pc.b;
    t_begin = pc.t0;
    t_end = pc.t0 + pc.n;
  }
  if (t_end <= t_begin) return;
  const bool final = MODE == LIN_WHOLE || t_end == span_of(a, b).end;
  if (MODE == LIN_STATES && final) return;      // no segment waits for the last one's state
  const int64_t slot = a.slot_idx[b];
  if (!slot_in_pool(slot, a.num_slots)) return;
  const int64_t rstep = int64_t(a.H) * D;
  const uint16_t* kp = static_cast<const uint16_t*>(a.k) + int64_t(head) * D;
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + int64_t(head) * D;
  const int col = (D / 4) * w + MD * r;           // this lane's first value column
  const uint16_t* vp = static_cast<const uint16_t*>(a.v) + int64_t(head) * D + col;
  uint16_t* op = static_cast<uint16_t*>(a.out) + int64_t(head) * D + col;
  float* pool = a.pool + ((slot * a.H + head) * D) * int64_t(D) + col;
  float* states = MODE == LIN_WHOLE ? nullptr : sg.states + int64_t(unit) * D * D + col;

  f32x4 S[XT][MD];   // S[x][m][i]: key channel 16 x + 4 g + i, value column col + m
  {
    const float* from = MODE == LIN_SEGMENTS ? states : MODE == LIN_WHOLE && a.resume && a.resume[b] != 0 ? pool : nullptr;
#pragma unroll
    for (int x = 0; x < XT; ++x)
#pragma unroll
      for (int m = 0; m < MD; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[x][m][i] = from ? from[(16 * x + 4 * g + i) * D + m] : 0.0f;
  }

  // one chunk's rows, in registers until LDS is free for them: rows past the end are zero
  constexpr int RW = D / 32;                      // 16-byte pieces of K (and of Q) per thread
  uint4 kr[RW], qr[RW];
  uint32_t tr[2][8], vr[2][8];                    // K by columns (64 channel groups x 8 token octets), V
  const auto load_rows = [&](int t0) {
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      const int x = tid + 256 * j, t = t0 + x / (D / 8), c = x % (D / 8);
      if constexpr (kReadout) {
        const bool live = t < t_end;
        const int64_t at = min(t, t_end - 1) * rstep + c * 8;
        kr[j] = *reinterpret_cast<const uint4*>(kp + at);
        qr[j] = *reinterpret_cast<const uint4*>(qp + at);
        if (!live) kr[j] = qr[j] = make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int x = tid + 256 * j, c = x % 64, o = x / 64;   // channels MD c .., tokens 8 o ..
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int t = t0 + 8 * o + i;
        const uint16_t* p = kp + min(t, t_end - 1) * rstep + MD * c;
        tr[j][i] = MD == 2 ? *reinterpret_cast<const uint32_t*>(p) : *p;
        if (t >= t_end) tr[j][i] = 0;
      }
    }
  };
  const auto load_v = [&](int t0) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int t = t0 + 32 * x + 8 * g + j;
        const uint16_t* p = vp + min(t, t_end - 1) * rstep;
        vr[x][j] = MD == 2 ? *reinterpret_cast<const uint32_t*>(p) : *p;
        if (t >= t_end) vr[x][j] = 0;
      }
  };
  const auto store_logs = [&](int t0, int to) {   // by one wave, a chunk ahead
    const double gs = chunk_logs<DECAY>(a, t0, min(kC, t_end - t0), head, lane);
    const double end = __shfl(gs, 63);
    logs[to][lane] = split_logs(gs);
    eg[to][lane] = pow2(static_cast<float>(gs));
    wc[to][lane] = pow2(static_cast<float>(end - gs));
    if (lane == 0) ends[to] = end;
  };

  double total = 0.0;
  load_rows(t_begin);
  load_v(t_begin);
  if (w == 0) store_logs(t_begin, 0);
  int at = 0;
  for (int t0 = t_begin; t0 < t_end; t0 += kC, at ^= 1) {
    const bool more = t_end - t0 > kC;
    if constexpr (kReadout) {
#pragma unroll
      for (int j = 0; j < RW; ++j) {
        const int x = tid + 256 * j;
        *reinterpret_cast<uint4*>(&ks[x / (D / 8)][(x % (D / 8)) * 8]) = kr[j];
        *reinterpret_cast<uint4*>(&qs[x / (D / 8)][(x % (D / 8)) * 8]) = qr[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int x = tid + 256 * j, c = x % 64, o = x / 64;
#pragma unroll
      for (int m = 0; m < MD; ++m) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = __builtin_amdgcn_perm(tr[j][2 * i + 1], tr[j][2 * i], m ? 0x07060302u : 0x05040100u);
        *reinterpret_cast<uint4*>(&kt[MD * c + m][8 * o]) = make_uint4(u[0], u[1], u[2], u[3]);
      }
    }
    __syncthreads();
    if (more) load_rows(t0 + kC);
    if constexpr (kReadout) {
      Frag qf[KS];
#pragma unroll
      for (int x = 0; x < KS; ++x) qf[x] = load_frag(&qs[16 * w + r][x * 32 + g * 8]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        f32x4 p{0.0f, 0.0f, 0.0f, 0.0f};
        const int s = 16 * c + r;
        if (c <= w) {
#pragma unroll
          for (int x = 0; x < KS; ++x) p = mfma(qf[x], load_frag(&ks[s][x * 32 + g * 8]), p);
          const Logs ls = logs[at][s];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = 16 * w + 4 * g + i;
            p[i] = s <= t ? p[i] * decay_between(logs[at][t], ls) : 0.0f;
          }
        }
        if ((c | 1) > (w | 1)) continue;          // no product reads these
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          uint32_t u[2];
          split_bf16<2>(p[i], p[i + 1], u);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            pp[x][16 * w + 4 * g + i][s] = static_cast<uint16_t>(u[x]);
            pp[x][16 * w + 4 * g + i + 1][s] = static_cast<uint16_t>(u[x] >> 16);
          }
        }
      }
      __syncthreads();
      f32x4 o[4][MD];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int m = 0; m < MD; ++m) o[rt][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        Frag sf[2][MD];
#pragma unroll
        for (int m = 0; m < MD; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t u[2];
            split_bf16<2>(S[2 * x + j / 2][m][2 * (j & 1)], S[2 * x + j / 2][m][2 * (j & 1) + 1], u);
            sf[0][m].w[j] = u[0];
            sf[1][m].w[j] = u[1];
          }
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          const Frag q = load_frag2(&qs[16 * rt + r][x * 32 + g * 4], &qs[16 * rt + r][x * 32 + 16 + g * 4]);
#pragma unroll
          for (int m = 0; m < MD; ++m) {
            o[rt][m] = mfma(q, sf[0][m], o[rt][m]);
            o[rt][m] = mfma(q, sf[1][m], o[rt][m]);
          }
        }
      }
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) {
        const float4 e = *reinterpret_cast<const float4*>(&eg[at][16 * rt + 4 * g]);
#pragma unroll
        for (int m = 0; m < MD; ++m) {
          o[rt][m][0] *= e.x; o[rt][m][1] *= e.y; o[rt][m][2] *= e.z; o[rt][m][3] *= e.w;
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        Frag vf[MD];
#pragma unroll
        for (int m = 0; m < MD; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            vf[m].w[j] = __builtin_amdgcn_perm(vr[x][2 * j + 1], vr[x][2 * j], m ? 0x07060302u : 0x05040100u);
#pragma unroll
        for (int rt = 2 * x; rt < 4; ++rt)         // tokens 32 x .. reach rows from 32 x on
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const Frag pf = load_frag(&pp[p][16 * rt + r][x * 32 + g * 8]);
#pragma unroll
            for (int m = 0; m < MD; ++m) o[rt][m] = mfma(pf, vf[m], o[rt][m]);
          }
      }
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = t0 + 16 * rt + 4 * g + i;
          if (t < t_end) {
            if constexpr (MD == 2) *reinterpret_cast<uint32_t*>(op + t * rstep) = pack_bf16(o[rt][0][i], o[rt][1][i]);
            else op[t * rstep] = float_to_bf16_bits(o[rt][0][i]);
          }
        }
    }
    // S = 2^G_C S + K^T (2^(G_C - G) V)
    const float last = pow2(static_cast<float>(ends[at]));
    total += ends[at];
#pragma unroll
    for (int x = 0; x < XT; ++x)
#pragma unroll
      for (int m = 0; m < MD; ++m) S[x][m] *= last;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      Frag vf[3][MD];
      const float4 w0 = *reinterpret_cast<const float4*>(&wc[at][32 * x + 8 * g]), w1 = *reinterpret_cast<const float4*>(&wc[at][32 * x + 8 * g + 4]);
      const float f[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int m = 0; m < MD; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = vr[x][2 * j], hi = vr[x][2 * j + 1];
          uint32_t u[3];
          split_bf16<3>((m ? bf16_hi(lo) : bf16_lo(lo)) * f[2 * j], (m ? bf16_hi(hi) : bf16_lo(hi)) * f[2 * j + 1], u);
#pragma unroll
          for (int p = 0; p < 3; ++p) vf[p][m].w[j] = u[p];
        }
#pragma unroll
      for (int y = 0; y < XT; ++y) {
        const Frag kf = load_frag(&kt[16 * y + r][x * 32 + g * 8]);
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int m = 0; m < MD; ++m) S[y][m] = mfma(kf, vf[p][m], S[y][m]);
      }
    }
    if (more) {
      load_v(t0 + kC);
      if (w == 0) store_logs(t0 + kC, at ^ 1);
    }
    __syncthreads();
  }
  float* to = MODE == LIN_STATES ? states : final ? pool : nullptr;
  if (to) {
#pragma unroll
    for (int x = 0; x < XT; ++x)
#pragma unroll
      for (int m = 0; m < MD; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) to[(16 * x + 4 * g + i) * D + m] = S[x][m][i];
  }
  if (MODE == LIN_STATES && tid == 0) sg.decays[unit] = static_cast<float>(total);
}

// The segments' own states turned into the states before each segment, 4 values a thread.
__global__ __launch_bounds__(256) void linear_scan_kernel(const PromptArgs a, const Segments sg, int dd4) {
  const int64_t x = int64_t(__builtin_amdgcn_workgroup_id_x()) * 256 + __builtin_amdgcn_workitem_id_x();
  const int64_t u = x / dd4;
  if (u >= int64_t(a.B) * a.H) return;
  const int b = static_cast<int>(u / a.H), head = static_cast<int>(u - int64_t(b) * a.H), e = static_cast<int>(x - u * dd4);
  const int64_t slot = a.slot_idx[b];
  if (!slot_in_pool(slot, a.num_slots)) return;
  const Span sp = span_of(a, b);
  f32x4 in{0.0f, 0.0f, 0.0f, 0.0f};
  if (a.resume && a.resume[b] != 0 && sp.end > sp.begin)
    in = reinterpret_cast<const f32x4*>(a.pool + (slot * a.H + head) * dd4 * 4)[e];
  const int64_t first = sp.begin / sg.len + b;
  const int n = (sp.end - sp.begin + sg.len - 1) / sg.len;
  for (int j = 0; j < n; ++j) {
    const int64_t unit = (first + j) * a.H + head;
    f32x4* p = reinterpret_cast<f32x4*>(sg.states) + unit * dd4 + e;
    f32x4 own{0.0f, 0.0f, 0.0f, 0.0f};
    float f = 0.0f;
    if (j + 1 < n) {
      own = *p;
      f = pow2(sg.decays[unit]);
    }
    *p = in;
    in = in * f + own;
  }
}

// Segments of a call: none (whole prompts) where the prompts alone fill the chip.
int segment_len(int32_t B, int32_t T, int32_t H) {
  if (int64_t(B) * H >= 512 || T <= 4 * kC) return 0;
  const int64_t want = (int64_t(T) * H + 1023) / 1024;
  return static_cast<int>(std::max<int64_t>((want + kC - 1) / kC * kC, 4 * kC));
}

template <int D, int DECAY>
void linear_dd(const PromptArgs& a, hipStream_t s) {
  Segments sg{segment_len(a.B, a.T, a.H), nullptr, nullptr};
  if (sg.len == 0) {
    const dim3 grid(static_cast<unsigned>(a.B) * static_cast<unsigned>(a.H));
    hipLaunchKernelGGL((linear_chunk_kernel<D, DECAY, LIN_WHOLE>), grid, dim3(256), 0, s, a, sg);
    return;
  }
  const int64_t units = (int64_t(a.T / sg.len) + a.B) * a.H;
  sg.states = reinterpret_cast<float*>(a.ws);
  sg.decays = sg.states + units * D * D;
  const dim3 grid(static_cast<unsigned>(units));
  hipLaunchKernelGGL((linear_chunk_kernel<D, DECAY, LIN_STATES>), grid, dim3(256), 0, s, a, sg);
  const int64_t threads = int64_t(a.B) * a.H * (D * D / 4);
  hipLaunchKernelGGL(linear_scan_kernel, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, s, a, sg, D * D / 4);
  hipLaunchKernelGGL((linear_chunk_kernel<D, DECAY, LIN_SEGMENTS>), grid, dim3(256), 0, s, a, sg);
}

template <int D>
hipError_t linear_d(int decay, const PromptArgs& a, hipStream_t s) {
  if (decay == DECAY_HEAD) linear_dd<D, DECAY_HEAD>(a, s);
  else linear_dd<D, DECAY_SCALAR>(a, s);
  return hipGetLastError();
}

template <int D>
hipError_t delta_d(const PromptArgs& a, hipStream_t s) {
  const unsigned chunks = static_cast<unsigned>(a.T / kC + a.B) * static_cast<unsigned>(a.H);
  hipLaunchKernelGGL((delta_chunk_kernel<D>), dim3(chunks), dim3(256), 0, s, a);
  const unsigned units = static_cast<unsigned>(a.B) * static_cast<unsigned>(a.H);
  hipLaunchKernelGGL((delta_chain_kernel<D, 1>), dim3(units * (D / 16)), dim3(256), 0, s, a);
  return hipGetLastError();
}

// bf16 inputs with one decay per head run in chunks; the rest token by token.
bool chunked(int d, int decay, int bf16) { return bf16 && (d == 64 || d == 128) && decay != DECAY_KEY; }

}  // namespace

int64_t prefill_ws_bytes(bool delta, int d, int decay, int bf16, int32_t B, int32_t T, int32_t H) {
  if (!chunked(d, decay, bf16)) return 0;
  if (delta) return (int64_t(T) / kC + B) * H * kDeltaUnit;
  const int len = segment_len(B, T, H);
  return len ? (int64_t(T / len) + B) * H * (int64_t(d) * d + 1) * 4 : 0;
}

hipError_t launch_prefill(bool delta, int d, int decay, int bf16, const PromptArgs& a, hipStream_t s) {
  if (!chunked(d, decay, bf16)) return launch_prompt_token(d, delta, decay, bf16, a, s);
  if (!delta) return d == 64 ? linear_d<64>(decay, a, s) : linear_d<128>(decay, a, s);
  return d == 64 ? delta_d<64>(a, s) : delta_d<128>(a, s);
}

}  // namespace damp
