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
// Numerics. Exponents are sums of binary32 logarithms (v_log_f32, within 2^-23 of each, near 1 too), summed
// in binary64. Those between two tokens are differences of sums held as two binary32 numbers each, so that
// an exponent x is off by 2^-22 |x| at most whatever the sums themselves reach; 2^G_t, 2^(G_C - G_t), 2^G_C
// and the segments' decays start at a chunk's or segment's border and come from one binary32 exponent, to
// the same bound. A decay 2^x is then off by 2^-22 |x| ln 2 of itself and v_exp_f32's 2^-23: by less than
// 2^-22 of 1, while the relative error grows with |x| (2^-18 at 2^-16), as it does by the number of tokens
// where they are multiplied one by one. Keys, queries and values are exact bf16 operands; the state, E
// and X enter a product as bf16 pieces (prompt_common.h): three where the result feeds the state (2^-24; of
// X R the products of pieces i and j with i + j > 2, below 2^-24 of the product, are left out), two (2^-16)
// where it is a readout, whose rounding to bf16 is 2^-8. The state itself and all sums are binary32.
#include <algorithm>

#include "prompt_common.h"

namespace damp {
namespace {

constexpr int kC = 64;         // tokens per chunk
// LDS rows, measured on gfx950 (cycles of a wave's access on a busy CU): 16-byte operand reads of 16
// rows take 4 where the row is an odd number of 32-byte units and 8 where it is an odd number of
// 16-byte ones; 8-byte writes and reads of them take 16 and 4 against 8 and 2.4. Arrays that are
// written by 16-byte rows or 2-byte values and read as operands have the former, the others the latter.
constexpr int kLd = kC + 8;

// Chunks (or segments of `len` tokens) are numbered without a table: those of request b start at
// begin_b / len + b, which leaves room for each request's last, short one; some numbers are unused.
struct Piece {
  int b, t0, n;   // n = 0: none
};

// Where requests of at most kFew tokens go token by token and have none (FEW), the others' chunks start at
// begin_b / kFew: n > 32 tokens have at most n / 32 chunks of 64, so a request's numbers end before the next
// one's begin, and T / 32 numbers are enough however many requests there are. (A build of its own: the same
// test at run time cost ordinary calls 0.5%, 624.5 against 621.6 us for a prompt of 16,384 tokens.)
constexpr int kFew = kC / 2;

template <bool FEW>
__device__ __forceinline__ int first_piece(int b, int begin, int len) {
  return FEW ? begin / kFew : begin / len + b;
}

template <bool FEW>
__device__ __forceinline__ Piece piece_of(const PromptArgs& a, int i, int len) {
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first_piece<FEW>(mid, span_of(a, mid).begin, len) <= i) lo = mid; else hi = mid;
  }
  const Span sp = span_of(a, lo);
  const int j = i - first_piece<FEW>(lo, sp.begin, len);
  const int64_t t0 = sp.begin + int64_t(j) * len;
  if (j < 0 || t0 >= sp.end || (FEW && sp.end - sp.begin <= kFew)) return Piece{lo, 0, 0};
  return Piece{lo, static_cast<int>(t0), min(len, static_cast<int>(sp.end - t0))};
}

// Segments: numbered likewise by the most tokens one may hold, but a request's are of even length (a
// multiple of 64).
__device__ __forceinline__ int even_len(int tokens, int most) {
  const int n = (tokens + most - 1) / most;
  return ((tokens + n - 1) / n + kC - 1) / kC * kC;
}

__device__ __forceinline__ Piece segment_of(const PromptArgs& a, int i, int most) {
  const Piece pc = piece_of<false>(a, i, most);
  if (pc.n <= 0) return pc;
  const Span sp = span_of(a, pc.b);
  const int len = even_len(sp.end - sp.begin, most), t0 = sp.begin + (pc.t0 - sp.begin) / most * len;
  return Piece{pc.b, t0, max(0, min(len, sp.end - t0))};
}

// The request with the i-th most tokens (equal ones by number), so that the longest chains start first
// and share a CU with short ones; each wave finds it for itself, a request per lane. On one MI355X,
// 8,191 ragged tokens x 32 heads: 16 requests by the delta rule 245 us (255-295 us in the order given,
// by where the long ones stood), 12 of linear attention 155-158 us (151-170 us). More than 32 requests
// are taken as they come: for 64 of 128 tokens the search cost 8% (308 us against 284 us). Nor does
// the order matter where every workgroup has a CU to itself (`per_head`: workgroups a head).
__device__ __forceinline__ int request_by_length(const PromptArgs& a, int i, int per_head) {
  if (a.B > 32 || a.B * a.H * per_head <= 256) return i;
  const int lane = __builtin_amdgcn_workitem_id_x() & 63;
  int own = -1;
  if (lane < a.B) {
    const Span sp = span_of(a, lane);
    own = sp.end - sp.begin;
  }
  int rank = 0;
  for (int j = 0; j < a.B; ++j) {
    const int other = __builtin_amdgcn_readlane(own, j);
    rank += other > own || (other == own && j < lane);
  }
  return __builtin_ctzll(__ballot(lane < a.B && rank == i));   // (the ranks are a permutation)
}

// One lane's running sum of log2 decays over a chunk (lane = token; tokens past n add nothing).
__device__ __forceinline__ double chunk_logs(const PromptArgs& a, int t0, int n, int head, int lane) {
  float l = 0.0f;
  if (lane < n) l = log2_decay(a.alpha[int64_t(t0 + lane) * a.H + head]);
  return wave_scan(static_cast<double>(l), lane);
}

struct Logs {   // G = hi + lo
  float hi, lo;
};

__device__ __forceinline__ Logs split_logs(double g) {
  const float hi = static_cast<float>(g);
  return Logs{hi, static_cast<float>(g - hi)};
}

// 2^(G_t - G_s) where `live`, else 0, without a branch.
__device__ __forceinline__ float decay_between(Logs t, Logs s, bool live) {
  return pow2(live ? (t.hi - s.hi) + (t.lo - s.lo) : -4000.0f);
}

// ---- the delta rule: what a chunk's keys and gates give -------------------------------------
// Workspace of one chunk and head: X diag(b) in three bf16 pieces and P in two, then 2^G_t and
// 2^(G_C - G_t). A piece [64][64] lies as the chain's waves load it: for each 16 rows and 32 columns the
// 64 lanes' 16 bytes in a row (whole cache lines; the upper right quarter is neither written nor read).
constexpr int kPlane = kC * kC * 2;
constexpr int kGates = 5 * kPlane;
constexpr int kDeltaUnit = kGates + 2 * kC * 4;

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
// Bound by its stream: q and k in, 40.5 KB of workspace a chunk and head out. 16,384 tokens x 32 heads,
// d = 128: 138 us for 558 MB moved (302 read, 256 written), 4.0 TB/s of the 5.6 a copy reaches.
template <int D, bool FEW>
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
  const Piece pc = piece_of<FEW>(a, unit / a.H, kC);
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
    const double gs = chunk_logs(a, pc.t0, pc.n, head, lane);
    const double end = __shfl(gs, 63);
    logs[lane] = split_logs(gs);
    beta[lane] = lane < pc.n ? a.beta[int64_t(pc.t0 + lane) * a.H + head] : 0.0f;
    float* sc = reinterpret_cast<float*>(ws + kGates);
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
      const float f = decay_between(logs[t], ls, s <= t);
      kk[c][i] *= s == t ? 0.0f : beta[t] * f;
      qk[c][i] *= f;
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
  // 16 values of one row per thread: X's columns scaled by beta, in three pieces, and P in two
  const int t = tid >> 2, c0 = (tid & 3) * 16;
  if (t < 32 && c0 >= 32) return;
  uint32_t px[5][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t u[3];
    split_bf16<3>(xf[t][c0 + 2 * j] * beta[c0 + 2 * j], xf[t][c0 + 2 * j + 1] * beta[c0 + 2 * j + 1], u);
    px[0][j] = u[0]; px[1][j] = u[1]; px[2][j] = u[2];
    split_bf16<2>(pf[t][c0 + 2 * j], pf[t][c0 + 2 * j + 1], u);
    px[3][j] = u[0]; px[4][j] = u[1];
  }
  uint4* dst = reinterpret_cast<uint4*>(ws) + (t / 16 * 2 + c0 / 32) * 64 + c0 % 32 / 8 * 16 + t % 16;
#pragma unroll
  for (int p = 0; p < 5; ++p)
#pragma unroll
    for (int h = 0; h < 2; ++h) dst[p * (kPlane / 16) + 16 * h] = make_uint4(px[p][4 * h], px[p][4 * h + 1], px[p][4 * h + 2], px[p][4 * h + 3]);
}

// ---- the delta rule: the chain over the chunks ---------------------------------------------
// One workgroup of 4 waves per (request, head, 16 NT value columns): a chunk's work is split over
// token rows (16 per wave) and, for the state's update, key channels (D / 4 per wave), so a wave
// loads only its own rows of Q, X and P, straight into operand registers, one chunk ahead; K is
// staged in LDS, where it is read by rows and, transposed, by channels; the state, R and E change
// hands in LDS as [column][k] arrays of bf16 pieces. Three barriers a chunk.
// It is bound by the latency of a chunk's way from state to state, and by the state's many products
// with nothing to overlap them: 1.9 us a chunk (d = 128, 16 columns, one workgroup a CU). One prompt
// of 16,384 tokens x 32 heads 470-488 us; 8,191 ragged tokens of 16 prompts x 32 heads 181 us. Wider
// workgroups (8 waves) took as long or longer, and two state pieces instead of three in K S gained 2%
// and lost the state's last bits.
template <int D>
struct DeltaRows {   // one wave's operands of a chunk
  Frag q[D / 32], x[3][2], p[2][2];
  uint4 k[D / 32];       // this thread's share of K, on its way to LDS
  float eg[4], wc[4];    // 2^G and 2^(G_C - G) of rows 16 w + 4 g .. + 3
  float last;            // 2^G_C
};

// Blocks go to the 8 XCDs in turn, and each XCD has its own L2: numbers that differ by 8 share one.
// Of `count` * `group` blocks, the `group` ones of one item get such numbers (whole sets of 8 items;
// the rest, at the end, as they come).
struct Place {
  int item, part;
};

__device__ __forceinline__ Place place_of(unsigned id, unsigned count, unsigned group) {
  const unsigned set = id / (8 * group);
  if ((set + 1) * 8 <= count) {
    const unsigned k = id - set * 8 * group;
    return Place{static_cast<int>(set * 8 + k % 8), static_cast<int>(k / 8)};
  }
  return Place{static_cast<int>(id / group), static_cast<int>(id % group)};
}

// Chunk numbers of a call, and (request, head) pairs that a chain is started for.
int64_t chunks_of(bool few, int32_t B, int32_t T) { return few ? T / kFew : int64_t(T / kC) + B; }

template <bool FEW>
__host__ __device__ __forceinline__ unsigned chains_of(const PromptArgs& a) { return static_cast<unsigned>(FEW ? a.T / kFew : a.B) * a.H; }

template <int D, int NT, bool FEW>
__global__ __launch_bounds__(256, 2) void delta_chain_kernel(const PromptArgs a) {
  constexpr int KS = D / 32, MD = D / 64, LS = D + 8, NC = 16 * NT;
  __shared__ __align__(16) uint16_t kb[kC][LS];
  __shared__ __align__(16) uint16_t sp[3][NC][LS];
  __shared__ __align__(16) uint16_t rp[3][NC][kLd], ep[2][NC][kLd], wp[3][NC][kLd];
  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  constexpr int slices = D / NC;
  // the slices of a head read the same K, Q, X and P: one L2 for them
  const Place at = place_of(__builtin_amdgcn_workgroup_id_x(), chains_of<FEW>(a), slices);
  const int c0 = at.part * NC, head = at.item % a.H;
  int b = at.item / a.H;
  if constexpr (FEW) {   // a chain for each chunk number; it is the request's whose first chunk that is
    const Piece pc = piece_of<true>(a, b, kC);
    if (pc.n <= 0 || pc.t0 != span_of(a, pc.b).begin) return;
    b = pc.b;
  } else {
    b = request_by_length(a, b, slices);
  }
  const int64_t slot = a.slot_idx[b];
  if (!slot_in_pool(slot, a.num_slots)) return;
  const Span sp_b = span_of(a, b);
  if (sp_b.end <= sp_b.begin) return;
  const int64_t rstep = int64_t(a.H) * D;
  const uint16_t* kp = static_cast<const uint16_t*>(a.k) + int64_t(head) * D;
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + int64_t(head) * D;
  const uint16_t* vp = static_cast<const uint16_t*>(a.v) + int64_t(head) * D + c0;
  uint16_t* op = static_cast<uint16_t*>(a.out) + int64_t(head) * D + c0;
  const uint8_t* ws = a.ws + (int64_t(first_piece<FEW>(b, sp_b.begin, kC)) * a.H + head) * kDeltaUnit;
  const int64_t ws_step = int64_t(a.H) * kDeltaUnit;
  const int own = (D / 4) * w;                      // this wave's first key channel of the state
  float* pool = a.pool + ((slot * a.H + head) * D + own + 4 * g) * int64_t(D) + c0 + r;

  f32x4 S[MD][NT];   // S[m][nt][i]: key channel own + 16 m + 4 g + i, column c0 + 16 nt + r
  const bool resume = a.resume && a.resume[b] != 0;
#pragma unroll
  for (int m = 0; m < MD; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[m][nt][i] = resume ? pool[(16 * m + i) * D + 16 * nt] : 0.0f;

  const auto share_state = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int m = 0; m < MD; ++m) {
        uint32_t u0[3], u1[3];
        split_bf16<3>(S[m][nt][0], S[m][nt][1], u0);
        split_bf16<3>(S[m][nt][2], S[m][nt][3], u1);
#pragma unroll
        for (int p = 0; p < 3; ++p) *reinterpret_cast<uint2*>(&sp[p][16 * nt + r][own + 16 * m + 4 * g]) = make_uint2(u0[p], u1[p]);
      }
  };
  // A chunk's loads go through buffer resources that end with its last row: what lies past it reads
  // as 0 (and is not stored). A lane's offsets are the same in every chunk. Every load is made every
  // time and in the order of use, so that the waits on earlier ones can count the later ones.
  const uint32_t ostep = static_cast<uint32_t>(rstep) * 2;
  const uint32_t off_row = (16 * w + r) * ostep + g * 16;                  // rows of Q as operands
  const uint32_t off_k = (tid / (D / 8)) * ostep + (tid % (D / 8)) * 16;   // rows of K on their way to LDS
  const uint32_t off_val = (16 * w + 4 * g) * ostep + r * 2;               // rows of V and the readouts
  const uint32_t off_ws = (w * 128 + lane) * 16;                           // rows of X and P
  const uint32_t off_ws1 = w < 2 ? kDeltaUnit : off_ws + 1024;             // their right halves; none above the diagonal
  DeltaRows<D> f;
  uint16_t vv[NT][4];
  struct Chunk {        // a chunk's place: byte offsets of its rows and workspace, rows from there on
    int64_t row, ws;
    int left;
  };
  Chunk now{sp_b.begin * rstep * 2, 0, sp_b.end - sp_b.begin}, last_chunk = now;
  const auto rows = [&](const uint16_t* p, const Chunk& c, int width) {
    return make_rsrc(reinterpret_cast<const uint8_t*>(p) + c.row, (min(c.left, kC) - 1) * ostep + width * 2);
  };
  const auto chunk_ws = [&](const Chunk& c) { return make_rsrc(ws + c.ws, kDeltaUnit); };
  const auto frag = [](rsrc_t rs, uint32_t off, int imm) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b128(rs, off, imm, 0);
    return Frag{{v[0], v[1], v[2], v[3]}};
  };
  const auto load_q = [&](const Chunk& at) {
    const rsrc_t qr = rows(qp, at, D);
#pragma unroll
    for (int x = 0; x < KS; ++x) f.q[x] = frag(qr, off_row + x * 64, 0);
  };
  const auto load_v = [&](const Chunk& at) {
    const rsrc_t vr = rows(vp, at, NC), wr = chunk_ws(at);
    const auto e = __builtin_amdgcn_raw_buffer_load_b128(wr, kGates + (16 * w + 4 * g) * 4, 0, 0);
    const auto c = __builtin_amdgcn_raw_buffer_load_b128(wr, kGates + (kC + 16 * w + 4 * g) * 4, 0, 0);
    f.last = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(wr, kGates + (kC - 1) * 4, 0, 0));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f.eg[i] = __uint_as_float(e[i]);
      f.wc[i] = __uint_as_float(c[i]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) vv[nt][i] = __builtin_amdgcn_raw_buffer_load_b16(vr, off_val + i * ostep + 32 * nt, 0, 0);
  };
  const auto load_x = [&](const Chunk& at) {
    const rsrc_t wr = chunk_ws(at);
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      f.x[p][0] = frag(wr, off_ws + p * kPlane, 0);
      f.x[p][1] = frag(wr, off_ws1 + p * kPlane, 0);
    }
  };
  const auto load_p = [&](const Chunk& at) {
    const rsrc_t wr = chunk_ws(at);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      f.p[p][0] = frag(wr, off_ws + (3 + p) * kPlane, 0);
      f.p[p][1] = frag(wr, off_ws1 + (3 + p) * kPlane, 0);
    }
  };
  constexpr int kRows = 256 / (D / 8);   // rows of K that the threads' shares are apart
  const auto load_k = [&](const Chunk& at) {
    const rsrc_t kr = rows(kp, at, D);
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      const Frag v = frag(kr, off_k + j * kRows * ostep, 0);
      f.k[j] = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    }
  };
  const auto store_k = [&]() {
#pragma unroll
    for (int j = 0; j < KS; ++j) *reinterpret_cast<uint4*>(&kb[tid / (D / 8) + j * kRows][(tid % (D / 8)) * 8]) = f.k[j];
  };

  // O = 2^G Q S + P E of the chunk at t0, from registers alone; off the chain, it fills the wait for
  // the next chunk's operands (bytes = 0: there is no chunk before the first)
  f32x4 o[NT];
  Frag ef[NT][2][2];
  const auto readout = [&](const Chunk& at, bool some) {
    const rsrc_t out = make_rsrc(reinterpret_cast<uint8_t*>(op) + at.row, some ? (min(at.left, kC) - 1) * ostep + NC * 2 : 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4 pe[2];
      pe[0] = o[nt];
      pe[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = 0; x < 2; ++x) {   // (the right half of an upper row is zero)
        pe[0] = mfma(f.p[0][x], ef[nt][0][x], pe[0]);
        pe[1] = mfma(f.p[1][x], ef[nt][0][x], pe[1]);
        pe[0] = mfma(f.p[0][x], ef[nt][1][x], pe[0]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        __builtin_amdgcn_raw_buffer_store_b16(static_cast<short>(float_to_bf16_bits(pe[0][i] + pe[1][i])), out, off_val + i * ostep + 32 * nt, 0, 0);
    }
  };
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    o[nt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int x = 0; x < 2; ++x) ef[nt][p][x] = Frag{{0, 0, 0, 0}};
  }

  load_k(now);
  load_v(now);
  load_p(now);
  load_q(now);
  load_x(now);
  share_state();
  store_k();
  __syncthreads();
  for (int t0 = sp_b.begin; t0 < sp_b.end; t0 += kC) {
    Chunk next = now;     // the chunk to load next; the last one once more
    if (now.left > kC) next = Chunk{now.row + int64_t(kC) * ostep, now.ws + ws_step, now.left - kC};
    // K S; R = V - 2^G K S
    Frag kf[KS], s[NT][2][KS];
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      kf[x] = load_frag(&kb[16 * w + r][x * 32 + g * 8]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int p = 0; p < 2; ++p) s[nt][p][x] = load_frag(&sp[p][16 * nt + r][x * 32 + g * 8]);
    }
    __builtin_amdgcn_sched_barrier(0);
    load_k(next);
    readout(last_chunk, t0 > sp_b.begin);
    load_p(now);
    __builtin_amdgcn_sched_barrier(0);
    const float wc[4] = {f.wc[0], f.wc[1], f.wc[2], f.wc[3]}, last = f.last;
    float eg[4] = {f.eg[0], f.eg[1], f.eg[2], f.eg[3]};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      Frag s2[KS];   // the third piece, which the readout does without
#pragma unroll
      for (int x = 0; x < KS; ++x) s2[x] = load_frag(&sp[2][16 * nt + r][x * 32 + g * 8]);
      f32x4 ks[3];
#pragma unroll
      for (int p = 0; p < 3; ++p) ks[p] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = 0; x < KS; ++x)
#pragma unroll
        for (int p = 0; p < 3; ++p) ks[p] = mfma(kf[x], p < 2 ? s[nt][p][x] : s2[x], ks[p]);
      float rr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) rr[i] = fmaf(-eg[i], ks[0][i] + (ks[1][i] + ks[2][i]), __uint_as_float(uint32_t(vv[nt][i]) << 16));
      uint32_t u0[3], u1[3];
      split_bf16<3>(rr[0], rr[1], u0);
      split_bf16<3>(rr[2], rr[3], u1);
#pragma unroll
      for (int p = 0; p < 3; ++p) *reinterpret_cast<uint2*>(&rp[p][16 * nt + r][16 * w + 4 * g]) = make_uint2(u0[p], u1[p]);
    }
    load_v(next);
    __syncthreads();
    // E = X diag(b) R; Q S while R comes
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      Frag rf[3][2];
#pragma unroll
      for (int j = 0; j < 3; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) rf[j][x] = load_frag(&rp[j][16 * nt + r][x * 32 + g * 8]);
      __builtin_amdgcn_sched_barrier(0);
      f32x4 qs[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) qs[p] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = 0; x < KS; ++x)
#pragma unroll
        for (int p = 0; p < 2; ++p) qs[p] = mfma(f.q[x], s[nt][p][x], qs[p]);
      __builtin_amdgcn_sched_barrier(0);
      f32x4 ex[3];
#pragma unroll
      for (int j = 0; j < 3; ++j) ex[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = 0; x < 2; ++x)        // (the right half of an upper row of X is zero)
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
          for (int j = 0; i + j < 3; ++j) ex[j] = mfma(f.x[i][x], rf[j][x], ex[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[nt][i] = eg[i] * (qs[0][i] + qs[1][i]);
      const f32x4 e = ex[0] + (ex[1] + ex[2]);
      uint32_t u0[3], u1[3];
      split_bf16<3>(e[0] * wc[0], e[1] * wc[1], u0);
      split_bf16<3>(e[2] * wc[2], e[3] * wc[3], u1);
#pragma unroll
      for (int p = 0; p < 3; ++p) *reinterpret_cast<uint2*>(&wp[p][16 * nt + r][16 * w + 4 * g]) = make_uint2(u0[p], u1[p]);
      split_bf16<2>(e[0], e[1], u0);
      split_bf16<2>(e[2], e[3], u1);
#pragma unroll
      for (int p = 0; p < 2; ++p) *reinterpret_cast<uint2*>(&ep[p][16 * nt + r][16 * w + 4 * g]) = make_uint2(u0[p], u1[p]);
    }
    Frag kt[2][MD];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int m = 0; m < MD; ++m) {
        const uint16_t* from = &kb[32 * x + 8 * g + r / 4][own + 16 * m + 4 * (r % 4)];
        kt[x][m] = load_frag_t(from, from + 4 * LS);
      }
    load_q(next);
    __syncthreads();
    // S = 2^G_C S + K^T (2^(G_C - G) E)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      Frag wf[3][2];
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int x = 0; x < 2; ++x) wf[p][x] = load_frag(&wp[p][16 * nt + r][x * 32 + g * 8]);
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int x = 0; x < 2; ++x) ef[nt][p][x] = load_frag(&ep[p][16 * nt + r][x * 32 + g * 8]);
      __builtin_amdgcn_sched_barrier(0);
      if (nt == 0) load_x(next);
#pragma unroll
      for (int m = 0; m < MD; ++m) {
        f32x4 add[3];
        add[0] = S[m][nt] * last;
        add[1] = add[2] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int p = 0; p < 3; ++p) add[p] = mfma(kt[x][m], wf[p][x], add[p]);
        S[m][nt] = add[0] + (add[1] + add[2]);
      }
    }
    share_state();
    store_k();   // (K was last read before the barrier)
    last_chunk = now;
    now = next;
    __syncthreads();
  }
  readout(last_chunk, true);
#pragma unroll
  for (int m = 0; m < MD; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) pool[(16 * m + i) * D + 16 * nt] = S[m][nt][i];
}

// ---- linear attention ------------------------------------------------------------------------
// One workgroup of 4 waves per (segment of a prompt, head); wave w owns the value columns D / 4 * w
// .. of the state, the values and the readouts, so between the chunks nothing of the state leaves
// its registers: as the B operand of Q S it is the accumulator tiles as they stand (k permuted:
// mfma), and Q is read to match. K, Q and K^T are staged in LDS once per chunk for all waves, P is
// formed tile by tile by the waves in turn. Long prompts of few heads are cut into segments: a first
// launch (STATES) sums every segment's own state, a scan turns them into the states before each
// segment, and the readouts of all segments run at once.
// Bound by issue (splitting the state and the weights into pieces, their products, the LDS reads):
// 4.1 us a chunk with one workgroup a CU. 8,191 ragged tokens of 12 prompts x 32 heads, d = 128: 160 us,
// 71 us where 16 prompts are even, against 55 us of its 307 MB at the rate of a copy; the longest
// prompt's chain sets the ragged time. 8 waves a workgroup took 84 us where 4 took 72-74.
enum LinearMode : int { LIN_WHOLE = 0, LIN_STATES = 1, LIN_SEGMENTS = 2 };

struct Segments {
  int len;          // most tokens per segment, a multiple of 64; 0: whole prompts
  float* states;    // [segment number][H][D][D]: own states, then the states before
  float* decays;    // [segment number][H]: log2 of a segment's decay
};

template <int D, int DECAY, int MODE>
__global__ __launch_bounds__(256, 2) void linear_chunk_kernel(const PromptArgs a, const Segments sg) {
  constexpr int KS = D / 32, MD = D / 64, XT = D / 16, LK = D + 8, LR = D + 16, LP = kC + 16;
  constexpr bool kReadout = MODE != LIN_STATES;
  __shared__ __align__(16) uint16_t ks[kC][LR];
  __shared__ __align__(16) uint16_t qs[kReadout ? kC : 1][LK];
  __shared__ __align__(16) uint16_t pp[2][kReadout ? kC : 1][LP];
  __shared__ Logs logs[4][kC];                    // of four chunks
  __shared__ __align__(16) float eg[4][kC], wc[4][kC];
  __shared__ double ends[4];
  const int tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int unit = __builtin_amdgcn_workgroup_id_x();
  const int head = unit % a.H, seg = unit / a.H;
  int b = seg, t_begin, t_end;
  if constexpr (MODE == LIN_WHOLE) {
    b = request_by_length(a, seg, 1);
    const Span sp = span_of(a, b);
    t_begin = sp.begin;
    t_end = sp.end;
  } else {
    const Piece pc = segment_of(a, seg, sg.len);
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
  const uint32_t ostep = static_cast<uint32_t>(rstep) * 2;
  const uint16_t* kp = static_cast<const uint16_t*>(a.k) + int64_t(head) * D;
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + int64_t(head) * D;
  const uint16_t* vp = static_cast<const uint16_t*>(a.v) + int64_t(head) * D;
  uint16_t* op = static_cast<uint16_t*>(a.out) + int64_t(head) * D;
  const int col = (D / 4) * w + MD * r;           // this lane's first value column
  float* pool = a.pool + (slot * a.H + head) * int64_t(D * D);
  float* states = MODE == LIN_WHOLE ? nullptr : sg.states + int64_t(unit) * (D * D);
  const uint32_t off_state = (4 * g * D + col) * 4;

  f32x4 S[XT][MD];   // S[x][m][i]: key channel 16 x + 4 g + i, value column col + m
  {
    const bool some = MODE == LIN_SEGMENTS || (MODE == LIN_WHOLE && a.resume && a.resume[b] != 0);
    const rsrc_t from = make_rsrc(MODE == LIN_SEGMENTS ? states : pool, D * D * 4);
#pragma unroll
    for (int x = 0; x < XT; ++x)
#pragma unroll
      for (int m = 0; m < MD; ++m) S[x][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (some) {
#pragma unroll
      for (int x = 0; x < XT; ++x)
#pragma unroll
        for (int m = 0; m < MD; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            S[x][m][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(from, off_state + 4 * m, (16 * x + i) * D * 4, 0));
    }
  }

  // One chunk's rows, in registers until LDS is free for them, through buffer resources that end
  // with the segment's last row (rows past it read as 0 and are not stored).
  constexpr int kRows = 256 / (D / 8);            // rows of K that a thread's pieces are apart
  const uint32_t off_k = (tid / (D / 8)) * ostep + (tid % (D / 8)) * 16;
  const uint32_t off_v = 8 * g * ostep + col * 2;
  Frag kr[KS], qr[KS];
  uint32_t vr[2][8];                              // values of tokens 32 x + 8 g + j, columns col ..
  const auto rows = [&](const uint16_t* p, int t0) {
    return make_rsrc(p + t0 * rstep, (min(t_end - t0, kC) - 1) * ostep + D * 2);
  };
  const auto load_rows = [&](int t0) {
    const rsrc_t rk = rows(kp, t0), rq = rows(qp, t0);
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      const auto k4 = __builtin_amdgcn_raw_buffer_load_b128(rk, off_k + j * kRows * ostep, 0, 0);
      kr[j] = Frag{{k4[0], k4[1], k4[2], k4[3]}};
      if constexpr (kReadout) {
        const auto q4 = __builtin_amdgcn_raw_buffer_load_b128(rq, off_k + j * kRows * ostep, 0, 0);
        qr[j] = Frag{{q4[0], q4[1], q4[2], q4[3]}};
      }
    }
  };
  const auto store_rows = [&]() {
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      const int t = tid / (D / 8) + j * kRows, c = (tid % (D / 8)) * 8;
      *reinterpret_cast<uint4*>(&ks[t][c]) = make_uint4(kr[j].w[0], kr[j].w[1], kr[j].w[2], kr[j].w[3]);
      if constexpr (kReadout) *reinterpret_cast<uint4*>(&qs[t][c]) = make_uint4(qr[j].w[0], qr[j].w[1], qr[j].w[2], qr[j].w[3]);
    }
  };
  const auto load_v = [&](int t0) {
    const rsrc_t rv = rows(vp, t0);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t off = off_v + (32 * x + j) * ostep;
        vr[x][j] = MD == 2 ? __builtin_amdgcn_raw_buffer_load_b32(rv, off, 0, 0) : __builtin_amdgcn_raw_buffer_load_b16(rv, off, 0, 0);
      }
  };

  if constexpr (kReadout) {   // the tiles above the diagonal that a product reads
    for (int x = tid; x < 2 * 2 * 16 * 2; x += 256) {
      const int row = (x >> 1 & 15) + 32 * (x >> 5 & 1);
      *reinterpret_cast<uint4*>(&pp[x >> 6][row][16 + (row & 32) + 8 * (x & 1)]) = make_uint4(0, 0, 0, 0);
    }
  }
  float ahead;   // this lane's decay of the wave's chunk among the next four (1 past the end)
  const auto load_decays = [&](int t0) {
    const int t = t0 + kC * w + lane;
    ahead = a.alpha[DECAY == DECAY_HEAD ? head : (int64_t(min(t, t_end - 1)) * a.H + head)];
    if (t >= t_end) ahead = 1.0f;
  };
  double total = 0.0;
  load_decays(t_begin);
  load_rows(t_begin);
  load_v(t_begin);
  int at = 0;
  for (int t0 = t_begin; t0 < t_end; t0 += kC, at = (at + 1) & 3) {
    const int tn = t_end - t0 > kC ? t0 + kC : t0;   // the chunk to load next
    store_rows();
    if (at == 0) {   // the decays of this chunk and the next three, one a wave
      const double gs = wave_scan(static_cast<double>(log2_decay(ahead)), lane);
      const double end = __shfl(gs, 63);
      logs[w][lane] = split_logs(gs);
      eg[w][lane] = pow2(static_cast<float>(gs));
      wc[w][lane] = pow2(static_cast<float>(end - gs));
      if (lane == 0) ends[w] = end;
    }
    __syncthreads();
    load_rows(tn);
    if (at == 0) load_decays(t0 + 4 * kC);
    f32x4 o[kReadout ? 4 : 1][MD];
    if constexpr (kReadout) {
      // P: the 10 tiles on and below the diagonal, 2 or 3 a wave
      const unsigned tiles = w == 0 ? 0xc0f : w == 1 ? 0x54d : w == 2 ? 0x98e : 0xaff;   // row, column: 2 bits each
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const int rt = tiles >> (4 * (2 - j) + 2) & 3, c = tiles >> (4 * (2 - j)) & 3;
        if (j == 2 && (w == 0 || w == 3)) break;
        f32x4 p{0.0f, 0.0f, 0.0f, 0.0f};
        const int s = 16 * c + r;
#pragma unroll
        for (int x = 0; x < KS; ++x)
          p = mfma(load_frag(&qs[16 * rt + r][x * 32 + g * 8]), load_frag(&ks[s][x * 32 + g * 8]), p);
        const Logs ls = logs[at][s];
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const int t = 16 * rt + 4 * g + i;
          uint32_t u[2];
          split_bf16<2>(p[i] * decay_between(logs[at][t], ls, s <= t), p[i + 1] * decay_between(logs[at][t + 1], ls, s <= t + 1), u);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            pp[x][t][s] = static_cast<uint16_t>(u[x]);
            pp[x][t + 1][s] = static_cast<uint16_t>(u[x] >> 16);
          }
        }
      }
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int m = 0; m < MD; ++m) o[rt][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      Frag sf[2][2][MD];
      const auto split_state = [&](int x) {
#pragma unroll
        for (int m = 0; m < MD; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t u[2];
            split_bf16<2>(S[2 * x + j / 2][m][2 * (j & 1)], S[2 * x + j / 2][m][2 * (j & 1) + 1], u);
            sf[x & 1][0][m].w[j] = u[0];
            sf[x & 1][1][m].w[j] = u[1];
          }
      };
      split_state(0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        if (x + 1 < KS) split_state(x + 1);   // the next pieces between this step's products
        Frag q[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) q[rt] = load_frag2(&qs[16 * rt + r][x * 32 + g * 4], &qs[16 * rt + r][x * 32 + 16 + g * 4]);
        // (a product that continues a sum comes 4 MD products after the last of that sum)
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int rt = 0; rt < 4; ++rt)
#pragma unroll
            for (int m = 0; m < MD; ++m) o[rt][m] = mfma(q[rt], sf[x & 1][p][m], o[rt][m]);
#pragma unroll
        for (int j = 0; j < 8 * MD; ++j) {
          if (j == 0) __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
          __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x2, 3, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) {
        const float4 e = *reinterpret_cast<const float4*>(&eg[at][16 * rt + 4 * g]);
#pragma unroll
        for (int m = 0; m < MD; ++m) {
          o[rt][m][0] *= e.x; o[rt][m][1] *= e.y; o[rt][m][2] *= e.z; o[rt][m][3] *= e.w;
        }
      }
      __syncthreads();
      const rsrc_t out = rows(op, t0);
      uint32_t step = ostep;
      asm volatile("" : "+s"(step));   // (offsets formed here, not held in registers over the loop)
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
          const uint32_t off = (16 * rt + 4 * g + i) * step + col * 2;
          if constexpr (MD == 2) __builtin_amdgcn_raw_buffer_store_b32(pack_bf16(o[rt][0][i], o[rt][1][i]), out, off, 0, 0);
          else __builtin_amdgcn_raw_buffer_store_b16(static_cast<short>(float_to_bf16_bits(o[rt][0][i])), out, off, 0, 0);
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
      for (int y = 0; y < XT; y += 2) {
        Frag kf[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint16_t* from = &ks[32 * x + 8 * g + r / 4][16 * (y + h) + 4 * (r % 4)];
          kf[h] = load_frag_t(from, from + 4 * LR);
        }
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int m = 0; m < MD; ++m) S[y + h][m] = mfma(kf[h], vf[p][m], S[y + h][m]);
      }
    }
    load_v(tn);
    __syncthreads();
  }
  if (MODE == LIN_STATES || final) {
    const rsrc_t to = make_rsrc(MODE == LIN_STATES ? states : pool, D * D * 4);
#pragma unroll
    for (int x = 0; x < XT; ++x)
#pragma unroll
      for (int m = 0; m < MD; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[x][m][i]), to, off_state + 4 * m, (16 * x + i) * D * 4, 0);
  }
  if (MODE == LIN_STATES && tid == 0) sg.decays[unit] = static_cast<float>(total);
}

// The segments' own states turned into the states before each segment, 4 values a thread, read and
// written once: bound by that stream.
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

// Segments of a call: none (whole prompts) where the prompts alone fill the chip, or where all
// together are so short that three launches cost more. d = 128, 32 heads, on one MI355X: 8 prompts of
// 1,024 tokens 83 us whole, 115 us cut; 4 of 2,048 147 and 119 us; one of 8,192 531 and 126 us; one of
// 512 35 and 38 us. (Between 4 and 8 even prompts whole ones are faster, 95 against 131 us for 7, but the
// lengths are on the device, and one long prompt among them would take as long as alone.)
int segment_len(int32_t B, int32_t T, int32_t H) {
  if (int64_t(B) * H >= 256 || T <= 8 * kC) return 0;
  const int64_t want = (int64_t(T) * H + 511) / 512;
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
  // (the scan goes by the numbers, so the segments' lengths do not matter to it)
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

template <int D, bool FEW>
hipError_t delta_d(const PromptArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((delta_chunk_kernel<D, FEW>), dim3(static_cast<unsigned>(chunks_of(FEW, a.B, a.T) * a.H)), dim3(256), 0, s, a);
  const unsigned units = chains_of<FEW>(a);
  // 32 columns a workgroup read K, Q, X and P half as often, 16 give twice the workgroups. On one
  // MI355X, d = 128, 32 heads, 8,192 tokens in all, with 32 columns against 16: 64 states 264 against
  // 289 us, 128 states 229 against 288, 2,048 states 287 against 378; 32 states (one prompt) 431
  // against 321. d = 64: 128 states 138 against 143 us, 64 states 201 against 154.
  if (units * (D / 32) >= 256)
    hipLaunchKernelGGL((delta_chain_kernel<D, 2, FEW>), dim3(units * (D / 32)), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((delta_chain_kernel<D, 1, FEW>), dim3(units * (D / 16)), dim3(256), 0, s, a);
  return hipGetLastError();
}

// bf16 inputs with one decay per head run in chunks; the rest token by token. So do calls of the delta
// rule of few tokens: one launch instead of two, and no chunk's inverse. On one MI355X, d = 128, 32
// heads, one prompt of 1 token 4.0 us against 13.1, of 16 7.6 against 13.2, of 32 11.9 against 13.3, of
// 48 16.4 against 13.5. Calls of no more tokens than requests (a fixed list of which few are in use, or a
// token each) of more than 64 tokens take both forms, by the requests' lengths, which only the device knows:
// those of up to 32 tokens one, longer ones the other. 512 requests, all 512 tokens one's: 70 us, 171 all
// token by token, 75 all in chunks; a token each: 578, 568 and 1,061 us. At 64 tokens of 64 requests the
// two launches more are not worth it: 21.5 and 72 us against 23.4 and 68 (19 and 128 in chunks).
// (Linear attention's chunks need one launch too: 3.9 us against 8.5 for one token, but 67 against 43 for
// 64 requests of one, which stay in chunks.)
enum Form : int { TOKENS, CHUNKS, BY_LENGTH };

Form form_of(bool delta, int d, int decay, int bf16, int32_t B, int32_t T) {
  if (!bf16 || (d != 64 && d != 128) || decay == DECAY_KEY || (delta && (T <= kFew || T <= std::min(B, 2 * kFew))))
    return TOKENS;
  return delta && T <= B ? BY_LENGTH : CHUNKS;
}

}  // namespace

int64_t prefill_ws_bytes(bool delta, int d, int decay, int bf16, int32_t B, int32_t T, int32_t H) {
  const Form form = form_of(delta, d, decay, bf16, B, T);
  if (form == TOKENS) return 0;
  if (delta) return chunks_of(form == BY_LENGTH, B, T) * H * kDeltaUnit;
  const int len = segment_len(B, T, H);
  return len ? (int64_t(T / len) + B) * H * (int64_t(d) * d + 1) * 4 : 0;
}

hipError_t launch_prefill(bool delta, int d, int decay, int bf16, const PromptArgs& a, hipStream_t s) {
  const Form form = form_of(delta, d, decay, bf16, a.B, a.T);
  if (form == TOKENS) return launch_prompt_token(d, delta, decay, bf16, a, s);
  if (!delta) return d == 64 ? linear_d<64>(decay, a, s) : linear_d<128>(decay, a, s);
  if (form == CHUNKS) return d == 64 ? delta_d<64, false>(a, s) : delta_d<128, false>(a, s);
  PromptArgs few = a;
  few.few = kFew;
  const hipError_t e = launch_prompt_token(d, delta, decay, bf16, few, s);
  if (e != hipSuccess) return e;
  return d == 64 ? delta_d<64, true>(a, s) : delta_d<128, true>(a, s);
}

}  // namespace damp
