// attn_mask.h -- what the attention kernels of several tokens share: which positions a drafted token
// sees, the softmax weights as operands, and values that are not finite.
#pragma once

#include "prompt_common.h"

namespace damp {
namespace {

using u32x4 = __attribute__((ext_vector_type(4))) uint32_t;

// A request's drafted tokens: rows first .. first + n - 1 of the queries, kept inside [0, T) whatever
// cu holds, at the positions base .. base + n - 1.
struct Drafts {
  int first, n, base;
};

__device__ __forceinline__ Drafts drafts_of(const TreeArgs& a, int b) {
  if (!a.cu) return Drafts{b, 1, max(a.seq_lens[b], 0) - 1};
  const int lo = min(max(a.cu[b], 0), a.T), hi = min(max(a.cu[b + 1], lo), a.T);
  return Drafts{lo, hi - lo, max(a.seq_lens[b], 0) - (hi - lo)};
}

// Bit x: drafted token `token` sees position base + rel + x (x < 32, rel > -32): every one before base,
// from base on those in its mask, or without masks those up to its own.
__device__ __forceinline__ uint32_t seen_window(const TreeArgs& a, const Drafts& dr, int token, int rel) {
  const int from = max(rel, 0);
  uint32_t bits;
  if (a.mask) {
    const uint64_t* words = a.mask + int64_t(dr.first + token) * a.words;
    const int w = from >> 6, s = from & 63;
    uint64_t x = w < a.words ? words[w] >> s : 0;
    if (s > 32 && w + 1 < a.words) x |= words[w + 1] << (64 - s);
    bits = static_cast<uint32_t>(x);
  } else {
    const int n = token + 1 - from;
    bits = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1;
  }
  return rel >= 0 ? bits : (bits << -rel) | ((1u << -rel) - 1);
}

// Running sums over the 64 lanes, by moves inside the vector unit (a sixth of the time that moves through LDS
// take; this is on the way of every workgroup's first load).
template <typename T>
__device__ __forceinline__ T scan64(T x) {
  static_assert(sizeof(T) == 4);
#define DAMP_SCAN_STEP(ctrl, rows) x += __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), ctrl, rows, 0xf, false))
  DAMP_SCAN_STEP(0x111, 0xf);   // from 1, 2, 4, 8 lanes below, within 16 lanes
  DAMP_SCAN_STEP(0x112, 0xf);
  DAMP_SCAN_STEP(0x114, 0xf);
  DAMP_SCAN_STEP(0x118, 0xf);
  DAMP_SCAN_STEP(0x142, 0xa);   // the sum of the 16 lanes below to the odd 16s, of the lower 32 to the upper
  DAMP_SCAN_STEP(0x143, 0xc);
#undef DAMP_SCAN_STEP
  return x;
}

template <typename T>
__device__ __forceinline__ T last_lane(T x) { return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63)); }

// Each lane's 16 bytes at src into LDS at dst + 16 lane (dst the same for the wave), without a way through
// registers. The data is there after landed() and a barrier.
__device__ __forceinline__ void load_to_lds(const uint8_t* src, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src, (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

// All loads but the `later` youngest are back.
template <int later = 0>
__device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(later) : "memory"); }

// Rows loaded that way lie close together in LDS. So that operands are read without bank conflicts, piece p (16
// bytes) of row t lies at p ^ row_turn(t) where rows are read whole (one access of 16 lanes takes piece c of
// rows 0-3 and 12-15 and piece c + 1 of rows 4-11, or the other way round), at p ^ column_turn(t) where they
// are read transposed (32 lanes: the halves of two pieces of 8 rows). PIECES: of a row, 4, 8 or 16.
template <int PIECES>
__device__ __forceinline__ int row_turn(int t) { return PIECES == 4 ? -(t >> 2) & 3 : PIECES == 8 ? t >> 1 & 7 : t & 15; }

template <int PIECES>
__device__ __forceinline__ int column_turn(int t) { return PIECES == 8 ? t & 6 : (t & 3) * 2 + (t & 4) * 2; }

// Maximum over the lanes l, l ^ 16, l ^ 32 and l ^ 48 (as sum_row_slots adds).
__device__ __forceinline__ float max_row_slots(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const uint32_t u2 = __float_as_uint(x);
  const auto b = __builtin_amdgcn_permlane32_swap(u2, u2, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// sum + f x, where f is what a part of a row's tokens (a wave's, a run's) counts beside the others and x a channel
// of its readout. f may be 0, where the other parts' scores are higher by far or the part saw no token; the weights
// behind it are not, so an infinity counts all the same (0 * infinity is NaN).
__device__ __forceinline__ float add_part(float f, float x, float sum) { return fmaf(__builtin_isfinite(x) ? f : 1.0f, x, sum); }

// A row's running maximum stays as it is until a score passes it by more than this factor 2^kSlack: weights of
// up to 2^8 lose nothing in binary32 or bf16 (sums over n tokens overflow from values of 2^120 / n on), and most
// tiles then need neither the other lanes' maxima nor sums scaled down.
constexpr float kSlack = 8.0f;

// x, in a branch that few tiles take: what goes by it is not worked out before the branch (for all tiles, to be
// selected from).
template <typename T>
__device__ __forceinline__ T rarely(T x) {
  asm volatile("" : "+v"(x));
  return x;
}

// An operand of ones: its product with the weights is their sum, in every row of the C tile.
__device__ __forceinline__ Frag ones() { return Frag{{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u}}; }

// Softmax weights of one row as an operand of the product with V, in one of two ways. Rounded to bf16 (to
// 2^-8 of each), with a sum over the rounded ones, so that equal values come back as they are: what a row
// gets is then off by up to 2^-8 of the weighted mean of |v - o|, the size of its own rounding. Or in two pieces,
// the upper 16 bits of the weight (less 2^-12) and the rest rounded, good to 2^-15 + 2^-20 of it, the rest
// never 0 (an infinite value times 0 would be NaN): twice the products, which few rows have to spare.
__device__ __forceinline__ Frag round_weights(const float (&p)[8]) {
  return Frag{{pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]), pack_bf16(p[6], p[7])}};
}

__device__ __forceinline__ uint32_t round_pair(float x0, float x1, float& sum) {
  const uint32_t w = pack_bf16(x0, x1);
  sum += bf16_lo(w) + bf16_hi(w);
  return w;
}

__device__ __forceinline__ void split_pair(float x0, float x1, uint32_t& upper, uint32_t& rest, float& sum) {
  const uint32_t w0 = __float_as_uint(x0 * 0x1.ffep-1f), w1 = __float_as_uint(x1 * 0x1.ffep-1f);
  upper = __builtin_amdgcn_perm(w1, w0, 0x07060302u);
  rest = pack_bf16(x0 - __uint_as_float(w0 & 0xffff0000u), x1 - __uint_as_float(w1 & 0xffff0000u));
  sum += x0 + x1;
}

__device__ __forceinline__ void pack_weights(const float (&p)[8], Frag (&pf)[2], float& sum) {
#pragma unroll
  for (int i = 0; i < 4; ++i) split_pair(p[2 * i], p[2 * i + 1], pf[0].w[i], pf[1].w[i], sum);
}

// 0x8000 / 0x80000000 bits of the halves that hold an infinity or a NaN.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// Values that are not finite must not enter a product with rows that do not see their token: their
// weight there is 0, but 0 * NaN is NaN. In tiles that hold drafted tokens they are taken out, and in
// the end each row gets back those of the tokens that it sees (adding them up has their product's
// result, whatever the weights).
__device__ __forceinline__ uint32_t finite_only(uint32_t w) { return w & ~((not_finite(w) >> 15) * 0xffffu); }

__device__ __forceinline__ f32x4 add_odd(f32x4 o, uint2 v, bool seen) {   // 4 channels of one token
  const float x[4] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
  const uint32_t odd[2] = {not_finite(v.x), not_finite(v.y)};
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] += seen && (odd[i >> 1] >> (16 * (i & 1)) & 0x8000u) ? x[i] : 0.0f;
  return o;
}

}  // namespace
}  // namespace damp
