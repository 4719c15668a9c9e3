// prompt_common.h -- device building blocks shared by the linear-attention and prompt kernels:
// the tokens of a request, dispatch over the decay forms, bf16 conversion and splitting, and the
// matrix instructions these kernels use.
#pragma once

#include "step_common.h"

namespace damp {
namespace {

// The tokens of request b, kept inside [0, T) whatever cu holds.
struct Span {
  int begin, end;
};

__device__ __forceinline__ Span span_of(const PromptArgs& a, int b) {
  const int lo = min(max(a.cu[b], 0), a.T);
  return Span{lo, min(max(a.cu[b + 1], lo), a.T)};
}

template <typename F>
void with_decay(int decay, F&& f) {
  if (decay == DECAY_KEY) f.template operator()<DECAY_KEY>();
  else if (decay == DECAY_HEAD) f.template operator()<DECAY_HEAD>();
  else f.template operator()<DECAY_SCALAR>();
}

using bf16x2 = __attribute__((ext_vector_type(2))) __bf16;
using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;
using f32x2 = __attribute__((ext_vector_type(2))) float;
using f32x4 = __attribute__((ext_vector_type(4))) float;

// Two values rounded to nearest even, packed (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2 v = __builtin_convertvector(f32x2{lo, hi}, bf16x2);
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ uint16_t float_to_bf16_bits(float x) { return static_cast<uint16_t>(pack_bf16(x, x)); }

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two binary32 values as N packed bf16 pieces whose sum is the value to 8 N bits: each piece
// rounds what the earlier ones left, which is exact in binary32. Products of pieces then run on
// the bf16 matrix instructions with binary32 sums: three pieces (2^-24) carry a binary32 operand
// whole, two (2^-16, 6e-7 in the mean square) suffice where the result is rounded to bf16.
template <int N>
__device__ __forceinline__ void split_bf16(float x0, float x1, uint32_t* piece) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    piece[i] = pack_bf16(x0, x1);
    if (i + 1 < N) {
      x0 -= bf16_lo(piece[i]);
      x1 -= bf16_hi(piece[i]);
    }
  }
}

struct Frag {   // one lane's 8 bf16 values of a 16 x 32 operand
  uint32_t w[4];
};

// v_mfma_f32_16x16x32_bf16. A: lane l holds row l % 16, k = 8 (l / 16) .. + 7; B: column l % 16,
// the same k; C: column l % 16, rows 4 (l / 16) .. + 3. A permutation of k that both operands
// share changes nothing, which is how a C tile becomes a B operand without leaving the registers:
// rows 4 g .. + 3 of two stacked tiles are the k values of lane group g.
__device__ __forceinline__ f32x4 mfma(const Frag& a, const Frag& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// v_mfma_f32_16x16x4_f32. A: row l % 16, k = l / 16; B: column l % 16, k = l / 16; C as above.
__device__ __forceinline__ f32x4 mfma_f32(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ Frag load_frag(const void* p) {   // 16-byte aligned
  const uint4 v = *static_cast<const uint4*>(p);
  return Frag{{v.x, v.y, v.z, v.w}};
}

__device__ __forceinline__ Frag load_frag2(const void* p, const void* p2) {   // two 8-byte halves
  const uint2 v = *static_cast<const uint2*>(p), u = *static_cast<const uint2*>(p2);
  return Frag{{v.x, v.y, u.x, u.y}};
}

// ds_read_b64_tr_b16 twice: of a bf16 array in LDS with rows of k and neighbouring columns, 8 rows of
// one column per lane. Each 16 lanes read 4 rows x 16 columns: lane l passes the address of row l / 4,
// columns 4 (l % 4) .. + 3, and gets column l of the 4 rows.
__device__ __forceinline__ Frag load_frag_t(const uint16_t* rows_lo, const uint16_t* rows_hi) {
  using s16x4 = __attribute__((ext_vector_type(4))) short;
  using lds_ptr = __attribute__((address_space(3))) s16x4*;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)rows_lo);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)rows_hi);
  const uint2 u = __builtin_bit_cast(uint2, a), v = __builtin_bit_cast(uint2, b);
  return Frag{{u.x, u.y, v.x, v.y}};
}

// 2^x with results below binary32's normal range flushed or subnormal (v_exp_f32).
__device__ __forceinline__ float pow2(float x) { return __builtin_amdgcn_exp2f(x); }

// log2 of a decay; 0 (or a negative or subnormal value) counts as 2^-4000, whose products are 0. NaN stays NaN.
__device__ __forceinline__ float log2_decay(float a) { return a < 0x1p-126f ? -4000.0f : __builtin_amdgcn_logf(a); }

// Running sums over the 64 lanes of a wave, in binary64.
__device__ __forceinline__ double wave_scan(double x, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  return x;
}

}  // namespace
}  // namespace damp
