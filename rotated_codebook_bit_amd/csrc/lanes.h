// Exchanges between the lanes of a wave and 16-byte element access, shared by
// the norm, embedding and 8-bit product kernels.
#pragma once

#include "cq_internal.h"

namespace cq {

typedef __bf16 bf16_pair __attribute__((ext_vector_type(2)));
typedef float f32_pair __attribute__((ext_vector_type(2)));

// Two floats as a dword of bf16 (round to nearest even, NaN kept).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32_pair{a, b}), bf16_pair));
}
__device__ __forceinline__ uint16_t one_bf16(float a) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(a));
}
__device__ __forceinline__ float bf16_low(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }

template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// A butterfly between lanes pairs lane l with l ^ 1, l ^ 2, l ^ 7, l ^ 8
// (one DPP move each: two quad permutes, a mirror inside 8 lanes, a rotation
// by 8 inside 16), l ^ 16 and l ^ 32 (half swaps).  The masks are independent
// over GF(2), so lane l can stand for label lane_label(l), in which those
// pairs differ in exactly bit 0, 1, .., 5: the butterfly is the Sylvester
// transform over labels.  A kernel gives lane l the data of position
// lane_label(l); within 8 lanes only the upper four are reversed.
__device__ __forceinline__ int lane_label(int lane) { return lane ^ ((lane & 4) ? 3 : 0); }

// One butterfly stage over label bit BIT; `label` is this lane's label.  Bits
// 0 to 3: the lane whose bit is clear holds a and takes b + a, its partner
// holds b and takes b - a, the negated difference; both lanes of a later pair
// are negated alike, so label_sign() puts all signs right at the end.
template <int BIT, int N>
__device__ __forceinline__ void label_stage(float (&y)[N], int label) {
  const float sgn = ((label >> BIT) & 1) ? -1.0f : 1.0f;
  if constexpr (BIT < 4) {
    constexpr int kCtrl = BIT == 0 ? 0xB1 : BIT == 1 ? 0x4E : BIT == 2 ? 0x141 : 0x128;
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = __builtin_fmaf(dpp_move<kCtrl>(y[i]), sgn, y[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // Both operands the same value: the first result holds the bit-clear
      // lane's value in both lanes of a pair, the second the other's.
      const uint32_t u = __builtin_bit_cast(uint32_t, y[i]);
      const auto ab = BIT == 4 ? __builtin_amdgcn_permlane16_swap(u, u, false, false)
                               : __builtin_amdgcn_permlane32_swap(u, u, false, false);
      const uint32_t a = ab[0], b = ab[1];
      y[i] = __builtin_fmaf(sgn, __builtin_bit_cast(float, b), __builtin_bit_cast(float, a));
    }
  }
}

// Butterfly over `labels` lanes (a power of two, run time, 1 .. 64), times
// label_sign(label, labels).
template <int N>
__device__ __forceinline__ void label_butterfly(float (&y)[N], int label, int labels) {
  if (labels > 1) label_stage<0>(y, label);
  if (labels > 2) label_stage<1>(y, label);
  if (labels > 4) label_stage<2>(y, label);
  if (labels > 8) label_stage<3>(y, label);
  if (labels > 16) label_stage<4>(y, label);
  if (labels > 32) label_stage<5>(y, label);
}
__device__ __forceinline__ float label_sign(int label, int labels) {
  return __popc(label & (labels - 1) & 15) & 1 ? -1.0f : 1.0f;
}

// Butterfly stages of pair distances 1 .. N/2 inside a lane.
template <int N>
__device__ __forceinline__ void lane_butterfly(float (&y)[N]) {
#pragma unroll
  for (int h = 1; h < N; h <<= 1)
#pragma unroll
    for (int i = 0; i < N; i += 2 * h)
#pragma unroll
      for (int j = i; j < i + h; ++j) {
        const float a = y[j], b = y[j + h];
        y[j] = a + b;
        y[j + h] = a - b;
      }
}

// Reductions over the 64 lanes, the same value in every lane, in a fixed
// order.
template <class Op>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, Op op) {
  auto mov = [](uint32_t x, auto ctrl) {
    return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  v = op(v, mov(v, std::integral_constant<int, 0xB1>{}));
  v = op(v, mov(v, std::integral_constant<int, 0x4E>{}));
  v = op(v, mov(v, std::integral_constant<int, 0x141>{}));
  v = op(v, mov(v, std::integral_constant<int, 0x128>{}));
  const auto r16 = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = op(r16[0], r16[1]);
  const auto r32 = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return op(r32[0], r32[1]);
}
__device__ __forceinline__ float wave_sum(float v) {
  return __builtin_bit_cast(float, wave_reduce(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
  }));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  return wave_reduce(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// Elements of 16 bytes: 8 bf16 or 4 float32.
template <bool BF16>
struct Piece {
  static constexpr int kElems = BF16 ? 8 : 4;
  static constexpr int kBytes = BF16 ? 2 : 4;
};

// 16 bytes as floats.
template <bool BF16>
__device__ __forceinline__ void unpack_piece(const uint4& r, float* v) {
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (BF16) {
      v[2 * k] = bf16_low(u[k]);
      v[2 * k + 1] = bf16_high(u[k]);
    } else {
      v[k] = __builtin_bit_cast(float, u[k]);
    }
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack_piece(const float* v) {
  if constexpr (BF16)
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  else
    return make_uint4(__builtin_bit_cast(uint32_t, v[0]), __builtin_bit_cast(uint32_t, v[1]),
                      __builtin_bit_cast(uint32_t, v[2]), __builtin_bit_cast(uint32_t, v[3]));
}

// Element i of a float32 or bf16 array.
template <bool BF16>
__device__ __forceinline__ float load_elem(const uint8_t* p, int64_t i) {
  if constexpr (BF16)
    return bf16_low(reinterpret_cast<const uint16_t*>(p)[i]);
  else
    return reinterpret_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store_elem(uint8_t* p, int64_t i, float v) {
  if constexpr (BF16)
    reinterpret_cast<uint16_t*>(p)[i] = one_bf16(v);
  else
    reinterpret_cast<float*>(p)[i] = v;
}

}  // namespace cq
