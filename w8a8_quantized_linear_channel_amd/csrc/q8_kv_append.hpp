// What the appends to the paged 8-bit key/value cache share on the device
// (kv_append.hip, kv_append_norm.hip).
#pragma once
#include "q8_device.hpp"
#include "q8_kv.hpp"
#include "q8_kv_plan.hpp"

namespace q8 {
namespace {

// 8 consecutive elements as floats
template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t off, float* v) {
  if constexpr (DT == DT_F32) {
    const v4i* p = (const v4i*)((const float*)base + off);
    Chunk<DT>::decode(p[0], v);
    Chunk<DT>::decode(p[1], v + 4);
  } else {
    Chunk<DT>::decode(*(const v4i*)((const uint16_t*)base + off), v);
  }
}
template <int DT>
__device__ __forceinline__ void store8(void* base, int64_t off, const float* v) {
  if constexpr (DT == DT_F32) {
    v4f* p = (v4f*)((float*)base + off);
    p[0] = v4f{v[0], v[1], v[2], v[3]};
    p[1] = v4f{v[4], v[5], v[6], v[7]};
  } else {
    v4i o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (int)pack2_out<DT>(v[2 * i], v[2 * i + 1]);
    *(v4i*)((uint16_t*)base + off) = o;
  }
}

// cos and sin of the 8 features 8c .. 8c+7 of a head at a position, as their rotation uses them:
// 8 of each for pairs (i, i + r), 4 of each for pairs (2 i, 2 i + 1).
struct Turn {
  float co[8], si[8];
};
__device__ __forceinline__ void load_turn(const AppendArgs& a, int c, int pos, Turn& t) {
  const int half = a.rot >> 1;
  const int64_t row = (int64_t)(pos < a.positions ? pos : a.positions - 1) * half;
  if (a.interleaved) {
    Chunk<DT_F32>::decode(*(const v4i*)(a.cos + row + 4 * c), t.co);
    Chunk<DT_F32>::decode(*(const v4i*)(a.sin + row + 4 * c), t.si);
  } else {
    const int j = 8 * c < half ? 8 * c : 8 * c - half;
    load8<DT_F32>(a.cos, row + j, t.co);
    load8<DT_F32>(a.sin, row + j, t.si);
  }
}
// Every product and the sum are rounded on their own (no contraction), so the codes do not depend on
// how the compiler pairs them.  w: the partner features (pairs (i, i + r) only), low: v is the first
// of the two.
__device__ __forceinline__ void turn8(const Turn& t, bool interleaved, bool low, float* v, const float* w) {
#pragma clang fp contract(off)
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = v[2 * i], r = v[2 * i + 1];
      v[2 * i] = p * t.co[i] - r * t.si[i];
      v[2 * i + 1] = r * t.co[i] + p * t.si[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float side = low ? -w[i] : w[i];
      v[i] = v[i] * t.co[i] + side * t.si[i];      // (a cos - b sin: the negated product rounds alike)
    }
  }
}
// The exponent byte of a page and head: the least b with amax <= 448 2^(b - 127).
__device__ __forceinline__ int exponent_byte(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int b = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return b < 0 ? 0 : (b > 254 ? 254 : b);
}

// Four codes re-expressed at a scale 2^-shift times as fine
__device__ __forceinline__ uint32_t rescale4(uint32_t w, int shift) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  return pack4_e4m3(__builtin_ldexpf(lo[0], shift), __builtin_ldexpf(lo[1], shift), __builtin_ldexpf(hi[0], shift),
                    __builtin_ldexpf(hi[1], shift));
}

}  // namespace
}  // namespace q8
