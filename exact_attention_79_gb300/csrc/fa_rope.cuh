// Rotary positions: the angle of a pair of columns at a position, as cosine and sine.
//
// A pair's frequency is held as the part of a turn that one position is, in units of
// 2^-64 (an integer modulo 2^64), so that position * frequency modulo a whole turn is one
// wrapping multiplication: exact at any 32-bit position, where fp32 radians would be off by
// 2^-24 of the angle (1/16 radian at position 2^20). The upper 32 bits of it are the
// angle within 2^-32 of a turn. Its two leading bits, rounded, are the quadrant; what is left is
// within 1/8 of a turn, where the Taylor sums of sine (to x^9) and cosine (to x^10)
// end below 2^-27.
#pragma once
#include "fa_common.cuh"
#include "fa_kernels.h"

namespace fa {

__device__ __forceinline__ float2 cos_sin_turns(unsigned long long turns, int position) {
  const uint32_t phase = static_cast<uint32_t>((turns * static_cast<unsigned long long>(static_cast<long long>(position))) >> 32);
  const uint32_t quadrant = (phase + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int>(phase - (quadrant << 30))) * 1.4629180792671596e-9f;   // 2 pi / 2^32
  const float y = x * x;
  float s = fmaf(y, 1.f / 362880.f, -1.f / 5040.f);
  s = fmaf(y, s, 1.f / 120.f);
  s = fmaf(y, s, -1.f / 6.f);
  s = fmaf(x * y, s, x);
  float c = fmaf(y, -1.f / 3628800.f, 1.f / 40320.f);
  c = fmaf(y, c, -1.f / 720.f);
  c = fmaf(y, c, 1.f / 24.f);
  c = fmaf(y, c, -0.5f);
  c = fmaf(y, c, 1.f);
  float2 r = (quadrant & 1u) ? make_float2(s, c) : make_float2(c, s);
  r.x = __uint_as_float(__float_as_uint(r.x) ^ (((quadrant + 1u) & 2u) << 30));
  r.y = __uint_as_float(__float_as_uint(r.y) ^ ((quadrant & 2u) << 30));
  return r;
}

// The pair's cosine and sine at token `t` (row b of the positions); what an axis outside 0 .. axes - 1
// would read is never read.
__device__ __forceinline__ float2 rope_at(const RopePlan& r, int pair, long long b, int t) {
  const int axis = r.axis == nullptr ? 0 : max(0, min(r.axis[pair], r.axes - 1));
  return cos_sin_turns(static_cast<unsigned long long>(r.turns[pair]), r.positions[axis * r.pos_sa + b * r.pos_sb + t]);
}

// (a, b) turned by the angle.
__device__ __forceinline__ void rotate(float& a, float& b, float2 cs) {
  const float x = fmaf(a, cs.x, -(b * cs.y));
  b = fmaf(a, cs.y, b * cs.x);
  a = x;
}

// The same for two pairs (a0, b0) and (a1, b1), each step rounded as there.
__device__ __forceinline__ void rotate2(float& a0, float& a1, float& b0, float& b1, float c0, float c1, float s0, float s1) {
  asm("{\n\t.reg .b64 a, b, c, s, t, u;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tmov.b64 c, {%4, %5};\n\tmov.b64 s, {%6, %7};\n\t"
      "mul.rn.f32x2 t, b, s;\n\tmul.rn.f32x2 u, b, c;\n\t"
      "xor.b64 t, t, 0x8000000080000000;\n\t"
      "fma.rn.f32x2 t, a, c, t;\n\tfma.rn.f32x2 u, a, s, u;\n\t"
      "mov.b64 {%0, %1}, t;\n\tmov.b64 {%2, %3}, u;\n\t}"
      : "+f"(a0), "+f"(a1), "+f"(b0), "+f"(b1) : "f"(c0), "f"(c1), "f"(s0), "f"(s1));
}
// (a0, a1) *= m
__device__ __forceinline__ void mul2_bc(float& a0, float& a1, float m) {
  asm("{\n\t.reg .b64 a, m;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 m, {%2, %2};\n\t"
      "mul.rn.f32x2 a, a, m;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1) : "f"(m));
}

}  // namespace fa
