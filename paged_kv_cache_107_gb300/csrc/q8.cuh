// q8.cuh — 8-bit codes (pa_q8_format): widening, and the quantisation of a row.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_device.cuh"

namespace pa {

// Four codes of a word to fp16, exactly: codes (0, 1) and (2, 3), or (0, 2) and (1, 3) with
// STRIDED. E4M3 converts in hardware; an int8 code x sits in the low byte of the fp16 number
// 1024 + (x + 128), 1152 is taken off.
template <int FMT, bool STRIDED>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& a, uint32_t& b) {
  if constexpr (FMT == PA_Q8_E4M3) {
    if constexpr (STRIDED) w = __byte_perm(w, 0u, 0x3120);
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(w));
  } else {
    w ^= 0x80808080u;
    a = __byte_perm(w, 0x64646464u, STRIDED ? 0x4240 : 0x4140);
    b = __byte_perm(w, 0x64646464u, STRIDED ? 0x4341 : 0x4342);
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(a) : "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(b) : "r"(0x64806480u));
  }
}

// fp16 pair to fp32, exactly.
__device__ __forceinline__ float2 f16x2_f2(uint32_t w) {
  float2 f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(w));
  return f;
}

// Four codes of a word to fp32, exactly: an int8 code x is the low byte of 2^23 + (x + 128).
template <int FMT>
__device__ __forceinline__ void widen4_f32(uint32_t w, float (&x)[4]) {
  if constexpr (FMT == PA_Q8_E4M3) {
    uint32_t a, b;
    widen4<FMT, false>(w, a, b);
    const float2 lo = f16x2_f2(a), hi = f16x2_f2(b);
    x[0] = lo.x, x[1] = lo.y, x[2] = hi.x, x[3] = hi.y;
  } else {
    w ^= 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7650 + i)) - 8388736.f;
  }
}

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// A row's scale, and what its elements are multiplied with, from the row's largest magnitude.
// E4M3: mul = 1 / scale, both powers of two. INT8: with 2^E the exponent of t, mul = 127 * 2^-E
// and inv = 1 / (t * 2^-E), so that 127 x / t = (x mul) / (t 2^-E) stays in range for every t.
struct RowScale {
  float scale, mul, t, inv;
};

template <int FMT>
__device__ __forceinline__ RowScale row_scale(float top) {
  RowScale r;
  const uint32_t u = __float_as_uint(top);
  if constexpr (FMT == PA_Q8_E4M3) {
    // 448 = 1.75 * 2^8
    const int e = max((int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0), -126);
    r.scale = pow2f(e);
    r.mul = pow2f(-e);
    r.t = r.inv = 1.f;
  } else {
    const float t = fmaxf(top, 127.f * 1.17549435e-38f);
    const uint32_t ut = __float_as_uint(t);
    // t / 127: the remainder of the rounded product, exact, corrects it; equal to the rounded
    // quotient for every t of 11 bits (all of them tried)
    const float s0 = t * (1.f / 127.f);
    r.scale = fmaf(fmaf(-s0, 127.f, t), 1.f / 127.f, s0);
    // 127 / 64 * 2^(6 - E), E of -120 .. 127
    r.mul = __int_as_float(((133 + 127 - (int)(ut >> 23)) << 23) | 0x7e0000);
    r.t = __uint_as_float((ut & 0x7fffffu) | 0x3f800000u);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.inv) : "f"(r.t));
  }
  if (u == 0u) r.scale = 0.f;  // (its codes are 0 anyway)
  // a NaN or an infinity in the row: scale NaN, and the caller writes codes 0
  if (u >= 0x7f800000u) r.scale = __uint_as_float(0x7fc00000u);
  return r;
}

// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pair_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t pair_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Four codes of a row, packed.
//
// INT8: n = x mul is exact (7 bits by 11 at most), q0 = n inv has a relative error of 2^-22 (inv is
// the hardware's approximation), and the remainder n - q0 t, exact in one multiply-add (t has
// 11 bits), corrects it to 2^-44 before the last rounding. Where the quotient is a tie (an integer and a half, a number of fp32) that rounding
// gives it exactly; where it is none, it lies at least 2^-21 of itself from the next tie (a
// quotient of two 11-bit numbers, times 127), which one rounding of 2^-24 does not cross. So the
// integer rounding after it, an addition of 1.5 * 2^23, goes the way of the exact quotient.
template <int FMT>
__device__ __forceinline__ uint32_t quantise4(const RowScale& r, float x0, float x1, float x2,
                                              float x3) {
  if constexpr (FMT == PA_Q8_E4M3) {
    const uint64_t mul = pair2(r.mul, r.mul);
    const uint64_t lo = pair_mul(pair2(x0, x1), mul), hi = pair_mul(pair2(x2, x3), mul);
    uint32_t w;
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
        : "=r"(w)
        : "f"(__uint_as_float((uint32_t)lo)), "f"(__uint_as_float((uint32_t)(lo >> 32))),
          "f"(__uint_as_float((uint32_t)hi)), "f"(__uint_as_float((uint32_t)(hi >> 32))));
    return w;
  } else {
    const uint64_t mul = pair2(r.mul, r.mul), inv = pair2(r.inv, r.inv), t = pair2(-r.t, -r.t);
    const uint64_t magic = pair2(12582912.f, 12582912.f);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t n = pair_mul(i ? pair2(x2, x3) : pair2(x0, x1), mul);
      const uint64_t q0 = pair_mul(n, inv);
      const uint64_t q = pair_fma(pair_fma(q0, t, n), inv, q0);
      const uint64_t k = pair_add(q, magic);
      c[2 * i] = (uint32_t)k;
      c[2 * i + 1] = (uint32_t)(k >> 32);
    }
    return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  }
}

}  // namespace pa
