// Device building blocks shared by the atom-wise dense operators (norm.hip,
// dense.hip): element types, loads and stores of short runs, activations.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/eec.h"

namespace eec {
namespace dense {

typedef __bf16 bf16;
typedef _Float16 f16;
struct e4m3 {
  uint8_t bits;
};
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Elements of one 16-byte access.
template <typename T>
constexpr int VEC = 16 / (int)sizeof(T);

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef i32x4 i32x4_any __attribute__((aligned(1)));

// N consecutive elements as they are stored, of which the first `valid` exist; the
// others read as zero.  The pointer needs only its elements' alignment: 16-byte
// global accesses of any alignment are ordinary here (rows of odd width), and an
// aligned address makes the same instruction fast.  ONCE: what nobody reads again
// soon passes the L2 by, in both directions (norm backward 16384 x 4096 bf16: 157 us,
// 145 us with its stores so).
template <bool ONCE = false, typename T, int N>
__device__ __forceinline__ void load_raw(const T* __restrict__ p, int64_t valid, T (&v)[N]) {
  if (valid >= N) {
    if constexpr (ONCE && sizeof(v) % 16 == 0) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(v) / 16; ++i) {
        const i32x4 q = __builtin_nontemporal_load((const i32x4_any*)p + i);
        __builtin_memcpy((char*)v + 16 * i, &q, 16);
      }
    } else {
      __builtin_memcpy(v, p, sizeof(v));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < valid ? p[i] : T{};
  }
}
// The same as floats.
template <bool ONCE = false, typename T, int N>
__device__ __forceinline__ void load_run(const T* __restrict__ p, int64_t valid, float (&v)[N]) {
  T t[N];
  load_raw<ONCE>(p, valid, t);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = (float)t[i];
}

// The first `valid` of N floats, each rounded once to T (to nearest even); past the
// L2 unless `once` (uniform) is false.
template <typename T, int N>
__device__ __forceinline__ void store_run(T* __restrict__ p, int64_t valid, const float (&v)[N], bool once = true) {
  if (valid >= N) {
    T t[N];
#pragma unroll
    for (int i = 0; i < N; ++i) t[i] = (T)v[i];
    if constexpr (sizeof(t) == 16) {
      i32x4 q;
      __builtin_memcpy(&q, t, 16);
      if (once)
        __builtin_nontemporal_store(q, (i32x4_any*)p);
      else
        *(i32x4_any*)p = q;
    } else {
      __builtin_memcpy(p, t, sizeof(t));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < valid) p[i] = (T)v[i];
  }
}

// The same in e4m3 (values within +-448, or NaN, which keeps its code).
template <int N>
__device__ __forceinline__ void store_run_e4m3(uint8_t* __restrict__ p, int64_t valid, const float (&v)[N]) {
  static_assert(N % 4 == 0, "e4m3 runs are packed four to a register");
  int q[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    q[i] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
    q[i] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], q[i], true);
  }
  if (valid >= N) {
    __builtin_memcpy(p, q, N);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < valid) p[i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
  }
}

// exp(x) from k = x log2(e) as rounded and `lost`, what that rounding left out.
__device__ __forceinline__ float exp_and(float k, float lost) {
  const float e = __builtin_amdgcn_exp2f(k);
  return __builtin_fmaf(e, lost * 0.69314718055994531f, e);
}
// sigmoid(z) = 1 / (1 + exp(-z)) and sigmoid(-z), so that z sigmoid(z) and its slope are
// within 16 x 2^-24 of their size before a float32 output is rounded, down to
// exp(-|z|) = 2^-126: both from exp(-|z|), so that neither cancels, and its argument keeps
// what its rounding loses (130 x 2^-24 at z = -87).  Beside a 16-bit output all of that is
// below the output's rounding, and the shorter form has it down to z = -88 (32768 x 512 x 512
// bf16 forward with SiLU: 31.1 us in the long form, 29.5 in the short one).
template <typename O>
__device__ __forceinline__ void sigmoids(float z, float& plus, float& minus) {
  constexpr float C = -1.44269504088896341f, C_LOW = (float)(-1.44269504088896341 - (double)C);
  if constexpr (sizeof(O) == 4) {
    const float a = fabsf(z), k = a * C;
    const float e = a > 200.f ? 0.f : exp_and(k, __builtin_fmaf(a, C, -k) + a * C_LOW);
    const float r = __builtin_amdgcn_rcpf(1.f + e), small = e * r;
    plus = z < 0.f ? small : r;
    minus = z < 0.f ? r : small;
  } else {
    plus = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * C));
    minus = 1.f - plus;
  }
}

// GELU is z Phi(z), with Phi(-|z|) = erfc(|z| / sqrt 2) / 2.  For z < 0 that is taken as it
// is: 1 + erf would cancel (4 % off at z = -5 in float32, nothing left at -6).
//   half_erfcx   erfc(a) exp(a^2) / 2 at a = |z| / sqrt 2, a polynomial in t = 1 / (1 + 0.4 a)
//                fitted to a relative 5.9e-8 over 0 <= a <= 9.6, 7 x 2^-24 with its roundings
//                and those of t;
//   gauss        exp(-z^2 / 2).  Beside a float32 output what z^2 and its product with
//                log2(e) lose in rounding is put back (up to 120 x 2^-24 at |z| = 13); in 16
//                bits it is far below the output's rounding.
// So z Phi(z) and its slope are within 16 x 2^-24 of their size before they are rounded to
// the output, down to exp(-z^2 / 2) = 2^-126.  (32768 x 512 x 512 bf16 forward with GELU:
// 36.2 us, 34.5 with 1 + erf to 1.5e-7 in five terms.)
__device__ __forceinline__ float half_erfcx(float z) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(fabsf(z), 0.4f * 0.70710678118654752f, 1.f));
  float p = 4.047512263e-02f;
  p = __builtin_fmaf(p, t, -1.364949644e-01f);
  p = __builtin_fmaf(p, t, 7.599072903e-02f);
  p = __builtin_fmaf(p, t, 9.722977877e-02f);
  p = __builtin_fmaf(p, t, 7.326742262e-02f);
  p = __builtin_fmaf(p, t, 1.961983591e-01f);
  p = __builtin_fmaf(p, t, 2.011585832e-01f);
  p = __builtin_fmaf(p, t, 2.265470028e-01f);
  p = __builtin_fmaf(p, t, 2.256280333e-01f);
  return p * t * 0.5f;
}
template <typename O>
__device__ __forceinline__ float gauss(float z) {
  constexpr float C = -0.72134752044448170f, C_LOW = (float)(-0.72134752044448170 - (double)C);
  const float h = z * z, k = h * C;
  if constexpr (sizeof(O) == 4) {
    const float lost = __builtin_fmaf(h, C, -k) + (__builtin_fmaf(z, z, -h) * C + h * C_LOW);
    return h > 400.f ? 0.f : exp_and(k, lost);  // an infinity has no rest; a NaN stays one
  } else {
    return __builtin_amdgcn_exp2f(k);
  }
}

// act in place, for an output of type O; the branch is uniform over the launch and taken once per run.
template <typename O, int N>
__device__ __forceinline__ void act_values(float (&z)[N], int act) {
  if (act == EEC_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float p, q;
      sigmoids<O>(z[i], p, q);
      z[i] *= p;
    }
  } else if (act == EEC_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float q = half_erfcx(z[i]), e = gauss<O>(z[i]);
      z[i] = z[i] < 0.f ? z[i] * q * e : z[i] * (1.f - q * e);
    }
  } else if (act == EEC_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = z[i] < 0.f ? 0.f : z[i];  // a NaN stays one
  }
}
// g act'(z) in place of g.
template <typename O, int N>
__device__ __forceinline__ void act_slopes(float (&g)[N], const float (&z)[N], int act) {
  if (act == EEC_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float p, q;
      sigmoids<O>(z[i], p, q);
      g[i] *= p * (1.f + z[i] * q);
    }
  } else if (act == EEC_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float q = half_erfcx(z[i]), e = gauss<O>(z[i]), d = z[i] * 0.39894228040143268f;
      g[i] *= z[i] < 0.f ? e * (q + d) : 1.f + e * (d - q);
    }
  } else if (act == EEC_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) g[i] *= z[i] > 0.f ? 1.f : 0.f;
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
// Maximum that keeps a NaN.
__device__ __forceinline__ float nan_max(float a, float b) { return (a > b || a != a) ? a : b; }
__device__ __forceinline__ float wave_nan_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = nan_max(v, __shfl_xor(v, o));
  return v;
}

}  // namespace dense
}  // namespace eec
