// Device helpers of the 8-bit path's kernels.
#pragma once

#include "hxq_device.h"

namespace hxq {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kF32 = 0, kBf16 = 1, kE4m3 = 2;  // hxq_dtype

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two float32 as bf16 bits (nearest, ties to even), a in the low half: one
// instruction here (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}
__device__ __forceinline__ uint16_t to_bf16(float a) { return __builtin_bit_cast(uint16_t, (__bf16)a); }

template <int DT>
struct Elem;
template <>
struct Elem<kF32> {
  static constexpr int size = 4;
};
template <>
struct Elem<kBf16> {
  static constexpr int size = 2;
};

// Eight consecutive elements as fp32.  Rows of an odd width start at any
// element, so the 16-byte loads are declared with the element's alignment
// only (the hardware takes them in one instruction either way).
template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&v)[8]) {
  if constexpr (DT == kF32) {
    struct __attribute__((packed, aligned(4))) P {
      float f[4];
    };
    const P* p = reinterpret_cast<const P*>(static_cast<const float*>(base) + at);
    const P a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a.f[i];
      v[4 + i] = b.f[i];
    }
  } else {
    struct __attribute__((packed, aligned(2))) P {
      uint32_t u[4];
    };
    const P a = *reinterpret_cast<const P*>(static_cast<const uint16_t*>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a.u[i] << 16);
      v[2 * i + 1] = __uint_as_float(a.u[i] & 0xffff0000u);
    }
  }
}

template <int DT>
__device__ __forceinline__ float load1(const void* base, int64_t at) {
  if constexpr (DT == kF32) return static_cast<const float*>(base)[at];
  return bf16_to_f32(static_cast<const uint16_t*>(base)[at]);
}

// Columns col .. col + 7 of a row of K (zeros past its end).
template <int DT>
__device__ __forceinline__ void load_row8(const void* base, int64_t row0, int col, int K, float (&v)[8]) {
  if (col + 8 <= K) {
    load8<DT>(base, row0 + col, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = col + i < K ? load1<DT>(base, row0 + col + i) : 0.f;
  }
}

template <int DT>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&v)[8]) {
  if constexpr (DT == kF32) {
    struct __attribute__((packed, aligned(4))) P {
      float f[4];
    };
    P* p = reinterpret_cast<P*>(static_cast<float*>(base) + at);
    P a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a.f[i] = v[i];
      b.f[i] = v[4 + i];
    }
    p[0] = a;
    p[1] = b;
  } else {
    struct __attribute__((packed, aligned(2))) P {
      uint32_t u[4];
    };
    P a;
#pragma unroll
    for (int i = 0; i < 4; ++i) a.u[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<P*>(static_cast<uint16_t*>(base) + at) = a;
  }
}

template <int DT>
__device__ __forceinline__ void store_row8(void* base, int64_t row0, int col, int K, const float (&v)[8]) {
  if (col + 8 <= K) {
    store8<DT>(base, row0 + col, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (col + i < K) {
        if constexpr (DT == kF32)
          static_cast<float*>(base)[row0 + col + i] = v[i];
        else
          static_cast<uint16_t*>(base)[row0 + col + i] = to_bf16(v[i]);
      }
    }
  }
}

// The same for float32, past the caches.
__device__ __forceinline__ void stream_row8(float* base, int64_t row0, int col, int K, const float (&v)[8]) {
  typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
  float* p = base + row0 + col;
  if (col + 8 <= K) {
    __builtin_nontemporal_store(vec{v[0], v[1], v[2], v[3]}, reinterpret_cast<vec*>(p));
    __builtin_nontemporal_store(vec{v[4], v[5], v[6], v[7]}, reinterpret_cast<vec*>(p + 4));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < K) p[i] = v[i];
  }
}

// The e8m0 byte of the smallest power of two p >= 2^-126 with a <= 448 p, for
// the bit pattern of a finite a >= 0: 448 = 1.75 * 2^8, so the exponent field
// less 8, one more where the mantissa passes 1.75 (the addition then carries).
__device__ __forceinline__ int e8m0_of(uint32_t bits) { return max((int)((bits + 0x1fffffu) >> 23) - 8, 1); }

// The magnitude's bits, 0 for an infinity or NaN: they take no part in a
// group's scale (and become NaN, so they stay where they are).
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}

// Largest of the 16 lanes of a DPP row, in every lane.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xb1, 0xf, 0xf, false));   // pairs
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4e, 0xf, 0xf, false));   // quads
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, false));  // 8 lanes
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, false));  // 16 lanes
  return v;
}

// 8 values over a power of two (as its inverse) to e4m3, nearest, ties to
// even: |v * inv| <= 448, so nothing saturates; infinities and NaN give NaN.
__device__ __forceinline__ uint2 to_e4m3x8(const float (&v)[8], float inv) {
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = v[i] * inv;
    t[i] = fabsf(v[i]) < __builtin_inff() ? s : __builtin_nanf("");
  }
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(t[4], t[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(t[6], t[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// One thread's 8 columns of a 128-column group (16 lanes of a DPP row hold the
// group): returns the e4m3 bytes, and the group's e8m0 byte in `byte`.
__device__ __forceinline__ uint2 quant_group(const float (&v)[8], int& byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, finite_bits(v[i]));
  byte = e8m0_of(row16_max(m));
  return to_e4m3x8(v, __uint_as_float((uint32_t)(254 - byte) << 23));
}

// 8 e4m3 bytes times a power of two as bf16 (exact: 4 significant bits).
__device__ __forceinline__ bf16x8 widen8(int lo, int hi, float p) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, p, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, p, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, p, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, p, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

}  // namespace hxq
