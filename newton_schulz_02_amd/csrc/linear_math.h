// Device arithmetic of the 8-bit linear operators: eight values of a row, and the coders that
// turn values into codes (muon_linear.h has the definitions).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace muon {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 __attribute__((aligned(2))) u32x4_at2;
typedef u32x4 __attribute__((aligned(4))) u32x4_at4;
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
template <typename T>
using global_ptr = __attribute__((address_space(1))) T*;

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// Converted together, in one instruction (apart, two and two more to join them).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// Eight consecutive values of a row, read with 16-byte accesses at any alignment of the element
// type (gfx950 takes them); zeros behind the row's end.
template <typename T>
struct Eight;

template <>
struct Eight<uint16_t> {
  static constexpr bool kShort = true;  // few bits: see RowCoder
  u32x4 v;
  __device__ __forceinline__ void clear() { v = 0; }
  __device__ __forceinline__ void load(const uint16_t* row, int at, int cols) {
    clear();
    if (at + 8 <= cols) {
      v = *(global_ptr<const u32x4_at2>)(row + at);
    } else if (at < cols) {
      // All loads at once, without a branch for each.
      uint16_t x[7];
#pragma unroll
      for (int e = 0; e < 7; ++e) x[e] = *(global_ptr<const uint16_t>)(row + min(at + e, cols - 1));
#pragma unroll
      for (int e = 0; e < 7; ++e) v[e / 2] |= (at + e < cols ? uint32_t(x[e]) : 0u) << (16 * (e & 1));
    }
  }
  __device__ __forceinline__ float get(int e) const { return __uint_as_float(e & 1 ? v[e / 2] & 0xffff0000u : v[e / 2] << 16); }
  // Largest magnitudes as integers: infinity lies above all numbers, NaN above infinity.  Two at a
  // time, as bf16 (eight apart, as floats, were a third of a row's arithmetic).
  struct Tops {
    u16x2 m[4] = {};
    __device__ __forceinline__ void take(const Eight& x) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = x.v[i] & 0x7fff7fffu;
        m[i] = __builtin_elementwise_max(m[i], __builtin_bit_cast(u16x2, w));
      }
    }
    __device__ __forceinline__ uint32_t get(int e) const { return uint32_t(m[e / 2][e & 1]) << 16; }
    __device__ __forceinline__ uint32_t all() const {
      const u16x2 t = __builtin_elementwise_max(__builtin_elementwise_max(m[0], m[1]), __builtin_elementwise_max(m[2], m[3]));
      return uint32_t(max(t[0], t[1])) << 16;
    }
  };
  __device__ __forceinline__ uint4 raw() const { return make_uint4(v[0], v[1], v[2], v[3]); }
  __device__ __forceinline__ static void store(uint16_t* row, int at, int cols, const float (&f)[8]) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
    if (at + 8 <= cols) {
      __builtin_nontemporal_store(o, (global_ptr<u32x4_at2>)(row + at));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at + e < cols) *(global_ptr<uint16_t>)(row + at + e) = uint16_t(o[e / 2] >> (16 * (e & 1)));
    }
  }
};

template <>
struct Eight<float> {
  static constexpr bool kShort = false;
  u32x4 v[2];
  __device__ __forceinline__ void clear() { v[0] = 0, v[1] = 0; }
  __device__ __forceinline__ void load(const float* row, int at, int cols) {
    clear();
    if (at + 8 <= cols) {
      const global_ptr<const u32x4_at4> p = (global_ptr<const u32x4_at4>)(row + at);
      v[0] = p[0], v[1] = p[1];
    } else if (at < cols) {
      float x[7];
#pragma unroll
      for (int e = 0; e < 7; ++e) x[e] = *(global_ptr<const float>)(row + min(at + e, cols - 1));
#pragma unroll
      for (int e = 0; e < 7; ++e) v[e / 4][e % 4] = at + e < cols ? __float_as_uint(x[e]) : 0u;
    }
  }
  __device__ __forceinline__ float get(int e) const { return __uint_as_float(v[e / 4][e % 4]); }
  __device__ __forceinline__ uint32_t bits(int e) const { return v[e / 4][e % 4] & 0x7fffffffu; }
  struct Tops {
    uint32_t m[8] = {};
    __device__ __forceinline__ void take(const Eight& x) {
#pragma unroll
      for (int e = 0; e < 8; ++e) m[e] = max(m[e], x.bits(e));
    }
    __device__ __forceinline__ uint32_t get(int e) const { return m[e]; }
    __device__ __forceinline__ uint32_t all() const {
      return max(max(max(m[0], m[1]), max(m[2], m[3])), max(max(m[4], m[5]), max(m[6], m[7])));
    }
  };
  __device__ __forceinline__ static void store(float* row, int at, int cols, const float (&f)[8]) {
    if (at + 8 <= cols) {
      const global_ptr<u32x4_at4> p = (global_ptr<u32x4_at4>)(row + at);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __float_as_uint(f[4 * h + i]);
        p[h] = o;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at + e < cols) *(global_ptr<float>)(row + at + e) = f[e];
    }
  }
};

// Maximum over the 16 lanes of each row of a wave, and over the wave: rotations within a row, and
// scalars.  All lanes have to be active.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x128, 0xf, 0xf, true)));  // row_ror:8
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x124, 0xf, 0xf, true)));
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x122, 0xf, 0xf, true)));
  return max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x121, 0xf, 0xf, true)));
}
__device__ __forceinline__ uint32_t max64(uint32_t v) {
  v = max16(v);
  return max(max(uint32_t(__builtin_amdgcn_readlane(int(v), 0)), uint32_t(__builtin_amdgcn_readlane(int(v), 16))),
             max(uint32_t(__builtin_amdgcn_readlane(int(v), 32)), uint32_t(__builtin_amdgcn_readlane(int(v), 48))));
}

// Codes to global memory.
__device__ __forceinline__ void store_codes(int8_t* q, uint2 codes) { __builtin_nontemporal_store(u32x2{codes.x, codes.y}, (global_ptr<u32x2>)(q)); }

// Low bytes of four words, as one.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u), hi = __builtin_amdgcn_perm(d, c, 0x04000c0cu);
  return lo | hi;
}

// 3 * 2^22: a float from 2^23 to 2^24 has steps of 1, so the sum of this and a small value rounds to
// an integer, ties to even, and its low byte is that integer's.
constexpr float kToInt = 12582912.0f;

// Codes of a row from the bits of its largest magnitude.  The nearest integer n to 127 x / max is
// that of x (127 / max), whose error is below 127 * 2^-24 < 2^-17, unless it lies that near to the
// middle between two integers.
//
// bf16 values (8 bits) often lie in the middle.  Their quotient is corrected by its residual: with
// y = x (127 / max) rounded, r = 127/128 x - y (max / 128) is exact (a few bits, a few steps of y
// times max), and y + r (128 / max) rounds to the middle where the quotient is there.  Elsewhere
// the quotient of a 15-bit and an 8-bit number of up to 2^(7-j) is 2^(-9-j) from it, far more than
// y's error.
//
// A group of fp32 codes with one that comes within 2^-16 of the middle is made again: 127 |x| is
// compared with max times the middle, both exact in 64 bits (24 + 7 and 24 + 8 bits).  (With this
// for bf16 too, nearly every group was: 16384 rows of 4096 took 44.1 us, and 39.7 with the residual.)
struct RowCoder {
  float size, inverse;
  bool lost;  // a NaN or an infinity
  bool tiny;  // scaled by 2^100 first, so that 127 / max stays finite
  __device__ __forceinline__ explicit RowCoder(uint32_t top) : RowCoder(top, 0.0f) {
    inverse = size > 0.0f ? 127.0f / (tiny ? size * 0x1p100f : size) : 0.0f;
  }
  // Of another coder's maximum and `inverse`.
  __device__ __forceinline__ RowCoder(uint32_t top, float inv) : inverse(inv) {
    lost = top >= 0x7f800000u;
    size = lost ? 0.0f : __uint_as_float(top);
    tiny = size < 0x1p-100f;
  }
  __device__ __forceinline__ float scale() const { return lost ? __uint_as_float(0x7fc00000u) : size / 127.0f; }
  __device__ __forceinline__ uint32_t exact(float x) const {
    const float y = (tiny ? x * 0x1p100f : x) * inverse;
    float n = rintf(y);
    if (fabsf(y - n) > 0.5f - 0x1p-13f) {
      const float low = floorf(fabsf(y));
      const double have = fabs(double(x)) * 127.0, middle = double(size) * (double(low) + 0.5);
      n = copysignf(have > middle || (have == middle && (int(low) & 1)) ? low + 1.0f : low, x);
    }
    return uint32_t(int(n));
  }
  // The codes of N values (a multiple of 4), x(0) .. x(N - 1); SHORT: bf16 numbers.
  template <int N, bool SHORT, typename X>
  __device__ __forceinline__ void codes(uint32_t (&w)[N / 4], X&& x) const {
    uint32_t n[N];
    float near = tiny ? 1.0f : 0.0f;
    if constexpr (SHORT) {
      const float part = size * 0x1p-7f, back = inverse * (128.0f / 127.0f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float y = x(i) * inverse, r = fmaf(-y, part, x(i) * (127.0f / 128.0f));
        n[i] = __float_as_uint(fmaf(r, back, y) + kToInt);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float r = fmaf(x(i), inverse, kToInt);
        near = fmaxf(near, fabsf(fmaf(x(i), inverse, kToInt - r)));
        n[i] = __float_as_uint(r);
      }
    }
    if (__builtin_expect(near > 0.5f - 0x1p-16f, 0)) {  // out of the way of the instructions that run
#pragma unroll
      for (int i = 0; i < N; ++i) n[i] = exact(x(i));
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = lost ? 0u : low_bytes(n[4 * i], n[4 * i + 1], n[4 * i + 2], n[4 * i + 3]);
  }
  template <typename V>
  __device__ __forceinline__ uint2 eight(const V& v) const {
    uint32_t w[2];
    codes<8, V::kShort>(w, [&](int e) { return v.get(e); });
    return make_uint2(w[0], w[1]);
  }
};

// Codes of a block.  With max = m 2^E, 1 <= m < 2, the smallest power of two s with max <= 127 s
// is 2^(E-6) where m <= 127/64, else 2^(E-5); x / s is exact.
struct BlockCoder {
  int e;
  bool lost;
  __device__ __forceinline__ explicit BlockCoder(uint32_t top) {
    lost = top >= 0x7f800000u;
    e = int(top >> 23) - 127 - 6 + ((top & 0x7fffffu) > 0x7e0000u ? 1 : 0);
    e = min(121, max(-126, e));
  }
  __device__ __forceinline__ float scale() const { return __uint_as_float(lost ? 0x7fc00000u : uint32_t(e + 127) << 23); }
  template <typename V>
  __device__ __forceinline__ uint2 eight(const V& v) const {
    const float inverse = __uint_as_float(uint32_t(127 - e) << 23);
    uint32_t n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = __float_as_uint(__builtin_amdgcn_fmed3f(v.get(i) * inverse, -127.0f, 127.0f) + kToInt);
    return make_uint2(lost ? 0u : low_bytes(n[0], n[1], n[2], n[3]), lost ? 0u : low_bytes(n[4], n[5], n[6], n[7]));
  }
};

// Code e (0..3) of a word.
__device__ __forceinline__ float code_of(uint32_t w, int e) { return float(int32_t(w << (24 - 8 * e)) >> 24); }

__device__ __forceinline__ void decode8(uint2 q, float s, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = code_of(e < 4 ? q.x : q.y, e % 4) * s;
}

}  // namespace muon
