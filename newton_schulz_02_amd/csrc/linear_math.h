// Device arithmetic of the 8-bit linear operators: eight values of a row, and the coders that
// turn values into codes (muon_linear.h has the definitions).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace muon {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 __attribute__((aligned(2))) u32x4_at2;
typedef u32x4 __attribute__((aligned(4))) u32x4_at4;
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
  u32x4 v;
  __device__ __forceinline__ void clear() { v = 0; }
  __device__ __forceinline__ void load(const uint16_t* row, int at, int cols) {
    clear();
    if (at + 8 <= cols) {
      v = *(global_ptr<const u32x4_at2>)(row + at);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at + e < cols) v[e / 2] |= uint32_t(*(global_ptr<const uint16_t>)(row + at + e)) << (16 * (e & 1));
    }
  }
  __device__ __forceinline__ float get(int e) const { return __uint_as_float(e & 1 ? v[e / 2] & 0xffff0000u : v[e / 2] << 16); }
  __device__ __forceinline__ uint32_t bits(int e) const { return __float_as_uint(get(e)) & 0x7fffffffu; }
  // The largest magnitude as an integer: infinity lies above all numbers, NaN above infinity.
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) t = max(t, bits(e));
    return t;
  }
  __device__ __forceinline__ uint4 raw() const { return make_uint4(v[0], v[1], v[2], v[3]); }
  __device__ __forceinline__ static void store(uint16_t* row, int at, int cols, const float (&f)[8]) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
    if (at + 8 <= cols) {
      *(global_ptr<u32x4_at2>)(row + at) = o;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at + e < cols) *(global_ptr<uint16_t>)(row + at + e) = uint16_t(o[e / 2] >> (16 * (e & 1)));
    }
  }
};

template <>
struct Eight<float> {
  u32x4 v[2];
  __device__ __forceinline__ void clear() { v[0] = 0, v[1] = 0; }
  __device__ __forceinline__ void load(const float* row, int at, int cols) {
    clear();
    if (at + 8 <= cols) {
      const global_ptr<const u32x4_at4> p = (global_ptr<const u32x4_at4>)(row + at);
      v[0] = p[0], v[1] = p[1];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at + e < cols) v[e / 4][e % 4] = __float_as_uint(*(global_ptr<const float>)(row + at + e));
    }
  }
  __device__ __forceinline__ float get(int e) const { return __uint_as_float(v[e / 4][e % 4]); }
  __device__ __forceinline__ uint32_t bits(int e) const { return v[e / 4][e % 4] & 0x7fffffffu; }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) t = max(t, bits(e));
    return t;
  }
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

__device__ __forceinline__ void store_codes(int8_t* q, uint2 codes) { *reinterpret_cast<uint2*>(q) = codes; }

// Codes of a row from the bits of its largest magnitude.  The nearest integer to 127 x / max is
// that of x (127 / max), whose two roundings move it by less than 127 * 2^-23 < 2^-16, unless
// the result lies that near to the middle between two integers: there 127 |x| is compared with
// max times the middle, both exact in 64 bits (24 + 7 and 24 + 8 bits).
struct RowCoder {
  float size, up, inverse;  // up: tiny rows are scaled first, so that 127 / max stays finite
  bool lost;                // a NaN or an infinity
  __device__ __forceinline__ explicit RowCoder(uint32_t top) {
    lost = top >= 0x7f800000u;
    size = lost ? 0.0f : __uint_as_float(top);
    up = size < 0x1p-100f ? 0x1p100f : 1.0f;
    inverse = size > 0.0f ? 127.0f / (size * up) : 0.0f;
  }
  __device__ __forceinline__ float scale() const { return lost ? __uint_as_float(0x7fc00000u) : size / 127.0f; }
  __device__ __forceinline__ int one(float x) const {
    const float y = (x * up) * inverse;
    float n = rintf(y);
    if (fabsf(y - n) > 0.5f - 0x1p-14f) {
      const float low = floorf(fabsf(y));
      const double have = fabs(double(x)) * 127.0, middle = double(size) * (double(low) + 0.5);
      const bool up_one = have > middle || (have == middle && (int(low) & 1));
      n = copysignf(up_one ? low + 1.0f : low, x);
    }
    return lost ? 0 : int(n);
  }
  template <typename V>
  __device__ __forceinline__ uint2 eight(const V& v) const {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e / 4] |= uint32_t(one(v.get(e)) & 255) << (8 * (e % 4));
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
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = rintf(fminf(fmaxf(v.get(i) * inverse, -127.0f), 127.0f));
      w[i / 4] |= uint32_t((lost ? 0 : int(n)) & 255) << (8 * (i % 4));
    }
    return make_uint2(w[0], w[1]);
  }
};

__device__ __forceinline__ void decode8(uint2 q, float s, float (&f)[8]) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = float(int32_t(w[e / 4] << (24 - 8 * (e % 4))) >> 24) * s;
}

}  // namespace muon
