// fp4_quant.cuh: 16 neighbouring elements of a row as the 4-bit quantiser takes them, for
// its own kernels and for the product that quantises a row on the way.
#pragma once

#include <type_traits>

#include "fp4.cuh"

namespace dg {

constexpr int kUnit = 16;  // elements a thread takes at a time

// Where 16-byte blocks may be read: the bytes from a matrix's first element to its last,
// gaps between its rows among them.
struct Span {
  const uint8_t *begin, *end;
};

// 16 neighbouring elements as loaded.
template <typename T>
struct Unit16 {
  static constexpr int kWords = sizeof(T) * kUnit / 4;
  uint32_t w[kWords];

  // The first `valid` of the elements at p, zeros after them.  Rows that do not start on
  // 16 bytes are read in the 16-byte blocks that hold them, shifted into place (element
  // by element 1000 x 8191 bf16 took 13.4 us instead of 8.8).
  __device__ __forceinline__ void load(const T* p, int valid, const Span& span) {
    const uint8_t* const at = reinterpret_cast<const uint8_t*>(p);
    const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(p)) & 15u;
    const uint4* const block = reinterpret_cast<const uint4*>(at - off);
    if (valid >= kUnit && off == 0) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 a = __ldg(block + i);
        w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
      }
    } else if (valid >= kUnit && at - off >= span.begin &&
               at - off + 4 * kWords + 16 <= span.end) {
      uint32_t v[kWords + 4];
#pragma unroll
      for (int i = 0; i < kWords / 4 + 1; ++i) {
        const uint4 a = __ldg(block + i);
        v[4 * i] = a.x; v[4 * i + 1] = a.y; v[4 * i + 2] = a.z; v[4 * i + 3] = a.w;
      }
      if (off & 8u) {
#pragma unroll
        for (int j = 0; j < kWords + 2; ++j) v[j] = v[j + 2];
      }
      if (off & 4u) {
#pragma unroll
        for (int j = 0; j < kWords + 1; ++j) v[j] = v[j + 1];
      }
#pragma unroll
      for (int j = 0; j < kWords; ++j)
        w[j] = sizeof(T) == 2 && (off & 2u) ? __funnelshift_r(v[j], v[j + 1], 16) : v[j];
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
      for (int j = 0; j < kUnit; ++j) {
        if (j >= valid) continue;
        if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(float(p[j]));
        else w[j / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(p)[j]) << (16 * (j & 1));
      }
    }
  }
  // Elements 2 j and 2 j + 1.
  __device__ __forceinline__ float2 pair(int j) const {
    if constexpr (sizeof(T) == 4) {
      return make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
    } else if constexpr (std::is_same<T, __half>::value) {
      __half2 h;
      __builtin_memcpy(&h, &w[j], 4);
      return __half22float2(h);
    } else {
      return make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
    }
  }
  // The largest finite magnitude; `odd`: there is a non-finite element.
  __device__ __forceinline__ float amax(bool& odd) const {
    float m;
    if constexpr (sizeof(T) == 4) {
      uint32_t most = 0;
#pragma unroll
      for (int j = 0; j < kUnit; ++j) most = max(most, w[j] & 0x7fffffffu);
      m = __uint_as_float(most);
    } else {
      uint32_t most = 0;
#pragma unroll
      for (int j = 0; j < kWords; ++j) most = __vmaxu2(most, w[j] & 0x7fff7fffu);
      const uint16_t h = uint16_t(max(most & 0xffffu, most >> 16));
      T v;
      __builtin_memcpy(&v, &h, 2);
      if constexpr (std::is_same<T, __half>::value) m = __half2float(v);
      else m = __bfloat162float(v);
    }
    odd = !(m < INFINITY);
    if (odd) {
      m = 0.f;
#pragma unroll
      for (int j = 0; j < kUnit / 2; ++j) {
        const float2 x = pair(j);
        if (fabsf(x.x) < INFINITY) m = fmaxf(m, fabsf(x.x));
        if (fabsf(x.y) < INFINITY) m = fmaxf(m, fabsf(x.y));
      }
    }
    return m;
  }
};

// (x a, y a), one instruction.
__device__ __forceinline__ float2 mul2(float2 x, float a) {
  float2 r;
  asm("{\n\t.reg .b64 p, q;\n\t"
      "mov.b64 p, {%2, %3};\n\t"
      "mov.b64 q, {%4, %4};\n\t"
      "mul.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(a));
  return r;
}

}  // namespace dg
