// Layout and codes of an 8-bit pool.
//
// A block is one record of block_bytes: codes [2][Hkv][16][D], one byte each,
// then fp32 scales [2][Hkv] (K, then V), padded to a multiple of 128 bytes so
// that every (block, K|V, head) tile starts on a 128-byte line. A block copied
// or swapped as bytes takes its scales along. An element is code * scale of
// its tile, the code being an int8 in [-127, 127] or an e4m3 number.
#pragma once

#include <cuda_fp16.h>

#include <cfloat>

#include "common.cuh"

namespace pagedkv {

struct Q8Layout {
  int64_t block_bytes;
  int64_t scale_offset;  // bytes from a block's start to its scales
};

inline Q8Layout q8_layout(int32_t num_kv_heads, int32_t head_dim) {
  Q8Layout l;
  l.scale_offset = (int64_t)2 * num_kv_heads * 16 * head_dim;
  l.block_bytes = (l.scale_offset + (int64_t)8 * num_kv_heads + 127) / 128 * 128;
  return l;
}

// Scale of (block, kv, head) inside a pool.
__device__ __forceinline__ size_t q8_scale_at(const Q8Layout& l, int64_t blk, int32_t kv, int32_t g, int32_t hkv) {
  return (size_t)blk * l.block_bytes + l.scale_offset + ((size_t)kv * hkv + g) * 4;
}

// Scale and code rules of the two code types. All in fp32, with no step that
// contraction or another order could change, so codes and scales are
// reproducible bit for bit:
//   first(a)          the scale of a tile that starts afresh with largest
//                     magnitude a (0 for a tile of zeros)
//   grown(s, a)       the scale of a tile of scale s that gains rows of largest
//                     magnitude a; s when they fit. int8 grows to exactly
//                     a / 127: its error is half a step everywhere, so a step
//                     larger than needed costs every element. e4m3 grows by a
//                     power of two: its error is relative, so the larger scale
//                     costs nothing, and coding the kept rows again is exact
//                     but for values that fall below the smallest normal, by
//                     half a step there (2^-10 of the grown scale).
struct CodeInt8 {
  static constexpr float kMax = 127.0f;
  static constexpr float kInvMax = 1.0f / 127.0f;
  __device__ __forceinline__ static float grown(float s, float a) { return fmaxf(s, __fmul_rn(a, kInvMax)); }
  __device__ __forceinline__ static uint32_t encode(float x) {
    return (uint32_t)max(-127, min(127, __float2int_rn(x))) & 0xffu;
  }
  // Four codes of one word, of values within [-127.5, 127.5): adding 1.5 * 2^23
  // rounds to the integer, ties to even, and leaves it in the low bits.
  __device__ __forceinline__ static uint32_t encode4(float a, float b, float c, float d) {
    const float big = 12582912.f;
    const uint32_t ab = __byte_perm(__float_as_uint(__fadd_rn(a, big)), __float_as_uint(__fadd_rn(b, big)), 0x0040);
    const uint32_t cd = __byte_perm(__float_as_uint(__fadd_rn(c, big)), __float_as_uint(__fadd_rn(d, big)), 0x0040);
    return __byte_perm(ab, cd, 0x5410);
  }
  __device__ __forceinline__ static float decode(uint32_t c) { return (float)(int8_t)c; }
};
struct CodeE4m3 {
  static constexpr float kMax = 448.0f;
  static constexpr float kInvMax = 1.0f / 448.0f;
  __device__ __forceinline__ static float grown(float s, float a) {
    const float room = __fmul_rn(s, kMax);
    if (!(a > room)) return s;
    if (s == 0.f) return __fmul_rn(a, kInvMax);
    // smallest k with room * 2^k >= a, from exponents and significands: the quotient
    // of the two may be more than fp32 holds
    int32_t ea, er;
    const float ma = frexpf(a, &ea), mr = frexpf(room, &er);
    return ldexpf(s, ea - er + (ma > mr ? 1 : 0));
  }
  __device__ __forceinline__ static uint32_t encode(float x) {
    uint16_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(0.f), "f"(x));
    return h & 0xffu;
  }
  __device__ __forceinline__ static uint32_t encode4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | (uint32_t)hi << 16;
  }
  __device__ __forceinline__ static float decode(uint32_t c) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)c));
    return __half2float(__ushort_as_half((unsigned short)(h2 & 0xffffu)));
  }
};

// Four codes of one word -> two fp16 pairs: (b0, b1), (b2, b3) of the bytes.
__device__ __forceinline__ void q8_unpack(CodeInt8, uint32_t w, bool interleaved, uint32_t& p, uint32_t& q) {
  const uint32_t u = w ^ 0x80808080u;  // code + 128
  const uint32_t a = __byte_perm(u, 0x64646464u, interleaved ? 0x4240 : 0x4140);
  const uint32_t b = __byte_perm(u, 0x64646464u, interleaved ? 0x4341 : 0x4342);
  const uint32_t bias = 0x64806480u;   // 1024 + 128
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p) : "r"(a), "r"(bias));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(q) : "r"(b), "r"(bias));
}
__device__ __forceinline__ void q8_unpack(CodeE4m3, uint32_t w, bool interleaved, uint32_t& p, uint32_t& q) {
  if (interleaved) w = __byte_perm(w, 0, 0x3120);  // (b0, b2), (b1, b3)
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(p), "=r"(q)
      : "r"(w));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

}  // namespace pagedkv
