// View of a paged key-value cache held in 8 bits with a scale for each block of tokens and head, and the codes' arithmetic.
//
// A page holds page_size slots of every key/value head; `block` slots that follow one another (block divides page_size)
// share a scale. The value of a code is code * scale, whichever type the code is of: int8, or E4M3.
#pragma once
#include <cuda_fp8.h>

#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sage {

// c.k, c.v and the strides are in bytes; c.mass and c.pos are null.
struct Q8View {
  PagedView c;
  float* ks; float* vs;  // [num_pages, hkv, blocks]
  int block, blocks;     // slots per scale, scales per page
  int k_type, v_type;    // SAGE_S8 or SAGE_E4M3
};

// The least scale: smaller magnitudes count as zero, and no reciprocal overflows.
constexpr float kLeastScale = 0x1p-100f;

// Host: checks a cache description and its layout; *align: the largest of 1, 2, 4, 8, 16 that every address, stride
// and the head_dim are multiples of.
int make_q8_view(const sage_q8_cache* cache, int batch, int heads_kv, int head_dim, int tensor_layout, Q8View* view,
                 int* align);

__device__ __forceinline__ int64_t scale_at(const Q8View& v, int page, int h, int slot) {
  return ((int64_t)page * v.c.hkv + h) * v.blocks + slot / v.block;
}

// Scale that values up to `most` need. int8: most / 127, which maps the largest to the last code. E4M3: the smallest
// power of two with most <= 448 scale: a floating code gains nothing from a finer scale, and codes that move to a larger
// scale lose no bit but those that become subnormal.
template <int TYPE>
__device__ __forceinline__ float needed_scale(float most) {
  float s;
  if (TYPE == SAGE_S8) {
    s = __fdiv_rn(most, 127.0f);
  } else {
    // most = m 2^e with m in [1, 2); 448 = 1.75 * 2^8
    const unsigned bits = __float_as_uint(most);
    const int e = (int)(bits >> 23) + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0) - 8;  // (subnormals end below the least scale)
    s = e > 0 ? __uint_as_float((unsigned)min(e, 254) << 23) : 0.f;
  }
  return fmaxf(s, kLeastScale);
}
// Codes of eight values in units of the scale, rounded to nearest even. (int8: the low byte of 3 * 2^22 + u, whose unit is one:
// u is rounded as by rint. The product that gave u must be rounded before: by __fmul_rn, since a packed product is fused with
// this addition, which gives other codes near halves. `clamped`: values may lie beyond the codes' range.)
template <int TYPE>
__device__ __forceinline__ uint2 to_codes(float (&u)[8], bool clamped = false) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float* v = u + 4 * i;
    if constexpr (TYPE == SAGE_S8) {
      if (clamped) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = fminf(fmaxf(v[e], -127.f), 127.f);
      }
      constexpr float kUnit = 12582912.0f;
      add2(v[0], v[1], v[0], v[1], kUnit, kUnit);
      add2(v[2], v[3], v[2], v[3], kUnit, kUnit);
      w[i] = __byte_perm(__byte_perm(__float_as_uint(v[0]), __float_as_uint(v[1]), 0x0040),
                         __byte_perm(__float_as_uint(v[2]), __float_as_uint(v[3]), 0x0040), 0x5410);
    } else {
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[1]), "f"(v[0]));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[3]), "f"(v[2]));
      w[i] = lo | (uint32_t)hi << 16;
    }
  }
  return make_uint2(w[0], w[1]);
}
// Four codes as numbers.
template <int TYPE>
__device__ __forceinline__ void from_codes(uint32_t c, float& f0, float& f1, float& f2, float& f3) {
  if constexpr (TYPE == SAGE_S8) {
    const uint32_t u = c ^ 0x80808080u;  // code + 128, in the last byte of 2^23 + code + 128
    constexpr float kBias = 8388736.0f;
    f0 = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440));
    f1 = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441));
    f2 = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7442));
    f3 = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7443));
    add2(f0, f1, f0, f1, -kBias, -kBias);
    add2(f2, f3, f2, f3, -kBias, -kBias);
  } else {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo)), b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    f0 = a.x; f1 = a.y; f2 = b.x; f3 = b.y;
  }
}

}  // namespace sage
