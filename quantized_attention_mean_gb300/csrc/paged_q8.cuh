// View of a paged key-value cache held in 8 bits with a scale for each block of tokens and head, and the codes' arithmetic.
//
// A page holds page_size slots of every key/value head; `block` slots that follow one another (block divides page_size)
// share a scale. The value of a code is code * scale, whichever type the code is of: int8, or E4M3.
#pragma once
#include <cuda_fp8.h>

#include "paged.cuh"

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
// Code of a value in units of the scale: round to nearest even.
template <int TYPE>
__device__ __forceinline__ uint8_t to_code(float u) {
  if (TYPE == SAGE_S8) return (uint8_t)(int8_t)max(-127, min(127, __float2int_rn(u)));
  return (uint8_t)__nv_cvt_float_to_fp8(u, __NV_SATFINITE, __NV_E4M3);
}
template <int TYPE>
__device__ __forceinline__ float from_code(uint8_t c) {
  if (TYPE == SAGE_S8) return (float)(int8_t)c;
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3)));
}

}  // namespace sage
