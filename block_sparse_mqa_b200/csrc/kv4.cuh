// The 4-bit paged cache: format, addressing and element conversions shared by
// the kernels that write it (kv4_cache.cu) and read it (kv4_cache.cu,
// simt_kv4_decode.cu, tc_kv4_decode.cu).
//
// A row of `width` elements (a multiple of 32) is G = width / 32 groups, each
// one scale and 32 codes.  A page of `ps` rows holds, in this order,
//   codes   [G][ps][16 bytes]          group-major: the same group of
//                                       consecutive rows is contiguous
//   scales  [ceil(G / 4)][ps][4 bytes]  byte g % 4 of word g / 4 is group g's
// so that threads that own consecutive rows read consecutive 16-byte units and
// consecutive words.  Code n in 0..15 stands for (n - 8) * scale.  The scale
// byte is the upper half of an fp16 number without its sign (5 exponent and 3
// mantissa bits, subnormals included): fp16 bits = byte << 7.  A code has at
// most 4 significant bits (|n - 8| <= 8, so 3 for the codes that are written)
// and a scale 4, so every value is exact in bf16 (8 bits) and in fp32.
//
// In a group's four 32-bit words, word w holds elements 8w .. 8w + 7: element
// 8w + 2k in bits 4k .. 4k + 3 and element 8w + 2k + 1 in bits 16 + 4k ..
// 19 + 4k, so (word >> 4k) & 0x000f000f is a pair of neighbours in the two
// halves of a 32-bit register.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "hs_device.cuh"
#include "hs_internal.h"

namespace hs {
namespace kv4 {

constexpr float kMaxScale = 61440.f;     // 1.875 * 2^15, the largest finite scale
constexpr uint32_t kNanScale = 0xffu;    // a group that held NaN or infinity

__host__ __device__ __forceinline__ int groups(int width) { return width / 32; }
__host__ __device__ __forceinline__ int64_t page_bytes(int width, int ps) {
  const int g = groups(width);
  return (int64_t)ps * (16 * g + 4 * ((g + 3) / 4));
}
// Byte offsets inside a page.
__host__ __device__ __forceinline__ int64_t code_off(int g, int slot, int ps) {
  return ((int64_t)g * ps + slot) * 16;
}
__host__ __device__ __forceinline__ int64_t scale_off(int g, int slot, int ps, int ngroups) {
  return (int64_t)ngroups * ps * 16 + ((int64_t)(g >> 2) * ps + slot) * 4 + (g & 3);
}

// The cached positions a query attends: the first `nf` positions, then
// [w0, len).  Index x in [0, n) walks them in ascending order.
struct KeyList {
  int nf, w0, n;
  __device__ __forceinline__ int pos(int x) const { return x < nf ? x : w0 + (x - nf); }
};
// window 0: every position.
__device__ __forceinline__ KeyList key_list(int len, int window, int first) {
  KeyList k;
  k.nf = window > 0 ? min(first, len) : 0;
  k.w0 = window > 0 ? max(k.nf, len - window) : 0;
  k.n = k.nf + (len - k.w0);
  return k;
}

// Page of cached position pos, or -1 (recorded) where the table is too narrow
// or holds a page that does not exist.
__device__ __forceinline__ int page_of(const int32_t* __restrict__ row, int table_width,
                                       int num_pages, int pos, int ps_log2, int* status) {
  const int e = pos >> ps_log2;
  if (e >= table_width) {
    record_status(status, HS_ERR_INVALID_INDEX);
    return -1;
  }
  const int pg = __ldg(row + e);
  if (pg < 0 || pg >= num_pages) {
    record_status(status, HS_ERR_INVALID_INDEX);
    return -1;
  }
  return pg;
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

// Scale of a group with largest magnitude amax (finite): the smallest scale s
// with 7 s >= amax.  A truncated product with 1/7 is at most two steps low, and
// 7 s is exact (3 bits times 4), so the comparison decides.
__device__ __forceinline__ float group_scale(float amax) {
  const float r = amax * 0.142857134f;  // just under 1 / 7
  float s;
  if (r >= 6.103515625e-05f) {  // 2^-14: normal, 4 significant bits
    uint32_t u = __float_as_uint(r) & ~0xfffffu;
    u += 7.f * __uint_as_float(u) < amax ? 0x100000u : 0u;
    u += 7.f * __uint_as_float(u) < amax ? 0x100000u : 0u;
    s = __uint_as_float(u);
  } else {  // steps of 2^-17
    const float step = 7.62939453125e-06f;
    s = floorf(r * 131072.f) * step;
    s += 7.f * s < amax ? step : 0.f;
    s += 7.f * s < amax ? step : 0.f;
  }
  return fminf(s, kMaxScale);
}
__device__ __forceinline__ uint32_t scale_byte(float s) {
  return (uint32_t)__half_as_ushort(__float2half_rn(s)) >> 7;  // exact: 4 significant bits
}

// Low four bits: rint(x / s), half to even, as a two's complement number; |x| <=
// 7 s, inv = 1 / s rounded.  The product's rounding can miss a border between
// two codes, so the remainder, which is exact (a few bits beyond s), decides.
__device__ __forceinline__ uint32_t code_bits(float x, float s, float inv) {
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
  float y = fmaf(x, inv, kRound);
  const float d = fmaf(kRound - y, s, x), half = 0.5f * s;
  if (fabsf(d) > half || (fabsf(d) == half && (__float_as_uint(y) & 1u))) y += copysignf(1.f, d);
  return __float_as_uint(y) & 15u;
}
// Eight codes (rint + 8) in the order of a word.
__device__ __forceinline__ uint32_t code_word(const float (&x)[8], float s, float inv) {
  uint32_t w = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) w |= code_bits(x[e], s, inv) << (4 * (e >> 1) + 16 * (e & 1));
  return w ^ 0x88888888u;  // n mod 16 -> n + 8
}

}  // namespace kv4
}  // namespace hs
