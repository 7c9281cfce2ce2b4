// Shared by the kernels of the caller-owned 8-bit paged cache (page planning, quantised append,
// attention): the page layout, e4m3 conversions and the argument checks of its C entry points.
#pragma once
#include "../../include/dflash.h"
#include "common.cuh"

namespace dflash {

constexpr int KV8_MAX_REQ = 4096;
constexpr int KV8_MIN_EXP = -64;          // smallest scale 2^-64: a page of zeros has one too

// Bytes of one (page, kv head) block of K or V; a pool of 2^24 pages passes 2^31 blocks of bytes.
__device__ __forceinline__ size_t kv8_block(int page, int h, int nkv, int hd) {
  return ((size_t)page * nkv + h) * (size_t)(KV_PAGE * hd);
}

// two e4m3 bytes (the low 16 bits) as f16 pair: exact, e4m3 is a subset of f16
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t b) {
  uint32_t r;
  asm("{\n .reg .b16 t;\n cvt.u16.u32 t, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}\n" : "=r"(r) : "r"(b));
  return r;
}
// four of them as two pairs
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t b, uint32_t &lo, uint32_t &hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(lo), "=r"(hi) : "r"(b));
}
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t b) {
  const uint32_t h = e4m3x2_to_f16x2(b);
  float2 v;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}\n"
      : "=f"(v.x), "=f"(v.y) : "r"(h));
  return v;
}
// two fp32 values as e4m3 bytes (a in the low one), to nearest even, finite values saturating;
// NaN stays NaN (0x7f)
__device__ __forceinline__ uint32_t f32_to_e4m3x2(float a, float b) {
  uint32_t r;
  asm("{\n .reg .b16 t;\n cvt.rn.satfinite.e4m3x2.f32 t, %2, %1;\n cvt.u32.u16 %0, t;\n}\n" : "=r"(r) : "f"(a), "f"(b));
  return r;
}

// the same from f16 pairs, and to e5m2
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t h) {
  uint32_t r;
  asm("{\n .reg .b16 t;\n cvt.rn.satfinite.e4m3x2.f16x2 t, %1;\n cvt.u32.u16 %0, t;\n}\n" : "=r"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_to_e5m2x2(uint32_t h) {
  uint32_t r;
  asm("{\n .reg .b16 t;\n cvt.rn.satfinite.e5m2x2.f16x2 t, %1;\n cvt.u32.u16 %0, t;\n}\n" : "=r"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// d += a b: m16n8k16 of f16 with fp32 sums
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// bytes 0x7f / 0xff (e4m3 NaN) of a word, as 0x80 in each
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// smallest e >= KV8_MIN_EXP with amax <= 448 * 2^e = 1.75 * 2^(e + 8), from amax's own bits
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, KV8_MIN_EXP);
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// four e4m3 bytes times a factor, rounded again
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  const float2 a = e4m3x2_to_f32(w), b = e4m3x2_to_f32(w >> 16);
  return f32_to_e4m3x2(a.x * f, a.y * f) | f32_to_e4m3x2(b.x * f, b.y * f) << 16;
}

inline bool aligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline int dtype_bytes(int dtype) { return dtype == DFLASH_BF16 ? 2 : 4; }

inline bool kv8_cache_ok(const dflash_kv8_cache *c, bool pointers = true) {
  if (!c || c->n_pages < 1 || c->n_pages > (1 << 24) || c->n_kv_heads < 1 || c->n_kv_heads > 128 ||
      (c->head_dim != 64 && c->head_dim != 128))
    return false;
  return !pointers || (c->k_pages && c->v_pages && c->k_scale && c->v_scale && aligned(c->k_pages, 16) &&
                       aligned(c->v_pages, 16) && aligned(c->k_scale, 4) && aligned(c->v_scale, 4));
}

}  // namespace dflash
