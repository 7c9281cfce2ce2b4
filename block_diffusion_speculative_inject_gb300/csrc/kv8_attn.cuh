// Shared by the two attention kernels over the 8-bit cache: small device helpers and the merge of the
// partial results of split items.
#pragma once
#include "kv8_sched.cuh"
#include "tc_ptx.cuh"

namespace dflash {

constexpr int KV8_SMS = 152;                           // one CTA per SM
constexpr float LN2 = 0.693147180559945309f;

// a (low half) and b as f16, to nearest even
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t h) {
  float2 v;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}\n" : "=f"(v.x), "=f"(v.y) : "r"(h));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t mbar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(mbar) : "memory");
}
__device__ __forceinline__ uint32_t byte_mask(uint32_t high_bits) { return (high_bits >> 7) * 0xffu; }

// ---------------------------------------------------------------- merge of split items
// CTA (w - 1, y) looks at the descriptor of worker w: if w's first piece continues an item that worker w - 1
// began, it merges rows of that item, a warp each: the partial (m, l, O) of worker w - 1's
// last piece and of the first pieces of w, w + 1, .. up to the item's end. It is all latency, so nothing but the
// descriptor is waited for before the loads: lanes fetch the maxima and sums of 32 pieces at once
// while the first eight pieces' O (a lane owns four dims) are on their way.
template <typename T, int HD, int M>
__global__ void __launch_bounds__(128) k_kv8_combine(const Kv8AttnArgs a) {
  pdl_trigger();
  pdl_wait();
  const int w = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = 4 * lane;
  const int4 d0 = *(const int4 *)&a.desc[w];
  const int h = a.desc[w].h, n = d0.x, slot0 = d0.y, row0 = d0.z, rows = d0.w;
  if (n == 0) return;
  for (int row = 4 * blockIdx.y + warp; row < rows; row += 4 * gridDim.y) {
    auto slot_of = [&](int x) { return (size_t)(x == 0 ? slot0 : 2 * (w - 1 + x)) * M + row; };
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x0 = 0; x0 < n; x0 += 32) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (x0 + lane < n) ml = *(const float2 *)(a.part_ml + slot_of(x0 + lane) * 2);
      const int k = min(32, n - x0);
      float4 v[8];
#pragma unroll
      for (int z = 0; z < 8; ++z) v[z] = z < k && c < HD ? *(const float4 *)(a.part_o + slot_of(x0 + z) * HD + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float top = fmaxf(m, warp_max(ml.x)), ref = top == -INFINITY ? 0.f : top;
      const float wt = exp2f(ml.x - ref), back = exp2f(m - ref);
      m = top;
      l = l * back + warp_sum(ml.y * wt);
      o.x *= back, o.y *= back, o.z *= back, o.w *= back;
      for (int x = 0; x < k; x += 8) {
        if (x) {
#pragma unroll
          for (int z = 0; z < 8; ++z)
            v[z] = x + z < k && c < HD ? *(const float4 *)(a.part_o + slot_of(x0 + x + z) * HD + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int z = 0; z < 8; ++z) {
          const float e = __shfl_sync(0xffffffffu, wt, x + z);
          o.x = fmaf(v[z].x, e, o.x);
          o.y = fmaf(v[z].y, e, o.y);
          o.z = fmaf(v[z].z, e, o.z);
          o.w = fmaf(v[z].w, e, o.w);
        }
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int group = a.nq / a.nkv;
    const size_t at = (size_t)(row0 + row / group) * a.nq + h * group + row % group;
    T *out = (T *)a.out + at * HD + c;
    if (c < HD) {
      if constexpr (sizeof(T) == 2) {
        __nv_bfloat162 b[2] = {__floats2bfloat162_rn(o.x * inv, o.y * inv), __floats2bfloat162_rn(o.z * inv, o.w * inv)};
        *(uint2 *)out = *(const uint2 *)b;
      } else {
        *(float4 *)out = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      }
    }
    if (a.lse && lane == 0) a.lse[at] = l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * LN2;
  }
}

// Bounded wait for an mbarrier phase: false if the CTA was aborted or two seconds went by (which aborts it).
// Reading the timer in every round also keeps a waiting warp from polling away the issue slots of the
// working ones (129 against 140 us for 64 requests of one token with a bare polling loop).
__device__ __forceinline__ bool kv8_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
#pragma unroll 1
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (global_ns() - t0 > TC_WAIT_NS) *abort_flag = 1;
  }
}

// The kernel for many query rows (bf16): tiles of 128 rows, one worker per SM.
constexpr int KT_ROWS = 128;
cudaError_t launch_kv8_tiles(const Kv8AttnArgs &a, int hd, cudaStream_t s);
// The kernel for few rows over listed blocks (rows: 8 or 16 of a tile; wide: bf16).
cudaError_t launch_kv8_rows_listed(const Kv8AttnArgs &a, bool wide, int hd, int rows, cudaStream_t s);

}  // namespace dflash
