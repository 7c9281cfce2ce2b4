// Per-head RMSNorm with rotary positions in one pass (dflash_qk_norm_rope) and its gradient.
//
// A head x [hd] at position p becomes y = R(p) n, n = x r w, r = 1 / sqrt(mean(x^2) + eps). Its gradient from
// that of y: n' = R^T y', g = n' w, x' = r (g - x r^2 mean(g x)), w' = sum of n' x r over rows and heads.
//
// Every element is read and written once, which bounds both. A head belongs to G lanes of a warp (the smallest
// power of two that its chunks need, at most 32), which hold it in registers between the sum of squares and the
// rotation; a chunk is V dims and, in the half layout, their partners, or the V dims that follow.
//
// 32768 rows of 48 x 128 bf16 take 128 us (805 MB, 6.3 TB/s), the gradient of 16384 rows of 40 x 128 98 us with the sum over
// its CTAs (503 MB, 5.1 TB/s; latencies at two CTAs per SM). What paid, in the forward pass: sines in registers for all heads
// of a row (219 us when every head read them from shared memory, four lanes to a bank), copies ahead through shared memory,
// paired arithmetic and packed conversions (248 without these two), as many CTAs as are resident (146 with a third more), and
// no more copies ahead than two (142 with one, 138 with four: the shared memory is the first-level cache's). The gradient
// keeps both weights' sums, 128 registers for two CTAs per SM, with 36 bytes spilled (110 us at 154 registers and one CTA; 105
// with three copies ahead, 101 with two, 98 with half as many groups to a row).
// 16384 rows of 40 x 128 take 58 us in bf16, 114 in fp32 (its gradient 161). Where the rotated dims, a stride or an address do not
// keep a 16-byte boundary, every access is of two elements or of one, in instances sized for heads of 256: with 20
// dims of 128 turned 174 us, and 255 for the gradient.
#include <cmath>

#include "rope.cuh"

namespace dflash {

constexpr int QN_THREADS = 256;
constexpr int QN_CTAS = 152 * 3, QN_CTAS_GRAD = 152 * 2;      // most CTAs: as many as are resident
constexpr int QN_DEPTH = 3, QN_DEPTH_GRAD = 3;        // heads of a lane that are held or on their way

struct NormArgs {
  uint64_t turn[128];
  float magnitude, eps;
  int rot, inter, rows, nq, nk, hd;
  int chunks, lanes;                                  // chunks of a head, lanes of a head
  int step;                                           // groups of lanes that share a row
  unsigned by_pairs;                                  // 2^20 / pairs, rounded up
  const int32_t *positions;
  const void *qw, *kw;
  const void *q, *k, *gq, *gk;                        // inputs; gradients of the outputs (backward)
  void *qo, *ko;                                      // outputs, or gradients of the inputs
  int64_t qs, ks, gqs, gks, qos, kos;
  float *part;                                        // [CTAs][2][hd] partial sums of the weights' gradients
};

// Two fp32 at a time.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n fma.rn.f32x2 x, x, y, z;\n"
      " mov.b64 {%0, %1}, x;\n}\n" : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Chunk c of a head: dims lo .. lo + V - 1 and hi .. hi + V - 1 (none from hd on), turned if c is below the rotated ones.
template <int V>
struct Chunk {
  int lo, hi;
  bool turns;
  Chunk() = default;
  __device__ __forceinline__ Chunk(const NormArgs &a, int c) {
    const int rot_chunks = a.rot / (2 * V);
    turns = c < rot_chunks;
    lo = turns && !a.inter ? c * V : c * 2 * V;
    hi = turns && !a.inter ? lo + a.rot / 2 : lo + V;
    if (c >= a.chunks) lo = hi = a.hd;
  }
};

// 2 V stored values of a chunk, V of each half, as V pairs: neighbours of a half (V = 1: the two).
template <typename T, int V>
__device__ __forceinline__ void unpack(const Vec<T, V> &lo, const Vec<T, V> &hi, float2 (&x)[V]) {
  if constexpr (V == 1) {
    x[0] = make_float2(to_f(lo.v[0]), to_f(hi.v[0]));
  } else {
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      if constexpr (sizeof(T) == 2) {
        const uint32_t a = ((const uint32_t *)&lo)[j], b = ((const uint32_t *)&hi)[j];
        x[j] = make_float2(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
        x[V / 2 + j] = make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
      } else {
        x[j] = make_float2(to_f(lo.v[2 * j]), to_f(lo.v[2 * j + 1]));
        x[V / 2 + j] = make_float2(to_f(hi.v[2 * j]), to_f(hi.v[2 * j + 1]));
      }
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void pack(const float2 *x, Vec<T, V> &v) {
#pragma unroll
  for (int j = 0; j < V / 2; ++j) {
    if constexpr (sizeof(T) == 2) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[j].x, x[j].y);
      ((uint32_t *)&v)[j] = *(const uint32_t *)&b;
    } else {
      v.v[2 * j] = from_f<T>(x[j].x);
      v.v[2 * j + 1] = from_f<T>(x[j].y);
    }
  }
}

// A lane's part of a head as stored: R chunks, zeros past the head's end. FULL: no lane has a place past it.
template <typename T, int V, int R, bool FULL>
struct Part {
  typedef Vec<T, V> VT;
  VT v[2 * R];
  static __device__ __forceinline__ int dim(const Chunk<V> (&c)[R], int i) { return i & 1 ? c[i / 2].hi : c[i / 2].lo; }
  __device__ __forceinline__ void zero(int i) {
#pragma unroll
    for (int j = 0; j < V; ++j) v[i].v[j] = from_f<T>(0.f);
  }
  __device__ __forceinline__ void load(const T *p, const Chunk<V> (&c)[R], int hd) {
#pragma unroll
    for (int i = 0; i < 2 * R; ++i) {
      if (FULL || dim(c, i) < hd) v[i] = *(const VT *)(p + dim(c, i));
      else zero(i);
    }
  }
  __device__ __forceinline__ void chunk(int i, float2 (&x)[V]) const { unpack<T, V>(v[2 * i], v[2 * i + 1], x); }
};
template <typename T, int V, bool FULL>
__device__ __forceinline__ void store_chunk(T *p, const Chunk<V> &c, int hd, const float2 (&x)[V]) {
  Vec<T, V> lo, hi;
  if constexpr (V == 1) {
    lo.v[0] = from_f<T>(x[0].x);
    hi.v[0] = from_f<T>(x[0].y);
  } else {
    pack<T, V>(x, lo);
    pack<T, V>(x + V / 2, hi);
  }
  if (FULL || c.lo < hd) *(Vec<T, V> *)(p + c.lo) = lo;
  if (FULL || c.hi < hd) *(Vec<T, V> *)(p + c.hi) = hi;
}

// Copies ahead: every thread's own ring of DEPTH parts (of OPS operands) in shared memory, which no other reads.
template <typename T, int V, int R, int OPS, int DEPTH, bool FULL>
struct Ring {
  typedef Vec<T, V> VT;
  typedef Part<T, V, R, FULL> P;
  static constexpr size_t BYTES = sizeof(VT) * 2 * R * OPS * DEPTH * QN_THREADS;
  VT *mine;
  __device__ __forceinline__ Ring(void *base) : mine((VT *)base + threadIdx.x) {}
  __device__ __forceinline__ VT *at(int slot, int op, int i) const { return mine + ((slot * OPS + op) * 2 * R + i) * QN_THREADS; }
  __device__ __forceinline__ void fetch(int slot, int op, const T *p, const Chunk<V> (&c)[R], int hd) const {
#pragma unroll
    for (int i = 0; i < 2 * R; ++i) {
      const int d = P::dim(c, i);
      if (!FULL && d >= hd) continue;
      VT *to = at(slot, op, i);
      if constexpr (sizeof(VT) == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(p + d) : "memory");
      else if constexpr (sizeof(VT) >= 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(p + d), "n"(sizeof(VT)) : "memory");
      else
        *to = *(const VT *)(p + d);
    }
  }
  __device__ __forceinline__ void commit() const { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // the oldest of DEPTH - 1 groups has arrived
  __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 2) : "memory"); }
  __device__ __forceinline__ void take(int slot, int op, P &x, const Chunk<V> (&c)[R], int hd) const {
#pragma unroll
    for (int i = 0; i < 2 * R; ++i) {
      if (FULL || P::dim(c, i) < hd) x.v[i] = *at(slot, op, i);
      else x.zero(i);
    }
  }
};

// the chunk's 2 V values turned in place by its pairs' cosines and sines
template <int V>
__device__ __forceinline__ void turn_chunk(bool inter, bool turns, const float *cos, const float *sin, float2 (&x)[V]) {
  if (!turns) return;
  if (inter || V == 1) {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = turned(x[j].x, x[j].y, make_float2(cos[j], sin[j]));
  } else {
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      const float2 c = make_float2(cos[2 * j], cos[2 * j + 1]), s = make_float2(sin[2 * j], sin[2 * j + 1]);
      const float2 l = x[j], h = x[V / 2 + j], m = mul2(h, s);
      x[j] = make_float2(fmaf(l.x, c.x, -m.x), fmaf(l.y, c.y, -m.y));
      x[V / 2 + j] = fma2(h, c, mul2(l, s));
    }
  }
}

__device__ __forceinline__ float head_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// 1 / sqrt(x): the approximation and a step of Newton's method
__device__ __forceinline__ float inv_sqrt(float x) {
  const float r = rsqrtf(x);
  return fmaf(0.5f * r, fmaf(-x * r, r, 1.f), r);
}

// Forward and gradient. A CTA takes a share of the rows, a tile at a time. A group of lanes stays with a row of the tile
// for all of its heads there (every a.step-th of q's and k's), so that sines and cosines are in registers; those of the
// next tile are made while this one is worked on. Heads to come are copied ahead.
template <typename T, int V, int R, bool FULL, bool GRAD>
__global__ void __launch_bounds__(QN_THREADS, GRAD ? 2 : 3) k_qk_norm(const __grid_constant__ NormArgs a) {
  constexpr int OPS = GRAD ? 2 : 1, DEPTH = GRAD ? QN_DEPTH_GRAD : QN_DEPTH;
  typedef Ring<T, V, R, OPS, DEPTH, FULL> Copies;
  extern __shared__ __align__(16) uint8_t qn_smem[];
  __shared__ uint64_t s_turn[128];
  const Copies ring(qn_smem);
  float *cs = (float *)(qn_smem + Copies::BYTES);      // [2][cosines, sines][tile][pairs]
  pdl_trigger();
  const int pairs = a.rot / 2, heads = a.nq + a.nk;
  for (int i = threadIdx.x; i < pairs; i += QN_THREADS) s_turn[i] = a.turn[i];
  // rows from `first` on, counted from there (that of many rows has many CTAs: no sum below passes 2^31)
  const int first = (int)((int64_t)a.rows * blockIdx.x / gridDim.x);
  const int end = (int)((int64_t)a.rows * (blockIdx.x + 1) / gridDim.x) - first;
  const int group = threadIdx.x / a.lanes, lane = threadIdx.x % a.lanes;
  const int tile = QN_THREADS / a.lanes / a.step;
  const int my_row = group / a.step, my_head = group % a.step, per_tile = (heads + a.step - 1) / a.step;
  Chunk<V> c[R];
#pragma unroll
  for (int i = 0; i < R; ++i) c[i] = Chunk<V>(a, lane + i * a.lanes);
  pdl_wait();
  // the copies: DEPTH - 1 steps ahead
  int f_row = my_row, f_head = my_head, f_slot = 0;
  auto fetch = [&]() {
    if (f_row < end && f_head < heads) {
      const bool isk = f_head >= a.nq;
      const int64_t from = (int64_t)(isk ? f_head - a.nq : f_head) * a.hd;
      ring.fetch(f_slot, 0, (const T *)(isk ? a.k : a.q) + (first + f_row) * (isk ? a.ks : a.qs) + from, c, a.hd);
      if constexpr (GRAD) ring.fetch(f_slot, 1, (const T *)(isk ? a.gk : a.gq) + (first + f_row) * (isk ? a.gks : a.gqs) + from, c, a.hd);
    }
    ring.commit();
    f_slot = f_slot + 1 == DEPTH ? 0 : f_slot + 1;
    f_head += a.step;
    if (f_head >= per_tile * a.step) {
      f_head = my_head;
      f_row += tile;
    }
  };
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) fetch();
  __syncthreads();                                    // s_turn is there
  auto angles = [&](int row0, float *to) {
    const int n = min(tile, end - row0) * pairs;
    for (int i = threadIdx.x; i < n; i += QN_THREADS) {
      const int r = (int)(i * a.by_pairs >> 20);       // i / pairs: i is below 2048 where pairs is above 1
      const float2 t = phase_cs((uint64_t)(int64_t)a.positions[first + row0 + r] * s_turn[i - r * pairs]);
      to[i] = t.x * a.magnitude;
      to[tile * pairs + i] = t.y * (GRAD ? -a.magnitude : a.magnitude);        // (the gradient turns back)
    }
  };
  Part<T, V, R, FULL> qw, kw;
  qw.load((const T *)a.qw, c, a.hd);
  if (a.nk) kw.load((const T *)a.kw, c, a.hd);
  else kw = qw;
  const float inv_hd = 1.f / (float)a.hd;
  float2 wsum[2][GRAD ? R : 1][V];
  if constexpr (GRAD) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) wsum[k][i][j] = make_float2(0.f, 0.f);
  }
  if (end > 0) angles(0, cs);
  int slot = 0;
  for (int row0 = 0, buf = 0; row0 < end; row0 += tile, buf ^= 1) {
    __syncthreads();                                  // this tile's angles are there, the last one's are done with
    if (row0 + tile < end) angles(row0 + tile, cs + 2 * (buf ^ 1) * tile * pairs);
    const int row = row0 + my_row;
    float cosine[R][V], sine[R][V];
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (c[i].turns) {
        const float *from = cs + (2 * buf * tile + my_row) * pairs + (a.inter ? c[i].lo / 2 : c[i].lo);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          cosine[i][j] = from[j];
          sine[i][j] = from[tile * pairs + j];
        }
      }
    for (int h = my_head, n = 0; n < per_tile; ++n, h += a.step) {     // (all lanes of a warp stay for the sums)
      ring.wait();
      Part<T, V, R, FULL> x, g;
      ring.take(slot, 0, x, c, a.hd);
      if constexpr (GRAD) ring.take(slot, 1, g, c, a.hd);
      fetch();
      slot = slot + 1 == DEPTH ? 0 : slot + 1;
      const bool isk = h >= a.nq;
      float2 u[R][V], z[R][V], w[R][V];
      float2 ss = make_float2(0.f, 0.f), dot = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        x.chunk(i, u[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) ss = fma2(u[i][j], u[i][j], ss);
        Part<T, V, 1, FULL> both_w;
        both_w.v[0] = isk ? kw.v[2 * i] : qw.v[2 * i];
        both_w.v[1] = isk ? kw.v[2 * i + 1] : qw.v[2 * i + 1];
        both_w.chunk(0, w[i]);
        if constexpr (GRAD) {
          g.chunk(i, z[i]);
          turn_chunk<V>(a.inter, c[i].turns, cosine[i], sine[i], z[i]);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            w[i][j] = mul2(z[i][j], w[i][j]);
            dot = fma2(w[i][j], u[i][j], dot);
          }
        }
      }
      const float inv = inv_sqrt(fmaf(head_sum(ss.x + ss.y, a.lanes), inv_hd, a.eps));
      float m = 0.f;
      if constexpr (GRAD) m = head_sum(dot.x + dot.y, a.lanes) * inv * inv_hd;       // r mean(g x)
      if (row >= end || h >= heads) continue;
      const int64_t to = (int64_t)(isk ? h - a.nq : h) * a.hd;
      T *dst = (T *)(isk ? a.ko : a.qo) + (first + row) * (isk ? a.kos : a.qos) + to;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float2 y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          u[i][j] = mul2(u[i][j], both(inv));
          if constexpr (GRAD) y[j] = mul2(fma2(u[i][j], both(-m), w[i][j]), both(inv));
          else y[j] = mul2(u[i][j], w[i][j]);
        }
        if constexpr (!GRAD) turn_chunk<V>(a.inter, c[i].turns, cosine[i], sine[i], y);
        store_chunk<T, V, FULL>(dst, c[i], a.hd, y);
      }
      if constexpr (GRAD) {
        if (isk) {
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) wsum[1][i][j] = fma2(z[i][j], u[i][j], wsum[1][i][j]);
        } else {
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) wsum[0][i][j] = fma2(z[i][j], u[i][j], wsum[0][i][j]);
        }
      }
    }
  }
  if constexpr (GRAD) {
    // the weights' gradients over the CTA, in a fixed order
    __syncthreads();
    float *sums = (float *)qn_smem;                   // [warps][2][hd]
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float2 v = wsum[k][i][j];
          for (int o = a.lanes; o < 32; o <<= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
          }
          // (V = 1: the two halves; else neighbours, the first half's and then the other's)
          const int d0 = V == 1 ? c[i].lo : j < V / 2 ? c[i].lo + 2 * j : c[i].hi + 2 * j - V, d1 = V == 1 ? c[i].hi : d0 + 1;
          if ((threadIdx.x & 31) < a.lanes) {
            if (d0 < a.hd) sums[(2 * warp + k) * a.hd + d0] = v.x;
            if (d1 < a.hd) sums[(2 * warp + k) * a.hd + d1] = v.y;
          }
        }
    __syncthreads();
    for (int d = threadIdx.x; d < 2 * a.hd; d += QN_THREADS) {
      float v = 0.f;
      for (int x = 0; x < QN_THREADS / 32; ++x) v += sums[2 * x * a.hd + d];
      a.part[(size_t)blockIdx.x * 2 * a.hd + d] = v;
    }
  }
}

// dweight[d] = the sum of the CTAs' partial sums: 32 dims of a CTA, 32 threads each
__global__ void __launch_bounds__(1024) k_qk_norm_weights(int ctas, int hd, const float *part, float *dqw, float *dkw) {
  __shared__ float s[32][33];
  pdl_trigger();
  pdl_wait();
  const int k = blockIdx.y, d = blockIdx.x * 32 + threadIdx.x, y = threadIdx.y;
  float v = 0.f;
  if (d < hd)
    for (int i = y; i < ctas; i += 32) v += part[((size_t)i * 2 + k) * hd + d];
  s[y][threadIdx.x] = v;
  __syncthreads();
  v = warp_sum(s[threadIdx.x][y]);
  const int dim = blockIdx.x * 32 + y;
  if (threadIdx.x == 0 && dim < hd) (k ? dkw : dqw)[dim] = v;
}

template <typename T, int V, int R, bool FULL, bool GRAD>
cudaError_t launch_norm(const NormArgs &a, int ctas, cudaStream_t s) {
  const int tile = QN_THREADS / a.lanes / a.step;
  size_t sm = Ring<T, V, R, GRAD ? 2 : 1, GRAD ? QN_DEPTH_GRAD : QN_DEPTH, FULL>::BYTES + 4ull * tile * (a.rot / 2) * sizeof(float);
  const size_t sums = (size_t)QN_THREADS / 32 * 2 * a.hd * sizeof(float);
  sm = GRAD && sm < sums ? sums : sm;
  const cudaError_t e = cudaFuncSetAttribute(k_qk_norm<T, V, R, FULL, GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, 112 << 10);
  return e != cudaSuccess ? e : launch_pdl(k_qk_norm<T, V, R, FULL, GRAD>, dim3(ctas), dim3(QN_THREADS), sm, s, a);
}

// width: elements of an access. Returns the CTAs in *ctas.
template <typename T, bool GRAD>
cudaError_t launch_norm(NormArgs &a, int width, int *ctas, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  a.chunks = (a.hd + 2 * width - 1) / (2 * width);
  a.lanes = 1;
  while (a.lanes < a.chunks && a.lanes < 32) a.lanes *= 2;
  const int per = QN_THREADS / a.lanes, heads = a.nq + a.nk;
  a.by_pairs = ((1u << 20) + a.rot / 2 - 1) / (a.rot / 2);
  constexpr int most = GRAD ? QN_CTAS_GRAD : QN_CTAS;
  // Groups of lanes that share a row: 8, for more than one row's angles at a time, 4 in the gradient (forward and gradient
  // above with 4 129 and 98 us, with 8 128 and 101); all of them where that leaves too few CTAs, and no more than the
  // power of two that holds the heads.
  a.step = 1;
  while (a.step < per && a.step < heads && (a.step < (GRAD ? 4 : 8) || (int64_t)a.rows * a.step < (int64_t)most * per)) a.step *= 2;
  const int tile = per / a.step;
  const int64_t tiles = ((int64_t)a.rows + tile - 1) / tile;
  *ctas = tiles < most ? (int)tiles : most;
  if (width == W && a.lanes == a.chunks && a.hd % (2 * W) == 0) return launch_norm<T, W, 1, true, GRAD>(a, *ctas, s);
  if (width == W) return launch_norm<T, W, 1, false, GRAD>(a, *ctas, s);
  return width == 2 ? launch_norm<T, 2, 2, false, GRAD>(a, *ctas, s) : launch_norm<T, 1, 4, false, GRAD>(a, *ctas, s);
}

}  // namespace dflash

using namespace dflash;

namespace {
bool norm_ok(const dflash_rope *rope, int rows, int nq, int nk, int hd, int dtype, float eps) {
  return rope && rows >= 0 && nq >= 1 && nk >= 0 && nq <= (1 << 20) && nk <= (1 << 20) && nq + nk <= (1 << 20) &&
         (dtype == DFLASH_F32 || dtype == DFLASH_BF16) && rope->rot_dim >= 2 && rope->rot_dim % 2 == 0 &&
         rope->rot_dim <= hd && hd <= 256 && !(rope->interleaved & ~1) && eps > 0.f && std::isfinite(eps);
}
NormArgs norm_args(const dflash_rope *rope, int rows, int nq, int nk, int hd, float eps, const int32_t *positions) {
  NormArgs a{};
  for (int i = 0; i < 128; ++i) a.turn[i] = rope->turn[i];
  a.magnitude = rope->magnitude;
  a.rot = rope->rot_dim;
  a.inter = rope->interleaved;
  a.eps = eps;
  a.rows = rows;
  a.nq = nq;
  a.nk = nk;
  a.hd = hd;
  a.positions = positions;
  return a;
}
// Elements that every access may take: 16 bytes where all rows, heads and chunks keep that boundary, else two, else one.
struct Fit {
  const void *p;
  int64_t stride;
};
int access_width(const NormArgs &a, unsigned es, const Fit *f, int n) {
  for (int w : {16 / (int)es, 2}) {
    bool ok = a.hd % w == 0 && a.rot % (2 * w) == 0;
    for (int i = 0; i < n; ++i) ok = ok && aligned(f[i].p, w * es) && f[i].stride % w == 0;
    if (ok) return w;
  }
  return 1;
}
}  // namespace

extern "C" dflash_status dflash_qk_norm_rope(void *stream, const dflash_rope *rope, int32_t rows, int32_t n_q_heads,
                                             int32_t n_k_heads, int32_t head_dim, dflash_dtype dtype,
                                             const int32_t *positions, float eps, const void *q_weight,
                                             const void *k_weight, const void *q, int64_t q_stride, const void *k,
                                             int64_t k_stride, void *q_out, int64_t q_out_stride, void *k_out,
                                             int64_t k_out_stride) {
  if (!norm_ok(rope, rows, n_q_heads, n_k_heads, head_dim, dtype, eps)) return DFLASH_ERR_INVALID_ARG;
  const int nk = k ? n_k_heads : 0;
  const int64_t qw = (int64_t)n_q_heads * head_dim, kw = (int64_t)nk * head_dim;
  if (q_stride < qw || q_out_stride < qw || (nk && (k_stride < kw || k_out_stride < kw))) return DFLASH_ERR_INVALID_ARG;
  if (rows == 0) return DFLASH_OK;
  const unsigned es = dtype_bytes(dtype);
  if (!positions || !aligned(positions, 4)) return DFLASH_ERR_INVALID_ARG;
  const Fit f[] = {{q, q_stride}, {q_out, q_out_stride}, {q_weight, 0}, {k, k_stride}, {k_out, k_out_stride}, {k_weight, 0}};
  const int n = nk ? 6 : 3;
  for (int i = 0; i < n; ++i)
    if (!f[i].p || !aligned(f[i].p, es)) return DFLASH_ERR_INVALID_ARG;
  if ((q == q_out && q_stride != q_out_stride) || (nk && k == k_out && k_stride != k_out_stride) ||
      (nk && (q_out == k || q_out == k_out || k_out == q)))
    return DFLASH_ERR_INVALID_ARG;
  NormArgs a = norm_args(rope, rows, n_q_heads, nk, head_dim, eps, positions);
  a.qw = q_weight, a.kw = k_weight;
  a.q = q, a.k = k, a.qo = q_out, a.ko = k_out;
  a.qs = q_stride, a.ks = k_stride, a.qos = q_out_stride, a.kos = k_out_stride;
  const int w = access_width(a, es, f, n);
  const cudaStream_t s = (cudaStream_t)stream;
  int ctas;
  const cudaError_t e = dtype == DFLASH_BF16 ? launch_norm<bf16, false>(a, w, &ctas, s) : launch_norm<float, false>(a, w, &ctas, s);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

extern "C" int64_t dflash_qk_norm_rope_workspace(void) { return (int64_t)QN_CTAS_GRAD * 2 * 256 * sizeof(float); }

extern "C" dflash_status dflash_qk_norm_rope_backward(void *stream, const dflash_rope *rope,
                                                      const dflash_qk_norm_rope_grad *x) {
  if (!x || !norm_ok(rope, x->rows, x->n_q_heads, x->n_k_heads, x->head_dim, x->dtype, x->eps)) return DFLASH_ERR_INVALID_ARG;
  // (with no rows k may be an empty tensor's null pointer)
  const int nk = x->k || (!x->rows && x->dk_weight) ? x->n_k_heads : 0, hd = x->head_dim;
  const int64_t qw = (int64_t)x->n_q_heads * hd, kw = (int64_t)nk * hd;
  if (x->q_stride < qw || x->grad_q_out_stride < qw || x->dq_stride < qw ||
      (nk && (x->k_stride < kw || x->grad_k_out_stride < kw || x->dk_stride < kw)))
    return DFLASH_ERR_INVALID_ARG;
  if (!x->dq_weight || !aligned(x->dq_weight, 4) || (nk && (!x->dk_weight || !aligned(x->dk_weight, 4))) ||
      !x->workspace || !aligned(x->workspace, 256) || x->workspace_bytes < dflash_qk_norm_rope_workspace())
    return DFLASH_ERR_INVALID_ARG;
  const unsigned es = dtype_bytes(x->dtype);
  const Fit f[] = {{x->q, x->q_stride}, {x->grad_q_out, x->grad_q_out_stride}, {x->dq, x->dq_stride}, {x->q_weight, 0},
                   {x->k, x->k_stride}, {x->grad_k_out, x->grad_k_out_stride}, {x->dk, x->dk_stride}, {x->k_weight, 0}};
  const int n = nk ? 8 : 4;
  if (x->rows) {
    if (!x->positions || !aligned(x->positions, 4)) return DFLASH_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
      if (!f[i].p || !aligned(f[i].p, es)) return DFLASH_ERR_INVALID_ARG;
    if (x->dq == x->q ||
        (nk && (x->dk == x->k || x->dk == x->q || x->dk == x->grad_q_out || x->dq == x->k || x->dq == x->grad_k_out || x->dq == x->dk)) ||
        (x->dq == x->grad_q_out && x->dq_stride != x->grad_q_out_stride) ||
        (nk && x->dk == x->grad_k_out && x->dk_stride != x->grad_k_out_stride))
      return DFLASH_ERR_INVALID_ARG;
  }
  NormArgs a = norm_args(rope, x->rows, x->n_q_heads, nk, hd, x->eps, x->positions);
  a.qw = x->q_weight, a.kw = x->k_weight;
  a.q = x->q, a.k = x->k, a.gq = x->grad_q_out, a.gk = x->grad_k_out, a.qo = x->dq, a.ko = x->dk;
  a.qs = x->q_stride, a.ks = x->k_stride, a.gqs = x->grad_q_out_stride, a.gks = x->grad_k_out_stride;
  a.qos = x->dq_stride, a.kos = x->dk_stride;
  a.part = (float *)x->workspace;
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  int ctas = 0;
  if (x->rows) {
    const int w = access_width(a, es, f, n);
    e = x->dtype == DFLASH_BF16 ? launch_norm<bf16, true>(a, w, &ctas, s) : launch_norm<float, true>(a, w, &ctas, s);
  }
  if (e == cudaSuccess)
    e = launch_pdl(k_qk_norm_weights, dim3((hd + 31) / 32, nk ? 2 : 1), dim3(32, 32), 0, s, ctas, hd,
                   (const float *)a.part, x->dq_weight, x->dk_weight);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
