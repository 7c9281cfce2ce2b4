// Per-head RMSNorm with rotary positions in one pass (dflash_qk_norm_rope) and its gradient.
//
// A head x [hd] at position p becomes y = R(p) n, n = x r w, r = 1 / sqrt(mean(x^2) + eps). Its gradient from
// that of y: n' = R^T y', g = n' w, x' = r (g - x r^2 mean(g x)), w' = sum of n' x r over rows and heads.
//
// Every element is read and written once, which bounds both. A head belongs to G lanes of a warp (the smallest
// power of two that its chunks need, at most 32), which hold it in registers between the sum of squares and the
// rotation; a chunk is V dims and, in the half layout, their partners, or the V dims that follow. Sines and
// cosines of a row are made once, in shared memory, for all of its heads.
#include <cmath>

#include "rope.cuh"

namespace dflash {

constexpr int QN_THREADS = 256;
constexpr int QN_CTAS = 152 * 4;                      // CTAs of the gradient, one partial sum of the weights' each

struct NormArgs {
  uint64_t turn[128];
  float magnitude, eps;
  int rot, inter, rows, nq, nk, hd;
  int chunks, lanes, tile;                            // chunks of a head, lanes of a head, rows of a CTA's tile
  const int32_t *positions;
  const void *qw, *kw;
  const void *q, *k, *gq, *gk;                        // inputs; gradients of the outputs (backward)
  void *qo, *ko;                                      // outputs, or gradients of the inputs
  int64_t qs, ks, gqs, gks, qos, kos;
  float *part;                                        // [CTAs][2][hd] partial sums of the weights' gradients
};

// Chunk c of a head: dims lo .. lo + V - 1 and hi .. hi + V - 1 (none where hi >= hd), turned if c is below the rotated ones.
template <int V>
struct Chunk {
  int lo, hi;
  bool turns;
  __device__ __forceinline__ Chunk(const NormArgs &a, int c) {
    const int rot_chunks = a.rot / (2 * V);
    turns = c < rot_chunks;
    lo = turns && !a.inter ? c * V : c * 2 * V;
    hi = turns && !a.inter ? lo + a.rot / 2 : lo + V;
    if (c >= a.chunks) lo = hi = a.hd;
  }
};

template <typename T, int V>
__device__ __forceinline__ void load_dims(const T *p, int d, int hd, float *x) {
  if (d < hd) {
    const Vec<T, V> v = *(const Vec<T, V> *)(p + d);
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = to_f(v.v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = 0.f;
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_dims(T *p, int d, int hd, const float *x) {
  if (d >= hd) return;
  Vec<T, V> v;
#pragma unroll
  for (int j = 0; j < V; ++j) v.v[j] = from_f<T>(x[j]);
  *(Vec<T, V> *)(p + d) = v;
}

// the chunk's 2 V values turned in place by cs (its row's pairs)
template <int V>
__device__ __forceinline__ void turn_chunk(const NormArgs &a, const Chunk<V> &c, const float2 *cs, float *x) {
  if (!c.turns) return;
  if (a.inter) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float2 z = turned(x[2 * j], x[2 * j + 1], cs[c.lo / 2 + j]);
      x[2 * j] = z.x;
      x[2 * j + 1] = z.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float2 z = turned(x[j], x[V + j], cs[c.lo + j]);
      x[j] = z.x;
      x[V + j] = z.y;
    }
  }
}

__device__ __forceinline__ float head_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// cos and sin of the tile's rows; sign -1: the transposed rotation
__device__ __forceinline__ void tile_angles(const NormArgs &a, int row0, int rows, float sign, float2 *cs) {
  const int pairs = a.rot / 2;
  for (int i = threadIdx.x; i < rows * pairs; i += QN_THREADS) {
    const int r = i / pairs, p = i - r * pairs;
    float2 t = phase_cs((uint64_t)(int64_t)a.positions[row0 + r] * a.turn[p]);
    t.x *= a.magnitude;
    t.y *= sign * a.magnitude;
    cs[i] = t;
  }
}

// R: chunks of a lane
template <typename T, int V, int R>
__global__ void __launch_bounds__(QN_THREADS) k_qk_norm(const __grid_constant__ NormArgs a) {
  extern __shared__ float2 cs[];                      // [tile][pairs]
  pdl_trigger();
  pdl_wait();
  const int row0 = blockIdx.x * a.tile, rows = min(a.tile, a.rows - row0), heads = a.nq + a.nk;
  const int per = QN_THREADS / a.lanes, lane = threadIdx.x % a.lanes, total = rows * heads;
  tile_angles(a, row0, rows, 1.f, cs);
  __syncthreads();
  for (int s0 = 0; s0 < total; s0 += per) {           // (all lanes of a warp stay for the sums)
    const int s = s0 + threadIdx.x / a.lanes;
    const bool live = s < total;
    const int r = live ? s / heads : 0;
    int h = live ? s - r * heads : 0;
    const bool isk = h >= a.nq;
    if (isk) h -= a.nq;
    const size_t row = row0 + r;
    const T *src = (isk ? (const T *)a.k + row * a.ks : (const T *)a.q + row * a.qs) + (size_t)h * a.hd;
    T *dst = (isk ? (T *)a.ko + row * a.kos : (T *)a.qo + row * a.qos) + (size_t)h * a.hd;
    const T *w = (const T *)(isk ? a.kw : a.qw);
    float x[R][2 * V];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const Chunk<V> c(a, lane + i * a.lanes);
      load_dims<T, V>(src, live ? c.lo : a.hd, a.hd, x[i]);
      load_dims<T, V>(src, live ? c.hi : a.hd, a.hd, x[i] + V);
#pragma unroll
      for (int j = 0; j < 2 * V; ++j) ss = fmaf(x[i][j], x[i][j], ss);
    }
    const float inv = __frsqrt_rn(head_sum(ss, a.lanes) / (float)a.hd + a.eps);
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const Chunk<V> c(a, lane + i * a.lanes);
      float y[2 * V];
      load_dims<T, V>(w, c.lo, a.hd, y);
      load_dims<T, V>(w, c.hi, a.hd, y + V);
#pragma unroll
      for (int j = 0; j < 2 * V; ++j) y[j] *= x[i][j] * inv;
      turn_chunk<V>(a, c, cs + r * (a.rot / 2), y);
      store_dims<T, V>(dst, c.lo, a.hd, y);
      store_dims<T, V>(dst, c.hi, a.hd, y + V);
    }
  }
}

// The gradient: CTAs walk the tiles, q's heads and then k's, each lane with the same chunks of every head, whose sums
// of n' x r it keeps; they are added up over the CTA at the end, in a fixed order.
template <typename T, int V, int R>
__global__ void __launch_bounds__(QN_THREADS) k_qk_norm_grad(const __grid_constant__ NormArgs a) {
  extern __shared__ float2 cs[];                      // [tile][pairs], then [warps][hd] sums
  pdl_trigger();
  pdl_wait();
  const int per = QN_THREADS / a.lanes, lane = threadIdx.x % a.lanes;
  float wsum[2][R][2 * V];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 2 * V; ++j) wsum[k][i][j] = 0.f;
  const int tiles = (a.rows + a.tile - 1) / a.tile;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int row0 = t * a.tile, rows = min(a.tile, a.rows - row0);
    tile_angles(a, row0, rows, -1.f, cs);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int heads = k ? a.nk : a.nq, total = rows * heads;
      const T *w = (const T *)(k ? a.kw : a.qw);
      const int64_t xs = k ? a.ks : a.qs, gs = k ? a.gks : a.gqs, os = k ? a.kos : a.qos;
      for (int s0 = 0; s0 < total; s0 += per) {
        const int s = s0 + threadIdx.x / a.lanes;
        const bool live = s < total;
        const int r = live ? s / heads : 0, h = live ? s - r * heads : 0;
        const size_t row = row0 + r;
        const T *src = (const T *)(k ? a.k : a.q) + row * xs + (size_t)h * a.hd;
        const T *up = (const T *)(k ? a.gk : a.gq) + row * gs + (size_t)h * a.hd;
        T *dst = (T *)(k ? a.ko : a.qo) + row * os + (size_t)h * a.hd;
        float x[R][2 * V], g[R][2 * V];
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const Chunk<V> c(a, lane + i * a.lanes);
          load_dims<T, V>(src, live ? c.lo : a.hd, a.hd, x[i]);
          load_dims<T, V>(src, live ? c.hi : a.hd, a.hd, x[i] + V);
          load_dims<T, V>(up, live ? c.lo : a.hd, a.hd, g[i]);
          load_dims<T, V>(up, live ? c.hi : a.hd, a.hd, g[i] + V);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const Chunk<V> c(a, lane + i * a.lanes);
          turn_chunk<V>(a, c, cs + r * (a.rot / 2), g[i]);
          float y[2 * V];
          load_dims<T, V>(w, c.lo, a.hd, y);
          load_dims<T, V>(w, c.hi, a.hd, y + V);
#pragma unroll
          for (int j = 0; j < 2 * V; ++j) {
            ss = fmaf(x[i][j], x[i][j], ss);
            dot = fmaf(g[i][j] * y[j], x[i][j], dot);
          }
        }
        ss = head_sum(ss, a.lanes);
        dot = head_sum(dot, a.lanes);
        const float inv = __frsqrt_rn(ss / (float)a.hd + a.eps), m = dot * inv / (float)a.hd;   // r mean(g x)
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const Chunk<V> c(a, lane + i * a.lanes);
          float y[2 * V];
          load_dims<T, V>(w, c.lo, a.hd, y);
          load_dims<T, V>(w, c.hi, a.hd, y + V);
#pragma unroll
          for (int j = 0; j < 2 * V; ++j) {
            const float u = x[i][j] * inv;
            wsum[k][i][j] = fmaf(g[i][j], u, wsum[k][i][j]);
            y[j] = inv * fmaf(g[i][j], y[j], -u * m);
          }
          store_dims<T, V>(dst, c.lo, a.hd, y);
          store_dims<T, V>(dst, c.hi, a.hd, y + V);
        }
      }
    }
    __syncthreads();                                  // the angles are done with
  }
  float *sums = (float *)cs;
  const int warp = threadIdx.x >> 5;
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const Chunk<V> c(a, lane + i * a.lanes);
#pragma unroll
      for (int j = 0; j < 2 * V; ++j) {
        float v = k ? wsum[1][i][j] : wsum[0][i][j];
        for (int o = a.lanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        const int first = j < V ? c.lo : c.hi, d = first + j % V;
        if ((threadIdx.x & 31) < a.lanes && first < a.hd) sums[warp * a.hd + d] = v;
      }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < a.hd; d += QN_THREADS) {
      float v = 0.f;
      for (int x = 0; x < QN_THREADS / 32; ++x) v += sums[x * a.hd + d];
      a.part[((size_t)blockIdx.x * 2 + k) * a.hd + d] = v;
    }
    __syncthreads();
  }
}

// dweight[d] = sum of n partial sums: 32 dims of a CTA, 32 threads each
__global__ void __launch_bounds__(1024) k_qk_norm_weights(int n, int hd, const float *part, float *dqw, float *dkw) {
  __shared__ float s[32][33];
  pdl_trigger();
  pdl_wait();
  const int k = blockIdx.y, d = blockIdx.x * 32 + threadIdx.x, y = threadIdx.y;
  float v = 0.f;
  if (d < hd)
    for (int i = y; i < n; i += 32) v += part[((size_t)i * 2 + k) * hd + d];
  s[y][threadIdx.x] = v;
  __syncthreads();
  v = warp_sum(s[threadIdx.x][y]);
  const int dim = blockIdx.x * 32 + y;
  if (threadIdx.x == 0 && dim < hd) (k ? dkw : dqw)[dim] = v;
}

template <typename T, int V, int R>
cudaError_t launch_norm(const NormArgs &a, int *parts, cudaStream_t s) {
  const size_t angles = (size_t)a.tile * (a.rot / 2) * sizeof(float2);
  const int tiles = (a.rows + a.tile - 1) / a.tile;
  if (!parts) return launch_pdl(k_qk_norm<T, V, R>, dim3(tiles), dim3(QN_THREADS), angles, s, a);
  const size_t sums = (size_t)QN_THREADS / 32 * a.hd * sizeof(float);
  *parts = tiles < QN_CTAS ? tiles : QN_CTAS;
  return launch_pdl(k_qk_norm_grad<T, V, R>, dim3(*parts), dim3(QN_THREADS), angles > sums ? angles : sums, s, a);
}

// width: elements of an access; parts: gets the number of partial sums of the gradient (null: forward)
template <typename T>
cudaError_t launch_norm(NormArgs a, int width, int *parts, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  a.chunks = (a.hd + 2 * width - 1) / (2 * width);
  a.lanes = 1;
  while (a.lanes < a.chunks && a.lanes < 32) a.lanes *= 2;
  // a tile of rows has as many heads as the CTA takes at once, but no more than 8 rows
  const int per = QN_THREADS / a.lanes, heads = parts ? (a.nk ? a.nk : a.nq) : a.nq + a.nk;
  a.tile = (per + heads - 1) / heads;
  a.tile = a.tile > 8 ? 8 : a.tile;
  if (width == W) return launch_norm<T, W, 1>(a, parts, s);
  return width == 2 ? launch_norm<T, 2, 2>(a, parts, s) : launch_norm<T, 1, 4>(a, parts, s);
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
  if ((q == q_out && q_stride != q_out_stride) || (nk && k == k_out && k_stride != k_out_stride))
    return DFLASH_ERR_INVALID_ARG;
  NormArgs a = norm_args(rope, rows, n_q_heads, nk, head_dim, eps, positions);
  a.qw = q_weight, a.kw = k_weight;
  a.q = q, a.k = k, a.qo = q_out, a.ko = k_out;
  a.qs = q_stride, a.ks = k_stride, a.qos = q_out_stride, a.kos = k_out_stride;
  const int w = access_width(a, es, f, n);
  const cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = dtype == DFLASH_BF16 ? launch_norm<bf16>(a, w, nullptr, s) : launch_norm<float>(a, w, nullptr, s);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

extern "C" int64_t dflash_qk_norm_rope_workspace(void) { return (int64_t)QN_CTAS * 2 * 256 * sizeof(float); }

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
    if (x->dq == x->q || (nk && x->dk == x->k) || (x->dq == x->grad_q_out && x->dq_stride != x->grad_q_out_stride) ||
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
  int parts = 0;
  if (x->rows) {
    const int w = access_width(a, es, f, n);
    e = x->dtype == DFLASH_BF16 ? launch_norm<bf16>(a, w, &parts, s) : launch_norm<float>(a, w, &parts, s);
  }
  if (e == cudaSuccess)
    e = launch_pdl(k_qk_norm_weights, dim3((hd + 31) / 32, nk ? 2 : 1), dim3(32, 32), 0, s, parts, hd,
                   (const float *)a.part, x->dq_weight, x->dk_weight);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
