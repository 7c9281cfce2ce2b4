// Rotary positions (dflash_rope_init / dflash_rope_apply).
//
// Pair i turns by position * f_i. The host keeps F_i = frac(f_i / 2 pi) * 2^64, to the nearest integer;
// the 64-bit product position * F_i, whose overflow drops whole turns, is then the angle as a fraction
// of a turn. Its error is position * 2^-65 turns, 2^-34 turns (4e-10 rad) at the last int32 position and thus
// below fp32's own everywhere, and there is no table: no memory, no position limit.
//
// Every element of q and k is read and written once, which bounds it: the sine and cosine of a
// row's pairs (at most 128) are computed once in shared memory and used by all of its heads.
#include <cmath>

#include "rope.cuh"

namespace dflash {

constexpr int ROPE_THREADS = 256;

struct RopeArgs {
  uint64_t turn[128];
  float magnitude;
  int rot, rows, nq, nk, hd, transpose;
  const int32_t *positions;
  const void *q, *k;
  void *qo, *ko;
  int64_t qs, ks, qos, kos;
};

// A CTA turns one row; V elements per access (16 or 8 bytes, or two elements or one where a row, a
// head or the rotated part does not keep the alignment). EARLY: for rows of one chunk per thread, whose loads are then on
// their way while the angles are made (5003 rows of 16 x 64 fp32: 10.1 against 13.7 us). Longer rows have more
// loads after the first, and the registers held across the barrier cost them more (32768 rows of 48 x 128 bf16: 152
// against 123 us, 6.5 TB/s).
template <typename T, int V, bool INTER, bool EARLY>
__global__ void __launch_bounds__(ROPE_THREADS) k_rope(const __grid_constant__ RopeArgs a) {
  extern __shared__ float2 cs[];                      // [pairs]
  pdl_trigger();
  pdl_wait();
  const int pairs = a.rot / 2, row = blockIdx.x;
  // Chunks of a head: the half layout takes V dims of the first half with their partners, the
  // interleaved one V neighbouring dims (V / 2 pairs, one pair where V is 1); then the copied tail.
  constexpr int IW = INTER && V == 1 ? 2 : V;         // dims of an interleaved chunk
  const int rot_chunks = INTER ? a.rot / IW : pairs / V;
  const int chunks = rot_chunks + (a.hd - a.rot) / V;
  const int per_row = (a.nq + a.nk) * chunks;
  typedef Vec<T, V> VT;
  VT early_x, early_y;
  if (EARLY && threadIdx.x < per_row) {
    int h = threadIdx.x / chunks;
    const int c = threadIdx.x - h * chunks, d = c >= rot_chunks ? a.rot + (c - rot_chunks) * V : c * IW;
    const bool isk = h >= a.nq;
    if (isk) h -= a.nq;
    const T *src = (isk ? (const T *)a.k + (size_t)row * a.ks : (const T *)a.q + (size_t)row * a.qs) + (size_t)h * a.hd + d;
    early_x = *(const VT *)src;
    if (!INTER && c < rot_chunks) early_y = *(const VT *)(src + pairs);
  }
  for (int p = threadIdx.x; p < pairs; p += ROPE_THREADS) {
    float2 t = phase_cs((uint64_t)(int64_t)a.positions[row] * a.turn[p]);
    t.x *= a.magnitude;
    t.y *= a.transpose ? -a.magnitude : a.magnitude;
    cs[p] = t;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < per_row; i += ROPE_THREADS) {
    int h = i / chunks;
    const int c = i - h * chunks;
    const bool isk = h >= a.nq;
    if (isk) h -= a.nq;
    const T *src = isk ? (const T *)a.k + (size_t)row * a.ks : (const T *)a.q + (size_t)row * a.qs;
    T *dst = isk ? (T *)a.ko + (size_t)row * a.kos : (T *)a.qo + (size_t)row * a.qos;
    src += (size_t)h * a.hd;
    dst += (size_t)h * a.hd;
    if (c >= rot_chunks) {
      const int d = a.rot + (c - rot_chunks) * V;
      if (src != dst) *(VT *)(dst + d) = EARLY ? early_x : *(const VT *)(src + d);
    } else if (INTER) {
      const int d = c * IW;
      if constexpr (V == 1) {
        const float2 z = turned(to_f(src[d]), to_f(src[d + 1]), cs[c]);
        dst[d] = from_f<T>(z.x);
        dst[d + 1] = from_f<T>(z.y);
      } else {
        VT x = EARLY ? early_x : *(const VT *)(src + d);
#pragma unroll
        for (int j = 0; j < V; j += 2) {
          const float2 z = turned(to_f(x.v[j]), to_f(x.v[j + 1]), cs[(d + j) / 2]);
          x.v[j] = from_f<T>(z.x);
          x.v[j + 1] = from_f<T>(z.y);
        }
        *(VT *)(dst + d) = x;
      }
    } else {
      const int d = c * V;
      VT x = EARLY ? early_x : *(const VT *)(src + d), y = EARLY ? early_y : *(const VT *)(src + d + pairs);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float2 z = turned(to_f(x.v[j]), to_f(y.v[j]), cs[d + j]);
        x.v[j] = from_f<T>(z.x);
        y.v[j] = from_f<T>(z.y);
      }
      *(VT *)(dst + d) = x;
      *(VT *)(dst + d + pairs) = y;
    }
  }
}

template <typename T, int V, bool EARLY>
cudaError_t launch_rope(const RopeArgs &a, bool inter, cudaStream_t s) {
  const dim3 g(a.rows), b(ROPE_THREADS);
  const size_t sm = (size_t)(a.rot / 2) * sizeof(float2);
  return inter ? launch_pdl(k_rope<T, V, true, EARLY>, g, b, sm, s, a) : launch_pdl(k_rope<T, V, false, EARLY>, g, b, sm, s, a);
}
// width: elements that every access may take at once
template <typename T>
cudaError_t launch_rope(const RopeArgs &a, bool inter, int width, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int chunks = (inter ? a.rot / V : a.rot / 2 / V) + (a.hd - a.rot) / V;
  if (width == V && (int64_t)(a.nq + a.nk) * chunks <= ROPE_THREADS) return launch_rope<T, V, true>(a, inter, s);
  if (width == V) return launch_rope<T, V, false>(a, inter, s);
  if (width == V / 2) return launch_rope<T, V / 2, false>(a, inter, s);
  return width == 2 ? launch_rope<T, 2, false>(a, inter, s) : launch_rope<T, 1, false>(a, inter, s);
}

}  // namespace dflash

using namespace dflash;

namespace {
// A double's 53 bits would leave position * 2^-54 turns, 7e-7 rad at 2^31. The table is made in sums of two doubles
// instead (over 100 bits), with error-free sums and products (Dekker 1971), the same on every host: products are
// kept from being contracted into the sums that follow.
struct Two {
  double hi, lo;
};
Two sum(double a, double b) {
  const double s = a + b, t = s - a;
  return Two{s, (a - (s - t)) + (b - t)};
}
Two add(Two a, Two b) {
  const Two s = sum(a.hi, b.hi);
  return sum(s.hi, s.lo + (a.lo + b.lo));
}
Two mul(Two a, Two b) {
  volatile double p = a.hi * b.hi;
  const double e = std::fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi);
  return sum(p, e);
}
Two div(Two a, Two b) {
  const double q = a.hi / b.hi;
  const Two p = mul(Two{q, 0}, b), r = add(a, Two{-p.hi, -p.lo});
  return sum(q, r.hi / b.hi);
}
// e^x for |x| < 90: 18 terms of the series at x / 1024, then squared ten times
Two exponential(Two x) {
  const Two y{x.hi / 1024, x.lo / 1024};
  Two e{1, 0};
  for (int n = 18; n > 0; --n) e = add(Two{1, 0}, mul(div(y, Two{(double)n, 0}), e));
  for (int n = 0; n < 10; ++n) e = mul(e, e);
  return e;
}
// ln x: one step of Newton's method from the double
Two logarithm(double x) {
  const double l = std::log(x);
  const Two e = mul(Two{x, 0}, exponential(Two{-l, 0}));
  return add(Two{l, 0}, add(e, Two{-1, 0}));
}
}  // namespace

extern "C" dflash_status dflash_rope_init(const dflash_rope_params *p, dflash_rope *rope) {
  if (!p || !rope || p->rot_dim < 2 || p->rot_dim > 256 || p->rot_dim % 2 || (p->interleaved & ~1) ||
      p->scaling < DFLASH_ROPE_NONE || p->scaling > DFLASH_ROPE_YARN || !(p->theta > 1.f) || !std::isfinite(p->theta))
    return DFLASH_ERR_INVALID_ARG;
  if (p->scaling != DFLASH_ROPE_NONE && (!(p->factor >= 1.f) || !std::isfinite(p->factor))) return DFLASH_ERR_INVALID_ARG;
  if (p->scaling == DFLASH_ROPE_YARN &&
      (!(p->original_positions > 0.f) || !std::isfinite(p->original_positions) || !(p->beta_slow > 0.f) ||
       !(p->beta_fast > p->beta_slow) || !std::isfinite(p->beta_fast)))
    return DFLASH_ERR_INVALID_ARG;
  const double pi = 3.14159265358979323846, rot = p->rot_dim, lt = std::log((double)p->theta);
  const Two log_theta = logarithm(p->theta), per_turn{0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};   // 1 / (2 pi)
  double lo = 0, hi = 0;
  if (p->scaling == DFLASH_ROPE_YARN) {
    auto dim = [&](double beta) { return rot * std::log(p->original_positions / (beta * 2 * pi)) / (2 * lt); };
    lo = std::fmax(std::floor(dim(p->beta_fast)), 0.0);
    hi = std::fmin(std::ceil(dim(p->beta_slow)), rot - 1);
  }
  for (int i = 0; i < 128; ++i) {
    rope->turn[i] = 0;
    if (i >= p->rot_dim / 2) continue;
    Two f = exponential(div(mul(log_theta, Two{-2.0 * i, 0}), Two{rot, 0}));
    if (p->scaling == DFLASH_ROPE_LINEAR) f = div(f, Two{p->factor, 0});
    if (p->scaling == DFLASH_ROPE_YARN && i > lo) {
      const double past = i - lo, width = std::fmax(hi - lo, 0.001);
      const Two g = past < width ? div(Two{past, 0}, Two{width, 0}) : Two{1, 0};
      f = add(mul(div(f, Two{p->factor, 0}), g), mul(f, add(Two{1, 0}, Two{-g.hi, -g.lo})));
    }
    // f <= 1, so the fraction of a turn is below 0.16 and fits 64 bits
    f = mul(f, per_turn);
    const double turns = f.hi * 0x1p64, whole = std::floor(turns);
    rope->turn[i] = (uint64_t)whole + (uint64_t)(int64_t)std::floor((turns - whole) + f.lo * 0x1p64 + 0.5);
  }
  rope->magnitude = p->scaling == DFLASH_ROPE_YARN ? (float)(0.1 * std::log((double)p->factor) + 1.0) : 1.f;
  rope->rot_dim = p->rot_dim;
  rope->interleaved = p->interleaved;
  return DFLASH_OK;
}

extern "C" dflash_status dflash_rope_apply(void *stream, const dflash_rope *rope, int32_t rows, int32_t n_q_heads,
                                           int32_t n_k_heads, int32_t head_dim, dflash_dtype dtype,
                                           const int32_t *positions, int32_t transpose, const void *q,
                                           int64_t q_stride, const void *k, int64_t k_stride, void *q_out,
                                           int64_t q_out_stride, void *k_out, int64_t k_out_stride) {
  if (!rope || rows < 0 || n_q_heads < 1 || n_k_heads < 0 || n_q_heads > (1 << 20) || n_k_heads > (1 << 20) ||
      n_q_heads + n_k_heads > (1 << 20) || (dtype != DFLASH_F32 && dtype != DFLASH_BF16) || (transpose & ~1) ||
      rope->rot_dim < 2 || rope->rot_dim % 2 || rope->rot_dim > head_dim || head_dim > 256 || (rope->interleaved & ~1))
    return DFLASH_ERR_INVALID_ARG;
  const int nk = k ? n_k_heads : 0;
  const int64_t qw = (int64_t)n_q_heads * head_dim, kw = (int64_t)nk * head_dim;
  if (q_stride < qw || q_out_stride < qw || (nk && (k_stride < kw || k_out_stride < kw))) return DFLASH_ERR_INVALID_ARG;
  if (rows == 0) return DFLASH_OK;
  const unsigned es = dtype_bytes(dtype);
  if (!positions || !q || !q_out || (nk && !k_out) || !aligned(positions, 4) || !aligned(q, es) || !aligned(q_out, es) ||
      (nk && (!aligned(k, es) || !aligned(k_out, es))))
    return DFLASH_ERR_INVALID_ARG;
  if ((q == q_out && q_stride != q_out_stride) || (nk && k == k_out && k_stride != k_out_stride))
    return DFLASH_ERR_INVALID_ARG;
  RopeArgs a;
  for (int i = 0; i < 128; ++i) a.turn[i] = rope->turn[i];
  a.magnitude = rope->magnitude;
  a.rot = rope->rot_dim;
  a.rows = rows;
  a.nq = n_q_heads;
  a.nk = nk;
  a.hd = head_dim;
  a.transpose = transpose;
  a.positions = positions;
  a.q = q;
  a.k = k;
  a.qo = q_out;
  a.ko = k_out;
  a.qs = q_stride;
  a.ks = k_stride;
  a.qos = q_out_stride;
  a.kos = k_out_stride;
  // Wide accesses need every row, every head and both rotated halves on their boundary: 16 bytes, else 8, else
  // two elements, else one (33870 rows of 18 x 64 bf16, 20 dims rotated: 66 us by four, 94 by two, 124 by one).
  auto fits = [&](int n) {
    bool y = aligned(q, n * es) && aligned(q_out, n * es) && q_stride % n == 0 && q_out_stride % n == 0 && head_dim % n == 0 &&
             a.rot % (rope->interleaved ? n : 2 * n) == 0;
    if (nk) y = y && aligned(k, n * es) && aligned(k_out, n * es) && k_stride % n == 0 && k_out_stride % n == 0;
    return y;
  };
  const int V = 16 / es, width = fits(V) ? V : fits(V / 2) ? V / 2 : fits(2) ? 2 : 1;
  const cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = dtype == DFLASH_BF16 ? launch_rope<bf16>(a, rope->interleaved, width, st)
                                             : launch_rope<float>(a, rope->interleaved, width, st);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
