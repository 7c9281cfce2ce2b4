// The choice of blocks for attention over a part of a long context (8-bit paged cache): bounds of a page's keys
// (dflash_kv8_bounds) and the choice by the score that they give (dflash_kv8_select).
#include "kv8_sched.cuh"

namespace dflash {

// ---------------------------------------------------------------- bounds
// A warp per (page, kv head): lanes read 16 bytes of a row each, several rows at a time, and keep the least and the
// largest of their 16 dims. 47 us for 8 prompts of 16384 .. 32768 tokens of 8 x 128 (208 MB of keys, 215 with the bounds
// and the tables, 4.6 TB/s); 65 with a conversion of every pair to f16, 56 with shifts and masks in its place. What is left
// is latency (45% of the issue slots, 58% of DRAM, and 12 of a warp's 16 cycles an instruction are the wait for its
// rows): a page of a head is a chain of its own, table entry, rows, shuffles, store. More of them hide it better: 8 x 16384
// tokens take 33 us, the next 8 x 16384 24.5 (5.6 TB/s).
constexpr int KB_THREADS = 256;
constexpr int KB_CTAS = 152 * 4;

struct BoundsArgs {
  int n_req, width, n_pages, nkv;
  const int32_t *old_len, *new_len, *table;
  const uint8_t *kp;
  int8_t *bounds;
};

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *(const __half2 *)&x; }
__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t x) { return *(const __nv_bfloat162 *)&x; }

template <int HD>
__global__ void __launch_bounds__(KB_THREADS) k_kv8_bounds(const BoundsArgs a) {
  extern __shared__ long long kb_pre[];               // [n_req + 1]: pages touched by the requests before
  __shared__ long long warp_tot[KB_THREADS / 32];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long cap = (long long)a.width * KV_PAGE;
  auto lens = [&](int b, int &first, int &end) {      // rows [first, end) of request b
    first = (int)max(0ll, min((long long)a.old_len[b], cap));
    end = (int)max(0ll, min((long long)a.new_len[b], cap));
  };
  const int ipt = (a.n_req + KB_THREADS - 1) / KB_THREADS;
  long long mine = 0;
  for (int i = 0; i < ipt; ++i) {
    const int b = tid * ipt + i;
    if (b >= a.n_req) break;
    int s, e;
    lens(b, s, e);
    if (e > s) mine += (e + KV_PAGE - 1) / KV_PAGE - s / KV_PAGE;
  }
  long long inc = warp_scan_ll(mine);
  if (lane == 31) warp_tot[warp] = inc;
  __syncthreads();
  for (int i = 0; i < warp; ++i) inc += warp_tot[i];
  long long run = inc - mine;
  for (int i = 0; i < ipt; ++i) {
    const int b = tid * ipt + i;
    if (b >= a.n_req) break;
    int s, e;
    lens(b, s, e);
    kb_pre[b] = run;
    if (e > s) run += (e + KV_PAGE - 1) / KV_PAGE - s / KV_PAGE;
  }
  if (tid == KB_THREADS - 1) kb_pre[a.n_req] = inc;
  __syncthreads();
  const long long tasks = kb_pre[a.n_req] * a.nkv, step = (long long)gridDim.x * (KB_THREADS / 32);
  constexpr int LPR = HD / 16, RPI = 32 / LPR;        // lanes of a row, rows at a time
  for (long long t = (long long)blockIdx.x * (KB_THREADS / 32) + warp; t < tasks; t += step) {
    const long long pg = t / a.nkv;
    const int h = (int)(t - pg * a.nkv);
    int lo = 0, hi = a.n_req - 1;                      // the last request whose pages begin at or before pg
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (kb_pre[m] <= pg) lo = m;
      else hi = m - 1;
    }
    int s, e;
    lens(lo, s, e);
    const int blk = s / KV_PAGE + (int)(pg - kb_pre[lo]);
    const int page = a.table[(size_t)lo * a.width + blk];
    if (page < 0 || page >= a.n_pages) continue;
    const int rows = min(KV_PAGE, e - blk * KV_PAGE);
    const uint8_t *src = a.kp + kv8_block(page, h, a.nkv, HD) + lane * 16;
    // Per word of four bytes the pairs (0, 2) and (1, 3). Read as bf16, a pair with its values in the high bytes is in their
    // order whatever the low bytes hold (they only decide between equals), so that a word takes one shift and no
    // conversion. NaN passes every value or is left out; where it shows (0x7f in the result), or nothing does, the scan is
    // made again in f16, which leaves NaN out.
    auto load = [&](int r0, uint4 (&w)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // (past the end: the first row again)
        const int r = r0 + i * RPI < rows ? r0 + i * RPI : r0;
        w[i] = *(const uint4 *)(src + (size_t)(r - lane / LPR) * HD);
      }
    };
    __nv_bfloat162 least[8], most[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      least[j] = as_bf162(0x7f7f7f7fu);
      most[j] = as_bf162(0xff7fff7fu);
    }
#pragma unroll 1
    for (int r0 = lane / LPR; r0 < rows; r0 += 8 * RPI) {
      uint4 w[8];
      load(r0, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 e = as_bf162(v[j] << 8), o = as_bf162(v[j]);
          least[2 * j] = __hmin2(least[2 * j], e);
          most[2 * j] = __hmax2(most[2 * j], e);
          least[2 * j + 1] = __hmin2(least[2 * j + 1], o);
          most[2 * j + 1] = __hmax2(most[2 * j + 1], o);
        }
      }
    }
    __syncwarp();
    uint32_t nan = 0;
    uint32_t out[8];                                   // the least (the largest) of dims 4 (j / 2) + (j & 1) and two further, in the second and fourth byte
    const bool up = lane >= LPR;                       // the first row's lanes write the least, the second's the largest
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) {
        least[j] = __hmin2(least[j], __shfl_xor_sync(0xffffffffu, least[j], o));
        most[j] = __hmax2(most[j], __shfl_xor_sync(0xffffffffu, most[j], o));
      }
      const uint32_t l = *(const uint32_t *)&least[j], m = *(const uint32_t *)&most[j];
      nan |= nan_bytes(l) | nan_bytes(m);
      out[j] = up ? m : l;
    }
    if (__any_sync(0xffffffffu, (nan & 0x80008000u) != 0)) {
      __half2 lh[8], mh[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        lh[j] = as_half2(0x7c007c00u);
        mh[j] = as_half2(0xfc00fc00u);
      }
#pragma unroll 1
      for (int r = lane / LPR; r < rows; r += RPI) {
        const uint4 w = *(const uint4 *)(src + (size_t)(r - lane / LPR) * HD);
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t p0, p1;
          e4m3x4_to_f16(v[j], p0, p1);
          const __half2 e = as_half2(__byte_perm(p0, p1, 0x5410)), o = as_half2(__byte_perm(p0, p1, 0x7632));
          lh[2 * j] = __hmin2(lh[2 * j], e);
          mh[2 * j] = __hmax2(mh[2 * j], e);
          lh[2 * j + 1] = __hmin2(lh[2 * j + 1], o);
          mh[2 * j + 1] = __hmax2(mh[2 * j + 1], o);
        }
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) {
          lh[j] = __hmin2(lh[j], __shfl_xor_sync(0xffffffffu, lh[j], o));
          mh[j] = __hmax2(mh[j], __shfl_xor_sync(0xffffffffu, mh[j], o));
        }
        // back to bytes (exact); a dim of nothing but NaN: 0
        const float2 l = __half22float2(lh[j]), m = __half22float2(mh[j]);
        const uint32_t x = f32_to_e4m3x2(l.x > m.x ? 0.f : up ? m.x : l.x, l.y > m.y ? 0.f : up ? m.y : l.y);
        out[j] = __byte_perm(x, 0, 0x1404);
      }
    }
    if (lane < 2 * LPR) {
      uint32_t b[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 v = e4m3x2_to_f32(__byte_perm(out[j], 0, 0x4431));
        const int x = (int)(up ? ceilf(v.x * 0.25f) : floorf(v.x * 0.25f)), y = (int)(up ? ceilf(v.y * 0.25f) : floorf(v.y * 0.25f));
        b[j / 2] |= ((uint32_t)(x & 255) | (uint32_t)(y & 255) << 16) << 8 * (j & 1);
      }
      *(uint4 *)(a.bounds + ((size_t)page * a.nkv + h) * (2 * HD) + lane * 16) = make_uint4(b[0], b[1], b[2], b[3]);
    }
  }
}

// ---------------------------------------------------------------- scores
// score[block] = max over rows of (q+ . hi + q- . lo) unit * 4 scale, q+ = max(q, 0) and q- = min(q, 0) in whole
// numbers of at most 1024: two m16n8k16 products of 16 blocks with 8 rows, in f16 with fp32 sums. Products are at most
// 2^17 and the sums of a row at most 2^24, so every partial sum is a whole number that fp32 (and an accumulator that
// truncates) holds. Contraction indices are permuted as in the attention for few rows: a lane's 16 bytes are the dims of
// four steps.
//
// The bounds are few bytes (26 MB for 8 x 16 rows of 40 heads over 1024 .. 2049 blocks, 4 us), and what takes 25 us there are
// the latencies of a round (table, bounds, the products' chains of sums) with 16 warps per SM, and the reads of q's
// fragments from shared memory. Both halves of q are kept there (46 us when they were made at every use), and all
// of a CTA's rows are loaded at once.
constexpr int KS_THREADS = 256;
constexpr int KS_TILE = KS_THREADS / 2;               // blocks of a CTA at once: 16 of a warp
// Rows of q staged at once: 16 rows of the most heads to a kv head, 8. More rows take another round, which reads the table
// and converts the bounds again. 8 x 16 rows over 1024 .. 2049 blocks with 80, 96 and 128: 47.8, 48.1 and 41.8 us for 8
// heads to a kv head, 44.9, 45.3 and 38.8 for 7, 32.6, 32.7 and 32.7 for 5; 16 single tokens over 513 blocks 14.9, 15.0 and
// 15.1. (A 64-bit division a row instead of the product took 0.9 us of the first three.)
constexpr int KS_ROWS = 128;
template <int HD>
constexpr size_t KS_SMEM = (size_t)KS_ROWS / 8 * (HD / 16) * 32 * sizeof(uint4) + KS_ROWS * sizeof(float);

struct SelectArgs {
  Kv8AttnArgs a;
  int n_select, first, last;
  const int8_t *bounds;
  float *score;                                       // [n_req][nkv][width]
  int32_t *blocks;
};

// four signed bytes as two f16 pairs: byte + 128 in the low bits of 1024 + .., less 1152
__device__ __forceinline__ void s8x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
  const uint32_t u = w ^ 0x80808080u;
  lo = sub_f16x2(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u);
  hi = sub_f16x2(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u);
}

template <typename T>
struct Vec4;
template <>
struct Vec4<bf16> {
  uint2 w;
  __device__ __forceinline__ void get(float (&v)[4]) const {
    v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xffff0000u);
  }
};
template <>
struct Vec4<float> {
  float4 w;
  __device__ __forceinline__ void get(float (&v)[4]) const { v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w; }
};

template <typename T, int HD>
__global__ void __launch_bounds__(KS_THREADS, 2) k_kv8_scores(const SelectArgs x) {
  constexpr int KS = HD / 16, C = HD / 64;
  extern __shared__ uint4 ks_smem[];
  uint4(*qf)[KS][32] = (uint4(*)[KS][32])ks_smem;      // [KS_ROWS / 8]: fragments of q+ and of q-
  float *unit = (float *)(qf + KS_ROWS / 8);           // [KS_ROWS], 0: a row that has no say
  const Kv8AttnArgs &a = x.a;
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.z, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const Kv8Req r = kv8_req(a, b);
  const int blocks = (r.len + KV_PAGE - 1) / KV_PAGE, group = a.nq / a.nkv;
  if (r.n == 0 || blocks <= x.n_select || blockIdx.x * KS_TILE >= blocks) return;
  const long long rows = (long long)r.n * group;
  float *score = x.score + ((size_t)b * a.nkv + h) * a.width;
  const uint32_t inv_group = 65536u / group + 1;       // (exact for the 135 rows and 8 heads at most that it is used for)
  for (long long r0 = 0; r0 < rows; r0 += KS_ROWS) {
    // q in whole numbers: HD / 4 lanes a row, four dims each
    constexpr int LPR = HD / 4, N = KS_ROWS * LPR / KS_THREADS;
    const int here = (int)min((long long)KS_ROWS, rows - r0), tiles = (here + 7) / 8;
    const int i0 = threadIdx.x / LPR, l = threadIdx.x % LPR;
    typedef Vec4<T> Q4;
    const long long token0 = r0 / group;
    const int rest = (int)(r0 - token0 * group);
    const T *q0 = (const T *)a.q + (r.row0 + token0) * a.q_stride + (int64_t)h * group * HD + 4 * l;
    Q4 in[N];                                         // all loads first
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = i0 + n * (KS_THREADS / LPR);
      const int token = (int)((uint32_t)(rest + i) * inv_group >> 16);          // (rest + i) / group
      in[n] = i < here ? *(const Q4 *)(q0 + token * a.q_stride + (rest + i - token * group) * HD) : Q4{};
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = i0 + n * (KS_THREADS / LPR);
      if (n * (KS_THREADS / LPR) >= tiles * 8) break;  // (the same for the CTA)
      float v[4];
      in[n].get(v);
      uint32_t top = 0;                               // bits of the largest magnitude: NaN and infinity are the largest
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const bool fin = top < 0x7f800000u;
      // top = m 2^k, m in [1/2, 1): unit 2^(k - 10)
      const int k = max((int)(top >> 23) - 126, -100);
      const float up = __uint_as_float((uint32_t)(137 - k) << 23);
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const __half2 y = __floats2half2_rn(fin ? rintf(v[2 * j] * up) : 0.f, fin ? rintf(v[2 * j + 1] * up) : 0.f);
        const __half2 p = __hmax2(y, as_half2(0)), m = __hmin2(y, as_half2(0));
        w[j] = *(const uint32_t *)&p;
        w[2 + j] = *(const uint32_t *)&m;
      }
      // dims 4 l .. + 3 are word l & 3 of lane l / 4 & 3's 16 bytes in chunk l / 16
      qf[i / 8][l / 16 * 4 + (l & 3)][(i & 7) * 4 + (l >> 2 & 3)] = make_uint4(w[0], w[1], w[2], w[3]);
      if (l == 0) unit[i] = i < here && fin ? __uint_as_float((uint32_t)(117 + k) << 23) : 0.f;
    }
    __syncthreads();
    auto page_at = [&](int p) { return p < blocks ? a.table[(size_t)b * a.width + p] : -1; };
    const int p_first = blockIdx.x * KS_TILE + warp * 16, p_step = gridDim.x * KS_TILE;
    int ahead[2] = {page_at(p_first + g), page_at(p_first + g + 8)};
    for (int p0 = p_first; p0 < blocks; p0 += p_step) {
      int page[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        page[y] = ahead[y] >= a.n_pages ? -1 : ahead[y];
        ahead[y] = page_at(p0 + p_step + g + 8 * y);
      }
      uint32_t lo[KS][4], hi[KS][4];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int8_t *src = x.bounds + ((size_t)max(page[y], 0) * a.nkv + h) * (2 * HD) + 16 * t;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const uint4 l4 = page[y] >= 0 ? *(const uint4 *)(src + 64 * c) : make_uint4(0, 0, 0, 0);
          const uint4 h4 = page[y] >= 0 ? *(const uint4 *)(src + HD + 64 * c) : make_uint4(0, 0, 0, 0);
          const uint32_t lw[4] = {l4.x, l4.y, l4.z, l4.w}, hw[4] = {h4.x, h4.y, h4.z, h4.w};
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            s8x4_to_f16(lw[s], lo[4 * c + s][y], lo[4 * c + s][2 + y]);
            s8x4_to_f16(hw[s], hi[4 * c + s][y], hi[4 * c + s][2 + y]);
          }
        }
      }
      float best[2] = {-INFINITY, -INFINITY};
      // two tiles of rows at a time, whose chains of sums interleave (an odd last one is its own partner)
      for (int n = 0; n < tiles; n += 2) {
        const int at[2] = {n, min(n + 1, tiles - 1)};
        float up[2][4], dn[2][4];
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
          for (int i = 0; i < 4; ++i) up[z][i] = dn[z][i] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const uint4 q = qf[at[z]][k][lane];
            mma_f16(up[z], hi[k], q.x, q.y);
            mma_f16(dn[z], lo[k], q.z, q.w);
          }
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float u0 = unit[8 * at[z] + 2 * t], u1 = unit[8 * at[z] + 2 * t + 1];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            if (u0 > 0.f) best[y] = fmaxf(best[y], (up[z][2 * y] + dn[z][2 * y]) * u0);
            if (u1 > 0.f) best[y] = fmaxf(best[y], (up[z][2 * y + 1] + dn[z][2 * y + 1]) * u1);
          }
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        best[y] = fmaxf(best[y], __shfl_xor_sync(0xffffffffu, best[y], 1));
        best[y] = fmaxf(best[y], __shfl_xor_sync(0xffffffffu, best[y], 2));
        const int p = p0 + g + 8 * y;
        if (t || p >= blocks) continue;
        float v = page[y] < 0 ? -INFINITY : best[y] * (4.f * x.a.ks[(size_t)page[y] * a.nkv + h]);
        if (!(v == v)) v = -INFINITY;
        score[p] = r0 ? fmaxf(score[p], v) : v;
      }
    }
  }
}

// ---------------------------------------------------------------- the n_select best
// A CTA per (request, kv head). Keys rank as the scores do (fixed blocks above all); four passes over the keys' bytes,
// each a histogram of the keys that agree with the threshold so far, find the last key that is taken and how many of
// those equal to it; the passes end where all keys of the last bin are taken, and the chosen ones are then written in
// order. It is latency: 9 us for 2049 keys, most of it barriers.
constexpr int KC_THREADS = 512;
constexpr int KC_HELD = 4096;                         // keys that are kept in shared memory

__global__ void __launch_bounds__(KC_THREADS) k_kv8_choose(const SelectArgs x) {
  __shared__ int hist[256], warp_tot[KC_THREADS / 32];
  __shared__ uint32_t held[KC_HELD];
  __shared__ int s_bin, s_left, s_all;
  const Kv8AttnArgs &a = x.a;
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Kv8Req r = kv8_req(a, b);
  const int blocks = r.n ? (r.len + KV_PAGE - 1) / KV_PAGE : 0;
  int32_t *out = x.blocks + ((size_t)b * a.nkv + h) * x.n_select;
  if (blocks <= x.n_select) {
    for (int i = tid; i < x.n_select; i += KC_THREADS) out[i] = i < blocks ? i : -1;
    return;
  }
  const float *score = x.score + ((size_t)b * a.nkv + h) * a.width;
  // floor((len - n) / 64) - last; the rows may be more than the context
  const int d = r.len - r.n, own = (d >= 0 ? d / KV_PAGE : -((-d + KV_PAGE - 1) / KV_PAGE)) - x.last;
  auto key_of = [&](int j) {
    if (j < x.first || j >= own) return 0xffffffffu;
    const uint32_t u = __float_as_uint(score[j] + 0.f);                 // (-0 as 0)
    return u & 0x80000000u ? ~u : u | 0x80000000u;
  };
  const bool fits = blocks <= KC_HELD;
  if (fits)
    for (int j = tid; j < blocks; j += KC_THREADS) held[j] = key_of(j);        // (read by the thread that wrote it)
  auto key = [&](int j) { return fits ? held[j] : key_of(j); };
  uint32_t prefix = 0;
  int left = x.n_select;                               // of the keys that begin with prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += KC_THREADS) hist[i] = 0;
    __syncthreads();
    for (int j = tid; j < blocks; j += KC_THREADS) {
      const uint32_t k = key(j);
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[k >> shift & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {                                   // from the top: the bin where the count passes left
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += c[i] = hist[255 - 8 * lane - i];
      int inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      int before = inc - sum;
      if (before < left && inc >= left) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < left && before + c[i] >= left) {
            s_bin = 255 - 8 * lane - i;
            s_left = left - before;
            s_all = c[i] == left - before;
          }
          before += c[i];
        }
      }
    }
    __syncthreads();
    prefix |= (uint32_t)s_bin << shift;
    left = s_left;
    const bool all = s_all;
    __syncthreads();
    if (all) {                                         // every key that begins so is taken: none is below prefix
      --prefix;                                        // (never below 0: then all keys would be taken, which are more)
      left = 0;
      break;
    }
  }
  // keys above prefix, and the first `left` equal to it
  int done = 0, equal = 0;
  for (int j0 = 0; j0 < blocks; j0 += KC_THREADS) {
    const int j = j0 + tid;
    const uint32_t k = j < blocks ? key(j) : 0;
    const bool eq = j < blocks && k == prefix, over = j < blocks && k > prefix;
    const unsigned be = __ballot_sync(0xffffffffu, eq), bo = __ballot_sync(0xffffffffu, over), lt = (1u << lane) - 1;
    if (lane == 0) warp_tot[warp] = __popc(be) | __popc(bo) << 16;
    __syncthreads();
    int tot = 0, mine = 0;
#pragma unroll
    for (int i = 0; i < KC_THREADS / 32; ++i) {
      if (i == warp) mine = tot;
      tot += warp_tot[i];
    }
    const int e = equal + (mine & 0xffff) + __popc(be & lt), o = (mine >> 16) + __popc(bo & lt);
    // equal ones before this one that are taken
    if (over || (eq && e < left)) out[done + o + min(e, left) - min(equal, left)] = j;
    const int all = equal + (tot & 0xffff);
    done += (tot >> 16) + min(all, left) - min(equal, left);
    equal = all;
    __syncthreads();
  }
}

}  // namespace dflash

using namespace dflash;

extern "C" dflash_status dflash_kv8_bounds(void *stream, const dflash_kv8_cache *c, int8_t *bounds, int32_t n_req,
                                           int32_t max_blocks, const int32_t *old_len, const int32_t *new_len,
                                           const int32_t *block_table) {
  if (!kv8_cache_ok(c) || n_req < 1 || n_req > KV8_MAX_REQ || max_blocks < 1 || max_blocks > (1 << 24) || !bounds ||
      !aligned(bounds, 16) || !old_len || !new_len || !block_table || !aligned(old_len, 4) || !aligned(new_len, 4) ||
      !aligned(block_table, 4))
    return DFLASH_ERR_INVALID_ARG;
  const BoundsArgs a{n_req, max_blocks, c->n_pages, c->n_kv_heads, old_len, new_len, block_table,
                     (const uint8_t *)c->k_pages, bounds};
  const int64_t most = ((int64_t)n_req * max_blocks * c->n_kv_heads + KB_THREADS / 32 - 1) / (KB_THREADS / 32);
  const dim3 g((unsigned)(most < KB_CTAS ? most : KB_CTAS)), t(KB_THREADS);
  const size_t sm = (size_t)(n_req + 1) * sizeof(long long);
  const cudaError_t e = c->head_dim == 128 ? launch_pdl(k_kv8_bounds<128>, g, t, sm, (cudaStream_t)stream, a)
                                           : launch_pdl(k_kv8_bounds<64>, g, t, sm, (cudaStream_t)stream, a);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

namespace {
bool choice_ok(const dflash_kv8_cache *c, const dflash_kv8_choice *x) {
  constexpr int most = 1 << 24;
  if (!c || !x || c->n_pages < 1 || c->n_pages > most || c->n_kv_heads < 1 || c->n_kv_heads > 128 ||
      (c->head_dim != 64 && c->head_dim != 128) || x->n_req < 1 || x->n_req > KV8_MAX_REQ || x->rows < 0 ||
      x->n_q_heads < 1 || x->n_q_heads % c->n_kv_heads || x->n_q_heads / c->n_kv_heads > 8 || x->max_blocks < 1 ||
      x->max_blocks > most || x->n_select < 1 || x->n_select > most || x->keep_first < 0 || x->keep_first > most ||
      x->keep_last < 0 || x->keep_last > most || (x->dtype != DFLASH_F32 && x->dtype != DFLASH_BF16))
    return false;
  return (int64_t)x->n_req * c->n_kv_heads * x->n_select < (1ll << 31) &&
         x->q_stride >= (int64_t)x->n_q_heads * c->head_dim && x->q_stride % (16 / dtype_bytes(x->dtype)) == 0;
}
template <typename T, int HD>
cudaError_t launch_scores(const SelectArgs &x, dim3 g, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(k_kv8_scores<T, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)KS_SMEM<HD>);
  return e != cudaSuccess ? e : launch_pdl(k_kv8_scores<T, HD>, g, dim3(KS_THREADS), KS_SMEM<HD>, s, x);
}
template <typename T>
cudaError_t launch_select(const SelectArgs &x, int hd, cudaStream_t s) {
  // CTAs of a (request, kv head), which take KS_TILE blocks at a time in turn: as many as are resident (64 items over
  // 1024 .. 2049 blocks with 2 each 43.5 us, 4 34.4, 5 36.2, 8 37.2, 17 40.8: each makes q's whole numbers for itself)
  const long items = (long)x.a.n_req * x.a.nkv, want = items < 304 ? 304 / items : 1;
  const long most = ((long)x.a.width + KS_TILE - 1) / KS_TILE;
  const dim3 g((unsigned)(want < most ? want : most), x.a.nkv, x.a.n_req);
  cudaError_t e = cudaSuccess;
  if (x.a.width > x.n_select) e = hd == 128 ? launch_scores<T, 128>(x, g, s) : launch_scores<T, 64>(x, g, s);
  if (e == cudaSuccess) e = launch_pdl(k_kv8_choose, dim3(x.a.nkv, x.a.n_req), dim3(KC_THREADS), 0, s, x);
  return e;
}
}  // namespace

extern "C" int64_t dflash_kv8_select_workspace(const dflash_kv8_cache *c, const dflash_kv8_choice *x) {
  if (!choice_ok(c, x)) return -1;
  return (int64_t)x->n_req * c->n_kv_heads * x->max_blocks * (int64_t)sizeof(float);
}

extern "C" dflash_status dflash_kv8_select(void *stream, const dflash_kv8_cache *c, const dflash_kv8_choice *x) {
  if (!choice_ok(c, x) || !c->k_scale || !aligned(c->k_scale, 4)) return DFLASH_ERR_INVALID_ARG;
  if (!x->cu_q || !x->ctx_len || !x->block_table || !x->bounds || !x->blocks || !x->workspace || (x->rows && !x->q) ||
      !aligned(x->cu_q, 4) || !aligned(x->ctx_len, 4) || !aligned(x->block_table, 4) || !aligned(x->bounds, 16) ||
      !aligned(x->blocks, 4) || !aligned(x->workspace, 256) || !aligned(x->q, 16) ||
      x->workspace_bytes < dflash_kv8_select_workspace(c, x))
    return DFLASH_ERR_INVALID_ARG;
  SelectArgs s{};
  s.a.n_req = x->n_req, s.a.rows = x->rows, s.a.nq = x->n_q_heads, s.a.nkv = c->n_kv_heads, s.a.width = x->max_blocks;
  s.a.n_pages = c->n_pages, s.a.q = x->q, s.a.q_stride = x->q_stride;
  s.a.cu_q = x->cu_q, s.a.ctx_len = x->ctx_len, s.a.table = x->block_table, s.a.ks = c->k_scale;
  s.n_select = x->n_select, s.first = x->keep_first, s.last = x->keep_last;
  s.bounds = x->bounds, s.score = (float *)x->workspace, s.blocks = x->blocks;
  const cudaError_t e = x->dtype == DFLASH_BF16 ? launch_select<bf16>(s, c->head_dim, (cudaStream_t)stream)
                                                : launch_select<float>(s, c->head_dim, (cudaStream_t)stream);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
