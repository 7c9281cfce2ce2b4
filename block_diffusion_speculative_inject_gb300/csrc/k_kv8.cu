// The caller-owned 8-bit paged cache: block tables and slot maps from request lengths
// (dflash_page_plan), the quantised write (dflash_kv8_append) and its inspection (dflash_kv8_read).
#include "kv8.cuh"

namespace dflash {

// ---------------------------------------------------------------- page planning
// Per request: pages asked for, pages given back and rows added, as prefix sums over the requests.
// Every CTA computes the same sums from the same inputs (a few KB, read from L2) and then writes
// its share of the rows, so one launch does without a second pass or a grid barrier; that is why
// outputs may not be inputs. It is bound by latency: two block scans and a few dependent loads.
constexpr int PP_THREADS = 512;
constexpr int PP_IPT = KV8_MAX_REQ / PP_THREADS;      // requests per thread, at most

struct PlanArgs {
  int n, width, n_pages, max_rows;
  const int32_t *ctx_len, *n_new;
  int32_t *table, *stack;
  const int32_t *n_free;
  int32_t *new_len, *n_free_out, *cu_rows, *refused;
  int64_t *slot_map;
  int32_t *positions;
};

struct Sum3 {
  long long need, rows, gone;                         // (4096 lengths of 2^24 pages: up to 2^36)
};
__device__ __forceinline__ Sum3 add3(const Sum3 &a, const Sum3 &b) {
  return Sum3{a.need + b.need, a.rows + b.rows, a.gone + b.gone};
}
// exclusive prefix of x over the block's threads; total gets the sum
__device__ __forceinline__ Sum3 block_scan(Sum3 x, Sum3 *warp_tot, Sum3 &total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  Sum3 inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    Sum3 t;
    t.need = __shfl_up_sync(0xffffffffu, inc.need, o);
    t.rows = __shfl_up_sync(0xffffffffu, inc.rows, o);
    t.gone = __shfl_up_sync(0xffffffffu, inc.gone, o);
    if (lane >= o) inc = add3(inc, t);
  }
  __syncthreads();                                    // warp_tot may be in use by an earlier scan
  if (lane == 31) warp_tot[w] = inc;
  __syncthreads();
  Sum3 before{0, 0, 0};
  total = Sum3{0, 0, 0};
#pragma unroll
  for (int i = 0; i < PP_THREADS / 32; ++i) {
    if (i == w) before = total;
    total = add3(total, warp_tot[i]);
  }
  return Sum3{before.need + inc.need - x.need, before.rows + inc.rows - x.rows, before.gone + inc.gone - x.gone};
}

// largest i in [0, n) with pre[i] <= x (pre[0] = 0 <= x, rising)
__device__ __forceinline__ int find_pre(const int *pre, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if (pre[m] <= x) lo = m;
    else hi = m - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(PP_THREADS) k_page_plan(const PlanArgs a) {
  extern __shared__ int pp_smem[];
  __shared__ Sum3 warp_tot[PP_THREADS / 32];
  int *s_need = pp_smem, *s_rows = s_need + a.n + 1, *s_gone = s_rows + a.n + 1, *s_len = s_gone + a.n + 1,
      *s_new = s_len + a.n;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const int ipt = (a.n + PP_THREADS - 1) / PP_THREADS;
  const long long cap = (long long)a.width * KV_PAGE;

  Sum3 mine{0, 0, 0};
  unsigned bad = 0;                                   // bit i: request tid * ipt + i needs too wide a table
  int len[PP_IPT], to[PP_IPT];
#pragma unroll
  for (int i = 0; i < PP_IPT; ++i) {
    const int b = tid * ipt + i;
    len[i] = to[i] = 0;
    if (i >= ipt || b >= a.n) continue;
    const long long l = max(0ll, min((long long)a.ctx_len[b], cap));
    long long t = max(0ll, l + a.n_new[b]);
    if (t > cap) {
      bad |= 1u << i;
      t = l;
    }
    len[i] = (int)l;
    to[i] = (int)t;
    const int op = (int)((l + KV_PAGE - 1) / KV_PAGE), np = (int)((t + KV_PAGE - 1) / KV_PAGE);
    mine = add3(mine, Sum3{max(0, np - op), max(0ll, t - l), max(0, op - np)});
  }
  Sum3 total;
  Sum3 pre = block_scan(mine, warp_tot, total);
  const int n_free = max(0, min(a.n_free[0], a.n_pages));
  const int have = (int)min((long long)a.n_pages, n_free + total.gone);
  if (total.need > have || total.rows > a.max_rows) {  // uniform: some request is refused
    Sum3 run = pre, kept{0, 0, 0};
#pragma unroll
    for (int i = 0; i < PP_IPT; ++i) {
      const int b = tid * ipt + i;
      if (i >= ipt || b >= a.n) continue;
      const int op = (len[i] + KV_PAGE - 1) / KV_PAGE, np = (to[i] + KV_PAGE - 1) / KV_PAGE;
      const int need = max(0, np - op), rows = max(0, to[i] - len[i]);
      run.need += need;
      run.rows += rows;
      if ((need && run.need > have) || (rows && run.rows > a.max_rows)) {
        bad |= 1u << i;
        to[i] = len[i];
      } else {
        kept = add3(kept, Sum3{need, rows, max(0, op - np)});
      }
    }
    pre = block_scan(kept, warp_tot, total);
  }
#pragma unroll
  for (int i = 0; i < PP_IPT; ++i) {
    const int b = tid * ipt + i;
    if (i >= ipt || b >= a.n) continue;
    s_need[b] = (int)pre.need;
    s_rows[b] = (int)pre.rows;
    s_gone[b] = (int)min(pre.gone, 1ll << 30);        // only the first n_pages <= 2^24 are looked up
    s_len[b] = len[i];
    s_new[b] = to[i];
    const int op = (len[i] + KV_PAGE - 1) / KV_PAGE, np = (to[i] + KV_PAGE - 1) / KV_PAGE;
    pre = add3(pre, Sum3{max(0, np - op), max(0, to[i] - len[i]), max(0, op - np)});
    if (blockIdx.x == 0) {
      a.new_len[b] = to[i];
      a.refused[b] = (bad >> i) & 1;
      a.cu_rows[b] = s_rows[b];
    }
  }
  if (tid == 0) {
    s_need[a.n] = (int)total.need;
    s_rows[a.n] = (int)total.rows;
    s_gone[a.n] = (int)min(total.gone, 1ll << 30);
    if (blockIdx.x == 0) {
      a.cu_rows[a.n] = (int)total.rows;
      a.n_free_out[0] = have - (int)total.need;
    }
  }
  __syncthreads();
  // page of the j-th grant: the top of the stack is the last page given back
  auto granted = [&](int j) {
    const int at = have - 1 - j;
    if (at < n_free) return a.stack[at];
    const int x = at - n_free, b = find_pre(s_gone, a.n, x);
    return a.table[(size_t)b * a.width + (s_new[b] + KV_PAGE - 1) / KV_PAGE + x - s_gone[b]];
  };
  const int t0 = blockIdx.x * PP_THREADS + tid, step = gridDim.x * PP_THREADS;
  for (int j = t0; j < s_need[a.n]; j += step) {
    const int b = find_pre(s_need, a.n, j);
    a.table[(size_t)b * a.width + (s_len[b] + KV_PAGE - 1) / KV_PAGE + j - s_need[b]] = granted(j);
  }
  for (int x = t0; x < have - n_free; x += step) {
    const int b = find_pre(s_gone, a.n, x);
    a.stack[n_free + x] = a.table[(size_t)b * a.width + (s_new[b] + KV_PAGE - 1) / KV_PAGE + x - s_gone[b]];
  }
  for (uint32_t u = t0; u < (uint32_t)a.max_rows; u += step) {     // (the last step may pass 2^31)
    const int r = (int)u;
    int64_t slot = -1;
    int pos = 0;
    if (r < s_rows[a.n]) {
      const int b = find_pre(s_rows, a.n, r);
      pos = s_len[b] + (r - s_rows[b]);
      const int i = pos / KV_PAGE, op = (s_len[b] + KV_PAGE - 1) / KV_PAGE;
      const int page = i < op ? a.table[(size_t)b * a.width + i] : granted(s_need[b] + i - op);
      slot = (int64_t)page * KV_PAGE + pos % KV_PAGE;
    }
    a.slot_map[r] = slot;
    a.positions[r] = pos;
  }
}

// ---------------------------------------------------------------- quantised append
// One CTA of (window of rows, kv head, K or V) walks the runs that begin in its window: a run is the
// consecutive rows of one page, so a page has one writer. Per run: the rows are read once into
// registers; the largest finite |x| gives the scale 2^e; the values are scaled (exact), rounded to e4m3
// once and stored. A page that grows its scale has its kept rows rounded again. V goes through a
// shared tile, since its pages are transposed: a thread holds neighbouring tokens of its dims, so that
// the tile is written in words of four tokens.
//
// Bound by latency for a few rows (8 x 16 rows of 8 x 128 take 7.7 us: slots, then rows and scale, then stores. Rows wait
// for the slots because a thread's registers go by the offset in the page, not because their addresses need them)
// and by instructions for many (8 x 4096 rows: 42.0 us, 4.8 TB/s), so the maximum is taken on pairs, bytes are
// turned with permutes and a whole page of V is copied 16 bytes at a time (59.7 us without these). Six CTAs
// per SM are asked for (44.5 us with five). A warp looks for a window's next run in 64 slots at once: row by
// row, 7849 rows of 4 x 128 took 34.8 us, now 16.2.
// The slots of a run are found by every warp for itself (a run whose slots rise by one, which is what a
// plan makes, needs no barrier); only two barriers are left, around the CTA's maximum and V's tile.
constexpr int KA_THREADS = 256;
constexpr int KV8_CTAS = 152 * 8;                     // CTAs that a call is cut into before its windows grow: a wave of the
                                                      // six per SM that fit, and a third of one

template <typename T>
struct AppendArgs {
  int rows, window, nkv, n_pages;
  const T *k, *v;
  int64_t ks, vs;
  const int64_t *slot;
  uint8_t *kp, *vp;
  float *kscale, *vscale;
};

// smallest e >= KV8_MIN_EXP with amax <= 448 * 2^e = 1.75 * 2^(e + 8), from amax's own bits
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, KV8_MIN_EXP);
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The largest |x| of 16 bytes, NaN left out; and with infinities left out too.
template <typename T>
__device__ __forceinline__ float largest(const uint4 &q) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if constexpr (sizeof(T) == 4)
    return fmaxf(fmaxf(fabsf(__uint_as_float(w[0])), fabsf(__uint_as_float(w[1]))),
                 fmaxf(fabsf(__uint_as_float(w[2])), fabsf(__uint_as_float(w[3]))));
  __nv_bfloat162 m = __habs2(*(const __nv_bfloat162 *)&w[0]);
#pragma unroll
  for (int j = 1; j < 4; ++j) m = __hmax2(m, __habs2(*(const __nv_bfloat162 *)&w[j]));
  return fmaxf(__low2float(m), __high2float(m));
}
template <typename T>
__device__ __forceinline__ float largest_finite(const uint4 &q) {
  const T *t = (const T *)&q;
  float big = 0.f;
#pragma unroll
  for (int j = 0; j < (int)(16 / sizeof(T)); ++j) {
    const float x = fabsf(to_f(t[j]));
    if (x <= 3.402823466e38f) big = fmaxf(big, x);
  }
  return big;
}

// four e4m3 bytes times a factor, rounded again
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  const float2 a = e4m3x2_to_f32(w), b = e4m3x2_to_f32(w >> 16);
  return f32_to_e4m3x2(a.x * f, a.y * f) | f32_to_e4m3x2(b.x * f, b.y * f) << 16;
}

template <typename T, int HD>
__global__ void __launch_bounds__(KA_THREADS, 6) k_kv8_append(const AppendArgs<T> a) {
  constexpr int V = 16 / sizeof(T);                   // values of a 16-byte load
  constexpr int TPR = HD / V;                         // threads of a row
  constexpr int NP = KV_PAGE * TPR / KA_THREADS;      // neighbouring rows of a thread
  __shared__ int owner[KV_PAGE];                      // row that stays at each offset, -1: none
  __shared__ int s_end;
  __shared__ float s_max[KA_THREADS / 32];
  __shared__ __align__(16) uint32_t tile[HD * (KV_PAGE / 4)];   // word w of dim d at w ^ (d / 8 & 15)
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, h = blockIdx.y;
  const bool isv = blockIdx.z != 0;
  const T *src = isv ? a.v : a.k;
  const int64_t stride = isv ? a.vs : a.ks;
  const int64_t n_slots = (int64_t)a.n_pages * KV_PAGE;
  auto slot_of = [&](int r) {                         // -1: a skipped row, or none
    const int64_t s = r >= 0 && r < a.rows ? a.slot[r] : -1;
    return s < n_slots && s >= 0 ? s : -1;
  };
  const int w0 = blockIdx.x * a.window, w1 = min(w0 + a.window, a.rows);
  auto page_of = [&](int64_t x) { return x < 0 ? -1 : (int)(x / KV_PAGE); };
  for (int i = w0; i < w1;) {                         // uniform: all warps read the same slots
    // the run: slots s0, s0 + 1, .. as a rule
    const int64_t s1 = slot_of(i + lane), s2 = slot_of(i + 32 + lane);
    const int before = page_of(slot_of(i - 1));
    const int64_t s0 = __shfl_sync(0xffffffffu, s1, 0);
    const int page = page_of(s0);
    if (page < 0 || page == before) {                 // skipped, or of a run begun before: on to the row that begins one
      const int p1 = page_of(s1), p2 = page_of(s2), last = __shfl_sync(0xffffffffu, p1, 31);
      int b1 = __shfl_up_sync(0xffffffffu, p1, 1), b2 = __shfl_up_sync(0xffffffffu, p2, 1);
      if (lane == 0) b1 = before, b2 = last;
      const uint64_t begins = (uint64_t)__ballot_sync(0xffffffffu, p2 >= 0 && p2 != b2) << 32 |
                              __ballot_sync(0xffffffffu, p1 >= 0 && p1 != b1);
      if (!begins) break;                             // (a window has 64 rows at most)
      i += __ffsll((long long)begins) - 1;
      continue;
    }
    const uint64_t rising = (uint64_t)__ballot_sync(0xffffffffu, s2 == s0 + 32 + lane && s2 / KV_PAGE == page) << 32 |
                            __ballot_sync(0xffffffffu, s1 == s0 + lane && s1 / KV_PAGE == page);
    const int first = (int)(s0 % KV_PAGE), len = ~rising ? __ffsll(~rising) - 1 : 64;
    const int64_t after = slot_of(i + len);
    const bool plain = after < 0 || (int)(after / KV_PAGE) != page;
    int end = i + len;
    uint64_t owned;
    if (plain) {
      owned = (len == 64 ? ~0ull : (1ull << len) - 1) << first;
    } else {                                          // slots in any order, some of them twice: the last row stays
      __syncthreads();
      if (tid < KV_PAGE) owner[tid] = -1;
      if (tid == 0) s_end = a.rows;
      end = a.rows;
      __syncthreads();
      for (int r = i; r < end; r += KA_THREADS) {
        const int rr = r + tid;
        const int64_t s = slot_of(rr);
        const bool in = s >= 0 && (int)(s / KV_PAGE) == page;
        if (rr < a.rows && !in) atomicMin(&s_end, rr);
        __syncthreads();
        end = s_end;
        if (rr < end) atomicMax(&owner[(int)(s % KV_PAGE)], rr);
        __syncthreads();
      }
      owned = (uint64_t)__ballot_sync(0xffffffffu, owner[32 + lane] >= 0) << 32 |
              __ballot_sync(0xffffffffu, owner[lane] >= 0);
    }
    // the CTA's rows of the page, one 16-byte piece per thread and row
    const int c = tid % TPR, off0 = tid / TPR * NP;
    const uint32_t mine = (uint32_t)(owned >> off0);   // bit p: row p of the thread
    uint4 q[NP];
    float big = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int off = off0 + p, row = plain ? i + off - first : owner[off];
      q[p] = mine >> p & 1 ? *(const uint4 *)(src + (int64_t)row * stride + (int64_t)h * HD + c * V) : make_uint4(0, 0, 0, 0);
    }
    float *sp = (isv ? a.vscale : a.kscale) + (size_t)page * a.nkv + h;
    const bool fresh = owned & 1;
    const float old = fresh ? 0.f : *sp;
#pragma unroll
    for (int p = 0; p < NP; ++p) big = fmaxf(big, largest<T>(q[p]));
    if (!(big <= 3.402823466e38f)) {                  // infinities and NaN have no say
      big = 0.f;
#pragma unroll
      for (int p = 0; p < NP; ++p) big = fmaxf(big, largest_finite<T>(q[p]));
    }
    big = warp_max(big);
    if (lane == 0) s_max[tid >> 5] = big;
    __syncthreads();                                  // (and every thread has read *sp)
#pragma unroll
    for (int j = 0; j < KA_THREADS / 32; ++j) big = fmaxf(big, s_max[j]);
    float scale = pow2f(scale_exp(big)), again = 1.f;
    if (old >= scale) scale = old;
    else if (!fresh) again = old / scale;             // powers of two: exact
    const int last = 63 - __clzll(owned);
    const uint64_t kept = fresh || again == 1.f ? 0 : (last == 63 ? ~0ull : (2ull << last) - 1) & ~owned;
    const float inv = 1.f / scale;                    // exact
    if (tid == 0) *sp = scale;
    uint8_t *blk = (isv ? a.vp : a.kp) + kv8_block(page, h, a.nkv, HD);
    uint32_t w[NP][V / 4];                            // four dims of a row each
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const T *t = (const T *)&q[p];
#pragma unroll
      for (int j = 0; j < V; j += 4)
        w[p][j / 4] = f32_to_e4m3x2(to_f(t[j]) * inv, to_f(t[j + 1]) * inv) |
                      f32_to_e4m3x2(to_f(t[j + 2]) * inv, to_f(t[j + 3]) * inv) << 16;
    }
    if (!isv) {
      const uint32_t keep = (uint32_t)(kept >> off0);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int off = off0 + p;
        uint8_t *dst = blk + off * HD + c * V;
        if (keep >> p & 1) {
#pragma unroll
          for (int j = 0; j < V / 4; ++j) w[p][j] = rescale4(*(const uint32_t *)(dst + 4 * j), again);
        } else if (!(mine >> p & 1)) {
          continue;
        }
        if constexpr (V == 8) *(uint2 *)dst = make_uint2(w[p][0], w[p][1]);
        else *(uint32_t *)dst = w[p][0];
      }
      __syncthreads();                                // s_max and owner are free again
    } else {
      auto at = [&](int d, int off) { return &tile[d * (KV_PAGE / 4) + ((off >> 2) ^ (d >> 3 & 15))]; };
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const int d = c * V + j;
        if constexpr (NP >= 4) {
#pragma unroll
          for (int p = 0; p < NP; p += 4) {           // four tokens' four dims turned into four dims' four tokens
            const uint32_t x0 = w[p][j / 4], x1 = w[p + 1][j / 4], x2 = w[p + 2][j / 4], x3 = w[p + 3][j / 4];
            const uint32_t a0 = __byte_perm(x0, x1, 0x5140), a1 = __byte_perm(x2, x3, 0x5140);
            const uint32_t b0 = __byte_perm(x0, x1, 0x7362), b1 = __byte_perm(x2, x3, 0x7362);
            *at(d, off0 + p) = __byte_perm(a0, a1, 0x5410);
            *at(d + 1, off0 + p) = __byte_perm(a0, a1, 0x7632);
            *at(d + 2, off0 + p) = __byte_perm(b0, b1, 0x5410);
            *at(d + 3, off0 + p) = __byte_perm(b0, b1, 0x7632);
          }
        } else {
          const uint32_t a = __byte_perm(w[0][j / 4], w[1][j / 4], 0x5140), b = __byte_perm(w[0][j / 4], w[1][j / 4], 0x7362);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *((uint16_t *)at(d + k, off0) + (off0 >> 1 & 1)) = (uint16_t)((k < 2 ? a : b) >> 16 * (k & 1));
        }
      }
      __syncthreads();
      if (!~owned) {                                  // a whole page: 16 tokens of a dim at a time
#pragma unroll
        for (int t = tid; t < HD * (KV_PAGE / 16); t += KA_THREADS) {
          const int d = t / (KV_PAGE / 16), o = t % (KV_PAGE / 16) * 4, x = d >> 3 & 15;
          const uint32_t *row = &tile[d * (KV_PAGE / 4)];
          *(uint4 *)(blk + 16 * t) = make_uint4(row[o ^ x], row[(o + 1) ^ x], row[(o + 2) ^ x], row[(o + 3) ^ x]);
        }
      } else {
#pragma unroll 4
        for (int t = tid; t < HD * (KV_PAGE / 4); t += KA_THREADS) {
          const int d = t / (KV_PAGE / 4), o = t % (KV_PAGE / 4);
          const uint32_t mo = (uint32_t)(owned >> (4 * o)) & 15, mk = (uint32_t)(kept >> (4 * o)) & 15;
          if (!(mo | mk)) continue;
          uint32_t *dst = (uint32_t *)(blk + 4 * t);
          uint32_t x = tile[d * (KV_PAGE / 4) + (o ^ (d >> 3 & 15))];
          if (mo != 15) {                               // keep or round anew the word's other bytes
            const uint32_t was = *dst, re = mk ? rescale4(was, again) : was;
            uint32_t bo = 0, bk = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              bo |= (mo >> j & 1) ? 0xffu << 8 * j : 0;
              bk |= (mk >> j & 1) ? 0xffu << 8 * j : 0;
            }
            x = (x & bo) | (re & bk) | (was & ~(bo | bk));
          }
          *dst = x;
        }
      }
      __syncthreads();                                // the tile, s_max and owner are free again
    }
    i = end;
  }
}

template <typename T>
cudaError_t launch_append(const dflash_kv8_cache *c, int rows, const void *k, int64_t ks, const void *v, int64_t vs,
                          const int64_t *slot, cudaStream_t s) {
  AppendArgs<T> a{rows, 1, c->n_kv_heads, c->n_pages, (const T *)k, (const T *)v, ks, vs, slot,
                  (uint8_t *)c->k_pages, (uint8_t *)c->v_pages, c->k_scale, c->v_scale};
  // Rows of a window: one, so that every row of a few may start a page of its own at once, up to a
  // page's worth when that leaves KV8_CTAS CTAs (half of it, for twice as many: 11.8 against 9.8 us at 33 x 8
  // rows of 8 x 128, 8.4 against 5.9 us at 29 x 48 .. 96 of 1 x 64, 13.4 against 16.7 at 7849 rows of 4 x 128).
  const long ctas = (long)rows * c->n_kv_heads * 2;
  a.window = (int)(ctas / KV8_CTAS);
  a.window = a.window < 1 ? 1 : a.window > KV_PAGE ? KV_PAGE : a.window;
  const dim3 g((rows + a.window - 1) / a.window, c->n_kv_heads, 2), b(KA_THREADS);
  return c->head_dim == 128 ? launch_pdl(k_kv8_append<T, 128>, g, b, 0, s, a)
                            : launch_pdl(k_kv8_append<T, 64>, g, b, 0, s, a);
}

// ---------------------------------------------------------------- inspection
__global__ void __launch_bounds__(256) k_kv8_read(int rows, int nkv, int hd, int n_pages, const int64_t *slot,
                                                  const uint8_t *kp, const uint8_t *vp, const float *ks,
                                                  const float *vs, float *ko, float *vo) {
  pdl_trigger();
  pdl_wait();
  const size_t per = (size_t)nkv * hd, n = (size_t)rows * per;
  for (size_t i = blockIdx.x * 256ull + threadIdx.x; i < n; i += gridDim.x * 256ull) {
    const size_t r = i / per;
    const int h = (int)(i % per) / hd, d = (int)(i % hd);
    const int64_t s = slot[r];
    float k = 0.f, v = 0.f;
    if (s >= 0 && s < (int64_t)n_pages * KV_PAGE) {
      const int page = (int)(s / KV_PAGE), off = (int)(s % KV_PAGE);
      const size_t blk = kv8_block(page, h, nkv, hd), sc = (size_t)page * nkv + h;
      k = e4m3x2_to_f32(kp[blk + (size_t)off * hd + d]).x * ks[sc];
      v = e4m3x2_to_f32(vp[blk + (size_t)d * KV_PAGE + off]).x * vs[sc];
    }
    ko[i] = k;
    vo[i] = v;
  }
}

}  // namespace dflash

using namespace dflash;

extern "C" dflash_status dflash_page_plan(void *stream, int32_t n_req, int32_t max_blocks, int32_t n_pages,
                                          int32_t max_rows, const int32_t *ctx_len, const int32_t *n_new,
                                          int32_t *block_table, int32_t *free_list, const int32_t *n_free,
                                          int32_t *new_len, int32_t *n_free_out, int32_t *cu_rows, int32_t *refused,
                                          int64_t *slot_map, int32_t *positions) {
  if (n_req < 1 || n_req > KV8_MAX_REQ || max_blocks < 1 || max_blocks > (1 << 24) || n_pages < 1 ||
      n_pages > (1 << 24) || max_rows < 0)
    return DFLASH_ERR_INVALID_ARG;
  if (!ctx_len || !n_new || !block_table || !free_list || !n_free || !new_len || !n_free_out || !cu_rows || !refused ||
      (max_rows && (!slot_map || !positions)))
    return DFLASH_ERR_INVALID_ARG;
  const void *ins[] = {ctx_len, n_new, n_free, block_table, free_list};
  const void *outs[] = {new_len, n_free_out, cu_rows, refused, slot_map, positions};
  for (const void *o : outs)
    for (const void *x : ins)
      if (o && o == x) return DFLASH_ERR_INVALID_ARG;
  for (const void *x : ins)
    if (!aligned(x, 4)) return DFLASH_ERR_INVALID_ARG;
  for (const void *o : outs)
    if (!aligned(o, o == slot_map ? 8 : 4)) return DFLASH_ERR_INVALID_ARG;
  const PlanArgs a{n_req, max_blocks, n_pages, max_rows, ctx_len, n_new, block_table, free_list, n_free,
                   new_len, n_free_out, cu_rows, refused, slot_map, positions};
  const size_t sm = (size_t)(5 * n_req + 3) * sizeof(int);
  const cudaError_t at = cudaFuncSetAttribute(k_page_plan, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              (5 * KV8_MAX_REQ + 3) * (int)sizeof(int));
  if (at != cudaSuccess) return DFLASH_ERR_CUDA;
  long ctas = ((long)max_rows + 4 * PP_THREADS - 1) / (4 * PP_THREADS);
  ctas = ctas < 1 ? 1 : ctas > 152 ? 152 : ctas;
  const cudaError_t e = launch_pdl(k_page_plan, dim3((unsigned)ctas), dim3(PP_THREADS), sm, (cudaStream_t)stream, a);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

extern "C" dflash_status dflash_kv8_append(void *stream, const dflash_kv8_cache *cache, int32_t rows,
                                           dflash_dtype dtype, const void *k, int64_t k_stride, const void *v,
                                           int64_t v_stride, const int64_t *slot_map) {
  if (!kv8_cache_ok(cache) || rows < 0 || (dtype != DFLASH_F32 && dtype != DFLASH_BF16)) return DFLASH_ERR_INVALID_ARG;
  const int64_t w = (int64_t)cache->n_kv_heads * cache->head_dim, V = 16 / dtype_bytes(dtype);
  if (k_stride < w || v_stride < w || k_stride % V || v_stride % V) return DFLASH_ERR_INVALID_ARG;
  if (rows == 0) return DFLASH_OK;
  if (!k || !v || !slot_map || !aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 8)) return DFLASH_ERR_INVALID_ARG;
  const cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = dtype == DFLASH_BF16 ? launch_append<bf16>(cache, rows, k, k_stride, v, v_stride, slot_map, s)
                                             : launch_append<float>(cache, rows, k, k_stride, v, v_stride, slot_map, s);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

extern "C" dflash_status dflash_kv8_read(void *stream, const dflash_kv8_cache *cache, int32_t rows,
                                         const int64_t *slot_map, float *k_out, float *v_out) {
  if (!kv8_cache_ok(cache) || rows < 0) return DFLASH_ERR_INVALID_ARG;
  if (rows == 0) return DFLASH_OK;
  if (!slot_map || !k_out || !v_out || !aligned(slot_map, 8) || !aligned(k_out, 4) || !aligned(v_out, 4))
    return DFLASH_ERR_INVALID_ARG;
  const long n = ((long)rows * cache->n_kv_heads * cache->head_dim + 255) / 256;
  const cudaError_t e = launch_pdl(k_kv8_read, dim3((unsigned)(n < 152 * 16 ? n : 152 * 16)), dim3(256), 0,
                                   (cudaStream_t)stream, (int)rows, (int)cache->n_kv_heads, (int)cache->head_dim,
                                   (int)cache->n_pages, slot_map, (const uint8_t *)cache->k_pages,
                                   (const uint8_t *)cache->v_pages, (const float *)cache->k_scale,
                                   (const float *)cache->v_scale, k_out, v_out);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
