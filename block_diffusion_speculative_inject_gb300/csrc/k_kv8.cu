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
  long long need, rows;
  int gone;
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
  const int have = min(a.n_pages, n_free + total.gone);
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
    s_gone[b] = pre.gone;
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
    s_gone[a.n] = total.gone;
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
  for (int r = t0; r < a.max_rows; r += step) {
    int64_t slot = -1;
    int pos = 0;
    if (r < s_rows[a.n]) {
      const int b = find_pre(s_rows, a.n, r);
      pos = s_len[b] + r - s_rows[b];
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
// consecutive rows of one page, so a page has one writer. Per run: the largest finite |x| gives
// the scale 2^e; the rows are read once into registers, scaled (exact), rounded to e4m3 once and
// stored. A page that grows its scale has its kept rows rounded again. V goes through a shared
// tile, since its pages are transposed.
constexpr int KA_THREADS = 256;

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

__device__ __forceinline__ float finite_abs(float x) {
  x = fabsf(x);
  return x <= 3.402823466e38f ? x : 0.f;              // infinities and NaN have no say
}

// four e4m3 bytes times a factor, rounded again
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  const float2 a = e4m3x2_to_f32(w), b = e4m3x2_to_f32(w >> 16);
  return f32_to_e4m3x2(a.x * f, a.y * f) | f32_to_e4m3x2(b.x * f, b.y * f) << 16;
}

template <typename T, int HD>
__global__ void __launch_bounds__(KA_THREADS) k_kv8_append(const AppendArgs<T> a) {
  constexpr int V = 16 / sizeof(T);                   // values of a 16-byte load
  constexpr int TPR = HD / V;                         // threads of a row
  constexpr int RPP = KA_THREADS / TPR;               // rows of a pass
  constexpr int NP = KV_PAGE / RPP;                   // passes of a page
  __shared__ int owner[KV_PAGE];                      // row that stays at each offset, -1: none
  __shared__ int s_end;
  __shared__ float s_max[KA_THREADS / 32];
  __shared__ __align__(16) uint8_t tile[HD][KV_PAGE + 4];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, h = blockIdx.y;
  const bool isv = blockIdx.z != 0;
  const T *src = isv ? a.v : a.k;
  const int64_t stride = isv ? a.vs : a.ks;
  const int64_t n_slots = (int64_t)a.n_pages * KV_PAGE;
  auto page_of = [&](int r) {                         // -1: a skipped row
    const int64_t s = a.slot[r];
    return s < 0 || s >= n_slots ? -1 : (int)(s / KV_PAGE);
  };
  const int w0 = blockIdx.x * a.window, w1 = min(w0 + a.window, a.rows);
  int i = w0, before = -2;                            // page of the last row that was not skipped
  while (i < w1) {
    const int page = page_of(i);                      // uniform: all threads read the same slot
    if (page < 0) {
      ++i;
      continue;
    }
    if (before == -2) {                               // the window's first row: look back past its start
      before = -1;
      for (int r = i - 1; r >= 0 && before < 0; --r) before = page_of(r);
    }
    if (page == before) {                             // a run that an earlier row began
      ++i;
      continue;
    }
    before = page;
    // the run's rows, and the row that stays at each offset
    __syncthreads();
    if (tid < KV_PAGE) owner[tid] = -1;
    if (tid == 0) s_end = a.rows;
    __syncthreads();
    int end = a.rows;
    for (int r = i; r < end; r += KA_THREADS) {
      const int rr = r + tid;
      if (rr < a.rows) {
        const int p = page_of(rr);
        if (p >= 0 && p != page) atomicMin(&s_end, rr);
      }
      __syncthreads();
      end = s_end;
      if (rr < end && page_of(rr) == page) atomicMax(&owner[(int)(a.slot[rr] % KV_PAGE)], rr);
      __syncthreads();
    }
    uint64_t owned = 0;
    {
      const uint32_t lo = __ballot_sync(0xffffffffu, owner[tid & 31] >= 0);
      const uint32_t hi = __ballot_sync(0xffffffffu, owner[32 + (tid & 31)] >= 0);
      owned = (uint64_t)hi << 32 | lo;
    }
    // rows of the page, one 16-byte piece per thread and pass
    const int c = tid % TPR, rp = tid / TPR;
    float x[NP][V];
    float big = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int row = owner[p * RPP + rp];
      if (row >= 0) {
        const T *g = src + (int64_t)row * stride + (int64_t)h * HD + c * V;
        const uint4 q = *(const uint4 *)g;
        const T *t = (const T *)&q;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          x[p][j] = to_f(t[j]);
          big = fmaxf(big, finite_abs(x[p][j]));
        }
      }
    }
    big = warp_max(big);
    if ((tid & 31) == 0) s_max[tid >> 5] = big;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < KA_THREADS / 32; ++j) big = fmaxf(big, s_max[j]);
    float *sp = (isv ? a.vscale : a.kscale) + (size_t)page * a.nkv + h;
    float scale = pow2f(scale_exp(big)), again = 1.f;
    const bool fresh = owned & 1;
    if (!fresh) {
      const float old = *sp;
      if (old >= scale) scale = old;
      else again = old / scale;                       // powers of two: exact
    }
    const int last = 63 - __clzll(owned);
    const uint64_t below = last == 63 ? ~0ull : (2ull << last) - 1;
    const uint64_t kept = fresh || again == 1.f ? 0 : below & ~owned;
    const float inv = 1.f / scale;                    // exact
    __syncthreads();                                  // every thread has read *sp
    if (tid == 0) *sp = scale;
    uint8_t *blk = (isv ? a.vp : a.kp) + kv8_block(page, h, a.nkv, HD);
    if (!isv) {
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int off = p * RPP + rp;
        uint8_t *dst = blk + off * HD + c * V;
        uint32_t w[V / 4];
        if (owned >> off & 1) {
#pragma unroll
          for (int j = 0; j < V; j += 4)
            w[j / 4] = f32_to_e4m3x2(x[p][j] * inv, x[p][j + 1] * inv) |
                       f32_to_e4m3x2(x[p][j + 2] * inv, x[p][j + 3] * inv) << 16;
        } else if (kept >> off & 1) {
#pragma unroll
          for (int j = 0; j < V; j += 4) w[j / 4] = rescale4(*(const uint32_t *)(dst + j), again);
        } else {
          continue;
        }
        if constexpr (V == 8) *(uint2 *)dst = make_uint2(w[0], w[1]);
        else *(uint32_t *)dst = w[0];
      }
    } else {
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int off = p * RPP + rp;
        if (!(owned >> off & 1)) continue;
#pragma unroll
        for (int j = 0; j < V; j += 2) {
          const uint32_t w = f32_to_e4m3x2(x[p][j] * inv, x[p][j + 1] * inv);
          tile[c * V + j][off] = (uint8_t)w;
          tile[c * V + j + 1][off] = (uint8_t)(w >> 8);
        }
      }
      __syncthreads();
      for (int t = tid; t < HD * (KV_PAGE / 4); t += KA_THREADS) {
        const int d = t / (KV_PAGE / 4), o4 = t % (KV_PAGE / 4) * 4;
        const uint32_t mo = (uint32_t)(owned >> o4) & 15, mk = (uint32_t)(kept >> o4) & 15;
        if (!(mo | mk)) continue;
        uint32_t *dst = (uint32_t *)(blk + d * KV_PAGE + o4);
        uint32_t w = *(const uint32_t *)&tile[d][o4];
        if (mo != 15) {                               // keep or round anew the word's other bytes
          const uint32_t was = *dst, re = mk ? rescale4(was, again) : was;
          uint32_t bo = 0, bk = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            bo |= (mo >> j & 1) ? 0xffu << 8 * j : 0;
            bk |= (mk >> j & 1) ? 0xffu << 8 * j : 0;
          }
          w = (w & bo) | (re & bk) | (was & ~(bo | bk));
        }
        *dst = w;
      }
    }
    i = min(end, w1);
  }
}

template <typename T>
cudaError_t launch_append(const dflash_kv8_cache *c, int rows, const void *k, int64_t ks, const void *v, int64_t vs,
                          const int64_t *slot, cudaStream_t s) {
  AppendArgs<T> a{rows, 1, c->n_kv_heads, c->n_pages, (const T *)k, (const T *)v, ks, vs, slot,
                  (uint8_t *)c->k_pages, (uint8_t *)c->v_pages, c->k_scale, c->v_scale};
  // Rows of a window: one, so that every row of a few may start a page of its own at once, up to a
  // page's worth when there are CTAs enough for about two waves of 8 per SM without.
  const long ctas = (long)rows * c->n_kv_heads * 2;
  a.window = (int)(ctas / (152 * 8 * 2));
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
