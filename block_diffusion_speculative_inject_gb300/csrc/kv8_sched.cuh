// The work of one attention call over the 8-bit cache, cut into equal pieces on the GPU.
//
// An item is (request, tile of query tokens, kv head); its units are the U-token stretches of the
// context that its rows may see. All items, in the order requests > tiles > heads, each as C + its units
// long (C: what its start and end cost a worker), form one line that is cut into equal chunks, one per
// worker (longer ones where an item would fall into too many pieces). A worker thus owns at most two pieces
// of items that others also work on (its first and its last), whose partial results go to the workspace
// and are merged by k_kv8_combine. An item whose first C fall to a worker without any of its units begins
// with the next worker. Every worker finds its start by itself from the lengths on the GPU: lengths of 32
// requests are summed by a warp, the sums of those groups sit in shared memory, and the lengths inside a
// request have a closed form.
#pragma once
#include "kv8.cuh"

namespace dflash {

constexpr int KV8_GROUPS = KV8_MAX_REQ / 32;
// The longest item is cut into about this many pieces at most, since its merge takes eight of them at a time:
// a token with 8 heads over 65536 tokens of one kv head took 70 us in 1025 pieces, 34 in 64, 26 in 128, 25 in 256;
// one with 2 heads of 64 over 48222 tokens 31, 25, 21 and 24. (The tiles' 152 workers are not held back.)
constexpr int KV8_PIECES = 152;

struct Kv8AttnArgs {
  int n_req, rows, nq, nkv, width, mask, words, n_pages;
  float scale;
  const void *q;
  int64_t q_stride;
  const int32_t *cu_q, *ctx_len, *table;
  const uint32_t *tree;
  void *out;
  float *lse;
  const uint8_t *kp, *vp;
  const float *ks, *vs;
  // workspace: one descriptor per worker, then two partial results per worker
  struct Kv8Desc *desc;
  float *part_o, *part_ml;     // [2 workers][M][hd], [2 workers][M][2] (max in log2 units, sum)
};

// What the merge needs to know of a worker's first piece: 0 pieces unless it continues an item that the worker
// before it began.
struct alignas(16) Kv8Desc {
  int pieces, slot0;           // partial results to merge: slot0, then the first ones of this and the next workers
  int row0, rows, h, pad[3];   // first query row (token) of the tile, its rows (tokens x heads), kv head
};

// sum over i < n of floor((a i + b) / m), for a, b >= 0 (called, not inlined, as what follows: the start of a kernel is
// mostly the fetching of its code)
static __device__ __noinline__ long long floor_sum(long long n, long long m, long long a, long long b) {
  long long s = 0;
  while (n > 0) {
    if (a >= m) s += (n - 1) * n / 2 * (a / m), a %= m;
    if (b >= m) s += n * (b / m), b %= m;
    const long long y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const long long t = m;
    m = a;
    a = t;
  }
  return s;
}

// weight of a causal request's tiles before qt; first: position of its first row
static __device__ __noinline__ long long kv8_before_causal(int U, int C, int tpt, int qt, int first) {
  if (qt == 0) return 0;
  const int t0 = first < 0 ? min(qt, -first / tpt) : 0;          // tiles that see nothing have one unit
  return (long long)qt * C + t0 + floor_sum(qt - t0, U, tpt, first + (long long)(t0 + 1) * tpt + U - 1);
}

struct Kv8Req {
  int n, len, row0;            // rows, context length, first row
};
__device__ __forceinline__ Kv8Req kv8_req(const Kv8AttnArgs &a, int b) {
  Kv8Req r;
  r.row0 = max(0, min(a.cu_q[b], a.rows));
  r.n = max(r.row0, min(a.cu_q[b + 1], a.rows)) - r.row0;
  r.len = (int)max(0ll, min((long long)a.ctx_len[b], (long long)a.width * KV_PAGE));
  return r;
}

// Tokens of a tile, tokens it may see, units: M rows of a tile hold M / group tokens.
template <int U, int M, int C>
struct Kv8Tiles {
  int tpt, nkv, causal;
  __device__ __forceinline__ Kv8Tiles(const Kv8AttnArgs &a)
      : tpt(M / (a.nq / a.nkv)), nkv(a.nkv), causal(a.mask == DFLASH_MASK_CAUSAL) {}
  __device__ __forceinline__ int tiles(const Kv8Req &r) const { return (r.n + tpt - 1) / tpt; }
  // the tokens [0, limit) hold all that some row of the tile sees
  __device__ __forceinline__ int limit(const Kv8Req &r, int qt) const {
    return causal ? max(0, (int)min((long long)r.len, (long long)r.len - r.n + min((long long)(qt + 1) * tpt, (long long)r.n)))
                  : r.len;
  }
  __device__ __forceinline__ int units(const Kv8Req &r, int qt) const { return max(1, (limit(r, qt) + U - 1) / U); }
  // what an item takes on the line: C units for its start and end, then its units
  __device__ __forceinline__ long long weight(const Kv8Req &r, int qt) const { return C + (long long)units(r, qt); }
  __device__ __forceinline__ int longest(const Kv8Req &r) const { return r.n ? units(r, tiles(r) - 1) : 0; }
  // weight of one head's tiles before qt, for qt < tiles
  __device__ __forceinline__ long long before(const Kv8Req &r, int qt) const {
    return causal ? kv8_before_causal(U, C, tpt, qt, r.len - r.n) : qt * weight(r, 0);
  }
  __device__ __forceinline__ long long total(const Kv8Req &r) const {
    const int nt = tiles(r);
    return nt ? nkv * (before(r, nt - 1) + weight(r, nt - 1)) : 0;
  }
};

// A worker's place on the line: the item, its unit range for this worker.
struct Kv8Piece {
  Kv8Req r;
  int b, qt, h;
  int u0, u1, units;           // [u0, u1) of the item's units
  long long left;              // of the worker's stretch after this piece; 0: no more pieces
};

// x / y for 0 <= x, 0 < y: one 32-bit division where both fit
static __device__ __noinline__ long long div_wide(long long x, long long y) { return x / y; }
__device__ __forceinline__ long long div_ll(long long x, long long y) {
  return ((x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : div_wide(x, y);
}

__device__ __forceinline__ long long warp_scan_ll(long long x) {       // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += t;
  }
  return x;
}

// The start of worker `me` of `workers`: false if it has nothing to do. The whole CTA calls it (s_grp is for more
// than 32 requests only); chunk gets a worker's length of the line, item_begin where the first
// piece's item begins. For up to 32 requests every warp sums them up by itself, without a barrier.
template <int U, int M, int C>
__device__ __forceinline__ bool kv8_start(const Kv8AttnArgs &a, long long *s_grp, int me, int workers, Kv8Piece &p,
                                          long long &chunk, long long &item_begin) {
  const Kv8Tiles<U, M, C> tl(a);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int groups = (a.n_req + 31) / 32;
  long long total = 0;
  int longest = 0;                                     // units of the longest item
  __shared__ int s_longest[KV8_GROUPS];
  if (groups > 1) {
    for (int g = warp; g < groups; g += warps) {
      const int b = g * 32 + lane;
      long long t = 0;
      int u = 0;
      if (b < a.n_req) {
        const Kv8Req r = kv8_req(a, b);
        t = tl.total(r);
        u = tl.longest(r);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      u = __reduce_max_sync(0xffffffffu, u);
      if (lane == 0) {
        s_grp[g + 1] = t;
        s_longest[g] = u;
      }
    }
    if (threadIdx.x == 0) s_grp[0] = 0;
    __syncthreads();
    if (warp == 0) {
      long long before = 0;
      for (int g0 = 1; g0 <= groups; g0 += 32) {
        const long long x = warp_scan_ll(g0 + lane <= groups ? s_grp[g0 + lane] : 0);
        if (g0 + lane <= groups) s_grp[g0 + lane] = before + x;
        before += __shfl_sync(0xffffffffu, x, 31);
      }
    }
    __syncthreads();
    total = s_grp[groups];
    for (int g = lane; g < groups; g += 32) longest = max(longest, s_longest[g]);
  }
  Kv8Req r{0, 0, 0};
  long long mine = 0, inc = 0, pos = 0, base = 0;
  int b0 = 0;
  if (groups == 1) {
    if (lane < a.n_req) {
      r = kv8_req(a, lane);
      mine = tl.total(r);
      longest = tl.longest(r);
    }
    inc = warp_scan_ll(mine);
    total = __shfl_sync(0xffffffffu, inc, 31);
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  chunk = max(div_ll(total + workers - 1, workers), (long long)(longest + KV8_PIECES - 1) / KV8_PIECES);
  pos = me * chunk;
  if (pos >= total) return false;
  if (groups > 1) {
    int lo = 0, hi = groups - 1;                       // last group with s_grp <= pos
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (s_grp[m] <= pos) lo = m;
      else hi = m - 1;
    }
    b0 = lo * 32;
    base = s_grp[lo];
    if (b0 + lane < a.n_req) {
      r = kv8_req(a, b0 + lane);
      mine = tl.total(r);
    }
    inc = warp_scan_ll(mine);
  }
  const int who = __ffs(__ballot_sync(0xffffffffu, base + inc > pos)) - 1;     // the request that holds pos
  p.b = b0 + who;
  p.r.n = __shfl_sync(0xffffffffu, r.n, who);
  p.r.len = __shfl_sync(0xffffffffu, r.len, who);
  p.r.row0 = __shfl_sync(0xffffffffu, r.row0, who);
  const long long off = pos - base - __shfl_sync(0xffffffffu, inc - mine, who);
  const long long count = min(chunk, total - pos);
  p.qt = 0;
  if (!tl.causal) {
    p.qt = (int)div_ll(off, tl.weight(p.r, 0) * a.nkv);
  } else {
    int l = 0, h = tl.tiles(p.r) - 1;
    while (l < h) {
      const int m = (l + h + 1) >> 1;
      if (tl.before(p.r, m) * a.nkv <= off) l = m;
      else h = m - 1;
    }
    p.qt = l;
  }
  p.units = tl.units(p.r, p.qt);
  const long long in_tile = off - tl.before(p.r, p.qt) * a.nkv;
  const long long w = C + (long long)p.units;
  p.h = (int)div_ll(in_tile, w);
  const long long x0 = in_tile - p.h * w, x1 = min(w, x0 + count);
  item_begin = pos - x0;
  p.u0 = (int)max(0ll, x0 - C);
  p.u1 = (int)max(0ll, x1 - C);
  p.left = count - (x1 - x0);
  if (p.left <= C) p.left = 0;                         // the next item's units are all the next worker's
  return p.u1 > 0;
}

// The descriptor of worker `me`, whose first piece is p.
template <int U, int M, int C>
__device__ __forceinline__ Kv8Desc kv8_desc(const Kv8AttnArgs &a, const Kv8Piece &p, int me, long long chunk, long long item_begin) {
  Kv8Desc d{0, 0, 0, 0, 0, {0, 0, 0}};
  const long long pos = me * chunk;
  const long long begin = item_begin + C;              // the item's first unit
  if (begin < pos && begin >= pos - chunk) {
    const Kv8Tiles<U, M, C> tl(a);
    d.pieces = (int)div_ll(begin + p.units - 1, chunk) - me + 2;       // up to the worker of the last unit
    d.slot0 = 2 * (me - 1) + (item_begin <= pos - chunk ? 0 : 1);
    d.row0 = p.r.row0 + p.qt * tl.tpt;
    d.rows = min(tl.tpt, p.r.n - p.qt * tl.tpt) * (a.nq / a.nkv);
    d.h = p.h;
  }
  return d;
}

// The next piece of the same worker; p.left > 0.
template <int U, int M, int C>
__device__ __forceinline__ void kv8_next_piece(const Kv8AttnArgs &a, Kv8Piece &p) {
  const Kv8Tiles<U, M, C> tl(a);
  if (++p.h == a.nkv) {
    p.h = 0;
    if (++p.qt == tl.tiles(p.r)) {
      p.qt = 0;
      do {
        if (++p.b >= a.n_req) {                        // (not reached: left counts what there is)
          p.u0 = p.u1 = 0;
          p.left = 0;
          return;
        }
        p.r = kv8_req(a, p.b);
      } while (p.r.n == 0);
    }
    p.units = tl.units(p.r, p.qt);
  }
  p.u0 = 0;
  p.u1 = (int)min((long long)p.units, p.left - C);
  p.left -= C + p.u1;
  if (p.left <= C) p.left = 0;
}

// Which of the 64 tokens of page `page_no` the row of `token` (index among the request's rows) sees,
// apart from whether the page is in the pool.
__device__ __forceinline__ uint64_t kv8_visible(const Kv8AttnArgs &a, const Kv8Req &r, int token, int page_no) {
  const int p0 = page_no * KV_PAGE;
  auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; };   // tokens 0 .. n - 1
  const uint64_t in = below(r.len - p0);
  const int first = r.len - r.n;
  if (a.mask == DFLASH_MASK_NONE) return in;
  if (a.mask == DFLASH_MASK_CAUSAL) return in & below(first + token + 1 - p0);
  // tree: bit i of the page is token p0 + i, bit p0 + i - first of the row's mask
  uint64_t bits = below(first - p0);                   // the context before the rows
  const uint32_t *w = a.tree + (size_t)(r.row0 + token) * a.words;
  const int j0 = p0 - first;                           // mask bit of the page's first token
  const int wd = j0 >> 5, sh = j0 & 31;                // floor division: j0 may be negative
  auto word = [&](int i) { return i >= 0 && i < a.words ? w[i] : 0u; };
  const uint32_t x0 = word(wd), x1 = word(wd + 1), x2 = word(wd + 2);
  bits |= (uint64_t)__funnelshift_r(x0, x1, sh) | (uint64_t)__funnelshift_r(x1, x2, sh) << 32;
  return in & bits;
}

}  // namespace dflash
