// Attention over the 8-bit paged cache (dflash_kv8_attention): the entry point, the kernel for few
// query rows per kv head (and for fp32), and the merge of split contexts.
//
// Few rows (a decoding step, a short block): the cache's bytes bound it, each read once. A worker is
// a warp with its own ring of K and V pages in shared memory, filled by bulk copies that it issues
// itself, so that warps never wait for one another. Per page of 64 tokens, with m16n8k16 products of up to
// 16 query rows (tokens x heads of a kv head):
//   S[16, 64] = Q . K^T      K bytes widened to f16 in registers (exact)
//   P = 2^(S c + log2 s_v - m), S = sum in log2 units, c = scale log2(e) s_k 2^row exponent
//   O[16, hd] += P . V       V bytes likewise, P in f16
// (m16n8k32 on the bytes themselves, with q in two 8-bit parts, was slower: 157 against 129 us.)
// The contraction indices are permuted so that no fragment needs a shuffle and both contractions run
// along 16 contiguous bytes: lane (g, t) of a B fragment holds dims 32 t .. 32 t + 31 of token
// 16 (g >> 1) + 2 j + (g & 1) for K, and tokens 16 t .. 16 t + 15 of a value dim for V, which makes the S
// accumulators of a lane exactly its part of the P fragments.
// V's page scale goes into the exponent (P carries s_v, the row sum divides it out again), so that
// O of pages of very different scale adds up in one accumulator. f16 holds q exactly (bf16 times a
// power of two per row, whose largest is at 2^14; entries below 2^-31 of it lose bits) and P to 11 bits with
// its largest at 2^14, so P is normal down to 2^-28 of that. Rounded so, P adds 0.1% to the error that the
// rounding of a bf16 output makes (1.650e-3 against 1.648e-3 of plain fp32, relative, 64 requests of one token).
// For fp32, q and P are pairs of f16: off by 2^-23 of a value at most (2^-39 of the row's largest for small ones),
// where fp32 itself rounds by 2^-24. Every product is two.
#include <cmath>

#include "kv8_attn.cuh"

namespace dflash {

constexpr int KM_WARPS = 8;
constexpr int KM_THREADS = 32 * KM_WARPS;
constexpr int KM_COST = 2;                             // what an item's start and end cost, in pages (measured on 64
                                                       // requests of one token alone: 92.8 us with 0, 91.4 with 2, 92.0 with 4)
constexpr float KM_BIAS = 14.f;                        // P's largest value is 2^14

template <int HD>
struct KmLayout {
  static constexpr int SLOT = KV_PAGE * HD;            // bytes of a K or V page of one head
  // 16 KB per warp: a page of K and one of V under way. 64 requests of one token took 91.7 us, 96.8 with three
  // slots (8 warps); with two, 93.1 with 6 warps and 95.0 with 12; 102.3 with 4 warps of four.
  static constexpr int SLOTS = HD == 128 ? 2 : 4;
  static constexpr int RING = SLOT * SLOTS;
  static constexpr int SIDE = 4;                       // units whose page and scales are kept
  static constexpr size_t SMEM = 128 + (size_t)KM_WARPS * (RING + SLOTS * 8 + SIDE * 16);
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// an 8 x 8 tile of 16-bit values over the warp (row g, columns 2 t and 2 t + 1 in lane (g, t)) transposed
__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// The warp's copies: pages of its units in order, K then V, each into the next slot of its ring.
template <int HD>
struct KmFeed {
  Kv8Piece p;                                          // piece of the next copy
  int u, tab_u, tab;                                   // next unit; the 32 table entries from tab_u on
  uint32_t seq;                                        // copies issued
  bool v, done;
};

// ROWS 16: S = Q K^T and O = P V with the query rows as M. ROWS 8: S^T = K Q^T and O^T = V^T P^T, the query rows
// as N, half the products and half the registers.
template <typename T, int HD, int ROWS>
__global__ void __launch_bounds__(KM_THREADS, 1) k_kv8_attn_rows(const Kv8AttnArgs a) {
  typedef KmLayout<HD> Lay;
  constexpr bool SWAP = ROWS == 8;
  constexpr int KS = HD / 16;                          // k steps of S
  constexpr int ST = SWAP ? 4 : 8;                     // tiles of S: 16 or 8 tokens each
  constexpr int OT = SWAP ? HD / 16 : HD / 8;          // tiles of O: 16 or 8 dims each
  constexpr int QF = SWAP ? 2 : 4;                     // registers of a fragment of q or P
  constexpr int PL = sizeof(T) == 4 ? 2 : 1;           // f16 planes of q and P
  extern __shared__ __align__(128) uint8_t km_smem[];
  __shared__ long long s_grp[KV8_GROUPS + 1];
  __shared__ int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t *base = km_smem;
  uint8_t *my_ring = base + warp * Lay::RING;
  const uint32_t ring = smem_u32(my_ring);
  uint64_t *bars = (uint64_t *)(base + KM_WARPS * Lay::RING) + warp * Lay::SLOTS;
  const uint32_t bar0 = smem_u32(bars);
  // per unit: page id (-1: not in the pool) and the two scales
  struct Side { int page; float ks, vs, pad; };
  Side *side = (Side *)(base + KM_WARPS * (Lay::RING + Lay::SLOTS * 8)) + warp * Lay::SIDE;
  pdl_trigger();
  if (lane < Lay::SLOTS) mbar_init(bar0 + 8 * lane, 1);
  if (threadIdx.x == 0) s_abort = 0;
  fence_mbar_init();
  __syncthreads();                                     // every warp reads s_abort, every lane the warp's barriers
  pdl_wait();
  const int me = warp * gridDim.x + blockIdx.x;        // few workers spread over all SMs
  long long chunk, item_begin;
  Kv8Piece pc;
  if (!kv8_start<KV_PAGE, ROWS, KM_COST>(a, s_grp, me, gridDim.x * KM_WARPS, pc, chunk, item_begin)) {
    if (lane == 0) a.desc[me].pieces = 0;
    return;                                            // (no barrier of the whole CTA follows)
  }
  if (lane == 0) a.desc[me] = kv8_desc<KV_PAGE, ROWS, KM_COST>(a, pc, me, chunk, item_begin);
  bool first = true;

  KmFeed<HD> f;
  f.p = pc;
  f.u = pc.u0;
  f.tab_u = -32;
  f.tab = 0;
  f.seq = 0;
  f.v = f.done = false;
  auto feed = [&]() {
    if (!f.done) {
      if (f.u >= f.tab_u + 32 || f.tab_u < 0) {        // the next 32 table entries of this piece
        f.tab_u = f.u;
        f.tab = f.u + lane < f.p.u1 ? a.table[(size_t)f.p.b * a.width + f.u + lane] : -1;
        if (f.p.r.len == 0) f.tab = -1;
      }
      const int page = __shfl_sync(0xffffffffu, f.tab, f.u - f.tab_u);
      const bool in = page >= 0 && page < a.n_pages;
      const uint32_t unit = f.seq >> 1;
      Side *sd = side + unit % Lay::SIDE;
      const uint32_t slot = f.seq % Lay::SLOTS;
      if (lane == 0) {
        // a page outside the pool is not copied; its arrival is a plain one
        if (in) {
          mbar_expect_tx(bar0 + 8 * slot, Lay::SLOT);
          bulk_load(ring + slot * Lay::SLOT, (f.v ? a.vp : a.kp) + kv8_block(page, f.p.h, a.nkv, HD), Lay::SLOT, bar0 + 8 * slot);
        } else {
          mbar_arrive(bar0 + 8 * slot);
        }
        if (!f.v) sd->page = in ? page : -1;
      }
      if (!f.v && in && lane < 2) {
        const float *src = (lane ? a.vs : a.ks) + (size_t)page * a.nkv + f.p.h;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&sd->ks + lane)), "l"(src) : "memory");
      }
      ++f.seq;
      f.v = !f.v;
      if (!f.v && ++f.u == f.p.u1) {
        if (f.p.left > 0) {
          kv8_next_piece<KV_PAGE, ROWS, KM_COST>(a, f.p);
          f.u = f.p.u0;
          f.tab_u = -32;
        } else {
          f.done = true;
        }
      }
      if (f.v) asm volatile("cp.async.commit_group;" ::: "memory");   // one group per unit, with its K page
    } else {
      // keep one group per unit ahead of the reader
      if (f.v ^= true) asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
#pragma unroll 1
  for (int i = 0; i < Lay::SLOTS; ++i) feed();

  const int group = a.nq / a.nkv, tpt = ROWS / group;
  uint32_t take = 0;                                   // pages taken from the ring
  bool ok = true;
  auto wait = [&]() {                                  // the slot of the next page
    const uint32_t slot = take % Lay::SLOTS;
    ok = ok && kv8_wait(bar0 + 8 * slot, take / Lay::SLOTS & 1, (volatile int *)&s_abort);
    ok = __all_sync(0xffffffffu, ok);
    return my_ring + slot * Lay::SLOT;
  };

  for (;;) {
    // ---------------- this piece's query rows, as f16 fragments
    // lanes load row g (and, of 16, g + 8) of the tile: token row / group, head row % group
    uint32_t qf[PL][KS][QF];
    float rs[2];                                       // scale log2(e) 2^(row exponent)
    bool bad[2];
    int tok[2];
#pragma unroll
    for (int rr = 0; rr < (SWAP ? 1 : 2); ++rr) {
      const int row = g + 8 * rr, tk = pc.qt * tpt + row / group;
      const bool live = row < tpt * group && tk < pc.r.n;
      tok[rr] = live ? tk : -1;
      float x[HD / 4];                                 // dims (HD / 4) t .. + HD / 4 - 1
      float big = 0.f;
      bool fin = true;
      if (live) {
        const T *src = (const T *)a.q + (int64_t)(pc.r.row0 + tk) * a.q_stride + (int64_t)(pc.h * group + row % group) * HD + t * (HD / 4);
#pragma unroll
        for (int i = 0; i < HD / 4; i += 16 / sizeof(T)) {
          const uint4 w = *(const uint4 *)(src + i);
          const T *e = (const T *)&w;
#pragma unroll
          for (int j = 0; j < 16 / (int)sizeof(T); ++j) x[i + j] = to_f(e[j]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < HD / 4; ++i) x[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < HD / 4; ++i) {
        big = fmaxf(big, fabsf(x[i]));
        fin = fin && fabsf(x[i]) <= 3.402823466e38f;
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      const unsigned fb = __ballot_sync(0xffffffffu, fin);
      bad[rr] = (fb >> (lane & ~3) & 15) != 15;
      // q * 2^(14 - e): the largest is in [2^14, 2^15)
      const int e = bad[rr] ? 0 : max(-100, (int)(__float_as_uint(big) >> 23) - 127);
      const float up = bad[rr] ? 0.f : exp2f((float)(14 - e));
      rs[rr] = a.scale * 1.44269504088896341f * exp2f((float)(e - 14));
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int z = 0; z < 2; ++z) {                  // dims 4 k + 2 z, + 1 of the lane's
          const float y0 = bad[rr] ? 0.f : x[4 * k + 2 * z] * up, y1 = bad[rr] ? 0.f : x[4 * k + 2 * z + 1] * up;
          const uint32_t h = pack_f16(y0, y1);
          qf[0][k][SWAP ? z : 2 * z + rr] = h;
          if constexpr (PL == 2) {
            const float2 f = unpack_f16(h);
            qf[PL - 1][k][SWAP ? z : 2 * z + rr] = pack_f16(y0 - f.x, y1 - f.y);
          }
        }
    }
    if constexpr (SWAP) {
      // from here on a lane keeps rows 2 t and 2 t + 1 (of 16: g and g + 8)
      const float rs0 = rs[0];
      const int state = (tok[0] << 1) | (int)bad[0];
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        rs[rr] = __shfl_sync(0xffffffffu, rs0, (2 * t + rr) * 4);
        const int st = __shfl_sync(0xffffffffu, state, (2 * t + rr) * 4);
        tok[rr] = st >> 1;
        bad[rr] = st & 1;
      }
    }
    float o[OT][4];
#pragma unroll
    for (int i = 0; i < OT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    // tokens from `open` on are hidden from some row of the request
    const int open = a.mask == DFLASH_MASK_NONE ? pc.r.len : max(0, pc.r.len - pc.r.n);

#pragma unroll 1
    for (int u = pc.u0; u < pc.u1; ++u) {
      const uint8_t *kslot = wait();
      asm volatile("cp.async.wait_group %0;" ::"n"(Lay::SLOTS / 2 - 1) : "memory");
      __syncwarp();
      const Side sd = side[take / 2 % Lay::SIDE];
      if (!ok) break;
      ++take;
      float s[ST][4];
      // two tiles at a time, whose chains of sums interleave
#pragma unroll
      for (int j = 0; j < ST; j += 2) {
        uint32_t w[2][SWAP ? 2 : 1][HD / 16];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
#pragma unroll
          for (int y = 0; y < (SWAP ? 2 : 1); ++y) {
            const int token = 16 * (g >> 1) + (g & 1) + (SWAP ? 4 : 2) * (j + z) + 2 * y;
#pragma unroll
            for (int c = 0; c < HD / 64; ++c)
              *(uint4 *)&w[z][y][4 * c] = *(const uint4 *)(kslot + token * HD + t * (HD / 4) + 16 * c);
          }
          s[j + z][0] = s[j + z][1] = s[j + z][2] = s[j + z][3] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            uint32_t f[4];
            if constexpr (SWAP) {
              e4m3x4_to_f16(w[z][0][k], f[0], f[2]);
              e4m3x4_to_f16(w[z][SWAP ? 1 : 0][k], f[1], f[3]);
#pragma unroll
              for (int pl = 0; pl < PL; ++pl) mma_f16(s[j + z], f, qf[pl][k][0], qf[pl][k][1]);
            } else {
              e4m3x4_to_f16(w[z][0][k], f[0], f[1]);
#pragma unroll
              for (int pl = 0; pl < PL; ++pl) mma_f16(s[j + z], *(const uint32_t(*)[4])qf[pl][k], f[0], f[1]);
            }
          }
      }
      __syncwarp();                                    // every lane has read the K page
      feed();
      // value i < 2 ST of row rr (of 16: tokens 16 t + i; of 8: 16 (g >> 1) + (g & 1) + 2 i)
      auto val = [&](int rr, int i) -> float & { return SWAP ? s[i >> 1][rr + 2 * (i & 1)] : s[i >> 1][2 * rr + (i & 1)]; };
      auto across = [&](float v, bool sum) {           // over the lanes that share the row
#pragma unroll
        for (int z = 0; z < (SWAP ? 3 : 2); ++z) {
          const float w = __shfl_xor_sync(0xffffffffu, v, (SWAP ? 4 : 1) << z);
          v = sum ? v + w : fmaxf(v, w);
        }
        return v;
      };
      const bool out = sd.page < 0;                    // not in the pool: nothing of it is seen
      const bool partial = out || (long long)(u + 1) * KV_PAGE > open;
      const float ev = out ? 0.f : log2f(sd.vs), iv = out ? 1.f : 1.f / sd.vs;
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const float c = out ? 0.f : rs[rr] * sd.ks;
#pragma unroll
        for (int i = 0; i < 2 * ST; ++i) val(rr, i) = fmaf(val(rr, i), c, ev);
      }
      if (partial) {
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          const uint64_t see = out || tok[rr] < 0 ? 0 : kv8_visible(a, pc.r, tok[rr], u);
          const uint32_t hidden = ~(uint32_t)(see >> (SWAP ? 16 * (g >> 1) + (g & 1) : 16 * t));
#pragma unroll
          for (int i = 0; i < 2 * ST; ++i)
            if (hidden >> (SWAP ? 2 * i : i) & 1) val(rr, i) = -INFINITY;
        }
      }
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
#pragma unroll
        for (int i = 0; i < 2 * ST; i += 2) mx[rr] = fmaxf(mx[rr], fmaxf(val(rr, i), val(rr, i + 1)));
        mx[rr] = fmaxf(across(mx[rr], false), m[rr]);
      }
      float alpha[2], ref[2];
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const float top = mx[rr] == -INFINITY ? 0.f : mx[rr];
        ref[rr] = top - KM_BIAS;
        alpha[rr] = ex2(m[rr] - top);
        m[rr] = mx[rr];
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 2 * ST; ++i) {
          float &x = val(rr, i);
          x = ex2(x - ref[rr]);
          sum[i & 1] += x;
        }
        l[rr] = fmaf(l[rr], alpha[rr], (sum[0] + sum[1]) * iv);
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < OT; ++i) {
          o[i][0] *= alpha[0], o[i][1] *= alpha[SWAP ? 1 : 0];
          o[i][2] *= alpha[SWAP ? 0 : 1], o[i][3] *= alpha[1];
        }
      }
      uint32_t pf[PL][4][QF];                          // P fragments of 16 tokens each
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < QF; ++i) {
          // of 16 rows: fragments of S as they are; of 8: S^T's tokens (g) x rows (2 t) turned over
          const float x0 = SWAP ? s[k][2 * i] : s[SWAP ? 0 : 2 * k + (i >> 1)][2 * (i & 1)];
          const float x1 = SWAP ? s[k][2 * i + 1] : s[SWAP ? 0 : 2 * k + (i >> 1)][2 * (i & 1) + 1];
          const uint32_t h = pack_f16(x0, x1);
          pf[0][k][i] = SWAP ? turn8x8(h) : h;
          if constexpr (PL == 2) {
            const float2 f = unpack_f16(h);
            const uint32_t lo = pack_f16(x0 - f.x, x1 - f.y);
            pf[PL - 1][k][i] = SWAP ? turn8x8(lo) : lo;
          }
        }
      uint8_t *vslot = wait();
      if (!ok) break;
      ++take;
      bool nan = false;
      if (partial) {
        // Bytes of tokens that no row sees (a page's tail) may be anything, and a NaN must not meet the zero
        // weight of a row that does not see it: each lane puts its own bytes in order where they lie.
        const int tail = out ? 0 : min(16, max(0, pc.r.len - u * KV_PAGE - 16 * t));
#pragma unroll 1
        for (int i = 0; i < HD / 8; ++i) {
          uint4 *at = (uint4 *)(vslot + (8 * i + g) * KV_PAGE + 16 * t);
          uint4 v = *at;
          uint32_t *w = (uint32_t *)&v;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int n = tail - 4 * k;
            w[k] = n >= 4 ? w[k] : n <= 0 ? 0u : w[k] & ((1u << 8 * n) - 1);
            const uint32_t nb = nan_bytes(w[k]);
            nan |= nb != 0;
            w[k] &= ~byte_mask(nb);
          }
          *at = v;
        }
        fence_proxy_async_smem();                      // before the next copy into the slot
      }
#pragma unroll
      for (int i = 0; i < OT; i += 2) {                // two tiles at a time again
        uint32_t w[2][SWAP ? 2 : 1][4];
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
          for (int y = 0; y < (SWAP ? 2 : 1); ++y)
            *(uint4 *)w[z][y] = *(const uint4 *)(vslot + ((SWAP ? 16 : 8) * (i + z) + 8 * y + g) * KV_PAGE + 16 * t);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            uint32_t f[4];
            if constexpr (SWAP) {
              e4m3x4_to_f16(w[z][0][k], f[0], f[2]);
              e4m3x4_to_f16(w[z][SWAP ? 1 : 0][k], f[1], f[3]);
#pragma unroll
              for (int pl = 0; pl < PL; ++pl) mma_f16(o[i + z], f, pf[pl][k][0], pf[pl][k][1]);
            } else {
              e4m3x4_to_f16(w[z][0][k], f[0], f[1]);
#pragma unroll
              for (int pl = 0; pl < PL; ++pl) mma_f16(o[i + z], *(const uint32_t(*)[4])pf[pl][k], f[0], f[1]);
            }
          }
      }
      if (partial && __any_sync(0xffffffffu, nan)) {   // rows that see a NaN value get it (rare)
        const uint64_t vis0 = tok[0] < 0 ? 0 : kv8_visible(a, pc.r, tok[0], u);
        const uint64_t vis1 = tok[1] < 0 ? 0 : kv8_visible(a, pc.r, tok[1], u);
        const uint8_t *page = a.vp + kv8_block(sd.page, pc.h, a.nkv, HD);
        uint32_t hit0 = 0, hit1 = 0;                   // bit 2 i + e: the lane's dim e of tile i holds one
#pragma unroll 1
        for (int d = 0; d < 2 * OT; ++d) {
          const int dim = SWAP ? 16 * (d >> 1) + 8 * (d & 1) + g : 8 * (d >> 1) + 2 * t + (d & 1);
          uint64_t at = 0;                             // tokens whose value is NaN in that dim
#pragma unroll 1
          for (int k = 0; k < KV_PAGE; ++k) at |= (uint64_t)((page[dim * KV_PAGE + k] & 0x7f) == 0x7f) << k;
          hit0 |= (uint32_t)((at & vis0) != 0) << d;
          hit1 |= (uint32_t)((at & vis1) != 0) << d;
        }
#pragma unroll
        for (int i = 0; i < OT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // adding 0 or NaN, so that no lane branches
            o[i][SWAP ? 2 * e : e] += __uint_as_float((uint32_t)((int)(hit0 << (31 - 2 * i - e)) >> 31) & 0x7fc00000u);
            o[i][SWAP ? 2 * e + 1 : 2 + e] += __uint_as_float((uint32_t)((int)(hit1 << (31 - 2 * i - e)) >> 31) & 0x7fc00000u);
          }
      }
      __syncwarp();                                    // every lane has read the V page
      feed();
    }
    if (!ok) break;

    // ---------------- the piece's result
    const bool whole = pc.u1 - pc.u0 == pc.units;
    const int slot = 2 * me + (first ? 0 : 1);
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
#pragma unroll
      for (int z = 0; z < (SWAP ? 3 : 2); ++z) l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], (SWAP ? 4 : 1) << z);
      if (tok[rr] < 0) continue;
      const int row = SWAP ? 2 * t + rr : g + 8 * rr;
      if (bad[rr]) l[rr] = NAN;
      const bool one = SWAP ? g == 0 : t == 0;         // one lane of the row
      if (whole) {
        const size_t at = (size_t)(pc.r.row0 + tok[rr]) * a.nq + pc.h * group + row % group;
        const float inv = l[rr] == 0.f ? 0.f : 1.f / l[rr];
        T *out = (T *)a.out + at * HD;
#pragma unroll
        for (int i = 0; i < OT; ++i) {
          if constexpr (SWAP) {
            out[16 * i + g] = from_f<T>(o[i][rr] * inv);
            out[16 * i + 8 + g] = from_f<T>(o[i][2 + rr] * inv);
          } else if constexpr (PL == 1) {
            *(__nv_bfloat162 *)(out + 8 * i + 2 * t) = __floats2bfloat162_rn(o[i][2 * rr] * inv, o[i][2 * rr + 1] * inv);
          } else {
            *(float2 *)(out + 8 * i + 2 * t) = make_float2(o[i][2 * rr] * inv, o[i][2 * rr + 1] * inv);
          }
        }
        if (a.lse && one) a.lse[at] = l[rr] == 0.f ? -INFINITY : (m[rr] - KM_BIAS + log2f(l[rr])) * LN2;
      } else {
        float *po = a.part_o + ((size_t)slot * ROWS + row) * HD;
#pragma unroll
        for (int i = 0; i < OT; ++i) {
          if constexpr (SWAP) {
            po[16 * i + g] = o[i][rr];
            po[16 * i + 8 + g] = o[i][2 + rr];
          } else {
            *(float2 *)(po + 8 * i + 2 * t) = make_float2(o[i][2 * rr], o[i][2 * rr + 1]);
          }
        }
        if (one) *(float2 *)(a.part_ml + ((size_t)slot * ROWS + row) * 2) = make_float2(m[rr] - KM_BIAS, l[rr]);
      }
    }
    if (pc.left <= 0) break;
    kv8_next_piece<KV_PAGE, ROWS, KM_COST>(a, pc);
    first = false;
  }
  if (!ok) {
    // A wait ran out of time: the rows that this worker still owes become NaN, and its copies in
    // flight are waited for, with a limit.
    for (;;) {
      const int slot = 2 * me + (first ? 0 : 1);
      for (int row = 0; row < tpt * group; ++row) {
        const int tk = pc.qt * tpt + row / group;
        if (tk >= pc.r.n) break;
        const size_t at = (size_t)(pc.r.row0 + tk) * a.nq + pc.h * group + row % group;
        if (pc.u1 - pc.u0 == pc.units) {
          for (int d = lane; d < HD; d += 32) ((T *)a.out)[at * HD + d] = from_f<T>(NAN);
          if (a.lse && lane == 0) a.lse[at] = NAN;
        } else if (lane == 0) {
          *(float2 *)(a.part_ml + ((size_t)slot * ROWS + row) * 2) = make_float2(0.f, NAN);
        }
      }
      if (pc.left <= 0) break;
      kv8_next_piece<KV_PAGE, ROWS, KM_COST>(a, pc);
      first = false;
    }
    const unsigned long long t0 = global_ns();
    for (; take < f.seq; ++take)
      while (!mbar_try_wait(bar0 + 8 * (take % Lay::SLOTS), take / Lay::SLOTS & 1) && global_ns() - t0 < TC_WAIT_NS) {
      }
  }
}

template <typename T, int HD, int ROWS>
cudaError_t launch_rows(const Kv8AttnArgs &a, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(k_kv8_attn_rows<T, HD, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)KmLayout<HD>::SMEM);
  if (e == cudaSuccess) e = launch_pdl(k_kv8_attn_rows<T, HD, ROWS>, dim3(KV8_SMS), dim3(KM_THREADS), KmLayout<HD>::SMEM, s, a);
  if (e == cudaSuccess)
    e = launch_pdl(k_kv8_combine<T, HD, ROWS>, dim3(KV8_SMS * KM_WARPS - 1, 2), dim3(128), 0, s, a);
  return e;
}
template <typename T, int ROWS>
cudaError_t launch_rows(const Kv8AttnArgs &a, int hd, cudaStream_t s) {
  return hd == 128 ? launch_rows<T, 128, ROWS>(a, s) : launch_rows<T, 64, ROWS>(a, s);
}

}  // namespace dflash

using namespace dflash;

namespace {
bool attn_ok(const dflash_kv8_cache *c, const dflash_kv8_attn *x, bool pointers) {
  if (!kv8_cache_ok(c, pointers) || !x) return false;
  if (x->n_req < 1 || x->n_req > KV8_MAX_REQ || x->rows < 0 || x->n_q_heads < 1 || x->n_q_heads % c->n_kv_heads ||
      x->n_q_heads / c->n_kv_heads > 8 || x->max_blocks < 1 || x->max_blocks > (1 << 24) || x->max_q < 0 ||
      (x->dtype != DFLASH_F32 && x->dtype != DFLASH_BF16) || x->mask < DFLASH_MASK_NONE || x->mask > DFLASH_MASK_TREE ||
      (x->mask == DFLASH_MASK_TREE && x->tree_words < 1) || !(x->scale > 0.f) || !std::isfinite(x->scale))
    return false;
  const int64_t V = 16 / dtype_bytes(x->dtype);
  if (x->q_stride < (int64_t)x->n_q_heads * c->head_dim || x->q_stride % V) return false;
  if (!pointers || x->rows == 0) return true;
  return x->q && x->cu_q && x->ctx_len && x->block_table && x->out && aligned(x->q, 16) && aligned(x->out, 16) &&
         aligned(x->cu_q, 4) && aligned(x->ctx_len, 4) && aligned(x->block_table, 4) && aligned(x->lse, 4) &&
         (x->mask != DFLASH_MASK_TREE || (x->tree_mask && aligned(x->tree_mask, 4)));
}

// Workspace: descriptors, then partial maxima and sums, then partial outputs.
struct Space {
  int64_t desc, ml, o, bytes;
};
Space space_of(int hd) {
  const int64_t workers = KV8_SMS * KM_WARPS, m = 16;   // the tiles' 152 workers of 128 rows need as much
  Space s;
  s.desc = 0;
  s.ml = (workers * (int64_t)sizeof(Kv8Desc) + 255) / 256 * 256;
  s.o = s.ml + workers * 2 * m * 8;
  s.bytes = s.o + workers * 2 * m * hd * 4;
  return s;
}
}  // namespace

extern "C" int64_t dflash_kv8_attention_workspace(const dflash_kv8_cache *cache, const dflash_kv8_attn *args) {
  if (!attn_ok(cache, args, false)) return -1;
  return space_of(cache->head_dim).bytes;
}

extern "C" dflash_status dflash_kv8_attention(void *stream, const dflash_kv8_cache *c, const dflash_kv8_attn *x) {
  if (!attn_ok(c, x, true)) return DFLASH_ERR_INVALID_ARG;
  if (x->rows == 0) return DFLASH_OK;
  const Space sp = space_of(c->head_dim);
  if (!x->workspace || !aligned(x->workspace, 256) || x->workspace_bytes < sp.bytes) return DFLASH_ERR_INVALID_ARG;
  uint8_t *ws = (uint8_t *)x->workspace;
  const Kv8AttnArgs a{x->n_req, x->rows, x->n_q_heads, c->n_kv_heads, x->max_blocks, x->mask, x->tree_words, c->n_pages,
                      x->scale, x->q, x->q_stride, x->cu_q, x->ctx_len, x->block_table, x->tree_mask, x->out, x->lse,
                      (const uint8_t *)c->k_pages, (const uint8_t *)c->v_pages, c->k_scale, c->v_scale,
                      (Kv8Desc *)(ws + sp.desc), (float *)(ws + sp.o), (float *)(ws + sp.ml)};
  const cudaStream_t s = (cudaStream_t)stream;
  // Rows of a request and kv head, as far as the host knows: up to 8 go to the kernel for 8, up to 16 to the one
  // for 16, which reads the cache once where two tiles of 8 would read it twice. Above, bf16 goes to the tensor
  // memory tiles; fp32 stays with 16 rows at a time. 8 requests x 8 kv heads of 128 over 32768 tokens, us:
  //   rows       8      12      16      24      64
  //   8 a go    88     124     124     244     455
  //   16        90      92      94     147     325
  //   tiles    121     121     121     122     133
  // and over 2048 tokens 8 rows 14 / 15 / 23, 16 rows 18.5 / 17.7 / 23, 24 rows 22.7 / 22.0 / 23.4, 64 rows 42 / 32 / 25.
  const int64_t most = (int64_t)x->max_q * (x->n_q_heads / c->n_kv_heads);
  const bool wide = x->dtype == DFLASH_BF16;
  const int hd = c->head_dim;
  const cudaError_t e = most <= 8 ? (wide ? launch_rows<bf16, 8>(a, hd, s) : launch_rows<float, 8>(a, hd, s))
                        : !wide ? launch_rows<float, 16>(a, hd, s)
                        : most <= 16 ? launch_rows<bf16, 16>(a, hd, s) : launch_kv8_tiles(a, hd, s);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
