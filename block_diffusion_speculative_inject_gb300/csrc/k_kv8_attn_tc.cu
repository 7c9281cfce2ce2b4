// Attention over the 8-bit paged cache for many query rows per kv head (bf16): verify blocks, draft
// trees, prompt chunks. One persistent CTA per SM walks its share of the work (kv8_sched.cuh) in tiles
// of 128 rows (tokens x query heads of the kv head) and 128 tokens (two pages):
//   S[128, 128] = Q . K^T        kind::f8f6f4, A = Q in tensor memory, B = the K pages as they are
//   P = 2^(S c + log2 s_v - m)   two threads per row, one page each; f16, written over S
//   O[128, hd] += P . V          kind::f16, A = P in tensor memory, B = V pages widened to f16
// Q's row, scaled by a power of two so that its largest entry is in [128, 256), is the sum of an e4m3 and
// an e5m2 part: bf16 has 8 significant bits, e4m3 takes 4, and what rounding to nearest leaves is at
// most 8 units of the last place, which e5m2's 3 bits hold exactly. So K needs no conversion, and S is
// exact for entries of q down to 2^-14 of the row's largest (below, q is off by at most 2^-21 of it).
// P could not go the same way: rows with one loud token and many quiet ones need its small values, so
// P is f16 (11 bits, largest 2^7 .. 2^15, normal to 2^-14) and two warps widen V (exact) into a second
// pair of tiles. That costs shared-memory traffic of 3x V's bytes per tile, 144 KB in all with the MMAs'
// own reads, about 0.6 us at 128 B/clk against 0.74 us that an SM's share of HBM takes for the tile's 32 KB.
//
// The running maximum is lazy: O is rescaled only when a row's maximum grows by more than 2^8. The
// pages' scales enter as in the few-row kernel: s_k in c, s_v in the exponent of P.
//
// Tensor memory (512 columns): S/P at 0 and 128 (tile parity), O at 256, Q at 384 and 448 (piece
// parity: 32 columns of the e4m3 part, then 32 of the e5m2 part). P of the 64 tokens of a half row lies in
// the first 32 of their own 64 columns of S.
//
// Roles (384 threads): warp 0 copies K (TMA, 128- or 64-byte swizzle) and V (bulk, as stored) into
// rings of 4 tiles; warp 1 issues the MMAs, S of the next tile ahead of P.V of this one, across
// piece borders; warps 2-9 load Q (of the next piece, ahead), run the softmax and write
// results; warps 10-11 widen V. All waits are bounded; rows whose wait ran out become NaN.
#include "kv8_attn.cuh"

namespace dflash {

constexpr int KT_THREADS = 384;
constexpr int KT_WIDEN = 64;                            // threads that widen V
constexpr int KT_STAGES = 4;
constexpr int KT_SIDE = 2 * KT_STAGES;                 // tiles whose page ids and scales are kept
constexpr float KT_BIAS = 7.f;
constexpr uint32_t TM_O = 256, TM_Q = 384;

struct KtParams {
  CUtensorMap kmap;
  Kv8AttnArgs a;
};

template <int HD>
struct KtLayout {
  static constexpr uint32_t PAGE8 = KV_PAGE * HD;      // a K or V page, 8 bits
  static constexpr uint32_t PAGE16 = KV_PAGE * HD * 2; // a V page in f16
  static constexpr uint32_t K0 = 0, V0 = K0 + KT_STAGES * 2 * PAGE8, W0 = V0 + KT_STAGES * 2 * PAGE8;
  static constexpr uint32_t END = W0 + 2 * 2 * PAGE16;
};

struct KtSide {
  int page[2];                                         // -1: not there, nothing of it is seen
  float ks[2], vs[2];
};

struct KtShared {
  uint64_t kfull[KT_STAGES], kempty[KT_STAGES], vfull[KT_STAGES], vempty[KT_STAGES];
  uint64_t s_full[2], p_full[2], w_full[2], w_empty[2], q_full[2], o_full, o_empty, pv_done, drain;
  KtSide side[KT_SIDE];
  float xmax[2][2][128], xsum[2][128];
  int xok[2][2][4];
  int nan_piece[4];                                    // per piece ordinal mod 4 (two are ahead): ordinal + 1 if V held a NaN
  int abort;
  uint32_t tmem;
  long long grp[KV8_GROUPS + 1];
};

template <int HD>
constexpr size_t kt_smem() { return 1024 + KtLayout<HD>::END + sizeof(KtShared); }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"((uint64_t)map), "r"(c0), "r"(c1), "r"(c2), "r"(mbar) : "memory");
}
__device__ __forceinline__ void umma_f8_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
               " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
               "r"(acc) : "memory");
}
// K-major descriptor of rows of 64 bytes in the 64-byte swizzle: 8-row atoms of 512 bytes
__device__ __forceinline__ uint64_t sw64_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(512 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)4 << 61;
}
// D fp32, M = 128, N columns; A and B formats as the kind numbers them
constexpr uint32_t idesc_of(int a_fmt, int b_fmt, int N) {
  return (1u << 4) | (uint32_t)a_fmt << 7 | (uint32_t)b_fmt << 10 | (uint32_t)(N >> 3) << 17 | (128u >> 4) << 24;
}
__device__ __forceinline__ uint32_t f32_to_e5m2x2(float a, float b) {
  uint32_t r;
  asm("{\n .reg .b16 t;\n cvt.rn.satfinite.e5m2x2.f32 t, %2, %1;\n cvt.u32.u16 %0, t;\n}\n" : "=r"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
}
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t *w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}

template <int HD>
__global__ void __launch_bounds__(KT_THREADS, 1) k_kv8_attn_tiles(const __grid_constant__ KtParams p) {
  typedef KtLayout<HD> Lay;
  typedef Kv8Tiles<KT_TOKENS, KT_ROWS> Tiles;
  const Kv8AttnArgs &a = p.a;
  extern __shared__ uint8_t kt_raw[];
  const uint32_t raw = smem_u32(kt_raw), base = (raw + 1023u) & ~1023u;
  KtShared &sh = *(KtShared *)(kt_raw + (base - raw) + Lay::END);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](uint64_t &b) { return smem_u32(&b); };
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < KT_STAGES; ++i) {
      mbar_init(bar(sh.kfull[i]), 1);
      mbar_init(bar(sh.kempty[i]), 1);
      mbar_init(bar(sh.vfull[i]), 1);
      mbar_init(bar(sh.vempty[i]), KT_WIDEN / 32);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(sh.s_full[i]), 2);                 // the MMAs, and their issuer for the side words that it has seen
      mbar_init(bar(sh.p_full[i]), 8);
      mbar_init(bar(sh.w_full[i]), KT_WIDEN / 32);
      mbar_init(bar(sh.w_empty[i]), 1);
      mbar_init(bar(sh.q_full[i]), 8);
    }
    mbar_init(bar(sh.o_full), 1);
    mbar_init(bar(sh.o_empty), 8);
    mbar_init(bar(sh.pv_done), 1);
    mbar_init(bar(sh.drain), 1);
    sh.abort = 0;
    for (int i = 0; i < 4; ++i) sh.nan_piece[i] = 0;
    fence_mbar_init();
  }
  pdl_wait();
  kv8_group_sums<KT_TOKENS, KT_ROWS>(a, sh.grp);
  const long long total = sh.grp[(a.n_req + 31) / 32];
  const long long chunk = (total + gridDim.x - 1) / gridDim.x, pos = (long long)blockIdx.x * chunk;
  if (pos >= total) {                                  // uniform for the CTA
    if (threadIdx.x == 0) a.desc[blockIdx.x].units = 0;
    return;
  }
  long long item_begin;
  Kv8Piece pc = kv8_first_piece<KT_TOKENS, KT_ROWS>(a, sh.grp, pos, min(chunk, total - pos), item_begin);
  if (threadIdx.x == 0) a.desc[blockIdx.x] = Kv8Desc{item_begin, chunk, pc.units, pc.b, pc.qt, pc.h};
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int *abort_flag = (volatile int *)&sh.abort;
  auto wait = [&](uint64_t &b, uint32_t parity) { return mbar_wait(bar(b), parity & 1, abort_flag, nullptr, 0); };

  if (warp == 0) {
    // ---------------- copies
    if (lane == 0) tma_prefetch_map(&p.kmap);
    uint32_t i = 0;
    bool go = true;
    for (;;) {
      const int limit = Tiles(a).limit(pc.r, pc.qt);
      int tab_u = -32, page = -1;                      // lane x: page x of the 16 tiles from tab_u on
      float ks = 1.f, vs = 1.f;
      for (int u = pc.u0; u < pc.u1 && go; ++u, ++i) {
        if (tab_u < 0 || u >= tab_u + 16) {
          tab_u = u;
          const int x = 2 * u + lane;
          page = (long long)x * KV_PAGE < limit && x < 2 * pc.u1 ? a.table[(size_t)pc.b * a.width + x] : -1;
          if (page < 0 || page >= a.n_pages) page = -1;
          ks = vs = 1.f;
          if (page >= 0) {
            ks = a.ks[(size_t)page * a.nkv + pc.h];
            vs = a.vs[(size_t)page * a.nkv + pc.h];
          }
        }
        const int at = 2 * (u - tab_u);
        const int stg = i % KT_STAGES;
        const uint32_t use = i / KT_STAGES;
        KtSide sd;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          sd.page[x] = __shfl_sync(0xffffffffu, page, at + x);
          sd.ks[x] = __shfl_sync(0xffffffffu, ks, at + x);
          sd.vs[x] = __shfl_sync(0xffffffffu, vs, at + x);
        }
        if (lane == 0) {
          if (use > 0) go = wait(sh.kempty[stg], use - 1) && wait(sh.vempty[stg], use - 1);
          if (go) {
            sh.side[i % KT_SIDE] = sd;
            const uint32_t there = (sd.page[0] >= 0) + (sd.page[1] >= 0);
            if (there) {
              mbar_expect_tx(bar(sh.kfull[stg]), there * Lay::PAGE8);
              mbar_expect_tx(bar(sh.vfull[stg]), there * Lay::PAGE8);
            } else {
              mbar_arrive(bar(sh.kfull[stg]));
              mbar_arrive(bar(sh.vfull[stg]));
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (sd.page[x] >= 0) {
                tma_load_3d(base + Lay::K0 + (2 * stg + x) * Lay::PAGE8, &p.kmap, 0, 0, sd.page[x] * a.nkv + pc.h, bar(sh.kfull[stg]));
                bulk_load(base + Lay::V0 + (2 * stg + x) * Lay::PAGE8, a.vp + kv8_block(sd.page[x], pc.h, a.nkv, HD), Lay::PAGE8,
                          bar(sh.vfull[stg]));
              }
          }
        }
        go = __shfl_sync(0xffffffffu, (int)go, 0) != 0;
        if (!go) break;
      }
      if (!go || pc.left <= 0) break;
      kv8_next_piece<KT_TOKENS, KT_ROWS>(a, pc);
    }
    if (lane == 0) {
      // copies in flight end before the CTA does (bounded; at once unless a wait ran out)
      const unsigned long long t0 = global_ns();
      for (uint32_t j = i > KT_STAGES ? i - KT_STAGES : 0; j < i; ++j)
        while (!(mbar_try_wait(bar(sh.kfull[j % KT_STAGES]), j / KT_STAGES & 1) &&
                 mbar_try_wait(bar(sh.vfull[j % KT_STAGES]), j / KT_STAGES & 1)) && global_ns() - t0 < TC_WAIT_NS) {
        }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- MMAs
      constexpr uint32_t idS0 = idesc_of(0, 0, KT_TOKENS), idS1 = idesc_of(1, 0, KT_TOKENS), idO = idesc_of(0, 0, HD);
      Kv8Piece sp = pc;                                // the piece whose S is issued next
      int su = sp.u0;
      uint32_t si = 0, spn = 0;                        // its tile and piece ordinals
      bool more = true;
      auto issue_s = [&]() {
        if (su == sp.u0 && !wait(sh.q_full[spn & 1], spn >> 1)) return false;
        const int stg = si % KT_STAGES;
        if (!wait(sh.kfull[stg], si / KT_STAGES)) return false;
        tc_fence_after();
        const uint32_t ks = base + Lay::K0 + 2 * stg * Lay::PAGE8, d = tmem + (si & 1) * 128, q = tmem + TM_Q + (spn & 1) * 64;
#pragma unroll
        for (int pl = 0; pl < 2; ++pl)
#pragma unroll
          for (int k = 0; k < HD / 32; ++k)
            umma_f8_ts(d, q + 32 * pl + 8 * k, HD == 128 ? sw128_desc(ks + 32 * k) : sw64_desc(ks + 32 * k), pl ? idS1 : idS0,
                       (pl | k) ? 1u : 0u);
        umma_commit(bar(sh.kempty[stg]));
        mbar_arrive(bar(sh.s_full[si & 1]));
        umma_commit(bar(sh.s_full[si & 1]));
        ++si;
        if (++su == sp.u1) {
          if (sp.left > 0) {
            kv8_next_piece<KT_TOKENS, KT_ROWS>(a, sp);
            su = sp.u0;
            ++spn;
          } else {
            more = false;
          }
        }
        return true;
      };
      bool go = issue_s();
      uint32_t i = 0;
      for (uint32_t pn = 0; go; ++pn) {
        for (int u = pc.u0; go && u < pc.u1; ++u, ++i) {
          if (more && !(go = issue_s())) break;
          const int par = i & 1;
          if (!(go = wait(sh.p_full[par], i >> 1))) break;
          if (!(go = wait(sh.w_full[par], i >> 1))) break;
          if (u == pc.u0 && pn > 0 && !(go = wait(sh.o_empty, pn - 1))) break;
          tc_fence_after();
          const uint32_t w = base + Lay::W0 + 2 * par * Lay::PAGE16;
#pragma unroll
          for (int k = 0; k < 8; ++k)                  // 16 tokens each; k >> 2: the page
            umma_bf16_ts(tmem + TM_O, tmem + par * 128 + 64 * (k >> 2) + 8 * (k & 3),
                         sw128_desc(w + (k >> 2) * Lay::PAGE16 + (k & 3) * 32), idO, (u > pc.u0 || k) ? 1u : 0u);
          umma_commit(bar(sh.w_empty[par]));
          umma_commit(bar(sh.pv_done));
        }
        if (!go) break;
        umma_commit(bar(sh.o_full));
        if (pc.left <= 0) break;
        kv8_next_piece<KT_TOKENS, KT_ROWS>(a, pc);
      }
      // MMAs in flight end before the tensor memory is given back
      umma_commit(bar(sh.drain));
      const unsigned long long t0 = global_ns();
      while (!mbar_try_wait(bar(sh.drain), 0) && global_ns() - t0 < TC_WAIT_NS) {
      }
    }
  } else if (warp < 10) {
    // ---------------- Q, softmax, results: warps w and w + 4 share the rows of lane quarter w % 4
    const int q = warp & 3, half = (warp - 2) >> 2, r = q * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16);
    const int group = a.nq / a.nkv, tpt = Tiles(a).tpt;
    bool ok = true;
    // writes Q of a piece; returns the row's factor (NaN: the row holds an infinity or NaN)
    auto load_q = [&](const Kv8Piece &x, uint32_t pn) {
      const int tk = x.qt * tpt + r / group;
      const bool live = r < tpt * group && tk < x.r.n;
      constexpr int N = HD / 2;                        // this half's dims
      float v[N];
      float big = 0.f;
      bool fin = true;
      const bf16 *src = (const bf16 *)a.q + (int64_t)(x.r.row0 + tk) * a.q_stride + (int64_t)(x.h * group + r % group) * HD + N * half;
      uint4 w[N / 8];
#pragma unroll
      for (int i = 0; i < N / 8; ++i) w[i] = live ? *(const uint4 *)(src + 8 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < N / 8; ++i) {
        const uint32_t e[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[8 * i + 2 * j] = __uint_as_float(e[j] << 16);
          v[8 * i + 2 * j + 1] = __uint_as_float(e[j] & 0xffff0000u);
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        big = fmaxf(big, fabsf(v[i]));
        fin = fin && fabsf(v[i]) <= 3.402823466e38f;
      }
      if (!fin) big = INFINITY;
      sh.xsum[half][r] = big;
      pair_sync(1 + q);
      big = fmaxf(big, sh.xsum[half ^ 1][r]);
      pair_sync(1 + q);                                // (the row sums reuse the words)
      const bool bad = !(big <= 3.402823466e38f);
      const int e = bad ? 0 : max(-100, (int)(__float_as_uint(big) >> 23) - 127);
      const float up = bad ? 0.f : exp2f((float)(7 - e));
      const uint32_t dst = lane_base + TM_Q + (pn & 1) * 64 + half * (N / 4);
#pragma unroll
      for (int c = 0; c < N / 4; c += 8) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float y[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) y[z] = bad ? 0.f : v[4 * (c + j) + z] * up;
          const uint32_t h0 = f32_to_e4m3x2(y[0], y[1]), h1 = f32_to_e4m3x2(y[2], y[3]);
          const float2 f0 = e4m3x2_to_f32(h0), f1 = e4m3x2_to_f32(h1);
          hi[j] = h0 | h1 << 16;
          lo[j] = f32_to_e5m2x2(y[0] - f0.x, y[1] - f0.y) | f32_to_e5m2x2(y[2] - f1.x, y[3] - f1.y) << 16;
        }
        tmem_st8(dst + c, hi);
        tmem_st8(dst + 32 + c, lo);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sh.q_full[pn & 1]));
      return bad ? NAN : a.scale * 1.44269504088896341f * exp2f((float)(e - 7));
    };
    float rs_next = load_q(pc, 0);
    uint32_t i = 0, pn = 0;
    bool first = true;
    for (;; ++pn) {
      const float rs = rs_next;
      Kv8Piece nx = pc;
      if (pc.left > 0) {
        kv8_next_piece<KT_TOKENS, KT_ROWS>(a, nx);
        rs_next = load_q(nx, pn + 1);
      }
      const int tk = pc.qt * tpt + r / group;
      const bool live = r < tpt * group && tk < pc.r.n;
      const bool quiet = !__any_sync(0xffffffffu, live);       // no row of this warp: only the barriers
      const int open = a.mask == DFLASH_MASK_NONE ? pc.r.len : max(0, pc.r.len - pc.r.n);
      const float fac = live && rs == rs ? rs : 0.f;
      float m_used = -INFINITY, l = 0.f;
      for (int u = pc.u0; u < pc.u1; ++u, ++i) {
        const int par = i & 1;
        const bool got = __all_sync(0xffffffffu, ok && wait(sh.s_full[par], i >> 1));
        const uint32_t sa = lane_base + par * 128 + half * 64;   // my 64 tokens: page 2 u + half
        float sc[64];
        float mt = -INFINITY;
        const KtSide &sd = sh.side[i % KT_SIDE];
        float c = 0.f, ev = 0.f, iv = 1.f;
        if (got && !quiet) {
          const int page = sd.page[half];
          c = fac * sd.ks[half];
          ev = log2f(sd.vs[half]);
          iv = 1.f / sd.vs[half];
          tc_fence_after();
#pragma unroll
          for (int c0 = 0; c0 < 64; c0 += 16) {
            uint32_t t[16];
            tmem_ld16(sa + c0, t);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) sc[c0 + j] = __uint_as_float(t[j]);
          }
          const int pgn = 2 * u + half;
          if (page < 0 || (pgn + 1) * KV_PAGE > open) {
            const uint64_t see = page < 0 || !live ? 0 : kv8_visible(a, pc.r, tk, pgn);
            const uint32_t s0 = (uint32_t)see, s1 = (uint32_t)(see >> 32);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (!(s0 >> j & 1)) sc[j] = -INFINITY;
              if (!(s1 >> j & 1)) sc[32 + j] = -INFINITY;
            }
          }
#pragma unroll
          for (int j = 0; j < 64; ++j) mt = fmaxf(mt, sc[j]);
          mt = mt == -INFINITY ? mt : fmaf(mt, c, ev);
        }
        sh.xmax[par][half][r] = mt;
        if (lane == 0) sh.xok[par][half][q] = got;
        pair_sync(1 + q);
        const float mp = sh.xmax[par][half ^ 1][r];
        ok = got && *(volatile int *)&sh.xok[par][half ^ 1][q] != 0;
        if (!ok) break;
        mt = fmaxf(mt, mp);
        if (u == pc.u0) {
          m_used = mt;
        } else if (__any_sync(0xffffffffu, mt > m_used + 8.f)) {
          const float m_new = fmaxf(m_used, mt);
          const float corr = m_used == -INFINITY ? 0.f : ex2(m_used - m_new);
          m_used = m_new;
          // P.V of the previous tile must have retired (the one before it has: its end preceded this S)
          if (!__all_sync(0xffffffffu, wait(sh.pv_done, i - 1))) {
            ok = false;                                // the partner learns of it at the next exchange
            continue;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < HD / 2; c0 += 16) {
            uint32_t t[16];
            const uint32_t oa = lane_base + TM_O + (HD / 2) * half + c0;
            tmem_ld16(oa, t);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) t[j] = __float_as_uint(__uint_as_float(t[j]) * corr);
            tmem_st16(oa, t);
          }
          l *= corr;
        }
        if (!quiet) {
          const float off = ev - (m_used == -INFINITY ? 0.f : m_used) + KT_BIAS;
          float sum = 0.f;
#pragma unroll
          for (int c0 = 0; c0 < 64; c0 += 32) {
            uint32_t pw[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float s0 = sc[c0 + 2 * j], s1 = sc[c0 + 2 * j + 1];
              // (a factor of zero must not meet the -infinity of a hidden token: such rows are not written)
              const float e0 = ex2(fmaf(s0, c, off)), e1 = ex2(fmaf(s1, c, off));
              sum += e0 + e1;
              pw[j] = pack_f16(e0, e1);
            }
            tmem_st16(sa + c0 / 2, pw);
          }
          l = fmaf(sum, iv, l);
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.p_full[par]));
      }
      // the row's sum over both halves (run by both warps of the pair)
      sh.xsum[half][r] = l;
      if (lane == 0) sh.xok[0][half][q] = ok;
      pair_sync(1 + q);
      float l_row = l + sh.xsum[half ^ 1][r];
      ok = ok && *(volatile int *)&sh.xok[0][half ^ 1][q] != 0;
      pair_sync(1 + q);
      ok = __all_sync(0xffffffffu, ok && wait(sh.o_full, pn));
      tc_fence_after();
      const bool whole = pc.u1 - pc.u0 == pc.units;
      const size_t slot = 2 * blockIdx.x + (first ? 0 : 1);
      const size_t at = (size_t)(pc.r.row0 + tk) * a.nq + pc.h * group + r % group;
      if (!ok || rs != rs) l_row = NAN;
      const bool nan_v = ok && *(volatile int *)&sh.nan_piece[pn & 3] == (int)pn + 1;
      if (live && half == 0) {
        if (!whole) *(float2 *)(a.part_ml + (slot * KT_ROWS + r) * 2) = make_float2(m_used - KT_BIAS, l_row);
        else if (a.lse) a.lse[at] = l_row == 0.f ? -INFINITY : (m_used - KT_BIAS + log2f(l_row)) * LN2;
      }
      const float inv = l_row == 0.f ? 0.f : 1.f / l_row;
#pragma unroll 1
      for (int c0 = 0; c0 < HD / 2; c0 += 16) {
        uint32_t t[16];
        if (ok) {
          tmem_ld16(lane_base + TM_O + (HD / 2) * half + c0, t);
          tmem_ld_wait();
        }
        if (!live) continue;
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = ok ? __uint_as_float(t[j]) : NAN;
        const int d0 = (HD / 2) * half + c0;
        if (nan_v) {                                   // rows that see a NaN value get it (rare)
          uint32_t hit = 0;
          const int lim = Tiles(a).limit(pc.r, pc.qt);
#pragma unroll 1
          for (int x = max(2 * pc.u0, open / KV_PAGE); x < 2 * pc.u1 && (long long)x * KV_PAGE < lim; ++x) {
            const int page = a.table[(size_t)pc.b * a.width + x];
            if (page < 0 || page >= a.n_pages) continue;
            const uint64_t see = kv8_visible(a, pc.r, tk, x);
            const uint8_t *vb = a.vp + kv8_block(page, pc.h, a.nkv, HD);
#pragma unroll 1
            for (int z = 0; z < 16 * KV_PAGE; ++z)
              if ((see >> (z % KV_PAGE) & 1) && (vb[(d0 + z / KV_PAGE) * KV_PAGE + z % KV_PAGE] & 0x7f) == 0x7f) hit |= 1u << z / KV_PAGE;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (hit >> j & 1) v[j] = NAN;
        }
        if (whole) {
          uint32_t h[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j] * inv, v[2 * j + 1] * inv);
            h[j] = *(const uint32_t *)&b;
          }
          uint4 *dst = (uint4 *)((bf16 *)a.out + at * HD + d0);
          dst[0] = make_uint4(h[0], h[1], h[2], h[3]);
          dst[1] = make_uint4(h[4], h[5], h[6], h[7]);
        } else {
          float4 *dst = (float4 *)(a.part_o + (slot * KT_ROWS + r) * HD + d0);
#pragma unroll
          for (int j = 0; j < 4; ++j) dst[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sh.o_empty));
      if (pc.left <= 0) break;
      pc = nx;
      first = false;
    }
  } else {
    // ---------------- V pages to f16: [hd][64 tokens] of 128-byte rows in the 128-byte swizzle
    const int tid = threadIdx.x - 320;
    uint32_t i = 0;
    bool go = true;
    for (uint32_t pn = 0; go; ++pn) {
      const int open = a.mask == DFLASH_MASK_NONE ? pc.r.len : max(0, pc.r.len - pc.r.n);
      for (int u = pc.u0; u < pc.u1; ++u, ++i) {
        const int stg = i % KT_STAGES, par = i & 1;
        go = wait(sh.vfull[stg], i / KT_STAGES) && (i < 2 || wait(sh.w_empty[par], (i >> 1) - 1));
        go = __all_sync(0xffffffffu, go);
        if (!go) break;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const bool there = sh.side[i % KT_SIDE].page[x] >= 0;
          const int p0 = (2 * u + x) * KV_PAGE;        // the page's first token
          const bool partial = p0 + KV_PAGE > open;
          const uint32_t src = base + Lay::V0 + (2 * stg + x) * Lay::PAGE8, dst = base + Lay::W0 + (2 * par + x) * Lay::PAGE16;
          bool nan = false;
#pragma unroll
          for (int j = 0; j < HD * 4 / KT_WIDEN; ++j) {   // 16 tokens of one dim at a time
            const int it = tid + KT_WIDEN * j, d = it >> 2, c = it & 3;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (there) v = lds128(src + it * 16);
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            if (partial) {
              const int tail = pc.r.len - p0 - 16 * c;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int n = tail - 4 * k;            // tokens that exist: the rest may be anything
                w[k] = n >= 4 ? w[k] : n <= 0 ? 0u : w[k] & ((1u << 8 * n) - 1);
                const uint32_t nb = nan_bytes(w[k]);   // must not meet the zero weight of a row that does not see it
                nan |= nb != 0;
                w[k] &= ~byte_mask(nb);
              }
            }
            uint32_t f[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              f[2 * k] = e4m3x2_to_f16x2(w[k]);
              f[2 * k + 1] = e4m3x2_to_f16x2(w[k] >> 16);
            }
            sts128(dst + d * 128 + (((2 * c) ^ (d & 7)) << 4), f);
            sts128(dst + d * 128 + (((2 * c + 1) ^ (d & 7)) << 4), f + 4);
          }
          if (nan) *(volatile int *)&sh.nan_piece[pn & 3] = (int)pn + 1;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(sh.w_full[par]));
          mbar_arrive(bar(sh.vempty[stg]));
        }
      }
      if (!go || pc.left <= 0) break;
      kv8_next_piece<KT_TOKENS, KT_ROWS>(a, pc);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

namespace {
template <int HD>
cudaError_t launch(const KtParams &p, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(k_kv8_attn_tiles<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kt_smem<HD>());
  if (e == cudaSuccess) e = launch_pdl(k_kv8_attn_tiles<HD>, dim3(KV8_SMS), dim3(KT_THREADS), kt_smem<HD>(), s, p);
  if (e == cudaSuccess)
    e = launch_pdl(k_kv8_combine<bf16, HD, KT_TOKENS, KT_ROWS>, dim3(KV8_SMS - 1, 8), dim3(128), 0, s, p.a);
  return e;
}
}  // namespace

cudaError_t launch_kv8_tiles(const Kv8AttnArgs &a, int hd, cudaStream_t s) {
  void *fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
  if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
  typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                             const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  KtParams p;
  p.a = a;
  // K pages as [page x head][64 tokens][hd bytes], one block per box
  const cuuint64_t dims[3] = {(cuuint64_t)hd, KV_PAGE, (cuuint64_t)a.n_pages * a.nkv};
  const cuuint64_t strides[2] = {(cuuint64_t)hd, (cuuint64_t)hd * KV_PAGE};
  const cuuint32_t box[3] = {(cuuint32_t)hd, KV_PAGE, 1}, ones[3] = {1, 1, 1};
  const CUresult r = ((Encode)fn)(&p.kmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, (void *)a.kp, dims, strides, box, ones,
                                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                                  hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
  return hd == 128 ? launch<128>(p, s) : launch<64>(p, s);
}

}  // namespace dflash
