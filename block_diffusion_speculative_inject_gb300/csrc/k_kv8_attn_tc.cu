// Attention over the 8-bit paged cache for many query rows per kv head (bf16): verify blocks, draft
// trees, prompt chunks. One persistent CTA per SM walks its share of the work (kv8_sched.cuh) in tiles
// of 128 rows (tokens x query heads of the kv head) and 128 tokens (two pages):
//   S[128, 128] = Q . K^T        kind::f8f6f4, both operands in shared memory, the K pages as they are
//   P = 2^(S c + log2 s_v - m)   f16, written over S
//   O[128, hd] += P . V          kind::f16, A = P in tensor memory, B = V pages widened to f16
// Q's row, scaled by a power of two so that its largest entry is in [128, 256), is the sum of an e4m3 and
// an e5m2 part: bf16 has 8 significant bits, e4m3 takes 4, and what rounding to nearest leaves is at
// most 8 units of the last place, which e5m2's 3 bits hold exactly. So K needs no conversion, and q is
// exact for entries down to 2^-6 scaled, 2^-13 of the row's largest. Below, e4m3 is subnormal and leaves up to 16
// units and more, and e5m2 rounds those by 2^-14 at most: 2^-21 of the row's largest.
// P could not go the same way: rows with one loud token and many quiet ones need its small values, so
// P is f16 (11 bits, largest 2^7 .. 2^15, normal to 2^-14) and two warps widen V (exact) into a second
// pair of tiles. That costs shared-memory traffic of 3x V's bytes per tile, 176 KB in all with the MMAs'
// own reads, 1400 cycles at 128 B/clk against 1400 that an SM's share of HBM takes for the tile's 32 KB.
//
// The running maximum is lazy: O is rescaled only when a row's maximum grows by more than 2^8. The
// pages' scales enter as in the few-row kernel: s_k in c, s_v in the exponent of P.
//
// Tensor memory (512 columns): S/P at 0, 128 and 256 (tile modulo 3), O at 384. P of a page's 64 tokens lies in
// the first 32 of their own 64 columns of S. With three buffers S of tile i + 2 need not wait for P.V of tile i;
// with Q in tensor memory and two, the block below took 134 us and the trees 146.
//
// Roles (384 threads, 168 registers): warp 0 copies K (TMA, 128- or 64-byte swizzle) and V (bulk, as stored)
// into rings of 3 tiles, is ahead of all, finds the pieces and leaves them in a ring. Warp 1 issues the MMAs, S
// two tiles ahead of P.V within a piece; it runs converged, with the MMAs themselves predicated on one
// lane, which leaves the descriptors to the uniform datapath (a lone lane took over twice as long to issue a
// tile as the tensor cores take to do it). Warps 2-9 run the softmax, two threads per row, one page each:
// warps w and w + 4 share the rows of lane quarter w % 4 and trade their maxima. They also load Q (of the
// next piece as soon as S of this one's last tile is there) and write results, half of the dims each, in both
// four lanes to a row. Warps 10-11 widen V. All waits are bounded; rows whose wait ran out become NaN.
//
// Code that runs once a piece is mostly fetched rather than run, so what is not a tile's inner work is
// rolled up: V widened a page at a time took the trees from 168 to 148 us. Measured, with the merge: 8 x 16
// rows x 40 heads over 32768 tokens 126 us (537 MB, 4.3 TB/s), 8 trees of 256 rows x 32 heads over 1000 .. 5000
// tokens 134 us; about 1700 cycles a tile, of which the MMAs are 1030 and the softmax's arithmetic 840. No one part
// bounds it: the block takes 116 us without the trade of maxima, 119 without exponentials or without the widening,
// 120 and 123 with a quarter of the products of S and of P.V, 103 without loads of S and stores of P.
#include "kv8_attn.cuh"

namespace dflash {

constexpr int KT_TOKENS = 128;                         // tokens of a tile: two pages
constexpr int KT_THREADS = 384;
constexpr int KT_WIDEN = 64;                           // threads that widen V
constexpr int KT_STAGES = 3;
constexpr int KT_SIDE = 8;                             // tiles whose page ids and scales are kept
constexpr int KT_COST = 8;                             // what an item's start and end cost, in tiles (measured on the
                                                       // trees above alone: 141 us with 4, 134 with 6 and 8, 138 with 12)
constexpr int KT_RING = 16;                            // pieces kept: the one found last is at most 7 ahead of the one written
constexpr float KT_BIAS = 7.f;
constexpr uint32_t TM_O = 384;

struct KtParams {
  CUtensorMap kmap;
  Kv8AttnArgs a;
};

template <int HD>
struct KtLayout {
  static constexpr uint32_t PAGE8 = KV_PAGE * HD;      // a K or V page, 8 bits
  static constexpr uint32_t PAGE16 = KV_PAGE * HD * 2; // a V page in f16
  static constexpr uint32_t K0 = 0, V0 = K0 + KT_STAGES * 2 * PAGE8, W0 = V0 + KT_STAGES * 2 * PAGE8;
  static constexpr uint32_t PLANE = 128 * HD;          // Q's e4m3 part; the e5m2 part follows
  static constexpr uint32_t Q0 = W0 + 2 * 2 * PAGE16, OUT0 = Q0 + 2 * PLANE, END = OUT0 + 8 * 2048;   // per softmax warp 32 rows x 64 bytes of results
};

struct KtSide {
  int page[2];                                         // -1: not there, nothing of it is seen
  float ks[2], ev[2], iv[2];                           // K's scale, log2 of V's and 1 over it
};

struct KtShared {
  uint64_t kfull[KT_STAGES], kempty[KT_STAGES], vfull[KT_STAGES], vempty[KT_STAGES];
  uint64_t s_full[3], p_full[3], w_full[2], pv_done[2], q_full, o_full, o_empty, drain[1];
  uint64_t x_ready[2][4];                              // maxima traded: per tile parity and lane quarter
  uint64_t l_ready[2][2][4];                           // row sums: per piece parity, half and lane quarter
  KtSide side[KT_SIDE];
  float xmax[2][2][128], lsum[2][2][128];              // per tile (piece) parity, half and row
  int xgrow[2][2][4];                                  // a row of the warp outgrew its reference
  uint64_t known[KT_RING];
  Kv8Piece ring[KT_RING];                              // pieces by ordinal, found by the copying warp for all
  Kv8Piece piece[8];                                   // of each softmax warp (it has no registers to spare)
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
// MMAs and commits of the one thread with `lead` set; the whole warp runs them. hi: the descriptors' upper word
__device__ __forceinline__ void mma_f8(uint32_t lead, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc) {
  asm volatile("{\n .reg .pred p, q;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n setp.ne.b32 q, %6, 0;\n mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
               " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, p;\n}\n" ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(hi),
               "r"(idesc), "r"(acc), "r"(lead) : "memory");
}
__device__ __forceinline__ void mma_f16(uint32_t lead, uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, uint32_t acc) {
  asm volatile("{\n .reg .pred p, q;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n setp.ne.b32 q, %6, 0;\n mov.b64 b, {%2, %3};\n"
               " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(d), "r"(a), "r"(b_lo), "r"(b_hi),
               "r"(idesc), "r"(acc), "r"(lead) : "memory");
}
__device__ __forceinline__ void commit_lead(uint32_t lead, uint32_t mbar) {
  asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
               " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(mbar), "r"(lead) : "memory");
}
// K-major descriptor of rows of 64 bytes in the 64-byte swizzle: 8-row atoms of 512 bytes
__device__ __forceinline__ uint64_t sw64_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(512 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)4 << 61;
}
// D fp32, M = 128, N columns; A and B formats as the kind numbers them
constexpr uint32_t idesc_of(int a_fmt, int b_fmt, int N) {
  return (1u << 4) | (uint32_t)a_fmt << 7 | (uint32_t)b_fmt << 10 | (uint32_t)(N >> 3) << 17 | (128u >> 4) << 24;
}
// 32 columns of this thread's lane, without the wait
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *r) {
  uint32_t *u = (uint32_t *)r;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
      "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]), "=r"(u[9]),
        "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]),
        "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]),
        "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr));
}
// (a.x * b + c, a.y * b + c) and a + b in one paired instruction each
__device__ __forceinline__ float2 fma2(float2 a, float b, float c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %4};\n mov.b64 z, {%5, %5};\n fma.rn.f32x2 x, x, y, z;\n"
      " mov.b64 {%0, %1}, x;\n}\n" : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t *w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}

template <int HD>
__global__ void __launch_bounds__(KT_THREADS, 1) k_kv8_attn_tiles(const __grid_constant__ KtParams p) {
  typedef KtLayout<HD> Lay;
  typedef Kv8Tiles<KT_TOKENS, KT_ROWS, KT_COST> Tiles;
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
      mbar_init(bar(sh.w_full[i]), KT_WIDEN / 32);
      mbar_init(bar(sh.pv_done[i]), 1);
      for (int j = 0; j < 4; ++j) {
        mbar_init(bar(sh.x_ready[i][j]), 2);
        mbar_init(bar(sh.l_ready[i][0][j]), 1);
        mbar_init(bar(sh.l_ready[i][1][j]), 1);
      }
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(bar(sh.s_full[i]), 2);                 // the MMAs, and their issuer for the side words that it has seen
      mbar_init(bar(sh.p_full[i]), 8);
    }
    mbar_init(bar(sh.q_full), 8);
    for (int i = 0; i < KT_RING; ++i) mbar_init(bar(sh.known[i]), 1);
    mbar_init(bar(sh.o_full), 1);
    mbar_init(bar(sh.drain[0]), 1);
    mbar_init(bar(sh.o_empty), 8);
    sh.abort = 0;
    for (int i = 0; i < 4; ++i) sh.nan_piece[i] = 0;
    fence_mbar_init();
  }
  pdl_wait();
  long long chunk, item_begin;
  Kv8Piece pc;
  if (!kv8_start<KT_TOKENS, KT_ROWS, KT_COST>(a, sh.grp, blockIdx.x, gridDim.x, pc, chunk, item_begin)) {   // uniform for the CTA
    if (threadIdx.x == 0) a.desc[blockIdx.x].pieces = 0;
    return;
  }
  if (threadIdx.x == 0) a.desc[blockIdx.x] = kv8_desc<KT_TOKENS, KT_ROWS, KT_COST>(a, pc, blockIdx.x, chunk, item_begin);
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int *abort_flag = (volatile int *)&sh.abort;
  auto wait = [&](uint64_t &b, uint32_t parity) { return kv8_wait(bar(b), parity & 1, abort_flag); };
  auto known = [&](uint32_t n) { return __all_sync(0xffffffffu, wait(sh.known[n % KT_RING], n / KT_RING)) != 0; };

  if (warp == 0) {
    // ---------------- copies
    if (lane == 0) tma_prefetch_map(&p.kmap);
    uint32_t i = 0;
    bool go = true;
    auto publish = [&](const Kv8Piece &x, uint32_t n) {
      if (lane == 0) {
        sh.ring[n % KT_RING] = x;
        mbar_arrive(bar(sh.known[n % KT_RING]));
      }
    };
    // lane x: page x (and its scales) of 16 tiles of a piece, and of the 16 after them (of the next
    // piece's first), whose table entries and then scales are fetched while these are used
    auto table = [&](const Kv8Piece &x, int from) {
      const int pg = 2 * from + lane;
      return (long long)pg * KV_PAGE < Tiles(a).limit(x.r, x.qt) && pg < 2 * x.u1 ? a.table[(size_t)x.b * a.width + pg] : -1;
    };
    auto scales = [&](int h, int &pg, float &k, float &v) {
      if (pg < 0 || pg >= a.n_pages) pg = -1;
      k = v = 1.f;
      if (pg >= 0) {
        k = a.ks[(size_t)pg * a.nkv + h];
        v = a.vs[(size_t)pg * a.nkv + h];
      }
    };
    float ks, vs, next_ks = 1.f, next_vs = 1.f, piece_ks = 1.f, piece_vs = 1.f;
    int page = table(pc, pc.u0), next_page = -1, piece_page = -1;
    publish(pc, 0);
    scales(pc.h, page, ks, vs);
    Kv8Piece nx = pc;
    for (uint32_t pn = 0;; ++pn) {
      int tab_u = pc.u0;
      float ev = log2f(vs), iv = 1.f / vs;
      for (int u = pc.u0; u < pc.u1 && go; ++u, ++i) {
        if (u == tab_u + 16) {
          tab_u = u;
          page = next_page;
          ks = next_ks;
          ev = log2f(next_vs);
          iv = 1.f / next_vs;
        }
        if (u == tab_u + 4) next_page = table(pc, tab_u + 16);
        if (u == tab_u + 10) scales(pc.h, next_page, next_ks, next_vs);
        const int at = 2 * (u - tab_u), stg = i % KT_STAGES;
        const uint32_t use = i / KT_STAGES;
        go = use == 0 || (wait(sh.kempty[stg], use - 1) && wait(sh.vempty[stg], use - 1));
        go = __all_sync(0xffffffffu, go);
        if (!go) break;
        const int x = lane - at;                       // the two lanes that hold the tile's pages write and copy them
        const unsigned there = __popc(__ballot_sync(0xffffffffu, (x == 0 || x == 1) && page >= 0));
        if (x == 0 || x == 1) {
          KtSide &sd = sh.side[i % KT_SIDE];
          sd.page[x] = page;
          sd.ks[x] = ks;
          sd.ev[x] = ev;
          sd.iv[x] = iv;
        }
        __syncwarp();
        if (lane == 0) {
          if (there) {
            mbar_expect_tx(bar(sh.kfull[stg]), there * Lay::PAGE8);
            mbar_expect_tx(bar(sh.vfull[stg]), there * Lay::PAGE8);
          } else {
            mbar_arrive(bar(sh.kfull[stg]));
            mbar_arrive(bar(sh.vfull[stg]));
          }
        }
        __syncwarp();
        if ((x == 0 || x == 1) && page >= 0) {
          tma_load_3d(base + Lay::K0 + (2 * stg + x) * Lay::PAGE8, &p.kmap, 0, 0, page * a.nkv + pc.h, bar(sh.kfull[stg]));
          bulk_load(base + Lay::V0 + (2 * stg + x) * Lay::PAGE8, a.vp + kv8_block(page, pc.h, a.nkv, HD), Lay::PAGE8, bar(sh.vfull[stg]));
        }
        if (pc.left > 0) {
          if (u == pc.u0) {
            kv8_next_piece<KT_TOKENS, KT_ROWS, KT_COST>(a, nx);
            publish(nx, pn + 1);
            piece_page = table(nx, nx.u0);
          }
          if (u == min(pc.u0 + 1, pc.u1 - 1)) scales(nx.h, piece_page, piece_ks, piece_vs);
        }
      }
      if (!go || pc.left <= 0) break;
      pc = nx;
      page = piece_page;
      ks = piece_ks;
      vs = piece_vs;
    }
    // copies in flight end before the CTA does (bounded; at once unless a wait ran out)
    const unsigned long long t0 = global_ns();
    for (uint32_t j = i > KT_STAGES ? i - KT_STAGES : 0; j < i; ++j)
      while (!(mbar_try_wait(bar(sh.kfull[j % KT_STAGES]), j / KT_STAGES & 1) &&
               mbar_try_wait(bar(sh.vfull[j % KT_STAGES]), j / KT_STAGES & 1)) && global_ns() - t0 < TC_WAIT_NS) {
      }
  } else if (warp == 1) {
    // ---------------- MMAs
    constexpr uint32_t idS0 = idesc_of(0, 0, KT_TOKENS), idS1 = idesc_of(1, 0, KT_TOKENS), idO = idesc_of(0, 0, HD);
    const uint32_t lead = lane == 0;
    auto wait_all = [&](uint64_t &b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };
    const uint64_t k0 = HD == 128 ? sw128_desc(base + Lay::K0) : sw64_desc(base + Lay::K0), w0 = sw128_desc(base + Lay::W0);
    const uint32_t k_hi = (uint32_t)(k0 >> 32), w_hi = (uint32_t)(w0 >> 32);
    const uint32_t qd = (uint32_t)k0 + ((Lay::Q0 - Lay::K0) >> 4);
    uint32_t si = 0;                                   // tiles whose S is issued
    auto issue_s = [&]() {
      const uint32_t stg = si % KT_STAGES, sb = si % 3;
      if (!wait_all(sh.kfull[stg], si / KT_STAGES)) return false;
      tc_fence_after();
      const uint32_t kd = (uint32_t)k0 + stg * (2 * Lay::PAGE8 >> 4), d = tmem + sb * 128;
#pragma unroll
      for (int pl = 0; pl < 2; ++pl)
#pragma unroll
        for (int k = 0; k < HD / 32; ++k)
          mma_f8(lead, d, qd + pl * (Lay::PLANE >> 4) + 2 * k, kd + 2 * k, k_hi, pl ? idS1 : idS0, (pl | k) ? 1u : 0u);
      commit_lead(lead, bar(sh.s_full[sb]));
      commit_lead(lead, bar(sh.kempty[stg]));
      if (lead) mbar_arrive(bar(sh.s_full[sb]));
      ++si;
      return true;
    };
    bool go = true;
    uint32_t i = 0;
    for (uint32_t pn = 0; go; ++pn) {
      if (!(go = known(pn) && wait_all(sh.q_full, pn))) break;
      const Kv8Piece &now = sh.ring[pn % KT_RING];
      const int n = now.u1 - now.u0;
      for (int x = -2; x < n; ++x) {                   // S two tiles ahead of P.V, within the piece
        if (x + 2 < n && !(go = issue_s())) break;
        if (x < 0) continue;
        const uint32_t par = i & 1, sb = i % 3;
        if (!(go = wait_all(sh.w_full[par], i >> 1))) break;
        if (x == 0 && pn > 0 && !(go = wait_all(sh.o_empty, pn - 1))) break;
        if (!(go = wait_all(sh.p_full[sb], i / 3))) break;
        tc_fence_after();
        const uint32_t wd = (uint32_t)w0 + par * (2 * Lay::PAGE16 >> 4), pa = tmem + sb * 128;
#pragma unroll
        for (int k = 0; k < 8; ++k)                    // 16 tokens each; k >> 2: the page
          mma_f16(lead, tmem + TM_O, pa + 64 * (k >> 2) + 8 * (k & 3), wd + (k >> 2) * (Lay::PAGE16 >> 4) + (k & 3) * 2, w_hi, idO,
                  k ? 1u : (uint32_t)(x > 0));
        commit_lead(lead, bar(sh.pv_done[par]));
        ++i;
      }
      if (!go) break;
      commit_lead(lead, bar(sh.o_full));
      if (now.left <= 0) break;
    }
    // MMAs in flight end before the tensor memory is given back
    __syncwarp();
    commit_lead(lead, bar(sh.drain[0]));
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait(bar(sh.drain[0]), 0) && global_ns() - t0 < TC_WAIT_NS) {
    }
  } else if (warp < 10) {
    // ---------------- Q, softmax, results: row r, page `half` of each tile
    const int q = warp & 3, half = (warp - 2) >> 2, r = q * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16);
    const int group = a.nq / a.nkv, tpt = Tiles(a).tpt;
    bool ok = true;
    // writes this half of the dims of Q of a piece; returns the row's factor (NaN: the row holds
    // an infinity or NaN)
    auto load_q = [&](const Kv8Piece &x) {
      const int tk = x.qt * tpt + r / group;
      const unsigned alive = __ballot_sync(0xffffffffu, r < tpt * group && tk < x.r.n);
      constexpr int N = HD / 2, R = N / 32;            // dims of a half, rounds of 64 bytes of each row
      const int64_t from = (int64_t)(x.r.row0 + tk) * a.q_stride + (int64_t)(x.h * group + r % group) * HD;
      // Four lanes read a row, 16 bytes each: this half of 8 rows at a time, the other half for the row's
      // maximum only.
      float factor = NAN;
#pragma unroll 1
      for (int k0 = 0; k0 < 4; k0 += 2) {
        uint4 mine[R][2], other[R][2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int y = 8 * (k0 + k) + (lane >> 2);
          const bf16 *src = (const bf16 *)a.q + __shfl_sync(0xffffffffu, from, y) + 8 * (lane & 3);
          const bool there = alive >> y & 1;
#pragma unroll
          for (int z = 0; z < R; ++z) {
            mine[z][k] = there ? *(const uint4 *)(src + N * half + 32 * z) : make_uint4(0, 0, 0, 0);
            other[z][k] = there ? *(const uint4 *)(src + N * (half ^ 1) + 32 * z) : make_uint4(0, 0, 0, 0);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t top = 0;                            // largest magnitudes of the row's even and odd dims; NaN stays
          auto take = [&](uint32_t e) {
            const __nv_bfloat162 m = __hmax2_nan(*(const __nv_bfloat162 *)&top, __habs2(*(const __nv_bfloat162 *)&e));
            top = *(const uint32_t *)&m;
          };
#pragma unroll
          for (int z = 0; z < R; ++z) {
            take(mine[z][k].x), take(mine[z][k].y), take(mine[z][k].z), take(mine[z][k].w);
            take(other[z][k].x), take(other[z][k].y), take(other[z][k].z), take(other[z][k].w);
          }
          take(__shfl_xor_sync(0xffffffffu, top, 1));
          take(__shfl_xor_sync(0xffffffffu, top, 2));
          const float t0 = __uint_as_float(top << 16), t1 = __uint_as_float(top & 0xffff0000u);
          const bool fin = t0 <= 3.402823466e38f && t1 <= 3.402823466e38f;
          const int e = fin ? max(-100, (int)(__float_as_uint(fmaxf(t0, t1)) >> 23) - 127) : 0;
          const float up = __uint_as_float((uint32_t)(134 - e) << 23);           // 2^(7 - e)
          const uint32_t keep = fin ? ~0u : 0u;
          const int y = q * 32 + 8 * (k0 + k) + (lane >> 2), swz = HD == 128 ? y & 7 : y >> 1 & 3;
#pragma unroll
          for (int z = 0; z < R; ++z) {
            const uint32_t w[4] = {mine[z][k].x, mine[z][k].y, mine[z][k].z, mine[z][k].w};
            uint32_t h[4], l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {              // f16 holds the scaled value and the difference exactly
              const uint32_t v = w[j] & keep, x16 = pack_f16(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xffff0000u) * up);
              h[j] = f16x2_to_e4m3x2(x16);
              l[j] = f16x2_to_e5m2x2(sub_f16x2(x16, e4m3x2_to_f16x2(h[j])));
            }
            const int c = (N * half + 32 * z) / 16 + (lane >> 1 & 1);          // 16-byte chunk of the row
            const uint32_t dst = base + Lay::Q0 + y * HD + 16 * (c ^ swz) + 8 * (lane & 1);
            sts64(dst, h[0] | h[1] << 16, h[2] | h[3] << 16);
            sts64(dst + Lay::PLANE, l[0] | l[1] << 16, l[2] | l[3] << 16);
          }
          const float f = fin ? a.scale * 1.44269504088896341f * __uint_as_float((uint32_t)(120 + e) << 23) : NAN;
          const float own = __shfl_sync(0xffffffffu, f, 4 * (lane & 7));         // of row 8 k + lane % 8
          if (lane >> 3 == k0 + k) factor = own;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sh.q_full));
      return factor;
    };
    Kv8Piece &mine = sh.piece[warp - 2];
    auto keep = [&](const Kv8Piece &x) {
      __syncwarp();
      if (lane == 0) mine = x;
      __syncwarp();
    };
    keep(pc);
    uint32_t i = 0, pn = 0;                            // tile and piece ordinals
    float rs_next = load_q(pc);
    bool first = true;
    for (;; ++pn) {
      const float rs = rs_next;
      const int tk = mine.qt * tpt + r / group;
      const bool live = r < tpt * group && tk < mine.r.n;
      const bool quiet = !__any_sync(0xffffffffu, live);       // no row of this warp: only the barriers
      const int u0 = mine.u0, u1 = mine.u1;
      // pages from `open` on hold a token that some row of the request does not see
      const int open = (a.mask == DFLASH_MASK_NONE ? mine.r.len : max(0, mine.r.len - mine.r.n)) / KV_PAGE;
      const float fac = live && rs == rs ? rs : 0.f;
      float m_used = -INFINITY, l = 0.f;
      for (int u = u0; u < u1; ++u, ++i) {
        const int par = i & 1, sb = i % 3;
        ok = __all_sync(0xffffffffu, ok && wait(sh.s_full[sb], i / 3));
        if (!ok) break;
        const uint32_t sa = lane_base + sb * 128 + half * 64;    // my 64 tokens
        const KtSide &sd = sh.side[i % KT_SIDE];
        // Never zero, so that the -infinity of a hidden token stays one: a row of zeros (factor 2^-110 or so) and a page of
        // zero keys (scale 2^-64) would underflow. |S| is below 2^24, so a score moves by 2^-102 at most. (A maximum in
        // place of the sum, an instruction more on the way to P, cost 1% of the time.)
        const float c = fmaf(fac, sd.ks[half], 1.17549435e-38f), ev = sd.ev[half];
        const bool partial = sd.page[half] < 0 || 2 * u + half >= open;
        // S of my tokens, without what the row does not see
        auto load_s = [&](float *sc) {
          tmem_ld32(sa, sc);
          tmem_ld32(sa + 32, sc + 32);
          tmem_ld_wait();
          if (partial) {
            const uint64_t see = live && sd.page[half] >= 0 ? kv8_visible(a, mine.r, tk, 2 * u + half) : 0;
            const uint32_t s0 = (uint32_t)see, s1 = (uint32_t)(see >> 32);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (!(s0 >> j & 1)) sc[j] = -INFINITY;
              if (!(s1 >> j & 1)) sc[32 + j] = -INFINITY;
            }
          }
        };
        // P of 32 tokens for the present reference, as f16 pairs; returns their sum
        auto exps = [&](const float *v, uint32_t *pw) {
          const float off = ev + KT_BIAS - (m_used == -INFINITY ? 0.f : m_used);
          float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float2 e = fma2(make_float2(v[2 * j], v[2 * j + 1]), c, off);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            sum[j & 1] = add2(sum[j & 1], e);
            pw[j] = pack_f16(e.x, e.y);
          }
          sum[0] = add2(sum[0], sum[1]);
          return sum[0].x + sum[0].y;
        };
        float sc[64];
        uint32_t pw[16];
        float mt = -INFINITY, sum = 0.f;
        if (!quiet) {
          tc_fence_after();
          load_s(sc);
          float mx[4];                                 // four chains, three values a step
#pragma unroll
          for (int j = 0; j < 4; ++j) mx[j] = fmaxf(sc[16 * j], sc[16 * j + 1]);
#pragma unroll
          for (int k = 2; k < 16; k += 2)
#pragma unroll
            for (int j = 0; j < 4; ++j) mx[j] = fmaxf(fmaxf(mx[j], sc[16 * j + k]), sc[16 * j + k + 1]);
          mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          mt = mt == -INFINITY ? mt : fmaf(mt, c, ev);
        }
        // The maxima are traded with the other half's warp. A first tile waits for them; any other keeps the
        // reference and makes half of its P meanwhile, in vain only if some row of the pair outgrew
        // its reference by 2^8.
        bool grow = u == u0 || __any_sync(0xffffffffu, mt > m_used + 8.f);
        sh.xmax[par][half][r] = mt;
        if (lane == 0) sh.xgrow[par][half][q] = grow;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.x_ready[par][q]));
#pragma unroll 1
        for (bool traded = false;; traded = true) {    // (one copy of the code for before and after the trade)
          if ((traded || !grow) && !quiet) sum = exps(sc, pw);
          if (traded) break;
          ok = __all_sync(0xffffffffu, wait(sh.x_ready[par][q], i >> 1));
          if (!ok) break;
          grow = grow || *(volatile int *)&sh.xgrow[par][half ^ 1][q] != 0;
          if (!grow) break;
          const float m_new = fmaxf(m_used, fmaxf(mt, sh.xmax[par][half ^ 1][r]));
          const float corr = m_used == -INFINITY ? 0.f : ex2(m_used - m_new);
          m_used = m_new;
          if (u == u0) continue;
          // O so far is scaled down (P.V of the tile before must be done; this one's waits for this warp)
          l *= corr;
          ok = __all_sync(0xffffffffu, wait(sh.pv_done[par ^ 1], (i - 1) >> 1));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < HD / 2; c0 += 16) {
            const uint32_t oa = lane_base + TM_O + (HD / 2) * half + c0;
            tmem_ld16(oa, pw);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) pw[j] = __float_as_uint(__uint_as_float(pw[j]) * corr);
            tmem_st16(oa, pw);
          }
        }
        if (!ok) break;
        if (!quiet) {
          tmem_st16(sa, pw);
          sum += exps(sc + 32, pw);
          tmem_st16(sa + 16, pw);
          l = fmaf(sum, sd.iv[half], l);
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.p_full[sb]));
      }
      // the next piece's Q: this one's products are done with it, as its last S is there
      if (mine.left > 0 && known(pn + 1)) rs_next = load_q(sh.ring[(pn + 1) % KT_RING]);
      // the row's sum over both halves (by piece parity: the other warp may be a piece ahead)
      const Kv8Piece pc = mine;
      float l_row = 0.f;
      const int pp = pn & 1;
      sh.lsum[pp][half][r] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sh.l_ready[pp][half][q]));
      ok = __all_sync(0xffffffffu, ok && wait(sh.l_ready[pp][half ^ 1][q], pn >> 1));
      if (ok) l_row = sh.lsum[pp][0][r] + sh.lsum[pp][1][r];
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
      // A warp's results go through shared memory, 64 bytes of each row at a time, so that four lanes
      // write a row: a store of one row per lane costs a cycle per row.
      const uint32_t stage = base + Lay::OUT0 + (warp - 2) * 2048;
      const uint32_t put = stage + lane * 64;          // chunk c of row x at c ^ (x >> 1 & 3)
      const int64_t to = whole ? (int64_t)at * HD * 2 : (int64_t)(slot * KT_ROWS + r) * HD * 4;
      uint8_t *dst = whole ? (uint8_t *)a.out : (uint8_t *)a.part_o;
      const unsigned alive = __ballot_sync(0xffffffffu, live);
      auto flush = [&](int byte) {                     // 64 bytes of each row, from `byte` of the row on
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int x = 8 * k + (lane >> 2), c = lane & 3;
          const int64_t row = __shfl_sync(0xffffffffu, to, x);
          const uint4 y = lds128(stage + x * 64 + 16 * (c ^ (x >> 1 & 3)));
          if (alive >> x & 1) *(uint4 *)(dst + row + byte + 16 * c) = y;
        }
        __syncwarp();
      };
#pragma unroll 1
      for (int c0 = 0; c0 < HD / 2; c0 += 16) {
        uint32_t t[16];
        const int d0 = (HD / 2) * half + c0;
        if (quiet) break;
        if (ok) {
          tmem_ld16(lane_base + TM_O + d0, t);
          tmem_ld_wait();
        }
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = ok ? __uint_as_float(t[j]) : NAN;
        if (nan_v && live) {                           // rows that see a NaN value get it (rare)
          uint32_t hit = 0;
          const int lim = Tiles(a).limit(pc.r, pc.qt);
#pragma unroll 1
          for (int x = max(2 * pc.u0, open); x < 2 * pc.u1 && (long long)x * KV_PAGE < lim; ++x) {
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
        uint32_t h[16];
        const int sw = lane >> 1 & 3;
        if (whole) {                                   // 32 bytes of the row: two rounds fill the 64
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j] * inv, v[2 * j + 1] * inv);
            h[j] = *(const uint32_t *)&b;
          }
          const int c = c0 >> 3 & 2;
          sts128(put + 16 * (c ^ sw), h);
          sts128(put + 16 * ((c + 1) ^ sw), h + 4);
          if (c) flush(2 * (d0 - 16));
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) h[j] = __float_as_uint(v[j]);
#pragma unroll
          for (int c = 0; c < 4; ++c) sts128(put + 16 * (c ^ sw), h + 4 * c);
          flush(4 * d0);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sh.o_empty));
      if (pc.left <= 0) break;
      if (known(pn + 1)) {
        keep(sh.ring[(pn + 1) % KT_RING]);
      } else {                                         // a wait ran out: the rows left become NaN all the same
        Kv8Piece nx = pc;
        kv8_next_piece<KT_TOKENS, KT_ROWS, KT_COST>(a, nx);
        keep(nx);
      }
      first = false;
    }
  } else {
    // ---------------- V pages to f16: [hd][64 tokens] of 128-byte rows in the 128-byte swizzle
    const int tid = threadIdx.x - 320;
    uint32_t i = 0;
    bool go = true;
    for (uint32_t pn = 0; go; ++pn) {
      if (!(go = known(pn))) break;
      const Kv8Piece pc = sh.ring[pn % KT_RING];
      const int open = a.mask == DFLASH_MASK_NONE ? pc.r.len : max(0, pc.r.len - pc.r.n);
      for (int u = pc.u0; u < pc.u1; ++u, ++i) {
        const int stg = i % KT_STAGES, par = i & 1;
        go = wait(sh.vfull[stg], i / KT_STAGES) && (i < 2 || wait(sh.pv_done[par], (i >> 1) - 1));
        go = __all_sync(0xffffffffu, go);
        if (!go) break;
        // row d of V^T in 128-byte rows, its 16-byte chunk c at c ^ (d & 7); d & 7 is the same for all j
        const uint32_t c0 = (2 * (tid & 3)) ^ (tid >> 2 & 7), c1 = c0 ^ 1;
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          constexpr int N = HD * 4 / KT_WIDEN;         // pieces of 16 tokens of one dim: all loads first
          uint4 v[N];
          const uint32_t src = base + Lay::V0 + (2 * stg + x) * Lay::PAGE8 + tid * 16;
#pragma unroll
          for (int j = 0; j < N; ++j) v[j] = lds128(src + KT_WIDEN * 16 * j);
          const int page = sh.side[i % KT_SIDE].page[x];
          const long long end = (long long)(2 * u + x + 1) * KV_PAGE;
          if (page < 0 || end > open) {
            // tokens that exist, from this thread's 16: the rest may be anything
            const int tail = page < 0 ? 0 : pc.r.len - (2 * u + x) * KV_PAGE - 16 * (tid & 3);
            uint32_t any = 0;                          // some row does not see some token: a NaN must not meet its zero weight
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int n = tail - 4 * k;
              const uint32_t there = n >= 4 ? ~0u : n <= 0 ? 0u : (1u << 8 * n) - 1;
#pragma unroll
              for (int j = 0; j < N; ++j) {
                uint32_t &w = ((uint32_t *)&v[j])[k];
                w &= there;
                any |= nan_bytes(w);
              }
            }
            if (any) {
#pragma unroll
              for (int j = 0; j < 4 * N; ++j) {
                uint32_t &w = ((uint32_t *)&v[j / 4])[j % 4];
                w &= ~byte_mask(nan_bytes(w));
              }
              *(volatile int *)&sh.nan_piece[pn & 3] = (int)pn + 1;
            }
          }
          const uint32_t dst = base + Lay::W0 + (2 * par + x) * Lay::PAGE16 + (tid >> 2) * 128;
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
            uint32_t f[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) e4m3x4_to_f16(w[k], f[2 * k], f[2 * k + 1]);
            sts128(dst + j * (KT_WIDEN / 4 * 128) + 16 * c0, f);
            sts128(dst + j * (KT_WIDEN / 4 * 128) + 16 * c1, f + 4);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(sh.w_full[par]));
          mbar_arrive(bar(sh.vempty[stg]));
        }
      }
      if (!go || pc.left <= 0) break;
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
    e = launch_pdl(k_kv8_combine<bf16, HD, KT_ROWS>, dim3(KV8_SMS - 1, 16), dim3(128), 0, s, p.a);
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
