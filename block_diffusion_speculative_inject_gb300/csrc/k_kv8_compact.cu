// Kept rows moved down in place in the 8-bit paged cache, in all layers of a model at once (dflash_kv8_compact).
//
// A CTA per (request, kv head, layer, K or V) takes the pages that rows go to one after another, from the first: a row
// goes to its own place or below, so a page's rows come from that page or later ones, and none that is still to
// be read has been written. Per page: the rows' bytes go to shared memory with their pages' scales, the largest
// value gives the page's scale as the append's does, and the bytes are written anew. 8 rows of one layer of 8 x 128 take 4.6 us,
// all latency: lengths, the rows' places, their pages, their bytes. 8 paths of 1 .. 16 rows in 32 layers take 24 us (49 with 256
// threads a CTA that went over the whole page). A page of V keeps the 64 tokens of a dim together, so that a row's 128 values
// lie in as many sectors of 32 bytes: the 67 rows are 9 MB to read and write, their sectors 58 MB (9 us at the copy
// rate; 64 MB by the counters). The rest is that chain, which each of 4096 CTAs goes through for itself in 1.7 waves, though
// its first links are the same for all layers, heads, K and V. 200 rows of each request take 235 us, 48 in one layer.
#include "kv8.cuh"

namespace dflash {

constexpr int KP_THREADS = 128;
constexpr int KP_LAYERS = 128;

struct CompactArgs {
  int width, max_keep, n_pages, nkv;
  const int32_t *base, *keep, *n_keep, *table;
  struct Layer {
    uint8_t *kp, *vp;
    float *ks, *vs;
  } layer[KP_LAYERS];
};

template <int HD>
__global__ void __launch_bounds__(KP_THREADS) k_kv8_compact(const __grid_constant__ CompactArgs a) {
  __shared__ __align__(16) uint8_t tile[KV_PAGE * HD];  // K: [64][HD], V: [HD][64]
  __shared__ int from[KV_PAGE];                        // slot of the row that goes to each place, -1: none
  __shared__ float from_scale[KV_PAGE];
  __shared__ unsigned s_owned[2];
  __shared__ float s_max[KP_THREADS / 32];
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const bool isv = blockIdx.z & 1;
  const CompactArgs::Layer &ly = a.layer[blockIdx.z >> 1];
  uint8_t *pages = isv ? ly.vp : ly.kp;
  float *scales = isv ? ly.vs : ly.ks;
  const long long cap = (long long)a.width * KV_PAGE;
  const long long base = max(0ll, min((long long)a.base[b], cap));
  const int count = max(0, min(a.n_keep[b], a.max_keep));
  const long long end = min(cap, base + count);
  const int32_t *table = a.table + (size_t)b * a.width;
  for (long long blk = base / KV_PAGE; blk * KV_PAGE < end; ++blk) {
    const int page = table[blk];
    const long long to = blk * KV_PAGE + tid;
    const int k = tid < KV_PAGE && to >= base && to < end ? a.keep[(size_t)b * a.max_keep + (to - base)] : -1;
    if (page < 0 || page >= a.n_pages) continue;       // (the same for the CTA)
    if (tid < KV_PAGE) {
      int slot = -1;
      float sc = 0.f;
      {
        const long long src = base + k;
        if (k >= 0 && src < cap) {
          const int sp = table[src / KV_PAGE];
          if (sp >= 0 && sp < a.n_pages) {
            slot = sp * KV_PAGE + (int)(src % KV_PAGE);
            sc = scales[(size_t)sp * a.nkv + h];
          }
        }
      }
      from[tid] = slot;
      from_scale[tid] = sc;
      const unsigned o = __ballot_sync(0xffffffffu, slot >= 0);
      if (lane == 0) s_owned[tid >> 5] = o;
    }
    __syncthreads();
    const uint64_t owned = (uint64_t)s_owned[1] << 32 | s_owned[0];
    const int o0 = owned ? __ffsll((long long)owned) - 1 : 0, last = owned ? 63 - __clzll(owned) : -1;
    const int w0 = o0 / 4, words = last < 0 ? 0 : last / 4 - w0 + 1;   // of V's places
    // the rows' bytes, and the largest value among them (NaN and what passes fp32 left out)
    float big = 0.f;
    auto largest = [&](uint32_t m, float sc) {
      const float v = e4m3x2_to_f32(m).x * sc;
      if (m != 0x7f && v <= 3.402823466e38f) big = fmaxf(big, v);
    };
    auto take = [&](uint32_t w, float sc) {            // four bytes of one row
#pragma unroll
      for (int j = 0; j < 4; ++j) largest(w >> 8 * j & 0x7f, sc);
    };
    if (!isv) {
      for (int i = o0 * (HD / 16) + tid; i < (last + 1) * (HD / 16); i += KP_THREADS) {
        const int o = i / (HD / 16), c = i % (HD / 16);
        if (!(owned >> o & 1)) continue;
        const uint4 w = *(const uint4 *)(pages + kv8_block(from[o] / KV_PAGE, h, a.nkv, HD) + (from[o] % KV_PAGE) * HD + 16 * c);
        *(uint4 *)(tile + o * HD + 16 * c) = w;
        take(w.x, from_scale[o]), take(w.y, from_scale[o]), take(w.z, from_scale[o]), take(w.w, from_scale[o]);
      }
    } else {
      for (int x = tid; x < HD * words; x += KP_THREADS) {
        const int d = x / words, i = d * (KV_PAGE / 4) + w0 + x - d * words, o = i % (KV_PAGE / 4) * 4;
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (owned >> (o + j) & 1) {
            const uint32_t y = pages[kv8_block(from[o + j] / KV_PAGE, h, a.nkv, HD) + d * KV_PAGE + from[o + j] % KV_PAGE];
            w |= y << 8 * j;
            largest(y & 0x7f, from_scale[o + j]);
          }
        *(uint32_t *)(tile + 4 * i) = w;
      }
    }
    float *sp = scales + (size_t)page * a.nkv + h;
    const bool fresh = owned & 1;
    const float old = fresh ? 0.f : *sp;
    big = warp_max(big);
    if (lane == 0) s_max[tid >> 5] = big;
    __syncthreads();                                   // (every byte and every scale is read)
#pragma unroll
    for (int j = 0; j < KP_THREADS / 32; ++j) big = fmaxf(big, s_max[j]);
    if (owned) {
      float scale = pow2f(scale_exp(big)), again = 1.f;
      if (old >= scale) scale = old;
      else if (!fresh) again = old / scale;
      const uint64_t kept = fresh || again == 1.f ? 0 : (last == 63 ? ~0ull : (2ull << last) - 1) & ~owned;
      const float inv = 1.f / scale;
      if (tid == 0) *sp = scale;
      uint8_t *blkp = pages + kv8_block(page, h, a.nkv, HD);
      auto moved = [&](uint32_t w, float sc) {         // four bytes of one row at the new scale
        const float2 x = e4m3x2_to_f32(w), y = e4m3x2_to_f32(w >> 16);
        return f32_to_e4m3x2(x.x * sc * inv, x.y * sc * inv) | f32_to_e4m3x2(y.x * sc * inv, y.y * sc * inv) << 16;
      };
      const int from0 = kept ? 0 : o0;                 // the first place that is written
      if (!isv) {
        for (int i = from0 * (HD / 4) + tid; i < (last + 1) * (HD / 4); i += KP_THREADS) {
          const int o = i / (HD / 4);
          uint32_t *dst = (uint32_t *)(blkp + 4 * i);
          if (owned >> o & 1) *dst = moved(*(const uint32_t *)(tile + 4 * i), from_scale[o]);
          else if (kept >> o & 1) *dst = rescale4(*dst, again);
        }
      } else {
        const int f0 = from0 / 4, n = last / 4 - f0 + 1;
        for (int z = tid; z < HD * n; z += KP_THREADS) {
          const int d = z / n, i = d * (KV_PAGE / 4) + f0 + z - d * n, o = i % (KV_PAGE / 4) * 4;
          const uint32_t mo = (uint32_t)(owned >> o) & 15, mk = (uint32_t)(kept >> o) & 15;
          if (!(mo | mk)) continue;
          uint32_t *dst = (uint32_t *)(blkp + 4 * i);
          const uint32_t was = mo == 15 ? 0 : *dst, re = mk ? rescale4(was, again) : was, w = *(const uint32_t *)(tile + 4 * i);
          const float2 x = e4m3x2_to_f32(w), y = e4m3x2_to_f32(w >> 16);
          const uint32_t nw = f32_to_e4m3x2(x.x * from_scale[o] * inv, x.y * from_scale[o + 1] * inv) |
                              f32_to_e4m3x2(y.x * from_scale[o + 2] * inv, y.y * from_scale[o + 3] * inv) << 16;
          uint32_t bo = 0, bk = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            bo |= (mo >> j & 1) ? 0xffu << 8 * j : 0;
            bk |= (mk >> j & 1) ? 0xffu << 8 * j : 0;
          }
          *dst = (nw & bo) | (re & bk) | (was & ~(bo | bk));
        }
      }
    }
    __syncthreads();                                   // the tile is free, the page is written
  }
}

}  // namespace dflash

using namespace dflash;

extern "C" dflash_status dflash_kv8_compact(void *stream, int32_t n_layers, const dflash_kv8_cache *c, int32_t n_req,
                                            int32_t max_blocks, int32_t max_keep, const int32_t *base_len,
                                            const int32_t *keep, const int32_t *n_keep, const int32_t *block_table) {
  constexpr int most = 1 << 24;
  if (!c || n_layers < 1 || n_layers > KP_LAYERS || n_req < 1 || n_req > KV8_MAX_REQ || max_blocks < 1 || max_blocks > most ||
      max_keep < 1 || max_keep > most || !base_len || !keep || !n_keep || !block_table || !aligned(base_len, 4) ||
      !aligned(keep, 4) || !aligned(n_keep, 4) || !aligned(block_table, 4))
    return DFLASH_ERR_INVALID_ARG;
  CompactArgs a;
  a.width = max_blocks, a.max_keep = max_keep, a.n_pages = c->n_pages, a.nkv = c->n_kv_heads;
  a.base = base_len, a.keep = keep, a.n_keep = n_keep, a.table = block_table;
  for (int i = 0; i < n_layers; ++i) {
    if (!kv8_cache_ok(&c[i]) || c[i].n_pages != c->n_pages || c[i].n_kv_heads != c->n_kv_heads || c[i].head_dim != c->head_dim)
      return DFLASH_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)                        // a cache twice would be moved twice at once
      if (c[j].k_pages == c[i].k_pages || c[j].v_pages == c[i].v_pages || c[j].k_scale == c[i].k_scale ||
          c[j].v_scale == c[i].v_scale)
        return DFLASH_ERR_INVALID_ARG;
    a.layer[i] = CompactArgs::Layer{(uint8_t *)c[i].k_pages, (uint8_t *)c[i].v_pages, c[i].k_scale, c[i].v_scale};
  }
  const dim3 g(n_req, c->n_kv_heads, 2 * n_layers), t(KP_THREADS);
  const cudaError_t e = c->head_dim == 128 ? launch_pdl(k_kv8_compact<128>, g, t, 0, (cudaStream_t)stream, a)
                                           : launch_pdl(k_kv8_compact<64>, g, t, 0, (cudaStream_t)stream, a);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
