// Attention over the 8-bit paged cache: the entry points (dflash_kv8_attention, dflash_kv8_attention_blocks) and their choice of
// kernel.
#include <cmath>

#include "kv8_attn_rows.cuh"

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

namespace {
dflash_status attend(void *stream, const dflash_kv8_cache *c, const dflash_kv8_attn *x, const int32_t *blocks, int n_blocks) {
  if (!attn_ok(c, x, true)) return DFLASH_ERR_INVALID_ARG;
  if (x->rows == 0) return DFLASH_OK;
  const Space sp = space_of(c->head_dim);
  if (!x->workspace || !aligned(x->workspace, 256) || x->workspace_bytes < sp.bytes) return DFLASH_ERR_INVALID_ARG;
  uint8_t *ws = (uint8_t *)x->workspace;
  const Kv8AttnArgs a{x->n_req, x->rows, x->n_q_heads, c->n_kv_heads, x->max_blocks, x->mask, x->tree_words, c->n_pages,
                      x->scale, x->q, x->q_stride, x->cu_q, x->ctx_len, x->block_table, x->tree_mask, x->out, x->lse,
                      (const uint8_t *)c->k_pages, (const uint8_t *)c->v_pages, c->k_scale, c->v_scale,
                      (Kv8Desc *)(ws + sp.desc), (float *)(ws + sp.o), (float *)(ws + sp.ml), blocks, n_blocks};
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
  cudaError_t e;
  if (most <= 16 || !wide)
    e = blocks ? launch_kv8_rows_listed(a, wide, hd, most <= 8 ? 8 : 16, s) : launch_rows<false>(a, wide, hd, most <= 8 ? 8 : 16, s);
  else
    e = launch_kv8_tiles(a, hd, s);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
}  // namespace

extern "C" dflash_status dflash_kv8_attention(void *stream, const dflash_kv8_cache *c, const dflash_kv8_attn *x) {
  return attend(stream, c, x, nullptr, 0);
}

extern "C" dflash_status dflash_kv8_attention_blocks(void *stream, const dflash_kv8_cache *c, const dflash_kv8_attn *x,
                                                     const int32_t *blocks, int32_t n_blocks) {
  if (n_blocks < 1 || n_blocks > (1 << 24) || !blocks || !aligned(blocks, 4)) return DFLASH_ERR_INVALID_ARG;
  return attend(stream, c, x, blocks, n_blocks);
}
