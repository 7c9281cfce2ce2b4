// Attention over the 8-bit paged cache (dflash_kv8_attention): one warp per query row and head,
// lanes over 32 keys at a time, a running maximum and sum, everything in fp32.
#include <cmath>

#include "kv8.cuh"

namespace dflash {

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
};

template <typename T, int HD>
__global__ void __launch_bounds__(128) k_kv8_attn_rows(const Kv8AttnArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ float sq[4][HD];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long id = (long)blockIdx.x * 4 + w;
  if (id >= (long)a.rows * a.nq) return;
  const int row = (int)(id / a.nq), h = (int)(id % a.nq), kvh = h / (a.nq / a.nkv);
  int lo = 0, hi = a.n_req;                            // first b with cu_q[b + 1] > row
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (a.cu_q[m + 1] > row) hi = m;
    else lo = m + 1;
  }
  if (lo == a.n_req || a.cu_q[lo] > row) return;
  const int b = lo, i = row - a.cu_q[b], n = min(a.cu_q[b + 1], a.rows) - a.cu_q[b];
  const int len = max(0, (int)min((long)a.ctx_len[b], (long)a.width * KV_PAGE));
  const int first = len - n;                           // position of the request's first row
  const T *q = (const T *)a.q + row * a.q_stride + (int64_t)h * HD;
  bool bad = false;
  for (int d = lane; d < HD; d += 32) {
    const float x = to_f(q[d]);
    bad |= !(fabsf(x) <= 3.402823466e38f);
    sq[w][d] = x;
  }
  bad = __any_sync(0xffffffffu, bad);
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[HD / 32] = {};
  for (int p0 = 0; p0 < len; p0 += 32) {
    const int p = p0 + lane, page = a.table[(size_t)b * a.width + p / KV_PAGE];
    bool see = p < len && page >= 0 && page < a.n_pages;
    if (a.mask == DFLASH_MASK_CAUSAL) see = see && p <= first + i;
    if (a.mask == DFLASH_MASK_TREE && p >= first && see) {
      const int j = p - first;
      see = j < 32 * a.words && (a.tree[(size_t)row * a.words + j / 32] >> (j % 32) & 1);
    }
    const size_t blk = see ? kv8_block(page, kvh, a.nkv, HD) : 0;
    float s = -INFINITY;
    if (see) {
      const uint8_t *k = a.kp + blk + (size_t)(p % KV_PAGE) * HD;
      s = 0.f;
      for (int d = 0; d < HD; d += 4) {
        const uint32_t u = *(const uint32_t *)(k + d);
        const float2 x = e4m3x2_to_f32(u & 0xffff), y = e4m3x2_to_f32(u >> 16);
        s += sq[w][d] * x.x + sq[w][d + 1] * x.y + sq[w][d + 2] * y.x + sq[w][d + 3] * y.y;
      }
      s *= a.scale * a.ks[(size_t)page * a.nkv + kvh];
    }
    const float top = fmaxf(m, warp_max(s));
    if (top == -INFINITY && !__any_sync(0xffffffffu, see)) continue;
    const float base = top == -INFINITY ? 0.f : top;
    const float pr = see ? expf(s - base) : 0.f, c = expf(m - base);
    const float pv = see ? pr * a.vs[(size_t)page * a.nkv + kvh] : 0.f;
    l = l * c + warp_sum(pr);
    m = top;
    for (int d = 0; d < HD / 32; ++d) o[d] *= c;
    for (int j = 0; j < 32; ++j) {
      const float pj = __shfl_sync(0xffffffffu, pv, j);
      const bool sj = __shfl_sync(0xffffffffu, (int)see, j);
      const size_t bj = __shfl_sync(0xffffffffu, blk, j);
      if (!sj) continue;
      for (int d = 0; d < HD / 32; ++d)
        o[d] = fmaf(pj, e4m3x2_to_f32(a.vp[bj + (size_t)(lane + 32 * d) * KV_PAGE + (p0 + j) % KV_PAGE]).x, o[d]);
    }
  }
  const float inv = bad ? NAN : l == 0.f ? 0.f : 1.f / l;
  T *out = (T *)a.out + ((size_t)row * a.nq + h) * HD;
  for (int d = 0; d < HD / 32; ++d) out[lane + 32 * d] = from_f<T>(bad ? NAN : o[d] * inv);
  if (a.lse && lane == 0) a.lse[(size_t)row * a.nq + h] = bad ? NAN : m + logf(l);
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
}  // namespace

extern "C" int64_t dflash_kv8_attention_workspace(const dflash_kv8_cache *cache, const dflash_kv8_attn *args) {
  if (!attn_ok(cache, args, false)) return -1;
  return 256;
}

extern "C" dflash_status dflash_kv8_attention(void *stream, const dflash_kv8_cache *c, const dflash_kv8_attn *x) {
  if (!attn_ok(c, x, true)) return DFLASH_ERR_INVALID_ARG;
  if (x->rows == 0) return DFLASH_OK;
  if (!x->workspace || !aligned(x->workspace, 256) || x->workspace_bytes < dflash_kv8_attention_workspace(c, x))
    return DFLASH_ERR_INVALID_ARG;
  const Kv8AttnArgs a{x->n_req, x->rows, x->n_q_heads, c->n_kv_heads, x->max_blocks, x->mask, x->tree_words, c->n_pages,
                      x->scale, x->q, x->q_stride, x->cu_q, x->ctx_len, x->block_table, x->tree_mask, x->out, x->lse,
                      (const uint8_t *)c->k_pages, (const uint8_t *)c->v_pages, c->k_scale, c->v_scale};
  const cudaStream_t s = (cudaStream_t)stream;
  const dim3 g((unsigned)(((long)x->rows * x->n_q_heads + 3) / 4)), b(128);
  const cudaError_t e = x->dtype == DFLASH_BF16
      ? (c->head_dim == 128 ? launch_pdl(k_kv8_attn_rows<bf16, 128>, g, b, 0, s, a) : launch_pdl(k_kv8_attn_rows<bf16, 64>, g, b, 0, s, a))
      : (c->head_dim == 128 ? launch_pdl(k_kv8_attn_rows<float, 128>, g, b, 0, s, a) : launch_pdl(k_kv8_attn_rows<float, 64>, g, b, 0, s, a));
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
