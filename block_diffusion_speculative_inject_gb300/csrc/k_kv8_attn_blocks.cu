// Attention over listed blocks of the 8-bit paged cache for few query rows: the instances of kv8_attn_rows.cuh.
// 16 requests of one token, 32 heads over 8, 64 of 513 blocks each: 32 us (135 MB, 20 us at the copy rate). 256 blocks take 92.5,
// so a block of all requests and heads costs 0.32 us, which is the copy rate, and 12 us are beside the pages: the start, the
// list's and the table's reads, and the merge, since a worker has 7 pages and every item is cut. fp32 33 us.
// Tiles (k_kv8_attn_tc.cu): 8 x 16 rows x 40 heads over 96 blocks 38 us, over 256 74.6: 0.23 us a block, which with 64 items
// on 152 workers is 2100 cycles a tile of 128 tokens, and 17 us beside them (12 for a list of two blocks): the pieces'
// search, Q, the drain and the merge with its launch. What an item's start and end count for in the cutting
// (KM_COST, KT_COST) was measured on long whole contexts, not on lists.
#include "kv8_attn_rows.cuh"

namespace dflash {

cudaError_t launch_kv8_rows_listed(const Kv8AttnArgs &a, bool wide, int hd, int rows, cudaStream_t s) {
  return launch_rows<true>(a, wide, hd, rows, s);
}

}  // namespace dflash
