// Attention over listed blocks of the 8-bit paged cache for few query rows: the instances of kv8_attn_rows.cuh.
// 16 requests of one token, 32 heads over 8, 64 of 513 blocks each: 32 us (135 MB, 20 us at the copy rate), of which the start,
// the list's and the table's reads and the merge are 10: a worker has 7 pages. Tiles (k_kv8_attn_tc.cu): 8 x 16 rows x 40
// heads over 96 blocks 38 us, as its whole contexts' 1700 cycles a tile and 8 tiles' worth for each item's start and end.
#include "kv8_attn_rows.cuh"

namespace dflash {

cudaError_t launch_kv8_rows_listed(const Kv8AttnArgs &a, bool wide, int hd, int rows, cudaStream_t s) {
  return launch_rows<true>(a, wide, hd, rows, s);
}

}  // namespace dflash
