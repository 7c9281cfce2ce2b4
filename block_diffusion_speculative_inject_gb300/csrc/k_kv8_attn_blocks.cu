// Attention over listed blocks of the 8-bit paged cache for few query rows: the instances of kv8_attn_rows.cuh.
#include "kv8_attn_rows.cuh"

namespace dflash {

cudaError_t launch_kv8_rows_listed(const Kv8AttnArgs &a, bool wide, int hd, int rows, cudaStream_t s) {
  return launch_rows<true>(a, wide, hd, rows, s);
}

}  // namespace dflash
