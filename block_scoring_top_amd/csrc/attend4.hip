// Attention of single tokens over the paged 4-bit cache (include/idx_cache4.h,
// idx_attend4): the rows' kernel of attend_rows.hpp over the tile of attend4.hpp. Bound by
// reading the cache, 136 bytes a token and KV head: 128 rows of 256 selected pages, 4 heads,
// 286 MB in 57 us, 5.0 TB/s (a plain read reaches 5.8 on this card; the same loads without
// the arithmetic take 53.5); 4 rows of 4096 to 131072 tokens, 8 heads, 294 MB in 64 us and 5
// of joining. What led there: 64 and 85 us with each lane making all factors of its unit's
// value scales and masks taken in every tile; 57 and 75 with the factors made once and masks
// behind branches; then occupancy and the cut (attend_rows.hpp). The next tile's loads held in
// registers: 59 and 80 (two waves a SIMD instead of three).
#include <hip/hip_runtime.h>

#include "attend4.hpp"
#include "attend_rows.hpp"
#include "launch.h"

namespace idxk {

AttnSplit attend4_rows_split(int64_t R, int Hkv, int64_t units) {
  return attend_rows_split(R, Hkv, units);
}

int launch_attend4_rows(const AttnArgs& a, AttnSplit sp, void* stream) {
  return launch_rows_of<Cache4>(a, sp, stream);
}

}  // namespace idxk
