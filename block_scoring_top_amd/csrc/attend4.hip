// Attention of single tokens over the paged 4-bit cache (include/idx_cache4.h,
// idx_attend4): the rows' kernel of attend_rows.hpp over the tile of attend4.hpp. Bound by
// reading the cache, 136 bytes a token and KV head: 128 rows of 256 selected pages, 4 heads,
// 286 MB in 57 us, 5.0 TB/s (a plain read reaches 5.8 on this card; the same loads without
// the arithmetic take 53.5); 4 rows of 4096 to 131072 tokens, 8 heads, 294 MB in 65 us and 5
// of joining. What led there: 64 and 85 us with each lane making all factors of its unit's
// value scales and masks taken in every tile; 57 and 75 with the factors made once and masks
// behind branches; then occupancy and the cut (attend_rows.hpp). The next tile's loads held in
// registers: 59 and 80 (two waves a SIMD instead of three).
#include <hip/hip_runtime.h>

#include "attend4.hpp"
#include "attend_rows.hpp"
#include "launch.h"

namespace idxk {

// Rows are cut as the 8-bit cache's (attend.hip), into chunks that would give eight
// workgroups a CU if all rows were of the longest length, so that ragged ones balance; but for
// two a CU, all that it holds, where a chunk is more than its start and its part of the join:
// groups above 16 heads, whose instance has two workgroups a CU and twice the partial sums
// (16 rows of 8192 to 32768 tokens, 64 heads on 2: 51 us with eight, 40 with two; 4 of 4096 to
// 131072: 45 and 37), and a row by itself (131072 tokens, 32 heads on 8: 41 and 36). Several rows
// of smaller groups are ragged as a rule (4096 to 131072, 32 heads on 8: two 42 us with eight, 46
// with two; four 70 and 82; 16 259 and 293); equal ones lose a little by it (two of 131072 64
// and 59, four 114 and 109). From 512 rows times heads on rows stay whole, two workgroups a CU
// or more (64 rows of 8192 tokens, 8 heads: 105 us whole, 115 in two; of 2048 to 32768: 277
// and 309).
AttnSplit attend4_rows_split(int64_t R, int Hkv, int G, int64_t units) {
  const int64_t tiles = (units + 3) / 4, pairs = R * Hkv;
  const int64_t want = G > 16 || R == 1 ? 512 : 2048;
  int64_t splits = pairs >= 512 ? 1 : (want + pairs - 1) / pairs;
  if (splits > tiles / kAtWaves) splits = tiles / kAtWaves;
  if (splits < 1) splits = 1;
  const int64_t chunk = (tiles + splits - 1) / splits;
  return {(int)chunk, (int)((tiles + chunk - 1) / chunk), 0};
}

int launch_attend4_rows(const AttnArgs& a, AttnSplit sp, void* stream) {
  return launch_rows_of<Cache4>(a, sp, stream);
}

}  // namespace idxk
