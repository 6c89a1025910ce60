// Attention of single tokens over the paged 4-bit cache (include/idx_cache4.h,
// idx_attend4): the rows' kernel of attend_rows.hpp over the tile of attend4.hpp. Bound by
// reading the cache, 136 bytes a token and KV head.
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
