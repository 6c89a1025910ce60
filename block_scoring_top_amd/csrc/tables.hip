// One step of the page allocator: page lists and slot maps from request lengths
// (include/idx_cache.h, idx_page_tables).
//
// Everything the step decides follows from prefix sums over the requests:
//   token rows   T_b = sum_{b'<=b} max(n_new, 0)
//   pages needed N_b = sum_{b'<=b} need,  need = ceil(after/page) - ceil(before/page)
//                of the requests that grow within max_pages and n_tokens
//   served       need == 0 or N_b <= free
//   pages held   P_b = sum_{b'<b} ceil(after/page), pages given back G_b likewise.
// A request's outputs then need only its own prefixes, so every workgroup runs
// the sums over all requests for itself (the lengths are a few KB, in L2) and
// fills the lists of its own requests: one launch, no workspace, no atomics, and
// nothing that depends on the order in which workgroups run. New pages come from
// the ring in front of the free count, pages given back go behind it, so no
// workgroup writes an entry that another reads.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "launch.h"

namespace idxk {

namespace {

constexpr int kTabNT = 256;
constexpr int kTabWaves = kTabNT / kWave;
constexpr int kTabOwn = 16;  // most requests of one workgroup

struct TabReq {
  int64_t have, after;  // tokens before and after the step
  int64_t tok;          // first token row
  int old_pages, new_pages;
  int grown, gave;      // first new page, first page given back
  int kv;               // first entry in kv_indices
  int fresh;            // token rows
  bool served;
};

// inclusive prefix sum over the workgroup of one value per thread; `total` gets
// the sum
__device__ int64_t block_scan(int64_t v, int64_t* lds, int64_t& total) {
  const int lane = lane_id(), w = threadIdx.x / kWave;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const int64_t o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();  // the previous scan's sums have been read
  if (lane == kWave - 1) lds[w] = v;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kTabWaves; ++i) {
    const int64_t s = lds[i];
    before += i < w ? s : 0;
    total += s;
  }
  return v + before;
}

__global__ __launch_bounds__(kTabNT) void page_tables_kernel(
    const int32_t* __restrict__ seq_len, const int32_t* __restrict__ n_new,
    const int32_t* __restrict__ cursor, int32_t* table, int32_t* ring,
    int32_t* __restrict__ seq_out, int32_t* __restrict__ cursor_out,
    int32_t* __restrict__ kv_indptr, int32_t* __restrict__ kv_indices,
    int32_t* __restrict__ tok_indptr, int32_t* __restrict__ slots,
    int32_t* __restrict__ tok_req, int32_t* __restrict__ tok_len, int B, int max_pages,
    int page_size, int n_pages, int64_t n_indices, int n_tok, int own, int per_thread) {
  __shared__ int64_t lds[kTabWaves];
  __shared__ TabReq mine[kTabOwn];
  const int tid = threadIdx.x;
  const int b0 = blockIdx.x * own, b1 = min(b0 + own, B);
  const int64_t most = (int64_t)max_pages * page_size;
  const int64_t head = (((int64_t)cursor[0] % n_pages) + n_pages) % n_pages;
  const int64_t free_n = min(max((int64_t)cursor[1], (int64_t)0), (int64_t)n_pages);

  // this thread's requests: per_thread consecutive ones
  const int first = tid * per_thread, last = min(first + per_thread, B);
  auto load = [&](int b, int64_t& have, int64_t& after, int64_t& fresh) {
    have = min(max((int64_t)seq_len[b], (int64_t)0), most);
    const int64_t d = n_new[b];
    after = max(have + d, (int64_t)0);
    fresh = max(d, (int64_t)0);
  };
  auto pages = [&](int64_t tokens) { return (tokens + page_size - 1) / page_size; };

  int64_t have, after, fresh, total_tok, total_need, total_pages, total_gave, n_refused;
  int64_t tok = 0;
  for (int b = first; b < last; ++b) {
    load(b, have, after, fresh);
    tok += fresh;
  }
  tok = block_scan(tok, lds, total_tok) - tok;  // before this thread's requests
  // pages needed by request b, whose token rows end at row `end`
  auto need_of = [&](int64_t end, bool& fits) {
    fits = after <= most && (fresh == 0 || end <= n_tok);
    return fits ? max(pages(after) - pages(have), (int64_t)0) : (int64_t)0;
  };
  int64_t need = 0, t = tok;
  bool fits;
  for (int b = first; b < last; ++b) {
    load(b, have, after, fresh);
    t += fresh;
    need += need_of(t, fits);
  }
  need = block_scan(need, lds, total_need) - need;
  int64_t held = 0, gave = 0, refused = 0, taken = 0, n = need;
  t = tok;
  for (int b = first; b < last; ++b) {
    load(b, have, after, fresh);
    t += fresh;
    const int64_t k = need_of(t, fits);
    n += k;
    const bool served = fits && (k == 0 || n <= free_n);
    const int64_t np = pages(served ? after : have);
    held += np;
    gave += max(pages(have) - np, (int64_t)0);
    taken += served ? k : 0;
    refused += served ? 0 : 1;
  }
  int64_t total_taken;
  const int64_t held0 = block_scan(held, lds, total_pages) - held;
  const int64_t gave0 = block_scan(gave, lds, total_gave) - gave;
  block_scan(taken, lds, total_taken);
  block_scan(refused, lds, n_refused);

  // the prefixes of this workgroup's own requests
  if (first < b1 && last > b0) {
    t = tok;
    n = need;
    int64_t h = held0, g = gave0;
    for (int b = first; b < last; ++b) {
      load(b, have, after, fresh);
      const int64_t t0 = t;
      t += fresh;
      const int64_t k = need_of(t, fits);
      const bool served = fits && (k == 0 || n + k <= free_n);
      const int64_t np = pages(served ? after : have);
      if (b >= b0 && b < b1) {
        TabReq& r = mine[b - b0];
        r.have = have;
        r.after = served ? after : have;
        r.tok = t0;
        r.old_pages = (int)pages(have);
        r.new_pages = (int)np;
        r.grown = (int)n;
        r.gave = (int)g;
        r.kv = (int)h;
        r.fresh = (int)min(fresh, (int64_t)n_tok);
        r.served = served;
      }
      n += k;
      h += np;
      g += max(pages(have) - np, (int64_t)0);
    }
  }
  __syncthreads();

  const bool lead = blockIdx.y == 0;  // writes the per-request words
  for (int b = b0; b < b1; ++b) {
    const TabReq r = mine[b - b0];
    int32_t* row = table + (int64_t)b * max_pages;
    // page of list entry i: held before, or taken from the ring in this step
    auto fresh_page = [&](int i) {
      return ring[(head + r.grown + (i - r.old_pages)) % n_pages];
    };
    const int step = gridDim.y * kTabNT;
    for (int i = blockIdx.y * kTabNT + tid; i < r.new_pages; i += step) {
      int32_t p;
      if (i < r.old_pages) {
        p = row[i];
      } else {
        p = fresh_page(i);
        row[i] = p;
      }
      const int64_t at = (int64_t)r.kv + i;
      if (at < n_indices) kv_indices[at] = p;
    }
    // pages given back join the ring behind the free ones (more than the ring has
    // room for can only come from an inconsistent state: they are dropped)
    for (int i = r.new_pages + blockIdx.y * kTabNT + tid; i < r.old_pages; i += step) {
      const int64_t j = free_n + r.gave + (i - r.new_pages);
      if (j < n_pages) ring[(head + j) % n_pages] = row[i];
    }
    for (int64_t i = blockIdx.y * kTabNT + tid; i < r.fresh; i += step) {
      const int64_t at = r.tok + i;
      if (at >= n_tok) break;
      int32_t slot = -1, len = 0;
      if (r.served) {
        const int64_t pos = r.have + i;
        const int e = (int)(pos / page_size);
        const int32_t p = e < r.old_pages ? row[e] : fresh_page(e);
        if (p >= 0 && p < n_pages) {  // else: not an entry that a step handed out
          slot = p * page_size + (int)(pos % page_size);
          len = (int)pos + 1;
        }
      }
      slots[at] = slot;
      tok_req[at] = b;
      tok_len[at] = len;
    }
    if (lead && tid == 0) {
      seq_out[b] = (int32_t)r.after;
      kv_indptr[b] = r.kv;
      tok_indptr[b] = (int32_t)min(r.tok, (int64_t)n_tok);
      if (b == B - 1) {
        kv_indptr[B] = (int32_t)total_pages;
        tok_indptr[B] = (int32_t)min(total_tok, (int64_t)n_tok);
      }
    }
  }
  // the rows past the last token
  if (blockIdx.x == gridDim.x - 1) {
    for (int64_t i = min(total_tok, (int64_t)n_tok) + blockIdx.y * kTabNT + tid; i < n_tok;
         i += gridDim.y * kTabNT) {
      slots[i] = -1;
      tok_req[i] = -1;
      tok_len[i] = 0;
    }
  }
  if (blockIdx.x == 0 && lead && tid == 0) {
    cursor_out[0] = (int32_t)((head + total_taken) % n_pages);
    cursor_out[1] = (int32_t)min(free_n - total_taken + total_gave, (int64_t)n_pages);
    cursor_out[2] = (int32_t)n_refused;
  }
}

}  // namespace

int launch_page_tables(const int32_t* seq_len, const int32_t* n_new, const int32_t* cursor,
                       int32_t* table, int32_t* ring, int32_t* seq_out, int32_t* cursor_out,
                       int32_t* kv_indptr, int32_t* kv_indices, int32_t* tok_indptr,
                       int32_t* slots, int32_t* tok_req, int32_t* tok_len, int B, int max_pages,
                       int page_size, int n_pages, int64_t n_indices, int n_tok, void* stream) {
  const int own = (B + 1023) / 1024;  // at most kTabOwn for B <= 16384
  const int gx = (B + own - 1) / own;
  int gy = 1;  // a few requests: several workgroups for each
  const int64_t longest = (max_pages > n_tok ? max_pages : n_tok);
  while (gy < 16 && gx * gy < 256 && (int64_t)gy * kTabNT < longest) gy *= 2;
  hipLaunchKernelGGL(page_tables_kernel, dim3(gx, gy), dim3(kTabNT), 0,
                     static_cast<hipStream_t>(stream), seq_len, n_new, cursor, table, ring,
                     seq_out, cursor_out, kv_indptr, kv_indices, tok_indptr, slots, tok_req,
                     tok_len, B, max_pages, page_size, n_pages, n_indices, n_tok, own,
                     (B + kTabNT - 1) / kTabNT);
  return (int)hipGetLastError();
}

}  // namespace idxk
