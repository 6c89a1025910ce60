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
// the sums over all requests for itself (the lengths are a few KB, in L2; a thread holds
// up to 16 requests in registers) and fills the lists of its own requests: one launch,
// no workspace, no atomics, and nothing that depends on the order in which workgroups
// run. New pages come from the ring in front of the free count, pages given back go
// behind it, so no workgroup writes an entry that another reads.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "launch.h"

namespace idxk {

namespace {

constexpr int kTabOwn = 64;  // most requests of one workgroup

struct TabReq {
  uint32_t tok;         // first token row
  int have, after;      // tokens before and after the step
  int old_pages, new_pages;
  int grown, gave;      // first new page, first page given back
  int kv;               // first entry in kv_indices
  int fresh;            // token rows (at most n_tok)
  bool served;
};

// Sums that stop at 2^32 - 1 (a count of token rows past every array, when they do);
// where no sum gets there they are the plain ones.
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) {
  return __builtin_elementwise_add_sat(a, b);
}
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ uint32_t scan_step(uint32_t v) {
  return add_sat(v, dpp_u32<CTRL, ROW_MASK>(v));
}
__device__ __forceinline__ uint32_t wave_scan_sat(uint32_t v) {
  v = scan_step<kDppRowShr1>(v);
  v = scan_step<kDppRowShr1 + 1>(v);
  v = scan_step<kDppRowShr1 + 3>(v);
  v = scan_step<kDppRowShr1 + 7>(v);
  v = scan_step<kDppRowBcast15, 0xA>(v);
  return scan_step<kDppRowBcast31, 0xC>(v);
}

// Exclusive prefix sums over the workgroup's threads of N values at once; v becomes the
// sum of the threads before, total that of all. The waves' sums are scanned by every wave
// for itself, a lane for each.
template <int NT, int N>
__device__ __forceinline__ void block_scan(uint32_t (&v)[N], uint32_t (*lds)[NT / kWave],
                                           uint32_t (&total)[N]) {
  constexpr int WAVES = NT / kWave;
  static_assert(WAVES <= 16, "the waves' sums lie in one row of lanes");
  const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  uint32_t sum[N];
#pragma unroll
  for (int i = 0; i < N; ++i) sum[i] = wave_scan_sat(v[i]);
  __syncthreads();  // the previous sums have been read
  if (lane == kWave - 1)
#pragma unroll
    for (int i = 0; i < N; ++i) lds[i][w] = sum[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t s = lane < WAVES ? lds[i][lane] : 0;
    s = scan_step<kDppRowShr1>(s);
    s = scan_step<kDppRowShr1 + 1>(s);
    s = scan_step<kDppRowShr1 + 3>(s);
    s = scan_step<kDppRowShr1 + 7>(s);
    total[i] = readlane<uint32_t>(s, WAVES - 1);
    const uint32_t before = w == 0 ? 0 : readlane<uint32_t>(s, w - 1);
    // this thread's inclusive sum less its own value: the neighbour's, in the same wave
    const uint32_t left = (uint32_t)__shfl_up((int)sum[i], 1);
    v[i] = add_sat(before, lane == 0 ? 0 : left);
  }
}

// NT threads, PER requests a thread (NT * PER >= B).
template <int NT, int PER>
__global__ __launch_bounds__(NT) void page_tables_kernel(
    const int32_t* __restrict__ seq_len, const int32_t* __restrict__ n_new,
    const int32_t* __restrict__ cursor, int32_t* table, int32_t* ring,
    int32_t* __restrict__ seq_out, int32_t* __restrict__ cursor_out,
    int32_t* __restrict__ kv_indptr, int32_t* __restrict__ kv_indices,
    int32_t* __restrict__ tok_indptr, int32_t* __restrict__ slots,
    int32_t* __restrict__ tok_req, int32_t* __restrict__ tok_len, int B, int max_pages,
    int page_size, int n_pages, int64_t n_indices, int n_tok, int own,
    int shift) {
  __shared__ uint32_t lds[4][NT / kWave];
  __shared__ TabReq mine[kTabOwn];
  const int tid = threadIdx.x;
  const int b0 = blockIdx.x * own, b1 = min(b0 + own, B);
  const int most = max_pages * page_size;

  // this thread's requests: PER consecutive ones
  int have[PER], change[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    have[i] = b < B ? min(max(seq_len[b], 0), most) : 0;
    change[i] = b < B ? n_new[b] : 0;
  }
  const int turn = cursor[0] % n_pages, head = turn < 0 ? turn + n_pages : turn;
  const int free_n = min(max(cursor[1], 0), n_pages);
  // division by page_size, a shift where it is a power of two
  auto div = [&](uint32_t x) {
    return (int)(shift >= 0 ? x >> shift : x / (uint32_t)page_size);
  };
  auto pages = [&](int tokens) { return div((uint32_t)tokens + (page_size - 1)); };

  uint32_t tok[1] = {0}, total_tok[1];
#pragma unroll
  for (int i = 0; i < PER; ++i) tok[0] = add_sat(tok[0], max(change[i], 0));
  block_scan<NT>(tok, lds, total_tok);

  // pages needed; -1 marks a request that cannot be served whatever is free
  int need[PER];
  uint32_t sum[1] = {0}, total_need[1];
  uint32_t t = tok[0];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    t = add_sat(t, max(change[i], 0));
    const int64_t after = max((int64_t)have[i] + change[i], (int64_t)0);
    const bool fits = after <= most && (change[i] <= 0 || t <= (uint32_t)n_tok);
    need[i] = fits ? max(pages((int)after) - pages(have[i]), 0) : -1;
    sum[0] += max(need[i], 0);
  }
  block_scan<NT>(sum, lds, total_need);

  uint32_t v[4] = {0, 0, 0, 0}, total[4];  // pages held, given back, taken; refused
  uint32_t n = sum[0];
  auto step = [&](int i, int& after, int& np) {  // whether request i is served
    n += max(need[i], 0);
    const bool served = need[i] == 0 || (need[i] > 0 && n <= (uint32_t)free_n);
    after = served ? (int)max((int64_t)have[i] + change[i], (int64_t)0) : have[i];
    np = pages(after);
    return served;
  };
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    int after, np;
    const bool served = step(i, after, np);
    v[0] += np;
    v[1] += max(pages(have[i]) - np, 0);
    v[2] += served ? need[i] : 0;
    v[3] += !served && tid * PER + i < B ? 1 : 0;
  }
  block_scan<NT>(v, lds, total);

  // the prefixes of this workgroup's own requests
  if (tid * PER < b1 && (tid + 1) * PER > b0) {
    t = tok[0];
    n = sum[0];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = tid * PER + i, grown = (int)n;
      int after, np;
      const bool served = step(i, after, np);
      if (b >= b0 && b < b1)
        mine[b - b0] = TabReq{t,  have[i], after,     pages(have[i]), np, grown, (int)v[1],
                              (int)v[0], min(max(change[i], 0), n_tok), served};
      t = add_sat(t, max(change[i], 0));
      v[0] += np;
      v[1] += max(pages(have[i]) - np, 0);
    }
  }
  __syncthreads();

  // a wave fills a request's lists; the whole workgroup (and gridDim.y of them) if it
  // has one request only
  const int team = own > 1 ? kWave : NT;
  const int at0 = blockIdx.y * team + tid % team, step_n = gridDim.y * team;
  const bool lead = blockIdx.y == 0 && tid % team == 0;  // writes the per-request words
  for (int k = tid / team; k < b1 - b0; k += NT / team) {
    const TabReq r = mine[k];
    const int b = b0 + k;
    int32_t* row = table + (int64_t)b * max_pages;
    // a page taken from the ring in this step
    auto new_page = [&](int64_t i) {
      return ring[((int64_t)head + r.grown + (i - r.old_pages)) % n_pages];
    };
    for (int64_t i = at0; i < r.new_pages; i += step_n) {
      int32_t p;
      if (i < r.old_pages) {
        p = row[i];
      } else {
        p = new_page(i);
        row[i] = p;
      }
      const int64_t at = (int64_t)r.kv + i;
      if (at < n_indices) kv_indices[at] = p;
    }
    // pages given back join the ring behind the free ones (more than the ring has
    // room for can only come from an inconsistent state: they are dropped)
    for (int64_t i = (int64_t)r.new_pages + at0; i < r.old_pages; i += step_n) {
      const int64_t j = (int64_t)free_n + r.gave + (i - r.new_pages);
      if (j < n_pages) ring[(head + j) % n_pages] = row[i];
    }
    for (int64_t i = at0; i < r.fresh; i += step_n) {
      const int64_t at = (int64_t)r.tok + i;
      if (at >= n_tok) break;
      int32_t slot = -1, len = 0;
      if (r.served) {
        const int pos = r.have + (int)i, e = div((uint32_t)pos);
        const int32_t p = e < r.old_pages ? row[e] : new_page(e);
        if (p >= 0 && p < n_pages) {  // else: not an entry that a step handed out
          slot = p * page_size + (pos - e * page_size);
          len = pos + 1;
        }
      }
      slots[at] = slot;
      tok_req[at] = b;
      tok_len[at] = len;
    }
    if (lead) {
      seq_out[b] = r.after;
      kv_indptr[b] = r.kv;
      tok_indptr[b] = (int32_t)min(r.tok, (uint32_t)n_tok);
    }
  }
  // the rows past the last token, and what belongs to no request
  if (blockIdx.x == gridDim.x - 1)
    for (int64_t i = min(total_tok[0], (uint32_t)n_tok) + blockIdx.y * NT + tid; i < n_tok;
         i += gridDim.y * NT) {
      slots[i] = -1;
      tok_req[i] = -1;
      tok_len[i] = 0;
    }
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) {
    kv_indptr[B] = (int32_t)total[0];
    tok_indptr[B] = (int32_t)min(total_tok[0], (uint32_t)n_tok);
    cursor_out[0] = (int32_t)(((int64_t)head + total[2]) % n_pages);
    cursor_out[1] =
        (int32_t)min((int64_t)free_n - total[2] + (int64_t)total[1], (int64_t)n_pages);
    cursor_out[2] = (int32_t)total[3];
  }
}

}  // namespace

int launch_page_tables(const int32_t* seq_len, const int32_t* n_new, const int32_t* cursor,
                       int32_t* table, int32_t* ring, int32_t* seq_out, int32_t* cursor_out,
                       int32_t* kv_indptr, int32_t* kv_indices, int32_t* tok_indptr,
                       int32_t* slots, int32_t* tok_req, int32_t* tok_len, int B, int max_pages,
                       int page_size, int n_pages, int64_t n_indices, int n_tok, void* stream) {
  // up to 256 requests: one thread and one workgroup (or several) for each; more: a
  // wave for each, 256 workgroups running the sums (4096 requests: 65 us with a
  // workgroup of 256 threads for each four, which reread the lengths, 13 so)
  const int own = B <= 256 ? 1 : (B + 255) / 256;
  const int gx = (B + own - 1) / own;
  int gy = 1;  // a few requests: several workgroups for each
  const int64_t longest = (max_pages > n_tok ? max_pages : n_tok);
  while (gy < 16 && gx * gy < 256 && (int64_t)gy * 256 < longest) gy *= 2;
  int shift = -1;
  for (int i = 0; i < 31; ++i)
    if (page_size == 1 << i) shift = i;
#define IDX_TABLES(NT, PER)                                                                      \
  hipLaunchKernelGGL((page_tables_kernel<NT, PER>), dim3(gx, gy), dim3(NT), 0,                   \
                     static_cast<hipStream_t>(stream), seq_len, n_new, cursor, table, ring,      \
                     seq_out, cursor_out, kv_indptr, kv_indices, tok_indptr, slots, tok_req,     \
                     tok_len, B, max_pages, page_size, n_pages, n_indices, n_tok, own, shift)
  if (B <= 256) IDX_TABLES(256, 1);
  else if (B <= 1024) IDX_TABLES(1024, 1);
  else if (B <= 4096) IDX_TABLES(1024, 4);
  else IDX_TABLES(1024, 16);
#undef IDX_TABLES
  return (int)hipGetLastError();
}

}  // namespace idxk
