// tables.cu -- the index tables of a serving step (cu_seqlens, positions, page table, slot map)
// from the requests' lengths, in one launch (definition in gdn.h).
//
// Two prefix sums over the requests (tokens and new pages) and two expansions (tokens to rows,
// new pages to table entries).  What it has to move is small (12 bytes per row), so the time is
// that of one launch and of its longest chain of dependent loads.  Hence one kernel and no
// hand-over between CTAs: every CTA goes over all lengths itself (from L2), kTabBlock requests at a
// time, and expands its own share of the rows and pages of each block of requests by binary search
// in shared memory.  Nothing may be written before the totals are checked: with one block of
// requests the prefix sums give them, with more a pass over all lengths comes first.
// Replayed from a graph: 256 single tokens 5.4 us, 8 prompts of up to 8192 tokens 5.7, 4096 requests
// of up to 128 8.6.
#include <cuda_runtime.h>

#include <algorithm>

#include "args.cuh"
#include "common.cuh"

namespace gdn {

constexpr int kTabThreads = 1024;
constexpr int kTabPer = 4;                          // requests per thread of a block of requests
constexpr int kTabBlock = kTabThreads * kTabPer;
constexpr int kTabRows = 2 * kTabThreads;           // rows per CTA

struct TableArgs {
  const int32_t* ctx;
  const int32_t* fresh;  // new_lens
  const int32_t* slot;
  int32_t* table;
  const int32_t* free_pages;
  const int32_t* head;
  int32_t* cu;
  int32_t* pos;
  int64_t* map;
  int32_t* head_out;
  int32_t* status;
  int num_slots, N, max_pages, num_free, page, rows;
  int shift;  // log2(page), or -1
  // v / page
  __device__ __forceinline__ uint32_t pages(uint32_t v) const {
    return shift >= 0 ? v >> shift : v / (uint32_t)page;
  }
};

struct Request {
  int ctx, tokens, held, pages;  // pages: those it lacks
  bool ok;
};

// Request n as the call counts it: one that breaks a rule brings no token.
__device__ __forceinline__ Request request_of(const TableArgs& a, int n) {
  Request r{0, 0, 0, 0, true};
  if (n >= a.N) return r;
  const int c = a.ctx ? __ldg(a.ctx + n) : 0, v = __ldg(a.fresh + n);
  const int sl = state_row(a.slot, n, a.num_slots);
  const int64_t all = (int64_t)c + v;
  r.ok = c >= 0 && v >= 0 && sl >= 0 && all <= INT32_MAX;
  if (!r.ok) return r;
  const uint32_t held = a.pages((uint32_t)c + a.page - 1);
  const uint32_t need = a.pages((uint32_t)all + a.page - 1);
  r.ok = need <= (uint32_t)a.max_pages;
  if (!r.ok) return r;
  r.ctx = c;
  r.tokens = v;
  r.held = (int)held;
  r.pages = (int)(need - held);
  return r;
}

// Index of the last entry of first[0 .. m) that is <= v (first[0] <= v).
__device__ __forceinline__ int last_at_most(const int* first, int m, int v) {
  int lo = 0, hi = m;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kTabThreads) batch_tables_kernel(TableArgs a) {
  __shared__ int tok_s[kTabBlock], page_s[kTabBlock];   // first token / first new page
  __shared__ int64_t sum_s[2][kTabThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool first_cta = blockIdx.x == 0, one = a.N <= kTabBlock;
  const int head = __ldg(a.head);
  const int r0 = blockIdx.x * kTabRows;
  const int r1 = (int)min((int64_t)a.rows, (int64_t)r0 + kTabRows);

  // The checks on the totals: what does not fit takes nothing.  Also this CTA's rows behind the
  // last token.  The same in all CTAs.
  auto admit = [&](int64_t tok, int64_t pages, bool bad) {
    const bool fits = head >= 0 && head <= a.num_free && tok <= a.rows;
    const bool take = fits && pages <= a.num_free - head;
    if (first_cta && tid == 0) {
      if (bad || !fits) report_status(a.status, GDN_ERR_INVALID_ARG);
      else if (!take) report_status(a.status, GDN_ERR_PAGES);
      *a.head_out = take ? head + (int)pages : head;
      a.cu[a.N] = take ? (int)tok : 0;
    }
    const int total = take ? (int)tok : 0;
    for (uint32_t r = max(r0, total) + tid; r < (uint32_t)r1; r += kTabThreads) {
      if (a.pos) a.pos[r] = -1;
      if (a.map) a.map[r] = -1;
    }
    if (!take)
      for (uint32_t n = blockIdx.x * kTabThreads + tid; n < (uint32_t)a.N;
           n += gridDim.x * kTabThreads)
        a.cu[n] = 0;
    return take;
  };
  if (!one) {
    int64_t tok = 0, pages = 0;
    bool bad = false;
    for (int n = tid; n < a.N; n += kTabThreads) {
      const Request r = request_of(a, n);
      tok += r.tokens;
      pages += r.pages;
      bad |= !r.ok;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      tok += __shfl_xor_sync(0xffffffffu, tok, o);
      pages += __shfl_xor_sync(0xffffffffu, pages, o);
    }
    if (lane == 0) {
      sum_s[0][warp] = tok;
      sum_s[1][warp] = pages;
    }
    bad = __syncthreads_or(bad);
    tok = pages = 0;
    for (int w = 0; w < kTabThreads / 32; ++w) {
      tok += sum_s[0][w];
      pages += sum_s[1][w];
    }
    if (!admit(tok, pages, bad)) return;
  }

  // ---- prefix sums, a block of requests at a time
  int64_t tok0 = 0, page0 = 0;  // sums before the block
  for (int base = 0; base < a.N || base == 0; base += kTabBlock) {
    Request r[kTabPer];
    int64_t t_sum = 0, p_sum = 0;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < kTabPer; ++k) {
      r[k] = request_of(a, base + tid * kTabPer + k);
      t_sum += r[k].tokens;
      p_sum += r[k].pages;
      bad |= !r[k].ok;
    }
    int64_t t_inc = t_sum, p_inc = p_sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t_up = __shfl_up_sync(0xffffffffu, t_inc, o);
      const int64_t p_up = __shfl_up_sync(0xffffffffu, p_inc, o);
      if (lane >= o) {
        t_inc += t_up;
        p_inc += p_up;
      }
    }
    __syncthreads();  // the previous block's arrays (and the totals) have been read
    if (lane == 31) {
      sum_s[0][warp] = t_inc;
      sum_s[1][warp] = p_inc;
    }
    bad = __syncthreads_or(bad);
    // sums of the warps before, and of all: lane w looks at warp w
    const int64_t tw = sum_s[0][lane], pw = sum_s[1][lane];
    int64_t t_all = tw, p_all = pw, t_bef = lane < warp ? tw : 0, p_bef = lane < warp ? pw : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      t_all += __shfl_xor_sync(0xffffffffu, t_all, o);
      p_all += __shfl_xor_sync(0xffffffffu, p_all, o);
      t_bef += __shfl_xor_sync(0xffffffffu, t_bef, o);
      p_bef += __shfl_xor_sync(0xffffffffu, p_bef, o);
    }
    if (one && !admit(t_all, p_all, bad)) return;
    int t_at = (int)(tok0 + t_bef + t_inc - t_sum), p_at = (int)(page0 + p_bef + p_inc - p_sum);
    const int m = min(kTabBlock, a.N - base);
#pragma unroll
    for (int k = 0; k < kTabPer; ++k) {
      const int i = tid * kTabPer + k;
      tok_s[i] = t_at;
      page_s[i] = p_at;
      t_at += r[k].tokens;
      p_at += r[k].pages;
    }
    __syncthreads();
    if ((base / kTabBlock) % gridDim.x == blockIdx.x)
      for (int i = tid; i < m; i += kTabThreads) a.cu[base + i] = tok_s[i];
    const int t_lo = (int)tok0, p_lo = (int)page0, t_hi = (int)(tok0 + t_all),
              p_hi = (int)(page0 + p_all);
    // this CTA's rows that belong to the block
    const int b1 = min(r1, t_hi);
    for (uint32_t u = max(r0, t_lo) + tid; u < (uint32_t)b1; u += kTabThreads) {
      const int row = (int)u;
      const int i = last_at_most(tok_s, m, row);
      const int ctx = a.ctx ? __ldg(a.ctx + base + i) : 0, pos = ctx + (row - tok_s[i]);
      if (a.pos) a.pos[row] = pos;
      if (a.map) {
        const int held = (int)a.pages((uint32_t)ctx + a.page - 1), p = (int)a.pages((uint32_t)pos);
        const int slot = state_row(a.slot, base + i, a.num_slots);
        // a page taken by this call comes from the free list itself: no wait for the table
        const int id = p >= held ? __ldg(a.free_pages + head + page_s[i] + (p - held))
                                 : a.table[(size_t)slot * a.max_pages + p];
        if (id < 0) report_status(a.status, GDN_ERR_INVALID_ARG);
        a.map[row] = id < 0 ? -1 : (int64_t)id * a.page + (pos - p * a.page);
      }
    }
    // new pages to the table, spread over all CTAs
    // (32-bit counters without a sign here and above: a last step may pass 2^31)
    for (uint32_t u = p_lo + blockIdx.x * kTabThreads + tid; u < (uint32_t)p_hi;
         u += gridDim.x * kTabThreads) {
      const int p = (int)u;
      const int i = last_at_most(page_s, m, p);
      const int ctx = a.ctx ? __ldg(a.ctx + base + i) : 0;
      const int held = (int)a.pages((uint32_t)ctx + a.page - 1);
      const int slot = state_row(a.slot, base + i, a.num_slots);
      a.table[(size_t)slot * a.max_pages + held + (p - page_s[i])] = __ldg(a.free_pages + head + p);
    }
    tok0 += t_all;
    page0 += p_all;
  }
}

}  // namespace gdn

extern "C" int gdn_batch_tables(const int32_t* ctx_lens, const int32_t* new_lens,
                                const int32_t* slot_idx, int32_t num_slots, int32_t num_reqs,
                                int32_t* page_table, int32_t max_pages, const int32_t* free_pages,
                                int32_t num_free, const int32_t* free_head, int32_t page_size,
                                int32_t num_rows, int32_t* cu_seqlens, int32_t* positions,
                                int64_t* slot_map, int32_t* free_head_out, int32_t* dev_status,
                                void* stream) {
  if (num_reqs < 0 || num_slots < 0 || max_pages < 0 || num_free < 0 || num_rows < 0 ||
      page_size < 1)
    return GDN_ERR_INVALID_ARG;
  if (!cu_seqlens || !free_head || !free_head_out || free_head == free_head_out)
    return GDN_ERR_INVALID_ARG;
  if (num_reqs > 0 && (!new_lens || (!slot_idx && num_slots < num_reqs))) return GDN_ERR_INVALID_ARG;
  if (num_reqs > 0 && max_pages > 0 && num_slots > 0 && !page_table) return GDN_ERR_INVALID_ARG;
  if (num_free > 0 && !free_pages) return GDN_ERR_INVALID_ARG;
  if (num_reqs > (1 << 30)) return GDN_ERR_UNSUPPORTED;  // 32-bit request indices
  const void* ptrs[] = {ctx_lens,   new_lens,  slot_idx, page_table,    free_pages, free_head,
                        cu_seqlens, positions, slot_map, free_head_out, dev_status};
  for (const void* p : ptrs)
    if (p && (reinterpret_cast<uintptr_t>(p) & 3u)) return GDN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(slot_map) & 7u) return GDN_ERR_INVALID_ARG;
  gdn::TableArgs a{ctx_lens,  new_lens,      slot_idx,   page_table, free_pages, free_head,
                   cu_seqlens, positions,    slot_map,   free_head_out, dev_status,
                   num_slots, num_reqs,      max_pages,  num_free,   page_size,  num_rows, -1};
  for (int b = 0; b < 31; ++b)
    if (page_size == (1 << b)) a.shift = b;
  const int grid = std::max(1, (int)(((int64_t)num_rows + gdn::kTabRows - 1) / gdn::kTabRows));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  gdn_host::trace_begin("batch_tables", s);
  gdn::batch_tables_kernel<<<grid, gdn::kTabThreads, 0, s>>>(a);
  gdn_host::trace_end(s);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
