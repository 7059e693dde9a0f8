// paged_plan.cu -- xattn_paged_plan: block table and slot map of a paged cache,
// built on the GPU from the requests' lengths.
#include <cuda_runtime.h>

#include "host.cuh"
#include "paged.cuh"

namespace xattn {
namespace {

constexpr int kThreads = 1024;

struct PlanArgs {
  int nseq, shift, num_pages, max_pages, max_tokens;
  const int32_t *lens, *fresh, *pool;
  int32_t *ring, *table, *lens_out, *pool_out, *starts, *slots;
  int* status;
};

// What one request does in this step.
struct Change {
  int len, grow, have, need, back;  // tokens held and added; pages held, taken and given back
  bool bad;
};

__device__ __forceinline__ int pages_of(long long tokens, int shift) {
  return static_cast<int>((tokens + (1 << shift) - 1) >> shift);
}

__device__ __forceinline__ Change change_of(const PlanArgs& a, int i) {
  Change c = {0, 0, 0, 0, 0, false};
  if (i >= a.nseq) return c;
  const int len = a.lens[i], fresh = a.fresh[i];
  const long long after = static_cast<long long>(len) + max(fresh, 0);
  const long long cap = static_cast<long long>(a.max_pages) << a.shift;
  c.bad = len < 0 || fresh < -1 || after > cap;
  if (c.bad) return c;
  c.len = len;
  c.grow = max(fresh, 0);
  c.have = pages_of(len, a.shift);
  c.need = pages_of(after, a.shift) - c.have;
  c.back = fresh < 0 ? c.have : 0;
  return c;
}

// Inclusive scan of a 64-bit value over the block; *total gets the block's sum.
__device__ long long block_scan(long long v, long long* total) {
  __shared__ long long part[33];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int o = 1; o < 32; o *= 2) {
    const long long w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  __syncthreads();
  if (lane == 31) part[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long p = part[lane];
    for (int o = 1; o < 32; o *= 2) {
      const long long w = __shfl_up_sync(0xffffffffu, p, o);
      if (lane >= o) p += w;
    }
    part[lane] = p;
  }
  __syncthreads();
  *total = part[31];
  return v + (warp > 0 ? part[warp - 1] : 0);
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanArgs a) {
  const int tid = threadIdx.x;
  const int head = a.pool[0], free_pages = a.pool[1];
  // whether the step can be done, from the totals
  long long tokens = 0, need = 0, back = 0, bad = 0;
  for (int i0 = 0; i0 < a.nseq; i0 += kThreads) {
    const Change c = change_of(a, i0 + tid);
    tokens += c.grow;
    need += c.need;
    back += c.back;
    bad += c.bad;
  }
  long long all_tokens, all_need, all_back, all_bad;
  block_scan(tokens, &all_tokens);
  block_scan(need, &all_need);
  block_scan(back, &all_back);
  block_scan(bad, &all_bad);
  const bool wrong = all_bad != 0 || all_tokens > a.max_tokens || head < 0 ||
                     head >= a.num_pages || free_pages < 0 ||
                     free_pages + all_back > a.num_pages;
  const bool lacking = !wrong && all_need > free_pages;
  if (wrong || lacking) {
    for (int i = tid; i < a.nseq; i += kThreads) a.lens_out[i] = a.lens[i];
    for (int i = tid; i <= a.nseq; i += kThreads) a.starts[i] = 0;
    for (int t = tid; t < a.max_tokens; t += kThreads) a.slots[t] = -1;
    if (tid == 0) {
      a.pool_out[0] = head;
      a.pool_out[1] = free_pages;
      atomicExch(a.status, wrong ? kStatusBadCache : kStatusNoPages);
    }
    return;
  }
  long long token0 = 0, need0 = 0, back0 = 0;
  bool bad_page = false;
  for (int i0 = 0; i0 < a.nseq; i0 += kThreads) {
    const int i = i0 + tid;
    const Change c = change_of(a, i);
    long long sum;
    const long long t_at = token0 + block_scan(c.grow, &sum) - c.grow;
    token0 += sum;
    const long long n_at = need0 + block_scan(c.need, &sum) - c.need;
    need0 += sum;
    const long long b_at = back0 + block_scan(c.back, &sum) - c.back;
    back0 += sum;
    if (i >= a.nseq) continue;
    int32_t* row = a.table + static_cast<long long>(i) * a.max_pages;
    for (int j = 0; j < c.need; ++j)
      row[c.have + j] = a.ring[(head + n_at + j) % a.num_pages];
    for (int j = 0; j < c.back; ++j)
      a.ring[(head + free_pages + b_at + j) % a.num_pages] = row[j];
    a.starts[i] = static_cast<int32_t>(t_at);
    a.lens_out[i] = c.back > 0 ? 0 : c.len + c.grow;
  }
  if (tid == 0) {
    a.starts[a.nseq] = static_cast<int32_t>(all_tokens);
    a.pool_out[0] = static_cast<int32_t>((head + all_need) % a.num_pages);
    a.pool_out[1] = static_cast<int32_t>(free_pages - all_need + all_back);
  }
  __syncthreads();
  for (int t = tid; t < a.max_tokens; t += kThreads) {
    int slot = -1;
    if (t < all_tokens) {
      int lo = 0, hi = a.nseq - 1;  // the last request whose start is at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.starts[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const int at = a.starts[lo];
      const int pos = a.lens_out[lo] - (a.starts[lo + 1] - at) + (t - at);
      const int page = a.table[static_cast<long long>(lo) * a.max_pages + (pos >> a.shift)];
      if (page >= 0 && page < a.num_pages)
        slot = (page << a.shift) + (pos & ((1 << a.shift) - 1));
      else
        bad_page = true;
    }
    a.slots[t] = slot;
  }
  if (bad_page) atomicExch(a.status, kStatusBadCache);
}

}  // namespace
}  // namespace xattn

using namespace xattn;
using namespace xattn::host;

extern "C" int xattn_paged_plan(int nseq, int page_size, int num_pages, int max_pages,
                                int max_tokens, const int32_t* lens, const int32_t* fresh,
                                const int32_t* pool, int32_t* ring, int32_t* table,
                                int32_t* lens_out, int32_t* pool_out, int32_t* starts,
                                int32_t* slots, void* stream) {
  int rc = check_pool(nseq, page_size, num_pages, max_pages);
  if (rc != XATTN_OK) return rc;
  if (max_tokens < 0 || !lens || !fresh || !pool || !ring || !table || !lens_out || !pool_out ||
      !starts || (!slots && max_tokens > 0))
    return XATTN_ERR_INVALID_ARG;
  DeviceState* ds = nullptr;
  if ((rc = device_state(&ds)) != XATTN_OK) return rc;
  const PlanArgs a = {nseq, page_shift_of(page_size), num_pages, max_pages, max_tokens,
                      lens, fresh, pool, ring, table, lens_out, pool_out, starts, slots,
                      ds->status};
  plan_kernel<<<1, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cuda_status(cudaGetLastError());
}
