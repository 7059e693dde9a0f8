// paged_plan.cu -- xattn_paged_plan: block table and slot map of a paged cache,
// built on the GPU from the requests' lengths.
//
// With have = ceil(len / P), need = ceil((len + grow) / P) - have and the exclusive
// prefix sums tok, off, rel of grow, need and the pages given back, over the
// requests in row order:
//   table[i, have + j]               = ring[head + off_i + j],  j < need_i
//   ring[head + free + rel_i + j]    = table[i, j],             j < have_i, if i ends
//   slots[tok_i + t]                 = page * P + (len_i + t) % P,
// the page of a token being table's where the request had it and the ring's where it
// is new, so no output waits for another. The call moves a few bytes a
// request, page and token and is bound by latency: the launch, the read of the
// lengths, two barriers a scan and one read of a page id.
//
// One launch of one cluster. Every CTA reads all lengths and does the scans for
// itself, then the cluster's threads share the pages and tokens out by their
// number in the sums, whoever the request (a request that ends may hold
// thousands of pages): each finds its request by bisection of the sums in shared
// memory. Lengths and the ring's state may be updated in place, so they are
// written last, behind a cluster barrier that tells that every CTA has read
// them. The slots of a large step are left to a second kernel on the whole GPU.
// Device time: 8 requests 6.6 us; 1024, of which 41 end, 10.7 us; 64 prompts with
// 505K tokens 12.7 us.
#include <cuda_runtime.h>

#include "host.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace xattn {
namespace {

constexpr int kThreads = 1024;  // also the requests of a scan

struct PlanArgs {
  int nseq, shift, num_pages, max_pages, max_tokens;
  bool slots_here;  // in the plan kernel, or by slots_kernel behind it
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

struct Sums {
  long long tok, need, back;
};
__device__ __forceinline__ Sums operator+(const Sums& x, const Sums& y) {
  return {x.tok + y.tok, x.need + y.need, x.back + y.back};
}

// Inclusive sums over the block's threads; *total gets the block's.
__device__ __forceinline__ Sums block_scan(Sums v, Sums* total) {
  __shared__ Sums part[32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  auto warp_scan = [&](Sums x) {
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const Sums y = {__shfl_up_sync(0xffffffffu, x.tok, o),
                      __shfl_up_sync(0xffffffffu, x.need, o),
                      __shfl_up_sync(0xffffffffu, x.back, o)};
      if (lane >= o) x = x + y;
    }
    return x;
  };
  v = warp_scan(v);
  __syncthreads();  // the last call's readers are done
  if (lane == 31) part[warp] = v;
  __syncthreads();
  const Sums p = warp_scan(part[lane]);  // every warp for itself: one barrier less
  *total = {__shfl_sync(0xffffffffu, p.tok, 31), __shfl_sync(0xffffffffu, p.need, 31),
            __shfl_sync(0xffffffffu, p.back, 31)};
  const int before = max(warp - 1, 0);
  const Sums q = {__shfl_sync(0xffffffffu, p.tok, before),
                  __shfl_sync(0xffffffffu, p.need, before),
                  __shfl_sync(0xffffffffu, p.back, before)};
  return warp > 0 ? v + q : v;
}

// The last of n sums that is at or below x, of those with sums[0] <= x < sums[n].
__device__ __forceinline__ int find(const int* sums, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (sums[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ int s_tok[kThreads + 1], s_need[kThreads + 1], s_back[kThreads + 1];
  __shared__ int s_len[kThreads];
  const int tid = threadIdx.x;
  const unsigned all = gridDim.x * kThreads, me = blockIdx.x * kThreads + tid;  // of the cluster
  const int head = a.pool[0], free_pages = a.pool[1];
  const bool one_scan = a.nseq <= kThreads;

  // the step's totals, and whether it can be done
  Change c = change_of(a, tid);
  Sums sum = {c.grow, c.need, c.back}, total;
  bool bad = c.bad;
  for (int i = tid + kThreads; i < a.nseq; i += kThreads) {
    const Change d = change_of(a, i);
    sum = sum + Sums{d.grow, d.need, d.back};
    bad = bad || d.bad;
  }
  sum = block_scan(sum, &total);
  const bool wrong = __syncthreads_or(bad) || total.tok > a.max_tokens || head < 0 ||
                     head >= a.num_pages || free_pages < 0 ||
                     free_pages + total.back > a.num_pages;
  const bool lacking = !wrong && total.need > free_pages;
  if (wrong || lacking) {
    if (a.slots_here)
      for (unsigned t = me; t < static_cast<unsigned>(a.max_tokens); t += all) a.slots[t] = -1;
    for (int i = me; i <= a.nseq; i += all) a.starts[i] = 0;
    for (int i = me; i < a.nseq; i += all) a.lens_out[i] = a.lens[i];
    if (me == 0) {
      a.pool_out[0] = head;
      a.pool_out[1] = free_pages;
      atomicExch(a.status, wrong ? kStatusBadCache : kStatusNoPages);
    }
    return;
  }

  // position x of the ring, counted from its head (x <= num_pages)
  auto ring_at = [&](int x) -> int32_t& {
    x += head;
    return a.ring[x >= a.num_pages ? x - a.num_pages : x];
  };
  bool bad_page = false;
  Sums before = {0, 0, 0};
  for (int i0 = 0; i0 < a.nseq; i0 += kThreads) {
    const int n = min(kThreads, a.nseq - i0);
    if (!one_scan) {
      c = change_of(a, i0 + tid);
      sum = before + block_scan({c.grow, c.need, c.back}, &total);
      before = before + total;
    }
    s_tok[tid + 1] = static_cast<int>(sum.tok);
    s_need[tid + 1] = static_cast<int>(sum.need);
    s_back[tid + 1] = static_cast<int>(sum.back);
    s_len[tid] = c.len;
    if (tid == 0) {
      s_tok[0] = static_cast<int>(sum.tok) - c.grow;
      s_need[0] = static_cast<int>(sum.need) - c.need;
      s_back[0] = static_cast<int>(sum.back) - c.back;
    }
    if (tid < n && (i0 + tid) / kThreads % gridDim.x == blockIdx.x)
      a.starts[i0 + tid] = static_cast<int>(sum.tok) - c.grow;
    __syncthreads();
    // pages taken
    for (int x = s_need[0] + me; x < s_need[n]; x += all) {
      const int i = find(s_need, n, x);
      a.table[static_cast<long long>(i0 + i) * a.max_pages + pages_of(s_len[i], a.shift) + x -
              s_need[i]] = ring_at(x);
    }
    // pages given back
    for (int x = s_back[0] + me; x < s_back[n]; x += all) {
      const int i = find(s_back, n, x);
      const int page = a.table[static_cast<long long>(i0 + i) * a.max_pages + x - s_back[i]];
      bad_page = bad_page || page < 0 || page >= a.num_pages;
      ring_at(free_pages + x) = page;
    }
    // slots, a token a thread, whose reads of page ids overlap four at a time;
    // from the last thread on, as the first ones have more of the pages
    if (a.slots_here) {
      const unsigned end = s_tok[n];  // unsigned: must not wrap past 2^31 - 1
      for (unsigned t = s_tok[0] + all - 1 - me; t < end; t += 4 * all) {
        int page[4], pos[4];
#pragma unroll
        for (unsigned x = 0; x < 4; ++x) {
          const unsigned u = t + x * all;
          if (u >= end) continue;
          const int i = find(s_tok, n, static_cast<int>(u));
          pos[x] = s_len[i] + static_cast<int>(u) - s_tok[i];
          const int at = pos[x] >> a.shift, have = pages_of(s_len[i], a.shift);
          page[x] = at < have ? a.table[static_cast<long long>(i0 + i) * a.max_pages + at]
                              : ring_at(s_need[i] + at - have);
        }
#pragma unroll
        for (unsigned x = 0; x < 4; ++x) {
          if (t + x * all >= end) continue;
          const bool good = page[x] >= 0 && page[x] < a.num_pages;
          bad_page = bad_page || !good;
          a.slots[t + x * all] =
              good ? (page[x] << a.shift) + (pos[x] & ((1 << a.shift) - 1)) : -1;
        }
      }
    }
    if (!one_scan) __syncthreads();
  }
  const int tokens = one_scan ? static_cast<int>(total.tok) : static_cast<int>(before.tok);
  const long long need = one_scan ? total.need : before.need;
  const long long back = one_scan ? total.back : before.back;
  if (a.slots_here)
    for (unsigned t = tokens + me; t < static_cast<unsigned>(a.max_tokens); t += all)
      a.slots[t] = -1;
  if (bad_page) atomicExch(a.status, kStatusBadCache);

  cluster_sync();  // every CTA has read the lengths and the ring's state
  for (int i = me; i < a.nseq; i += all) {
    const int len = a.lens[i], fresh = a.fresh[i];
    a.lens_out[i] = fresh < 0 ? 0 : len + fresh;
  }
  if (me == 0) {
    a.starts[a.nseq] = tokens;
    const int at = head + static_cast<int>(need);
    a.pool_out[0] = at >= a.num_pages ? at - a.num_pages : at;
    a.pool_out[1] = static_cast<int>(free_pages - need + back);
  }
}

constexpr int kSlotWarps = 8;
constexpr int kRun = 512;  // tokens of a warp: on 33 pages at most

// The slot map of a large step, from the finished plan: a cluster sits in one part
// of the GPU, whose writes alone would take 6 us for 500K tokens. A warp takes a
// run of tokens, most often of one request, reads its page ids a lane each and
// passes them round.
__global__ void __launch_bounds__(kSlotWarps * 32) slots_kernel(const PlanArgs a) {
  const int lane = threadIdx.x % 32;
  const bool aligned = (reinterpret_cast<uintptr_t>(a.slots) & 15) == 0;
  bool bad_page = false;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const unsigned tokens = a.starts[a.nseq], room = a.max_tokens;
  auto page_of = [&](int i, int at) {
    const int page = a.table[static_cast<long long>(i) * a.max_pages + at];
    if (page >= 0 && page < a.num_pages) return page;
    bad_page = true;
    return -1;
  };
  auto slot_of = [&](int page, int pos) {
    return page < 0 ? -1 : (page << a.shift) + (pos & ((1 << a.shift) - 1));
  };
  for (unsigned lo = (blockIdx.x * kSlotWarps + threadIdx.x / 32) * kRun; lo < room;
       lo += gridDim.x * kSlotWarps * kRun) {
    const unsigned hi = min(lo + kRun, tokens);
    if (lo < tokens) {
      int i = 0;  // the last request whose start is at or before lo: 32 probes a step
      for (int n = a.nseq; n > 1;) {
        const int step = (n + 31) / 32;
        const bool below =
            lane * step < n && static_cast<unsigned>(a.starts[i + lane * step]) <= lo;
        const int at = 31 - __clz(static_cast<int>(__ballot_sync(0xffffffffu, below)));
        i += at * step;
        n = min(step, n - at * step);
      }
      // the requests of the run in turn
      for (unsigned from = lo; from < hi; ++i) {
        const unsigned next = a.starts[i + 1], to = min(hi, next);
        if (next <= from) continue;
        const int pos0 = a.lens_out[i] - static_cast<int>(next - from);  // of token `from`
        const int at0 = pos0 >> a.shift, last = (pos0 + static_cast<int>(to - from) - 1) >> a.shift;
        const int page = at0 + lane <= last ? page_of(i, at0 + lane) : -1;
        const int page32 = at0 + 32 <= last ? page_of(i, at0 + 32) : -1;
        for (unsigned t0 = from / 128 * 128; t0 < to; t0 += 128) {
          const unsigned t = t0 + lane * 4;
          int slot[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int pos = pos0 + static_cast<int>(t + y - from), at = (pos >> a.shift) - at0;
            const int of_lane = __shfl_sync(0xffffffffu, page, at & 31);
            slot[y] = slot_of(at == 32 ? page32 : of_lane, pos);
          }
          if (aligned && t >= from && t + 4 <= to) {
            *reinterpret_cast<int4*>(a.slots + t) = make_int4(slot[0], slot[1], slot[2], slot[3]);
          } else {
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (t + y >= from && t + y < to) a.slots[t + y] = slot[y];
          }
        }
        from = to;
      }
    }
    for (unsigned t = max(lo, tokens) + lane; t < min(lo + kRun, room); t += 32) a.slots[t] = -1;
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
  // one CTA for a small step, a cluster of 8 as there is more to share out
  const bool slots_here = max_tokens <= 32 * kThreads;
  const int ctas = max_tokens <= 4 * kThreads && nseq <= 256 ? 1 : 8;
  const PlanArgs a = {nseq, page_shift_of(page_size), num_pages, max_pages, max_tokens, slots_here,
                      lens, fresh, pool, ring, table, lens_out, pool_out, starts, slots,
                      ds->status};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, plan_kernel, a);
  if (e != cudaSuccess || slots_here) return cuda_status(e);
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  const long long runs = (static_cast<long long>(max_tokens) + kRun - 1) / kRun;
  cfg.gridDim = dim3(static_cast<unsigned>(
      min((runs + kSlotWarps - 1) / kSlotWarps, static_cast<long long>(ds->num_sms) * 8)));
  cfg.blockDim = dim3(kSlotWarps * 32);
  return cuda_status(cudaLaunchKernelEx(&cfg, slots_kernel, a));
}
