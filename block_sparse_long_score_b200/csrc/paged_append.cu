// paged_append.cu -- xattn_paged_append: keys and values of new tokens into the
// slots of a paged cache.
//
// A copy, bound by memory: every byte of K and V is read once and written once
// (one 128K prompt, 8 KV heads of 128, bf16: 1.07 GB in 168.7 us, 97 % of the copy
// rate; 64 tokens of a step 4.4 us, the launch and two dependent reads). A CTA takes a few
// tokens with all their heads. Where each token's rows come from and go is worked
// out once, by a thread a token, in shared memory; the copy itself is shifts and
// adds, kAhead 16-byte pieces of K and of V a thread in flight.
#include <cuda_runtime.h>

#include "host.cuh"
#include "paged.cuh"

namespace xattn {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;
constexpr int kMostTokens = 16;  // of a CTA

struct AppendArgs {
  PagedDims D;
  int tokens, per;   // tokens in all, and of a CTA (a power of two: 1 << per)
  int vec_shift;     // log2 of a row's 16-byte pieces
  long long kv_stride;
  const int32_t *slots, *starts;
  const uint4 *K, *V;
  uint4 *k_pages, *v_pages;
  int* status;
};

// Where a token's rows are, in 16-byte pieces: head h's at from + h * step in K and
// V, and at to + h * (head stride) in the pages. from < 0: the token is left out.
struct Place {
  long long from, step, to;
};

// The last request whose start is at or before t, by a whole warp: 32 probes a
// step (0 where there is none).
__device__ int request_of(const AppendArgs& a, long long t) {
  const int lane = threadIdx.x % 32;
  int lo = 0, n = a.D.nseq;  // it is one of lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 31) / 32, i = lo + lane * step;
    const bool below = lane * step < n && a.starts[i] <= t;
    const int at = max(31 - __clz(static_cast<int>(__ballot_sync(0xffffffffu, below))), 0);
    n = min(step, n - at * step);
    lo += at * step;
  }
  return lo;
}

// The same from `lo` on, by one thread: most often it is there or a row further, but
// rows that wait lie between busy ones by the thousand (two prompts in the first and
// last of 65536 rows: 4321 us row by row), so the step doubles, then halves.
__device__ int request_from(const AppendArgs& a, int lo, long long t) {
  int step = 1;
  while (lo + step < a.D.nseq && a.starts[lo + step] <= t) {
    lo += step;
    step *= 2;
  }
  for (; step > 0; step /= 2)  // it is one of lo .. lo + 2 * step - 1
    if (lo + step < a.D.nseq && a.starts[lo + step] <= t) lo += step;
  return lo;
}

// Of token t; `request` is that of an earlier one (XATTN_HEAD_MAJOR).
template <bool kHeadMajor>
__device__ Place place_of(const AppendArgs& a, int t, int request) {
  const PagedDims& D = a.D;
  Place p = {-1, 0, 0};
  const int slot = a.slots[t];
  const int per = 16 / D.esize;
  if (kHeadMajor) {
    if (t >= a.starts[D.nseq]) return p;
    request = request_from(a, request, t);
    const long long at = a.starts[request], end = a.starts[request + 1];
    if (at < 0 || t < at || t >= end || end > a.tokens) {  // not a prefix sum
      atomicExch(a.status, kStatusBadCache);
      return p;
    }
    p.step = (end - at) * (D.d / per);
    p.from = (at * D.hkv + (t - at)) * (D.d / per);
  } else {
    p.step = D.d / per;
    p.from = t * a.kv_stride / per;
  }
  if (slot < 0 || (slot >> D.page_shift) >= D.num_pages) {
    if (slot != -1) atomicExch(a.status, kStatusBadCache);
    p.from = -1;
    return p;
  }
  p.to = ((slot >> D.page_shift) * D.page_stride + (slot & (D.page - 1)) * D.token_stride) / per;
  return p;
}

template <bool kHeadMajor>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a) {
  __shared__ Place places[kMostTokens];
  const int tid = threadIdx.x, n = 1 << a.per;
  if (tid < 32) {
    const long long t0 = static_cast<long long>(blockIdx.x) << a.per, t = t0 + tid;
    const int request = kHeadMajor ? request_of(a, t0) : 0;
    if (tid < n)
      places[tid] = t < a.tokens ? place_of<kHeadMajor>(a, static_cast<int>(t), request)
                                 : Place{-1, 0, 0};
  }
  __syncthreads();
  // pieces of a row vary first, then tokens, then heads: neighbouring threads
  // read and write neighbouring rows where they are neighbours in memory
  const int all = a.D.hkv << (a.per + a.vec_shift);
  const long long head_step = a.D.head_stride / (16 / a.D.esize);
  for (int x0 = tid; x0 < all; x0 += kThreads * kAhead) {
    uint4 k[kAhead], v[kAhead];
    long long to[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int x = x0 + i * kThreads;
      to[i] = -1;
      if (x >= all) continue;
      const int row = x >> a.vec_shift, piece = x & ((1 << a.vec_shift) - 1);
      const int h = row >> a.per;
      const Place p = places[row & (n - 1)];
      if (p.from < 0) continue;
      to[i] = p.to + h * head_step + piece;
      const long long from = p.from + h * p.step + piece;
      k[i] = __ldcs(a.K + from);  // read once
      v[i] = __ldcs(a.V + from);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (to[i] < 0) continue;
      a.k_pages[to[i]] = k[i];
      a.v_pages[to[i]] = v[i];
    }
  }
}

}  // namespace
}  // namespace xattn

using namespace xattn;
using namespace xattn::host;

extern "C" int xattn_paged_append(const void* K, const void* V, const xattn_paged* cache,
                                  int tokens, int layout, long long kv_stride,
                                  const int32_t* slots, const int32_t* starts, void* k_pages,
                                  void* v_pages, void* stream) {
  PagedDims D;
  int rc = check_paged(cache, false, &D);
  if (rc != XATTN_OK) return rc;
  if (tokens < 0 || (layout != XATTN_TOKEN_MAJOR && layout != XATTN_HEAD_MAJOR))
    return XATTN_ERR_INVALID_ARG;
  if (tokens == 0) return XATTN_OK;
  if (!K || !V || !slots || !k_pages || !v_pages || k_pages == v_pages)
    return XATTN_ERR_INVALID_ARG;
  if (!aligned16(K) || !aligned16(V) || !aligned16(k_pages) || !aligned16(v_pages))
    return XATTN_ERR_INVALID_ARG;
  if (layout == XATTN_HEAD_MAJOR) {
    if (!starts) return XATTN_ERR_INVALID_ARG;
  } else if (kv_stride < static_cast<long long>(D.hkv) * D.d || kv_stride > (1ll << 31) ||
             kv_stride * D.esize % 16 != 0) {
    return XATTN_ERR_INVALID_ARG;
  }
  DeviceState* ds = nullptr;
  if ((rc = device_state(&ds)) != XATTN_OK) return rc;
  AppendArgs a = {D, tokens, 0, 0, kv_stride, slots, starts, static_cast<const uint4*>(K),
                  static_cast<const uint4*>(V), static_cast<uint4*>(k_pages),
                  static_cast<uint4*>(v_pages), ds->status};
  while (16 << a.vec_shift < D.d * D.esize) ++a.vec_shift;
  // as many tokens a CTA as leave four CTAs to an SM
  while (2 << a.per <= kMostTokens && (tokens >> (a.per + 1)) >= 4 * ds->num_sms) ++a.per;
  const unsigned grid = static_cast<unsigned>((tokens + (1ll << a.per) - 1) >> a.per);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (layout == XATTN_HEAD_MAJOR)
    append_kernel<true><<<grid, kThreads, 0, st>>>(a);
  else
    append_kernel<false><<<grid, kThreads, 0, st>>>(a);
  return cuda_status(cudaGetLastError());
}
