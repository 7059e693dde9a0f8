// paged_append.cu -- xattn_paged_append: keys and values of new tokens into the
// slots of a paged cache.
#include <cuda_runtime.h>

#include "host.cuh"
#include "paged.cuh"

namespace xattn {
namespace {

constexpr int kThreads = 256;

struct AppendArgs {
  PagedDims D;
  int tokens;
  long long kv_stride;
  const int32_t *slots, *starts;
  const uint4 *K, *V;
  uint4 *k_pages, *v_pages;
  int* status;
};

// A thread moves 16 bytes of K and of V.
template <bool kHeadMajor>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a) {
  const int vecs = a.D.d * a.D.esize / 16, per = 16 / a.D.esize;
  const long long n = static_cast<long long>(a.tokens) * a.D.hkv * vecs;
  for (long long x = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; x < n;
       x += static_cast<long long>(gridDim.x) * kThreads) {
    const int v = static_cast<int>(x % vecs);
    const int h = static_cast<int>(x / vecs % a.D.hkv);
    const int t = static_cast<int>(x / vecs / a.D.hkv);
    const int slot = a.slots[t];
    if (slot < 0 || (slot >> a.D.page_shift) >= a.D.num_pages) {
      if (slot != -1) atomicExch(a.status, kStatusBadCache);
      continue;
    }
    long long from;
    if (kHeadMajor) {
      if (t >= a.starts[a.D.nseq]) continue;
      int lo = 0, hi = a.D.nseq - 1;  // the last request whose start is at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.starts[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const long long at = a.starts[lo], end = a.starts[lo + 1], size = end - at;
      if (at < 0 || t < at || t >= end || end > a.tokens) {  // not a prefix sum
        atomicExch(a.status, kStatusBadCache);
        continue;
      }
      from = (at * a.D.hkv + h * size + (t - at)) * a.D.d;
    } else {
      from = t * a.kv_stride + static_cast<long long>(h) * a.D.d;
    }
    const long long to = (slot >> a.D.page_shift) * a.D.page_stride + h * a.D.head_stride +
                         (slot & (a.D.page - 1)) * a.D.token_stride;
    a.k_pages[to / per + v] = a.K[from / per + v];
    a.v_pages[to / per + v] = a.V[from / per + v];
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
  const AppendArgs a = {D, tokens, kv_stride, slots, starts, static_cast<const uint4*>(K),
                        static_cast<const uint4*>(V), static_cast<uint4*>(k_pages),
                        static_cast<uint4*>(v_pages), ds->status};
  const long long n = static_cast<long long>(tokens) * D.hkv * (D.d * D.esize / 16);
  const long long most = static_cast<long long>(ds->num_sms) * 8;
  const unsigned grid = static_cast<unsigned>(min((n + kThreads - 1) / kThreads, most));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (layout == XATTN_HEAD_MAJOR)
    append_kernel<true><<<grid, kThreads, 0, st>>>(a);
  else
    append_kernel<false><<<grid, kThreads, 0, st>>>(a);
  return cuda_status(cudaGetLastError());
}
