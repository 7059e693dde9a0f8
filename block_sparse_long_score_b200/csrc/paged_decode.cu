// paged_decode.cu -- xattn_paged_decode: attention of one new token per request
// over a paged key-value cache.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "host.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace xattn {
namespace {

constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct DecodeArgs {
  PagedDims D;
  const void *Q, *k_pages, *v_pages;
  const int32_t *table, *lens;
  void* O;
  float* lse;
  int* status;
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(float x, float* y) { *y = x; }
__device__ __forceinline__ void from_float(float x, __nv_bfloat16* y) {
  *y = __float2bfloat16_rn(x);
}

// One CTA per (request, query head); a warp takes every kWarps-th token, a
// lane d / 32 of its features.
template <typename T, int kD>
__global__ void __launch_bounds__(kWarps * 32) decode_kernel(const DecodeArgs a) {
  constexpr int kPer = kD / 32;
  const PagedDims& D = a.D;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int i = blockIdx.x / D.hq, h = blockIdx.x % D.hq;
  const int most = D.max_pages << D.page_shift;
  int len = a.lens[i];
  bool bad = len < 0 || len > most;
  len = min(max(len, 0), most);
  const float scale = kLog2e / sqrtf(static_cast<float>(kD));
  const T* q = static_cast<const T*>(a.Q) + (static_cast<long long>(i) * D.hq + h) * kD;
  float qv[kPer], o[kPer], m = -INFINITY, l = 0.0f;
  for (int j = 0; j < kPer; ++j) {
    qv[j] = to_float(q[lane * kPer + j]) * scale;
    o[j] = 0.0f;
  }
  for (int t = warp; t < len; t += kWarps) {
    const int page = a.table[static_cast<long long>(i) * D.max_pages + (t >> D.page_shift)];
    if (page < 0 || page >= D.num_pages) {
      bad = true;
      continue;
    }
    const long long at = page * D.page_stride + (h / D.group) * D.head_stride +
                         (t & (D.page - 1)) * D.token_stride + lane * kPer;
    const T* k = static_cast<const T*>(a.k_pages) + at;
    const T* v = static_cast<const T*>(a.v_pages) + at;
    float s = 0.0f;
    for (int j = 0; j < kPer; ++j) s += qv[j] * to_float(k[j]);
    for (int x = 16; x > 0; x /= 2) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float m2 = fmaxf(m, s);
    const float base = m2 == -INFINITY ? 0.0f : m2;  // logits of -inf weigh nothing
    const float c = ex2(m - base), p = ex2(s - base);
    l = l * c + p;
    for (int j = 0; j < kPer; ++j) o[j] = o[j] * c + p * to_float(v[j]);
    m = m2;
  }
  if (bad && lane == 0) atomicExch(a.status, kStatusBadCache);
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][kD];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  for (int j = 0; j < kPer; ++j) so[warp][lane * kPer + j] = o[j];
  __syncthreads();
  if (warp != 0) return;
  float top = -INFINITY, total = 0.0f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  const float base = top == -INFINITY ? 0.0f : top;
  for (int w = 0; w < kWarps; ++w) total += sl[w] * ex2(sm[w] - base);
  T* out = static_cast<T*>(a.O) + (static_cast<long long>(i) * D.hq + h) * kD;
  for (int j = 0; j < kPer; ++j) {
    float x = 0.0f;
    for (int w = 0; w < kWarps; ++w) x += so[w][lane * kPer + j] * ex2(sm[w] - base);
    from_float(total == 0.0f ? 0.0f : x / total, out + lane * kPer + j);
  }
  if (lane == 0 && a.lse != nullptr)
    a.lse[static_cast<long long>(i) * D.hq + h] =
        total == 0.0f ? -INFINITY : base * kLn2 + logf(total);
}

template <typename T>
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(a.D.nseq) * a.D.hq;
  if (a.D.d == 32) decode_kernel<T, 32><<<grid, kWarps * 32, 0, st>>>(a);
  else if (a.D.d == 64) decode_kernel<T, 64><<<grid, kWarps * 32, 0, st>>>(a);
  else decode_kernel<T, 128><<<grid, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace xattn

using namespace xattn;
using namespace xattn::host;

extern "C" {

size_t xattn_paged_decode_workspace_bytes(const xattn_paged* cache) {
  PagedDims D;
  return check_paged(cache, true, &D) == XATTN_OK ? 256 : 0;
}

int xattn_paged_decode(const void* Q, const void* k_pages, const void* v_pages,
                       const xattn_paged* cache, const int32_t* table, const int32_t* lens,
                       void* O, float* lse, void* ws, size_t ws_bytes, void* stream) {
  PagedDims D;
  int rc = check_paged(cache, true, &D);
  if (rc != XATTN_OK) return rc;
  if (!Q || !k_pages || !v_pages || !table || !lens || !O) return XATTN_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(O) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
    return XATTN_ERR_INVALID_ARG;
  if (!ws || ws_bytes < xattn_paged_decode_workspace_bytes(cache)) return XATTN_ERR_WORKSPACE;
  if (!aligned16(ws)) return XATTN_ERR_INVALID_ARG;
  DeviceState* ds = nullptr;
  if ((rc = device_state(&ds)) != XATTN_OK) return rc;
  const DecodeArgs a = {D, Q, k_pages, v_pages, table, lens, O, lse, ds->status};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cuda_status(D.dtype == XATTN_BF16 ? launch_decode<__nv_bfloat16>(a, st)
                                           : launch_decode<float>(a, st));
}

}  // extern "C"
