/* A server step through the C ABI alone: a plan for the new tokens of every
 * request, their keys and values into the cache, and attention of one query a
 * request. Usage: paged in out nseq hq hkv d page_size num_pages max_pages fresh...
 * in: Q [nseq, hq, d], K [tokens, hkv, d], V, all bf16; out: O, then lse (fp32),
 * then slots (int32). */
#include <cuda_runtime.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "xattn.h"

#define CU(x)                                   \
  do {                                          \
    if ((x) != cudaSuccess) {                   \
      fprintf(stderr, "%s failed\n", #x);       \
      return 2;                                 \
    }                                           \
  } while (0)
#define XA(x)                                                  \
  do {                                                         \
    const int rc_ = (x);                                       \
    if (rc_ != XATTN_OK) {                                     \
      fprintf(stderr, "%s: %s\n", #x, xattn_strerror(rc_));    \
      return 3;                                                \
    }                                                          \
  } while (0)

static void* device(size_t bytes) {
  void* p = NULL;
  if (cudaMalloc(&p, bytes > 0 ? bytes : 1) != cudaSuccess) exit(4);
  cudaMemset(p, 0, bytes > 0 ? bytes : 1);
  return p;
}

int main(int argc, char** argv) {
  if (argc < 11) return 1;
  const int nseq = atoi(argv[3]), hq = atoi(argv[4]), hkv = atoi(argv[5]), d = atoi(argv[6]);
  const int page = atoi(argv[7]), pages = atoi(argv[8]), rows = atoi(argv[9]);
  if (argc != 10 + nseq) return 1;
  int32_t* fresh_host = malloc(sizeof(int32_t) * (size_t)nseq);
  int tokens = 0;
  for (int i = 0; i < nseq; ++i) tokens += fresh_host[i] = atoi(argv[10 + i]);
  const size_t q_bytes = (size_t)nseq * hq * d * 2, kv_bytes = (size_t)tokens * hkv * d * 2;
  const size_t pool_bytes = (size_t)pages * hkv * page * d * 2;
  char* host = malloc(q_bytes + 2 * kv_bytes);
  FILE* f = fopen(argv[1], "rb");
  if (!f || fread(host, 1, q_bytes + 2 * kv_bytes, f) != q_bytes + 2 * kv_bytes) return 1;
  fclose(f);

  void *Q = device(q_bytes), *K = device(kv_bytes), *V = device(kv_bytes), *O = device(q_bytes);
  void *k_pages = device(pool_bytes), *v_pages = device(pool_bytes);
  float* lse = device((size_t)nseq * hq * 4);
  int32_t *lens = device((size_t)nseq * 4), *fresh = device((size_t)nseq * 4), *pool = device(8);
  int32_t *ring = device((size_t)pages * 4), *table = device((size_t)nseq * rows * 4);
  int32_t *starts = device((size_t)(nseq + 1) * 4), *slots = device((size_t)tokens * 4);
  CU(cudaMemcpy(Q, host, q_bytes, cudaMemcpyHostToDevice));
  CU(cudaMemcpy(K, host + q_bytes, kv_bytes, cudaMemcpyHostToDevice));
  CU(cudaMemcpy(V, host + q_bytes + kv_bytes, kv_bytes, cudaMemcpyHostToDevice));
  CU(cudaMemcpy(fresh, fresh_host, (size_t)nseq * 4, cudaMemcpyHostToDevice));
  int32_t* ids = malloc(sizeof(int32_t) * (size_t)pages);
  for (int i = 0; i < pages; ++i) ids[i] = pages - 1 - i;
  const int32_t state[2] = {0, pages};
  CU(cudaMemcpy(ring, ids, (size_t)pages * 4, cudaMemcpyHostToDevice));
  CU(cudaMemcpy(pool, state, 8, cudaMemcpyHostToDevice));

  xattn_paged c;
  memset(&c, 0, sizeof(c));
  c.nseq = nseq;
  c.max_pages = rows;
  c.num_pages = pages;
  c.page_size = page;
  c.hq = hq;
  c.hkv = hkv;
  c.d = d;
  c.dtype = XATTN_BF16;
  c.token_stride = d;
  c.head_stride = (long long)page * d;
  c.page_stride = (long long)hkv * page * d;
  const size_t ws_bytes = xattn_paged_decode_workspace_bytes(&c);
  if (ws_bytes == 0) return 1;
  void* ws = device(ws_bytes);
  XA(xattn_paged_plan(nseq, page, pages, rows, tokens, lens, fresh, pool, ring, table, lens, pool,
                      starts, slots, NULL));
  XA(xattn_paged_append(K, V, &c, tokens, XATTN_TOKEN_MAJOR, (long long)hkv * d, slots, NULL,
                        k_pages, v_pages, NULL));
  XA(xattn_paged_decode(Q, k_pages, v_pages, &c, table, lens, O, lse, ws, ws_bytes, NULL));
  XA(xattn_get_device_status(NULL));

  f = fopen(argv[2], "wb");
  if (!f) return 1;
  const void* outs[3] = {O, lse, slots};
  const size_t sizes[3] = {q_bytes, (size_t)nseq * hq * 4, (size_t)tokens * 4};
  for (int i = 0; i < 3; ++i) {
    char* h = malloc(sizes[i]);
    CU(cudaMemcpy(h, outs[i], sizes[i], cudaMemcpyDeviceToHost));
    if (fwrite(h, 1, sizes[i], f) != sizes[i]) return 1;
    free(h);
  }
  fclose(f);
  return 0;
}
