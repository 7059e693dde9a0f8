// paged.cuh -- what the paged-cache entry points share: the checked shape of a
// cache and the address arithmetic of its pages.
#pragma once

#include "common.cuh"

namespace xattn {

struct PagedDims {
  int nseq, max_pages, num_pages, page, page_shift, hq, hkv, group, d, esize, dtype;
  long long page_stride, head_stride, token_stride;  // elements
};

namespace host {

// 5-D TMA view of a paged cache's K or V (see api.cu).
int make_pages_map(CUtensorMap* m, const void* ptr, const PagedDims& D, int box_d,
                   int box_tokens);

// log2 of a page size the kernels take, or -1.
inline int page_shift_of(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

// Sizes of the table and the pool (what the plan needs of a cache).
inline int check_pool(int nseq, int page_size, int num_pages, int max_pages) {
  if (nseq < 1 || page_size < 1 || num_pages < 1 || max_pages < 1) return XATTN_ERR_INVALID_ARG;
  if (page_shift_of(page_size) < 0) return XATTN_ERR_UNSUPPORTED;
  // slots and token positions are int32, the latter with room to count past the last
  if (static_cast<long long>(num_pages) * page_size > (1ll << 31) - 1 ||
      static_cast<long long>(max_pages) * page_size > 1ll << 30 || nseq > (1 << 20))
    return XATTN_ERR_UNSUPPORTED;
  return XATTN_OK;
}

// Checks the cache's shape; with_heads = false leaves hq out (append).
inline int check_paged(const xattn_paged* c, bool with_heads, PagedDims* D) {
  if (!c) return XATTN_ERR_INVALID_ARG;
  const int nseq = c->nseq, hkv = c->hkv, d = c->d;
  const int hq = with_heads ? c->hq : hkv, max_pages = with_heads ? c->max_pages : 1;
  if (hkv < 1 || hq < 1 || d < 1 || hq % hkv != 0) return XATTN_ERR_INVALID_ARG;
  if (c->dtype != XATTN_F32 && c->dtype != XATTN_BF16) return XATTN_ERR_INVALID_ARG;
  const int rc = check_pool(nseq, c->page_size, c->num_pages, max_pages);
  if (rc != XATTN_OK) return rc;
  if (hq > XATTN_MAX_HEADS) return XATTN_ERR_UNSUPPORTED;
  if (!(d == 64 || d == 128 || (d == 32 && c->dtype == XATTN_F32))) return XATTN_ERR_UNSUPPORTED;
  const int esize = c->dtype == XATTN_BF16 ? 2 : 4;
  for (long long s : {c->page_stride, c->head_stride, c->token_stride})
    // (a TMA view's strides are below 2^40 bytes)
    if (s < d || s >= (1ll << 40) || s * esize >= (1ll << 40) || (s * esize) % 16 != 0)
      return XATTN_ERR_INVALID_ARG;
  D->nseq = nseq;
  D->max_pages = max_pages;
  D->num_pages = c->num_pages;
  D->page = c->page_size;
  D->page_shift = page_shift_of(c->page_size);
  D->hq = hq;
  D->hkv = hkv;
  D->group = hq / hkv;
  D->d = d;
  D->esize = esize;
  D->dtype = c->dtype;
  D->page_stride = c->page_stride;
  D->head_stride = c->head_stride;
  D->token_stride = c->token_stride;
  return XATTN_OK;
}

}  // namespace host
}  // namespace xattn
