// Argument checks that the serving entry points share, on the host.
#pragma once
#include <cmath>
#include <cstdint>

#include "fa.h"

namespace fa {
namespace host {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The largest stride in elements that a tensor map takes (2^40 bytes, exclusive).
constexpr long long kMaxStride = (1LL << 39) - 8;

// A stride in elements of which `unit` are 16 bytes.
inline int check_stride(int64_t s, int unit = 8) {
  if (s <= 0 || s % unit != 0) return FA_ERR_INVALID_ARG;
  return s <= kMaxStride ? FA_OK : FA_ERR_UNSUPPORTED;
}

inline int check_rows(const fa_rows* r) {
  if (!r || !r->data) return FA_ERR_INVALID_ARG;
  if (!aligned16(r->data)) return FA_ERR_MISALIGNED;
  const int rc = check_stride(r->token_stride);
  return rc != FA_OK ? rc : check_stride(r->head_stride);
}

inline int check_sizes(int B, int T, int Hq, int Hkv, int d, int dtype, float scale) {
  if (B < 0 || T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || Hq / Hkv > 128 || Hq > 65535 || B > (1 << 20) || T > (1 << 30)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

inline bool page_size_ok(int page_size) {
  return page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128 || page_size == 256;
}

// unit: elements in 16 bytes (8, or 16 of a cache in 8 bits)
inline int check_pages(const fa_pages* c, int unit = 8) {
  if (!c || !c->k || !c->v || !c->table) return FA_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v)) return FA_ERR_MISALIGNED;
  for (int64_t s : {c->page_stride, c->head_stride, c->token_stride})
    if (const int rc = check_stride(s, unit); rc != FA_OK) return rc;
  if (c->n_pages < 1 || c->table_width < 1 || c->table_stride < c->table_width) return FA_ERR_INVALID_ARG;
  if (!page_size_ok(c->page_size)) return FA_ERR_UNSUPPORTED;
  if ((long long)c->table_width * c->page_size > (1 << 30)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// The scales of a cache in 8 bits with pages of page_size tokens.
inline int check_scales(const fa_scales* s, int page_size) {
  if (!s || !s->k || !s->v) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(s->k) & 3u) || (reinterpret_cast<uintptr_t>(s->v) & 3u)) return FA_ERR_MISALIGNED;
  if (s->page_stride < 1 || s->head_stride < 1) return FA_ERR_INVALID_ARG;
  if (!page_size_ok(s->block) || s->block > page_size) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

inline int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

}  // namespace host
}  // namespace fa
