// tokens_checks.hpp - argument checks that the token operators' C ABI sources
// share. Host code; nothing here calls the HIP runtime.
#pragma once

#include "gkdtokens.h"
#include "status.hpp"
#include "tokens_launch.hpp"

namespace gkd {

inline Heads heads(const gkd_heads* h) {
  if (h == nullptr) return Heads{nullptr, 0, 0, 0};
  return Heads{h->data, (long long)h->batch, (long long)h->token, (long long)h->head};
}

// One operand of heads, `n` bytes of alignment for its data and strides
// (`size` bytes an element).
inline gkd_status check_heads(const char* fn, const char* name, const gkd_heads* h, unsigned size, unsigned n) {
  if (h == nullptr || h->data == nullptr) return fail(GKD_ERR_NULL, "%s: NULL %s", fn, name);
  if (h->batch < 0 || h->token < 0 || h->head < 0)
    return fail(GKD_ERR_SHAPE, "%s: a negative stride of %s", fn, name);
  const int64_t unit = n / size;
  if (!aligned(h->data, n) || h->batch % unit != 0 || h->token % unit != 0 || h->head % unit != 0)
    return fail(GKD_ERR_ALIGN, "%s: %s needs %u-byte aligned data and strides", fn, name, n);
  return GKD_OK;
}

// An output, of which no two elements may share a place: no stride of a size
// above one is 0.
inline gkd_status check_out(const char* fn, const char* name, const gkd_heads* h, unsigned size, unsigned n, int B,
                     int T, int H) {
  const gkd_status st = check_heads(fn, name, h, size, n);
  if (st != GKD_OK) return st;
  if ((B > 1 && h->batch == 0) || (T > 1 && h->token == 0) || (H > 1 && h->head == 0))
    return fail(GKD_ERR_SHAPE, "%s: a stride of %s is 0", fn, name);
  return GKD_OK;
}

inline gkd_status check_workspace(const char* fn, const void* ws, size_t bytes, size_t need) {
  if (need == 0) return GKD_OK;
  if (ws == nullptr) return fail(GKD_ERR_NULL, "%s: NULL workspace", fn);
  if (!aligned(ws, 256)) return fail(GKD_ERR_ALIGN, "%s: the workspace needs 256-byte alignment", fn);
  if (bytes < need)
    return fail(GKD_ERR_VALUE, "%s: workspace of %zu bytes, needs %zu", fn, bytes, need);
  return GKD_OK;
}

}  // namespace gkd
