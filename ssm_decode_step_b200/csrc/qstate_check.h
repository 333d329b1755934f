// Argument checks shared by the C entry points (include/qstate.h): field
// ranges, alignment and overlap of caller buffers.  Host only.
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/qstate.h"

namespace qs {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void* p, size_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + bytes};
}

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

// Field ranges of the configuration; 0 = fine, else the status to return.
inline qs_status check_config(const qs_config* c) {
  if (c == nullptr) return QS_ERR_INVALID_ARG;
  if (c->num_tiles < 0) return QS_ERR_INVALID_ARG;
  if (c->dk < 1 || c->dv < 1) return QS_ERR_INVALID_ARG;
  if (c->bits != 4 && c->bits != 8) return QS_ERR_INVALID_ARG;
  if (c->group < 1 || c->dk % c->group != 0) return QS_ERR_INVALID_ARG;
  if (c->delta != 0 && c->delta != 1) return QS_ERR_INVALID_ARG;
  if (c->decay != QS_DECAY_SCALAR && c->decay != QS_DECAY_DIAGONAL) return QS_ERR_INVALID_ARG;
  if (c->policy != QS_SCALE_DYNAMIC && c->policy != QS_SCALE_PERSISTENT && c->policy != QS_SCALE_YOKED)
    return QS_ERR_INVALID_ARG;
  if (c->rounding != QS_ROUND_NEAREST && c->rounding != QS_ROUND_BDR) return QS_ERR_INVALID_ARG;
  // what this build has kernels for
  if (c->dk != 64 && c->dk != 128) return QS_ERR_UNSUPPORTED;
  if (c->dv % 16 != 0 || c->dv > 4096) return QS_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->num_tiles) * (c->dv / 8) > 0x7fffffffLL) return QS_ERR_UNSUPPORTED;
  if (c->group != 32 && c->group != 64 && c->group != 128) return QS_ERR_UNSUPPORTED;
  return QS_OK;
}

struct Sizes {
  size_t codes, scales, shadow, vec_k, vec_v, alpha, tile_scalars;
};

inline Sizes sizes_of(const qs_config* c) {
  const size_t T = static_cast<size_t>(c->num_tiles);
  Sizes s;
  s.codes = T * c->dv * c->dk * c->bits / 8;
  s.scales = T * c->dv * (c->dk / c->group) * sizeof(float);
  s.shadow = c->policy == QS_SCALE_YOKED ? T * c->dv * c->dk * sizeof(float) : 0;
  s.vec_k = T * c->dk * sizeof(float);
  s.vec_v = T * c->dv * sizeof(float);
  s.alpha = c->decay == QS_DECAY_DIAGONAL ? s.vec_k : T * sizeof(float);
  s.tile_scalars = T * sizeof(float);
  return s;
}

inline qs_status from_cuda(cudaError_t e) { return e == cudaSuccess ? QS_OK : QS_ERR_CUDA; }

// Written buffers must not overlap each other or any input.
inline bool any_overlap(const Range* written, int nw, const Range* read, int nr) {
  for (int i = 0; i < nw; ++i) {
    for (int j = i + 1; j < nw; ++j)
      if (overlap(written[i], written[j])) return true;
    for (int j = 0; j < nr; ++j)
      if (overlap(written[i], read[j])) return true;
  }
  return false;
}

inline size_t dtype_bytes(int dtype) { return dtype == QS_F32 ? 4 : 2; }

inline bool valid_dtype(int d) { return d == QS_F32 || d == QS_F16 || d == QS_BF16; }

// A batch's tiles fit 32-bit row block counts (row blocks of 8 or 16 rows).
inline bool batch_fits(const qs_config* c, long long entries, long long heads) {
  return entries * heads * (c->dv / 8) <= 0x7fffffffLL;
}

struct TokenRanges {
  Range q, k, v, o;
};

// The layout of q, k, v, o in `b`, and the pointers' alignment.
inline qs_status check_tokens(const qs_config* c, const qs_tokens* b, const void* q, const void* k, const void* v,
                       const void* o, TokenRanges* r) {
  const size_t e = dtype_bytes(b->dtype);
  const size_t qk = static_cast<size_t>(b->qk_heads) * c->dk, vo = static_cast<size_t>(b->heads) * c->dv;
  const int64_t strides[4] = {b->q_stride, b->k_stride, b->v_stride, b->o_stride};
  const size_t width[4] = {qk, qk, vo, vo};
  const void* ptr[4] = {q, k, v, o};
  Range out[4];
  for (int i = 0; i < 4; ++i) {
    out[i] = range_of(nullptr, 0);
    if (ptr[i] == nullptr) continue;
    // a token's stride fits a tensor map's 40 bits of bytes, and the whole batch 62
    if (strides[i] < static_cast<int64_t>(width[i]) || strides[i] > (1LL << 37)) return QS_ERR_INVALID_ARG;
    if (strides[i] > (1LL << 60) / b->tokens) return QS_ERR_INVALID_ARG;
    if ((static_cast<size_t>(strides[i]) * e) % 16 != 0 || !aligned(ptr[i], 16)) return QS_ERR_INVALID_ARG;
    out[i] = range_of(ptr[i], (static_cast<size_t>(b->tokens - 1) * strides[i] + width[i]) * e);
  }
  *r = {out[0], out[1], out[2], out[3]};
  return QS_OK;
}

inline qs_status check_batch(const qs_tokens* b) {
  if (b == nullptr || b->tokens < 0 || b->heads < 1 || b->qk_heads < 1 || b->heads % b->qk_heads != 0 ||
      !valid_dtype(b->dtype))
    return QS_ERR_INVALID_ARG;
  return QS_OK;
}

}  // namespace qs
