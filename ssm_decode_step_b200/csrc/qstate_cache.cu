// C entry points of the state cache (include/qstate.h): argument checks and
// dispatch.  No memory is allocated.

#include "qstate_cache.cuh"
#include "qstate_check.h"
#include "qstate_launch.h"

namespace {

using namespace qs;

// The pool: the family's fields, heads that divide its tiles.
qs_status check_pool(const qs_config* c, int heads) {
  const qs_status st = check_config(c);
  if (st != QS_OK) return st;
  if (heads < 1 || c->num_tiles % heads != 0) return QS_ERR_INVALID_ARG;
  return QS_OK;
}

template <int BITS, int DK>
cudaError_t launch_cache(bool write, int dtype, const CacheParams& p0, int n, cudaStream_t stream) {
  CacheParams p = p0;
  constexpr int RPB = CachePlace<DK>::RPB * kCacheUnroll;
  p.blocks = (p.rows + RPB - 1) / RPB;
  const dim3 grid(static_cast<unsigned>(n) * p.blocks), block(kCacheThreads);
  if (write) {
    if (dtype == QS_F32) cache_write_kernel<BITS, DK, F32><<<grid, block, 0, stream>>>(p);
    if (dtype == QS_F16) cache_write_kernel<BITS, DK, F16><<<grid, block, 0, stream>>>(p);
    if (dtype == QS_BF16) cache_write_kernel<BITS, DK, BF16><<<grid, block, 0, stream>>>(p);
  } else {
    if (dtype == QS_F32) cache_read_kernel<BITS, DK, F32><<<grid, block, 0, stream>>>(p);
    if (dtype == QS_F16) cache_read_kernel<BITS, DK, F16><<<grid, block, 0, stream>>>(p);
    if (dtype == QS_BF16) cache_read_kernel<BITS, DK, BF16><<<grid, block, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

// Checks and launch shared by write and read.
qs_status cache_move(bool write, const qs_config* cfg, int heads, int n, const int32_t* slots, const void* S,
                     int dtype, const void* codes, const float* scales, cudaStream_t stream) {
  const qs_status st = check_pool(cfg, heads);
  if (st != QS_OK) return st;
  if (n < 0 || !valid_dtype(dtype)) return QS_ERR_INVALID_ARG;
  if (write && cfg->policy == QS_SCALE_YOKED) return QS_ERR_UNSUPPORTED;
  if (!batch_fits(cfg, n, heads)) return QS_ERR_UNSUPPORTED;
  if (n == 0 || cfg->num_tiles == 0) return QS_OK;
  if (!slots || !S || !codes || !scales) return QS_ERR_INVALID_ARG;
  if (!aligned(slots, 4) || !aligned(S, 32) || !aligned(codes, 32) || !aligned(scales, 16)) return QS_ERR_INVALID_ARG;
  const Sizes z = sizes_of(cfg);
  const Range rs = range_of(S, static_cast<size_t>(n) * heads * cfg->dv * cfg->dk * dtype_bytes(dtype));
  const Range rc = range_of(codes, z.codes), rg = range_of(scales, z.scales);
  const Range ri = range_of(slots, static_cast<size_t>(n) * 4);
  if (write) {
    const Range w[2] = {rc, rg}, r[2] = {rs, ri};
    if (any_overlap(w, 2, r, 2)) return QS_ERR_INVALID_ARG;
  } else {
    const Range w[1] = {rs}, r[3] = {rc, rg, ri};
    if (any_overlap(w, 1, r, 3)) return QS_ERR_INVALID_ARG;
  }
  CacheParams p;
  p.slots = slots;
  p.codes = static_cast<uint8_t*>(const_cast<void*>(codes));
  p.scales = const_cast<float*>(scales);
  p.S = const_cast<void*>(S);
  p.num_slots = cfg->num_tiles / heads;
  p.group = cfg->group;
  p.rows = static_cast<unsigned>(heads) * cfg->dv;
  p.blocks = 0;
  p.two23 = 0x4B000000u;
  cudaError_t e;
  if (cfg->bits == 4)
    e = cfg->dk == 64 ? launch_cache<4, 64>(write, dtype, p, n, stream) : launch_cache<4, 128>(write, dtype, p, n, stream);
  else
    e = cfg->dk == 64 ? launch_cache<8, 64>(write, dtype, p, n, stream) : launch_cache<8, 128>(write, dtype, p, n, stream);
  return from_cuda(e);
}

template <int BITS, int DK>
cudaError_t dispatch_cache_step(const qs_config* c, const StreamParams& p, int tiles, cudaStream_t s) {
  const bool bdr = c->rounding == QS_ROUND_BDR, delta = c->delta == 1, diag = c->decay == QS_DECAY_DIAGONAL;
  const int sel = (c->policy * 8) + (bdr ? 4 : 0) + (delta ? 2 : 0) + (diag ? 1 : 0);
  switch (sel) {
#define QS_CASE(P, R, DE, DI) \
  case (P * 8 + R * 4 + DE * 2 + DI): return launch_cache_step<BITS, DK, P, R, DE, DI>(p, tiles, c->dv, s);
    QS_CASE(0, 0, 0, 0) QS_CASE(0, 0, 0, 1) QS_CASE(0, 0, 1, 0) QS_CASE(0, 0, 1, 1)
    QS_CASE(0, 1, 0, 0) QS_CASE(0, 1, 0, 1) QS_CASE(0, 1, 1, 0) QS_CASE(0, 1, 1, 1)
    QS_CASE(1, 0, 0, 0) QS_CASE(1, 0, 0, 1) QS_CASE(1, 0, 1, 0) QS_CASE(1, 0, 1, 1)
    QS_CASE(1, 1, 0, 0) QS_CASE(1, 1, 0, 1) QS_CASE(1, 1, 1, 0) QS_CASE(1, 1, 1, 1)
#undef QS_CASE
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

extern "C" {

qs_status qstate_cache_write(const qs_config* cfg, int heads, int n, const int32_t* slots, const void* S,
                             qs_dtype dtype, void* codes, float* scales, cudaStream_t stream) {
  return cache_move(true, cfg, heads, n, slots, S, dtype, codes, scales, stream);
}

qs_status qstate_cache_read(const qs_config* cfg, int heads, int n, const int32_t* slots, const void* codes,
                            const float* scales, void* S, qs_dtype dtype, cudaStream_t stream) {
  return cache_move(false, cfg, heads, n, slots, S, dtype, codes, scales, stream);
}

qs_status qstate_cache_step(const qs_config* cfg, const qs_tokens* batch, const int32_t* slots, void* codes,
                            float* scales, const void* q, const void* k, const void* v, const float* alpha,
                            const float* beta, void* o, cudaStream_t stream) {
  qs_status st = check_batch(batch);
  if (st != QS_OK) return st;
  st = check_pool(cfg, batch->heads);
  if (st != QS_OK) return st;
  if (cfg->policy == QS_SCALE_YOKED) return QS_ERR_UNSUPPORTED;
  if (batch->tokens == 0 || cfg->num_tiles == 0) return QS_OK;
  const bool diag = cfg->decay == QS_DECAY_DIAGONAL;
  if (!slots || !codes || !scales || !k || !v || !alpha || !beta || (o && !q)) return QS_ERR_INVALID_ARG;
  if (!aligned(slots, 4) || !aligned(codes, 32) || !aligned(scales, 16) || !aligned(alpha, diag ? 16 : 4) ||
      !aligned(beta, 4))
    return QS_ERR_INVALID_ARG;
  TokenRanges t;
  st = check_tokens(cfg, batch, q, k, v, o, &t);
  if (st != QS_OK) return st;
  if (!batch_fits(cfg, batch->tokens, batch->heads)) return QS_ERR_UNSUPPORTED;
  const Sizes z = sizes_of(cfg);
  const size_t tiles = static_cast<size_t>(batch->tokens) * batch->heads;
  const Range w[3] = {range_of(codes, z.codes), range_of(scales, z.scales), t.o};
  const Range r[6] = {t.q, t.k, t.v, range_of(alpha, tiles * (diag ? cfg->dk : 1) * 4), range_of(beta, tiles * 4),
                      range_of(slots, static_cast<size_t>(batch->tokens) * 4)};
  if (any_overlap(w, 3, r, 6)) return QS_ERR_INVALID_ARG;
  StreamParams p{};
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = scales;
  p.q = static_cast<const float*>(q);
  p.k = static_cast<const float*>(k);
  p.v = static_cast<const float*>(v);
  p.alpha = alpha;
  p.beta = beta;
  p.o = static_cast<float*>(o);
  p.group = cfg->group;
  p.slots = slots;
  p.num_slots = cfg->num_tiles / batch->heads;
  p.heads = static_cast<unsigned>(batch->heads);
  p.share = static_cast<unsigned>(batch->heads / batch->qk_heads);
  p.dtype = batch->dtype;
  p.q_stride = batch->q_stride;
  p.k_stride = batch->k_stride;
  p.v_stride = batch->v_stride;
  p.o_stride = batch->o_stride;
  const int n = static_cast<int>(tiles);
  cudaError_t e;
  if (cfg->bits == 4)
    e = cfg->dk == 64 ? dispatch_cache_step<4, 64>(cfg, p, n, stream) : dispatch_cache_step<4, 128>(cfg, p, n, stream);
  else
    e = cfg->dk == 64 ? dispatch_cache_step<8, 64>(cfg, p, n, stream) : dispatch_cache_step<8, 128>(cfg, p, n, stream);
  return from_cuda(e);
}

}  // extern "C"
