// C entry points of the packed prefill (include/qstate.h): argument checks,
// choice of the kernel, and its launch.  No memory is allocated.
#include <mutex>

#include "qstate_check.h"
#include "qstate_launch.h"
#include "qstate_packed_tc.cuh"

namespace {

using namespace qs;

// The recurrence's fields of cfg, the packed batch and the number of prompts.
qs_status check_packed(const qs_config* cfg, const qs_tokens* b, int sequences, qs_config* out) {
  if (cfg == nullptr) return QS_ERR_INVALID_ARG;
  qs_config c = *cfg;  // storage fields do not matter here
  c.num_tiles = 0;
  c.bits = 8;
  c.group = 32;
  c.policy = QS_SCALE_PERSISTENT;
  c.rounding = QS_ROUND_NEAREST;
  qs_status st = check_config(&c);
  if (st != QS_OK) return st;
  st = check_batch(b);
  if (st != QS_OK) return st;
  if (sequences < 0) return QS_ERR_INVALID_ARG;
  if (c.delta != 0 || c.decay != QS_DECAY_SCALAR) return QS_ERR_UNSUPPORTED;
  if (!batch_fits(&c, sequences, b->heads)) return QS_ERR_UNSUPPORTED;
  *out = c;
  return QS_OK;
}

template <int DK, class E>
cudaError_t launch_recurrent(PackedParams p, int sequences, cudaStream_t stream) {
  constexpr int ROWS = kPackThreads / (DK / 16);
  p.blocks = (p.dv + ROWS - 1) / ROWS;
  packed_recurrent_kernel<DK, E><<<static_cast<unsigned>(sequences) * p.heads * p.blocks, kPackThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// q, k, v or o as [tokens][heads][width], in boxes of 64 tokens by `columns`
// of a head, swizzled over the box's row of 32, 64 or 128 bytes.
bool token_map(CUtensorMap* m, int dtype, const void* base, int width, int heads, int tokens, int64_t stride,
               int columns = 64) {
  const EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(width) * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(columns), 1, kPtChunk}, step[3] = {1, 1, 1};
  return fn(m, dtype == QS_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
            const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            columns == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
            : columns == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                            : CU_TENSOR_MAP_SWIZZLE_32B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of S that a CTA of the tensor-core kernel works on.
int tc_rows(int dv) { return dv <= 64 ? 64 : 128; }

// Segments that a prompt is cut into at most: what the SMs offer beyond the
// heads' row blocks, each at least kMinSegment chunks long.  The SM count is
// B200's, so that workspace sizes need no device.
constexpr int kSms = 148, kMinSegment = 4;
long long max_segments(int dv, int heads, int tokens) {
  const long long spread = kSms / (static_cast<long long>(heads) * ((dv + tc_rows(dv) - 1) / tc_rows(dv)));
  const long long chunks = (static_cast<long long>(tokens) + kPtChunk - 1) / kPtChunk;
  const long long most = chunks / kMinSegment;
  return spread < most ? spread : most;
}

// Tokens of a segment, or 0 where prompts are not cut: with one segment at
// most, or with an item for every SM already (two thirds of them: cutting
// costs a second pass over the keys and values) unless the batch is so long
// (kLongShare chunks for every SM) that one long prompt among short ones would
// matter more than the two launches.
constexpr int kLongShare = 32;
int segment_tokens(int dv, int heads, int tokens, int sequences) {
  const long long n = max_segments(dv, heads, tokens);
  if (n < 2) return 0;
  const long long tiles = static_cast<long long>(heads) * ((dv + tc_rows(dv) - 1) / tc_rows(dv));
  const long long chunks = (static_cast<long long>(tokens) + kPtChunk - 1) / kPtChunk;
  if (3 * tiles * sequences > 2 * kSms && chunks * tiles < static_cast<long long>(kLongShare) * kSms) return 0;
  return static_cast<int>((chunks + n - 1) / n) * kPtChunk;
}

// Bytes of the stored states and decays of n segments (a multiple of 256).
size_t segment_bytes(int dk, int dv, int heads, long long n, size_t* states) {
  const size_t s = (static_cast<size_t>(n + 1) * heads * dv * dk * sizeof(float) + 255) / 256 * 256;
  if (states) *states = s;
  return s + (static_cast<size_t>(n + 1) * heads * sizeof(float) + 255) / 256 * 256;
}

template <class E, int DK, int MDV>
cudaError_t launch_packed_tc(const PackedParams& p0, int sequences, void* workspace, cudaStream_t stream) {
  auto kernel = packed_tc_kernel<E, DK, MDV>;
  static std::once_flag flag;
  cudaError_t err = cudaSuccess;
  std::call_once(flag, [&] {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PtLayout<DK, MDV>::kBytes);
  });
  if (err != cudaSuccess) return err;
  PackedTcParams a;
  a.p = p0;
  a.p.blocks = (p0.dv + MDV - 1) / MDV;
  a.sequences = sequences;
  a.seg = segment_tokens(p0.dv, p0.heads, p0.tokens, sequences);
  a.local = false;
  a.states = a.decays = nullptr;
  const long long units = sequences + (a.seg > 0 ? p0.tokens / a.seg : 0);
  a.items = static_cast<int>(units * p0.heads * a.p.blocks);  // < 2^31: batch_fits, and few segments
  CUtensorMap mq, mk, mv, mo;
  const int qk_heads = p0.heads / p0.share;
  if (!token_map(&mk, E::kTag, p0.k, DK, qk_heads, p0.tokens, p0.k_stride) ||
      !token_map(&mv, E::kTag, p0.v, p0.dv, p0.heads, p0.tokens, p0.v_stride))
    return cudaErrorInvalidValue;
  mq = mo = mk;  // unused without outputs
  if (p0.o != nullptr && (!token_map(&mq, E::kTag, p0.q, DK, qk_heads, p0.tokens, p0.q_stride) ||
                          !token_map(&mo, E::kTag, p0.o, p0.dv, p0.heads, p0.tokens, p0.o_stride, MDV / 4)))
    return cudaErrorInvalidValue;
  const int sms = device_sm_count();
  const int grid = a.items < sms ? a.items : sms;
  if (a.seg > 0) {
    size_t states = 0;
    segment_bytes(DK, p0.dv, p0.heads, p0.tokens / a.seg, &states);
    a.states = static_cast<float*>(workspace);
    a.decays = reinterpret_cast<float*>(static_cast<char*>(workspace) + states);
    PackedTcParams first = a;
    first.local = true;
    first.p.o = nullptr;
    kernel<<<grid, kPtThreads, PtLayout<DK, MDV>::kBytes, stream>>>(mq, mk, mv, mo, first);
    const int quads = (p0.dv * DK / 4 + kJoinThreads - 1) / kJoinThreads;
    packed_join_kernel<DK><<<dim3(static_cast<unsigned>(quads) * sequences, p0.heads), kJoinThreads, 0, stream>>>(a, quads);
  }
  kernel<<<grid, kPtThreads, PtLayout<DK, MDV>::kBytes, stream>>>(mq, mk, mv, mo, a);
  return cudaGetLastError();
}

template <class E>
cudaError_t launch_tc(int dk, const PackedParams& p, int sequences, void* ws, cudaStream_t stream) {
  const bool small = tc_rows(p.dv) == 64;
  if (dk == 64)
    return small ? launch_packed_tc<E, 64, 64>(p, sequences, ws, stream) : launch_packed_tc<E, 64, 128>(p, sequences, ws, stream);
  return small ? launch_packed_tc<E, 128, 64>(p, sequences, ws, stream) : launch_packed_tc<E, 128, 128>(p, sequences, ws, stream);
}

}  // namespace

extern "C" {

qs_status qstate_prefill_packed_workspace(const qs_config* cfg, const qs_tokens* batch, int sequences,
                                          size_t* bytes) {
  qs_config c;
  const qs_status st = check_packed(cfg, batch, sequences, &c);
  if (st != QS_OK) return st;
  const long long n = batch->dtype == QS_F32 ? 0 : max_segments(c.dv, batch->heads, batch->tokens);
  if (bytes) *bytes = n < 2 ? 0 : segment_bytes(c.dk, c.dv, batch->heads, n, nullptr);
  return QS_OK;
}

qs_status qstate_prefill_packed(const qs_config* cfg, const qs_tokens* batch, int sequences, const int32_t* starts,
                                const float* S0, float* S1, const void* q, const void* k, const void* v,
                                const float* alpha, const float* beta, void* o, void* workspace,
                                size_t workspace_bytes, cudaStream_t stream) {
  qs_config c;
  qs_status st = check_packed(cfg, batch, sequences, &c);
  if (st != QS_OK) return st;
  if (sequences == 0) return QS_OK;
  const bool any = batch->tokens > 0;
  if (!starts || !S1 || (any && (!k || !v || !alpha || !beta || (o && !q)))) return QS_ERR_INVALID_ARG;
  if (!aligned(starts, 4) || !aligned(S1, 16) || (S0 && !aligned(S0, 16)) || !aligned(alpha, 4) || !aligned(beta, 4))
    return QS_ERR_INVALID_ARG;
  TokenRanges t = {};
  if (any) {
    st = check_tokens(&c, batch, q, k, v, o, &t);
    if (st != QS_OK) return st;
  }
  size_t need = 0;
  qstate_prefill_packed_workspace(cfg, batch, sequences, &need);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return QS_ERR_INVALID_ARG;
  const size_t tiles = static_cast<size_t>(sequences) * batch->heads;
  const size_t state = tiles * c.dv * c.dk * sizeof(float);
  const size_t gates = any ? static_cast<size_t>(batch->tokens) * batch->heads * sizeof(float) : 0;
  const Range w[3] = {range_of(S1, state), t.o, range_of(need ? workspace : nullptr, need)};
  const Range r[7] = {t.q, t.k, t.v, range_of(alpha, gates), range_of(beta, gates),
                      range_of(starts, (static_cast<size_t>(sequences) + 1) * 4),
                      range_of(S0 == S1 ? nullptr : S0, S0 && S0 != S1 ? state : 0)};
  if (any_overlap(w, 3, r, 7)) return QS_ERR_INVALID_ARG;
  PackedParams p;
  p.starts = starts;
  p.S0 = S0;
  p.S1 = S1;
  p.q = q;
  p.k = k;
  p.v = v;
  p.alpha = alpha;
  p.beta = beta;
  p.o = o;
  p.q_stride = batch->q_stride;
  p.k_stride = batch->k_stride;
  p.v_stride = batch->v_stride;
  p.o_stride = batch->o_stride;
  p.tokens = batch->tokens;
  p.heads = batch->heads;
  p.share = batch->heads / batch->qk_heads;
  p.dv = c.dv;
  p.blocks = 0;
  cudaError_t e;
  if (batch->dtype != QS_F32 && any) {
    e = batch->dtype == QS_F16 ? launch_tc<F16>(c.dk, p, sequences, workspace, stream)
                                  : launch_tc<BF16>(c.dk, p, sequences, workspace, stream);
    return from_cuda(e);
  }
#define QS_REC(DK) (batch->dtype == QS_F32 ? launch_recurrent<DK, F32>(p, sequences, stream) \
                    : batch->dtype == QS_F16 ? launch_recurrent<DK, F16>(p, sequences, stream) \
                                             : launch_recurrent<DK, BF16>(p, sequences, stream))
  e = c.dk == 64 ? QS_REC(64) : QS_REC(128);
#undef QS_REC
  return from_cuda(e);
}

qs_status qstate_prefill_packed_timeouts(unsigned int* count) {
  if (count == nullptr) return QS_ERR_INVALID_ARG;
  return from_cuda(cudaMemcpyFromSymbol(count, packed_timeouts, sizeof(unsigned int)));
}

}  // extern "C"
