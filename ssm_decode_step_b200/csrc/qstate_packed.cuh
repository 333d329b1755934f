// Prefill of packed prompts, token by token (qstate_prefill_packed): the
// recurrence as it stands, S <- alpha S + (beta v) k^T, o = S q, with the
// state in registers and every operation in FP32.
//
// One CTA per (prompt, head, block of rows).  A row of S lies in LPR = Dk/16
// neighbouring lanes, 16 columns each, in pieces of four that alternate
// between the lanes (so that k and q are read from shared memory without
// bank conflicts and S from global memory in whole lines).  Tokens are
// staged kPackStage at a time, widened to FP32.  Nothing is rounded but the
// outputs, once.  The loop over tokens is bound by its own latency (about
// 32 multiply-adds and log2(LPR) shuffles a token: 0.3 us a token with 16
// heads of 128 x 128), so this form serves FP32 activations and prompts of a
// few tokens (16384 tokens x 16 heads take 9.2 ms here, 0.12 ms on the tensor
// cores).
#pragma once

#include "qstate_kernels.cuh"
#include "qstate_types.cuh"

namespace qs {

constexpr int kPackThreads = 128;
constexpr int kPackStage = 16;

struct PackedParams {
  const int32_t* starts;
  const float* S0;
  float* S1;
  const void* q;
  const void* k;
  const void* v;
  const float* alpha;
  const float* beta;
  void* o;
  long long q_stride, k_stride, v_stride, o_stride;  // elements between tokens
  int tokens;
  int heads;
  int share;   // value heads of a q/k head
  int dv;
  int blocks;  // row blocks of a tile
};

// Rows [begin, end) of a prompt, clamped to the buffer.
__device__ __forceinline__ void prompt_bounds(const int32_t* starts, int i, int tokens, int& begin, int& end) {
  begin = min(max(__ldg(starts + i), 0), tokens);
  end = min(max(__ldg(starts + i + 1), begin), tokens);
}

template <int DK, class E>
__global__ void __launch_bounds__(kPackThreads) packed_recurrent_kernel(PackedParams p) {
  constexpr int LPR = DK / 16;
  constexpr int ROWS = kPackThreads / LPR;
  using T = typename E::T;
  __shared__ __align__(16) float sk[kPackStage][DK];
  __shared__ __align__(16) float sq[kPackStage][DK];
  __shared__ float sv[kPackStage][ROWS];
  __shared__ float sa[kPackStage], sb[kPackStage];
  const int blk = blockIdx.x % p.blocks;
  const int tile = blockIdx.x / p.blocks;
  const int seq = tile / p.heads, head = tile - seq * p.heads;
  const int tid = threadIdx.x, c = tid % LPR, r = tid / LPR;
  const int row = blk * ROWS + r;
  const bool live = row < p.dv;
  int begin, end;
  prompt_bounds(p.starts, seq, p.tokens, begin, end);
  const T* q = static_cast<const T*>(p.q) + static_cast<size_t>(head / p.share) * DK;
  const T* k = static_cast<const T*>(p.k) + static_cast<size_t>(head / p.share) * DK;
  const T* v = static_cast<const T*>(p.v) + static_cast<size_t>(head) * p.dv + blk * ROWS;
  T* o = static_cast<T*>(p.o) + static_cast<size_t>(head) * p.dv + row;
  const bool out = p.o != nullptr;

  const size_t sbase = (static_cast<size_t>(tile) * p.dv + row) * DK;
  float4 S[4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    S[u] = live && p.S0 != nullptr ? *reinterpret_cast<const float4*>(p.S0 + sbase + 4 * (c + LPR * u))
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int t0 = begin; t0 < end; t0 += kPackStage) {
    const int n = min(kPackStage, end - t0);
    __syncthreads();
    for (int i = tid; i < n * DK; i += kPackThreads) {
      const int t = i / DK, j = i % DK;
      sk[t][j] = E::widen(k[(t0 + t) * p.k_stride + j]);
      if (out) sq[t][j] = E::widen(q[(t0 + t) * p.q_stride + j]);
    }
    for (int i = tid; i < n * ROWS; i += kPackThreads) {
      const int t = i / ROWS, j = i % ROWS;
      sv[t][j] = blk * ROWS + j < p.dv ? E::widen(v[(t0 + t) * p.v_stride + j]) : 0.0f;
    }
    if (tid < n) {
      sa[tid] = __ldg(p.alpha + static_cast<size_t>(t0 + tid) * p.heads + head);
      sb[tid] = __ldg(p.beta + static_cast<size_t>(t0 + tid) * p.heads + head);
    }
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      const float a = sa[t], w = sb[t] * sv[t][r];
      float acc = 0.0f;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float4 kv = *reinterpret_cast<const float4*>(&sk[t][4 * (c + LPR * u)]);
        S[u].x = __fmaf_rn(w, kv.x, a * S[u].x);
        S[u].y = __fmaf_rn(w, kv.y, a * S[u].y);
        S[u].z = __fmaf_rn(w, kv.z, a * S[u].z);
        S[u].w = __fmaf_rn(w, kv.w, a * S[u].w);
      }
      if (out) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float4 qv = *reinterpret_cast<const float4*>(&sq[t][4 * (c + LPR * u)]);
          acc = __fmaf_rn(S[u].x, qv.x, acc);
          acc = __fmaf_rn(S[u].y, qv.y, acc);
          acc = __fmaf_rn(S[u].z, qv.z, acc);
          acc = __fmaf_rn(S[u].w, qv.w, acc);
        }
#pragma unroll
        for (int d = 1; d < LPR; d <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
        if (c == 0 && live) o[(t0 + t) * p.o_stride] = E::narrow(acc);
      }
    }
  }
  if (!live) return;
#pragma unroll
  for (int u = 0; u < 4; ++u) *reinterpret_cast<float4*>(p.S1 + sbase + 4 * (c + LPR * u)) = S[u];
}

}  // namespace qs
