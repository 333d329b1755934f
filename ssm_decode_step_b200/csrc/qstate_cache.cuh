// State-cache kernels: quantize states into slots, and read slots back as
// values (include/qstate.h, the state-cache section).
//
// Both are one pass over the data and bound by memory: a state element costs
// its own bytes plus bits/8 + 4/group.  A lane owns 8 consecutive columns of
// a row (32 bytes of FP32 or 16 of a 16-bit type: one load or store; 8 or 4
// bytes of codes), so a warp's access to either side is one contiguous run;
// a group's maximum takes log2(group / 8) xor shuffles.  A thread works on
// kCacheUnroll row passes with their loads issued together.
#pragma once

#include "qstate_kernels.cuh"
#include "qstate_types.cuh"

namespace qs {

constexpr int kCacheThreads = 256;
constexpr int kCacheUnroll = 4;

struct CacheParams {
  const int32_t* slots;
  uint8_t* codes;
  float* scales;
  void* S;
  int num_slots;
  int group;
  unsigned rows;        // rows of a slot: heads * dv
  unsigned blocks;      // CTAs of an entry
};

template <class E>
__device__ __forceinline__ void load8(float (&x)[8], const typename E::T* p) {
  if constexpr (E::kTag == QS_F32) {
    asm volatile("ld.global.cg.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                 : "l"(p));
  } else {
    uint32_t w[4];
    asm volatile("ld.global.cg.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = E::widen2(w[i]);
      x[2 * i] = t.x;
      x[2 * i + 1] = t.y;
    }
  }
}

template <class E>
__device__ __forceinline__ void store8(typename E::T* p, const float (&x)[8]) {
  if constexpr (E::kTag == QS_F32) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
                 "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
  } else {
    uint4 w;
    w.x = E::narrow2(x[0], x[1]);
    w.y = E::narrow2(x[2], x[3]);
    w.z = E::narrow2(x[4], x[5]);
    w.w = E::narrow2(x[6], x[7]);
    *reinterpret_cast<uint4*>(p) = w;
  }
}

// The rows a thread of one entry's CTA works on: pass u takes row
// (block * kCacheUnroll + u) * RPB + row-in-pass, of `rows`.
template <int DK>
struct CachePlace {
  static constexpr int LPR = DK / 8;                 // lanes per row
  static constexpr int RPB = kCacheThreads / LPR;    // rows of one pass of a CTA
  unsigned entry, row0;
  int col;
  __device__ __forceinline__ explicit CachePlace(unsigned blocks) {
    entry = blockIdx.x / blocks;
    row0 = (blockIdx.x - entry * blocks) * (RPB * kCacheUnroll) + threadIdx.x / LPR;
    col = 8 * (threadIdx.x % LPR);
  }
};

// scale = max|x| / qmax, code = x * (1 / scale) rounded to nearest even (the
// exact product): the dynamic rule, as qstate_init.
template <int BITS, int DK, class E>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(CacheParams p) {
  constexpr int QMAX = BITS == 4 ? 7 : 127;
  constexpr float kOff = kMagic + (BITS == 4 ? 8.0f : 128.0f);
  constexpr float kQ = static_cast<float>(QMAX);
  using Pl = CachePlace<DK>;
  const Pl at(p.blocks);
  const int slot = __ldg(p.slots + at.entry);
  if (slot < 0 || slot >= p.num_slots) return;
  const typename E::T* src = static_cast<const typename E::T*>(p.S) + static_cast<size_t>(at.entry) * p.rows * DK;
  const size_t pool_row = static_cast<size_t>(slot) * p.rows;
  float x[kCacheUnroll][8];
#pragma unroll
  for (int u = 0; u < kCacheUnroll; ++u) {
    const unsigned r = at.row0 + u * Pl::RPB;
    if (r < p.rows) {
      load8<E>(x[u], src + static_cast<size_t>(r) * DK + at.col);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[u][i] = 0.0f;
    }
  }
#pragma unroll
  for (int u = 0; u < kCacheUnroll; ++u) {
    const unsigned r = at.row0 + u * Pl::RPB;
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[u][i]));
    // every lane of the warp takes the shuffles, rows behind the last too
    for (int d = 1; d < p.group / 8; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float s = div_qmax_rn<QMAX>(m);
    uint32_t w[2] = {0u, 0u};
    if (s > 0.0f) {
      const float inv = recip_rn(s);
      const bool general = !(s >= 0x1p-126f && s < 0x1p126f);
      uint32_t f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float y = __fmaf_rn(x[u][i], inv, kOff);
        if (general) y = fminf(fmaxf(y, kOff - kQ), kOff + kQ);
        f[i] = __float_as_uint(y);
      }
      if constexpr (BITS == 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[h] = __byte_perm(__byte_perm(f[4 * h], f[4 * h + 1], 0x0040u),
                             __byte_perm(f[4 * h + 2], f[4 * h + 3], 0x0040u), 0x5410u) ^ 0x80808080u;
      } else {
        uint32_t by[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) by[b] = (f[2 * b + 1] << 4) + f[2 * b];
        w[0] = __byte_perm(__byte_perm(by[0], by[1], 0x0040u), __byte_perm(by[2], by[3], 0x0040u), 0x5410u) ^
               0x88888888u;
      }
    }
    if (r >= p.rows) continue;
    const size_t row = pool_row + r;
    uint8_t* c = p.codes + (row * DK + at.col) * BITS / 8;
    if constexpr (BITS == 8) {
      *reinterpret_cast<uint2*>(c) = make_uint2(w[0], w[1]);
    } else {
      *reinterpret_cast<uint32_t*>(c) = w[0];
    }
    if (at.col % p.group == 0) p.scales[row * (DK / p.group) + at.col / p.group] = s;
  }
}

// S = code * scale.
template <int BITS, int DK, class E>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(CacheParams p) {
  using Pl = CachePlace<DK>;
  const Pl at(p.blocks);
  const int slot = __ldg(p.slots + at.entry);
  if (slot < 0 || slot >= p.num_slots) return;
  typename E::T* dst = static_cast<typename E::T*>(p.S) + static_cast<size_t>(at.entry) * p.rows * DK;
  const size_t pool_row = static_cast<size_t>(slot) * p.rows;
  uint2 w[kCacheUnroll];
  float s[kCacheUnroll];
#pragma unroll
  for (int u = 0; u < kCacheUnroll; ++u) {
    const unsigned r = at.row0 + u * Pl::RPB;
    w[u] = make_uint2(0u, 0u);
    s[u] = 0.0f;
    if (r < p.rows) {
      const size_t row = pool_row + r;
      const uint8_t* c = p.codes + (row * DK + at.col) * BITS / 8;
      if constexpr (BITS == 8) {
        w[u] = __ldcg(reinterpret_cast<const uint2*>(c));
      } else {
        w[u].x = __ldcg(reinterpret_cast<const uint32_t*>(c));
      }
      s[u] = __ldg(p.scales + row * (DK / p.group) + at.col / p.group);
    }
  }
#pragma unroll
  for (int u = 0; u < kCacheUnroll; ++u) {
    const unsigned r = at.row0 + u * Pl::RPB;
    if (r >= p.rows) continue;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int code;
      if constexpr (BITS == 8) {
        code = static_cast<int>((i < 4 ? w[u].x : w[u].y) << (24 - 8 * (i & 3))) >> 24;
      } else {
        code = static_cast<int>(w[u].x << (28 - 4 * i)) >> 28;
      }
      x[i] = __fmul_rn(static_cast<float>(code), s[u]);
    }
    store8<E>(dst + static_cast<size_t>(r) * DK + at.col, x);
  }
}

}  // namespace qs
