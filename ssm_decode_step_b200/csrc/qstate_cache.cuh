// State-cache kernels: quantize states into slots, and read slots back as
// values (include/qstate.h, the state-cache section).
//
// Both are one pass over the data; a state element costs its own bytes plus
// bits/8 + 4/group, and that is little enough that instructions bind before
// memory does.  So a lane owns 16 consecutive columns of a row, which shares
// the scale's arithmetic (a group's maximum takes log2(group / 16) xor
// shuffles) and the addresses among 16 elements, and works on pairs with the
// packed FP32 instructions: no integer conversions, codes are joined to and
// split from the mantissa of 2^23 as in the step kernel.  A thread works on
// kCacheUnroll rows with their loads issued together.  Measured on a B200: 256
// states of 16 heads of 128 x 128, FP32 to INT8, 53.3 us (344 MB, 99% of the
// measured copy bandwidth; 8 columns a lane: 65 us); INT4 to FP32 50.4 us
// (306 MB, 93%); 100 states of 24 heads of 80 x 128 in bf16, to INT4 and back,
// 13.7 + 9.5 us (129 MB), where the issue slots of 16-bit conversion bind.
#pragma once

#include "qstate_kernels.cuh"
#include "qstate_types.cuh"

namespace qs {

constexpr int kCacheThreads = 256;
constexpr int kCacheUnroll = 2;
constexpr int kCacheCols = 16;  // columns of a lane

struct CacheParams {
  const int32_t* slots;
  uint8_t* codes;
  float* scales;
  void* S;
  int num_slots;
  int group;
  unsigned rows;        // rows of a slot: heads * dv
  unsigned blocks;      // CTAs of an entry
  uint32_t two23;       // the bits of 2^23 (see StreamParams)
};

template <class E>
__device__ __forceinline__ void load8(float (&x)[8], const typename E::T* p) {
  static_assert(E::kTag == QS_F32, "32 bytes");
  asm volatile("ld.global.cg.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
               : "l"(p));
}

template <class E>
__device__ __forceinline__ void store8(typename E::T* p, const float (&x)[8]) {
  static_assert(E::kTag == QS_F32, "32 bytes");
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
               "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}

// A lane's 16 elements as they are in memory: 16 words of FP32, 8 of a
// 16-bit type.
template <class E>
struct Row16 {
  static constexpr int W = E::kTag == QS_F32 ? 16 : 8;
  uint32_t w[W];
  __device__ __forceinline__ void load(const typename E::T* p) {
#pragma unroll
    for (int i = 0; i < W; i += 8)
      asm volatile("ld.global.cg.v8.u32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]),
                     "=r"(w[i + 6]), "=r"(w[i + 7])
                   : "l"(reinterpret_cast<const uint32_t*>(p) + i));
  }
  __device__ __forceinline__ void store(typename E::T* p) const {
#pragma unroll
    for (int i = 0; i < W; i += 8)
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(reinterpret_cast<uint32_t*>(p) + i),
                   "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]),
                   "r"(w[i + 7])
                   : "memory");
  }
  __device__ __forceinline__ float2 pair(int m) const {
    if constexpr (E::kTag == QS_F32) {
      return make_float2(__uint_as_float(w[2 * m]), __uint_as_float(w[2 * m + 1]));
    } else {
      return E::widen2(w[m]);
    }
  }
  __device__ __forceinline__ void set(int m, float2 v) {
    if constexpr (E::kTag == QS_F32) {
      w[2 * m] = __float_as_uint(v.x);
      w[2 * m + 1] = __float_as_uint(v.y);
    } else {
      w[m] = E::narrow2(v.x, v.y);
    }
  }
};

// The rows a thread of one entry's CTA works on: row0 + u * RPB, of `rows`,
// at columns col .. col + 15.
template <int DK>
struct CachePlace {
  static constexpr int LPR = DK / kCacheCols;       // lanes per row
  static constexpr int RPB = kCacheThreads / LPR;   // rows of one pass of a CTA
  unsigned entry, row0, col;
  __device__ __forceinline__ explicit CachePlace(unsigned blocks) {
    entry = blockIdx.x / blocks;
    row0 = (blockIdx.x - entry * blocks) * (RPB * kCacheUnroll) + threadIdx.x / LPR;
    col = kCacheCols * (threadIdx.x % LPR);
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
  const typename E::T* src = static_cast<const typename E::T*>(p.S) +
                             (static_cast<size_t>(at.entry) * p.rows + at.row0) * DK + at.col;
  Row16<E> in[kCacheUnroll];
#pragma unroll
  for (int u = 0; u < kCacheUnroll; ++u) {
    if (at.row0 + u * Pl::RPB < p.rows) {
      in[u].load(src + u * Pl::RPB * DK);
    } else {
#pragma unroll
      for (int i = 0; i < Row16<E>::W; ++i) in[u].w[i] = 0u;
    }
  }
  const int slot = __ldg(p.slots + at.entry);  // the states' loads above do not wait for it
  if (slot < 0 || slot >= p.num_slots) return;
  const size_t row = static_cast<size_t>(slot) * p.rows + at.row0;
  uint8_t* const codes = p.codes + (row * DK + at.col) * BITS / 8;
  const unsigned ng = DK / p.group;
  float* const scales = p.scales + row * ng + at.col / p.group;
  const bool writes_scale = at.col % p.group == 0;
#pragma unroll
  for (int u = 0; u < kCacheUnroll; ++u) {
    float2 x[8];
    float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = in[u].pair(i);
      m0 = fmaxf(m0, fabsf(x[i].x));
      m1 = fmaxf(m1, fabsf(x[i].y));
    }
    float m = fmaxf(m0, m1);
    // every lane of the warp takes the shuffles, rows behind the last too
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    if (p.group >= 64) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (p.group >= 128) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
    const float s = div_qmax_rn<QMAX>(m);
    const bool zero = !(s > 0.0f), general = !(s >= 0x1p-126f && s < 0x1p126f);
    const float inv = zero ? 0.0f : recip_rn(s);
    float2 y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __ffma2_rn(x[i], f2(inv), f2(kOff));
    if (general) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i].x = zero ? kOff : fminf(fmaxf(y[i].x, kOff - kQ), kOff + kQ);
        y[i].y = zero ? kOff : fminf(fmaxf(y[i].y, kOff - kQ), kOff + kQ);
      }
    }
    if (at.row0 + u * Pl::RPB >= p.rows) continue;
    uint8_t* const c = codes + u * (Pl::RPB * DK * BITS / 8);
    if constexpr (BITS == 8) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = __byte_perm(__byte_perm(__float_as_uint(y[2 * q].x), __float_as_uint(y[2 * q].y), 0x0040u),
                           __byte_perm(__float_as_uint(y[2 * q + 1].x), __float_as_uint(y[2 * q + 1].y), 0x0040u),
                           0x5410u) ^ 0x80808080u;
      *reinterpret_cast<uint4*>(c) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      uint32_t w[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t by[4];
#pragma unroll
        for (int b = 0; b < 4; ++b)
          by[b] = (__float_as_uint(y[4 * q + b].y) << 4) + __float_as_uint(y[4 * q + b].x);
        w[q] = __byte_perm(__byte_perm(by[0], by[1], 0x0040u), __byte_perm(by[2], by[3], 0x0040u), 0x5410u) ^ 0x88888888u;
      }
      *reinterpret_cast<uint2*>(c) = make_uint2(w[0], w[1]);
    }
    if (writes_scale) scales[u * Pl::RPB * ng] = s;
  }
}

// S = code * scale.
template <int BITS, int DK, class E>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(CacheParams p) {
  constexpr int CW = BITS / 2;  // code words of a lane
  using Pl = CachePlace<DK>;
  const Pl at(p.blocks);
  const int slot = __ldg(p.slots + at.entry);
  if (slot < 0 || slot >= p.num_slots) return;
  typename E::T* const dst = static_cast<typename E::T*>(p.S) +
                             (static_cast<size_t>(at.entry) * p.rows + at.row0) * DK + at.col;
  const size_t row = static_cast<size_t>(slot) * p.rows + at.row0;
  const uint8_t* const codes = p.codes + (row * DK + at.col) * BITS / 8;
  const unsigned ng = DK / p.group;
  const float* const scales = p.scales + row * ng + at.col / p.group;
  uint32_t w[kCacheUnroll][CW];
  float s[kCacheUnroll];
#pragma unroll
  for (int u = 0; u < kCacheUnroll; ++u) {
    s[u] = 0.0f;
#pragma unroll
    for (int i = 0; i < CW; ++i) w[u][i] = 0u;
    if (at.row0 + u * Pl::RPB < p.rows) {
      const uint8_t* const c = codes + u * (Pl::RPB * DK * BITS / 8);
      if constexpr (BITS == 8) {
        const uint4 t = __ldcg(reinterpret_cast<const uint4*>(c));
        w[u][0] = t.x, w[u][1] = t.y, w[u][2] = t.z, w[u][3] = t.w;
      } else {
        const uint2 t = __ldcg(reinterpret_cast<const uint2*>(c));
        w[u][0] = t.x, w[u][1] = t.y;
      }
      s[u] = __ldcg(scales + u * Pl::RPB * ng);
    }
  }
#pragma unroll
  for (int u = 0; u < kCacheUnroll; ++u) {
    if (at.row0 + u * Pl::RPB >= p.rows) continue;
    Row16<E> out;
#pragma unroll
    for (int q = 0; q < CW; ++q) {
      if constexpr (BITS == 8) {
        // 2^23 + (code + 128), less the offset
        const uint32_t x = w[u][q] ^ 0x80808080u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 c = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(x, p.two23, 0x7540u | (2 * h))),
                                                  __uint_as_float(__byte_perm(x, p.two23, 0x7540u | (2 * h + 1)))),
                                      f2(-(0x1p23f + 128.0f)));
          out.set(2 * q + h, __fmul2_rn(c, f2(s[u])));
        }
      } else {
        // 2^23 + 16^i (code + 8) for nibble i of a 16-bit half, scaled back
        // and less the offset in one exact multiply-add
        const float2 r01 = make_float2(1.0f, 0x1p-4f), r23 = make_float2(0x1p-8f, 0x1p-12f);
        const float2 b01 = make_float2(-(0x1p23f + 8.0f), -(0x1p19f + 8.0f));
        const float2 b23 = make_float2(-(0x1p15f + 8.0f), -(0x1p11f + 8.0f));
        const uint32_t lo = w[u][q] ^ 0x88888888u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t v = h ? lo >> 16 : lo;
          const float2 c0 = __ffma2_rn(make_float2(__uint_as_float((v & 0xFu) | p.two23), __uint_as_float((v & 0xF0u) | p.two23)), r01, b01);
          const float2 c1 = __ffma2_rn(make_float2(__uint_as_float((v & 0xF00u) | p.two23), __uint_as_float((v & 0xF000u) | p.two23)), r23, b23);
          out.set(4 * q + 2 * h, __fmul2_rn(c0, f2(s[u])));
          out.set(4 * q + 2 * h + 1, __fmul2_rn(c1, f2(s[u])));
        }
      }
    }
    out.store(dst + u * Pl::RPB * DK);
  }
}

}  // namespace qs
