// Counter-based dropout masks and 8-column access to rows of float32 or bfloat16, shared by the
// kernels of the residual stream (dropout.cu, embedding.cu, block_norm.cu).
//
// Element (r, c) of a [rows, cols] tensor has 16 random bits, a function of (seed, offset, r, c) alone:
// the generator is Philox4x32-10 (J. Salmon et al., "Parallel random numbers: as easy as 1, 2, 3",
// SC 2011), its counter (b, o) of two 64-bit words, b = r * ceil(cols / 8) + c / 8, its key the seed; the
// eight elements of a block take the halves of the four output words in order.  So one call serves the
// 16 bytes of bfloat16 that a thread loads, and any kernel that meets the element, forward or backward
// and whatever its layout, finds the same bits.  16 bits, not 32: the ten rounds are 20 wide products,
// and at four elements a call they, not the memory, would bound a bfloat16 pass.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"

namespace esm {

// A dropout as the kernels take it: rng NULL: none; kept if the 16 bits are >= threshold (1..65536),
// kept values times scale = 65536 / (65536 - threshold).
struct DropMask {
  const unsigned long long* rng;  // device: seed, base
  unsigned long long offset;      // added to the base
  unsigned threshold;
  float scale;
};

// n / d for n below 2^31 by a product: with s = ceil(log2 d) and m = ceil(2^(31 + s) / d), m d exceeds 2^(31 + s)
// by less than d <= 2^s, so floor(n m / 2^(31 + s)) is exact (Granlund and Montgomery, PLDI 1994).
struct FastDiv {
  uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return FastDiv{d, (uint32_t)(((1ull << (31 + s)) + d - 1) / d), s};
}

#ifdef __CUDACC__

__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv& f) {
  return (uint32_t)(((unsigned long long)n * f.m) >> 31 >> f.s);
}

// ---- eight values as four pairs (two to an instruction) ----
using Pairs = uint64_t[4];

__device__ __forceinline__ uint64_t f2_both(float x) { return f2_pack(x, x); }
__device__ __forceinline__ float f2_lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float f2_hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ float f2_sum(uint64_t v) { return f2_lo(v) + f2_hi(v); }
__device__ __forceinline__ uint64_t bf16x2_pair(uint32_t w) {
  return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pair_bf16x2(uint64_t v) { return pack_bf16x2(f2_lo(v), f2_hi(v)); }
__device__ __forceinline__ void fill(Pairs& v, float x) { v[0] = v[1] = v[2] = v[3] = f2_both(x); }
__device__ __forceinline__ float sum(const Pairs& v) { return f2_sum(f2_add(f2_add(v[0], v[1]), f2_add(v[2], v[3]))); }

// ---- random bits ----
struct PhiloxState {
  uint32_t k0, k1;  // key
  uint32_t o0, o1;  // upper 64 bits of the counter
  uint32_t least;   // 65536 threshold
};

__device__ __forceinline__ PhiloxState philox_state(const DropMask& m) {
  if (m.rng == nullptr) return PhiloxState{0, 0, 0, 0, 0};
  const unsigned long long seed = __ldg(m.rng), o = __ldg(m.rng + 1) + m.offset;
  return PhiloxState{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)o, (uint32_t)(o >> 32), min(m.threshold, 65535u) << 16};
}

constexpr uint32_t kPhiloxKey0 = 0x9E3779B9u, kPhiloxKey1 = 0xBB67AE85u;

__device__ __forceinline__ void philox_round(uint4& c, uint32_t k0, uint32_t k1) {
  const unsigned long long p0 = (unsigned long long)c.x * 0xD2511F53u, p1 = (unsigned long long)c.z * 0xCD9E8D57u;
  c = make_uint4((uint32_t)(p1 >> 32) ^ c.y ^ k0, (uint32_t)p1, (uint32_t)(p0 >> 32) ^ c.w ^ k1, (uint32_t)p0);
}

// The four output words of block b; elements 2 j and 2 j + 1 of the block are kept if the lower and upper
// halves of word j are not below the threshold (which no half is without a dropout, and every half is at
// threshold 65536).
__device__ __forceinline__ uint4 drop_words(const DropMask& m, const PhiloxState& s, unsigned long long b) {
  if (m.rng == nullptr) return make_uint4(~0u, ~0u, ~0u, ~0u);
  if (m.threshold > 65535u) return make_uint4(0u, 0u, 0u, 0u);
  uint4 c = make_uint4((uint32_t)b, (uint32_t)(b >> 32), s.o0, s.o1);
#pragma unroll
  for (int i = 0; i < 10; ++i) philox_round(c, s.k0 + i * kPhiloxKey0, s.k1 + i * kPhiloxKey1);
  return c;
}

// The same with the ten rounds' keys in shared memory (written by philox_keys): one call has nothing to
// share the 18 additions with, and five 16-byte reads take their place.
struct PhiloxKeys {
  uint4 k[5];
};
__device__ __forceinline__ void philox_keys(const PhiloxState& s, PhiloxKeys* shared) {
  for (int i = threadIdx.x; i < 5; i += blockDim.x)
    shared->k[i] = make_uint4(s.k0 + 2 * i * kPhiloxKey0, s.k1 + 2 * i * kPhiloxKey1, s.k0 + (2 * i + 1) * kPhiloxKey0,
                              s.k1 + (2 * i + 1) * kPhiloxKey1);
}
__device__ __forceinline__ uint4 drop_words(const DropMask& m, const PhiloxState& s, const PhiloxKeys* shared,
                                            unsigned long long b) {
  if (m.rng == nullptr) return make_uint4(~0u, ~0u, ~0u, ~0u);
  if (m.threshold > 65535u) return make_uint4(0u, 0u, 0u, 0u);
  uint4 c = make_uint4((uint32_t)b, (uint32_t)(b >> 32), s.o0, s.o1);
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const uint4 k = shared->k[i];
    philox_round(c, k.x, k.y);
    philox_round(c, k.z, k.w);
  }
  return c;
}

// v where the element is kept, else 0 (whatever v is).
__device__ __forceinline__ uint64_t keep_pair(uint32_t word, uint32_t least, uint64_t v) {
  return f2_pack((word << 16) >= least ? f2_lo(v) : 0.f, word >= least ? f2_hi(v) : 0.f);
}
__device__ __forceinline__ void keep(const uint4& w, const PhiloxState& s, Pairs& v) {
  v[0] = keep_pair(w.x, s.least, v[0]);
  v[1] = keep_pair(w.y, s.least, v[1]);
  v[2] = keep_pair(w.z, s.least, v[2]);
  v[3] = keep_pair(w.w, s.least, v[3]);
}

// ---- eight values of a row per lane, 256 columns per warp and step ----
// VEC: lane l holds columns 8 l .. 8 l + 7 of the span (one access; a row's eights aligned);
// otherwise columns l, l + 32, ..., l + 224 (scalar accesses, coalesced whatever the rows' alignment).
template <bool VEC>
__device__ __forceinline__ int span_col(int lane, int k) {
  return VEC ? 8 * lane + k : 32 * k + lane;
}

// The words with a lane's eight columns' bits.  They come per block of eight consecutive columns, so without
// VEC lane l draws block l of the span, and the lanes exchange them: column 32 k + l is element l % 8 of block
// 4 k + l / 8.  Every lane of the warp takes part.
template <bool VEC>
__device__ __forceinline__ uint4 span_words(const DropMask& m, const uint4& own, int lane) {
  if constexpr (VEC) {
    return own;
  } else {
    if (m.rng == nullptr) return own;
    uint32_t out[4];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int from = 4 * k + lane / 8;
      const uint32_t a = __shfl_sync(0xffffffffu, own.x, from), b = __shfl_sync(0xffffffffu, own.y, from),
                     c = __shfl_sync(0xffffffffu, own.z, from), d = __shfl_sync(0xffffffffu, own.w, from);
      const uint32_t word = lane & 4 ? (lane & 2 ? d : c) : (lane & 2 ? b : a);
      const uint32_t half = lane & 1 ? word >> 16 : word & 0xffffu;
      out[k / 2] = k & 1 ? out[k / 2] | half << 16 : half;
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
  }
}

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ void ld8(const float* p, Pairs& v) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(p), b = *reinterpret_cast<const ulonglong2*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}
__device__ __forceinline__ void ld8(const __nv_bfloat16* p, Pairs& v) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  v[0] = bf16x2_pair(a.x); v[1] = bf16x2_pair(a.y); v[2] = bf16x2_pair(a.z); v[3] = bf16x2_pair(a.w);
}
__device__ __forceinline__ void st8(float* p, const Pairs& v) {
  asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p), "l"(v[0]), "l"(v[1]), "l"(v[2]), "l"(v[3]) : "memory");
}
__device__ __forceinline__ void st8(__nv_bfloat16* p, const Pairs& v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pair_bf16x2(v[0]), pair_bf16x2(v[1]), pair_bf16x2(v[2]), pair_bf16x2(v[3]));
}

// A lane's eight values of 256 in shared memory.  Of float32 ones four lanes in eight begin with the upper half, so
// that eight lanes meet all banks.
__device__ __forceinline__ void ld8_shared(const float* p, int lane, Pairs& v) {
  const bool upper = lane & 4;
  const int at = 8 * lane + (lane & 4);
  const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(p + at), s = *reinterpret_cast<const ulonglong2*>(p + (at ^ 4));
  v[0] = upper ? s.x : f.x; v[1] = upper ? s.y : f.y; v[2] = upper ? f.x : s.x; v[3] = upper ? f.y : s.y;
}
__device__ __forceinline__ void ld8_shared(const __nv_bfloat16* p, int lane, Pairs& v) { ld8(p + 8 * lane, v); }

// Eight values as they stand in memory, to be on the way in as few registers as they need.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void get(Pairs& out) const {
    if constexpr (sizeof(T) == 2) {
      out[0] = bf16x2_pair(v[0].x); out[1] = bf16x2_pair(v[0].y);
      out[2] = bf16x2_pair(v[0].z); out[3] = bf16x2_pair(v[0].w);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        out[2 * i] = (uint64_t)v[i].y << 32 | v[i].x;
        out[2 * i + 1] = (uint64_t)v[i].w << 32 | v[i].z;
      }
    }
  }
  // Of a row with aligned eights, `left` values to its end: those past it are 0.  Eight float32 are one access of 32
  // bytes, a whole sector: in two halves the 16384 x 1280 block norms took 48 and 81 us where they take 46 and 74.
  __device__ __forceinline__ void load(const T* p, int left) {
    if (left >= 8) {
      if constexpr (sizeof(T) == 4) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y),
                       "=r"(v[1].z), "=r"(v[1].w)
                     : "l"(p));
        return;
      }
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
      return;
    }
    T* to = reinterpret_cast<T*>(v);
#pragma unroll
    for (int k = 0; k < 8; ++k) to[k] = k < left ? p[k] : T(0.f);
  }
};

// A lane's eight values of the span that starts at `row` with `left` columns to the row's end; columns
// past the end read as 0 and are not written.
template <bool VEC, typename T>
__device__ __forceinline__ void span_load(const T* row, int left, int lane, Pairs& v) {
  if (VEC && 8 * lane + 8 <= left) {
    ld8(row + 8 * lane, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = span_col<VEC>(lane, 2 * i), d = span_col<VEC>(lane, 2 * i + 1);
    v[i] = f2_pack(c < left ? ld1(row + c) : 0.f, d < left ? ld1(row + d) : 0.f);
  }
}
template <bool VEC, typename T>
__device__ __forceinline__ void span_store(T* row, int left, int lane, const Pairs& v) {
  if (VEC && 8 * lane + 8 <= left) {
    st8(row + 8 * lane, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = span_col<VEC>(lane, 2 * i), d = span_col<VEC>(lane, 2 * i + 1);
    if (c < left) st1(row + c, f2_lo(v[i]));
    if (d < left) st1(row + d, f2_hi(v[i]));
  }
}
// 0 in the places past the row's end.
template <bool VEC>
__device__ __forceinline__ void span_trim(int left, int lane, Pairs& v) {
  if (VEC && 8 * lane + 8 <= left) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = f2_pack(span_col<VEC>(lane, 2 * i) < left ? f2_lo(v[i]) : 0.f,
                   span_col<VEC>(lane, 2 * i + 1) < left ? f2_hi(v[i]) : 0.f);
}

#endif  // __CUDACC__

}  // namespace esm
