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

// A dropout as the kernels take it: rng NULL: none; kept if the 16 bits are >= threshold (0..65536),
// kept values times scale = 65536 / (65536 - threshold).
struct DropMask {
  const unsigned long long* rng;  // device: seed, base
  unsigned long long offset;      // added to the base
  unsigned threshold;
  float scale;
};

#ifdef __CUDACC__

struct PhiloxState {
  uint32_t k0, k1;  // key
  uint32_t o0, o1;  // upper 64 bits of the counter
};

__device__ __forceinline__ PhiloxState philox_state(const DropMask& m) {
  if (m.rng == nullptr) return PhiloxState{0, 0, 0, 0};
  const unsigned long long seed = __ldg(m.rng), o = __ldg(m.rng + 1) + m.offset;
  return PhiloxState{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)o, (uint32_t)(o >> 32)};
}

__device__ __forceinline__ uint4 philox(const PhiloxState& s, unsigned long long b) {
  uint32_t c0 = (uint32_t)b, c1 = (uint32_t)(b >> 32), c2 = s.o0, c3 = s.o1, k0 = s.k0, k1 = s.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const unsigned long long p0 = (unsigned long long)c0 * 0xD2511F53u, p1 = (unsigned long long)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Bit j: element j of block b is kept (all of them without a dropout).  With n >= 1, bits u are kept if
// u > n - 1: the upper half of a word w is if w > (n - 1) * 65536 + 65535, the lower one if 65536 w is.
__device__ __forceinline__ uint32_t keep8(const DropMask& m, const PhiloxState& s, unsigned long long b) {
  if (m.rng == nullptr) return 0xffu;
  const uint4 w = philox(s, b);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w}, limit = (m.threshold << 16) - 1u;
  uint32_t bits = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if ((u[j] << 16) > limit) bits |= 1u << (2 * j);
    if (u[j] > limit) bits |= 2u << (2 * j);
  }
  return bits;
}

// ---- eight values of a row per lane, 256 columns per warp and step ----
// VEC: lane l holds columns 8 l .. 8 l + 7 of the span (16-byte accesses; rows on 16-byte boundaries);
// otherwise columns l, l + 32, ..., l + 224 (scalar accesses, coalesced whatever the rows' alignment).
template <bool VEC>
__device__ __forceinline__ int span_col(int lane, int k) {
  return VEC ? 8 * lane + k : 32 * k + lane;
}

// The keep bits of a lane's eight columns.  Bits come per block of eight consecutive columns, so without
// VEC lane l draws block l of the span and the lanes exchange them: column 32 k + l is element l % 8 of
// block 4 k + l / 8.  Every lane of the warp takes part.
template <bool VEC>
__device__ __forceinline__ uint32_t span_keep(const DropMask& m, const PhiloxState& s, unsigned long long first_block,
                                              int lane) {
  const uint32_t own = keep8(m, s, first_block + lane);
  if (VEC || m.rng == nullptr) return own;
  uint32_t bits = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) bits |= (__shfl_sync(0xffffffffu, own, 4 * k + lane / 8) >> (lane % 8) & 1u) << k;
  return bits;
}

__device__ __forceinline__ float2 bf16x2_to_f2(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ void ld8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void ld8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16x2_to_f2(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void st8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void st8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}

// A lane's eight values of the span that starts at `row` with `left` columns to the row's end; columns
// past the end read as 0 and are not written.
template <bool VEC, typename T>
__device__ __forceinline__ void span_load(const T* row, int left, int lane, float (&v)[8]) {
  if (VEC && 8 * lane + 8 <= left) {
    ld8(row + 8 * lane, v);
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = span_col<VEC>(lane, k) < left ? ld1(row + span_col<VEC>(lane, k)) : 0.f;
}
template <bool VEC, typename T>
__device__ __forceinline__ void span_store(T* row, int left, int lane, const float (&v)[8]) {
  if (VEC && 8 * lane + 8 <= left) {
    st8(row + 8 * lane, v);
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (span_col<VEC>(lane, k) < left) st1(row + span_col<VEC>(lane, k), v[k]);
}

// Eight values of a lane as they stand in memory: four registers for bfloat16, which kernels keep or stage.
template <typename T, bool VEC>
struct Span8 {
  float v[8];
  __device__ __forceinline__ void load(const T* row, int left, int lane) { span_load<VEC>(row, left, lane, v); }
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = x;
  }
  __device__ __forceinline__ void get(float (&out)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) out[k] = v[k];
  }
};
template <>
struct Span8<__nv_bfloat16, true> {
  uint32_t v[4];
  // (the row's length is a multiple of 8 here)
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int left, int lane) {
    const uint4 a = 8 * lane < left ? __ldg(reinterpret_cast<const uint4*>(row + 8 * lane)) : make_uint4(0, 0, 0, 0);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  }
  __device__ __forceinline__ void fill(float x) { v[0] = v[1] = v[2] = v[3] = pack_bf16x2(x, x); }
  __device__ __forceinline__ void get(float (&out)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = bf16x2_to_f2(v[i]);
      out[2 * i] = f.x;
      out[2 * i + 1] = f.y;
    }
  }
};

// ---- a thread's own eight values of rows to come, copied ahead into shared memory ----
// Chunk c of 16 bytes of thread t stands at (c * threads + t) * 16 of its stage, so a warp's accesses are
// conflict-free; a thread reads only what it copied itself, so waiting for its own copies is enough.
template <typename T>
constexpr int kChunks = sizeof(T) / 2;  // 16-byte chunks of eight values

template <typename T>
__device__ __forceinline__ void stage_copy(uint8_t* stage, int chunk, const T* row, int left, int lane) {
#pragma unroll
  for (int i = 0; i < kChunks<T>; ++i) {
    constexpr int per = 16 / sizeof(T);
    const bool in = 8 * lane + per * i < left;
    cp_async_16(stage + ((size_t)(chunk + i) * blockDim.x + threadIdx.x) * 16, row + (in ? 8 * lane + per * i : 0),
                in ? 16u : 0u);
  }
}
template <typename T>
__device__ __forceinline__ void stage_read(const uint8_t* stage, int chunk, float (&v)[8]) {
  const uint8_t* at = stage + ((size_t)chunk * blockDim.x + threadIdx.x) * 16;
  if constexpr (sizeof(T) == 2) {
    ld8(reinterpret_cast<const __nv_bfloat16*>(at), v);
  } else {
    const float4 a = *reinterpret_cast<const float4*>(at);
    const float4 b = *reinterpret_cast<const float4*>(at + (size_t)blockDim.x * 16);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

#endif  // __CUDACC__

}  // namespace esm
