// Embedding lookup with scaling and dropout, and its gradient:
//   out[t] = keep(t, c) * drop_scale * scale * row_scale[t] * table[id_t]     (id -1: zeros)
//   d_table[v] (+)= scale * sum over t with id_t = v of row_scale[t] * keep(t, c) * drop_scale * d_out[t]
// The sums run in a fixed order, so results do not depend on scheduling.
//
// Bound by memory: the rows met and the output; for the gradient d_out and the table's rows.  16384 tokens x 1280:
// lookup in 50021 float32 rows 25.2 us (4.5 TB/s of the bytes that it cannot do without); gradient of 33 ids 24.7 us,
// 22.0 without the dropout (3.8 TB/s; 16 where d_out still lies in the L2: the sort of a chunk before its first row's
// load and the second kernel over the chunks' sums are not hidden), of 50021 64.2 us, of which 38 clear the table.
#include <algorithm>
#include <type_traits>

#include "dropout.cuh"
#include "internal.h"

namespace esm {
namespace {

// An id that has a row, or -1; ids out of range latch ERRBIT_TOKEN.
__device__ __forceinline__ int checked_id(const EmbedArgs& a, int t, bool report) {
  const int id = __ldg(a.ids + t);
  if (id >= 0 && id < a.vocab) return id;
  if (!(a.none && id == -1) && report) latch_error(a.err, ERRBIT_TOKEN);
  return -1;
}

__device__ __forceinline__ float token_scale(const EmbedArgs& a, int t) {
  return a.row_scale ? a.scale * __ldg(a.row_scale + t) : a.scale;
}

// Blocks of eight columns in the order of the tokens, one to a thread: 64 warps an SM hide the way from the id to
// the row (four blocks to a thread and half as many warps took 29 us where this takes 25).  Rows with aligned eights.
template <typename TE, typename TO>
__global__ void __launch_bounds__(256, 8) embed_scaled_kernel(const EmbedArgs a, const FastDiv per_row, long long total) {
  const long long b = (long long)blockIdx.x * 256 + threadIdx.x;
  if (b >= total) return;
  const int t = total <= INT32_MAX ? (int)div_by((uint32_t)b, per_row) : (int)(b / per_row.d);
  const int col = (int)(b - (long long)t * per_row.d) * 8, left = a.cols - col;
  const int id = checked_id(a, t, col == 0);
  Raw8<TE> x;
  if (id >= 0) x.load(static_cast<const TE*>(a.table) + (long long)id * a.cols + col, left);
  const float f = token_scale(a, t) * a.mask.scale;
  Pairs v;
  fill(v, 0.f);
  if (id >= 0) {
    x.get(v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2_mul(v[i], f2_both(f));
    if (a.mask.rng) {
      const PhiloxState ps = philox_state(a.mask);
      keep(drop_words(a.mask, ps, (unsigned long long)b), ps, v);
    }
  }
  span_store<true>(static_cast<TO*>(a.out) + (long long)t * a.out_stride + col, left, 0, v);
}

// Rows whose eights are not aligned: one warp per 256 columns of a token.
template <typename TE, typename TO>
__global__ void __launch_bounds__(256) embed_rows_kernel(const EmbedArgs a, const FastDiv spans, long long total) {
  const PhiloxState ps = philox_state(a.mask);
  const int lane = threadIdx.x & 31;
  const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5), per_row = (a.cols + 7) / 8;
  if (i >= total) return;
  const int t = total <= INT32_MAX ? (int)div_by((uint32_t)i, spans) : (int)(i / spans.d);
  const int c0 = (int)(i - (long long)t * spans.d) * 256, left = a.cols - c0, id = checked_id(a, t, lane == 0 && c0 == 0);
  Pairs v;
  fill(v, 0.f);
  if (id >= 0) {
    span_load<false>(static_cast<const TE*>(a.table) + (long long)id * a.cols + c0, left, lane, v);
    const uint4 own = drop_words(a.mask, ps, (unsigned long long)(t * per_row + c0 / 8 + lane));
    const uint64_t f = f2_both(token_scale(a, t) * a.mask.scale);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = f2_mul(v[k], f);
    keep(span_words<false>(a.mask, own, lane), ps, v);
  }
  span_store<false>(static_cast<TO*>(a.out) + t * a.out_stride + c0, left, lane, v);
}

// acc += keep(token t, block of the lane) * f * g
template <bool VEC>
__device__ __forceinline__ void add_token(const EmbedArgs& a, const PhiloxState& ps, const PhiloxKeys* keys, int t, int c0,
                                          int lane, float f, Pairs& g, Pairs& acc) {
  if (a.mask.rng) {
    const unsigned long long b = (unsigned long long)t * ((a.cols + 7) / 8) + c0 / 8 + lane;
    keep(span_words<VEC>(a.mask, drop_words(a.mask, ps, keys, b), lane), ps, g);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = f2_fma(g[i], f2_both(f), acc[i]);
}

// One block per id and 256 columns: its eight warps look through all tokens, 32 at a time in turn, and add the rows
// that they find; their sums are then added in order.
template <typename TO, bool VEC>
__global__ void __launch_bounds__(256) embed_grad_kernel(const EmbedArgs a, const FastDiv spans) {
  __shared__ PhiloxKeys keys;
  __shared__ ulonglong2 sums[8][2][32];  // a lane's eight columns in two halves
  const PhiloxState ps = philox_state(a.mask);
  philox_keys(ps, &keys);
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int v = (int)div_by(blockIdx.x, spans), c0 = (int)(blockIdx.x - v * spans.d) * 256, left = a.cols - c0;
  float* dst = a.d_table + (long long)v * a.cols + c0;
  Pairs acc;
  fill(acc, 0.f);
  bool any = false;
  for (int t0 = 32 * warp; t0 < a.tokens; t0 += 256) {
    const int t = t0 + lane;
    const int id = t < a.tokens ? checked_id(a, t, blockIdx.x == 0) : -1;
    for (uint32_t hit = __ballot_sync(0xffffffffu, id == v); hit; hit &= hit - 1) {
      const int m = t0 + __ffs(hit) - 1;
      Pairs g;
      span_load<VEC>(static_cast<const TO*>(a.out) + m * a.out_stride + c0, left, lane, g);
      add_token<VEC>(a, ps, &keys, m, c0, lane, token_scale(a, m) * a.mask.scale, g, acc);
      any = true;
    }
  }
  sums[warp][0][lane] = make_ulonglong2(acc[0], acc[1]);
  sums[warp][1][lane] = make_ulonglong2(acc[2], acc[3]);
  any = __syncthreads_or(any);
  if (warp || (a.accumulate && !any)) return;
  fill(acc, 0.f);
  if (any) {
    if (a.accumulate) span_load<VEC>(dst, left, lane, acc);
    Pairs total;
    fill(total, 0.f);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const ulonglong2 lo = sums[w][0][lane], hi = sums[w][1][lane];
      total[0] = f2_add(total[0], lo.x); total[1] = f2_add(total[1], lo.y);
      total[2] = f2_add(total[2], hi.x); total[3] = f2_add(total[3], hi.y);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = f2_add(acc[k], total[k]);
  }
  span_store<VEC>(dst, left, lane, acc);
}

// Sums of `count` <= 32 places of a list sorted by id, lane l holding place l's (id, token) and factor, over 256
// columns: leave(id, last, sums) takes each id's.  VEC: aligned eights and cols % 8 == 0.  MASKS_AHEAD: the masks of four
// rows at once while they are on their way, for 16 registers more.
template <typename TO, bool VEC, bool MASKS_AHEAD, typename Leave>
__device__ __forceinline__ void sum_places(const EmbedArgs& a, const PhiloxState& ps, const PhiloxKeys* keys, int c0, int left,
                                           int lane, const uint2& own, float own_scale, int count, Leave leave) {
  constexpr int kAhead = 4;  // rows in flight
  int id = (int)__shfl_sync(0xffffffffu, own.x, 0);
  const bool active = 8 * lane < left;
  Pairs acc;
  fill(acc, 0.f);
  using Row = std::conditional_t<VEC, Raw8<TO>, Pairs>;
  for (int j0 = 0; j0 < count; j0 += kAhead) {
    Row g[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      // (past the end: the last row once more, which is not added)
      const int t = (int)__shfl_sync(0xffffffffu, own.y, min(j0 + j, count - 1));
      const TO* row = static_cast<const TO*>(a.out) + (size_t)t * a.out_stride + c0;
      if constexpr (VEC) g[j].load(row + (active ? 8 * lane : 0), 8);
      else span_load<false>(row, left, lane, g[j]);
    }
    uint4 words[MASKS_AHEAD ? kAhead : 1];
    if (MASKS_AHEAD && a.mask.rng) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const uint32_t t = __shfl_sync(0xffffffffu, own.y, min(j0 + j, count - 1));
        words[j] = drop_words(a.mask, ps, keys, (unsigned long long)t * ((a.cols + 7) / 8) + c0 / 8 + lane);
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int t = (int)__shfl_sync(0xffffffffu, own.y, j0 + j), v = (int)__shfl_sync(0xffffffffu, own.x, j0 + j);
      const float f = __shfl_sync(0xffffffffu, own_scale, j0 + j);
      if (j0 + j >= count) break;
      if (v != id) {
        leave(id, false, acc);
        id = v;
        fill(acc, 0.f);
      }
      Pairs p;
      if constexpr (VEC) {
        g[j].get(p);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = g[j][k];
      }
      if constexpr (MASKS_AHEAD) {
        if (a.mask.rng) keep(words[j], ps, p);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = f2_fma(p[k], f2_both(f), acc[k]);
      } else {
        add_token<VEC>(a, ps, keys, t, c0, lane, f, p, acc);
      }
    }
  }
  leave(id, true, acc);
}

// ---- the gradient of larger batches of few ids: chunks of up to 256 tokens, each sorted by its own block ----
// A block sums a chunk's rows over 256 columns into part[chunk][id]; a second kernel adds the chunks.  Its eight
// warps take up to 32 places each of the chunk's sorted list; an id that goes on over a warp's border leaves parts in
// shared memory, which the warp in which it begins joins in order.
constexpr int kChunk = 256, kShortChunk = 64, kChunkIds = 64, kChunkWarps = kChunk / 32;

template <typename TO, bool VEC>
__global__ void __launch_bounds__(kChunk, 3)
    embed_grad_chunks_kernel(const EmbedArgs a, float* __restrict__ part, const FastDiv spans, int length) {
  __shared__ PhiloxKeys keys;
  __shared__ int hist[kChunkWarps][kChunkIds];  // each warp's counts, then where its tokens of each id go
  __shared__ int counts[kChunkIds], total;
  __shared__ uint2 list[kChunk];  // (id, token)
  __shared__ float scales[kChunk];
  __shared__ ulonglong2 parts[kChunkWarps][2][2][32];  // as of the pieces below: a lane's eight columns in two halves
  grid_dependency_launch();
  const PhiloxState ps = philox_state(a.mask);
  philox_keys(ps, &keys);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = (int)div_by(blockIdx.x, spans), c0 = (int)(blockIdx.x - chunk * spans.d) * 256, left = a.cols - c0;
  for (int i = threadIdx.x; i < kChunkWarps * kChunkIds; i += kChunk) hist[i / kChunkIds][i % kChunkIds] = 0;
  const int t = chunk * length + threadIdx.x;
  const int my_id = (int)threadIdx.x < length && t < a.tokens ? checked_id(a, t, c0 == 0) : -1;
  const float my_scale = my_id >= 0 ? token_scale(a, t) * a.mask.scale : 0.f;
  const uint32_t peers = __match_any_sync(0xffffffffu, my_id);
  const int ahead = __popc(peers & ((1u << lane) - 1));
  __syncthreads();
  if (my_id >= 0 && ahead == 0) hist[warp][my_id] = __popc(peers);
  __syncthreads();
  if (warp == 0) {  // (two ids to a lane)
    int own[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int w = 0; w < kChunkWarps; ++w) own[k] += hist[w][2 * lane + k];
    int incl = own[0] + own[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    int at = incl - own[0] - own[1];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      counts[2 * lane + k] = own[k];
#pragma unroll
      for (int w = 0; w < kChunkWarps; ++w) {
        const int c = hist[w][2 * lane + k];
        hist[w][2 * lane + k] = at;
        at += c;
      }
    }
    if (lane == 31) total = incl;
  }
  __syncthreads();
  if (my_id >= 0) {
    const int place = hist[warp][my_id] + ahead;
    list[place] = make_uint2((uint32_t)my_id, (uint32_t)t);
    scales[place] = my_scale;
  }
  __syncthreads();
  // (four places to a step of a warp)
  const int n = total, per = (n + 4 * kChunkWarps - 1) / (4 * kChunkWarps) * 4, p0 = warp * per, end = p0 + per;
  const int count = min(per, n - p0);
  float* sums = part + (size_t)chunk * a.vocab * a.cols + c0;
  if (count > 0) {
    const uint2 own = lane < count ? list[p0 + lane] : make_uint2(0xffffffffu, 0);
    const float own_scale = lane < count ? scales[p0 + lane] : 0.f;
    const int before = p0 > 0 ? (int)list[p0 - 1].x : -1, after = end < n ? (int)list[end].x : -1;
    // (masks ahead with float32 rows: 30 us for 25)
    constexpr bool kMasksAhead = VEC && sizeof(TO) == 2;
    sum_places<TO, VEC, kMasksAhead>(a, ps, &keys, c0, left, lane, own, own_scale, count, [&](int id, bool last, Pairs& acc) {
      const bool from_before = id == before, goes_on = last && id == after;
      if (from_before || goes_on) {
        parts[warp][from_before ? 0 : 1][0][lane] = make_ulonglong2(acc[0], acc[1]);
        parts[warp][from_before ? 0 : 1][1][lane] = make_ulonglong2(acc[2], acc[3]);
      } else {
        span_store<VEC>(sums + (size_t)id * a.cols, left, lane, acc);
      }
    });
  }
  __syncthreads();
  Pairs acc;
  if (end < n) {
    const uint32_t id = list[end - 1].x;
    if (list[end].x == id && !(p0 > 0 && list[p0 - 1].x == id)) {
      fill(acc, 0.f);
      for (int w = warp; w < kChunkWarps && (w == warp || (per * w < n && list[per * w].x == id)); ++w) {
        const ulonglong2 lo = parts[w][w == warp][0][lane], hi = parts[w][w == warp][1][lane];
        acc[0] = f2_add(acc[0], lo.x); acc[1] = f2_add(acc[1], lo.y);
        acc[2] = f2_add(acc[2], hi.x); acc[3] = f2_add(acc[3], hi.y);
      }
      span_store<VEC>(sums + (size_t)id * a.cols, left, lane, acc);
    }
  }
  fill(acc, 0.f);
  for (int v = warp; v < a.vocab; v += kChunkWarps)
    if (counts[v] == 0) span_store<VEC>(sums + (size_t)v * a.cols, left, lane, acc);
}

// d_table (+)= the chunks' sums: warp w of a block adds chunks w, w + 8, ... of 128 elements, then the warps' sums
// are added in order.  VEC: four elements to a lane in one access.
template <bool VEC>
__global__ void __launch_bounds__(256) embed_grad_add_kernel(const EmbedArgs a, const float* __restrict__ part, int chunks) {
  __shared__ float sums[8][128];
  grid_dependency_wait();
  const size_t n = (size_t)a.vocab * a.cols, first = (size_t)blockIdx.x * 128;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if constexpr (VEC) {
    if (first + 4 * lane < n) {
#pragma unroll 8
      for (int k = warp; k < chunks; k += 8) {
        const float4 v = *reinterpret_cast<const float4*>(part + k * n + first + 4 * lane);
        s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
      }
    }
  } else {
#pragma unroll 2
    for (int k = warp; k < chunks; k += 8)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (first + 4 * lane + e < n) s[e] += part[k * n + first + 4 * lane + e];
  }
  *reinterpret_cast<float4*>(&sums[warp][4 * lane]) = make_float4(s[0], s[1], s[2], s[3]);
  __syncthreads();
  if (threadIdx.x >= 128 || first + threadIdx.x >= n) return;
  float v = a.accumulate ? a.d_table[first + threadIdx.x] : 0.f;
  float own = sums[0][threadIdx.x];
#pragma unroll
  for (int w = 1; w < 8; ++w) own += sums[w][threadIdx.x];
  a.d_table[first + threadIdx.x] = v + own;
}

// ---- the gradient of larger batches: tokens sorted by id, then summed in pieces of 32 ----
// Sorting: one cluster of eight blocks sorts (id, token) by id, token order kept (least significant digit
// first), so that every id's tokens stand together in rising order.  A warp owns a contiguous stretch of the
// list; per pass it counts its digits (lanes with equal digits find each other by match, so one lane writes
// each count and no atomics order anything), the blocks exchange their counts through distributed shared
// memory, and every warp then knows where each of its digits goes.  Up to 8 bits per pass: one pass for
// 256 ids, two for 65536 (16384 tokens: 15.7 us alone; it grows with the tokens, as eight SMs take them: a gradient of
// 65536 tokens of 300 ids takes 46 us at 128 columns, 62 at 480).  The rest of the grid meanwhile clears d_table (rows that the
// sort may not name left to the sums' launch: 69 us and more where all of it takes 66).
constexpr int kSortBlocks = 8, kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 8, kBins = 1 << kDigitBits;

struct SortArgs {
  uint2 *list, *other;  // (id, token); the last pass writes list
  int* valid;      // tokens with a row
  int passes, digit_bits;
};

__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __cluster_dims__(kSortBlocks, 1, 1) __launch_bounds__(kSortThreads)
    embed_sort_kernel(const EmbedArgs a, const SortArgs s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dependency_launch();
  if (blockIdx.x >= kSortBlocks) {
    // (d_table is zeroed in 16-byte steps where it allows them)
    const size_t n = (size_t)a.vocab * a.cols, step = (size_t)(gridDim.x - kSortBlocks) * kSortThreads;
    const size_t first = (size_t)(blockIdx.x - kSortBlocks) * kSortThreads + tid;
    const size_t n4 = (reinterpret_cast<uintptr_t>(a.d_table) & 15) == 0 ? n / 4 : 0;
    for (size_t i = first; i < n4; i += step) reinterpret_cast<float4*>(a.d_table)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (size_t i = 4 * n4 + first; i < n; i += step) a.d_table[i] = 0.f;
    return;
  }
  constexpr int kRow = kBins + 1;  // (lanes read a column without bank conflicts)
  __shared__ int hist[kSortWarps * kRow];  // each warp's counts, then the next place of each digit within the block
  __shared__ int block_count[kBins], start[kBins];
  __shared__ int warp_total[kSortWarps];
  const int rank = (int)cluster_ctarank(), bins = 1 << s.digit_bits;
  int* mine = hist + warp * kRow;
  int n = a.tokens;
  for (int pass = 0; pass < s.passes; ++pass) {
    const uint2* src = (s.passes - pass) & 1 ? s.other : s.list;
    uint2* dst = (s.passes - pass) & 1 ? s.list : s.other;
    const int shift = pass * s.digit_bits;
    const int stretch = ((n + kSortBlocks * kSortWarps - 1) / (kSortBlocks * kSortWarps) + 31) & ~31;
    const long long begin = (long long)(rank * kSortWarps + warp) * stretch;
    const int end = (int)min((long long)n, begin + stretch);
    for (int d = lane; d < bins; d += 32) mine[d] = 0;
    __syncwarp();
    auto item = [&](long long i) -> uint2 {  // an id of -1: none
      if (i >= end) return make_uint2(0xffffffffu, 0);
      if (pass) return __ldcg(src + i);
      return make_uint2((uint32_t)checked_id(a, (int)i, true), (uint32_t)i);
    };
    // (the first two steps' items are kept for the second time round)
    uint2 kept[2];
    uint32_t kept_peers[2];
    auto digit = [&](const uint2& v) { return v.x == 0xffffffffu ? kBins : (int)(v.x >> shift) & (bins - 1); };
    auto count = [&](int d, uint32_t peers) {
      if (d < kBins && lane == __ffs(peers) - 1) mine[d] += __popc(peers);
      __syncwarp();
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) kept[i] = item(begin + 32 * i + lane);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      kept_peers[i] = __match_any_sync(0xffffffffu, digit(kept[i]));
      count(digit(kept[i]), kept_peers[i]);
    }
    for (long long i0 = begin + 64; i0 < end; i0 += 32) {
      const int d = digit(item(i0 + lane));
      count(d, __match_any_sync(0xffffffffu, d));
    }
    __syncthreads();
    // counts of the warps before, and the block's: a warp per digit, a lane per warp's count
    for (int d = warp; d < bins; d += kSortWarps) {
      const int own = hist[lane * kRow + d];
      int incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      hist[lane * kRow + d] = incl - own;
      if (lane == 31) block_count[d] = incl;
    }
    __syncwarp();
    cluster_sync();
    int total = 0, before = 0;
    if (tid < bins) {
#pragma unroll
      for (int r = 0; r < kSortBlocks; ++r) {
        const int c = ld_cluster(map_to_rank(block_count + tid, r));
        total += c;
        if (r < rank) before += c;
      }
    }
    // where each digit starts: exclusive scan of the totals
    int incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) warp_total[warp] = incl;
    __syncthreads();
    int lower = 0, all = 0;
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = warp_total[w];
      if (w < warp) lower += c;
      all += c;
    }
    if (tid < bins) start[tid] = lower + incl - total + before;
    __syncthreads();
    const bool last = pass == s.passes - 1;
    if (last) cluster_arrive();  // (this block has read the others' counts)
    auto place = [&](const uint2& v, uint32_t peers) {
      const int d = digit(v), ahead = __popc(peers & ((1u << lane) - 1));
      if (d < kBins) dst[start[d] + mine[d] + ahead] = v;
      __syncwarp();
      if (d < kBins && ahead == 0) mine[d] += __popc(peers);
      __syncwarp();
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) place(kept[i], kept_peers[i]);
    for (long long i0 = begin + 64; i0 < end; i0 += 32) {
      const uint2 v = item(i0 + lane);
      place(v, __match_any_sync(0xffffffffu, digit(v)));
    }
    n = all;
    // the next pass reads what all blocks have placed; and none counts again, or leaves, while another still
    // reads its counts
    if (last) cluster_wait();
    else cluster_sync();
  }
  if (rank == 0 && tid == 0) *s.valid = n;
}

// Sums of 32 consecutive places of the sorted list and 256 columns by one warp.  An id whose tokens all lie
// within the piece is written at once; of an id that goes on over the piece's border the piece keeps its part:
// part[piece][0] for one that began before, part[piece][1] for one that begins here and goes on.
constexpr int kPiece = 32;

template <typename TO, bool VEC>
__global__ void __launch_bounds__(32, 24)
    embed_grad_pieces_kernel(const EmbedArgs a, const uint2* __restrict__ list, const int* __restrict__ valid,
                             float* __restrict__ part, const FastDiv spans, long long total) {
  __shared__ PhiloxKeys keys;
  const PhiloxState ps = philox_state(a.mask);
  philox_keys(ps, &keys);
  __syncthreads();
  grid_dependency_wait();
  grid_dependency_launch();
  const int lane = threadIdx.x, n = *valid;
  const long long i = blockIdx.x;
  const int piece = total <= INT32_MAX ? (int)div_by((uint32_t)i, spans) : (int)(i / spans.d);
  const int c0 = (int)(i - (long long)piece * spans.d) * 256, left = a.cols - c0;
  const int p0 = piece * kPiece, count = min(kPiece, n - p0);
  if (count <= 0) return;
  const uint2 own = lane < count ? list[p0 + lane] : make_uint2(0xffffffffu, 0);
  const float own_scale = lane < count ? token_scale(a, (int)own.y) * a.mask.scale : 0.f;
  const int before = p0 > 0 ? (int)list[p0 - 1].x : -1, after = p0 + kPiece < n ? (int)list[p0 + kPiece].x : -1;
  // (65536 x 1280, 65 ids: masks ahead 91.5 us, one by one 94.7; in bfloat16 84 and 106)
  sum_places<TO, VEC, VEC>(a, ps, &keys, c0, left, lane, own, own_scale, count, [&](int id, bool last, Pairs& acc) {
    const bool from_before = id == before, goes_on = last && id == after;
    if (from_before || goes_on) {
      span_store<VEC>(part + ((size_t)piece * 2 + (from_before ? 0 : 1)) * a.cols + c0, left, lane, acc);
      return;
    }
    float* dst = a.d_table + (size_t)id * a.cols + c0;
    if (a.accumulate) {
      Pairs old;
      span_load<VEC>(dst, left, lane, old);
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] = f2_add(acc[k], old[k]);
    }
    span_store<VEC>(dst, left, lane, acc);
  });
}

// Ids that cross borders: one warp per piece in which such an id begins and 256 columns adds its parts in order; one
// that goes on over more than kAlone further pieces is left to the block, whose warps add every eighth part, then
// their sums in order.  (131072 x 1280, 5000 ids: the whole gradient takes 193 us, 270 where all tokens have one id; with
// a block for every id it took 226 and 463.)
constexpr int kAlone = 8;

template <bool VEC>
__global__ void __launch_bounds__(256) embed_grad_join_kernel(const EmbedArgs a, const uint2* __restrict__ list,
                                                              const int* __restrict__ valid,
                                                              const float* __restrict__ part) {
  __shared__ ulonglong2 sums[8][2][32];
  __shared__ int further[8];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = *valid;
  const int spans = (a.cols + 255) / 256, pieces = (n + kPiece - 1) / kPiece;
  const long long total = (long long)spans * pieces;
  // acc += parts first, first + step, ... <= more of the id that begins in `piece`
  auto add_parts = [&](int piece, int c0, int first, int step, int more, Pairs& acc) {
    for (int k0 = first; k0 <= more; k0 += 4 * step) {
      Pairs p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = min(k0 + step * j, more);
        span_load<VEC>(part + ((size_t)(piece + k) * 2 + (k ? 0 : 1)) * a.cols + c0, a.cols - c0, lane, p[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (k0 + step * j > more) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = f2_add(acc[e], p[j][e]);
      }
    }
  };
  auto put = [&](int piece, int c0, Pairs& acc) {
    float* dst = a.d_table + (size_t)list[piece * (long long)kPiece + kPiece - 1].x * a.cols + c0;
    if (a.accumulate) {
      Pairs old;
      span_load<VEC>(dst, a.cols - c0, lane, old);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = f2_add(acc[e], old[e]);
    }
    span_store<VEC>(dst, a.cols - c0, lane, acc);
  };
  for (long long base = blockIdx.x * 8ll; base < total; base += gridDim.x * 8ll) {
    const long long i = base + warp;
    const int span = (int)(i / pieces), piece = (int)(i - (long long)span * pieces), c0 = span * 256, p0 = piece * kPiece;
    int more = 0;
    if (i < total && p0 + kPiece < n) {
      const uint32_t id = list[p0 + kPiece - 1].x;
      if (list[p0 + kPiece].x == id && !(p0 > 0 && list[p0 - 1].x == id)) {
        // the pieces that begin with this id: they follow one another
        for (int k0 = piece + 1;; k0 += 32) {
          const int k = k0 + lane;
          const int same = __popc(__ballot_sync(0xffffffffu, k < pieces && list[(size_t)min(k, pieces - 1) * kPiece].x == id));
          more += same;
          if (same < 32) break;
        }
      }
    }
    Pairs acc;
    fill(acc, 0.f);
    if (more > 0 && more <= kAlone) {
      add_parts(piece, c0, 0, 1, more, acc);
      put(piece, c0, acc);
    }
    if (lane == 0) further[warp] = more;
    __syncthreads();
    for (int w = 0; w < 8; ++w) {
      if (further[w] <= kAlone) continue;
      const int its_span = (int)((base + w) / pieces), its_piece = (int)(base + w - (long long)its_span * pieces),
                its_c0 = its_span * 256;
      fill(acc, 0.f);
      add_parts(its_piece, its_c0, warp, 8, further[w], acc);
      sums[warp][0][lane] = make_ulonglong2(acc[0], acc[1]);
      sums[warp][1][lane] = make_ulonglong2(acc[2], acc[3]);
      __syncthreads();
      if (warp == 0) {
        fill(acc, 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const ulonglong2 lo = sums[k][0][lane], hi = sums[k][1][lane];
          acc[0] = f2_add(acc[0], lo.x); acc[1] = f2_add(acc[1], lo.y);
          acc[2] = f2_add(acc[2], hi.x); acc[3] = f2_add(acc[3], hi.y);
        }
        put(its_piece, its_c0, acc);
      }
      __syncthreads();
    }
    __syncthreads();
  }
}

template <typename TE, typename TO>
cudaError_t launch_lookup(const EmbedArgs& a, cudaStream_t st) {
  if (rows_on_eights(a.table, a.cols, sizeof(TE)) && rows_on_eights(a.out, a.out_stride, sizeof(TO))) {
    const int per_row = (a.cols + 7) / 8;
    const long long total = (long long)a.tokens * per_row, grid = (total + 255) / 256;
    embed_scaled_kernel<TE, TO><<<(unsigned)grid, 256, 0, st>>>(a, fast_div(per_row), total);
  } else {
    const int spans = (a.cols + 255) / 256;
    const long long total = (long long)a.tokens * spans;
    embed_rows_kernel<TE, TO><<<(unsigned)((total + 7) / 8), 256, 0, st>>>(a, fast_div(spans), total);
  }
  return cudaGetLastError();
}

// Few ids: sums of every id per chunk (16384 x 1280: 64 ids 26.5 us, sorted 31; 65536 tokens 88.7 and 91.5: what the
// chunks leave grows with the ids).
bool by_chunks(int vocab) { return vocab <= kChunkIds; }
// Few tokens: a search through all of them for every id is one launch.  1280 columns, us with ids at random and all
// the same: 33 ids, 173 tokens 2.8 and 8.3, by chunks 5.2 and 5.5; 512 tokens 3.7 and 14.9, by chunks 5.5 and 5.6;
// 300 ids, 512 tokens 4.6 and 15, sorted 15 and 14.  The blocks of ids that are not met cost too: 1000 ids take 10,
// 2000 17, sorted 16.
bool direct(int tokens, int vocab, int cols) {
  return tokens <= (by_chunks(vocab) ? 256 : 512) && (long long)vocab * ((cols + 255) / 256) <= 8192;
}
// Tokens of a chunk: as many as give every SM three blocks, up to 256 (16384 x 1280, 33 ids: 192 tokens 24.8 us, 256
// 26.7; 2000 tokens 9.0 and 13.4).
int chunk_length(int tokens, int cols, int num_sms) {
  const long long blocks = 3ll * num_sms, spans = (cols + 255) / 256;
  const long long even = (tokens * spans + blocks - 1) / blocks;
  return (int)std::min((long long)kChunk, std::max((long long)kShortChunk, (even + 31) / 32 * 32));
}
// Chunks of any batch of up to `tokens`.
long long most_chunks(int tokens, int cols, int num_sms) {
  const long long spans = (cols + 255) / 256, wave = (3ll * num_sms + spans - 1) / spans;
  return std::max((tokens + kChunk - 1ll) / kChunk, std::min((tokens + kShortChunk - 1ll) / kShortChunk, wave));
}

struct GradWorkspace {
  size_t list[2], valid, part, total;
};
GradWorkspace grad_workspace(int tokens, int cols) {
  const size_t T = (size_t)std::max(tokens, 1), pieces = (T + kPiece - 1) / kPiece;
  auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  GradWorkspace w;
  w.list[0] = 0;
  w.list[1] = w.list[0] + up(sizeof(uint2) * T);
  w.valid = w.list[1] + up(sizeof(uint2) * T);
  w.part = w.valid + 256;
  w.total = w.part + up(sizeof(float) * pieces * 2 * cols);
  return w;
}

template <typename TO, bool VEC>
cudaError_t launch_grad(const EmbedArgs& a, void* workspace, int num_sms, cudaStream_t st) {
  const long long spans = (a.cols + 255) / 256;
  if (a.tokens == 0)
    return a.accumulate ? cudaSuccess : cudaMemsetAsync(a.d_table, 0, 4 * (size_t)a.vocab * a.cols, st);
  if (direct(a.tokens, a.vocab, a.cols)) {
    embed_grad_kernel<TO, VEC><<<(unsigned)(spans * a.vocab), 256, 0, st>>>(a, fast_div((uint32_t)spans));
    return cudaGetLastError();
  }
  if (by_chunks(a.vocab)) {
    float* part = static_cast<float*>(workspace);
    const int length = chunk_length(a.tokens, a.cols, num_sms), chunks = (a.tokens + length - 1) / length;
    embed_grad_chunks_kernel<TO, VEC><<<(unsigned)(spans * chunks), kChunk, 0, st>>>(a, part, fast_div((uint32_t)spans),
                                                                                     length);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_after(embed_grad_add_kernel<VEC>, (unsigned)(((size_t)a.vocab * a.cols + 127) / 128), 256, st, a,
                        (const float*)part, chunks);
  }
  const GradWorkspace w = grad_workspace(a.tokens, a.cols);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SortArgs s;
  s.list = reinterpret_cast<uint2*>(ws + w.list[0]);
  s.other = reinterpret_cast<uint2*>(ws + w.list[1]);
  s.valid = reinterpret_cast<int*>(ws + w.valid);
  int bits = 1;
  while (bits < 31 && (1ll << bits) < a.vocab) ++bits;
  s.passes = (bits + kDigitBits - 1) / kDigitBits;
  s.digit_bits = (bits + s.passes - 1) / s.passes;
  float* part = reinterpret_cast<float*>(ws + w.part);
  int clear = 0;  // blocks that clear d_table: one per 128 KB, in clusters of eight, up to two an SM
  if (!a.accumulate) {
    const size_t bytes = 4 * (size_t)a.vocab * a.cols;
    clear = (int)std::min((bytes + (1 << 17) - 1) >> 17, (size_t)num_sms * 2);
    clear = (clear + kSortBlocks - 1) / kSortBlocks * kSortBlocks;
  }
  embed_sort_kernel<<<kSortBlocks + clear, kSortThreads, 0, st>>>(a, s);
  const long long pieces = (a.tokens + kPiece - 1) / kPiece;
  // (each launch may start while the one before it still runs, and waits for it where it needs its results)
  cudaError_t e = launch_after(embed_grad_pieces_kernel<TO, VEC>, (unsigned)(spans * pieces), 32, st, a,
                               (const uint2*)s.list, (const int*)s.valid, part, fast_div((uint32_t)spans), spans * pieces);
  if (e != cudaSuccess) return e;
  const unsigned join = (unsigned)std::min((spans * pieces + 7) / 8, (long long)num_sms * 32);
  return launch_after(embed_grad_join_kernel<VEC>, join, 256, st, a, (const uint2*)s.list, (const int*)s.valid,
                      (const float*)part);
}

}  // namespace

cudaError_t launch_embed_scaled(const EmbedArgs& a, cudaStream_t st) {
  if (a.tokens <= 0) return cudaSuccess;
  using bf16 = __nv_bfloat16;
  if (a.table_bf16) return a.out_bf16 ? launch_lookup<bf16, bf16>(a, st) : launch_lookup<bf16, float>(a, st);
  return a.out_bf16 ? launch_lookup<float, bf16>(a, st) : launch_lookup<float, float>(a, st);
}

size_t embed_grad_workspace_bytes(int tokens, int vocab, int cols, int num_sms) {
  if (tokens == 0 || direct(tokens, vocab, cols)) return 256;
  if (by_chunks(vocab)) return ((size_t)most_chunks(tokens, cols, num_sms) * vocab * cols * 4 + 255) & ~size_t(255);
  return grad_workspace(tokens, cols).total;
}

cudaError_t launch_embed_grad(const EmbedArgs& a, void* workspace, int num_sms, cudaStream_t st) {
  const bool vec =
      a.cols % 8 == 0 && rows_on_eights(a.d_table, a.cols, 4) && rows_on_eights(a.out, a.out_stride, a.out_bf16 ? 2 : 4);
  if (a.out_bf16)
    return vec ? launch_grad<__nv_bfloat16, true>(a, workspace, num_sms, st)
               : launch_grad<__nv_bfloat16, false>(a, workspace, num_sms, st);
  return vec ? launch_grad<float, true>(a, workspace, num_sms, st) : launch_grad<float, false>(a, workspace, num_sms, st);
}

}  // namespace esm
