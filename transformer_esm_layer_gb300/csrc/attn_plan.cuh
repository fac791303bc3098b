// The work list of the windowed attention, straight from cu_seqlens.
#pragma once
#include "common.cuh"
#include "internal.h"

namespace esm {

// it / heads by a multiplication with ceil(2^32 / heads): at most one too large.
struct HeadDiv {
  uint32_t heads, magic;
  __device__ __forceinline__ void split(uint32_t it, uint32_t& entry, uint32_t& h) const {
    entry = heads == 1 ? it : __umulhi(it, magic);
    if (entry * heads > it) --entry;
    h = it - entry * heads;
  }
};

// A work item of the forward: its list entry (first query row, query rows, first key row, visible
// keys) and head.
struct RawItem {
  int4 w;
  int h;
};
// Item `it` from the offsets themselves, by a whole warp, for batches of at most 32 sequences whose
// items one grid takes in one round; reports malformed offsets like the kernel that writes the
// list, and counts the items.
template <int QT>
__device__ __forceinline__ RawItem find_item(const PackedBatch& b, int it, const HeadDiv& hd, int& n_items, unsigned* err) {
  const int lane = threadIdx.x & 31;
  int c0 = 0, L = 0;
  if (lane < b.B) {
    c0 = __ldg(b.cu + lane);
    int c1 = __ldg(b.cu + lane + 1);
    if ((lane == 0 && c0 != 0) || (lane == b.B - 1 && c1 != b.T) || c1 < c0 || c1 - c0 > b.max_seqlen ||
        c1 - c0 > b.max_positions || c0 < 0 || c1 > b.T) {
      if (threadIdx.x < 32) latch_error(err, ERRBIT_CU_SEQLENS);
      c0 = min(max(c0, 0), b.T);
      c1 = min(min(max(c1, c0), b.T), c0 + b.max_positions);
    }
    L = c1 - c0;
  }
  const int tiles = (L + QT - 1) / QT;
  int v = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  // Malformed offsets (segments that overlap) can hold more items than the grid was made for: a second
  // round would read a list that was never written.
  n_items = min(__shfl_sync(0xffffffffu, v, 31) * (int)hd.heads, (int)gridDim.x);
  uint32_t entry, h;
  hd.split((uint32_t)it, entry, h);
  const unsigned mine = __ballot_sync(0xffffffffu, (int)entry >= v - tiles && (int)entry < v);
  const int src = mine ? __ffs(mine) - 1 : 0;
  const int start = __shfl_sync(0xffffffffu, c0, src), len = __shfl_sync(0xffffffffu, L, src);
  const int off = ((int)entry - __shfl_sync(0xffffffffu, v - tiles, src)) * QT;
  return RawItem{make_int4(start + off, min(QT, len - off), start, len), (int)h};
}

// Sort key of a windowed item, longest first: its key tiles (forward) or query tiles (backward),
// exact up to 64 and in steps of 8 above.
constexpr int PLAN_CLASSES = 128;
__device__ __forceinline__ int plan_class(int pos, int rows, int len, const AttnWindow& win, bool backward) {
  const int before = backward ? win.right : win.left, after = backward ? win.left : win.right;
  const int lo = before < 0 ? 0 : max(0, pos - before), hi = after < 0 ? len : min(len, pos + rows + after);
  const int tiles = (max(0, hi - lo) + (!backward && lo > 0 ? (win.sinks + 15) / 16 * 16 : 0) + 127) / 128;
  return PLAN_CLASSES - 1 - min(PLAN_CLASSES - 1, tiles <= 64 ? tiles : 64 + (tiles - 64) / 8);
}

// One block of NT threads: the validated segment table of a packed batch and the windowed attention's
// items, for callers that need no positions.  A chunk of NT sequences at a time: their tiles are
// scanned, then all threads take the chunk's items, each found by bisection.  With more than
// sort_above items they are ordered longest first (a counting sort: one pass counts, one
// writes), so that the CTAs' static shares come out even: 47 packed sequences under a window of
// 128 + 128 hold items of one to four tiles, and in sequence order the busiest CTA had 1.17
// times the mean's work, sorted 1.07; with a causal window 1.29 and 1.02.  Items of one length
// stand in any order.  Malformed offsets can hold more items than the list has room for: the items
// past max_items are left out, of the count and of both passes alike.
template <int NT>
__device__ __forceinline__ void attn_plan(const AttnPlan& pl, const PackBuffers& pb, unsigned* err) {
  __shared__ int s_first[NT + 1];  // items before the chunk's sequence i, within the chunk
  __shared__ int s_start[NT], s_len[NT];
  __shared__ int s_warp[NT / 32];
  __shared__ int s_class[PLAN_CLASSES];    // items of a class, then the next place of one
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  // the chunk at b0: segments (written once) and s_first; returns its items
  auto scan_chunk = [&](int b0, bool write) -> int {
    const int i = b0 + tid;
    int tiles = 0;
    if (i < pl.B) {
      int c0 = pl.cu[i], c1 = pl.cu[i + 1];
      const bool bad = (i == 0 && c0 != 0) || (i == pl.B - 1 && c1 != pl.T) || c1 < c0 || c1 - c0 > pl.max_seqlen ||
                       c1 - c0 > pl.max_positions || c0 < 0 || c1 > pl.T;
      if (bad) {
        latch_error(err, ERRBIT_CU_SEQLENS);
        c0 = min(max(c0, 0), pl.T);
        c1 = min(min(max(c1, c0), pl.T), c0 + pl.max_positions);
      }
      const int L = c1 - c0;
      s_start[tid] = c0;
      s_len[tid] = L;
      if (write) {
        pb.seg_start[i] = c0;
        pb.seg_qlen[i] = pb.seg_klen[i] = L;
      }
      tiles = (L + pl.q_tile - 1) / pl.q_tile;
    }
    int v = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += n;
    }
    if (lane == 31) s_warp[wid] = v;
    __syncthreads();
    if (wid == 0) {
      int w = lane < NT / 32 ? s_warp[lane] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += n;
      }
      if (lane < NT / 32) s_warp[lane] = w;
    }
    __syncthreads();
    v += wid > 0 ? s_warp[wid - 1] : 0;
    s_first[tid] = v - tiles;
    if (tid == NT - 1) s_first[NT] = v;
    __syncthreads();
    return s_first[NT];
  };
  // item k of the chunk: its sequence's slot, and its first row there
  auto item = [&](int k, int& off) -> int {
    int lo = 0, hi = NT;  // the last sequence with s_first <= k (it has tiles)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_first[mid] <= k) lo = mid;
      else hi = mid;
    }
    off = (k - s_first[lo]) * pl.q_tile;
    return lo;
  };
  if (tid < PLAN_CLASSES) s_class[tid] = 0;
  __syncthreads();
  int total = 0;
  for (int b0 = 0; b0 < pl.B; b0 += NT) {
    const int n = min(scan_chunk(b0, true), pl.max_items - total);
    total += n;
    if (pl.max_items > pl.sort_above)
      for (int k = tid; k < n; k += NT) {
        int off;
        const int q = item(k, off);
        atomicAdd(&s_class[plan_class(off, min(pl.q_tile, s_len[q] - off), s_len[q], pl.win, pl.backward)], 1);
      }
    __syncthreads();
  }
  const bool sorted = total > pl.sort_above;
  if (sorted && wid == 0) {  // first place of every class
    int before = 0;
    for (int c = lane; c < PLAN_CLASSES; c += 32) {
      const int n = s_class[c];
      int v = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      s_class[c] = before + v - n;
      before += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  int base = 0;
  for (int b0 = 0; b0 < pl.B; b0 += NT) {
    // (a single chunk is still there)
    const int n = pl.B > NT ? min(scan_chunk(b0, false), pl.max_items - base) : total;
    for (int k = tid; k < n; k += NT) {
      int off;
      const int q = item(k, off), rows = min(pl.q_tile, s_len[q] - off);
      const int at = sorted ? atomicAdd(&s_class[plan_class(off, rows, s_len[q], pl.win, pl.backward)], 1) : base + k;
      reinterpret_cast<int4*>(pb.work)[at] = make_int4(s_start[q] + off, rows, s_start[q], s_len[q]);
    }
    base += n;
    __syncthreads();
  }
  if (tid == 0) pb.work_count[0] = total;
}

}  // namespace esm
