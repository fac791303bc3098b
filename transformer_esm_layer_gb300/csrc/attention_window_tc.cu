// Windowed variable-length attention on the tcgen05 tensor cores (head_dim 64, bf16 in, fp32
// softmax and accumulation), with the first tokens of a sequence (sinks) kept visible.
//
// Query i of a sequence sees key j of the same sequence if j <= i + right and (j >= i - left or
// j < sinks), a side below zero being unlimited:
//   o_i = sum_j p_ij v_j,  p_ij = exp(s_ij - lse_i),  s_ij = q_i . k_j / 8,
//   lse_i = log sum_j exp(s_ij) over the keys that i sees; a row that sees none is zero, one whose
//   visible scores are all -inf is NaN.
//
// A query tile's keys are the list [sinks | lo .. hi), with lo .. hi the band that any of its 128
// rows sees: first the sink rows, padded to a multiple of 16, then the band.  The key tiles are
// 128 consecutive entries of that list, so a few sinks cost their 16-row groups and not a tile
// of their own; the one tile that holds both is fetched as eight 16-row boxes.  Each row's
// visible columns of a tile are two runs, [0, cs) and [cl, ch), applied as bits; a tile that
// every row of a warp sees whole takes no mask.
//
// Persistent: two CTAs per SM walk the (sequence, 128-query tile, head) items of the work list in
// rounds of one item per CTA, in snake order; barrier phases run on across items.
//   warp 0       TMA: each item's Q tile (two buffers) and its K tiles into a 2-stage ring;
//   warp 2       TMA: the V tiles into their own 2-stage ring;
//   warp 1       one thread issues S = Q K^T (M = N = 128, K = 64) of every tile;
//   warp 3       one thread issues O += P V (N = 64; P read from tensor memory) of every tile, as
//                many 16-key steps as the list fills;
//   warps 4..7   softmax: thread r owns query row r, its 128 scores in registers.
// The reference maximum of a row moves only when a tile exceeds it by more than 8 (log2 units), so
// O is rescaled rarely and P <= 2^8; P = 2^(s log2(e) / 8 - m) is rounded to bf16 for the P V
// product, its sum is taken before the rounding in fp32.
// Tensor memory: S 128 columns, P 64 (bf16 pairs), O 64 -> 256 columns per CTA.  Every wait is
// bounded.
//
// What bounds it: latency, and the integer pipe in tiles that are seen in part.  A tile is a chain
// (scores from tensor memory, maximum, exponentials, P back, P V), on GB300 about 2800 cycles of
// which the arithmetic is half, and two CTAs per SM interleave two of them; no pipe is above half
// of its rate.  An item's O is brought out after the next item's first P has been handed over, from
// registers in 32-byte pieces, which hides the last P V and leaves Q's buffers to the loads.  Whole
// calls on 16384 packed tokens, 20 heads, window 128 + 128, one sink: 66 us (floor: 25 us of memory
// traffic); with O brought out at the item's end, 69 us; without masks a fifth less.  Measured and
// slower, on the same call: two threads per row (87 us, twice the waits), 64-key tiles with three
// CTAs per SM (77 us, the tensor pipe takes as long for 64 columns as for 128), skipping or not
// masking 32-column chunks by branches (69 to 79 us: the compiler then schedules each chunk by
// itself), and what a row sees kept for the epilogue through the tile loop (68 us).
#include "attn_plan.cuh"
#include "common.cuh"
#include "internal.h"

namespace esm {
namespace {

constexpr int DH = 64;
constexpr int QT = 128;
constexpr int KT = 128;
constexpr int STG = 2;
constexpr int TILE_BYTES = 128 * 128;  // 128 rows x 128 bytes
constexpr int THREADS = 256;
constexpr int CTAS_PER_SM = 2;
// Register budget per thread at launch and after the warpgroup-wide setmaxnreg: warpgroup 0 (TMA,
// MMA) gives up registers to the softmax warpgroup, whose threads hold a row of 128 scores.
constexpr int kRegsLaunch = 128, kRegsWg0 = 56, kRegsSoftmax = 200;
static_assert(128 * kRegsWg0 + 128 * kRegsSoftmax <= THREADS * kRegsLaunch, "register split");
constexpr uint32_t TMEM_COLS = 256;
constexpr uint32_t COL_S = 0, COL_P = 128, COL_O = 192;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr int NC = KT / 32;                // 32-column chunks of a score row

struct WinSmem {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[STG], k_empty[STG];  // K tile landed / read by its S = Q K^T
  uint64_t v_full[STG], v_empty[STG];  // V tile landed / read by its O += P V
  uint64_t s_full, s_free, p_full, pv_done, mma_done, pv_fin;
  uint32_t tmem_base;
  volatile int abort;
  int first[5];                        // the first item's list entry and head
};
// [Q0][Q1][K0][V0][K1][V1] then WinSmem
constexpr int SMEM_BYTES = TILE_BYTES * (2 + 2 * STG) + 1024 + (int)sizeof(WinSmem);

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// max of three (one instruction)
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 32 bytes to global memory: one store if the address allows it.
__device__ __forceinline__ void store32(uint8_t* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// The low n bits set (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

struct Item {
  int qrow0, qrows, krow0, klen, h;
  int qpos0;      // position of the first query in its sequence
  int nsink, s16; // sink rows and their padded count at the front of the key list
  int lo;         // first band key (position in the sequence)
  int n_keys;     // entries of the key list: s16 and the band's
  int nkb;        // key tiles
};

// Work item `it` = (work-list entry it / heads, head it % heads), in one 16-byte load.
__device__ __forceinline__ RawItem load_item(const PackBuffers& pb, int it, const HeadDiv& hd) {
  uint32_t entry, h;
  hd.split((uint32_t)it, entry, h);
  return RawItem{__ldg(reinterpret_cast<const int4*>(pb.work) + entry), (int)h};
}
__device__ __forceinline__ Item make_item(const RawItem& raw, const AttnWindow& win) {
  Item x;
  x.h = raw.h;
  x.qrow0 = raw.w.x;
  x.qrows = raw.w.y;
  x.krow0 = raw.w.z;
  x.klen = raw.w.w;
  x.qpos0 = x.qrow0 - x.krow0;
  x.lo = win.left < 0 ? 0 : max(0, x.qpos0 - win.left);
  if (win.sinks >= x.lo) x.lo = 0;  // sinks that reach the band make one run with it
  x.nsink = x.lo > 0 ? min(win.sinks, x.klen) : 0;
  x.s16 = (x.nsink + 15) & ~15;
  const int hi = win.right < 0 ? x.klen : min(x.klen, x.qpos0 + x.qrows + win.right);
  x.n_keys = x.s16 + max(0, hi - x.lo);
  // at least one tile, so that rows that see nothing (padding queries far past the last key) pass
  // through the same pipeline
  x.nkb = max(1, (x.n_keys + KT - 1) / KT);
  return x;
}

// 16-key steps of key tile j that hold any entry of the list (1 to 8).
__device__ __forceinline__ int key_steps(const Item& x, int j) {
  return max(1, min(KT / 16, (x.n_keys - j * KT + 15) >> 4));
}

// Key tile j of an item: entries 128 j .. of [sinks (s16 rows) | band from lo].
__device__ __forceinline__ void load_key_tile(uint8_t* dst, const CUtensorMap* tm, const CUtensorMap* tm16, int xcol,
                                              const Item& x, int j, uint64_t* bar) {
  const int c0 = j * KT;
  if (c0 >= x.s16) {
    tma_load_2d(dst, tm, xcol, x.krow0 + x.lo + c0 - x.s16, bar);
  } else if (c0 + KT <= x.s16) {
    tma_load_2d(dst, tm, xcol, x.krow0 + c0, bar);
  } else {  // c0 == 0 (at most 128 sinks): s16 sink rows, then the band's first rows
#pragma unroll 1
    for (int r = 0; r < KT; r += 16)
      tma_load_2d(dst + r * 128, tm16, xcol, x.krow0 + (r < x.s16 ? r : x.lo + r - x.s16), bar);
  }
}

// AMAX: a bf16 output also records its max |value| into amax_out (compiled only into the
// instantiation that needs it).
template <Act OUT, bool AMAX = false>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM)
    attention_window_tc_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tm16,
                               AttnWindow win, const __nv_bfloat16* __restrict__ qkv, void* __restrict__ o, int d,
                               HeadDiv hd, PackBuffers pb, PackedBatch batch, const float* q_scale, float* amax_out,
                               float* __restrict__ lse, int lse_stride, unsigned* err) {
  // the CTA's first item: from the work list, or (then its only one) from the offsets
  int n_items;
  RawItem first;
  if (batch.cu != nullptr) {
    first = find_item<QT>(batch, blockIdx.x, hd, n_items, err);
  } else {
    n_items = *pb.work_count * (int)hd.heads;
    if ((int)blockIdx.x < n_items) first = load_item(pb, blockIdx.x, hd);
  }
  if ((int)blockIdx.x >= n_items) return;  // whole CTA, before any barrier or TMEM use

  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;                       // buffer b: sQ + b * TILE_BYTES
  uint8_t* sK = base + 2 * TILE_BYTES;      // stage s: sK + 2 * s * TILE_BYTES
  uint8_t* sV = base + 3 * TILE_BYTES;      // stage s: sV + 2 * s * TILE_BYTES
  WinSmem* sm = reinterpret_cast<WinSmem*>(base + TILE_BYTES * (2 + 2 * STG));

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Items in rounds of gridDim.x, snake order: even rounds give CTA c item c of the round,
  // odd rounds item gridDim.x - 1 - c.
  auto item_at = [&](int rnd) -> int {
    return rnd * (int)gridDim.x + ((rnd & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
  };
  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm->q_full[b], 1);
      mbar_init(&sm->q_empty[b], 1);
    }
    for (int s = 0; s < STG; ++s) {
      mbar_init(&sm->k_full[s], 1);
      mbar_init(&sm->k_empty[s], 1);
      mbar_init(&sm->v_full[s], 1);
      mbar_init(&sm->v_empty[s], 1);
    }
    mbar_init(&sm->s_full, 1);
    mbar_init(&sm->s_free, 4);
    mbar_init(&sm->p_full, 4);
    mbar_init(&sm->pv_done, 1);
    mbar_init(&sm->mma_done, 1);
    mbar_init(&sm->pv_fin, 1);
    sm->abort = 0;
    sm->first[0] = first.w.x;
    sm->first[1] = first.w.y;
    sm->first[2] = first.w.z;
    sm->first[3] = first.w.w;
    sm->first[4] = first.h;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) tma_prefetch_desc(&tm);
  if (warp == 1) tmem_alloc(&sm->tmem_base, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  auto first_item = [&]() { return RawItem{make_int4(sm->first[0], sm->first[1], sm->first[2], sm->first[3]), sm->first[4]}; };
  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsWg0));

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ TMA producers
    // A K stage is free as soon as its S is done, a V stage only after its P V, so K never waits
    // behind V.
    if (lane == 0) {
      const bool kq = warp == 0;
      int g = 0, n_q = 0;  // key tiles and Q tiles asked for
      RawItem nxt = first_item();
      for (int rnd = 0, it = item_at(0); it < n_items && !sm->abort; it = item_at(++rnd)) {
        const Item x = make_item(nxt, win);
        if (item_at(rnd + 1) < n_items) nxt = load_item(pb, item_at(rnd + 1), hd);  // prefetch
        if (kq) {
          const int qb = n_q & 1;
          if (!mbar_wait(&sm->q_empty[qb], ((uint32_t)(n_q >> 1) & 1u) ^ 1u)) {
            latch_error(err, ERRBIT_TIMEOUT);
            sm->abort = 1;
            break;
          }
          mbar_arrive_expect_tx(&sm->q_full[qb], TILE_BYTES);
          tma_load_2d(sQ + qb * TILE_BYTES, &tm, x.h * DH, x.qrow0, &sm->q_full[qb]);
          ++n_q;
        }
        uint64_t* empty = kq ? sm->k_empty : sm->v_empty;
        uint64_t* full = kq ? sm->k_full : sm->v_full;
        uint8_t* dst0 = kq ? sK : sV;
        const int xcol = (kq ? d : 2 * d) + x.h * DH;
        for (int j = 0; j < x.nkb; ++j, ++g) {
          const int st = g % STG;
          if (!mbar_wait(&empty[st], ((uint32_t)(g / STG) & 1u) ^ 1u)) {
            latch_error(err, ERRBIT_TIMEOUT);
            sm->abort = 1;
            break;
          }
          mbar_arrive_expect_tx(&full[st], TILE_BYTES);
          load_key_tile(dst0 + 2 * st * TILE_BYTES, &tm, &tm16, xcol, x, j, &full[st]);
        }
      }
      // Copies still in flight can only exist if a consumer gave up early: then the last
      // STG stages (and Q tiles) are waited for (bounded) before the CTA exits.
      if (sm->abort) {
        uint64_t* full = kq ? sm->k_full : sm->v_full;
        for (int k = g - 1; k >= 0 && k >= g - STG; --k)
          if (!mbar_wait(&full[k % STG], (uint32_t)(k / STG) & 1u)) break;
        for (int k = n_q - 1; k >= 0 && k >= n_q - 2; --k)
          if (!mbar_wait(&sm->q_full[k & 1], (uint32_t)(k >> 1) & 1u)) break;
      }
    }
    __syncwarp();
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------ MMA issuers
    // Two threads issue to the one tensor pipe, each in tile order and each blocking only on its
    // own operands: a ready S never waits behind the P V MMAs the pipe is still accepting.
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16(QT, KT);
      constexpr uint32_t idesc_pv = idesc_bf16(QT, DH) | (1u << 16);  // B (= V) MN-major
      const bool is_s = warp == 1;
      const uint64_t qdesc0 = make_sw128_desc(smem_u32(sQ));  // buffer b: + b * (TILE_BYTES >> 4)
      const uint64_t kdesc0 = make_sw128_desc(smem_u32(sK));  // stage s: + 2 s (TILE_BYTES >> 4)
      const uint64_t vdesc0 = make_sw128_desc(smem_u32(sV));
      bool ok = true;
      int g = 0, qi = 0;
      RawItem nxt = first_item();
      for (int rnd = 0, it = item_at(0); it < n_items && ok && !sm->abort; it = item_at(++rnd), ++qi) {
        const Item x = make_item(nxt, win);
        if (item_at(rnd + 1) < n_items) nxt = load_item(pb, item_at(rnd + 1), hd);  // prefetch
        const int qb = qi & 1;
        for (int j = 0; j < x.nkb; ++j, ++g) {
          const int st = g % STG;
          if (is_s) {
            // the K tile has landed, the previous S has been read, the item's Q has landed
            if (!mbar_wait(&sm->k_full[st], (uint32_t)(g / STG) & 1u) ||
                (g > 0 && !mbar_wait(&sm->s_free, (uint32_t)(g - 1) & 1u)) ||
                (j == 0 && !mbar_wait(&sm->q_full[qb], (uint32_t)(qi >> 1) & 1u))) {
              ok = false;
              break;
            }
            tc_fence_after();
            // descriptor arithmetic on the low word (the start-address field cannot carry)
            const uint32_t alo = (uint32_t)qdesc0 + (uint32_t)((qb * TILE_BYTES) >> 4);
            const uint32_t blo = (uint32_t)kdesc0 + (uint32_t)((2 * st * TILE_BYTES) >> 4);
#pragma unroll
            for (int k = 0; k < DH / 16; ++k)  // 16 dims = 32 bytes of each 128-byte row
              mma_bf16_ss(tmem + COL_S, (qdesc0 & 0xFFFFFFFF00000000ull) | (uint64_t)(alo + 2u * (uint32_t)k),
                          (kdesc0 & 0xFFFFFFFF00000000ull) | (uint64_t)(blo + 2u * (uint32_t)k), idesc_s,
                          k > 0 ? 1u : 0u);
            mma_commit(&sm->s_full);
            mma_commit(&sm->k_empty[st]);
            if (j == x.nkb - 1) mma_commit(&sm->q_empty[qb]);
          } else {
            // P of this tile is in tensor memory and its V tile has landed
            if (!mbar_wait(&sm->p_full, (uint32_t)g & 1u) || !mbar_wait(&sm->v_full[st], (uint32_t)(g / STG) & 1u)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t vlo = (uint32_t)vdesc0 + (uint32_t)((2 * st * TILE_BYTES) >> 4);
            const int steps = key_steps(x, j);
#pragma unroll
            for (int k = 0; k < KT / 16; ++k) {  // 16 keys = 16 rows of V = 2048 bytes
              if (k >= steps) break;
              mma_bf16_ts(tmem + COL_O, tmem + COL_P + 8 * k,
                          (vdesc0 & 0xFFFFFFFF00000000ull) | (uint64_t)(vlo + 128u * (uint32_t)k), idesc_pv,
                          (j > 0 || k > 0) ? 1u : 0u);
            }
            mma_commit(&sm->pv_done);
            mma_commit(&sm->v_empty[st]);
          }
        }
      }
      if (!ok) {
        latch_error(err, ERRBIT_TIMEOUT);
        sm->abort = 1;
      }
      // every MMA of this thread has completed before tensor memory may be released
      uint64_t* fin = is_s ? &sm->mma_done : &sm->pv_fin;
      mma_commit(fin);
      mbar_wait(fin, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int wq = warp & 3;                                // TMEM lane quarter
    const int r = wq * 32 + lane;                           // query row of this thread
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t col_s = tmem + lane_off + COL_S, col_p = tmem + lane_off + COL_P, col_o = tmem + lane_off + COL_O;
    const float c = 1.4426950408889634f / 8.f;  // 1/sqrt(64), log2 units
    const float qs = (OUT == Act::E4M3) ? __ldg(q_scale) : 1.f;
    const bool wide = (reinterpret_cast<uintptr_t>(o) & 31) == 0;
    float amax = 0.f;
    bool ok = true;
    int g = 0;
    // The item whose P V may still run: its O goes to memory once the next item's first P has been
    // handed over, so that neither waits for the other.
    struct {
      Item x;
      // of this thread's row; inv = 0 where it sees no key (a padding query), inf where its scores are
      // all -inf (0 inf = NaN), NaN where one is NaN or +inf
      float m, inv;
      bool pending;
    } last;
    last.pending = false;
    auto load_o = [&](uint32_t (&u)[2][32]) {
      tmem_ld32_nowait(col_o, u[0]);
      tmem_ld32_nowait(col_o + 32, u[1]);
      tmem_ld_wait_regs(u[0]);
      tmem_ld_wait_regs(u[1]);
    };
    // the rows of O / l to global memory, 32 bytes at a time
    auto store_o = [&](uint32_t (&u)[2][32]) {
      const bool live = r < last.x.qrows;
      constexpr size_t kElem = (OUT == Act::BF16) ? 2 : 1;
      uint8_t* dst = static_cast<uint8_t*>(o) + ((size_t)(last.x.qrow0 + r) * d + (size_t)last.x.h * DH) * kElem;
      // A row that sees no key is zero.  A zero weight times an infinite or NaN value is NaN, so
      // values that a row does not see could reach it through the tile's product: a row whose sums
      // are not finite, but for its own scores, is set aside and summed over its visible keys alone below.
      uint64_t probe[4] = {0, 0, 0, 0};
      const uint64_t zero2 = f2_pack(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < DH; i += 2)
        probe[i >> 1 & 3] = f2_fma(f2_pack(__uint_as_float(u[i >> 5][i & 31]), __uint_as_float(u[i >> 5][i + 1 & 31])),
                                   zero2, probe[i >> 1 & 3]);
      float p0, p1;
      f2_unpack(f2_add(f2_add(probe[0], probe[1]), f2_add(probe[2], probe[3])), p0, p1);
      const bool odd = p0 + p1 != 0.f;
      const bool redo = odd && fabsf(last.inv) > 0.f && live;  // (false for NaN)
      if (odd || last.inv == 0.f) {
#pragma unroll
        for (int i = 0; i < DH; ++i) u[i >> 5][i & 31] = 0u;
      }
      const uint64_t inv2 = f2_pack(last.inv, last.inv);
      if constexpr (OUT == Act::BF16) {
#pragma unroll
        for (int i = 0; i < DH; i += 16) {
          uint32_t w[8];
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            float a0, a1;
            const uint32_t* v = &u[i >> 5][(i & 31) + k];
            f2_unpack(f2_mul(f2_pack(__uint_as_float(v[0]), __uint_as_float(v[1])), inv2), a0, a1);
            if (AMAX && live) amax = fmax3(amax, fabsf(a0), fabsf(a1));
            w[k >> 1] = pack_bf16x2(a0, a1);
          }
          if (live && !redo) store32(dst + 2 * i, w, wide);
        }
      } else {
#pragma unroll
        for (int i = 0; i < DH; i += 32) {
          uint32_t w[8];
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            float a0, a1, a2, a3;
            const uint32_t* v = &u[i >> 5][k];
            f2_unpack(f2_mul(f2_pack(__uint_as_float(v[0]), __uint_as_float(v[1])), inv2), a0, a1);
            f2_unpack(f2_mul(f2_pack(__uint_as_float(v[2]), __uint_as_float(v[3])), inv2), a2, a3);
            if (live) amax = fmax3(amax, fmaxf(fabsf(a0), fabsf(a1)), fmaxf(fabsf(a2), fabsf(a3)));
            __nv_fp8x4_e4m3 qv(make_float4(a0 * qs, a1 * qs, a2 * qs, a3 * qs));
            w[k >> 2] = *reinterpret_cast<uint32_t*>(&qv);
          }
          if (live && !redo) store32(dst + i, w, wide);
        }
      }
      // (rare) the whole warp per set-aside row: lane c computes head columns 2c and 2c + 1
      for (unsigned todo = __ballot_sync(0xffffffffu, redo); todo != 0u; todo &= todo - 1) {
        const int src = __ffs(todo) - 1, row = wq * 32 + src, qp = last.x.qpos0 + row;
        const float m = __shfl_sync(0xffffffffu, last.m, src), scale = __shfl_sync(0xffffffffu, last.inv, src);
        const int e = win.right < 0 ? last.x.klen : min(last.x.klen, qp + win.right + 1);
        const int lo = win.left < 0 ? 0 : max(0, qp - win.left), ns = min(win.sinks, min(lo, e));
        const __nv_bfloat16* seq = qkv + (size_t)last.x.krow0 * 3 * d + last.x.h * DH + 2 * lane;
        const float2 qv = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(seq + (size_t)qp * 3 * d));
        float2 acc = make_float2(0.f, 0.f);
        for (int j = 0; j < ns + max(0, e - lo); ++j) {
          const __nv_bfloat16* kr = seq + (size_t)(j < ns ? j : lo + j - ns) * 3 * d + d;
          const float2 kv = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(kr));
          const float2 vv = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(kr + d));
          float s = fmaf(qv.x, kv.x, qv.y * kv.y);
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
          const float p = ex2_approx(fmaf(s, c, -m));
          acc.x = fmaf(p, vv.x, acc.x);
          acc.y = fmaf(p, vv.y, acc.y);
        }
        acc.x *= scale;
        acc.y *= scale;
        if constexpr (OUT == Act::E4M3 || AMAX) amax = fmax3(amax, fabsf(acc.x), fabsf(acc.y));
        const size_t at = (size_t)(last.x.qrow0 + row) * d + (size_t)last.x.h * DH + 2 * lane;
        if constexpr (OUT == Act::BF16) {
          *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(o) + at) = pack_bf16x2(acc.x, acc.y);
        } else {
          __nv_fp8x2_e4m3 q8(make_float2(acc.x * qs, acc.y * qs));
          *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(o) + at) = *reinterpret_cast<uint16_t*>(&q8);
        }
      }
    };
    RawItem nxt = first_item();
    for (int rnd = 0, it = item_at(0); it < n_items && ok; it = item_at(++rnd)) {
      const Item x = make_item(nxt, win);
      if (item_at(rnd + 1) < n_items) nxt = load_item(pb, item_at(rnd + 1), hd);  // prefetch
      // visible columns of the key list: [0, cs0) (sinks) and [cl0, ch0) (band)
      const int q = x.qpos0 + r;
      const int end = win.right < 0 ? x.klen : min(x.klen, q + win.right + 1);
      const int shift = x.s16 - x.lo;  // column of key position 0
      const int cl0 = (win.left < 0 ? 0 : max(x.lo, q - win.left)) + shift, ch0 = end + shift;
      const int cs0 = x.lo > 0 ? x.nsink : min(win.sinks, end);
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < x.nkb; ++j, ++g) {
        const int cl = cl0 - j * KT, ch = ch0 - j * KT, cs = cs0 - j * KT;
        const bool whole = __all_sync(0xffffffffu, cl <= 0 && ch >= KT);
        if (!mbar_wait_warp(&sm->s_full, (uint32_t)g & 1u)) { ok = false; break; }
        tc_fence_after();
        // the row's scores into registers; S is then free for the next tile's Q K^T
        // (su[w] holds 32 scores, then their P as bf16 pairs in its first 16)
        uint32_t su[NC][32];
#pragma unroll
        for (int w = 0; w < NC; ++w) tmem_ld32_nowait(col_s + 32 * w, su[w]);
#pragma unroll
        for (int w = 0; w < NC; ++w) tmem_ld_wait_regs(su[w]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->s_free);
        if (!whole) {
#pragma unroll
          for (int w = 0; w < NC; ++w) {
            const uint32_t vis = low_bits(cs - 32 * w) | (low_bits(ch - 32 * w) & ~low_bits(cl - 32 * w));
#pragma unroll
            for (int i = 0; i < 32; ++i) su[w][i] = (vis >> i & 1u) ? su[w][i] : 0xff800000u;  // -inf
          }
        }
        auto sv = [&](int i) { return __uint_as_float(su[i >> 5][i & 31]); };
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < KT; i += 8) {
          mx[0] = fmax3(mx[0], sv(i), sv(i + 1));
          mx[1] = fmax3(mx[1], sv(i + 2), sv(i + 3));
          mx[2] = fmax3(mx[2], sv(i + 4), sv(i + 5));
          mx[3] = fmax3(mx[3], sv(i + 6), sv(i + 7));
        }
        const float mt = c * fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
        const bool need = mt > m_ref + kRescaleThreshold;
        const float m_new = need ? mt : m_ref;
        const float f = need ? ex2_approx(m_ref - m_new) : 1.f;  // 0 on the first tile
        l *= f;
        m_ref = m_new;
        // P = 2^(s*c - m) as bf16 pairs, computed while the previous P V may still be reading the P
        // columns (scale-subtract and row sums two scores per f32x2 instruction); a row that has
        // seen no key yet has m = -inf: 2^(-inf - 0) = 0 for all its keys
        const float nm = m_ref == -INFINITY ? 0.f : -m_ref;
        const uint64_t c2 = f2_pack(c, c), nm2 = f2_pack(nm, nm);
        uint64_t ls2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int w = 0; w < NC; ++w) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float p0, p1;
            f2_unpack(f2_fma(f2_pack(sv(32 * w + 2 * i), sv(32 * w + 2 * i + 1)), c2, nm2), p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            ls2[i & 1] = f2_add(ls2[i & 1], f2_pack(p0, p1));
            su[w][i] = pack_bf16x2(p0, p1);
          }
        }
        {
          float a0, a1, b0, b1;
          f2_unpack(ls2[0], a0, a1);
          f2_unpack(ls2[1], b0, b1);
          l += (a0 + a1) + (b0 + b1);
        }
        // P (and, within an item, O) may be rewritten once the previous P V is done
        if (g > 0) {
          if (!mbar_wait_warp(&sm->pv_done, (uint32_t)(g - 1) & 1u)) { ok = false; break; }
          tc_fence_after();
        } else {
          __syncwarp();  // (the wait brings the lanes together for the stores below)
        }
        auto hand_over = [&]() {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm->p_full);
        };
        if (j == 0 && last.pending) {  // O still holds the previous item's
          uint32_t u[2][32];
          load_o(u);
#pragma unroll
          for (int w = 0; w < NC; ++w) tmem_st16(col_p + 16 * w, su[w]);
          hand_over();
          store_o(u);
          continue;
        }
#pragma unroll
        for (int w = 0; w < NC; ++w) tmem_st16(col_p + 16 * w, su[w]);
        if (j > 0 && __any_sync(0xffffffffu, need)) {  // warp-collective TMEM round trip of O
#pragma unroll
          for (int ch2 = 0; ch2 < DH / 16; ++ch2) {
            float v[16];
            tmem_ld16(col_o + 16 * ch2, v);
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[i] * f);
            tmem_st16(col_o + 16 * ch2, w);
          }
        }
        hand_over();
      }
      if (!ok) break;
      // ---- the item's row statistics
      last.x = x;
      last.m = m_ref;
      last.inv = l == 0.f && q >= x.klen ? 0.f : 1.f / l;  // (a query before klen sees itself)
      last.pending = true;
      // the natural-log softmax normaliser, ln 2 (m + log2 l) in the base-2 units used above
      if (lse != nullptr && r < x.qrows)
        lse[(size_t)x.h * lse_stride + x.qrow0 + r] = 0.6931471805599453f * (m_ref + __log2f(l));
    }
    if (ok && last.pending) {
      ok = mbar_wait_warp(&sm->pv_done, (uint32_t)(g - 1) & 1u);
      if (ok) {
        tc_fence_after();
        uint32_t u[2][32];
        load_o(u);
        tc_fence_before();
        store_o(u);
      }
    }
    if (!ok) {
      latch_error(err, ERRBIT_TIMEOUT);
      sm->abort = 1;
    }
    if constexpr (OUT == Act::E4M3 || AMAX) {
      // a bf16 output's amax is that of the rounded values: rounding is monotone, so round the max
      if constexpr (OUT == Act::BF16) amax = __bfloat162float(__float2bfloat16_rn(amax));
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
      if (lane == 0) atomic_max_nonneg(amax_out, amax);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Persistent grid: at most CTAS_PER_SM CTAs per SM; CTAs past the (device-side) item count exit.
unsigned window_grid(long long items) {
  static int num_sms = 0;
  if (num_sms == 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || num_sms <= 0)
      num_sms = 148;
  }
  const long long cap = (long long)CTAS_PER_SM * num_sms;
  return (unsigned)(items < cap ? items : cap);
}

}  // namespace

bool attention_window_direct(int B, int max_items, int heads) {
  return B <= 32 && (long long)max_items * heads <= window_grid(1ll << 40);
}

cudaError_t launch_attention_window_tc(const CUtensorMap* tm_qkv, const CUtensorMap* tm_qkv16, const AttnWindow& win,
                                       const void* qkv, void* o, Act out, int d, int heads, int max_items,
                                       const PackBuffers& pb, const PackedBatch& batch, const float* q_scale,
                                       float* amax, unsigned* err, cudaStream_t st, float* lse, int lse_stride) {
  if (max_items <= 0) return cudaSuccess;
  static bool configured[3] = {false, false, false};
  const unsigned grid = window_grid((long long)max_items * heads);
  const HeadDiv hd{(uint32_t)heads, (uint32_t)(((1ull << 32) + heads - 1) / heads)};
  auto run = [&](auto kernel, int which) -> cudaError_t {
    if (!configured[which]) {
      cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
      if (e != cudaSuccess) return e;
      // the register split draws on the registers that the block is launched with
      cudaFuncAttributes a;
      if ((e = cudaFuncGetAttributes(&a, kernel)) != cudaSuccess) return e;
      if (a.numRegs < kRegsLaunch) return cudaErrorInvalidKernelImage;
      configured[which] = true;
    }
    kernel<<<grid, THREADS, SMEM_BYTES, st>>>(*tm_qkv, *tm_qkv16, win, static_cast<const __nv_bfloat16*>(qkv), o, d, hd,
                                              pb, batch, q_scale, amax, lse, lse_stride, err);
    return cudaGetLastError();
  };
  if (out == Act::E4M3) return run(attention_window_tc_kernel<Act::E4M3>, 1);
  if (amax != nullptr) return run(attention_window_tc_kernel<Act::BF16, true>, 2);
  return run(attention_window_tc_kernel<Act::BF16>, 0);
}

}  // namespace esm
