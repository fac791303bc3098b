// Backward of the windowed attention on the tcgen05 tensor cores (head_dim 64, bf16 operands, fp32
// accumulation).
//
// With S = Q K^T / 8, P = exp(S - lse) where the query sees the key and 0 elsewhere (rows:
// queries), O = P V and dO given, per head:
//   dV = P^T dO,  dP = dO V^T,  dS = P * (dP - D) with D_i = sum_c dO_ic O_ic,
//   dK = dS^T Q / 8,  dQ = dS K / 8.
//
// Key j is visible to query i if j <= i + right and (j >= i - left or j < sinks).  An item is a key
// tile of 128 rows and a head; its query tiles start at the first query that sees any of its keys
// and end behind the last, so each key row's visible queries are one run of columns.  The keys of
// the first tile that are sinks are seen by every later query.  The tile itself goes on kFarStart
// queries past its band; the queries behind that, of a long sequence, are cut into chunks of
// kFarQueries, each an item of its own with the same key tile, so that no one CTA walks the whole
// sequence.  Such chunks and the tile itself leave the sinks' dK and dV as fp32 partial sums in
// slots, which a last kernel adds in slot order.  Slot 0 of a sequence that starts at row s0 is
// s0 / kFarSlotTokens: a sequence long enough to have chunks spans more slots than it uses, so
// no list of them is needed.
//
// One CTA per SM walks the items in rounds, in snake order.  TMEM lanes are keys throughout; per
// (key tile, query tile) pair:
//   S^T  = K Q^T - 8 lse (M=128 keys, N=128 queries, K=64 + 16)   TMEM cols [0,128)
//   dP^T = V dO^T - D    (M=128, N=128, K=64 + 16)                 cols [128,256)
//   dV  += P^T dO       (M=128, N=64, K=128; P^T in cols [448,512), dO MN-major)  cols [384,448)
//   dK  += dS^T Q       (M=128, N=64, K=128; Q MN-major)           cols [320,384)
//   dQ_i = dS K         (M=128 queries, N=64, K=128 keys; dS and K MN-major)  cols [256,320)
// (the row terms -8 lse and -D are one more K step against rows of ones: read from shared memory
// by the threads that form P^T and dS^T, they waited behind the tensor core's own reads)
// Roles (512 threads; registers rebalanced per warpgroup with setmaxnreg):
//   warp 0       TMA: the Q and dO tiles of each pair into a 3-stage ring (straight from the packed
//                qkv and dO buffers), with their row terms: -8 lse and -D as sums of three bf16;
//   warp 2       TMA: the items' K tiles (two buffers) and V tiles (one: V is done with an item's
//                last dP^T);
//   warp 1       one thread issues S^T and dP^T of every pair, as soon as its operands are ready;
//   warp 3       one thread issues the three gradient products of every pair;
//   warps 4..11  two warpgroups, one per 64 queries of the tile; thread r owns key r: reads its
//                S^T and dP^T row segment, forms P^T = 2^(S^T log2(e) / 8) and dS^T = P^T dP^T
//                in registers (f32x2 pairs), hands S^T back, then writes dS^T into shared memory
//                (K-major, 128-byte swizzle; once the previous pair's dK and dQ products have read
//                it) and P^T into tensor memory (once its dV product has), both rounded to bf16 as
//                operands;
//   warps 12..15 thread r owns query r of the tile: reads dQ_i from TMEM, stages it in shared
//                memory and adds it into an fp32 accumulator in global memory with TMA
//                reduce-add (several key tiles contribute to each query row); after an item's last
//                pair they also bring out its dK (turned back through RoPE) and dV.
// Pairs run on across items.  Every mbarrier wait is bounded; on timeout the kernel latches an
// error bit and stops.
//
// What bounds it: the tensor core, by way of shared memory.  A pair is 34 MMAs of 75 to 100 cycles
// (M = 128 with N = 64 takes as long as N = 128: the operands' way out of shared memory), about
// 3400 cycles of the 4100 that a pair takes in long runs.  So the other readers of shared memory went
// where they could (row terms into the MMAs, P^T into tensor memory), and nothing waits for global
// memory or for the other warps' ends of items: three Q / dO stages, the next item's K and V loaded
// ahead, scores and gradient products from two threads.  Whole calls with fresh inputs, and in
// parentheses those of the first version, the full attention's form of the kernel with masks: 16384
// packed tokens, 20 heads, window 128 + 128, one sink 195 us (276), three quarters of it here; 34374
// tokens, left 512, four sinks 560 (791).  160 sequences of 100 tokens, one pair per item, 147 us a call
// after an L2 flush, where the full attention's backward takes 222.  What the call has beside this
// kernel is memory traffic: the row terms, the accumulator's zeros and its rounding to dq.
#include "attn_plan.cuh"
#include "common.cuh"
#include "internal.h"

namespace esm {
namespace {

constexpr int DH = 64;
constexpr int TB = 128;                 // rows of a key or query tile
constexpr int TILE = 128 * 128;         // 128 rows x 128 bytes (64 bf16)
constexpr int STG = 3;                  // Q, dO and row terms in flight
constexpr int kComputeWgs = 2;                      // P^T / dS^T warpgroups
constexpr int QPW = 128 / kComputeWgs;               // queries of a tile per compute warpgroup
constexpr int NSUB = QPW / 16;                       // 16-query sub-chunks per thread
// Warpgroups: 0 = TMA (warp 0), MMA (warp 1), two idle warps; 1..kComputeWgs = compute;
// the last = dQ.  Warp w reaches the TMEM lanes 32 (w % 4) .. + 31.
constexpr int kWarpCompute = 4, kWarpDq = 4 + 4 * kComputeWgs;
constexpr int THREADS = 32 * (kWarpDq + 4);
// Registers per thread at launch and after the warpgroup-wide setmaxnreg: warpgroup 0 and the dQ
// warpgroup give registers to the compute warpgroups (their P^T / dS^T pairs stay in registers
// until the shared buffers are free).
constexpr int kRegsLaunch = 128, kRegsWg0 = 96, kRegsDq = 96, kRegsCompute = 160;
static_assert(128 * (kRegsWg0 + kRegsDq) + 128 * kComputeWgs * kRegsCompute <= THREADS * kRegsLaunch,
              "register split");
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t COL_S = 0, COL_DP = 128, COL_DQ = 256, COL_DK = 320, COL_DV = 384, COL_P = 448;

struct BwdSmem {
  uint64_t k_full[2], k_empty[2], v_full, v_empty;
  uint64_t q_full[STG], q_empty[STG];
  uint64_t s_full, s_free, p_full, p_free, ds_free, dq_full, dq_free, acc_full, acc_free, s_done, mma_done;
  uint32_t tmem_base;
  volatile int abort;
};
// [dS^T 32K][Q 0..2][dO 0..2][K0][K1][V][dQ staging 4 x 4K][row terms 0..2][ones of S][ones of dP] then
// BwdSmem
constexpr int TERM_BYTES = 128 * 2 * kBwdTerms;  // 128 rows of 16 bf16
constexpr int OFF_DS = 0, OFF_Q = 2 * TILE, OFF_DO = OFF_Q + STG * TILE, OFF_K = OFF_DO + STG * TILE,
              OFF_V = OFF_K + 2 * TILE, OFF_DQ = OFF_V + TILE, OFF_TERM = OFF_DQ + TILE,
              OFF_ONE = OFF_TERM + STG * TERM_BYTES, OFF_BAR = OFF_ONE + 2 * TERM_BYTES;
constexpr int DQ_WARP_BYTES = 32 * 128;  // one dQ warp's 32 rows x 32 fp32, a box of the reduce-add
constexpr int SMEM_BYTES = OFF_BAR + (int)sizeof(BwdSmem) + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory of one CTA");

// 16-byte unit j of row r of a 128-row x 128-byte tile with the 128-byte swizzle.
__device__ __forceinline__ uint32_t swz(int r, int j) { return (uint32_t)(r * 128 + ((j ^ (r & 7)) << 4)); }

// Two 32-lane x 16-column TMEM loads (S^T and dP^T of the same queries) and one wait.
__device__ __forceinline__ void tmem_ld16x2(uint32_t ta, uint32_t tb, float (&a)[16], float (&b)[16]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
      "[%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(ta), "r"(tb)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    a[i] = __uint_as_float(r[i]);
    b[i] = __uint_as_float(r[16 + i]);
  }
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// 32 bytes to global memory: one store if the address allows it.
__device__ __forceinline__ void store32(__nv_bfloat16* p, const uint32_t (&w)[8], bool wide) {
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

// Shared-memory matrix descriptor of a K-major operand tile of 16 bf16 columns with the 32-byte swizzle
// (rows of 32 bytes, 8-row groups 256 bytes apart).
__device__ __forceinline__ uint64_t make_sw32_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);  // start address
  d |= (uint64_t)1u << 16;                    // leading byte offset (unused: one swizzle atom wide)
  d |= (uint64_t)(256u >> 4) << 32;           // stride byte offset: 8 rows x 32 B
  d |= (uint64_t)1u << 46;                    // descriptor version (tcgen05)
  d |= (uint64_t)6u << 61;                    // swizzle mode: 32 B
  return d;
}

// Queries past the first key tile's band that its own item still takes, queries of a chunk item,
// and tokens per slot.  A sequence has chunks from length 128 + left + 1 + kFarStart on, and
// 1 + ceil((L - kFarStart) / kFarQueries) <= L / kFarSlotTokens slots from there.
constexpr int kFarStart = 1024, kFarQueries = 2048, kFarSlotTokens = 512;

// Far chunks of the batch: count, then (s0, length, first query, slot) each.  count == NULL: none.
struct FarList {
  const int32_t* count;
  const int4* item;
  float* partial;  // [slot][heads][sinks][dK 64 | dV 64]
};

// Keys k0 .. k0 + krows - 1 (rows of the packed batch) of the sequence at row s0; its queries
// q0 .. q1 - 1 (positions in the sequence) in nq tiles.  slot: where the sinks' fp32 partial
// sums go (-1: nowhere, the gradients are written whole); far: a chunk item.
struct BItem {
  int k0, krows, s0, h, q0, q1, nq, slot;
  bool far;
};

// An item's list entry (loaded ahead), and its unpacking.
struct Raw {
  int4 w;
  int h;
  bool far;
};
__device__ __forceinline__ Raw load_item(const PackBuffers& pb, int it, const HeadDiv& hd, const FarList& fl,
                                         int n_far) {
  Raw raw;
  raw.far = it < n_far;  // the chunks first: they are the longest items
  uint32_t entry, h;
  hd.split((uint32_t)(raw.far ? it : it - n_far), entry, h);
  raw.h = (int)h;
  raw.w = __ldg((raw.far ? fl.item : reinterpret_cast<const int4*>(pb.work)) + entry);
  return raw;
}
__device__ __forceinline__ BItem make_item(const Raw& raw, const AttnWindow& win, const FarList& fl) {
  const int4& w = raw.w;
  BItem x;
  x.slot = -1;
  x.far = raw.far;
  x.h = raw.h;
  if (raw.far) {
    x.k0 = x.s0 = w.x;
    x.krows = win.sinks;
    x.q0 = w.z;
    x.q1 = min(w.y, w.z + kFarQueries);
    x.slot = w.w;
  } else {
    x.k0 = w.x;
    x.krows = w.y;
    x.s0 = w.z;
    const int p0 = w.x - w.z;
    x.q0 = win.right >= 0 ? max(0, p0 - win.right) : 0;
    x.q1 = w.w;
    if (win.left >= 0) {
      const int far0 = TB + win.left + 1 + kFarStart;
      x.q1 = min(w.w, p0 < win.sinks ? far0 : p0 + w.y + win.left);
      if (p0 < win.sinks && w.w > far0 && fl.count != nullptr) x.slot = w.z / kFarSlotTokens;
    }
  }
  x.nq = (x.q1 - x.q0 + TB - 1) / TB;
  return x;
}

__global__ void __launch_bounds__(THREADS, 1)
    attention_window_bwd_tc_kernel(const __grid_constant__ CUtensorMap tm_qkv,
                                   const __grid_constant__ CUtensorMap tm_do, const __grid_constant__ CUtensorMap tm_dq,
                                   const __grid_constant__ CUtensorMap tm_terms, AttnWindow win, FarList fl,
                                   __nv_bfloat16* __restrict__ dqkv, int T, int d,
                                   HeadDiv hd, PackBuffers pb, const float2* __restrict__ rope, int max_pos,
                                   unsigned* err) {
  const int heads = (int)hd.heads;
  const int n_far = fl.count != nullptr ? *fl.count * heads : 0;
  const int n_items = *pb.work_count * heads + n_far;
  if ((int)blockIdx.x >= n_items) return;  // whole CTA, before any barrier or TMEM use

  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  BwdSmem* sm = reinterpret_cast<BwdSmem*>(base + OFF_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Items in rounds of gridDim.x, snake order (the list is longest first, so this evens out loads).
  auto item_at = [&](int rnd) -> int {
    return rnd * (int)gridDim.x + ((rnd & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
  };

  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm->k_full[b], 1);
      mbar_init(&sm->k_empty[b], 1);
    }
    for (int b = 0; b < STG; ++b) {
      mbar_init(&sm->q_full[b], 1);
      mbar_init(&sm->q_empty[b], 1);
    }
    mbar_init(&sm->v_full, 1);
    mbar_init(&sm->v_empty, 1);
    mbar_init(&sm->ds_free, 1);
    mbar_init(&sm->s_full, 1);
    mbar_init(&sm->s_free, 4 * kComputeWgs);
    mbar_init(&sm->p_full, 4 * kComputeWgs);
    mbar_init(&sm->p_free, 1);
    mbar_init(&sm->dq_full, 1);
    mbar_init(&sm->dq_free, 4);
    mbar_init(&sm->acc_full, 1);
    mbar_init(&sm->acc_free, 4);
    mbar_init(&sm->s_done, 1);
    mbar_init(&sm->mma_done, 1);
    sm->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(&sm->tmem_base, TMEM_COLS);
  if (threadIdx.x < 256) {  // the rows of ones: columns 0..2 for S^T, 3..5 for dP^T, the others 0
    const int row = threadIdx.x & 127, which = threadIdx.x >> 7;
    uint4* dst = reinterpret_cast<uint4*>(base + OFF_ONE + which * TERM_BYTES + row * 32);
    const int at = (row >> 2) & 1;  // 32-byte swizzle: where the row's first 16 bytes lie
    dst[at] = which == 0 ? make_uint4(0x3f803f80u, 0x00003f80u, 0u, 0u) : make_uint4(0u, 0x3f800000u, 0x3f803f80u, 0u);
    dst[at ^ 1] = make_uint4(0u, 0u, 0u, 0u);
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsWg0));

  if (warp == 0) {
    // ------------------------------------------------------------ TMA: Q, dO and their row terms
    if (lane == 0) {
      tma_prefetch_desc(&tm_qkv);
      tma_prefetch_desc(&tm_do);
      int g = 0;
      for (int rnd = 0, it = item_at(0); it < n_items && !sm->abort; it = item_at(++rnd)) {
        const BItem x = make_item(load_item(pb, it, hd, fl, n_far), win, fl);
        for (int i = 0; i < x.nq; ++i, ++g) {
          const int st = g % STG;
          if (!mbar_wait(&sm->q_empty[st], (uint32_t)((g / STG) & 1) ^ 1u)) {
            latch_error(err, ERRBIT_TIMEOUT);
            sm->abort = 1;
            break;
          }
          mbar_arrive_expect_tx(&sm->q_full[st], 2 * TILE + TERM_BYTES);
          const int row = x.s0 + x.q0 + i * TB;
          tma_load_2d(base + OFF_Q + st * TILE, &tm_qkv, x.h * DH, row, &sm->q_full[st]);
          tma_load_2d(base + OFF_TERM + st * TERM_BYTES, &tm_terms, 0, x.h * T + row, &sm->q_full[st]);
          tma_load_2d(base + OFF_DO + st * TILE, &tm_do, x.h * DH, row, &sm->q_full[st]);
        }
      }
      // Copies still in flight can only exist if a consumer gave up early: they are waited for
      // (bounded) before the CTA exits.
      if (sm->abort)
        for (int k = g - 1; k >= 0 && k >= g - STG; --k)
          if (!mbar_wait(&sm->q_full[k % STG], (uint32_t)(k / STG) & 1u)) break;
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ TMA: K and V
    if (lane == 0) {
      int n = 0, n_v = 0;  // items; V tiles asked for (K: n_v or one more)
      for (int rnd = 0, it = item_at(0); it < n_items && !sm->abort; it = item_at(++rnd)) {
        const BItem x = make_item(load_item(pb, it, hd, fl, n_far), win, fl);
        const int kb = n & 1;
        bool in = mbar_wait(&sm->k_empty[kb], (uint32_t)((n >> 1) & 1) ^ 1u);
        if (in) {
          mbar_arrive_expect_tx(&sm->k_full[kb], TILE);
          tma_load_2d(base + OFF_K + kb * TILE, &tm_qkv, d + x.h * DH, x.k0, &sm->k_full[kb]);
          ++n;
          in = mbar_wait(&sm->v_empty, (uint32_t)(n_v & 1) ^ 1u);
        }
        if (!in) {
          latch_error(err, ERRBIT_TIMEOUT);
          sm->abort = 1;
          break;
        }
        mbar_arrive_expect_tx(&sm->v_full, TILE);
        tma_load_2d(base + OFF_V, &tm_qkv, 2 * d + x.h * DH, x.k0, &sm->v_full);
        ++n_v;
      }
      if (sm->abort) {
        for (int k = n - 1; k >= 0 && k >= n - 2; --k)
          if (!mbar_wait(&sm->k_full[k & 1], (uint32_t)(k >> 1) & 1u)) break;
        if (n_v > 0) mbar_wait(&sm->v_full, (uint32_t)(n_v - 1) & 1u);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer: S^T, dP^T
    // (A thread that issues is held until the tensor core accepts its MMA: with one issuer, scores
    // that were ready waited behind the 24 gradient MMAs before them.)
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16(TB, TB);
      const uint32_t sb = smem_u32(base);
      const uint64_t v_kmaj = make_sw128_desc(sb + OFF_V);
      const uint64_t ones_s = make_sw32_desc(sb + OFF_ONE), ones_dp = make_sw32_desc(sb + OFF_ONE + TERM_BYTES);
      bool ok = true;
      int g = 0, n = 0;
      for (int rnd = 0, it = item_at(0); it < n_items && ok && !sm->abort; it = item_at(++rnd), ++n) {
        const BItem x = make_item(load_item(pb, it, hd, fl, n_far), win, fl);
        const int kb = n & 1;
        if (!mbar_wait(&sm->k_full[kb], (uint32_t)(n >> 1) & 1u) || !mbar_wait(&sm->v_full, (uint32_t)n & 1u)) {
          ok = false;
          break;
        }
        const uint64_t k_kmaj = make_sw128_desc(sb + OFF_K + kb * TILE);
        for (int i = 0; i < x.nq; ++i, ++g) {
          const int st = g % STG;
          if (!mbar_wait(&sm->q_full[st], (uint32_t)(g / STG) & 1u) ||
              !mbar_wait(&sm->s_free, (uint32_t)(g & 1) ^ 1u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t q_kmaj = make_sw128_desc(sb + OFF_Q + st * TILE);
          const uint64_t do_kmaj = make_sw128_desc(sb + OFF_DO + st * TILE);
          const uint64_t terms = make_sw32_desc(sb + OFF_TERM + st * TERM_BYTES);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_bf16_ss(tmem + COL_S, k_kmaj + 2u * k, q_kmaj + 2u * k, idesc_s, k > 0 ? 1u : 0u);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_bf16_ss(tmem + COL_DP, v_kmaj + 2u * k, do_kmaj + 2u * k, idesc_s, k > 0 ? 1u : 0u);
          mma_bf16_ss(tmem + COL_S, ones_s, terms, idesc_s, 1u);
          mma_bf16_ss(tmem + COL_DP, ones_dp, terms, idesc_s, 1u);
          mma_commit(&sm->s_full);
          if (i == x.nq - 1) mma_commit(&sm->v_empty);
        }
      }
      if (!ok) {
        latch_error(err, ERRBIT_TIMEOUT);
        sm->abort = 1;
      }
      // every MMA of this thread has completed before tensor memory may be released
      mma_commit(&sm->s_done);
      mbar_wait(&sm->s_done, 0);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------ MMA issuer: dV, dK, dQ
    if (lane == 0) {
      constexpr uint32_t idesc_kv = idesc_bf16(TB, DH) | kIdescBMn;             // dV, dK
      constexpr uint32_t idesc_q = idesc_bf16(TB, DH) | kIdescAMn | kIdescBMn;  // dQ
      const uint32_t sb = smem_u32(base);
      const uint64_t ds_kmaj = make_sw128_desc(sb + OFF_DS);
      const uint64_t ds_mn = make_sw128_mn_desc(sb + OFF_DS, TILE);  // queries 64.. one tile further
      bool ok = true;
      int g = 0, n = 0;
      for (int rnd = 0, it = item_at(0); it < n_items && ok && !sm->abort; it = item_at(++rnd), ++n) {
        const BItem x = make_item(load_item(pb, it, hd, fl, n_far), win, fl);
        const int kb = n & 1;
        const uint64_t k_mn = make_sw128_mn_desc(sb + OFF_K + kb * TILE, TILE);
        for (int i = 0; i < x.nq; ++i, ++g) {
          const int st = g % STG;
          // the operands have landed (the pair's scores were made of them), P^T and dS^T are there,
          // the previous dQ has been read, and so have the previous item's dK and dV
          if (!mbar_wait(&sm->k_full[kb], (uint32_t)(n >> 1) & 1u) ||
              !mbar_wait(&sm->q_full[st], (uint32_t)(g / STG) & 1u) || !mbar_wait(&sm->p_full, (uint32_t)g & 1u) ||
              !mbar_wait(&sm->dq_free, (uint32_t)(g & 1) ^ 1u) ||
              (i == 0 && !mbar_wait(&sm->acc_free, (uint32_t)(n & 1) ^ 1u))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t q_mn = make_sw128_mn_desc(sb + OFF_Q + st * TILE, TILE);
          const uint64_t do_mn = make_sw128_mn_desc(sb + OFF_DO + st * TILE, TILE);
          // dK and dQ first: what the next pair writes into dS^T's place takes longest.  K = 128
          // queries (dQ: keys) in steps of 16
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            // K-major dS^T: queries 64.. live in the second 16 KB block
            const uint64_t koff = (uint64_t)(((k >> 2) * TILE) >> 4) + 2u * (uint64_t)(k & 3);
            mma_bf16_ss(tmem + COL_DK, ds_kmaj + koff, q_mn + 128u * (uint64_t)k, idesc_kv, (i > 0 || k > 0) ? 1u : 0u);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_bf16_ss(tmem + COL_DQ, ds_mn + 128u * (uint64_t)k, k_mn + 128u * (uint64_t)k, idesc_q,
                        k > 0 ? 1u : 0u);
          mma_commit(&sm->ds_free);
          mma_commit(&sm->dq_full);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_bf16_ts(tmem + COL_DV, tmem + COL_P + 8 * k, do_mn + 128u * (uint64_t)k, idesc_kv,
                        (i > 0 || k > 0) ? 1u : 0u);
          mma_commit(&sm->p_free);
          mma_commit(&sm->q_empty[st]);
          if (i == x.nq - 1) {
            mma_commit(&sm->acc_full);
            mma_commit(&sm->k_empty[kb]);
          }
        }
      }
      if (!ok) {
        latch_error(err, ERRBIT_TIMEOUT);
        sm->abort = 1;
      }
      mma_commit(&sm->mma_done);
      mbar_wait(&sm->mma_done, 0);
    }
    __syncwarp();
  } else if (warp >= kWarpCompute && warp < kWarpDq) {
    // ------------------------------------------------------------ P^T / dS^T
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsCompute));
    const int wg = (warp - kWarpCompute) >> 2;  // warpgroup: queries QPW wg .. QPW wg + QPW - 1 of each tile
    const int wq = warp & 3;
    const int r = wq * 32 + lane;    // key row of the tile (and index of the lse / D slot)
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    constexpr float kLog2e = 1.4426950408889634f;
    const float c = kLog2e / 8.f;  // scores scaled by 1/sqrt(64), in log2 units
    const uint64_t c2 = f2_pack(c, c);
    // this warpgroup's QPW queries of dS^T: 16-byte units unit0 .. of a 64-query block
    uint8_t* sDS = base + OFF_DS + ((QPW * wg) >> 6) * TILE;
    const int unit0 = ((QPW * wg) & 63) >> 3;
    const uint32_t col_p = tmem + lane_off + COL_P + QPW / 2 * wg;
    bool ok = true;
    int g = 0;
    for (int rnd = 0, it = item_at(0); it < n_items && ok; it = item_at(++rnd)) {
      const BItem x = make_item(load_item(pb, it, hd, fl, n_far), win, fl);
      const bool kval = r < x.krows;
      const int key = x.k0 - x.s0 + r;
      for (int i = 0; i < x.nq; ++i, ++g) {
        // the queries [cl, ch) of this warpgroup's half of the tile see this thread's key
        const int first = x.q0 + i * TB + QPW * wg;
        const int cl = win.right >= 0 ? key - win.right - first : 0;
        int ch = x.q1 - first;
        if (win.left >= 0 && key >= win.sinks) ch = min(ch, key + win.left + 1 - first);
        if (!kval) ch = 0;
        const bool full = __all_sync(0xffffffffu, cl <= 0 && ch >= QPW);
        if (!mbar_wait_warp(&sm->s_full, (uint32_t)g & 1u)) { ok = false; break; }
        tc_fence_after();
        // P^T and dS^T of this thread's key and QPW queries, as bf16 pairs, 16 queries at a time:
        // p = 2^(c s'), ds = p dp', with s' = s - 8 lse and dp' = dp - D from the tensor core, in
        // f32x2 pairs
        uint32_t pw[NSUB][8], dw[NSUB][8];
#pragma unroll
        for (int sub = 0; sub < NSUB; ++sub) {
          const int cq = QPW * wg + 16 * sub;  // first query (column) of the sub-chunk
          float sv[16], dp[16];
          tmem_ld16x2(tmem + lane_off + COL_S + cq, tmem + lane_off + COL_DP + cq, sv, dp);
          const uint32_t vis = low_bits(ch - 16 * sub) & ~low_bits(cl - 16 * sub);
#pragma unroll
          for (int j4 = 0; j4 < 4; ++j4) {
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
              const int j = 2 * j4 + h2;  // pair j: queries cq + 2j, cq + 2j + 1
              const uint64_t t = f2_mul(f2_pack(sv[2 * j], sv[2 * j + 1]), c2);
              float t0, t1;
              f2_unpack(t, t0, t1);
              float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
              if (!full) {
                p0 = (vis >> (2 * j) & 1u) ? p0 : 0.f;
                p1 = (vis >> (2 * j + 1) & 1u) ? p1 : 0.f;
              }
              const uint64_t pp = f2_pack(p0, p1);
              const uint64_t dd = f2_mul(pp, f2_pack(dp[2 * j], dp[2 * j + 1]));
              float d0, d1;
              f2_unpack(dd, d0, d1);
              pw[sub][j] = pack_bf16x2(p0, p1);
              dw[sub][j] = pack_bf16x2(d0, d1);
            }
          }
        }
        // S^T / dP^T are read: the tensor core may compute the next tile's
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->s_free);
        // dS^T may be overwritten once the previous pair's dK and dQ products have read it, P^T once its
        // dV product has
        if (!mbar_wait_warp(&sm->ds_free, (uint32_t)(g & 1) ^ 1u)) { ok = false; break; }
#pragma unroll
        for (int sub = 0; sub < NSUB; ++sub)
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2)
            *reinterpret_cast<uint4*>(sDS + swz(r, unit0 + 2 * sub + h2)) =
                make_uint4(dw[sub][4 * h2], dw[sub][4 * h2 + 1], dw[sub][4 * h2 + 2], dw[sub][4 * h2 + 3]);
        if (!mbar_wait_warp(&sm->p_free, (uint32_t)(g & 1) ^ 1u)) { ok = false; break; }
        tc_fence_after();
        static_assert(NSUB == 4, "two 16-column stores");
        tmem_st16(col_p, &pw[0][0]);
        tmem_st16(col_p + 16, &pw[2][0]);
        tmem_st_wait();
        tc_fence_before();
        fence_async_smem();  // generic-proxy writes of dS^T before the tensor core reads
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->p_full);
      }
    }
    if (!ok) {
      latch_error(err, ERRBIT_TIMEOUT);
      sm->abort = 1;
    }
  } else if (warp >= kWarpDq) {
    // ------------------------------------------------------------ dQ accumulation, dK / dV
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsDq));
    // Each warp adds its 32 rows of dQ_i (fp32) into the global accumulator with TMA reduce-add,
    // staged 32 columns at a time (128-byte swizzle); rows of queries past the sequence end hold
    // exact zeros (their dS columns are zero), so adding them is harmless.
    const int wq = warp & 3;  // lane l owns query row 32 wq + l of the tile
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    uint8_t* stage = base + OFF_DQ + wq * DQ_WARP_BYTES;
    if (lane == 0) tma_prefetch_desc(&tm_dq);
    const bool wide = (reinterpret_cast<uintptr_t>(dqkv) & 31) == 0;
    bool ok = true;
    int g = 0, n = 0;
    // An item's dK (scaled, RoPE undone) and dV, in 32-byte pieces straight from the threads that hold
    // a key each: four parts of 32 values, v = 0, 1 dV columns 32 v .. + 31 and v = 2, 3 dK's pairs
    // (j, j + 32), j in 16 (v - 2) .. + 15.
    auto take_out = [&](const BItem& x) {
      const int r = wq * 32 + lane, key = x.k0 + r;
      const bool kval = r < x.krows, part = x.slot >= 0 && (x.far || r < win.sinks);  // a sink's partial sums, fp32
      int p = key - x.s0;
      p = p < 0 ? 0 : (p >= max_pos ? max_pos - 1 : p);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const bool is_k = v >= 2;
        const int c0 = is_k ? 16 * (v - 2) : 32 * v, c1 = is_k ? c0 + 32 : c0 + 16;
        float a[16], b[16];
        const uint32_t acc = tmem + lane_off + (is_k ? COL_DK : COL_DV);
        tmem_ld16x2(acc + c0, acc + c1, a, b);
        if (v == 3) {  // the last TMEM read of the item
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm->acc_free);
        }
        if (kval && part) {
          float* dst = fl.partial + (((size_t)x.slot * heads + x.h) * win.sinks + r) * (2 * DH) + (is_k ? 0 : DH);
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            *reinterpret_cast<float4*>(dst + c0 + j) = make_float4(a[j], a[j + 1], a[j + 2], a[j + 3]);
            *reinterpret_cast<float4*>(dst + c1 + j) = make_float4(b[j], b[j + 1], b[j + 2], b[j + 3]);
          }
        } else if (kval) {
          if (is_k) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {  // pair (c0 + j, c0 + j + 32) turned back by its angle
              const float u = a[j] * 0.125f, w = b[j] * 0.125f;
              a[j] = u;
              b[j] = w;
              if (rope != nullptr) {
                const int jj = c0 + j;
                const float2 cs = __ldg(rope + ((size_t)(jj >> 1) * max_pos + p) * 2 + (jj & 1));
                a[j] = u * cs.x + w * cs.y;
                b[j] = w * cs.x - u * cs.y;
              }
            }
          }
          __nv_bfloat16* out = dqkv + (size_t)key * 3 * d + (is_k ? d : 2 * d) + x.h * DH;
          uint32_t w[2][8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            w[0][j] = pack_bf16x2(a[2 * j], a[2 * j + 1]);
            w[1][j] = pack_bf16x2(b[2 * j], b[2 * j + 1]);
          }
          store32(out + c0, w[0], wide);
          store32(out + c1, w[1], wide);
        }
        __syncwarp();  // the lanes part above; the next read of tensor memory takes them together
      }
    };
    for (int rnd = 0, it = item_at(0); it < n_items && ok; it = item_at(++rnd), ++n) {
      const BItem x = make_item(load_item(pb, it, hd, fl, n_far), win, fl);
      for (int i = 0; i < x.nq; ++i, ++g) {
        if (!mbar_wait_warp(&sm->dq_full, (uint32_t)g & 1u)) { ok = false; break; }
        tc_fence_after();
        if (i == x.nq - 1) {  // the item's accumulators first: the next item's products wait for them
          if (!mbar_wait_warp(&sm->acc_full, (uint32_t)n & 1u)) { ok = false; break; }
          tc_fence_after();
          take_out(x);
        }
        uint32_t a[2][32];
        tmem_ld32_nowait(tmem + lane_off + COL_DQ, a[0]);
        tmem_ld32_nowait(tmem + lane_off + COL_DQ + 32, a[1]);
        tmem_ld_wait_regs(a[0]);
        tmem_ld_wait_regs(a[1]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->dq_free);
        const int row = x.s0 + x.q0 + i * TB + wq * 32;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // the previous reduce must have finished reading the staging rows
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
#pragma unroll
          for (int u = 0; u < 8; ++u)
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((u ^ (lane & 7)) << 4)) =
                make_uint4(a[half][4 * u], a[half][4 * u + 1], a[half][4 * u + 2], a[half][4 * u + 3]);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_reduce_add_2d(&tm_dq, x.h * DH + 32 * half, row, stage);
            bulk_commit();
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();  // reduces complete before the CTA may exit
    __syncwarp();
    if (!ok) {
      latch_error(err, ERRBIT_TIMEOUT);
      sm->abort = 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Far chunks a batch can have (each needs more than 1024 tokens of its sequence), and slots.
int far_max_chunks(int T) { return T / kFarStart; }
int far_max_slots(int T) { return T / kFarSlotTokens + 1; }

// Lists the far chunks of the batch in sequence order; one CTA.
__global__ void __launch_bounds__(1024) attention_far_list_kernel(const int32_t* __restrict__ seg_start,
                                                                  const int32_t* __restrict__ seg_len, int B, int far0,
                                                                  int max_chunks, int32_t* count, int4* item) {
  __shared__ int warp_sum[32];
  __shared__ int base;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  if (threadIdx.x == 0) base = 0;
  __syncthreads();
  for (int b0 = 0; b0 < B; b0 += 1024) {
    const int b = b0 + threadIdx.x;
    const int s0 = b < B ? seg_start[b] : 0, len = b < B ? seg_len[b] : 0;
    const int n = len > far0 ? (len - far0 + kFarQueries - 1) / kFarQueries : 0;
    int v = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) warp_sum[wid] = v;
    __syncthreads();
    if (wid == 0) {
      int w = warp_sum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
      }
      warp_sum[lane] = w;
    }
    __syncthreads();
    const int at = base + (wid > 0 ? warp_sum[wid - 1] : 0) + v - n;
    for (int k = 0; k < n && at + k < max_chunks; ++k)
      item[at + k] = make_int4(s0, len, far0 + k * kFarQueries, s0 / kFarSlotTokens + 1 + k);
    __syncthreads();
    if (threadIdx.x == 1023) base = at + n;
    __syncthreads();
  }
  if (threadIdx.x == 0) *count = min(base, max_chunks);
}

// dK and dV of the sinks of sequences with far chunks: the slots' fp32 sums in slot order, dK
// scaled and turned back through RoPE, as bf16.  A block per (sequence, head); kSumRows sink rows at
// a time, each by a thread per pair (j, j + 32) (threads 0..31 of the row: dK, 32..63: dV).
constexpr int kSumRows = 8;
__global__ void __launch_bounds__(64 * kSumRows) attention_far_sum_kernel(const int32_t* __restrict__ seg_start,
                                                               const int32_t* __restrict__ seg_len, int far0, int sinks,
                                                               const float* __restrict__ partial,
                                                               __nv_bfloat16* __restrict__ dqkv, int d, int heads,
                                                               const float2* __restrict__ rope, int max_pos) {
  const int s0 = seg_start[blockIdx.x], len = seg_len[blockIdx.x], h = blockIdx.y;
  if (len <= far0) return;
  const int slots = 1 + (len - far0 + kFarQueries - 1) / kFarQueries;
  const int j = threadIdx.x & 31;
  const bool is_k = threadIdx.x < 32;
  const float* src = partial + ((size_t)(s0 / kFarSlotTokens) * heads + h) * sinks * (2 * DH) + (is_k ? 0 : DH) + j;
  for (int r = threadIdx.y; r < sinks; r += kSumRows) {
    float a = 0.f, b = 0.f;
#pragma unroll 8
    for (int k = 0; k < slots; ++k) {
      const float* at = src + ((size_t)k * heads * sinks + r) * (2 * DH);
      a += at[0];
      b += at[32];
    }
    if (is_k) {
      const float u = a * 0.125f, w = b * 0.125f;
      float2 cs = make_float2(1.f, 0.f);
      if (rope != nullptr) cs = __ldg(rope + ((size_t)(j >> 1) * max_pos + min(r, max_pos - 1)) * 2 + (j & 1));
      a = u * cs.x + w * cs.y;
      b = w * cs.x - u * cs.y;
    }
    __nv_bfloat16* row = dqkv + (size_t)(s0 + r) * 3 * d + (is_k ? d : 2 * d) + h * DH + j;
    row[0] = __float2bfloat16_rn(a);
    row[32] = __float2bfloat16_rn(b);
  }
}

// The row terms of the scores and of dP, per head and token 16 bf16: -8 lse and -D, D = sum_c dO_c O_c,
// as sums of three (hi, mid, lo: 24 bits), columns 0..2 and 3..5; and 0 into the token's and
// head's 64 values of the dQ accumulator.  Eight lanes per (token, head): lane p takes columns
// 8p .. 8p + 7, so the eight read the head's 128 bytes together.  With plan.cu the first block makes
// the work list instead (a launch of its own took 4 us of a small call).
constexpr int kTermThreads = 256;
__global__ void __launch_bounds__(kTermThreads)
    attention_bwd_terms_kernel(AttnPlan plan, PackBuffers pb, unsigned* err, const __nv_bfloat16* __restrict__ o,
                               const __nv_bfloat16* __restrict__ dout, const float* __restrict__ lse,
                               __nv_bfloat16* __restrict__ terms, float* __restrict__ dq_acc, int T, int d,
                               int heads) {
  if (plan.cu != nullptr && blockIdx.x == 0) {
    attn_plan<kTermThreads>(plan, pb, err);
    return;
  }
  const long long g = (long long)(blockIdx.x - (plan.cu != nullptr ? 1 : 0)) * kTermThreads + threadIdx.x;
  const long long i = g >> 3;
  const int p = (int)(g & 7);
  const bool ok = i < (long long)T * heads;
  const long long t = ok ? i / heads : 0;
  const int h = ok ? (int)(i % heads) : 0;
  float acc = 0.f;
  if (ok) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(o + t * d + h * DH) + p);
    const uint4 y = __ldg(reinterpret_cast<const uint4*>(dout + t * d + h * DH) + p);
    float4* z = reinterpret_cast<float4*>(dq_acc + t * d + h * DH) + p;
    z[0] = z[8] = make_float4(0.f, 0.f, 0.f, 0.f);
    const __nv_bfloat162* xh = reinterpret_cast<const __nv_bfloat162*>(&x);
    const __nv_bfloat162* yh = reinterpret_cast<const __nv_bfloat162*>(&y);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 xf = __bfloat1622float2(xh[k]), yf = __bfloat1622float2(yh[k]);
      acc = fmaf(xf.x, yf.x, acc);
      acc = fmaf(xf.y, yf.y, acc);
    }
  }
  acc += __shfl_xor_sync(0xffffffffu, acc, 1);
  acc += __shfl_xor_sync(0xffffffffu, acc, 2);
  acc += __shfl_xor_sync(0xffffffffu, acc, 4);
  if (!ok || p > 1) return;
  uint4* dst = reinterpret_cast<uint4*>(terms + ((size_t)h * T + t) * kBwdTerms);
  if (p == 1) {
    dst[1] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  auto split = [](float v, float (&out)[3]) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      out[k] = __bfloat162float(__float2bfloat16_rn(v));
      v -= out[k];
    }
  };
  float a[3], b[3];
  split(-8.f * __ldg(lse + (size_t)h * T + t), a);
  split(-acc, b);
  dst[0] = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], b[0]), pack_bf16x2(b[1], b[2]), 0u);
}

// Whether a batch of at most T tokens in sequences of at most max_len can have far chunks.
bool window_has_far(const AttnWindow& w, int T, int max_len) {
  return w.sinks > 0 && w.left >= 0 && (T < max_len ? T : max_len) > TB + w.left + 1 + kFarStart;
}

}  // namespace

// Scratch of the far chunks: [count, padded to 16 bytes][chunks][partial sums].
size_t attention_window_bwd_far_bytes(const AttnWindow& w, int T, int heads) {
  if (!window_has_far(w, T, T)) return 0;
  return 16 + 16 * (size_t)far_max_chunks(T) +
         sizeof(float) * (size_t)far_max_slots(T) * heads * w.sinks * (2 * DH);
}

cudaError_t launch_attention_window_bwd_tc(const CUtensorMap* tm_qkv, const CUtensorMap* tm_do,
                                           const CUtensorMap* tm_dq, const CUtensorMap* tm_terms, const AttnWindow& win,
                                           const __nv_bfloat16* o, const __nv_bfloat16* dout, const float* lse,
                                           __nv_bfloat16* terms, float* dq_acc,
                                           void* far, __nv_bfloat16* dqkv, int T, int B, int max_len, int d, int heads,
                                           int max_items, const PackBuffers& pb, const AttnPlan& plan,
                                           const float2* rope, int max_pos, int num_sms, unsigned* err,
                                           cudaStream_t st) {
  if (T <= 0 || max_items <= 0) return cudaSuccess;
  static bool configured = false;
  if (!configured) {
    cudaError_t e = cudaFuncSetAttribute(attention_window_bwd_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         SMEM_BYTES);
    if (e != cudaSuccess) return e;
    // the register split draws on the registers that the block is launched with
    cudaFuncAttributes a;
    if ((e = cudaFuncGetAttributes(&a, attention_window_bwd_tc_kernel)) != cudaSuccess) return e;
    if (a.numRegs < kRegsLaunch) return cudaErrorInvalidKernelImage;
    configured = true;
  }
  const long long th = (long long)T * heads;
  const unsigned blocks = (unsigned)((8 * th + kTermThreads - 1) / kTermThreads) + (plan.cu != nullptr ? 1u : 0u);
  attention_bwd_terms_kernel<<<blocks, kTermThreads, 0, st>>>(plan, pb, err, o, dout, lse, terms, dq_acc, T, d, heads);
  // (a sequence longer than max_len is malformed: it is reported and gets no chunks)
  const bool has_far = window_has_far(win, T, max_len);
  const int far0 = TB + win.left + 1 + kFarStart;
  FarList fl{};
  if (has_far) {
    int32_t* count = static_cast<int32_t*>(far);
    int4* item = reinterpret_cast<int4*>(count + 4);
    fl.count = count;
    fl.item = item;
    fl.partial = reinterpret_cast<float*>(item + far_max_chunks(T));
    attention_far_list_kernel<<<1, 1024, 0, st>>>(pb.seg_start, pb.seg_klen, B, far0, far_max_chunks(T), count, item);
  }
  const long long items = (long long)(max_items + (has_far ? far_max_chunks(T) : 0)) * heads;
  const unsigned grid = (unsigned)(items < num_sms ? items : num_sms);
  const HeadDiv hd{(uint32_t)heads, (uint32_t)(((1ull << 32) + heads - 1) / heads)};
  attention_window_bwd_tc_kernel<<<grid, THREADS, SMEM_BYTES, st>>>(*tm_qkv, *tm_do, *tm_dq, *tm_terms, win, fl,
                                                                    dqkv, T, d, hd, pb, rope, max_pos, err);
  if (has_far)
    attention_far_sum_kernel<<<dim3(B, heads), dim3(64, kSumRows), 0, st>>>(
        pb.seg_start, pb.seg_klen, far0, win.sinks, fl.partial, dqkv, d, heads, rope, max_pos);
  launch_attention_bwd_dq(dq_acc, dqkv, pb.pos_id, rope, max_pos, T, d, st);
  return cudaGetLastError();
}

}  // namespace esm
