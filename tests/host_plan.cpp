// The work list of the windowed attention (attn_plan.cuh) run on the host: a thread per CUDA thread of one
// block, a barrier per warp and one for the block behind the collectives that the header uses.
// ATTN_PLAN_SOURCE is the header's text without its includes.
#include <algorithm>
#include <atomic>
#include <barrier>
#include <cstdint>
#include <cstring>
#include <memory>
#include <thread>
#include <vector>

#define __device__
#define __forceinline__ inline
#define __shared__ static
using std::max;
using std::min;

struct int4 {
  int x, y, z, w;
};
static int4 make_int4(int x, int y, int z, int w) { return {x, y, z, w}; }
struct Dim {
  int x;
};
static thread_local Dim threadIdx{0};
static Dim gridDim{1};

struct Warp {
  std::barrier<> bar{32};
  int v[32];
};
static std::vector<std::unique_ptr<Warp>> warps;
static std::unique_ptr<std::barrier<>> block;

static Warp& warp() { return *warps[threadIdx.x >> 5]; }
template <typename F>
static auto exchange(int v, F f) {
  Warp& w = warp();
  w.v[threadIdx.x & 31] = v;
  w.bar.arrive_and_wait();
  auto r = f(w.v);
  w.bar.arrive_and_wait();
  return r;
}
static int __shfl_sync(unsigned, int v, int src) {
  return exchange(v, [=](const int* a) { return a[src & 31]; });
}
static int __shfl_up_sync(unsigned, int v, int o) {
  const int lane = threadIdx.x & 31;
  return exchange(v, [=](const int* a) { return a[lane >= o ? lane - o : lane]; });
}
static unsigned __ballot_sync(unsigned, bool p) {
  return exchange(p, [](const int* a) {
    unsigned m = 0;
    for (int i = 0; i < 32; ++i) m |= a[i] ? 1u << i : 0u;
    return m;
  });
}
static void __syncthreads() { block->arrive_and_wait(); }
static int __ffs(unsigned v) { return v ? __builtin_ctz(v) + 1 : 0; }
static uint32_t __umulhi(uint32_t a, uint32_t b) { return (uint32_t)((uint64_t)a * b >> 32); }
template <typename T>
static T __ldg(const T* p) { return *p; }
static int atomicAdd(int* p, int v) { return std::atomic_ref<int>(*p).fetch_add(v); }

static constexpr unsigned ERRBIT_CU_SEQLENS = 1u;
static void latch_error(unsigned* err, unsigned bit) { std::atomic_ref<unsigned>(*err).fetch_or(bit); }

namespace esm {
struct AttnWindow {
  int left, right, sinks;
};
struct PackBuffers {
  int32_t *pos_id, *seg_id, *seg_start, *seg_qlen, *seg_klen, *work, *work_count;
};
struct AttnPlan {
  const int32_t* cu;
  int B, T, max_seqlen, max_positions, q_tile, max_items;
  AttnWindow win;
  bool backward;
  int sort_above;
};
struct PackedBatch {
  const int32_t* cu;
  int B, T, max_seqlen, max_positions;
};
}  // namespace esm

#include ATTN_PLAN_SOURCE

template <typename F>
static void run_block(int threads, F f) {
  warps.clear();
  for (int i = 0; i < threads / 32; ++i) warps.push_back(std::make_unique<Warp>());
  block = std::make_unique<std::barrier<>>(threads);
  std::vector<std::thread> ts;
  for (int t = 0; t < threads; ++t)
    ts.emplace_back([=] {
      threadIdx.x = t;
      f(t);
    });
  for (auto& t : ts) t.join();
}

extern "C" {

// work: [max_items][4]; returns the listed items.
int host_attn_plan(const int32_t* cu, int B, int T, int max_seqlen, int max_positions, int max_items, int left, int right,
                   int sinks, int backward, int sort_above, int32_t* work, unsigned* err) {
  std::vector<int32_t> seg(3 * (size_t)B);
  int32_t count = -1;
  const esm::PackBuffers pb{nullptr, nullptr, seg.data(), seg.data() + B, seg.data() + 2 * B, work, &count};
  const esm::AttnPlan plan{cu, B, T, max_seqlen, max_positions, 128, max_items, {left, right, sinks}, backward != 0, sort_above};
  run_block(256, [&](int) { esm::attn_plan<256>(plan, pb, err); });
  return count;
}

// Item of block `it` in a grid of `grid` blocks: item[5] = row, rows, first key row, keys, head; returns the item count.
int host_find_item(const int32_t* cu, int B, int T, int max_seqlen, int max_positions, int heads, int grid, int it,
                   int32_t* item, unsigned* err) {
  gridDim.x = grid;
  const esm::HeadDiv hd{(uint32_t)heads, (uint32_t)(((1ull << 32) + heads - 1) / heads)};
  const esm::PackedBatch batch{cu, B, T, max_seqlen, max_positions};
  int count = -1;
  run_block(32, [&](int t) {
    int n = -1;
    const esm::RawItem raw = esm::find_item<128>(batch, it, hd, n, err);
    if (t > 0) return;
    count = n;
    const int v[5] = {raw.w.x, raw.w.y, raw.w.z, raw.w.w, raw.h};
    std::memcpy(item, v, sizeof v);
  });
  return count;
}

}  // extern "C"
