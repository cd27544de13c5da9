// dt_prompt_attention — causal attention over whole prompts, packed one after the other.
//
// Token i of a prompt sees its prompt's tokens 0..i: out[i][h] = softmax_j<=i(scale q[i][h].k_j) v_j, query head h
// reading key/value head h / (Hq / Hkv).
//
// GB300 design: bound by the tensor cores (long prompts) and by what a tile costs to start and finish (short ones). An
// item is 256 query rows of one head, as two tiles of 128, and walks its keys in blocks of 128 that both tiles share.
// Per tile and block: S = Q K^T (both operands in shared memory) into tensor memory, a softmax by the tile's own eight
// warps, the weights written back as bf16 over their own scores in tensor memory, and O += P V with P read from there,
// so that P never passes through shared memory. The tiles alternate: while one is in its softmax the tensor cores work
// on the other. Softmax in base 2, fp32; the running maximum is raised (and O rescaled) only past a headroom of 2^20
// (at d = 64 of up to 2^26), which leaves O alone in nearly every block. A block's weights are taken against the
// maximum so far, at d = 128 while its own is still being found, at d = 64 without it: the weights' sum shows a row that
// left its headroom. P is rounded to bf16, the only rounding before the output's (the tensor cores want it in the
// values' type); the row sums are taken in fp32 from the unrounded weights.
// One CTA per SM stays for all of its items: the loads of the next item and its first scores run under the last block
// and the epilogue of the one before. Items are dealt out longest first, from a counter in the workspace (the order
// changes no result).
// Measured, 32/8 heads: one prompt of 16384, d = 128: 1390 us, 1.58 PFLOP/s, 82% of cuBLAS' burst rate (tensor pipe 72%
// active; S = Q K^T takes all of shared memory's bandwidth). 12 prompts of 33 to 2500: 205 us, 1.06 PFLOP/s (a block of
// both tiles takes 1.5 us, an item's end and start 2). 5 prompts of 1000 to 4097, d = 64: 180 us, 0.88 PFLOP/s (issue
// slots 63% taken, exponentials 41%, tensor pipe 41%: the softmax's own chain).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "attn_common.cuh"

namespace dt {
namespace {

constexpr int kPrTile = 128;                 // query rows of a tile
constexpr int kPrRows = 2 * kPrTile;         // of a CTA
constexpr int kPrKeys = 128;                 // keys per block
constexpr int kPrThreads = 640;              // warps 0-3: load, MMA, items, MMA (D = 64); then eight a tile's softmax
constexpr int kPrSoft = 256;                 // softmax threads of a tile
constexpr int kPrAhead = 3;                  // items that may be known ahead
constexpr int kPrSorted = 8;                 // prompts a lane of the item warp keeps: up to 256 are dealt out sorted
// Of a thread's weights of a block and row, 32 at most, of up to 2^-6: a larger sum holds a larger weight. (A weight
// may come near 1 before that.)
constexpr float kPrSumMost = 1.f;
static_assert(32 * kAtWeightMost <= kPrSumMost, "a sum that is taken again raises the reference");
// the longest packed batch (2^30 rows), in blocks of 128 keys of four threads' sums, and the others' weights
static_assert(4 * kPrSumMost * kAtValueMost * (INT_MAX / 2 / 128) < 3e38, "a row's weighted values have a sum");
static_assert(kAtWeightMost * kAtValueMost * (INT_MAX / 2) < 3e38, "a row's weighted values have a sum");
constexpr uint32_t kPrBox = kPrKeys * 128;   // 128 rows x 64 elements: 16 KB

struct PrParams {
  int total, B, Hq, Hkv, G, slots, grid;
  const int32_t* cu;           // [B + 1]
  const unsigned short* v;     // re-read only for values that are not finite
  long long v_stride;
  float scale_log2;            // scale * log2(e)
  unsigned short* out;         // [total][Hq][D]
};
struct PrMaps {
  CUtensorMap q, k, v;  // [total][heads][D], box 64 x 1 x 128
};

// The prompt that owns tile slot `slot`. Prompt b's tiles start at slot cu[b] / 256 + b: its ceil(len / 256) tiles end
// before the next prompt's start, so the slots are found by search, without a scan of the lengths; some stay unused.
__device__ __forceinline__ int pr_start(const PrParams& p, int b) { return p.cu[b] / kPrRows + b; }
__device__ __forceinline__ int pr_find(const PrParams& p, int slot, int lane) {  // -1: before the first prompt
  int lo = 0, n = p.B;
  while (true) {  // 32-ary: `n` shrinks to ceil(n / 32) each round
    const int step = (n + 31) / 32;
    const int b = lo + lane * step;
    const bool in = lane * step < n && b < p.B && pr_start(p, b) <= slot;
    const unsigned hits = __ballot_sync(0xFFFFFFFFu, in);
    if (hits == 0u) return -1;
    lo += (31 - __clz(hits)) * step;
    if (step == 1) return lo;
    n = step;
  }
}

struct PrItem {  // 256 rows of a prompt (its first row `lo`, `len` rows) from row q0 on, one head; len 0: no more items
  int lo, len, q0, head;
  // blocks of each tile: up to its last row's own (the tiles start on block borders); a tile past the end has none
  __device__ __forceinline__ int n0() const { return q0 / kPrKeys + 1; }
  __device__ __forceinline__ int n1() const { return q0 + kPrTile < len ? q0 / kPrKeys + 2 : 0; }
  __device__ __forceinline__ int blocks() const { return q0 / kPrKeys + (q0 + kPrTile < len ? 2 : 1); }
};

// The items in order, by a whole warp. Up to 256 prompts: all prompts' tiles sorted by their number in the prompt,
// latest (longest) first, found by counting (a lane holds the tile counts of eight prompts). More: the tile slots from
// the last to the first, which is sorted within each prompt.
struct PrDealer {
  int first[kPrSorted], rows[kPrSorted], tiles[kPrSorted];  // of the lane's prompts 32 m + lane
  int total;  // tiles (sorted) or slots
  bool sorted;
  __device__ __forceinline__ int from(int i) const {  // tiles numbered i and up, over all prompts
    int n = 0;
#pragma unroll
    for (int m = 0; m < kPrSorted; ++m) n += max(tiles[m] - i, 0);
    return __reduce_add_sync(0xFFFFFFFFu, n);
  }
  __device__ __forceinline__ void init(const PrParams& p, int lane) {
    sorted = p.B <= 32 * kPrSorted;
#pragma unroll
    for (int m = 0; m < kPrSorted; ++m) {
      const int b = 32 * m + lane;
      const int lo = sorted && b < p.B ? p.cu[b] : 0, hi = sorted && b < p.B ? p.cu[b + 1] : 0;
      first[m] = lo;
      rows[m] = lo < 0 || hi > p.total || lo >= hi ? 0 : hi - lo;
      tiles[m] = (rows[m] + kPrRows - 1) / kPrRows;
    }
    total = sorted ? from(0) : p.slots;
  }
  __device__ __forceinline__ PrItem item(const PrParams& p, long long w, int lane) const {  // len 0: nothing there
    PrItem it{0, 0, 0, static_cast<int>(w % p.Hq)};
    const int r = static_cast<int>(w / p.Hq);
    if (sorted) {
      int top = 0;
#pragma unroll
      for (int m = 0; m < kPrSorted; ++m) top = max(top, tiles[m]);
      int lo = 0, hi = __reduce_max_sync(0xFFFFFFFFu, top) - 1;  // the last i with from(i) > r
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (from(mid) > r) lo = mid;
        else hi = mid - 1;
      }
      int left = r - from(lo + 1);  // in order among the prompts with a tile `lo`
      bool found = false;
#pragma unroll
      for (int m = 0; m < kPrSorted; ++m) {
        unsigned has = __ballot_sync(0xFFFFFFFFu, tiles[m] > lo);
        if (!found && left < __popc(has)) {
          found = true;
          for (int skip = left; skip > 0; --skip) has &= has - 1u;
          it.lo = __shfl_sync(0xFFFFFFFFu, first[m], __ffs(has) - 1);
          it.len = __shfl_sync(0xFFFFFFFFu, rows[m], __ffs(has) - 1);
        }
        left -= __popc(has);
      }
      it.q0 = lo * kPrRows;
    } else {
      const int slot = p.slots - 1 - r;
      const int b = pr_find(p, slot, lane);
      if (b < 0) return it;
      it.q0 = (slot - pr_start(p, b)) * kPrRows;
      const int lo = p.cu[b], hi = p.cu[b + 1];
      if (lo < 0 || hi > p.total || lo >= hi || it.q0 < 0 || it.q0 >= hi - lo) return it;
      it.lo = lo;
      it.len = hi - lo;
    }
    return it;
  }
};

template <int D>
__global__ void __launch_bounds__(kPrThreads, 1) prompt_attn_kernel(PrParams p, const __grid_constant__ PrMaps maps,
                                                                    WsHeader* hdr) {
  constexpr int kHalves = D / 64;
  constexpr uint32_t kTileBytes = kHalves * kPrBox;          // one Q tile, one K block or one V block
  constexpr unsigned kStages = D == 128 ? 5 : 8;             // ring entries: K and V blocks in turn
  // Tensor memory, 512 columns. D = 64 leaves room for P beside S: the next scores are computed while the softmax is at
  // work, and its warps go from block to block. D = 128: P lies over S, and the next scores follow P V.
  constexpr bool kApart = D == 64;
  constexpr uint32_t kColP = kApart ? 256 : 0, kStepP = kApart ? 64 : 128, kColO = kApart ? 384 : 256, kStepO = D;
  extern __shared__ float4 smem_f4[];
  unsigned char* sq =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_f4) + 1023) & ~uintptr_t(1023));
  unsigned char* skv = sq + 2 * kTileBytes;
  __shared__ uint64_t q_full[2], q_empty[2], kv_full[kStages], kv_empty[kStages], s_full[2], p_full[2][2];
  __shared__ uint64_t s_empty[2], p_empty[2], o_full[2], o_empty[2], it_full[kPrAhead], it_empty[kPrAhead];
  __shared__ PrItem s_items[kPrAhead];
  __shared__ uint32_t s_tmem;
  __shared__ unsigned s_issued, s_used[2], s_qi[2], s_qu[2];  // copies issued and waited for (failure drain)
  __shared__ int s_bad[2];  // by tile: the last item (from 1 on) in whose last block a value was not finite
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;

  if (t == 0) {
    for (unsigned i = 0; i < kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i][0], kPrSoft / 32);
      mbar_init(&p_full[i][1], kPrSoft / 32);
      mbar_init(&s_empty[i], kPrSoft / 32);
      mbar_init(&p_empty[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_empty[i], kPrSoft / 32);
      s_qi[i] = s_qu[i] = s_used[i] = 0u;
      s_bad[i] = 0;
    }
    for (int i = 0; i < kPrAhead; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], (kApart ? 3 : 2) + 2 * kPrSoft / 32);  // the loader, MMA threads, softmax warps
    }
    mbar_fence_init();
    s_issued = 0u;
  }
  if (warp == 0 && lane < 3)
    asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &maps.q : lane == 1 ? &maps.k : &maps.v) : "memory");
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = s_tmem;
  at_launch_order();
  bool ok = true;
  // Item k (from 0) as a reader sees it; `arrive`: this thread counts as one of the slot's readers.
  auto read_item = [&](int k, PrItem& it, bool arrive) {
    const int s = k % kPrAhead;
    if (!at_wait(&it_full[s], static_cast<unsigned>(k / kPrAhead) & 1u)) return false;
    it = s_items[s];
    if (arrive) mbar_arrive(&it_empty[s]);
    return true;
  };

  if (warp == 2) {  // the items
    PrDealer dealer;
    dealer.init(p, lane);
    const long long end = static_cast<long long>(dealer.total) * p.Hq;
    int k = 0;
    for (long long w = blockIdx.x; ok;) {
      PrItem it{0, 0, 0, 0};
      const long long at = w;
      if (w < end) {  // the next one, for when this one is through
        unsigned got = 0;
        if (lane == 0) got = atomicAdd(&hdr->deal_next, 1u);
        w = static_cast<long long>(p.grid) + __shfl_sync(0xFFFFFFFFu, got, 0);
      } else if (lane == 0 && atomicAdd(&hdr->deal_done, 1u) == static_cast<unsigned>(p.grid) - 1u) {
        hdr->deal_next = hdr->deal_done = 0u;  // every CTA is through with them: ready for the next call
      }
      if (at < end) {
        it = dealer.item(p, at, lane);
        if (it.len == 0) continue;
      }
      const int s = k % kPrAhead;
      if (k >= kPrAhead)
        ok = __all_sync(0xFFFFFFFFu, at_wait(&it_empty[s], static_cast<unsigned>(k / kPrAhead - 1) & 1u));
      if (!ok) break;
      if (lane == 0) {
        s_items[s] = it;
        mbar_arrive(&it_full[s]);
      }
      __syncwarp();
      ++k;
      if (it.len == 0) break;
    }
    if (blockIdx.x == 0) {  // lengths that contradict themselves are reported once, when the items are out
      bool bad = lane == 0 && (p.cu[0] < 0 || p.cu[p.B] > p.total);
      for (int b = lane; b < p.B; b += 32) bad = bad || p.cu[b] > p.cu[b + 1];
      if (bad) record_error(hdr, DT_ERR_INVALID_ARG);
    }
  } else if (warp == 0) {
    if (elect_one()) {  // TMA, per item: Q0, K0, Q1, V0, K1, V1, ..., a Q when its buffer is free
      unsigned st = 0, par = 1u, e = 0, uq[2] = {0u, 0u};
      for (int k = 0; ok; ++k) {
        PrItem it;
        ok = read_item(k, it, true);
        if (!ok || it.len == 0) break;
        const int kvh = it.head / p.G, nblk = it.blocks();
        bool pending[2] = {true, it.n1() > 0};
        auto load_q = [&](int i) {  // if it is still to come and can
          if (!pending[i] || (uq[i] > 0 && !at_test(&q_empty[i], (uq[i] - 1u) & 1u))) return;
          pending[i] = false;
          mbar_expect_tx(&q_full[i], kTileBytes);
          for (int h = 0; h < kHalves; ++h)
            tma_load_3d(sq + i * kTileBytes + h * kPrBox, &maps.q, 64 * h, it.head, it.lo + it.q0 + i * kPrTile,
                        &q_full[i]);
          s_qi[i] = ++uq[i];
        };
        auto load_kv = [&](const CUtensorMap* map, int j) {
          if (e >= kStages) {
            const uint64_t t0 = pending[0] || pending[1] ? global_timer_ns() : 0;
            while ((pending[0] || pending[1]) && !at_test(&kv_empty[st], par)) {  // whichever comes first
              load_q(0);
              load_q(1);
              if (global_timer_ns() - t0 > kAtBudgetNs) return false;
              __nanosleep(40);
            }
            if (!at_wait(&kv_empty[st], par)) return false;
          }
          mbar_expect_tx(&kv_full[st], kTileBytes);
          for (int h = 0; h < kHalves; ++h)
            tma_load_3d(skv + st * kTileBytes + h * kPrBox, map, 64 * h, kvh, it.lo + j * kPrKeys, &kv_full[st]);
          s_issued = ++e;
          if (++st == kStages) {
            st = 0;
            par ^= 1u;
          }
          return true;
        };
        for (int j = 0; j < nblk && ok; ++j) {
          load_q(0);
          ok = load_kv(&maps.k, j);
          load_q(1);
          if (ok) ok = load_kv(&maps.v, j);
        }
        for (int i = 0; i < 2 && ok; ++i) {
          if (pending[i]) ok = at_wait(&q_empty[i], (uq[i] - 1u) & 1u);
          if (ok) load_q(i);
        }
      }
    }
  } else if (warp < 4) {
    if ((kApart || warp == 1) && elect_one()) {  // MMA
      const uint32_t id_s = umma_idesc(kPrKeys, 128), id_o = umma_idesc(D, 128) | (1u << 16);  // O: V MN-major
      const uint64_t dq = umma_desc_sw128(smem_u32(sq)), dk = umma_desc_sw128(smem_u32(skv));
      const uint64_t dv = umma_desc_sw128_mn(smem_u32(skv), kPrBox, 1024u);
      auto wait = [&](uint64_t* bar, unsigned parity) {
        const bool done = at_wait(bar, parity);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        return done;
      };
      auto issue_s = [&](int i, unsigned st) {  // S_i = Q_i K^T, the keys in ring entry st
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kPrBox + (kk & 3) * 32u) >> 4;
          umma_f16(tmem + 128u * i, dq + (i * (kTileBytes >> 4) + off), dk + (st * (kTileBytes >> 4) + off), id_s,
                   kk > 0 ? 1u : 0u);
        }
        umma_commit(&s_full[i]);
      };
      auto issue_o = [&](int i, unsigned st, int half, bool fresh) {  // O_i += P_i V, 64 of the keys of ring entry st
#pragma unroll
        for (int k2 = 0; k2 < kPrKeys / 32; ++k2) {
          const int kk = half * (kPrKeys / 32) + k2;
          umma_f16_ts(tmem + kColO + kStepO * i, tmem + kColP + kStepP * i + 8u * kk,
                      dv + (st * (kTileBytes >> 4) + kk * (2048u >> 4)), id_o, fresh && kk == 0 ? 0u : 1u);
        }
      };
      if constexpr (kApart) {
        // Scores and outputs are independent: warp 1 issues the scores, warp 3 the outputs. (One thread's waits would
        // take longer than the products.)
        unsigned e = warp == 1 ? 0u : 1u, uses[2] = {0u, 0u}, first[2] = {0u, 0u};
        for (int k = 0; ok; ++k) {
          PrItem it;
          ok = read_item(k, it, true);
          if (!ok || it.len == 0) break;
          const int n[2] = {it.n0(), it.n1()}, nblk = it.blocks();
          for (int j = 0; j < nblk && ok; ++j, e += 2u) {
            const unsigned st = e % kStages;
            ok = wait(&kv_full[st], (e / kStages) & 1u);
            if (!ok) break;
            s_used[warp >> 1] = e + 1u;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!ok || j >= n[i]) continue;
              if (warp == 1) {
                if (j == 0) {
                  ok = wait(&q_full[i], first[i] & 1u);
                  if (!ok) continue;
                  s_qu[i] = ++first[i];
                }
                if (uses[i] > 0) ok = wait(&s_empty[i], (uses[i] - 1u) & 1u);  // the scores before have been read
                ++uses[i];
                if (!ok) continue;
                issue_s(i, st);
                if (j + 1 == n[i]) umma_commit(&q_empty[i]);
              } else {
                if (j == 0) {  // the epilogue before has read O
                  if (first[i] > 0) ok = wait(&o_empty[i], (first[i] - 1u) & 1u);
                  ++first[i];
                }
                if (ok) ok = wait(&p_full[i][1], uses[i] & 1u);
                ++uses[i];
                if (!ok) continue;
                issue_o(i, st, 0, j == 0);
                issue_o(i, st, 1, false);
                umma_commit(&p_empty[i]);
                if (j + 1 == n[i]) umma_commit(&o_full[i]);
              }
            }
            if (ok) umma_commit(&kv_empty[st]);
          }
        }
      } else {
        unsigned st = 0, par = 0, used = 0;  // ring entry last waited for and its parity: K_j, V_j, K_{j+1}, ...
        auto step = [&]() {
          if (++st == kStages) {
            st = 0;
            par ^= 1u;
          }
        };
        auto wait_entry = [&]() {
          const bool done = wait(&kv_full[st], par);
          if (done) s_used[0] = ++used;
          return done;
        };
        unsigned uq[2] = {0u, 0u}, up[2] = {0u, 0u}, uo[2] = {0u, 0u};  // uses so far
        // The first scores of tile i of an item whose K0 is in entry st; q_empty follows the last scores of a tile.
        auto start = [&](int i, int n) {
          if (n == 0) return true;
          if (!wait(&q_full[i], uq[i] & 1u)) return false;
          s_qu[i] = ++uq[i];
          issue_s(i, st);
          if (n == 1) umma_commit(&q_empty[i]);
          return true;
        };
        PrItem it;
        ok = read_item(0, it, true);
        int n[2] = {it.n0(), it.n1()}, nblk = it.blocks();
        bool more = ok && it.len > 0;
        if (more) {
          ok = wait_entry() && start(0, n[0]) && start(1, n[1]);
          if (ok) umma_commit(&kv_empty[0]);
        }
        for (int k = 0; ok && more; ++k) {
          ok = read_item(k + 1, it, true);
          if (!ok) break;
          more = it.len > 0;
          const int m[2] = {more ? it.n0() : 0, more ? it.n1() : 0};  // the next item's
          for (int j = 0; j < nblk && ok; ++j) {
            const bool last = j + 1 == nblk;
            step();
            const unsigned sv = st;
            ok = wait_entry();
            if (ok && (!last || more)) {  // the next block's keys, or the next item's first
              step();
              ok = wait_entry();
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!ok) continue;
              if (j < n[i]) {
                if (j == 0) {  // the epilogue before has read O
                  if (uo[i] > 0) ok = wait(&o_empty[i], (uo[i] - 1u) & 1u);
                  ++uo[i];
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                  if (ok) ok = wait(&p_full[i][half], up[i] & 1u);
                  if (ok) issue_o(i, sv, half, j == 0);
                }
                ++up[i];
                if (!ok) continue;
                if (j + 1 == n[i]) {
                  umma_commit(&o_full[i]);
                } else {  // the next scores overwrite P: the tensor cores run this thread's products in order
                  issue_s(i, st);
                  if (j + 2 == n[i]) umma_commit(&q_empty[i]);
                }
              }
              if (last) ok = start(i, m[i]);
            }
            if (ok) {
              umma_commit(&kv_empty[sv]);
              if (!last || more) umma_commit(&kv_empty[st]);
            }
          }
          n[0] = m[0];
          n[1] = m[1];
          nblk = it.blocks();
        }
      }
    }
  } else if (warp >= 4) {  // softmax of tile i
    // A warp owns 16 rows of its quarter of tensor memory; four neighbouring threads share two rows (ra, ra + 8), each
    // holding a quarter of their columns.
    const int i = (warp - 4) >> 3, tt = t - 128 - kPrSoft * i;
    const int lane0 = 32 * (warp & 3) + 16 * (((warp - 4) >> 2) & 1);
    const uint32_t lanes = static_cast<uint32_t>(lane0) << 16;
    const uint32_t ts = tmem + lanes + 128u * i, tp = tmem + lanes + kColP + kStepP * i;
    const uint32_t to = tmem + lanes + kColO + kStepO * i;
    const int ra = lane0 + (lane >> 2), quad = lane & 3, col = 2 * quad;
    unsigned base = 0, us = 0, uo = 0;  // ring entry of the item's K0; blocks and items of this tile so far
    for (int k = 0; ok; ++k) {
      ok = __all_sync(0xFFFFFFFFu, at_wait(&it_full[k % kPrAhead], static_cast<unsigned>(k / kPrAhead) & 1u));
      if (!ok) break;
      const PrItem& it = s_items[k % kPrAhead];  // stays until this warp is through with it
      if (it.len == 0) break;
      const int nb = i ? it.n1() : it.n0();
      const int row0 = it.q0 + i * kPrTile + ra;  // row ra's token in its prompt; the other row's is 8 further
      // minus the weights' reference: the running maximum of the scaled scores, as last raised, and kAtShift
      float nref[2] = {kAtNone, kAtNone};
      float l[2] = {0.f, 0.f};                    // sums of this thread's weights
      for (int j = 0; j < nb && ok; ++j, ++us) {
        const bool diag = j + 1 == nb;
        if (diag) {
          // The block where the tile's rows see different keys. A weight of zero does not hide a value that is not
          // finite from the tensor cores (0 x inf is NaN): rows past the prompt's end are cleared, and what is not
          // finite among the block's values is cleared too and added to the rows that see it at the end (its weight
          // there is positive, and any positive multiple of it gives the same sum).
          const unsigned e = base + 2u * j + 1u;
          ok = at_issued(&s_issued, e) && at_wait(&kv_full[e % kStages], (e / kStages) & 1u) && ok;
          unsigned char* sv = skv + (e % kStages) * kTileBytes;
          const int valid = it.len - j * kPrKeys;  // keys of the block inside the prompt
          __nv_bfloat162 acc = __floats2bfloat162_rn(0.f, 0.f);
          const __nv_bfloat162 zero = acc;
#pragma unroll 4
          for (int c = tt; c < kHalves * kPrKeys * 8; c += kPrSoft) {  // 16-byte pieces; eight a row
            uint4* at = reinterpret_cast<uint4*>(sv + 16 * c);
            if (((c >> 3) & (kPrKeys - 1)) >= valid) {
              *at = make_uint4(0u, 0u, 0u, 0u);
            } else {
              const uint4 x = *at;
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int k2 = 0; k2 < 4; ++k2)
                acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[k2]), zero, acc);  // x 0: NaN if not finite
            }
          }
          const float2 a2 = __bfloat1622float2(acc);
          if (!(a2.x == 0.f && a2.y == 0.f)) {  // rare
            for (int c = tt; c < kHalves * kPrKeys * 8; c += kPrSoft) {
              unsigned short* at = reinterpret_cast<unsigned short*>(sv + 16 * c);
              for (int k2 = 0; k2 < 8; ++k2)
                if ((at[k2] & 0x7F80u) == 0x7F80u) at[k2] = 0;
            }
            atomicMax(&s_bad[i], k + 1);
          }
        }
        ok = at_wait(&s_full[i], us & 1u) && ok;
        __syncwarp();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        float s[64];
        at_ld_s(ts, s);
        // Apart, the weights before have been read and their products are in O only after this.
        auto p_free = [&]() {
          if (kApart && us > 0) ok = at_wait(&p_empty[i], (us - 1u) & 1u) && ok;
          __syncwarp();
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        };
        auto mask = [&]() {
          const int lim = row0 - j * kPrKeys - col;  // row ra sees this thread's columns 8 g + e up to here
#pragma unroll
          for (int g = 0; g < 16; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (8 * g + (e & 1) > lim + 8 * (e >> 1)) s[4 * g + e] = -INFINITY;
        };
        if (diag) mask();
        float mx[2], alpha[2];
        auto rescale = [&]() {
          p_free();  // (not apart, S is full only after the products into O before it)
#pragma unroll 1
          for (int h = 0; h < D / 32; ++h) {
            float o[16];
            at_ld_o(to + 32u * h, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= alpha[(e >> 1) & 1];
            at_st_o(to + 32u * h, o);
          }
        };
        uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
        // half of the weights are in place: their products may start (apart, all of them start together)
        auto give = [&](int h, const uint32_t (&pk)[16]) {
          at_st_p(tp + 32u * h, pk);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          if (diag && h == 0) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the cleared values
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0 && (!kApart || h == 1)) mbar_arrive(&p_full[i][h]);
        };
        if (kApart) {
          if (j == 0) {  // the first block sets the reference
            at_max(s, p.scale_log2, mx);
            at_raise(mx, nref, l, alpha);
          }
          // Later blocks take their weights against the reference so far; their sums show a row that left its headroom.
          uint32_t pk[16], pk1[16];
          at_weights<0>(s, p.scale_log2, nref, ls, pk);
          at_weights<1>(s, p.scale_log2, nref, ls, pk1);
          float sum[2] = {0.f, 0.f};
          at_sums(ls, sum);
          if (__any_sync(0xFFFFFFFFu, !(sum[0] <= kPrSumMost && sum[1] <= kPrSumMost))) {  // rare (or NaN)
            at_ld_s(ts, s);
            if (diag) mask();
            at_max(s, p.scale_log2, mx);
            at_raise(mx, nref, l, alpha);
            if (j > 0) rescale();
#pragma unroll
            for (int c = 0; c < 4; ++c) ls[c] = 0ull;
            at_weights<0>(s, p.scale_log2, nref, ls, pk);
            at_weights<1>(s, p.scale_log2, nref, ls, pk1);
            sum[0] = sum[1] = 0.f;
            at_sums(ls, sum);
          }
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[i]);
          p_free();
          l[0] += sum[0];
          l[1] += sum[1];
          give(0, pk);
          give(1, pk1);
        } else {
          at_max(s, p.scale_log2, mx);
          auto raised = [&]() {
            return __any_sync(0xFFFFFFFFu, mx[0] + nref[0] > kAtMost || mx[1] + nref[1] > kAtMost);
          };
          if (j == 0) at_raise(mx, nref, l, alpha);  // the first block sets the reference
          // Later blocks' weights are taken against the reference so far while the maxima are being found.
          uint32_t pk[16];
          at_weights<0>(s, p.scale_log2, nref, ls, pk);
          if (j > 0 && raised()) {  // rare: take the scores and the weights again
            at_raise(mx, nref, l, alpha);
            rescale();
            at_ld_s(ts, s);
            if (diag) mask();
#pragma unroll
            for (int c = 0; c < 4; ++c) ls[c] = 0ull;
            at_weights<0>(s, p.scale_log2, nref, ls, pk);
          }
          give(0, pk);
          at_weights<1>(s, p.scale_log2, nref, ls, pk);
          give(1, pk);
          at_sums(ls, l);
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
      }
      if (!ok) break;
      base += 2u * it.blocks();
      if (nb == 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&it_empty[k % kPrAhead]);
        continue;
      }
      ok = __all_sync(0xFFFFFFFFu, at_wait(&o_full[i], uo & 1u));
      if (!ok) break;
      ++uo;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      float inv[2];
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2) {
        l[k2] += __shfl_xor_sync(0xFFFFFFFFu, l[k2], 1);
        l[k2] += __shfl_xor_sync(0xFFFFFFFFu, l[k2], 2);
        inv[k2] = at_rcp(l[k2]);  // the row's own key is visible; a sum of 0 or NaN gives NaN
      }
      // a later item's mark counts too: adding what is not finite to rows that see it changes nothing
      const volatile int* marks = s_bad;
      const bool bad = marks[0] > k || marks[1] > k;
      unsigned short* po = p.out + (static_cast<size_t>(it.lo + row0) * p.Hq + it.head) * D + 8 * quad;
      float o[D / 2];
      if constexpr (D == 128)
        at_ld_s(to, o);
      else
        at_ld_half(to, o);
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_empty[i]);  // O is free for the next item
      if (bad) {  // rare: tile 0's clearing reaches tile 1 too, which shares the block
        for (int key = (it.n0() - 1) * kPrKeys; key <= row0 + 8 && key < it.len; ++key) {
          const unsigned short* vr = p.v + static_cast<size_t>(it.lo + key) * p.v_stride + it.head / p.G * D + col;
#pragma unroll
          for (int e = 0; e < D / 2; ++e) {
            const uint32_t bits = static_cast<uint32_t>(vr[8 * (e >> 2) + (e & 1)]) << 16;
            if ((bits & 0x7F800000u) == 0x7F800000u && key <= row0 + 8 * ((e >> 1) & 1)) o[e] += __uint_as_float(bits);
          }
        }
      }
#pragma unroll
      for (int h = 0; h < D / 32; ++h)
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
          const uint4 x = at_row16(o + 16 * h, k2, inv[k2], quad);
          if (row0 + 8 * k2 < it.len)
            *reinterpret_cast<uint4*>(po + static_cast<size_t>(8 * k2) * p.Hq * D + 32 * h) = x;
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&it_empty[k % kPrAhead]);
    }
  }
  ok = __syncthreads_and(ok);
  if (!ok && t == 0) {
    record_error(hdr, DT_ERR_TIMEOUT);
    // copies issued but never waited for must land before the CTA leaves: wait for them too (bounded)
    // (with two MMA threads, entries one of them has seen may be counted again: their phase is over or comes)
    for (unsigned e = kApart ? min(s_used[0], s_used[1]) : s_used[0]; e < s_issued; ++e)
      mbar_wait(&kv_full[e % kStages], (e / kStages) & 1u, kAtBudgetNs);
    for (int i = 0; i < 2; ++i)
      for (unsigned e = s_qu[i]; e < s_qi[i]; ++e) mbar_wait(&q_full[i], e & 1u, kAtBudgetNs);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

template <int D>
dt_status pr_launch(const PrParams& p, const PrMaps& maps, WsHeader* hdr, cudaStream_t stream) {
  constexpr size_t smem = 1024 + (2 + (D == 128 ? 5 : 8)) * static_cast<size_t>(D / 64) * kPrBox;
  const void* fn = reinterpret_cast<const void*>(prompt_attn_kernel<D>);
  if (ensure_dynamic_smem(fn, smem) != cudaSuccess) return DT_ERR_CUDA;
  return at_launch(prompt_attn_kernel<D>, p.grid, kPrThreads, smem, stream, p, maps, hdr);
}

}  // namespace
}  // namespace dt

extern "C" size_t dt_prompt_attention_workspace_bytes(int total, int B, int Hq, int Hkv, int d) {
  if (total < 1 || B < 1 || Hq < 1 || Hkv < 1 || d < 1 || Hq % Hkv != 0) return 0;
  return sizeof(dt::WsHeader);
}

extern "C" dt_status dt_prompt_attention(int total, int B, int Hq, int Hkv, int d, const void* q, int64_t q_stride,
                                         const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                         dt_dtype dtype, const int32_t* cu_seqlens, float scale, void* out,
                                         void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  using namespace dt;
  if (total < 0 || B < 0 || Hq < 1 || Hkv < 1 || d < 1 || Hq % Hkv != 0) return DT_ERR_INVALID_ARG;
  if (dtype != DT_F32 && dtype != DT_BF16) return DT_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale * 1.4426950408889634f)) return DT_ERR_INVALID_ARG;
  if (total == 0 || B == 0) return DT_OK;
  const void* ptrs[] = {q, k, v, out, workspace};
  for (const void* x : ptrs)
    if (!x || !aligned16(x)) return DT_ERR_INVALID_ARG;
  if (!cu_seqlens || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u)) return DT_ERR_INVALID_ARG;
  if (workspace_bytes < sizeof(WsHeader)) return DT_ERR_INVALID_ARG;
  if (Hq > DT_MAX_HEADS) return DT_ERR_UNSUPPORTED;
  const int64_t width[3] = {static_cast<int64_t>(Hq) * d, static_cast<int64_t>(Hkv) * d, static_cast<int64_t>(Hkv) * d};
  const int64_t stride[3] = {q_stride, k_stride, v_stride};
  for (int i = 0; i < 3; ++i)
    if (stride[i] < width[i] || stride[i] % 8 != 0 || stride[i] > INT_MAX) return DT_ERR_INVALID_ARG;
  if (dtype != DT_BF16 || (d != 64 && d != 128)) return DT_ERR_UNSUPPORTED;
  const long long slots = total / kPrRows + static_cast<long long>(B);
  if (total > INT_MAX / 2 || slots * Hq > INT_MAX) return DT_ERR_UNSUPPORTED;
  PrParams p{};
  p.total = total; p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv; p.slots = static_cast<int>(slots);
  DeviceInfo di{};
  if (current_device_info(&di) != cudaSuccess) return DT_ERR_CUDA;
  p.grid = slots * Hq < di.sms ? static_cast<int>(slots * Hq) : di.sms;
  p.cu = cu_seqlens;
  p.v = static_cast<const unsigned short*>(v);
  p.v_stride = v_stride;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = static_cast<unsigned short*>(out);
  PrMaps maps{};
  const uint64_t dd = static_cast<uint64_t>(d), rows = static_cast<uint64_t>(total);
  if (!encode_bf16_3d_pitched(&maps.q, q, dd, static_cast<uint64_t>(Hq), rows, dd, static_cast<uint64_t>(q_stride), 64,
                              1, kPrTile) ||
      !encode_bf16_3d_pitched(&maps.k, k, dd, static_cast<uint64_t>(Hkv), rows, dd, static_cast<uint64_t>(k_stride), 64,
                              1, kPrKeys) ||
      !encode_bf16_3d_pitched(&maps.v, v, dd, static_cast<uint64_t>(Hkv), rows, dd, static_cast<uint64_t>(v_stride), 64,
                              1, kPrKeys))
    return DT_ERR_CUDA;
  WsHeader* hdr = static_cast<WsHeader*>(workspace);
  return d == 64 ? pr_launch<64>(p, maps, hdr, stream) : pr_launch<128>(p, maps, hdr, stream);
}
