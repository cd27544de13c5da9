// dt_paged_attention — attention of each request's newest tokens over its paged key/value cache.
//
// For request b, node i and query head h: out = softmax(scale q.k_j) v_j over the visible keys j. The newest n
// positions of the request's len[b] are the n query tokens' own: all earlier keys are visible to every node, and among
// the last n node i sees those its mask row names (n = 1: itself).
//
// GB300 design (flash decoding on the 5th-generation tensor cores): the n nodes of the G = Hq / Hkv query heads that
// share a key/value head are one block of R = G n <= 128 query rows, so each cached row is read once per (request,
// key/value head) and feeds R rows of dot products. Only the device knows the lengths: every CTA (one per SM) scans
// them, and the 128-key blocks of all (request, key/value head) pairs, laid end to end with a unit more for each pair
// (its start and end cost about what a block does), are split evenly over the CTAs.
// A CTA's run inside one pair is a segment; a segment that covers its pair writes the output, the others leave
// (O, m, l) in the CTA's two partial slots (only the first and the last segment of a share can be cut), and the CTA
// that finishes a cut pair last joins its segments in slot order, so the result does not depend on who that is.
// Bound by memory: the key and value rows are the bytes. Measured, 32/8 heads, d = 128: one new token for 64 requests
// of 1 to 8191, pages of 16: 165 us, 6.5 TB/s, 96% of the copy rate (1.077 GB read from DRAM for 1.074 needed); three
// of 100001 to 131072: 205 us, 102%; 64 trees of 16 nodes over 130 to 4099: 103 us, 82% (pairs of 2 to 33 blocks:
// starts, ends and joins); one of 2049: 10 us, a chain of latencies. d = 64: the same 64 requests 91 us with pages of
// 64 (5.9 TB/s, 87%) and 122 with pages of 16, whose 16 copies of 2 KB a block take longer than their bytes; the three
// long ones 111 (6.4 TB/s, 94%); the trees 69 (4.1 TB/s, 61%: starts, ends and joins cost what they do at d = 128).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "attn_common.cuh"
#include "paged_share.cuh"

namespace dt {
namespace {

constexpr int kPaThreads = 384;   // warps 0, 1: values kept from the tensor cores; 2: load; 3: MMA; 4-11: softmax
constexpr int kPaMaxStages = 12;
constexpr int kPaCleans = 8;      // barriers of cleaned blocks: more than the ring can hold
constexpr uint32_t kPaBox = kPaKeys * 128;  // 128 rows x 64 elements: 16 KB

struct PaParams : PaWork {
  int stages;
  uint32_t q_box;                  // one 64-element box of Q: rows rounded up to 8, x 128 bytes
  const unsigned short* v_cache;   // [num_pages][Hkv][page_size][D], re-read only for values that are not finite
  float scale_log2;                // scale * log2(e)
};
struct PaMaps {
  CUtensorMap q;     // [B][n][Hq][D], box 64 x G x n x 1
  CUtensorMap k, v;  // [num_pages * Hkv][page_size][D] in 8-row atoms, boxes of min(page_size, 128) rows
};

__device__ __forceinline__ bool nonfinite_bf16x2(uint32_t w) {
  return (w & 0x7F800000u) == 0x7F800000u || (w & 0x7F80u) == 0x7F80u;
}

// Roles: warp 2 loads (its lanes look the pages up and issue one page's boxes each), warp 3 issues the MMAs, the
// softmax warps own 16 query rows each (row r = node G + head, tensor memory lane r; four neighbouring threads share
// two rows), warps 0 and 1 clean values. Per block: S = Q K^T (M = 128, N = 128) into one of two buffers in tensor
// memory, so that the next block's scores are computed during a block's softmax, also across segments; softmax in
// base 2 with the running maximum raised only past a headroom of 2^20 (O is rescaled then); the weights over their
// scores as bf16; O += P V with P from tensor memory and V as an MN-major operand, into one of two buffers by segment.
// Rows past R are padding and are left to whatever their rows of Q hold. A block takes the tensor cores 1024 cycles at
// D = 128 and the softmax about as long, where its 64 KB take 2800 at the memory's rate.
template <int D>
__global__ void __launch_bounds__(kPaThreads, 1) paged_attn_kernel(PaParams p, const __grid_constant__ PaMaps maps,
                                                                   WsHeader* hdr) {
  constexpr int kHalves = D / 64;
  constexpr uint32_t kEntry = kHalves * kPaBox;  // a ring entry: a block's keys or values
  constexpr uint32_t kAtoms = kHalves * 1024;    // eight of its rows
  constexpr uint32_t kColO = 256, kStepO = D;    // tensor memory: S at 0 and 128, O behind
  extern __shared__ float4 smem_f4[];
  unsigned char* sq =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_f4) + 1023) & ~uintptr_t(1023));
  const uint32_t q_bytes = kHalves * p.q_box;
  unsigned char* skv = sq + 2 * q_bytes;
  int* cum = reinterpret_cast<int*>(skv + p.stages * kEntry);  // [B + 1]
  int* lens = cum + p.B + 1;                                   // [B]
  __shared__ uint64_t kv_full[kPaMaxStages], kv_empty[kPaMaxStages], v_clean[kPaCleans];
  __shared__ uint64_t s_full[2], p_full[2], o_done[2], q_full[2], q_empty[2], o_free[2], s_meet;
  __shared__ uint32_t s_tmem;
  __shared__ unsigned s_kv_issued, s_kv_used, s_q_issued, s_q_used;  // copies issued and waited for (failure drain)
  __shared__ int s_warp[kPaThreads / 32];
  __shared__ int s_bad, s_joins;
  __shared__ PaJoin s_join[2];
  __shared__ unsigned long long s_mbits[kPaCleans][kPaNodes];  // bit c: the key of node c is visible to the node
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int live_warps = (p.R + 15) / 16;
  const unsigned stages = static_cast<unsigned>(p.stages);
  if (t == 0) {
    for (unsigned i = 0; i < stages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < kPaCleans; ++i) mbar_init(&v_clean[i], 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], live_warps);
      mbar_init(&o_done[i], 1);
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&o_free[i], live_warps);
    }
    mbar_init(&s_meet, live_warps);
    mbar_fence_init();
    s_kv_issued = s_kv_used = s_q_issued = s_q_used = 0u;
    s_bad = s_joins = 0;
  }
  if (warp == 3) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 2 && lane < 3)
    asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &maps.q : lane == 1 ? &maps.k : &maps.v) : "memory");
  at_launch_order();
  // the plan: block counts scanned over the requests; rows of requests without blocks are zero
  int carry = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPaThreads) {
    const int b = b0 + t;
    bool bad = false;
    const int len = b < p.B ? pa_length(p, b, &bad) : 0;
    if (bad && blockIdx.x == 0) record_error(hdr, DT_ERR_INVALID_ARG);
    int total;
    const int units = len > 0 ? (len + kPaKeys - 1) / kPaKeys + p.extra : 0;
    const int before = block_exclusive_scan<kPaThreads / 32>(units, &total, s_warp);
    if (b < p.B) {
      cum[b] = carry + before;
      lens[b] = len;
    }
    carry += total;
  }
  if (t == 0) cum[p.B] = carry;
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = s_tmem;
  const long long W = static_cast<long long>(carry) * p.Hkv;
  for (int b = blockIdx.x; b < p.B; b += p.grid)
    if (cum[b + 1] == cum[b]) {
      uint4* o = reinterpret_cast<uint4*>(p.out + static_cast<size_t>(b) * p.n * p.Hq * D);
      for (int i = t; i < p.n * p.Hq * (D / 8); i += kPaThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  bool ok = true;
  const int ctas = W < p.grid ? static_cast<int>(W) : p.grid;  // that take a share: a block each at least
  PaWalk w = pa_walk(p, cum, W, ctas);

  if (warp == 2) {  // TMA: the whole warp, one page's boxes a lane
    unsigned st = 0, par = 1u, e = 0;  // ring entry, the parity of its last release, entries so far
    const int box_rows = p.page_size < kPaKeys ? p.page_size : kPaKeys;
    const int per_block = kPaKeys / box_rows;  // pages a block spans (1 when a page holds whole blocks)
    for (int si = 0; ok; ++si) {
      const PaSeg sg = pa_next(p, cum, w);
      if (sg.nblk == 0) break;
      const unsigned qb = static_cast<unsigned>(si) & 1u;
      const int used = (lens[sg.b] + p.page_size - 1) / p.page_size;  // pages the request holds
      const int32_t* table = p.page_table + static_cast<size_t>(sg.b) * p.max_pages;
      // page ids, 32 at a time and one window ahead
      int win = static_cast<int>(static_cast<long long>(sg.j0) * kPaKeys / p.page_size) / 32;
      int cur = 32 * win + lane < used ? table[32 * win + lane] : 0;
      int nxt = 32 * (win + 1) + lane < used ? table[32 * (win + 1) + lane] : 0;
      if (si >= 2) ok = __all_sync(0xFFFFFFFFu, at_wait(&q_empty[qb], static_cast<unsigned>((si >> 1) - 1) & 1u));
      if (!ok) break;
      if (lane == 0) {
        unsigned char* qd = sq + qb * q_bytes;
        mbar_expect_tx(&q_full[qb], static_cast<uint32_t>(kHalves * 128 * p.R));
        for (int h = 0; h < kHalves; ++h)
          tma_load_4d(qd + h * p.q_box, &maps.q, 64 * h, sg.kvh * p.G, 0, sg.b, &q_full[qb]);
        s_q_issued = static_cast<unsigned>(si) + 1u;
      }
      for (int j = 0; j < sg.nblk && ok; ++j) {
        const int key = (sg.j0 + j) * kPaKeys, first = key / p.page_size, row = key % p.page_size;
        if (first / 32 != win) {
          ++win;
          cur = nxt;
          nxt = 32 * (win + 1) + lane < used ? table[32 * (win + 1) + lane] : 0;
        }
        const int pages = used - first < per_block ? used - first : per_block;
        int page = __shfl_sync(0xFFFFFFFFu, cur, (first + lane) & 31);
        if (lane < pages && (page < 0 || page >= p.num_pages)) {
          record_error(hdr, DT_ERR_INVALID_ARG);
          page = 0;
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {  // the keys, then the values
          if (ok && e >= stages) ok = __all_sync(0xFFFFFFFFu, at_wait(&kv_empty[st], par));
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(&kv_full[st], static_cast<uint32_t>(pages * box_rows * 128 * kHalves));
          __syncwarp();
          if (lane < pages) {
            tma_load_5d(skv + st * kEntry + lane * box_rows * (128 * kHalves), kv ? &maps.v : &maps.k, 0, 0, 0, row / 8,
                        page * p.Hkv + sg.kvh, &kv_full[st]);
          }
          ++e;
          if (lane == 0) s_kv_issued = e;
          if (++st == stages) {
            st = 0;
            par ^= 1u;
          }
        }
      }
    }
  } else if (warp == 3) {
    if (elect_one()) {  // MMA
      const uint32_t id_s = umma_idesc(kPaKeys, 128), id_o = umma_idesc(D, 128) | (1u << 16);  // O: V MN-major
      const uint64_t dk = umma_desc_sw128_strided(smem_u32(skv), kAtoms);
      const uint64_t dv = umma_desc_sw128_mn(smem_u32(skv), 1024u, kAtoms);
      auto wait = [&](uint64_t* bar, unsigned parity) {
        const bool done = at_wait(bar, parity);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        return done;
      };
      unsigned st = 0, par = 0, seen = 0;  // the ring entry that comes next, in order: K, V, K, V, ...
      auto take = [&](unsigned& at) {
        at = st;
        if (!wait(&kv_full[st], par)) return false;
        s_kv_used = ++seen;
        if (++st == stages) {
          st = 0;
          par ^= 1u;
        }
        return true;
      };
      // The scores run one block ahead of the outputs, through the same segments.
      PaWalk ws = w;
      PaSeg ss{};
      int js = 0, sis = -1;
      unsigned gs = 0;
      auto scores = [&]() {  // of the next block, if there is one
        if (js == ss.nblk) {
          ss = pa_next(p, cum, ws);
          js = 0;
          if (ss.nblk == 0) return true;
          ++sis;
          if (!wait(&q_full[sis & 1], static_cast<unsigned>(sis >> 1) & 1u)) return false;
          s_q_used = static_cast<unsigned>(sis) + 1u;
        }
        unsigned at;
        if (!take(at)) return false;
        const uint64_t q0 = umma_desc_sw128(smem_u32(sq + (sis & 1) * q_bytes)), k0 = dk + at * (kEntry >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_f16(tmem + (gs & 1u) * kPaKeys, q0 + (((kk >> 2) * p.q_box + (kk & 3) * 32u) >> 4),
                   k0 + (((kk >> 2) * 1024u + (kk & 3) * 32u) >> 4), id_s, kk > 0 ? 1u : 0u);
        umma_commit(&s_full[gs & 1u]);
        umma_commit(&kv_empty[at]);
        if (++js == ss.nblk) umma_commit(&q_empty[sis & 1]);
        ++gs;
        return true;
      };
      unsigned g = 0, cleans = 0;
      ok = scores();
      for (int si = 0; ok; ++si) {
        const PaSeg sg = pa_next(p, cum, w);
        if (sg.nblk == 0) break;
        const unsigned qb = static_cast<unsigned>(si) & 1u;
        const uint32_t to = tmem + kColO + kStepO * qb;
        const int common = pa_common(p, lens[sg.b]);
        for (int j = 0; j < sg.nblk && ok; ++j, ++g) {
          unsigned sv;
          ok = take(sv);
          // its buffer was freed by block g - 1's softmax (waited for below, one block ago)
          if (ok) ok = scores();
          if (ok && j == 0 && si >= 2) ok = wait(&o_free[qb], static_cast<unsigned>((si >> 1) - 1) & 1u);
          if (ok && (sg.j0 + j + 1) * kPaKeys > common) {
            ok = wait(&v_clean[cleans % kPaCleans], (cleans / kPaCleans) & 1u);
            ++cleans;
          }
          if (ok) ok = wait(&p_full[g & 1u], (g >> 1) & 1u);
          if (!ok) break;
          const uint64_t v0 = dv + sv * (kEntry >> 4);
#pragma unroll
          for (int kk = 0; kk < kPaKeys / 16; ++kk)
            umma_f16_ts(to, tmem + (g & 1u) * kPaKeys + 8u * kk, v0 + kk * (2u * kAtoms >> 4), id_o,
                        (j > 0 || kk > 0) ? 1u : 0u);
          umma_commit(&kv_empty[sv]);
          umma_commit(&o_done[g & 1u]);
        }
      }
    }
  } else if (warp < 2) {
    // A weight of zero does not hide a value that is not finite from the tensor cores (0 x inf is NaN). So rows past
    // the request's end (stale, or left in the ring by another block) are cleared, and what is not finite among the
    // nodes' values is cleared here and added to the rows that see it at the end: its weight there is positive, and
    // any positive multiple of it gives the same sum.
    unsigned g = 0, cleans = 0;
    for (int si = 0; ok; ++si) {
      const PaSeg sg = pa_next(p, cum, w);
      if (sg.nblk == 0) break;
      const int len = lens[sg.b], common = pa_common(p, len);
      for (int j = 0; j < sg.nblk && ok; ++j, ++g) {
        const int kbase = (sg.j0 + j) * kPaKeys;
        if (kbase + kPaKeys <= common) continue;
        const unsigned e = 2u * g + 1u, at = e % stages;
        ok = __all_sync(0xFFFFFFFFu, at_issued(&s_kv_issued, e));
        if (!ok) break;
        if (t < p.n) {  // the nodes' mask rows, for the softmax
          unsigned long long bits = t == 63 ? ~0ull : (2ull << t) - 1ull;
          if (p.mask) {
            const uint8_t* mr = p.mask + (static_cast<size_t>(sg.b) * p.n + t) * p.n;
            bits = 0ull;
#pragma unroll 8
            for (int c = 0; c < p.n; ++c) bits |= static_cast<unsigned long long>(mr[c] != 0) << c;
          }
          s_mbits[cleans % kPaCleans][t] = bits;
        }
        ok = __all_sync(0xFFFFFFFFu, at_wait(&kv_full[at], (e / stages) & 1u));
        if (!ok) break;
        unsigned char* sv = skv + at * kEntry;
        bool found = false;
        for (int c = t; c < kHalves * kPaKeys * 8; c += 64) {  // 16-byte pieces; eight a row
          const int key = kbase + c / (kAtoms / 16) * 8 + ((c >> 3) & 7);
          uint4* piece = reinterpret_cast<uint4*>(sv + 16 * c);
          if (key >= len) {
            *piece = make_uint4(0u, 0u, 0u, 0u);
          } else if (key >= common) {
            uint4 x = *piece;
            uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
            bool hit = false;
#pragma unroll
            for (int k2 = 0; k2 < 4; ++k2)
              if (nonfinite_bf16x2(xw[k2])) {
                if ((xw[k2] & 0x7F80u) == 0x7F80u) xw[k2] &= 0xFFFF0000u;
                if ((xw[k2] & 0x7F800000u) == 0x7F800000u) xw[k2] &= 0xFFFFu;
                hit = true;
              }
            if (hit) {
              *piece = x;
              found = true;
            }
          }
        }
        if (found) atomicMax(&s_bad, si + 1);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMA reads V through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_clean[cleans % kPaCleans]);
        ++cleans;
      }
    }
  } else if (32 * (warp & 3) + 16 * ((warp - 4) >> 2) < p.R) {  // softmax
    const int lane0 = 32 * (warp & 3) + 16 * ((warp - 4) >> 2);
    const uint32_t lanes = static_cast<uint32_t>(lane0) << 16;
    const int ra = lane0 + (lane >> 2), quad = lane & 3, col = 2 * quad;
    int node[2], head[2];
    bool live[2];
#pragma unroll
    for (int k2 = 0; k2 < 2; ++k2) {
      live[k2] = ra + 8 * k2 < p.R;
      node[k2] = live[k2] ? (ra + 8 * k2) / p.G : 0;
      head[k2] = live[k2] ? (ra + 8 * k2) % p.G : 0;
    }
    unsigned g = 0, meet = 0, cleans = 0;
    for (int si = 0; ok; ++si) {
      const PaSeg sg = pa_next(p, cum, w);
      if (sg.nblk == 0) break;
      const unsigned qb = static_cast<unsigned>(si) & 1u;
      const uint32_t to = tmem + lanes + kColO + kStepO * qb;
      const int len = lens[sg.b], pre = len - p.n, common = pa_common(p, len);
      const int last_key = (sg.j0 + sg.nblk) * kPaKeys;
      unsigned long long mbits[2] = {0ull, 0ull};  // bit c: the key of node c is visible to the row's node
      float nref[2] = {kAtNone, kAtNone}, l[2] = {0.f, 0.f};
      for (int j = 0; j < sg.nblk && ok; ++j, ++g) {
        const uint32_t ts = tmem + lanes + (g & 1u) * kPaKeys;
        ok = at_wait(&s_full[g & 1u], (g >> 1) & 1u) && ok;
        __syncwarp();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        float s[64];
        at_ld_s(ts, s);
        const int kbase = (sg.j0 + j) * kPaKeys;
        if (kbase + kPaKeys > common) {
          ok = at_wait(&v_clean[cleans % kPaCleans], (cleans / kPaCleans) & 1u) && ok;
          __syncwarp();
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2) {
            mbits[k2] = s_mbits[cleans % kPaCleans][node[k2]];
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // bit i: column 64 half + i, from the thread's first, is visible
              const int at = kbase + col + 64 * half;
              const unsigned long long bits = pa_visible(pre - at, len - at, mbits[k2]);
#pragma unroll
              for (int g8 = 0; g8 < 8; ++g8)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (!((bits >> (8 * g8 + e)) & 1ull)) s[32 * half + 4 * g8 + 2 * k2 + e] = -INFINITY;
            }
          }
          ++cleans;
        }
        float mx[2];
        at_max(s, p.scale_log2, mx);
        if (__any_sync(0xFFFFFFFFu, mx[0] + nref[0] > kAtMost || mx[1] + nref[1] > kAtMost)) {  // rare: rescale O
          float alpha[2];
          at_raise(mx, nref, l, alpha);
          if (j > 0) {
            ok = at_wait(&o_done[(g - 1u) & 1u], ((g - 1u) >> 1) & 1u) && ok;
            __syncwarp();
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll 1
            for (int h = 0; h < D / 32; ++h) {
              float o[16];
              at_ld_o(to + 32u * h, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= alpha[(e >> 1) & 1];
              at_st_o(to + 32u * h, o);
            }
          }
        }
        uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
        uint32_t pk[16];
        at_weights<0>(s, p.scale_log2, nref, ls, pk);
        at_st_p(ts, pk);
        at_weights<1>(s, p.scale_log2, nref, ls, pk);
        at_st_p(ts + 32u, pk);
        at_sums(ls, l);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[g & 1u]);
        ok = __all_sync(0xFFFFFFFFu, ok);
      }
      if (!ok) break;
      ok = __all_sync(0xFFFFFFFFu, at_wait(&o_done[(g - 1u) & 1u], ((g - 1u) >> 1) & 1u));
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      float o[D / 2];
      if constexpr (D == 128)
        at_ld_s(to, o);
      else
        at_ld_half(to, o);
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[qb]);
      const bool whole = sg.nblk == sg.nb;
      // (a later segment's mark counts too: that is only slower)
      const bool bad = *reinterpret_cast<volatile int*>(&s_bad) > si;
      if (bad) {  // rare: the nodes' values that are not finite, from global memory
        for (int c = 0; c < p.n; ++c) {
          const int key = pre + c;
          if (key < sg.j0 * kPaKeys || key >= last_key) continue;
          const int page = p.page_table[static_cast<size_t>(sg.b) * p.max_pages + key / p.page_size];
          if (page < 0 || page >= p.num_pages) continue;
          const unsigned short* vr =
              p.v_cache + ((static_cast<size_t>(page) * p.Hkv + sg.kvh) * p.page_size + key % p.page_size) * D + col;
#pragma unroll
          for (int e = 0; e < D / 2; ++e) {
            const uint32_t bits = static_cast<uint32_t>(vr[8 * (e >> 2) + (e & 1)]) << 16;
            if ((bits & 0x7F800000u) == 0x7F800000u && ((mbits[(e >> 1) & 1] >> c) & 1ull))
              o[e] += __uint_as_float(bits);
          }
        }
      }
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2) {
        l[k2] += __shfl_xor_sync(0xFFFFFFFFu, l[k2], 1);
        l[k2] += __shfl_xor_sync(0xFFFFFFFFu, l[k2], 2);
      }
      if (whole) {
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
          // no visible key at all: zero; visible keys of weight 0 alone: NaN
          const float inv = l[k2] == 0.f && common == 0 && mbits[k2] == 0ull ? 0.f : 1.f / l[k2];
          unsigned short* po =
              p.out + ((static_cast<size_t>(sg.b) * p.n + node[k2]) * p.Hq + sg.kvh * p.G + head[k2]) * D + 8 * quad;
#pragma unroll
          for (int h = 0; h < D / 32; ++h) {
            const uint4 x = at_row16(o + 16 * h, k2, inv, quad);
            if (live[k2]) *reinterpret_cast<uint4*>(po + 32 * h) = x;
          }
        }
        continue;
      }
      const size_t unit = 2 * static_cast<size_t>(blockIdx.x) + (sg.j0 == 0 ? 1 : 0);
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2) {
        if (!live[k2]) continue;
        const size_t row = unit * p.R + ra + 8 * k2;
#pragma unroll
        for (int g8 = 0; g8 < D / 8; ++g8)
          *reinterpret_cast<float2*>(p.part + row * D + 8 * g8 + col) =
              make_float2(o[4 * g8 + 2 * k2], o[4 * g8 + 2 * k2 + 1]);
        if (quad == 0)
          *reinterpret_cast<float2*>(p.ml + 2 * row) = make_float2(nref[k2] == kAtNone ? -INFINITY : -nref[k2], l[k2]);
      }
      // the pair's last segment to finish joins them all, once the CTA is through its share
      const int c0 = pa_owner(sg.pair0, W, ctas), c1 = pa_owner(sg.pair0 + sg.nb - 1, W, ctas);
      ok = pa_sync(&s_meet, meet, lane);  // the ticket's release covers what the other warps wrote before it
      if (!ok) break;
      if (t == 128) {
        // a pair's ticket is a byte: it counts to the grid at most, and goes back to zero before it is used again
        const int shift = 8 * (c0 & 3);
        const unsigned done = ((atom_add_acq_rel_gpu(hdr->tickets + c0 / 4, 1u << shift) >> shift) & 0xFFu) + 1u;
        if (done == static_cast<unsigned>(c1 - c0 + 1)) {
          atomicSub(hdr->tickets + c0 / 4, done << shift);  // ready for the next call
          s_join[s_joins++] = PaJoin{sg.b, sg.kvh, c0, c1};
        }
      }
    }
  }
  ok = __syncthreads_and(ok);
  if (!ok && t == 0) {
    record_error(hdr, DT_ERR_TIMEOUT);
    // copies issued but never waited for must land before the CTA leaves: wait for them too (bounded)
    for (unsigned e = s_kv_used; e < s_kv_issued; ++e) mbar_wait(&kv_full[e % stages], (e / stages) & 1u, kAtBudgetNs);
    for (unsigned q = s_q_used; q < s_q_issued; ++q) mbar_wait(&q_full[q & 1u], (q >> 1) & 1u, kAtBudgetNs);
  }
  if (ok) {
    // the ticket's thread acquired the others' partials; the barrier above passed them on
    for (int i = 0; i < s_joins; ++i) {
      PaSum* red = reinterpret_cast<PaSum*>(skv);  // the ring is empty by now
      if (p.R * (D / 4) <= kPaThreads) pa_join<D, 1, kPaThreads>(p, s_join[i], red);
      else pa_join<D, 6, kPaThreads>(p, s_join[i], red);
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 3) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

template <int D>
dt_status pa_launch(PaParams& p, const PaMaps& maps, WsHeader* hdr, cudaStream_t stream) {
  const uint32_t halves = D / 64, entry = halves * kPaBox;
  p.q_box = static_cast<uint32_t>((p.R + 7) / 8 * 8) * 128;
  const size_t fixed = 1024 + 2 * halves * p.q_box + align_up(sizeof(int) * (2 * p.B + 1), 16);
  const int fit = static_cast<int>((kPaSmemCap - fixed) / entry);
  p.stages = fit > kPaMaxStages ? kPaMaxStages : fit;
  const size_t smem = fixed + static_cast<size_t>(p.stages) * entry;
  const void* fn = reinterpret_cast<const void*>(paged_attn_kernel<D>);
  if (ensure_dynamic_smem(fn, kPaSmemCap) != cudaSuccess) return DT_ERR_CUDA;
  return at_launch(paged_attn_kernel<D>, p.grid, kPaThreads, smem, stream, p, maps, hdr);
}

}  // namespace
}  // namespace dt

extern "C" size_t dt_paged_attention_workspace_bytes(int B, int n, int Hq, int Hkv, int d) {
  if (B < 1 || n < 1 || Hq < 1 || Hkv < 1 || d < 1 || Hq % Hkv != 0) return 0;
  const long long R = static_cast<long long>(Hq / Hkv) * n;
  if (R > dt::kPaRows || d > 256) return 0;  // outside the envelope
  dt::DeviceInfo di{};
  if (dt::current_device_info(&di) != cudaSuccess) return 0;
  return dt::pa_plan(static_cast<int>(R), d, di.sms).bytes;
}

extern "C" dt_status dt_paged_attention(int B, int n, int Hq, int Hkv, int d, const void* q, const void* k_cache,
                                        const void* v_cache, dt_dtype dtype, int num_pages, int page_size,
                                        const int32_t* page_table, int max_pages, const int32_t* lens,
                                        const uint8_t* mask, float scale, void* out, void* workspace,
                                        size_t workspace_bytes, cudaStream_t stream) {
  using namespace dt;
  if (B < 0 || n < 1 || Hq < 1 || Hkv < 1 || d < 1 || Hq % Hkv != 0 || num_pages < 1 || page_size < 1 || max_pages < 1)
    return DT_ERR_INVALID_ARG;
  if (dtype != DT_F32 && dtype != DT_BF16) return DT_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale * 1.4426950408889634f)) return DT_ERR_INVALID_ARG;
  if (B == 0) return DT_OK;
  const void* ptrs[] = {q, k_cache, v_cache, out, workspace};
  for (const void* x : ptrs)
    if (!x || !aligned16(x)) return DT_ERR_INVALID_ARG;
  const void* ints[] = {page_table, lens};
  for (const void* x : ints)
    if (!x || (reinterpret_cast<uintptr_t>(x) & 3u)) return DT_ERR_INVALID_ARG;
  const int G = Hq / Hkv;
  if (dtype != DT_BF16 || (d != 64 && d != 128)) return DT_ERR_UNSUPPORTED;
  if (n > kPaNodes || static_cast<long long>(G) * n > kPaRows || B > DT_PAGED_MAX_BATCH) return DT_ERR_UNSUPPORTED;
  if (Hq > DT_MAX_HEADS) return DT_ERR_UNSUPPORTED;
  if (page_size < DT_MIN_PAGE || page_size > DT_MAX_PAGE || (page_size & (page_size - 1))) return DT_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_pages) * page_size > INT_MAX || static_cast<long long>(num_pages) * Hkv > INT_MAX)
    return DT_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size > DT_PAGED_MAX_TOKENS) return DT_ERR_UNSUPPORTED;
  DeviceInfo di{};
  if (current_device_info(&di) != cudaSuccess) return DT_ERR_CUDA;
  const PaPlan P = pa_plan(G * n, d, di.sms);
  if (workspace_bytes < P.bytes) return DT_ERR_INVALID_ARG;
  PaParams p{};
  p.B = B; p.n = n; p.Hq = Hq; p.Hkv = Hkv; p.G = G; p.R = G * n; p.grid = P.grid; p.extra = 1;
  p.page_size = page_size; p.num_pages = num_pages; p.max_pages = max_pages;
  p.v_cache = static_cast<const unsigned short*>(v_cache);
  p.page_table = page_table; p.lens = lens; p.mask = mask;
  p.scale_log2 = scale * 1.4426950408889634f;
  char* ws = static_cast<char*>(workspace);
  p.part = reinterpret_cast<float*>(ws + P.part);
  p.ml = reinterpret_cast<float*>(ws + P.ml);
  p.out = static_cast<unsigned short*>(out);
  PaMaps maps{};
  const uint64_t dd = static_cast<uint64_t>(d), hkv = static_cast<uint64_t>(Hkv), ps = static_cast<uint64_t>(page_size),
                 np = static_cast<uint64_t>(num_pages);
  const uint32_t box = page_size < kPaKeys ? static_cast<uint32_t>(page_size) : kPaKeys;
  if (!encode_bf16_4d(&maps.q, q, dd, static_cast<uint64_t>(Hq), static_cast<uint64_t>(n), static_cast<uint64_t>(B), 64,
                      static_cast<uint32_t>(G), static_cast<uint32_t>(n)) ||
      !encode_bf16_atoms(&maps.k, k_cache, dd, ps, hkv * np, box) ||
      !encode_bf16_atoms(&maps.v, v_cache, dd, ps, hkv * np, box))
    return DT_ERR_CUDA;
  WsHeader* hdr = reinterpret_cast<WsHeader*>(ws);
  return d == 64 ? pa_launch<64>(p, maps, hdr, stream) : pa_launch<128>(p, maps, hdr, stream);
}
