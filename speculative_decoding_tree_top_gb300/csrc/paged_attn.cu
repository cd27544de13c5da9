// dt_paged_attention — attention of each request's newest tokens over its paged key/value cache.
//
// For request b, node i and query head h: out = softmax(scale q.k_j) v_j over the visible keys j. The newest n
// positions of the request's len[b] are the n query tokens' own: all earlier keys are visible to every node, and among
// the last n node i sees those its mask row names (n = 1: itself).
//
// GB300 design (flash decoding on the 5th-generation tensor cores): the n nodes of the G = Hq / Hkv query heads that
// share a key/value head are one block of R = G n <= 128 query rows, so each cached row is read once per (request,
// key/value head) and feeds R rows of dot products. Only the device knows the lengths: every CTA (one per SM) scans
// them, and the 64-key blocks of all (request, key/value head) pairs, laid end to end, are split evenly over the CTAs.
// A CTA's run inside one pair is a segment; a segment that covers its pair writes the output, the others leave
// (O, m, l) in the CTA's two partial slots (only the first and the last segment of a share can be cut), and the CTA
// that finishes a cut pair last joins its segments in slot order, so the result does not depend on who that is.
// Bound by memory: the key and value rows are the bytes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "dt_internal.cuh"
#include "umma.cuh"

namespace dt {
namespace {

constexpr int kPaRows = 128;      // query rows per pair: G n at most
constexpr int kPaNodes = 64;      // n at most (a node's mask row is one 64-bit word)
constexpr int kPaKeys = 64;       // keys per block
constexpr int kPaThreads = 256;
constexpr int kPaMaxStages = 10;
constexpr float kPaLazy = 8.f;    // log2 headroom before the running maximum is raised
constexpr uint64_t kPaBudgetNs = 4000000000ull;
constexpr uint32_t kPaBox = kPaKeys * 128;  // 64 rows x 64 elements: 8 KB
constexpr size_t kPaSmemCap = 232448 - 1024;  // opt-in shared memory of a CTA, less the static part

struct PaParams {
  int B, n, Hq, Hkv, G, R, grid, stages;
  int page_size, num_pages, max_pages;
  uint32_t q_box, p_bytes;         // one 64-element box of Q, one P buffer: rows rounded up to 64 or 128, x 128 bytes
  const unsigned short* v_cache;   // [num_pages][Hkv][page_size][D], re-read only for values that are not finite
  const int32_t* page_table;       // [B][max_pages]
  const int32_t* lens;             // [B]
  const uint8_t* mask;             // [B][n][n] or null: causal among the n
  float scale_log2;                // scale * log2(e)
  float* part;                     // [grid][2][R][D] unnormalised outputs of cut segments
  float* ml;                       // [grid][2][R][2] running maximum (base 2) and sum
  unsigned* tickets;               // [grid] by a cut pair's first CTA: segments finished; zero between calls
  unsigned short* out;             // [B][n][Hq][D] bf16
};
struct PaMaps {
  CUtensorMap q;     // [B][n][Hq][D], box 64 x G x n x 1
  CUtensorMap k, v;  // [num_pages][Hkv][page_size][D], box 64 x min(page_size, 64) x 1 x 1
};

__device__ __forceinline__ float pa_exp2(float x) {  // relative error about 2^-22, results below 2^-126 flushed
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pa_pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void pa_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void pa_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ bool nonfinite_bf16x2(uint32_t w) {
  return (w & 0x7F800000u) == 0x7F800000u || (w & 0x7F80u) == 0x7F80u;
}

// The softmax warps meet (a barrier whose wait is bounded); `count` is the meetings so far, the same in every warp.
__device__ __forceinline__ bool pa_sync(uint64_t* bar, unsigned& count, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, count++ & 1u, kPaBudgetNs));
}

// The lengths' plan. cum[b] = 64-key blocks of one head of requests before b; a request whose length is not in
// [n, max_pages * page_size] has none (0 and below: an unused row of the batch; otherwise an error).
__device__ __forceinline__ int pa_length(const PaParams& p, int b, bool* bad) {
  const int len = p.lens[b];
  if (len <= 0) return 0;
  if (len < p.n || len > static_cast<long long>(p.max_pages) * p.page_size) {
    *bad = true;
    return 0;
  }
  return len;
}
__device__ __forceinline__ long long pa_share(long long W, int grid, int c) { return W * c / grid; }
__device__ __forceinline__ int pa_owner(long long x, long long W, int grid) {
  return static_cast<int>(((x + 1) * grid - 1) / W);
}
struct PaSeg {
  int b, kvh, nb, j0, nblk;
  long long pair0;  // the pair's first block in the flattened order
  bool first;       // the CTA's first segment
};
struct PaWalk {  // a CTA's segments, in order
  int b;
  long long x0, x, x1;
};
__device__ __forceinline__ PaWalk pa_walk(const PaParams& p, const int* cum, long long W, int ctas) {
  PaWalk w{0, 0, 0, 0};
  if (static_cast<int>(blockIdx.x) >= ctas) return w;
  w.x0 = w.x = pa_share(W, ctas, blockIdx.x);
  w.x1 = pa_share(W, ctas, blockIdx.x + 1);
  int lo = 0, hi = p.B - 1;  // the last request that starts at or before x0
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<long long>(cum[mid]) * p.Hkv <= w.x0) lo = mid;
    else hi = mid - 1;
  }
  w.b = lo;
  return w;
}
__device__ __forceinline__ PaSeg pa_next(const PaParams& p, const int* cum, PaWalk& w) {  // call while w.x < w.x1
  while (static_cast<long long>(cum[w.b + 1]) * p.Hkv <= w.x) ++w.b;
  PaSeg s;
  s.b = w.b;
  s.nb = cum[w.b + 1] - cum[w.b];
  const long long rel = w.x - static_cast<long long>(cum[w.b]) * p.Hkv;
  s.kvh = static_cast<int>(rel / s.nb);
  s.j0 = static_cast<int>(rel - static_cast<long long>(s.kvh) * s.nb);
  s.pair0 = w.x - s.j0;
  const long long left = w.x1 - w.x;
  s.nblk = left < s.nb - s.j0 ? static_cast<int>(left) : s.nb - s.j0;
  s.first = w.x == w.x0;
  w.x += s.nblk;
  return s;
}

// A cut pair's segments: CTA c0's in slot `first`, those of c0 + 1 .. c1 in their slot 0.
struct PaJoin {
  int b, kvh, c0, c1, first;
};
// Joins them, a warp per query row: the lanes read 32 segments' (m, l) at a time, then each segment's row of O, D / 32
// columns a lane, with several segments' loads in flight.
template <int D>
__device__ __forceinline__ void pa_join(const PaParams& p, const PaJoin& jn, int warp, int lane) {
  constexpr int kCols = D / 32;
  const int nseg = jn.c1 - jn.c0 + 1;
  auto unit = [&](int i) { return 2 * static_cast<size_t>(jn.c0 + i) + (i == 0 ? jn.first : 0); };
  for (int r = warp; r < p.R; r += kPaThreads / 32) {
    float mx = -INFINITY;
    for (int i = lane; i < nseg; i += 32) mx = fmaxf(mx, __ldcg(p.ml + (unit(i) * p.R + r) * 2));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    const float mref = mx == -INFINITY ? 0.f : mx;
    float den = 0.f, num[kCols];
#pragma unroll
    for (int e = 0; e < kCols; ++e) num[e] = 0.f;
    for (int i0 = 0; i0 < nseg; i0 += 32) {
      float wgt = 0.f;
      if (i0 + lane < nseg) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.ml + (unit(i0 + lane) * p.R + r) * 2));
        wgt = exp2f(ml.x - mref);  // a segment without visible keys: 2^-inf = 0
        den += wgt * ml.y;
      }
      const int here = min(32, nseg - i0);
#pragma unroll 8
      for (int i = 0; i < here; ++i) {
        const float* src = p.part + (unit(i0 + i) * p.R + r) * D + kCols * lane;
        const float wi = __shfl_sync(0xFFFFFFFFu, wgt, i);
        if constexpr (kCols == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
          num[0] += wi * x.x;
          num[1] += wi * x.y;
          num[2] += wi * x.z;
          num[3] += wi * x.w;
        } else {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
          num[0] += wi * x.x;
          num[1] += wi * x.y;
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xFFFFFFFFu, den, o);
    const int node = r / p.G;
    bool none = p.mask && p.lens[jn.b] == p.n;  // no prefix: perhaps no visible key at all
    if (none)
      for (int c = 0; c < p.n; ++c) none = none && p.mask[(static_cast<size_t>(jn.b) * p.n + node) * p.n + c] == 0;
    const float inv = den == 0.f && none ? 0.f : 1.f / den;
    unsigned short* o =
        p.out + ((static_cast<size_t>(jn.b) * p.n + node) * p.Hq + jn.kvh * p.G + r % p.G) * D + kCols * lane;
    if constexpr (kCols == 4)
      *reinterpret_cast<uint2*>(o) = make_uint2(pa_pack(num[0] * inv, num[1] * inv), pa_pack(num[2] * inv, num[3] * inv));
    else
      *reinterpret_cast<uint32_t*>(o) = pa_pack(num[0] * inv, num[1] * inv);
  }
}

// Roles: warp 2 loads (its lanes look the pages up and issue one page's boxes each), warp 3 issues the MMAs, warps
// 4 to 7 run the softmax, thread r owning query row r = node G + head (TMEM lane r).
// Per block: S = Q K^T (M = 128, N = 64) into one of two TMEM buffers; softmax in base 2 with the running maximum
// raised only past a headroom of 2^8 (O is rescaled then), P rounded to bf16 into shared memory; O += P V with V as an
// MN-major operand. Rows past R are padding and are left to whatever their rows of Q and P hold.
template <int D>
__global__ void __launch_bounds__(kPaThreads, 1) paged_attn_rows(PaParams p, const __grid_constant__ PaMaps maps,
                                                                 WsHeader* hdr) {
  constexpr int kHalves = D / 64;
  constexpr uint32_t kStage = 2 * kHalves * kPaBox;  // K boxes, then V boxes
  extern __shared__ float4 smem_f4[];
  unsigned char* sq =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_f4) + 1023) & ~uintptr_t(1023));
  const uint32_t q_bytes = kHalves * p.q_box;
  unsigned char* sp = sq + 2 * q_bytes;
  unsigned char* skv = sp + 2 * p.p_bytes;
  int* cum = reinterpret_cast<int*>(skv + p.stages * kStage);  // [B + 1]
  __shared__ uint64_t kv_full[kPaMaxStages], kv_empty[kPaMaxStages], s_full[2], p_full[2], o_done[2];
  __shared__ uint64_t q_full[2], q_empty[2], o_free[2], s_meet;
  __shared__ uint32_t s_tmem;
  __shared__ unsigned s_kv_issued, s_kv_used, s_q_issued, s_q_used;
  __shared__ int s_warp[kPaThreads / 32];
  __shared__ int s_bad, s_joins;
  __shared__ PaJoin s_join[2];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int live_warps = (p.R + 31) / 32;
  if (t == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
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
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // the plan: block counts scanned over the requests; rows of requests without blocks are zero
  int carry = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPaThreads) {
    const int b = b0 + t;
    bool bad = false;
    const int len = b < p.B ? pa_length(p, b, &bad) : 0;
    if (bad && blockIdx.x == 0) record_error(hdr, DT_ERR_INVALID_ARG);
    int total;
    const int before = block_exclusive_scan<kPaThreads / 32>((len + kPaKeys - 1) / kPaKeys, &total, s_warp);
    if (b < p.B) cum[b] = carry + before;
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

  if (warp == 2) {  // TMA producer: the whole warp, one page's boxes a lane
    unsigned st = 0, use = 0, g = 0;
    const int box_rows = p.page_size < kPaKeys ? p.page_size : kPaKeys;
    const int per_block = kPaKeys / box_rows;  // pages a block spans (1 when a page holds whole blocks)
    for (int si = 0; w.x < w.x1 && ok; ++si) {
      const PaSeg sg = pa_next(p, cum, w);
      const unsigned qb = static_cast<unsigned>(si) & 1u;
      if (si >= 2) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&q_empty[qb], static_cast<unsigned>((si >> 1) - 1) & 1u, kPaBudgetNs));
      if (!ok) break;
      if (lane == 0) {
        unsigned char* qd = sq + qb * q_bytes;
        mbar_expect_tx(&q_full[qb], static_cast<uint32_t>(kHalves * 128 * p.R));
        for (int h = 0; h < kHalves; ++h)
          tma_load_4d(qd + h * p.q_box, &maps.q, 64 * h, sg.kvh * p.G, 0, sg.b, &q_full[qb]);
        s_q_issued = static_cast<unsigned>(si) + 1u;
      }
      const int used = (p.lens[sg.b] + p.page_size - 1) / p.page_size;  // pages the request holds
      const int32_t* table = p.page_table + static_cast<size_t>(sg.b) * p.max_pages;
      // page ids, 32 at a time and one window ahead
      int win = static_cast<int>(static_cast<long long>(sg.j0) * kPaKeys / p.page_size) / 32;
      int cur = 32 * win + lane < used ? table[32 * win + lane] : 0;
      int nxt = 32 * (win + 1) + lane < used ? table[32 * (win + 1) + lane] : 0;
      for (int j = 0; j < sg.nblk; ++j, ++g) {
        if (use > 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&kv_empty[st], (use - 1) & 1u, kPaBudgetNs));
        if (!ok) break;
        const int key = (sg.j0 + j) * kPaKeys, first = key / p.page_size, row = key % p.page_size;
        if (first / 32 != win) {
          ++win;
          cur = nxt;
          nxt = 32 * (win + 1) + lane < used ? table[32 * (win + 1) + lane] : 0;
        }
        const int pages = used - first < per_block ? used - first : per_block;
        if (lane == 0) mbar_expect_tx(&kv_full[st], static_cast<uint32_t>(pages * box_rows * 128 * 2 * kHalves));
        int page = __shfl_sync(0xFFFFFFFFu, cur, (first + lane) & 31);
        if (lane < pages) {
          if (page < 0 || page >= p.num_pages) {
            record_error(hdr, DT_ERR_INVALID_ARG);
            page = 0;
          }
          unsigned char* d = skv + st * kStage + lane * box_rows * 128;
          for (int h = 0; h < kHalves; ++h) {
            tma_load_4d(d + h * kPaBox, &maps.k, 64 * h, row, sg.kvh, page, &kv_full[st]);
            tma_load_4d(d + (kHalves + h) * kPaBox, &maps.v, 64 * h, row, sg.kvh, page, &kv_full[st]);
          }
        }
        if (lane == 0) s_kv_issued = g + 1u;
        if (++st == static_cast<unsigned>(p.stages)) {
          st = 0;
          ++use;
        }
      }
    }
  } else if (warp == 3 && lane == 0) {  // MMA issuer
    const uint32_t id_s = umma_idesc(kPaKeys, 128), id_o = umma_idesc(D, 128) | (1u << 16);  // O: V MN-major
    unsigned g = 0, st = 0;           // the block whose P V comes next, and its stage
    unsigned st_s = 0, par_s = 0;     // the same of the block whose S comes next
    unsigned gs = 0;
    for (int si = 0; w.x < w.x1 && ok; ++si) {
      const PaSeg sg = pa_next(p, cum, w);
      const unsigned qb = static_cast<unsigned>(si) & 1u;
      const uint32_t aq = smem_u32(sq + qb * q_bytes), to = tmem + 128u + 128u * qb;
      ok = mbar_wait(&q_full[qb], static_cast<unsigned>(si >> 1) & 1u, kPaBudgetNs);
      if (ok) s_q_used = static_cast<unsigned>(si) + 1u;
      if (ok && si >= 2) ok = mbar_wait(&o_free[qb], static_cast<unsigned>((si >> 1) - 1) & 1u, kPaBudgetNs);
      if (!ok) break;
      auto issue_s = [&]() {
        if (!mbar_wait(&kv_full[st_s], par_s, kPaBudgetNs)) return false;
        s_kv_used = gs + 1u;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t bk = smem_u32(skv + st_s * kStage);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_f16(tmem + (gs & 1u) * kPaKeys, umma_desc_sw128(aq + (kk >> 2) * p.q_box + (kk & 3) * 32u),
                   umma_desc_sw128(bk + (kk >> 2) * kPaBox + (kk & 3) * 32u), id_s, kk > 0 ? 1u : 0u);
        umma_commit(&s_full[gs & 1u]);
        ++gs;
        if (++st_s == static_cast<unsigned>(p.stages)) {
          st_s = 0;
          par_s ^= 1u;
        }
        return true;
      };
      ok = issue_s();
      if (ok && sg.nblk == 1) umma_commit(&q_empty[qb]);
      for (int j = 0; j < sg.nblk && ok; ++j, ++g) {
        if (j + 1 < sg.nblk) {  // its S buffer was freed by block g - 1's softmax (waited for below, one block ago)
          ok = issue_s();
          if (ok && j + 2 == sg.nblk) umma_commit(&q_empty[qb]);
        }
        if (ok) ok = mbar_wait(&p_full[g & 1u], (g >> 1) & 1u, kPaBudgetNs);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t ap = smem_u32(sp + (g & 1u) * p.p_bytes), bv = smem_u32(skv + st * kStage + kHalves * kPaBox);
#pragma unroll
        for (int kk = 0; kk < kPaKeys / 16; ++kk)
          umma_f16(to, umma_desc_sw128(ap + 32u * kk), umma_desc_sw128_mn(bv + 2048u * kk, kPaBox, 1024u), id_o,
                   (j > 0 || kk > 0) ? 1u : 0u);
        umma_commit(&kv_empty[st]);
        umma_commit(&o_done[g & 1u]);
        if (++st == static_cast<unsigned>(p.stages)) st = 0;
      }
    }
  } else if (warp >= 4 && warp - 4 < live_warps) {  // softmax
    const int r = t - 128;
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp - 4)) << 16);
    const bool live = r < p.R;
    const int node = live ? r / p.G : 0, gi = live ? r % p.G : 0;
    const int workers = 32 * live_warps;
    unsigned g = 0, st = 0, par = 0, meet = 0;
    for (int si = 0; w.x < w.x1 && ok; ++si) {
      const PaSeg sg = pa_next(p, cum, w);
      const unsigned qb = static_cast<unsigned>(si) & 1u;
      const uint32_t to = tl + 128u + 128u * qb;
      const int len = p.lens[sg.b], pre = len - p.n;  // keys below pre are visible to every node
      const int last_key = (sg.j0 + sg.nblk) * kPaKeys;
      unsigned long long mbits = 0;  // bit c: the key of node c is visible to this row's node
      if (live && (last_key > pre || p.n == 1)) {
        if (!p.mask) {
          mbits = node == 63 ? ~0ull : (2ull << node) - 1ull;
        } else {
          const uint8_t* mr = p.mask + (static_cast<size_t>(sg.b) * p.n + node) * p.n;
          for (int c = 0; c < p.n; ++c) mbits |= static_cast<unsigned long long>(mr[c] != 0) << c;
        }
      }
      float m = -INFINITY, l = 0.f;
      bool bad_v = false;  // a value of the segment's nodes is not finite
      for (int j = 0; j < sg.nblk && ok; ++j, ++g) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s_full[g & 1u], (g >> 1) & 1u, kPaBudgetNs));
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const int kbase = (sg.j0 + j) * kPaKeys;
        // A weight of zero does not hide a value that is not finite from the tensor cores (0 x inf is NaN). So rows
        // past the request's end (stale, or left in the ring by another block) are cleared, and what is not finite
        // among the nodes' values is cleared here and added to the rows that see it at the end: its weight there is
        // positive, and any positive multiple of it gives the same sum.
        const bool tail = kbase + kPaKeys > len, nodes = p.n > 1 && kbase + kPaKeys > pre;
        if (tail || nodes) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(&kv_full[st], par, kPaBudgetNs));  // done: S is complete
          if (!ok) break;
          unsigned char* sv = skv + st * kStage + kHalves * kPaBox;
          bool found = false;
          for (int i = t - 128; i < kPaKeys * kHalves; i += workers) {
            const int c = i % kPaKeys, key = kbase + c;
            uint4* row = reinterpret_cast<uint4*>(sv + (i / kPaKeys) * kPaBox + c * 128);
            if (key >= len) {
#pragma unroll
              for (int e = 0; e < 8; ++e) row[e] = make_uint4(0u, 0u, 0u, 0u);
            } else if (nodes && key >= pre) {
              for (int e = 0; e < 8; ++e) {
                uint4 x = row[e];
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
                  row[e] = x;
                  found = true;
                }
              }
            }
          }
          if (nodes) {
            if (found) s_bad = si + 1;
            ok = pa_sync(&s_meet, meet, lane);
            if (!ok) break;
            bad_v = bad_v || *reinterpret_cast<volatile int*>(&s_bad) > si;  // a later segment's counts too: only slower
          }
        }
        uint32_t sv[4][16];
#pragma unroll
        for (int h = 0; h < 4; ++h) pa_ld16(tl + (g & 1u) * kPaKeys + 16u * h, sv[h]);
        const int rel = pre - kbase, lim = len - kbase;
        unsigned long long visb = 0;
        if (live) {
          const unsigned long long pbits = rel >= 64 ? ~0ull : rel <= 0 ? 0ull : (1ull << rel) - 1ull;
          unsigned long long tbits = 0;
          if (rel < 64) tbits = rel >= 0 ? mbits << rel : rel > -64 ? mbits >> (-rel) : 0ull;
          const unsigned long long lbits = lim >= 64 ? ~0ull : lim <= 0 ? 0ull : (1ull << lim) - 1ull;
          visb = (pbits | tbits) & lbits;
        }
        float s[64];
        float bmax = -INFINITY;
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          s[c] = (visb >> c) & 1ull ? __uint_as_float(sv[c >> 4][c & 15]) * p.scale_log2 : -INFINITY;
          bmax = fmaxf(bmax, s[c]);
        }
        const bool raise = bmax > m + kPaLazy || (m == -INFINITY && bmax > -INFINITY);
        const bool rescale_o = raise && m > -INFINITY;
        const float mn = raise ? bmax : m;
        const float alpha = rescale_o ? pa_exp2(m - mn) : 1.f;
        m = mn;
        const float mref = m == -INFINITY ? 0.f : m;  // nothing visible yet: every weight is 2^-inf = 0
        float ls = 0.f;
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float a = pa_exp2(s[c] - mref), bb = pa_exp2(s[c + 1] - mref);
          ls += a + bb;
          pk[c >> 1] = pa_pack(a, bb);
        }
        l = l * alpha + ls;
        // P's buffer was last read by the O MMA of block g - 2; a rescale needs block g - 1's O MMA complete (of this
        // segment: m was finite). Commits complete in order.
        const bool any_rescale = __any_sync(0xFFFFFFFFu, rescale_o);
        if (g >= 2 || any_rescale) {
          const unsigned gw = any_rescale ? g - 1 : g - 2;
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(&o_done[gw & 1u], (gw >> 1) & 1u, kPaBudgetNs));
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        }
        if (any_rescale) {
#pragma unroll
          for (int h = 0; h < D / 16; ++h) {
            uint32_t ov[16];
            pa_ld16(to + 16u * h, ov);
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            pa_st16(to + 16u * h, ov);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        unsigned char* prow = sp + (g & 1u) * p.p_bytes + r * 128;
#pragma unroll
        for (int cc = 0; cc < 8; ++cc)
          *reinterpret_cast<uint4*>(prow + ((cc ^ (r & 7)) << 4)) =
              make_uint4(pk[4 * cc], pk[4 * cc + 1], pk[4 * cc + 2], pk[4 * cc + 3]);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMA reads P and V through the async proxy
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[g & 1u]);
        if (++st == static_cast<unsigned>(p.stages)) {
          st = 0;
          par ^= 1u;
        }
      }
      if (!ok) break;
      const unsigned gl = g - 1;
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&o_done[gl & 1u], (gl >> 1) & 1u, kPaBudgetNs));
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const bool whole = sg.nblk == sg.nb;
      const bool empty = pre == 0 && mbits == 0;  // (only read where l == 0)
      const size_t unit = 2 * static_cast<size_t>(blockIdx.x) + (sg.first ? 0 : 1);
      unsigned short* po = p.out + ((static_cast<size_t>(sg.b) * p.n + node) * p.Hq + sg.kvh * p.G + gi) * D;
      float* pp = p.part + (unit * p.R + r) * D;
      const float inv = l == 0.f && empty ? 0.f : 1.f / l;
#pragma unroll
      for (int h = 0; h < D / 16; ++h) {
        uint32_t ov[16];
        pa_ld16(to + 16u * h, ov);
        if (!live) continue;
        if (bad_v) {  // rare: the nodes' values that are not finite, from global memory
          for (int c = 0; c < p.n; ++c) {
            const int key = pre + c;
            if (!((mbits >> c) & 1ull) || key < sg.j0 * kPaKeys || key >= last_key) continue;
            const int page = p.page_table[static_cast<size_t>(sg.b) * p.max_pages + key / p.page_size];
            if (page < 0 || page >= p.num_pages) continue;
            const unsigned short* vr =
                p.v_cache + ((static_cast<size_t>(page) * p.Hkv + sg.kvh) * p.page_size + key % p.page_size) * D + 16 * h;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint32_t bits = static_cast<uint32_t>(vr[e]) << 16;
              if ((bits & 0x7F800000u) == 0x7F800000u)
                ov[e] = __float_as_uint(__uint_as_float(ov[e]) + __uint_as_float(bits));
            }
          }
        }
        if (whole) {
          uint32_t w8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            w8[e] = pa_pack(__uint_as_float(ov[2 * e]) * inv, __uint_as_float(ov[2 * e + 1]) * inv);
          *reinterpret_cast<uint4*>(po + 16 * h) = make_uint4(w8[0], w8[1], w8[2], w8[3]);
          *reinterpret_cast<uint4*>(po + 16 * h + 8) = make_uint4(w8[4], w8[5], w8[6], w8[7]);
        } else {
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4*>(pp + 16 * h + e) =
                make_float4(__uint_as_float(ov[e]), __uint_as_float(ov[e + 1]), __uint_as_float(ov[e + 2]),
                            __uint_as_float(ov[e + 3]));
        }
      }
      if (live && !whole) *reinterpret_cast<float2*>(p.ml + (unit * p.R + r) * 2) = make_float2(m, l);
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[qb]);
      if (whole) continue;
      // the pair's last segment to finish joins them all, once the CTA is through its share
      const int c0 = pa_owner(sg.pair0, W, ctas), c1 = pa_owner(sg.pair0 + sg.nb - 1, W, ctas);
      __threadfence();
      ok = pa_sync(&s_meet, meet, lane);
      if (!ok) break;
      if (t == 128) {
        const unsigned done = atom_add_acq_rel_gpu(p.tickets + c0, 1u) + 1u;
        if (done == static_cast<unsigned>(c1 - c0 + 1)) {
          p.tickets[c0] = 0u;  // ready for the next call
          s_join[s_joins++] = PaJoin{sg.b, sg.kvh, c0, c1, pa_share(W, ctas, c0) == sg.pair0 ? 0 : 1};
        }
      }
    }
  }
  ok = __syncthreads_and(ok);
  if (!ok && t == 0) {
    record_error(hdr, DT_ERR_TIMEOUT);
    // copies issued but never waited for must land before the CTA leaves: wait for them too (bounded)
    const unsigned ns = static_cast<unsigned>(p.stages);
    for (unsigned g = s_kv_used; g < s_kv_issued; ++g) mbar_wait(&kv_full[g % ns], (g / ns) & 1u, kPaBudgetNs);
    for (unsigned q = s_q_used; q < s_q_issued; ++q) mbar_wait(&q_full[q & 1u], (q >> 1) & 1u, kPaBudgetNs);
  }
  if (ok) {
    __threadfence();  // the ticket's thread acquired the others' partials; the barrier above passed them on
    for (int i = 0; i < s_joins; ++i) pa_join<D>(p, s_join[i], warp, lane);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

struct PaPlan {
  int grid;
  size_t tickets, part, ml, bytes;
};
inline PaPlan pa_plan(int R, int d, int sms) {
  PaPlan P{};
  P.grid = sms;
  P.tickets = align_up(sizeof(WsHeader));
  P.part = align_up(P.tickets + sizeof(unsigned) * P.grid);
  P.ml = align_up(P.part + sizeof(float) * 2 * P.grid * static_cast<size_t>(R) * d);
  P.bytes = align_up(P.ml + sizeof(float) * 2 * 2 * P.grid * static_cast<size_t>(R));
  return P;
}

template <int D>
dt_status pa_launch(PaParams& p, const PaMaps& maps, WsHeader* hdr, cudaStream_t stream) {
  const uint32_t rows = p.R <= 64 ? 64 : 128, halves = D / 64, stage = 2 * halves * kPaBox;
  p.q_box = rows * 128;
  p.p_bytes = rows * 128;
  const size_t fixed = 1024 + 2 * halves * p.q_box + 2 * p.p_bytes + align_up(sizeof(int) * (p.B + 1), 16);
  int stages = static_cast<int>((kPaSmemCap - fixed) / stage);
  p.stages = stages > kPaMaxStages ? kPaMaxStages : stages;
  const size_t smem = fixed + static_cast<size_t>(p.stages) * stage;
  const void* fn = reinterpret_cast<const void*>(paged_attn_rows<D>);
  if (ensure_dynamic_smem(fn, kPaSmemCap) != cudaSuccess) return DT_ERR_CUDA;
  paged_attn_rows<D><<<static_cast<unsigned>(p.grid), kPaThreads, smem, stream>>>(p, maps, hdr);
  return cuda_status(cudaGetLastError());
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
  if (!(scale > 0.f) || !std::isfinite(scale)) return DT_ERR_INVALID_ARG;
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
  if (static_cast<long long>(num_pages) * page_size > INT_MAX) return DT_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size > DT_PAGED_MAX_TOKENS) return DT_ERR_UNSUPPORTED;
  DeviceInfo di{};
  if (current_device_info(&di) != cudaSuccess) return DT_ERR_CUDA;
  const PaPlan P = pa_plan(G * n, d, di.sms);
  if (workspace_bytes < P.bytes) return DT_ERR_INVALID_ARG;
  PaParams p{};
  p.B = B; p.n = n; p.Hq = Hq; p.Hkv = Hkv; p.G = G; p.R = G * n; p.grid = P.grid;
  p.page_size = page_size; p.num_pages = num_pages; p.max_pages = max_pages;
  p.v_cache = static_cast<const unsigned short*>(v_cache);
  p.page_table = page_table; p.lens = lens; p.mask = mask;
  p.scale_log2 = scale * 1.4426950408889634f;
  char* ws = static_cast<char*>(workspace);
  p.tickets = reinterpret_cast<unsigned*>(ws + P.tickets);
  p.part = reinterpret_cast<float*>(ws + P.part);
  p.ml = reinterpret_cast<float*>(ws + P.ml);
  p.out = static_cast<unsigned short*>(out);
  PaMaps maps{};
  const uint64_t dd = static_cast<uint64_t>(d), hkv = static_cast<uint64_t>(Hkv), ps = static_cast<uint64_t>(page_size),
                 np = static_cast<uint64_t>(num_pages);
  const uint32_t box = page_size < kPaKeys ? static_cast<uint32_t>(page_size) : kPaKeys;
  if (!encode_bf16_4d(&maps.q, q, dd, static_cast<uint64_t>(Hq), static_cast<uint64_t>(n), static_cast<uint64_t>(B), 64,
                      static_cast<uint32_t>(G), static_cast<uint32_t>(n)) ||
      !encode_bf16_4d(&maps.k, k_cache, dd, ps, hkv, np, 64, box, 1) ||
      !encode_bf16_4d(&maps.v, v_cache, dd, ps, hkv, np, 64, box, 1))
    return DT_ERR_CUDA;
  WsHeader* hdr = reinterpret_cast<WsHeader*>(ws);
  return d == 64 ? pa_launch<64>(p, maps, hdr, stream) : pa_launch<128>(p, maps, hdr, stream);
}
