// How the attention kernels over a paged cache share their work among the CTAs, and how cut pairs are joined.
//
// The 128-key blocks of all (request, key/value head) pairs, laid end to end with some units more for each pair, are split
// evenly over the CTAs. A CTA's run inside one pair is a segment; a segment that covers its pair writes the output, the
// others leave (O, m, l) in the CTA's two partial slots, and the CTA that finishes a cut pair last joins its segments in
// slot order.
#pragma once

#include <cuda_runtime.h>

#include <cmath>

#include "attn_common.cuh"

namespace dt {
namespace {

constexpr int kPaRows = 128;  // query rows per pair: G n at most
constexpr int kPaNodes = 64;  // n at most (a node's mask row is one 64-bit word)
constexpr int kPaKeys = 128;  // keys per block
constexpr size_t kPaSmemCap = 232448 - 5120;  // opt-in shared memory of a CTA, less the static part
static_assert(kAtWeightMost * kAtValueMost * DT_PAGED_MAX_TOKENS < 1e38, "a request's weighted values have a sum");

struct PaWork {
  int B, n, Hq, Hkv, G, R, grid;
  int extra;                       // units of a pair before those of its blocks: what its start and end cost, in blocks
  int page_size, num_pages, max_pages;
  const int32_t* page_table;       // [B][max_pages]
  const int32_t* lens;             // [B]
  const uint8_t* mask;             // [B][n][n] or null: causal among the n
  float* part;                     // [grid][2][R][D] unnormalised outputs of cut segments
  float* ml;                       // [grid][2][R][2] the weights' reference (base 2) and their sum
  unsigned short* out;             // [B][n][Hq][D] bf16
};

// The lengths' plan. cum[b]: units of one head of the requests before b, a request's being its 128-key blocks and `extra`
// more; a request whose length is not in [n, max_pages * page_size] has none (0 and below: an unused row of the batch;
// otherwise an error).
__device__ __forceinline__ int pa_length(const PaWork& p, int b, bool* bad) {
  const int len = p.lens[b];
  if (len <= 0) return 0;
  if (len < p.n || len > static_cast<long long>(p.max_pages) * p.page_size) {
    *bad = true;
    return 0;
  }
  return len;
}
// CTA c's share of W units starts here; the CTA whose share holds unit x. (A 64-bit division takes half a microsecond
// on the way to the first load; a batch's units nearly always fit 32 bits.)
__device__ __forceinline__ long long pa_div(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}
__device__ __forceinline__ long long pa_share(long long W, int grid, int c) { return pa_div(W * c, grid); }
__device__ __forceinline__ int pa_owner(long long x, long long W, int grid) {
  return static_cast<int>(pa_div((x + 1) * grid - 1, W));
}
struct PaSeg {
  int b, kvh, nb, j0, nblk;  // blocks j0 .. j0 + nblk - 1 of the pair's nb
  long long pair0;           // the pair's first block in the flattened order (after the pair's extra units)
};
struct PaWalk {  // a CTA's segments, in order
  int b;
  long long x0, x, x1;
};
__device__ __forceinline__ PaWalk pa_walk(const PaWork& p, const int* cum, long long W, int ctas) {
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
// The next segment, nblk 0 when there is none.
__device__ __forceinline__ PaSeg pa_next(const PaWork& p, const int* cum, PaWalk& w) {
  PaSeg s{};
  while (w.x < w.x1) {
    while (static_cast<long long>(cum[w.b + 1]) * p.Hkv <= w.x) ++w.b;
    const int units = cum[w.b + 1] - cum[w.b];
    const long long start = static_cast<long long>(cum[w.b]) * p.Hkv;
    const int rel = static_cast<int>(w.x - start), kvh = rel / units, at = rel - kvh * units;  // rel < units Hkv < 2^26
    const long long left = w.x1 - w.x;
    const int take = left < units - at ? static_cast<int>(left) : units - at;
    w.x += take;
    const int skip = at >= p.extra ? 0 : p.extra - at < take ? p.extra - at : take;
    s.nblk = take - skip;
    if (s.nblk == 0) continue;  // the share ends among the pair's extra units
    s.b = w.b;
    s.kvh = kvh;
    s.nb = units - p.extra;
    s.j0 = at >= p.extra ? at - p.extra : 0;
    s.pair0 = start + static_cast<long long>(kvh) * units + p.extra;
    break;
  }
  return s;
}

// The softmax warps meet (a barrier whose wait is bounded); `count` is the meetings so far, the same in every warp.
__device__ __forceinline__ bool pa_sync(uint64_t* bar, unsigned& count, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
  return __all_sync(0xFFFFFFFFu, at_wait(bar, count++ & 1u));
}

// A cut pair's segments are those of CTAs c0 .. c1. A CTA's slot 1 holds the segment that starts its pair, slot 0 one
// that goes on with another CTA's.
struct PaJoin {
  int b, kvh, c0, c1;
};
// Joins them with every thread of the CTA: a thread takes four columns of a query row and runs through the segments
// with a maximum that may rise. Many rows: several at once, so that their loads are in flight together. Few rows
// (kAtOnce 1): as many threads a row as there are, each with every so many segments, joined in order through shared
// memory.
struct PaSum {
  float4 num;
  float m, den;
  __device__ __forceinline__ void add(const float4& x, float mx, float d) {
    const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.f : mn;  // nothing visible so far: 2^-inf = 0
    const float a = exp2f(m - ref), b = exp2f(mx - ref);
    m = mn;
    den = den * a + b * d;
    num.x = num.x * a + b * x.x;
    num.y = num.y * a + b * x.y;
    num.z = num.z * a + b * x.z;
    num.w = num.w * a + b * x.w;
  }
};
template <int D>
__device__ __forceinline__ void pa_join_out(const PaWork& p, const PaJoin& jn, int i, const PaSum& s) {
  constexpr int kQuads = D / 4;
  const int r = i / kQuads, node = r / p.G;
  // a cut pair has two blocks at least, and so a prefix that every node sees
  static_assert(kPaNodes < kPaKeys, "the nodes' own keys fill no block");
  const float inv = 1.f / s.den;
  unsigned short* o =
      p.out + ((static_cast<size_t>(jn.b) * p.n + node) * p.Hq + jn.kvh * p.G + r % p.G) * D + 4 * (i % kQuads);
  *reinterpret_cast<uint2*>(o) =
      make_uint2(at_pack(s.num.x * inv, s.num.y * inv), at_pack(s.num.z * inv, s.num.w * inv));
}
template <int D, int kAtOnce, int kThreads>
__device__ __forceinline__ void pa_join(const PaWork& p, const PaJoin& jn, PaSum* red) {
  constexpr int kQuads = D / 4, kSegments = kAtOnce == 1 ? 8 : 2;  // in flight: kAtOnce rows of kSegments segments
  const int nseg = jn.c1 - jn.c0 + 1, total = p.R * kQuads;
  const int groups = kAtOnce == 1 ? kThreads / total : 1, group = kAtOnce == 1 ? threadIdx.x / total : 0;
  const int first = kAtOnce == 1 ? static_cast<int>(threadIdx.x) % total : static_cast<int>(threadIdx.x);
  for (int i0 = first; i0 < total; i0 += kAtOnce * kThreads) {
    PaSum s[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) s[u] = PaSum{make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f};
    for (int c0 = group; group < groups && c0 < nseg; c0 += kSegments * groups) {
      float2 ml[kSegments][kAtOnce];
      float4 x[kSegments][kAtOnce];
#pragma unroll
      for (int k = 0; k < kSegments; ++k) {
        const int c = c0 + k * groups;
        const size_t unit = 2 * static_cast<size_t>(jn.c0 + c) + (c == 0 ? 1 : 0);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const int i = i0 + u * kThreads;
          const size_t row = unit * p.R + i / kQuads;
          ml[k][u] = make_float2(-INFINITY, 0.f);
          x[k][u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c < nseg && i < total) {
            ml[k][u] = __ldcg(reinterpret_cast<const float2*>(p.ml + 2 * row));
            x[k][u] = __ldcg(reinterpret_cast<const float4*>(p.part + row * D + 4 * (i % kQuads)));
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kSegments; ++k)
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) s[u].add(x[k][u], ml[k][u].x, ml[k][u].y);
    }
    if constexpr (kAtOnce == 1) {
      if (group > 0 && group < groups) red[threadIdx.x] = s[0];
      __syncthreads();
      if (group == 0) {
        for (int g = 1; g < groups; ++g) {
          const PaSum& other = red[g * total + i0];
          s[0].add(other.num, other.m, other.den);
        }
        pa_join_out<D>(p, jn, i0, s[0]);
      }
      __syncthreads();
      break;  // every thread had one
    } else {
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (i0 + u * kThreads < total) pa_join_out<D>(p, jn, i0 + u * kThreads, s[u]);
    }
  }
}

// The keys of a pair from here on are not the same for all rows (the nodes' own), or not all there (the last block's
// rows past the request's end): blocks that reach past it are masked, and their values cleaned.
__device__ __forceinline__ int pa_common(const PaWork& p, int len) { return p.n > 1 || p.mask ? len - p.n : len; }

// Of 64 consecutive keys: all before `own` are visible, key own + c where bit c of `nodes` is set, none from `end` on.
__device__ __forceinline__ unsigned long long pa_visible(int own, int end, unsigned long long nodes) {
  const unsigned long long before = own >= 64 ? ~0ull : own <= 0 ? 0ull : (1ull << own) - 1ull;
  const unsigned long long there = end >= 64 ? ~0ull : end <= 0 ? 0ull : (1ull << end) - 1ull;
  const unsigned long long tree = own >= 64 || own <= -64 ? 0ull : own >= 0 ? nodes << own : nodes >> -own;
  return (before | tree) & there;
}

struct PaPlan {
  int grid;
  size_t part, ml, bytes;  // behind the header nothing outlives a call
};
inline PaPlan pa_plan(int R, int d, int sms) {
  PaPlan P{};
  P.grid = sms < kWsTickets ? sms : kWsTickets;
  P.part = align_up(sizeof(WsHeader));
  P.ml = align_up(P.part + sizeof(float) * 2 * P.grid * static_cast<size_t>(R) * d);
  P.bytes = align_up(P.ml + sizeof(float) * 2 * 2 * P.grid * static_cast<size_t>(R));
  return P;
}

}  // namespace
}  // namespace dt
