// dt_paged_attention8 — attention of each request's newest tokens over its paged cache in 8 bits with scales.
//
// For request b, node i and query head h: out = softmax(scale q.k_j) v_j over the visible keys j, where k_j and v_j are
// e4m3 codes times the scales ks_j and vs_j of their block of rows. The scales stay outside the products:
//     score_j = ks_j (q . code_j),  out = sum_j (p_j vs_j) code_j / sum_j p_j.
//
// GB300 design. As in the bf16 kernel the R = G n query rows that share a key/value head read each cached row once, and
// the 128-key blocks of all pairs are split evenly over the CTAs. What bounds it is memory, at half the bytes a block, so
// little may be done to a code on its way. Keys and values are the left operands: S^T = K Q^T (a lane a key) and
// O^T = V^T W (a lane a column), so that the few query rows are N and a product costs little when R is small.
//   Keys go to the tensor cores as the e4m3 they are, from the ring that TMA fills. The queries then are e4m3 too: two
// terms, q = q1 + q2, which hold the eight significant bits of a bf16 between them (what q1 rounds away is at most eight
// steps of the eighth bit: four bits), so each key is multiplied twice, and once less is read than with a conversion.
//   Weights are not so kind: they need a wide range below their largest. They stay fp16, and values are brought to fp16
// (exactly) on the way from the ring to tensor memory: a transposing load of pairs of columns, a byte shuffle, one
// conversion for two codes.
//   A softmax thread owns a key: its scales are two registers, and a row's maximum is looked for only when some weight
// leaves the headroom.
//
// Measured (32/8 heads, d = 128): a token each for 64 requests of up to 8191 keys 95 us with pages of 64, 96 with pages of
// 16 (539 MB, 5.6 TB/s, 83% of the copy rate); 3 requests of up to 131072 keys 111 (710 MB, 6.4 TB/s, 94%): memory. 64
// trees of 16 nodes over up to 4099 keys 112 (of 8 81, of 3 64; their bytes take 43): the softmax, about 36 issue slots an
// element in all, and the chain of waits that a step is. d = 64, a token each 73 (floor 40): that chain. Keys brought to
// fp16 like the values instead of two products: 119 where this took 97. The maximum looked for after the weights, which
// are made again if one left the headroom: trees 118, of 8 nodes 88. A segment's outputs by the warps of the values: trees
// the same, pages of 16 112 for 100. The bf16 cache takes 167.6, 101.8 (of 8 97.1, of 3 92.3) and 92.6 for the first, the
// trees and the last: this one is the faster up to 32 rows at d = 128; at d = 64, where trees of 2, 3, 4 and 8 nodes take 49.4,
// 56.3, 58.1 and 74.3 here and 57.7, 57.4, 57.2 and 64.3 there, up to 8 rows. Past that it saves memory alone.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "attn_common.cuh"
#include "paged_share.cuh"

namespace dt {
namespace {

constexpr int kP8MaxStages = 24;
// Blocks whose scales are there: the load runs at most half a ring ahead of the keys that the tensor cores have read, and
// those two steps of up to two blocks ahead of the softmax.
constexpr int kP8Scales = 32;
static_assert(kP8MaxStages / 2 + 4 <= kP8Scales, "scales are not overwritten before they are read");
constexpr size_t kPa8SmemCap = 232448 - 11264;  // opt-in shared memory of a CTA, less the static part
// What a pair's start and end cost, in blocks (64 trees of 16 nodes: 2 123 us, 4 112, 6 115; a token each at d = 64 77, 76, 77).
constexpr int kP8Extra = 4;
// Weights times their values' scales are fp16: a row's largest starts out at 2^kP8Start and may grow to 2^kP8Most before
// the reference is raised. fp16 goes up to 2^16 and holds subnormal numbers in steps of 2^-24.
constexpr float kP8Start = 4.f, kP8Most = 15.f;
constexpr float kP8LeastScale = -64.f;  // log2: smaller scales of values do not pull the reference further down

struct Pa8Params : PaWork {
  int stages;
  int page_shift, block_shift;      // log2 of the rows of a page, and of those that share a scale
  int third;                        // whether a third warp copies boxes
  const unsigned short* q;          // [B][n][Hq][D]
  const unsigned char* v_cache;     // re-read only for codes that are NaN
  const float *k_scale, *v_scale;   // [num_pages][Hkv][page_size >> block_shift]
  float scale_log2;                 // scale * log2(e)
};
struct Pa8Maps {
  CUtensorMap k, v;  // [num_pages * Hkv][page_size][D], boxes of min(page_size, 128) rows
};

// Loads and stores of n columns of tensor memory with a row (lane) per thread: column c of the thread's lane is v[c]. Each
// load waits for itself.
template <int n>
__device__ __forceinline__ void p8_ld(uint32_t taddr, float* v);
template <int n>
__device__ __forceinline__ void p8_st(uint32_t taddr, const float* v);
template <>
__device__ __forceinline__ void p8_ld<4>(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
      : "r"(taddr)
      : "memory");
}
template <>
__device__ __forceinline__ void p8_ld<8>(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
      : "r"(taddr)
      : "memory");
}
template <>
__device__ __forceinline__ void p8_ld<16>(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}
template <>
__device__ __forceinline__ void p8_st<8>(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
      : "memory");
}
template <>
__device__ __forceinline__ void p8_st<16>(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
        "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
// 16 lanes x 64 columns: in each group of 4 columns thread l holds column l % 4 of lanes l / 4 and l / 4 + 8.
__device__ __forceinline__ void p8_st_v(uint32_t taddr, const uint32_t* v) {  // 64 columns of two fp16
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
        "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
        "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

__device__ __forceinline__ uint32_t p8_two(uint32_t codes) {  // the two e4m3 codes in the low half
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}
__device__ __forceinline__ void p8_four(uint32_t codes, uint32_t& lo, uint32_t& hi) {  // those of both halves
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
__device__ __forceinline__ uint32_t p8_code2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t p8_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint64_t p8_mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float p8_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Waits. try_wait holds a warp for some fifty cycles only, so a warp that waits is a warp that polls, and takes issue slots
// and instruction fetches from those that work. The roles that run ahead (load, queries, values) rest between their looks;
// the others poll in as few instructions as there can be. The long way stands in one place each.
__device__ __noinline__ bool p8_poll(uint64_t* bar, unsigned parity) {
  const uint64_t t0 = global_timer_ns();
  do {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, 0;\n"
        "LOOK:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
        "add.u32 n, n, 1;\n\tsetp.lt.u32 q, n, 1000;\n\t@q bra LOOK;\n"
        "DONE:\n\tselp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (done) return true;
  } while (global_timer_ns() - t0 <= kAtBudgetNs);
  return false;
}
__device__ __noinline__ bool p8_nap(uint64_t* bar, unsigned parity) {
  const uint64_t t0 = global_timer_ns();
  do {
#pragma unroll 1
    for (int i = 0; i < 1000; ++i) {
      __nanosleep(64);
      if (mbar_try_wait(bar, parity)) return true;
    }
  } while (global_timer_ns() - t0 <= kAtBudgetNs);
  return false;
}
__device__ __forceinline__ bool p8_wait(uint64_t* bar, unsigned parity) {
  return mbar_try_wait(bar, parity) || p8_poll(bar, parity);
}
__device__ __forceinline__ bool p8_rest(uint64_t* bar, unsigned parity) {
  return mbar_try_wait(bar, parity) || p8_nap(bar, parity);
}
// Of a block's pages, so many are copied by the loads of the keys and of the values, the rest of both by a third warp.
__device__ __forceinline__ int p8_own_pages(int per_block) { return per_block - (per_block + 1) / 3; }
// Entries announced to the third warp, and its wait for more than `g` of them (each has been found empty, and expects all
// of its bytes, by then).
__device__ __forceinline__ void p8_issue(unsigned* count, unsigned now) {
  asm volatile("st.release.cta.shared.u32 [%0], %1;" ::"r"(smem_u32(count)), "r"(now) : "memory");
}
__device__ __forceinline__ bool p8_issued(const unsigned* count, unsigned g) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (unsigned i = 0;; ++i) {
    unsigned now;
    asm volatile("ld.acquire.cta.shared.u32 %0, [%1];" : "=r"(now) : "r"(smem_u32(count)) : "memory");
    if (now > g) return true;
    if ((i & 1023u) == 0u) {
      const uint64_t t = global_timer_ns();
      if (i == 0u) t0 = t;
      if (t - t0 > kAtBudgetNs) return false;
    }
    __nanosleep(32);
  }
}
// Whether any of a group's threads says so; all of them come here, by whole warps.
template <int kThreads>
__device__ __forceinline__ bool p8_any(int id, bool x) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(id), "n"(kThreads)
      : "memory");
  return r != 0u;
}
template <int kThreads>
__device__ __forceinline__ void p8_meet(int id) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kThreads) : "memory");
}
// The warp's largest value of x; NaN counts for nothing.
__device__ __forceinline__ float p8_warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// The warp's sums of R values a lane: lane x returns that of value x / (32 / R).
template <int R>
__device__ __forceinline__ float p8_warp_sums(float (&v)[R], int lane) {
#pragma unroll
  for (int w = R / 2, h = 16; w >= 1; w /= 2, h /= 2) {
    const bool up = (lane & h) != 0;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float got = __shfl_xor_sync(0xFFFFFFFFu, up ? v[i] : v[i + w], h);
      v[i] = (up ? v[i + w] : v[i]) + got;
    }
  }
#pragma unroll
  for (int h = 16 / R; h >= 1; h /= 2) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], h);
  return v[0];
}
// Where 16-byte piece c of row r of a block lies in its ring entry.
template <int D>
__device__ __forceinline__ uint32_t p8_piece(int r, int c) {
  return D == 128 ? static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4))
                  : static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// The shape of one instance: N columns of query rows (R rounded up), of which a softmax thread has M for its key, kStep at
// a time, in each of its blocks: kPar blocks are a step.
template <int D, int N, int M, int kPar_, int kStep_>
struct P8 {
  static constexpr int kPar = kPar_;                     // blocks of a step: the softmax takes them at once
  static constexpr int kRowGroups = N > 16 ? N / M : 1;  // groups of four softmax warps share a block's rows
  static constexpr int kGroups = kPar * kRowGroups;
  static constexpr int kMeet = 128 * kPar;               // softmax threads that have the same rows
  static constexpr int kSoftmax = 8;                     // warps 0, 2, 3: load, 1: MMA, 4-7: values, then softmax
  static constexpr int kThreads = 32 * kSoftmax + 128 * kGroups;
  static constexpr bool kOwnQ = N <= 16;                 // a warp of its own for the queries, unless it is wanted for boxes
  static constexpr int kStep = kStep_;                   // rows taken at once
  static constexpr int kSteps = M / kStep;
  // a thread's sums: of its key and a row each, or, without the registers for so many, of its warp's keys
  static constexpr bool kWarpSums = M > 16;
  static constexpr int kSums = kWarpSums ? kSteps : M;
  static constexpr bool kKeep = M <= 8;                  // registers for the rows' factors and references
  static constexpr int kOut = M / kPar < 16 ? M / kPar : 16;  // rows of outputs that a thread takes at once
  static constexpr int kWs = 2;                          // steps whose weights have buffers
  static constexpr int kVs = N * kPar <= 64 ? 4 : 2;     // buffers of values
  static constexpr int kOs = N <= 64 ? 2 : 1;            // buffers of outputs
  static constexpr uint32_t kEntry = kPaKeys * D;        // a ring entry: a block's keys or values
  static constexpr uint32_t kTerm = N * D;               // one term of the queries
  static constexpr uint32_t kQ = 2 * kTerm;              // a buffer of queries
  static constexpr int kAtom = N < 64 ? N : 64;          // query rows in a row of the weights
  static constexpr uint32_t kRowW = kAtom * 2;
  static constexpr uint32_t kW = kPaKeys * N * 2;        // a buffer of weights
  // tensor memory
  static constexpr uint32_t kS = 0, kO = 2 * kPar * N, kV = kO + kOs * N;
  static_assert(kV + kVs * 64 <= 512, "tensor memory");
  static constexpr size_t kFixed = 1024 + 2 * kQ + kWs * kPar * kW;
};

// Roles. Load: pages to the ring, as in the bf16 kernel, and their scales, keys and values by a warp each, and some of
// both by a third where a block spans many pages (a box takes its warp about a hundred cycles to issue). Values: lane =
// column, two keys a register. Softmax: lane = key; its scales come with the keys (loaded by the softmax itself a block
// ahead they are late: a block takes less than a load). MMA: the scores run one step ahead of the outputs, through the
// segments. Queries: by the third warp of loads where there are few rows and it is not wanted for boxes, else by the
// warps of the values, a segment ahead.
template <int D, int N, int M, int kPar_, int kStep_>
__global__ void __launch_bounds__(P8<D, N, M, kPar_, kStep_>::kThreads, 1)
    paged_attn8_kernel(Pa8Params p, const __grid_constant__ Pa8Maps maps, WsHeader* hdr) {
  using C = P8<D, N, M, kPar_, kStep_>;
  constexpr int kThreads = C::kThreads, kPar = C::kPar, kMeet = C::kMeet, kStep = C::kStep, kVs = C::kVs, kOs = C::kOs;
  extern __shared__ float4 smem_f4[];
  unsigned char* sq =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_f4) + 1023) & ~uintptr_t(1023));
  unsigned char* sw = sq + 2 * C::kQ;
  unsigned char* skv = sw + C::kWs * kPar * C::kW;
  int* cum = reinterpret_cast<int*>(skv + p.stages * C::kEntry);  // [B + 1]
  int* lens = cum + p.B + 1;                                      // [B]
  __shared__ uint64_t kv_full[kP8MaxStages], kv_empty[kP8MaxStages];
  __shared__ uint64_t v_full[kVs], v_empty[kVs];
  __shared__ uint64_t s_full[2], w_full[2], o_done[2], q_full[2], o_free[2], s_meet;
  __shared__ uint32_t s_tmem;
  __shared__ unsigned s_issued[2];  // ring entries of keys, of values
  __shared__ int s_warp[kThreads / 32];
  __shared__ int s_bad, s_joins;
  __shared__ PaJoin s_join[2];
  __shared__ float s_scales[kP8Scales][2][kPaKeys / DT_MIN_PAGE];  // of a block's keys, then of its values
  __shared__ __align__(16) float s_factor[2][N], s_nref[N], s_alpha[N], s_red[4 * kPar][N];
  __shared__ unsigned long long s_sees[2][kPaNodes];  // bit i: node i sees the key of node c
  __shared__ int s_at[N];                             // a query row's place in a request's outputs
  __shared__ unsigned char s_node[N];                 // its node
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const unsigned stages = static_cast<unsigned>(p.stages);
  if (t == 0) {
    for (unsigned i = 0; i < stages; ++i) {
      mbar_init(&kv_full[i], i % 2 == 0 ? 33 : 1);  // keys: and each lane's copy of a scale
      mbar_init(&kv_empty[i], i % 2 == 0 ? 1 : 4);  // keys: by the tensor cores; values: by four warps
    }
    for (int i = 0; i < kVs; ++i) {
      mbar_init(&v_full[i], 4);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&w_full[i], 4 * C::kGroups);
      mbar_init(&o_done[i], 1);
      mbar_init(&q_full[i], C::kOwnQ && p.third == 0 ? 1 : 4);
      mbar_init(&o_free[i], 4 * C::kGroups);
    }
    mbar_init(&s_meet, 4 * C::kGroups);
    mbar_fence_init();
    s_issued[0] = s_issued[1] = 0u;
    s_bad = s_joins = 0;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 0 && lane < 2)
    asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &maps.k : &maps.v) : "memory");
  // rows of queries that there are not: zero, with a factor of zero
  for (int i = t; i < static_cast<int>(2 * C::kQ / 16); i += kThreads)
    if (static_cast<int>(i * 16 / D) % N >= p.R) reinterpret_cast<uint4*>(sq)[i] = make_uint4(0u, 0u, 0u, 0u);
  // and the weights of rows that no softmax thread has
  for (int i = t; i < static_cast<int>(C::kWs * kPar * C::kW / 16); i += kThreads)
    reinterpret_cast<uint4*>(sw)[i] = make_uint4(0u, 0u, 0u, 0u);
  for (int r = t; r < N; r += kThreads) {
    s_node[r] = static_cast<unsigned char>(r / p.G < kPaNodes ? r / p.G : kPaNodes - 1);
    s_at[r] = (r / p.G * p.Hq + r % p.G) * D;
  }
  for (int i = t; i < 2 * N; i += kThreads) s_factor[i / N][i % N] = 0.f;
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  at_launch_order();
  // the plan: block counts scanned over the requests; rows of requests without blocks are zero
  int carry = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + t;
    bool bad = false;
    const int len = b < p.B ? pa_length(p, b, &bad) : 0;
    if (bad && blockIdx.x == 0) record_error(hdr, DT_ERR_INVALID_ARG);
    int total;
    const int units = len > 0 ? (len + kPaKeys - 1) / kPaKeys + p.extra : 0;
    const int before = block_exclusive_scan<kThreads / 32>(units, &total, s_warp);
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
      for (int i = t; i < p.n * p.Hq * (D / 8); i += kThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  bool ok = true;
  const int ctas = W < p.grid ? static_cast<int>(W) : p.grid;  // that take a share: a block each at least
  PaWalk w = pa_walk(p, cum, W, ctas);

  // A segment's queries and its mask, by `of` warps.
  const bool third = C::kOwnQ && p.third != 0;  // warp 3 copies boxes
  const int own_pages = third ? p8_own_pages(kPaKeys >> p.page_shift) : kPaKeys;
  auto queries = [&](const PaSeg& sg, int si, int who, int of) {
    const unsigned qb = static_cast<unsigned>(si) & 1u;
    // the segment that had the buffer before is over: its factors and its mask are not read any more
    if (si >= 2) ok = __all_sync(0xFFFFFFFFu, p8_rest(&o_free[qb], static_cast<unsigned>((si >> 1) - 1) & 1u));
    if (!ok) return;
#pragma unroll 1
    for (int c = 32 * who + lane; c < p.n; c += 32 * of) {
      unsigned long long bits = ~0ull << c;
      if (p.mask) {
        const uint8_t* col = p.mask + static_cast<size_t>(sg.b) * p.n * p.n + c;
        bits = 0ull;
#pragma unroll 8
        for (int i = 0; i < p.n; ++i) bits |= static_cast<unsigned long long>(col[static_cast<size_t>(i) * p.n] != 0) << i;
      }
      s_sees[qb][c] = bits;
    }
    unsigned char* qd = sq + qb * C::kQ;
    // eight lanes a row, D / 8 elements each; four rows a step, several steps' loads in flight
    constexpr int kEach = D / 8, kAtOnce = 4;
    const int sub = lane & 7;
    const unsigned short* src = p.q + (static_cast<size_t>(sg.b) * p.n * p.Hq + sg.kvh * p.G) * D + kEach * sub;
#pragma unroll 1
    for (int r0 = 4 * kAtOnce * who; r0 < p.R; r0 += 4 * kAtOnce * of) {
      uint4 x[kAtOnce][kEach / 8];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int r = r0 + 4 * u + (lane >> 3);
#pragma unroll
        for (int i = 0; i < kEach / 8; ++i)
          x[u][i] = r < p.R ? *reinterpret_cast<const uint4*>(src + s_at[r] + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (r0 + 4 * u >= p.R) break;
        const int r = r0 + 4 * u + (lane >> 3);
        const uint32_t* bits = reinterpret_cast<const uint32_t*>(x[u]);
        unsigned most = 0u;  // the bits of the row's largest finite element, as a bf16
#pragma unroll
        for (int i = 0; i < kEach / 2; ++i) {
          const unsigned lo = bits[i] & 0x7FFFu, hi = (bits[i] >> 16) & 0x7FFFu;
          if (lo < 0x7F80u && lo > most) most = lo;
          if (hi < 0x7F80u && hi > most) most = hi;
        }
#pragma unroll
        for (int h = 4; h > 0; h >>= 1) {
          const unsigned other = __shfl_xor_sync(0xFFFFFFFFu, most, h);
          most = other > most ? other : most;
        }
        // the largest power of two that leaves it at 448 = 1.75 2^8 or less
        int up = ((most & 0x7Fu) > 0x60u ? 7 : 8) - (static_cast<int>(most >> 7) - 127);
        if (up > 100) up = 100;  // (nothing is lost: such a row's scores are zero whatever the keys are)
        const float by = __uint_as_float(static_cast<unsigned>(up + 127) << 23);
        uint32_t q1[kEach / 4], q2[kEach / 4];
#pragma unroll
        for (int i = 0; i < kEach / 4; ++i) q1[i] = q2[i] = 0u;
#pragma unroll
        for (int i = 0; i < kEach / 2; ++i) {
          const float a = __uint_as_float(bits[i] << 16) * by, b = __uint_as_float(bits[i] & 0xFFFF0000u) * by;
          const float a1 = fabsf(a) <= 448.f ? a : NAN, b1 = fabsf(b) <= 448.f ? b : NAN;
          const uint32_t c = p8_code2(a1, b1), two = p8_two(c);
          const float2 got = __half22float2(*reinterpret_cast<const __half2*>(&two));
          q1[i / 2] |= c << (16 * (i & 1));
          q2[i / 2] |= p8_code2(a1 - got.x, b1 - got.y) << (16 * (i & 1));
        }
        if (r < p.R) {
          if constexpr (D == 128) {
            unsigned char* at = qd + p8_piece<D>(r, sub);
            *reinterpret_cast<uint4*>(at) = make_uint4(q1[0], q1[1], q1[kEach / 4 - 2], q1[kEach / 4 - 1]);
            *reinterpret_cast<uint4*>(at + C::kTerm) = make_uint4(q2[0], q2[1], q2[kEach / 4 - 2], q2[kEach / 4 - 1]);
          } else {
            unsigned char* at = qd + p8_piece<D>(r, sub >> 1) + 8 * (sub & 1);
            *reinterpret_cast<uint2*>(at) = make_uint2(q1[0], q1[1]);
            *reinterpret_cast<uint2*>(at + C::kTerm) = make_uint2(q2[0], q2[1]);
          }
          if (sub == 0) s_factor[qb][r] = p.scale_log2 * __uint_as_float(static_cast<unsigned>(127 - up) << 23);
        }
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMA reads Q through the async proxy
    __syncwarp();
    if (lane == 0) mbar_arrive(&q_full[qb]);
  };

  if (warp == 0 || warp == 2) {  // load: the keys, the values; the whole warp, one page's box a lane
    const int kv = warp >> 1;
    const CUtensorMap* map = kv ? &maps.v : &maps.k;
    unsigned st = kv, par = 1u, g = 0;  // ring entry, the parity of its last release, entries so far
    const int box_rows = p.page_size < kPaKeys ? p.page_size : kPaKeys;
    const int per_block = kPaKeys / box_rows;  // pages a block spans (1 when a page holds whole blocks)
    const int per_scale = p.block_shift < 7 ? kPaKeys >> p.block_shift : 1;  // scales a block has
    while (ok) {
      const PaSeg sg = pa_next(p, cum, w);
      if (sg.nblk == 0) break;
      const int used = (lens[sg.b] + p.page_size - 1) >> p.page_shift;  // pages the request holds
      const int32_t* table = p.page_table + static_cast<size_t>(sg.b) * p.max_pages;
      // page ids, 32 at a time and one window ahead
      int win = ((sg.j0 * kPaKeys) >> p.page_shift) / 32;
      int cur = 32 * win + lane < used ? table[32 * win + lane] : 0;
      int nxt = 32 * (win + 1) + lane < used ? table[32 * (win + 1) + lane] : 0;
      for (int j = 0; j < sg.nblk && ok; ++j, ++g) {
        const int key = (sg.j0 + j) * kPaKeys, first = key >> p.page_shift, row = key & (p.page_size - 1);
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
        const int plane = page * p.Hkv + sg.kvh;  // num_pages Hkv < 2^31
        // the block's scales come with its keys, the values' too: the softmax needs both, and waits for no value. Lanes
        // 0-15 the keys', the others the values'
        const int at = row + ((lane & 15) << p.block_shift), from = __shfl_sync(0xFFFFFFFFu, plane, at >> p.page_shift);
        if (2 * g >= stages) ok = __all_sync(0xFFFFFFFFu, p8_rest(&kv_empty[st], par));
        if (!ok) break;
        if (lane == 0) {
          mbar_expect_tx(&kv_full[st], static_cast<uint32_t>(pages * box_rows * D));
          p8_issue(&s_issued[kv], g + 1u);
        }
        __syncwarp();
        if (lane < pages && lane < own_pages)
          tma_load_3d(skv + st * C::kEntry + lane * box_rows * D, map, 0, row, plane, &kv_full[st]);
        if (kv == 0 && (lane & 15) < per_scale && (at >> p.page_shift) < pages) {
          const float* src = (lane < 16 ? p.k_scale : p.v_scale) + (static_cast<size_t>(from) << (p.page_shift - p.block_shift)) +
                             ((at & (p.page_size - 1)) >> p.block_shift);
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(
                           &s_scales[g % kP8Scales][lane >> 4][lane & 15])),
                       "l"(src)
                       : "memory");
        }
        if (kv == 0) asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(&kv_full[st])) : "memory");
        st += 2;
        if (st >= stages) {
          st = kv;
          par ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {  // MMA
      // the same bits for e4m3 and for fp16; O: the weights MN-major
      const uint32_t id_s = umma_idesc_f16(N), id_o = umma_idesc_f16(N) | (1u << 16);
      const uint64_t dq = umma_desc_rows(smem_u32(sq), D), dk = umma_desc_rows(smem_u32(skv), D);
      const uint64_t dw = umma_desc_mn(smem_u32(sw), C::kRowW, kPaKeys * 128);
      auto wait = [&](uint64_t* bar, unsigned parity) {
        const bool done = p8_wait(bar, parity);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        return done;
      };
      PaWalk ws = w;
      PaSeg ss{};
      int js = 0, sis = -1;
      unsigned gs = 0, st = 0, par = 0;  // the ring entry of the next keys: every other one
      auto scores = [&]() {  // of the next step, if there is one
        if (js >= ss.nblk) {
          ss = pa_next(p, cum, ws);
          js = 0;
          if (ss.nblk == 0) return true;
          ++sis;
          if (!wait(&q_full[sis & 1], static_cast<unsigned>(sis >> 1) & 1u)) return false;
        }
        const uint64_t q0 = dq + static_cast<uint64_t>((sis & 1) * (C::kQ >> 4));
#pragma unroll 1
        for (int u = 0; u < kPar && js + u < ss.nblk; ++u) {
          if (!wait(&kv_full[st], par)) return false;
          const uint64_t k0 = dk + st * (C::kEntry >> 4);
          const uint32_t to = tmem + C::kS + ((gs & 1u) * kPar + u) * N;
#pragma unroll
          for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              umma_f8(to, k0 + 2u * kk, q0 + ((term * C::kTerm) >> 4) + 2u * kk, id_s, term + kk > 0 ? 1u : 0u);
          umma_commit(&kv_empty[st]);
          st += 2;
          if (st == stages) {
            st = 0;
            par ^= 1u;
          }
        }
        umma_commit(&s_full[gs & 1u]);
        js += kPar;
        ++gs;
        return true;
      };
      unsigned g = 0, step = 0;  // blocks and steps so far
      ok = scores();
      for (int si = 0; ok; ++si) {
        const PaSeg sg = pa_next(p, cum, w);
        if (sg.nblk == 0) break;
        const unsigned ob = static_cast<unsigned>(si) % kOs;
        for (int j = 0; j < sg.nblk && ok; j += kPar, ++step) {
          // their buffers were freed by the softmax of the step before (waited for below, one step ago); the next segment's
          // wait for its queries, and this one's outputs do not wait for them
          const bool early = js < ss.nblk;
          if (early) ok = scores();
          if (ok && j == 0 && si >= kOs) {  // the segment that had the buffer before has been read
            const int was = si - kOs;
            ok = wait(&o_free[was & 1], static_cast<unsigned>(was >> 1) & 1u);
          }
          if (ok) ok = wait(&w_full[step & 1u], (step >> 1) & 1u);
#pragma unroll 1
          for (int u = 0; u < kPar && j + u < sg.nblk && ok; ++u, ++g) {
            const unsigned vb = g % kVs;
            ok = wait(&v_full[vb], (g / kVs) & 1u);
            if (!ok) break;
            const uint64_t w0 = dw + (((step % C::kWs * kPar + u) * C::kW) >> 4);
#pragma unroll
            for (int kk = 0; kk < kPaKeys / 16; ++kk)
              umma_f16_ts(tmem + C::kO + ob * N, tmem + C::kV + vb * 64u + 8u * kk, w0 + ((kk * 16u * C::kRowW) >> 4), id_o,
                          (j + u > 0 || kk > 0) ? 1u : 0u);
            umma_commit(&v_empty[vb]);
          }
          if (!ok) break;
          umma_commit(&o_done[step & 1u]);
          if (!early) ok = scores();
        }
      }
    }
  } else if (warp == 3) {  // queries; or the other boxes of blocks that span many pages, once the load has announced them
    const int box_rows = p.page_size < kPaKeys ? p.page_size : kPaKeys;
    const int per_block = kPaKeys / box_rows;
    unsigned st = 0, g = 0;
    for (int si = 0; ok && C::kOwnQ; ++si) {
      const PaSeg sg = pa_next(p, cum, w);
      if (sg.nblk == 0) break;
      if (!third) {
        queries(sg, si, 0, 1);
        continue;
      }
      const int used = (lens[sg.b] + p.page_size - 1) >> p.page_shift;
      const int32_t* table = p.page_table + static_cast<size_t>(sg.b) * p.max_pages;
      int win = ((sg.j0 * kPaKeys) >> p.page_shift) / 32;
      int cur = 32 * win + lane < used ? table[32 * win + lane] : 0;
      int nxt = 32 * (win + 1) + lane < used ? table[32 * (win + 1) + lane] : 0;
      for (int j = 0; j < sg.nblk && ok; ++j, ++g) {
        const int first = ((sg.j0 + j) * kPaKeys) >> p.page_shift;
        if (first / 32 != win) {
          ++win;
          cur = nxt;
          nxt = 32 * (win + 1) + lane < used ? table[32 * (win + 1) + lane] : 0;
        }
        const int pages = used - first < per_block ? used - first : per_block;
        int page = __shfl_sync(0xFFFFFFFFu, cur, (first + lane) & 31);
        if (page < 0 || page >= p.num_pages) page = 0;  // (reported by the load)
        const int plane = page * p.Hkv + sg.kvh;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          ok = ok && __all_sync(0xFFFFFFFFu, p8_issued(&s_issued[kv], g));
          if (ok && lane >= own_pages && lane < pages)
            tma_load_3d(skv + (st + kv) * C::kEntry + lane * box_rows * D, kv ? &maps.v : &maps.k, 0, 0, plane,
                        &kv_full[st + kv]);
        }
        st += 2;
        if (st >= stages) st = 0;
      }
    }
  } else if (warp < C::kSoftmax) {  // values
    constexpr int kParts = D / 64;  // pieces of 16 columns a warp has
    const int part0 = (warp & 3) * kParts;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    unsigned g = 0, at = 1, par = 0;
    // queries, where they are these warps': a segment ahead, when the first buffers are full and nothing else is to do
    const bool ours = !C::kOwnQ || third;
    PaSeg sg = pa_next(p, cum, w), next{};
    if (ours && sg.nblk) queries(sg, 0, warp - 4, 4);
    for (int si = 0; ok && sg.nblk; sg = next, ++si) {
      const int len = lens[sg.b], common = pa_common(p, len);
      for (int j = 0; j < sg.nblk && ok; ++j, ++g) {
        if (j == (sg.nblk > kVs ? kVs : sg.nblk - 1)) {
          next = pa_next(p, cum, w);
          if (ours && next.nblk) queries(next, si + 1, warp - 4, 4);
          if (!ok) break;
        }
        const unsigned vb = g % kVs;
        const int kbase = (sg.j0 + j) * kPaKeys;
        ok = __all_sync(0xFFFFFFFFu, p8_rest(&kv_full[at], par));
        if (!ok) break;
        const uint32_t src = smem_u32(skv + at * C::kEntry);
        if (__builtin_expect(kbase + kPaKeys > common, 0)) {
          // A weight of zero does not hide a NaN from the tensor cores. Rows past the request's end are cleared; a NaN
          // among the nodes' codes is cleared here and given to the rows that see it at the end.
          bool found = false;
#pragma unroll 1
          for (int i = lane; i < kPaKeys * kParts; i += 32) {
            const int key = kbase + i / kParts;
            if (key < common) continue;
            uint4* piece = reinterpret_cast<uint4*>(skv + at * C::kEntry + p8_piece<D>(i / kParts, part0 + i % kParts));
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (key < len) {
              x = *piece;
              const uint4 nan = make_uint4(
                  __vcmpeq4(x.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu), __vcmpeq4(x.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu),
                  __vcmpeq4(x.z & 0x7F7F7F7Fu, 0x7F7F7F7Fu), __vcmpeq4(x.w & 0x7F7F7F7Fu, 0x7F7F7F7Fu));
              if ((nan.x | nan.y | nan.z | nan.w) == 0u) continue;
              found = true;
              x = make_uint4(x.x & ~nan.x, x.y & ~nan.y, x.z & ~nan.z, x.w & ~nan.w);
            }
            *piece = x;
          }
          if (found) atomicMax(&s_bad, si + 1);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the entry's next copy
          __syncwarp();
        }
        if (g >= kVs) {
          ok = __all_sync(0xFFFFFFFFu, p8_rest(&v_empty[vb], (g / kVs - 1) & 1u));
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        }
#pragma unroll 1
        for (int h = 0; h < kParts; ++h) {
          uint32_t r[32];
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            uint32_t x[4];
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                         : "r"(src + p8_piece<D>(32 * kk + lane, part0 + h))
                         : "memory");
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const uint32_t y = __byte_perm(x[m], 0u, 0x3120);  // two keys of a column, then of the next
              p8_four(y, r[2 * (4 * kk + m)], r[2 * (4 * kk + m) + 1]);
            }
          }
          p8_st_v(tmem + lanes + (static_cast<uint32_t>(16 * h) << 16) + C::kV + vb * 64u, r);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&kv_empty[at]);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[vb]);
        at += 2;
        if (at > stages) {
          at = 1;
          par ^= 1u;
        }
      }
    }
  } else {  // softmax
    const int group = (warp - C::kSoftmax) >> 2, quad = warp & 3, row = 32 * quad + lane;  // the thread's key of a block
    const int part = group / C::kRowGroups, first = group % C::kRowGroups * M;  // its block of a step, its first row
    const int bar = 1 + group % C::kRowGroups, mine = 128 * part + row, four = 4 * part + quad;
    const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
    // the column that the thread's lane of the outputs is, and the pair of columns that it writes
    const int column = D / 4 * quad + 16 * (lane >> 4) + 2 * (lane & 7) + ((lane >> 3) & 1);
    const bool has_column = D == 128 || lane < 16;
    const int my_scale = p.block_shift < 7 ? row >> p.block_shift : 0;
    unsigned g = part, step = 0, meet = 0;  // the thread's block, and the steps so far
    bool failed = false;                    // a wait ran out; those with the same rows leave together, at their next meeting
    for (int si = 0; ok; ++si) {
      const PaSeg sg = pa_next(p, cum, w);
      if (sg.nblk == 0) break;
      const unsigned qb = static_cast<unsigned>(si) & 1u;
      const uint32_t to = tmem + lanes + C::kO + (static_cast<unsigned>(si) % kOs) * N + first;
      const int len = lens[sg.b], pre = len - p.n, common = pa_common(p, len);
      float l[C::kSums], factors[C::kKeep ? M : 4], nrefs[C::kKeep ? M : 4];
#pragma unroll
      for (int i = 0; i < C::kSums; ++i) l[i] = 0.f;
      for (int j = part; j - part < sg.nblk && ok; j += kPar, g += kPar, ++step) {
        const bool there = j < sg.nblk;  // the step's last block may be missing
        const uint32_t ts = tmem + lanes + C::kS + ((step & 1u) * kPar + part) * N + first;
        if (!p8_wait(&s_full[step & 1u], (step >> 1) & 1u)) failed = true;
        __syncwarp();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if constexpr (C::kKeep) {
          if (j < kPar) {
#pragma unroll
            for (int i = 0; i < M; i += 4) {
              *reinterpret_cast<float4*>(factors + i) = *reinterpret_cast<const float4*>(&s_factor[qb][first + i]);
              nrefs[i] = nrefs[i + 1] = nrefs[i + 2] = nrefs[i + 3] = kAtNone;
            }
          }
        }
        float2 scales = make_float2(0.f, 0.f);
        if (there) scales = make_float2(s_scales[g % kP8Scales][0][my_scale], s_scales[g % kP8Scales][1][my_scale]);
        const float log_vs = fmaxf(p8_log2(fabsf(scales.y)), kP8LeastScale);
        const int key = (sg.j0 + j) * kPaKeys + row;
        const bool masked = (sg.j0 + j + 1) * kPaKeys > common;
        unsigned long long sees = ~0ull;  // bit i: row first + i sees the key
        if (__builtin_expect(masked && key >= pre, 0)) {
          sees = 0ull;
          if (key < len) {
            const unsigned long long nodes = s_sees[qb][key - pre];
#pragma unroll 4
            for (int i = 0; i < M; ++i) sees |= ((nodes >> s_node[first + i]) & 1ull) << i;
          }
        }
        const float value_scale = sees == 0ull ? 0.f : scales.y;
        __syncwarp();
        const bool fresh = j < kPar;  // a segment's first step: there are no references yet
        // kStep scores from row `r` of the thread's on, scaled, against the reference
        float x[kStep];
        auto load = [&](int r, bool against) {
          p8_ld<kStep>(ts + r, x);
          const uint64_t ks = at_pair(scales.x, scales.x);
#pragma unroll
          for (int i = 0; i < kStep; i += 4) {
            float4 f, n4 = make_float4(0.f, 0.f, 0.f, 0.f);
            if constexpr (C::kKeep) {
              f = make_float4(factors[i], factors[i + 1], factors[i + 2], factors[i + 3]);
              if (against) n4 = make_float4(nrefs[i], nrefs[i + 1], nrefs[i + 2], nrefs[i + 3]);
            } else {
              f = *reinterpret_cast<const float4*>(&s_factor[qb][first + r + i]);
              if (against) n4 = *reinterpret_cast<const float4*>(&s_nref[first + r + i]);
            }
            at_unpair(at_fma2(at_pair(x[i], x[i + 1]), p8_mul2(at_pair(f.x, f.y), ks), at_pair(n4.x, n4.y)), x[i],
                      x[i + 1]);
            at_unpair(at_fma2(at_pair(x[i + 2], x[i + 3]), p8_mul2(at_pair(f.z, f.w), ks), at_pair(n4.z, n4.w)), x[i + 2],
                      x[i + 3]);
          }
          if (__builtin_expect(masked, 0)) {
            const unsigned bits = static_cast<unsigned>(sees >> r);
#pragma unroll
            for (int i = 0; i < kStep; ++i)
              if (!((bits >> i) & 1u)) x[i] = -INFINITY;
          }
        };
#pragma unroll 1
        for (bool raised = false;; raised = true) {
          if (!fresh) {
            float top = -INFINITY;
            if (there) {
#pragma unroll 1
              for (int r = 0; r < M; r += kStep) {
                load(r, true);
#pragma unroll
                for (int i = 0; i < kStep; i += 2) top = at_max3(top, x[i], x[i + 1]);
              }
            }
            if (raised || __builtin_expect(!p8_any<kMeet>(bar, top + log_vs > kP8Most || failed), 1)) break;
          }
          // a segment's first step, and rarely later: raise references
          if (!fresh && p8_any<kMeet>(bar, failed)) {
            ok = false;
            break;
          }
#pragma unroll 1
          for (int r = 0; r < M; r += kStep) {
            float keep = -INFINITY;
            if (there) {
              load(r, false);
#pragma unroll
              for (int i = 0; i < kStep; ++i) {
                const float m = p8_warp_max(x[i] + log_vs);
                if (lane == i) keep = m;
              }
            }
            if (lane < kStep) s_red[four][first + r + lane] = keep;
          }
          p8_meet<kMeet>(bar);
          if (mine < M) {
            const int r = first + mine;
            float m = s_red[0][r];
#pragma unroll
            for (int i = 1; i < 4 * kPar; ++i) m = fmaxf(m, s_red[i][r]);
            const float was = fresh ? kAtNone : s_nref[r];
            const bool raise = m + was > kP8Most;
            const float now = raise ? kP8Start - m : was;
            s_alpha[r] = raise ? at_exp2(now - was) : 1.f;  // from nothing: 0
            s_nref[r] = now;
          }
          p8_meet<kMeet>(bar);
          if constexpr (C::kWarpSums) {
#pragma unroll
            for (int i = 0; i < C::kSums; ++i) l[i] *= s_alpha[first + kStep * i + lane / (32 / kStep)];
          } else if (!fresh) {
#pragma unroll
            for (int i = 0; i < M; i += 4) {
              const float4 a = *reinterpret_cast<const float4*>(&s_alpha[first + i]);
              l[i] *= a.x;
              l[i + 1] *= a.y;
              l[i + 2] *= a.z;
              l[i + 3] *= a.w;
            }
          }
          if constexpr (C::kKeep) {
#pragma unroll
            for (int i = 0; i < M; ++i) nrefs[i] = s_nref[first + i];
          }
          if (part == 0 && j > 0) {
            if (!p8_wait(&o_done[(step - 1u) & 1u], ((step - 1u) >> 1) & 1u)) failed = true;
            __syncwarp();
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll 1
            for (int r = 0; r < M; r += kStep) {
              float o[kStep];
              p8_ld<kStep>(to + r, o);
#pragma unroll
              for (int i = 0; i < kStep; i += 4) {
                const float4 a = *reinterpret_cast<const float4*>(&s_alpha[first + r + i]);
                o[i] *= a.x;
                o[i + 1] *= a.y;
                o[i + 2] *= a.z;
                o[i + 3] *= a.w;
              }
              p8_st<kStep>(to + r, o);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          }
          if constexpr (C::kSteps > 1) break;  // the scores are loaded again for the weights
          if (fresh) {
#pragma unroll
            for (int i = 0; i < kStep; i += 4) {
              const float4 n4 = *reinterpret_cast<const float4*>(&s_nref[first + i]);
              x[i] += n4.x;
              x[i + 1] += n4.y;
              x[i + 2] += n4.z;
              x[i + 3] += n4.w;
            }
            break;
          }
        }
        if (!ok) break;
        if (step >= C::kWs) {  // the product that read the buffer before is done
          if (!p8_wait(&o_done[(step - C::kWs) & 1u], ((step - C::kWs) >> 1) & 1u)) failed = true;
          __syncwarp();
        }
        if (there) {
          unsigned char* wrow = sw + (step % C::kWs * kPar + part) * C::kW + row * C::kRowW;
          const int turn = C::kRowW == 128 ? row & 7 : C::kRowW == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
          const uint64_t vs = at_pair(value_scale, value_scale);
#pragma unroll
          for (int r = 0; r < M; r += kStep) {
            if constexpr (C::kSteps > 1) load(r, true);
            float sums[kStep];
            uint32_t h[kStep / 2];
#pragma unroll
            for (int i = 0; i < kStep; i += 2) {
              float a = at_exp2(x[i]), b = at_exp2(x[i + 1]);
              if constexpr (C::kWarpSums) {
                sums[i] = a;
                sums[i + 1] = b;
              } else {
                at_unpair(at_add2(at_pair(l[r + i], l[r + i + 1]), at_pair(a, b)), l[r + i], l[r + i + 1]);
              }
              at_unpair(p8_mul2(at_pair(a, b), vs), a, b);
              h[i / 2] = p8_pack(a, b);
            }
            if constexpr (C::kWarpSums) l[r / kStep] += p8_warp_sums(sums, lane);
#pragma unroll
            for (int c = 0; c < kStep / 8; ++c) {
              const int at = first + r + 8 * c, atom = at / C::kAtom, piece = at % C::kAtom / 8;
              *reinterpret_cast<uint4*>(wrow + atom * (kPaKeys * 128) + ((piece ^ turn) << 4)) =
                  make_uint4(h[4 * c], h[4 * c + 1], h[4 * c + 2], h[4 * c + 3]);
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMA reads the weights through the async proxy
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&w_full[step & 1u]);
      }
      if (!ok) break;
      g -= kPar * ((sg.nblk + kPar - 1) / kPar) - sg.nblk;  // the blocks of the last step that were not there
      // the sums over the keys, while the last product runs: by warps, then over the warps
      if constexpr (C::kWarpSums) {
#pragma unroll
        for (int i = 0; i < C::kSums; ++i)
          if (lane % (32 / kStep) == 0) s_red[four][first + kStep * i + lane / (32 / kStep)] = l[i];
      } else {
        const float sum = p8_warp_sums(l, lane);
        if (lane % (32 / M) == 0) s_red[four][first + lane / (32 / M)] = sum;
      }
      ok = !p8_any<kMeet>(bar, failed);
      if (!ok) break;
      const bool whole = sg.nblk == sg.nb;
      const size_t unit = 2 * static_cast<size_t>(blockIdx.x) + (sg.j0 == 0 ? 1 : 0);
      if (mine < M) {
        const int r = first + mine;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4 * kPar; ++i) sum += s_red[i][r];
        float inv = 1.f / sum;
        if (sum == 0.f && pre == 0 && r < p.R) {  // no visible key at all: zero; visible keys of weight 0 alone: NaN
          bool any = false;
          for (int c = 0; c < p.n; ++c) any = any || ((s_sees[qb][c] >> s_node[r]) & 1ull);
          if (!any) inv = 0.f;
        }
        s_alpha[r] = whole ? inv : 1.f;
        if (!whole && r < p.R) {
          const float nref = s_nref[r];
          *reinterpret_cast<float2*>(p.ml + 2 * (unit * p.R + r)) = make_float2(nref == kAtNone ? -INFINITY : -nref, sum);
        }
      }
      if (!p8_wait(&o_done[(step - 1u) & 1u], ((step - 1u) >> 1) & 1u)) failed = true;
      ok = !p8_any<kMeet>(bar, failed);
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      unsigned short* out = p.out + (static_cast<size_t>(sg.b) * p.n * p.Hq + sg.kvh * p.G) * D + (column & ~1);
      float* partial = p.part + unit * p.R * D + (column & ~1);
      const bool bad = *reinterpret_cast<volatile int*>(&s_bad) > si;  // (a later segment's mark counts too: only slower)
      constexpr int kOut = C::kOut;
      const int from = M / kPar * part;
#pragma unroll 1
      for (int i0 = from; i0 < from + M / kPar; i0 += kOut) {
        float o[kOut];
        __syncwarp();
        p8_ld<kOut>(to + i0, o);
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        if (first + i0 >= p.R) continue;
        if (__builtin_expect(bad && has_column, 0)) {  // rare: NaN among the nodes' codes
#pragma unroll 1
          for (int c = 0; c < p.n; ++c) {
            const int key = pre + c;
            if (key < sg.j0 * kPaKeys || key >= (sg.j0 + sg.nblk) * kPaKeys) continue;
            const int page = p.page_table[static_cast<size_t>(sg.b) * p.max_pages + (key >> p.page_shift)];
            if (page < 0 || page >= p.num_pages) continue;
            const size_t at = (static_cast<size_t>(page) * p.Hkv + sg.kvh) * p.page_size + (key & (p.page_size - 1));
            if ((p.v_cache[at * D + column] & 0x7Fu) != 0x7Fu) continue;
            const unsigned long long nodes = s_sees[qb][c];
#pragma unroll
            for (int i = 0; i < kOut; ++i)
              if ((nodes >> s_node[first + i0 + i]) & 1ull) o[i] = NAN;
          }
        }
        // lanes 8 apart hold neighbouring columns: one of them takes both of a row, the other those of the next row
        const bool odd = (lane & 8) != 0;
#pragma unroll
        for (int i = 0; i < kOut; i += 2) {
          const int r = first + i0 + i + (odd ? 1 : 0);
          const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? o[i] : o[i + 1], 8);
          const float lo = odd ? got : o[i], hi = odd ? o[i + 1] : got, by = s_alpha[r];
          if (r >= p.R || !has_column) continue;
          if (whole) *reinterpret_cast<uint32_t*>(out + s_at[r]) = at_pack(lo * by, hi * by);
          else *reinterpret_cast<float2*>(partial + r * D) = make_float2(lo, hi);
        }
      }
      // (what the next segment's raise writes is behind its first meeting, and that behind this)
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[qb]);  // through with the segment's factors, mask and outputs
      if (whole) continue;
      // the pair's last segment to finish joins them all, once the CTA is through its share
      const int c0 = pa_owner(sg.pair0, W, ctas), c1 = pa_owner(sg.pair0 + sg.nb - 1, W, ctas);
      const bool met = pa_sync(&s_meet, meet, lane);  // the ticket's release covers what the other warps wrote before it
      ok = !p8_any<kMeet>(bar, !met);
      if (!ok) break;
      if (t == 32 * C::kSoftmax) {
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
    // copies issued must land before the CTA leaves: wait for the last of each entry too (bounded)
    for (unsigned kv = 0; kv < 2; ++kv)
      for (unsigned i = s_issued[kv] > stages / 2 ? s_issued[kv] - stages / 2 : 0u; i < s_issued[kv]; ++i)
        mbar_wait(&kv_full[(2 * i + kv) % stages], ((2 * i + kv) / stages) & 1u, kAtBudgetNs);
  }
  if (ok) {
    // the ticket's thread acquired the others' partials; the barrier above passed them on
    for (int i = 0; i < s_joins; ++i) {
      PaSum* red = reinterpret_cast<PaSum*>(skv);  // the ring is empty by now
      if (p.R * (D / 4) <= kThreads) pa_join<D, 1, kThreads>(p, s_join[i], red);
      else pa_join<D, kThreads <= 640 ? 4 : 2, kThreads>(p, s_join[i], red);
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

template <int D, int N, int M, int kPar_, int kStep_>
dt_status pa8_launch(Pa8Params& p, const Pa8Maps& maps, WsHeader* hdr, cudaStream_t stream) {
  using C = P8<D, N, M, kPar_, kStep_>;
  const size_t fixed = C::kFixed + align_up(sizeof(int) * (2 * p.B + 1), 16);
  const int fit = static_cast<int>((kPa8SmemCap - fixed) / C::kEntry);
  // an even number: a slot then always holds keys or always values
  p.stages = (fit > kP8MaxStages ? kP8MaxStages : fit) & ~1;
  const size_t smem = fixed + static_cast<size_t>(p.stages) * C::kEntry;
  if (ensure_dynamic_smem(reinterpret_cast<const void*>(paged_attn8_kernel<D, N, M, kPar_, kStep_>), kPa8SmemCap) != cudaSuccess)
    return DT_ERR_CUDA;
  return at_launch(paged_attn8_kernel<D, N, M, kPar_, kStep_>, p.grid, C::kThreads, smem, stream, p, maps, hdr);
}
// By the rows R = G n that share a head. Columns of the products: the next of 16, 32, 64 and 128 (16 is what the weights'
// layout allows). Softmax: two blocks a step wherever tensor memory holds two steps of their scores (not beside 128 rows),
// because a step waits more than it computes; and so many rows a thread that its warps find their registers. Measured in
// us, 32 query and 8 key/value heads, pages of 64, lengths from a 32nd of the largest up, D = 128 and D = 64:
//   R <= 8 (64 requests of up to 8191 keys): two blocks a step 92.9 and 74; one 94.1 and 82.8
//   R <= 16 (3 nodes each, up to 4099): two blocks, eight rows at once 64.4 and 57.1; sixteen 66.8 and 67.7; four blocks
//     69.3 and 63.8
//   R <= 32 (8 nodes): two blocks, 16 rows a thread 80.9 and 74.5; one block 95.8 and 86.5; 32 rows a thread 82.8 and 83.8
//   R <= 64 (16 nodes): two blocks, 32 rows a thread, sixteen at once 113.5 and 101.5; eight at once 115.1 and 107.3; one
//     block 120.0 and 116.1; 16 rows a thread 139.8 and 131.4
//   R <= 128 (32 requests of 32 nodes): 32 rows a thread, sixteen at once 102.8 and 95.0; eight at once 106.4 and 99.2 (in an
//     earlier form at D = 128, 64 rows a thread 148 where 32 took 134; 16 rows are more warps than a CTA has)
template <int D>
dt_status pa8_pick(Pa8Params& p, const Pa8Maps& maps, WsHeader* hdr, cudaStream_t stream) {
  if (p.R <= 8) return pa8_launch<D, 16, 8, 2, 8>(p, maps, hdr, stream);
  if (p.R <= 16) return pa8_launch<D, 16, 16, 2, 8>(p, maps, hdr, stream);
  if (p.R <= 32) return pa8_launch<D, 32, 16, 2, 8>(p, maps, hdr, stream);
  if (p.R <= 64) return pa8_launch<D, 64, 32, 2, 16>(p, maps, hdr, stream);
  return pa8_launch<D, 128, 32, 1, 16>(p, maps, hdr, stream);
}

}  // namespace
}  // namespace dt

extern "C" size_t dt_paged_attention8_workspace_bytes(int B, int n, int Hq, int Hkv, int d) {
  if (B < 1 || n < 1 || Hq < 1 || Hkv < 1 || d < 1 || Hq % Hkv != 0) return 0;
  const long long R = static_cast<long long>(Hq / Hkv) * n;
  if (R > dt::kPaRows || d > 256) return 0;  // outside the envelope
  dt::DeviceInfo di{};
  if (dt::current_device_info(&di) != cudaSuccess) return 0;
  return dt::pa_plan(static_cast<int>(R), d, di.sms).bytes;
}

extern "C" dt_status dt_paged_attention8(int B, int n, int Hq, int Hkv, int d, const void* q, const void* k_cache,
                                         const void* v_cache, const float* k_scale, const float* v_scale,
                                         dt_dtype dtype, int num_pages, int page_size, int scale_block,
                                         const int32_t* page_table, int max_pages, const int32_t* lens,
                                         const uint8_t* mask, float scale, void* out, void* workspace,
                                         size_t workspace_bytes, cudaStream_t stream) {
  using namespace dt;
  if (B < 0 || n < 1 || Hq < 1 || Hkv < 1 || d < 1 || Hq % Hkv != 0 || num_pages < 1 || page_size < 1 || max_pages < 1 ||
      scale_block < 1)
    return DT_ERR_INVALID_ARG;
  if (dtype != DT_F32 && dtype != DT_BF16) return DT_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale * 1.4426950408889634f)) return DT_ERR_INVALID_ARG;
  if (B == 0) return DT_OK;
  const void* ptrs[] = {q, k_cache, v_cache, out, workspace};
  for (const void* x : ptrs)
    if (!x || !aligned16(x)) return DT_ERR_INVALID_ARG;
  const void* words[] = {page_table, lens, k_scale, v_scale};
  for (const void* x : words)
    if (!x || (reinterpret_cast<uintptr_t>(x) & 3u)) return DT_ERR_INVALID_ARG;
  const int G = Hq / Hkv;
  if (dtype != DT_BF16 || (d != 64 && d != 128)) return DT_ERR_UNSUPPORTED;
  if (n > kPaNodes || static_cast<long long>(G) * n > kPaRows || B > DT_PAGED_MAX_BATCH) return DT_ERR_UNSUPPORTED;
  if (Hq > DT_MAX_HEADS) return DT_ERR_UNSUPPORTED;
  if (page_size < DT_MIN_PAGE || page_size > DT_MAX_PAGE || (page_size & (page_size - 1))) return DT_ERR_UNSUPPORTED;
  if (scale_block < DT_MIN_PAGE || scale_block > page_size || (scale_block & (scale_block - 1)))
    return DT_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_pages) * page_size > INT_MAX || static_cast<long long>(num_pages) * Hkv > INT_MAX)
    return DT_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size > DT_PAGED_MAX_TOKENS) return DT_ERR_UNSUPPORTED;
  DeviceInfo di{};
  if (current_device_info(&di) != cudaSuccess) return DT_ERR_CUDA;
  const PaPlan P = pa_plan(G * n, d, di.sms);
  if (workspace_bytes < P.bytes) return DT_ERR_INVALID_ARG;
  Pa8Params p{};
  p.B = B; p.n = n; p.Hq = Hq; p.Hkv = Hkv; p.G = G; p.R = G * n; p.grid = P.grid;
  p.extra = kP8Extra;
  p.page_size = page_size; p.num_pages = num_pages; p.max_pages = max_pages;
  while ((1 << p.page_shift) < page_size) ++p.page_shift;
  while ((1 << p.block_shift) < scale_block) ++p.block_shift;
  // Measured in us (64 requests of up to 8191 keys, a token each), a third warp for boxes and two: pages of 16 98.8 and 103.9,
  // at d = 64 89.8 and 98.3; pages of 32 96.2 and 96.7, 81.8 and 82.6.
  p.third = page_size <= 16 ? 1 : 0;
  p.q = static_cast<const unsigned short*>(q);
  p.v_cache = static_cast<const unsigned char*>(v_cache);
  p.k_scale = k_scale; p.v_scale = v_scale;
  p.page_table = page_table; p.lens = lens; p.mask = mask;
  p.scale_log2 = scale * 1.4426950408889634f;
  char* ws = static_cast<char*>(workspace);
  p.part = reinterpret_cast<float*>(ws + P.part);
  p.ml = reinterpret_cast<float*>(ws + P.ml);
  p.out = static_cast<unsigned short*>(out);
  Pa8Maps maps{};
  const uint64_t planes = static_cast<uint64_t>(num_pages) * static_cast<uint64_t>(Hkv);
  const uint32_t box = page_size < kPaKeys ? static_cast<uint32_t>(page_size) : kPaKeys;
  if (!encode_u8_rows(&maps.k, k_cache, static_cast<uint64_t>(d), static_cast<uint64_t>(page_size), planes, box) ||
      !encode_u8_rows(&maps.v, v_cache, static_cast<uint64_t>(d), static_cast<uint64_t>(page_size), planes, box))
    return DT_ERR_CUDA;
  WsHeader* hdr = reinterpret_cast<WsHeader*>(ws);
  return d == 64 ? pa8_pick<64>(p, maps, hdr, stream) : pa8_pick<128>(p, maps, hdr, stream);
}
