// What the attention kernels over the paged cache and over prompts share: packed fp32 arithmetic, loads and stores of
// tensor memory by 16 rows a warp, waits.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dt_internal.cuh"
#include "umma.cuh"

namespace dt {
namespace {

// Weights are powers of two relative to a reference: a row's maximum as last raised, and 2^kAtShift more, so that they
// start out at 2^-26 and a row's later keys may exceed the maximum by a headroom of 2^kAtLazy before it is raised. bf16
// and fp32 hold such weights with the relative rounding of weights below 1. The shift makes room for the sums: of
// 2^24 keys of weight 2^kAtMost with values of 2^100 (10^30) in size they stay finite in fp32, and products of weights
// with values of 2^-100 are normal numbers still.
constexpr float kAtLazy = 20.f, kAtShift = 26.f, kAtMost = kAtLazy - kAtShift;
constexpr double kAtValueMost = 1e30;  // as the public header states it
constexpr double kAtWeightMost = 1.0 / 64;
static_assert(kAtMost == -6.f, "log2 of kAtWeightMost");
// minus a reference that has seen nothing: any finite score raises it, a score of -inf has no weight under it, and NaN
// stays
constexpr float kAtNone = 3e38f;
constexpr uint64_t kAtBudgetNs = 4000000000ull;

// These kernels are launched so that their set-up (barriers, tensor memory, descriptors) may run while the kernel
// before them in the stream ends; everything they read or write in global memory comes after this. The kernel after
// them may be set up as soon as every CTA has come here; it waits for this one's end in the same way.
__device__ __forceinline__ void at_launch_order() {
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
}
template <class Kernel, class... Args>
inline dt_status at_launch(Kernel kernel, int grid, int threads, size_t smem, cudaStream_t stream,
                           const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, args...));
}

__device__ __forceinline__ float at_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float at_rcp(float x) {  // off by at most 2^-23 of it; 0 gives infinity
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t at_pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Pairs of fp32 in one 64-bit register: the packed FMA and add issue once for two elements.
__device__ __forceinline__ uint64_t at_pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void at_unpair(uint64_t d, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(d));
}
__device__ __forceinline__ uint64_t at_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t at_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float at_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Tensor memory by 16 lanes (rows) a warp: in each group of 8 columns thread l holds columns 2 (l % 4) and + 1 of rows
// l / 4 and l / 4 + 8 (v[4 g], v[4 g + 1], then v[4 g + 2], v[4 g + 3]). Each load waits for itself.
__device__ __forceinline__ void at_ld_s(uint32_t taddr, float (&v)[64]) {  // 16 groups: a block's scores
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,"
      "%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,"
      "%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]), "=f"(v[32]),
        "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]), "=f"(v[40]),
        "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]), "=f"(v[48]),
        "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]), "=f"(v[56]),
        "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void at_ld_half(uint32_t taddr, float (&v)[32]) {  // 8 groups
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
      "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void at_ld_o(uint32_t taddr, float (&v)[16]) {  // 4 groups
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void at_st_o(uint32_t taddr, const float* v) {  // 4 groups, as at_ld_o holds them
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
// The weights of 64 keys: a pair of bf16 per 32-bit column, so a group's two values of a row are one column.
__device__ __forceinline__ void at_st_p(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// A block's 128 scores as at_ld_s holds them: the thread's part of its two rows' maxima, scaled.
__device__ __forceinline__ void at_max(const float (&s)[64], float scale, float (&mx)[2]) {
#pragma unroll
  for (int k2 = 0; k2 < 2; ++k2) {
    float u = fmaxf(s[2 * k2], s[2 * k2 + 1]), w = fmaxf(s[2 * k2 + 4], s[2 * k2 + 5]);
#pragma unroll
    for (int g = 2; g < 16; g += 2) {
      u = at_max3(u, s[4 * g + 2 * k2], s[4 * g + 2 * k2 + 1]);
      w = at_max3(w, s[4 * g + 4 + 2 * k2], s[4 * g + 5 + 2 * k2]);
    }
    mx[k2] = fmaxf(u, w) * scale;
  }
}
// Raises the references of a warp's rows (nref: minus them) where a block's maxima leave the headroom; alpha: what the
// sums and outputs so far are multiplied by.
__device__ __forceinline__ void at_raise(float (&mx)[2], float (&nref)[2], float (&l)[2], float (&alpha)[2]) {
#pragma unroll
  for (int k2 = 0; k2 < 2; ++k2) {
    mx[k2] = fmaxf(mx[k2], __shfl_xor_sync(0xFFFFFFFFu, mx[k2], 1));
    mx[k2] = fmaxf(mx[k2], __shfl_xor_sync(0xFFFFFFFFu, mx[k2], 2));
    const bool raise = mx[k2] + nref[k2] > kAtMost;
    const float to = -mx[k2] - kAtShift;
    alpha[k2] = raise ? at_exp2(to - nref[k2]) : 1.f;  // from nothing: 0
    l[k2] *= alpha[k2];
    if (raise) nref[k2] = to;
  }
}
// The weights of half a block (64 keys), rounded to bf16 pairs; their sums are taken before the rounding.
template <int kHalf>
__device__ __forceinline__ void at_weights(const float (&s)[64], float scale, const float (&nref)[2], uint64_t (&ls)[4],
                                           uint32_t (&pk)[16]) {
  const uint64_t scale2 = at_pair(scale, scale);
  const uint64_t nref2[2] = {at_pair(nref[0], nref[0]), at_pair(nref[1], nref[1])};
#pragma unroll
  for (int c = 0; c < 16; ++c) {  // group 8 kHalf + c / 2, row c % 2
    const int at = 32 * kHalf + 2 * c;
    float a, b;
    at_unpair(at_fma2(at_pair(s[at], s[at + 1]), scale2, nref2[c & 1]), a, b);
    a = at_exp2(a);
    b = at_exp2(b);
    ls[c & 3] = at_add2(ls[c & 3], at_pair(a, b));
    pk[c] = at_pack(a, b);
  }
}
__device__ __forceinline__ void at_sums(const uint64_t (&ls)[4], float (&l)[2]) {
#pragma unroll
  for (int k2 = 0; k2 < 2; ++k2) {
    float a, b;
    at_unpair(at_add2(ls[k2], ls[k2 + 2]), a, b);
    l[k2] += a + b;
  }
}
// Four groups (32 columns) of one of the thread's two rows as bf16: four threads hold the four words of each 16 bytes,
// transposed among them so that thread `quad` of the four returns the 16 bytes of group `quad`.
__device__ __forceinline__ uint4 at_row16(const float* o, int k2, float factor, int quad) {
  uint32_t x[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) x[g] = at_pack(o[4 * g + 2 * k2] * factor, o[4 * g + 2 * k2 + 1] * factor);
#pragma unroll
  for (int g = 0; g < 4; g += 2) {
    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, quad & 1 ? x[g] : x[g + 1], 1);
    if (quad & 1) x[g] = got;
    else x[g + 1] = got;
  }
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, quad & 2 ? x[g] : x[g + 2], 2);
    if (quad & 2) x[g] = got;
    else x[g + 2] = got;
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// A phase that has ended is seen at once (45 cycles; the form with a time limit takes 100). Otherwise a wait in long
// sleeps: the hardware wakes the warp when the phase ends; a warp that polls takes issue slots from those that compute.
__device__ __forceinline__ bool at_try_wait(uint64_t* bar, unsigned parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool at_wait(uint64_t* bar, unsigned parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!at_try_wait(bar, parity))
    if (global_timer_ns() - t0 > kAtBudgetNs) return false;
  return true;
}

// Whether the phase has ended, without waiting.
__device__ __forceinline__ bool at_test(uint64_t* bar, unsigned parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// Waits until the loader has issued more than `e` ring entries (its count, in shared memory). A waiter that skips
// entries calls this before it waits for entry e's phase: by then the phase before, of the other parity, is over. It
// may have skipped a whole share (many long caches that end with a block): the time runs from the loader's last step.
__device__ __forceinline__ bool at_issued(const unsigned* count, unsigned e) {
  const volatile unsigned* seen = count;
  unsigned now = *seen;
  if (now > e) return true;
  uint64_t t0 = global_timer_ns();
  while (true) {
    const unsigned was = now;
    now = *seen;
    if (now > e) return true;
    if (now != was) t0 = global_timer_ns();
    if (global_timer_ns() - t0 > kAtBudgetNs) return false;
    __nanosleep(100);
  }
}

}  // namespace
}  // namespace dt
