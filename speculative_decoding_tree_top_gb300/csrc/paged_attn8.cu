// dt_paged_attention8 — attention of each request's newest tokens over its paged cache in 8 bits with scales.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "attn_common.cuh"
#include "paged_share.cuh"

namespace dt {
namespace {

struct Pa8Params : PaWork {
  int block;                        // rows of a page that share a scale
  const unsigned short* q;
  const unsigned char *k_cache, *v_cache;
  const float *k_scale, *v_scale;   // [num_pages][Hkv][page_size / block]
  float scale;
};

__device__ __forceinline__ float code_value(unsigned char c) {
  uint32_t two;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(static_cast<uint16_t>(c)));
  return __low2float(*reinterpret_cast<const __half2*>(&two));
}

// One query row a CTA, 128 keys at a time: a thread a key for the scores, a thread a column for the sums.
template <int D>
__global__ void __launch_bounds__(128) paged_attn8_kernel(Pa8Params p, WsHeader* hdr) {
  __shared__ float s_q[D], s_p[128], s_red[4];
  __shared__ size_t s_row[128];
  at_launch_order();
  const int t = threadIdx.x;
  const int h = blockIdx.x % p.Hq, node = blockIdx.x / p.Hq % p.n, b = blockIdx.x / p.Hq / p.n, kvh = h / p.G;
  unsigned short* out = p.out + ((static_cast<size_t>(b) * p.n + node) * p.Hq + h) * D;
  bool bad = false;
  const int len = pa_length(p, b, &bad);
  if (bad && t == 0) record_error(hdr, DT_ERR_INVALID_ARG);
  if (t < D) s_q[t] = __uint_as_float(static_cast<uint32_t>(p.q[out - p.out + t]) << 16);
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int k0 = 0; k0 < len; k0 += 128) {
    const int key = k0 + t;
    bool seen = key < len;
    if (seen && key >= len - p.n) {
      const int c = key - (len - p.n);
      seen = p.mask ? p.mask[(static_cast<size_t>(b) * p.n + node) * p.n + c] != 0 : c <= node;
    }
    float s = -INFINITY;
    __syncthreads();
    if (seen) {
      int page = p.page_table[static_cast<size_t>(b) * p.max_pages + key / p.page_size];
      if (page < 0 || page >= p.num_pages) {
        record_error(hdr, DT_ERR_INVALID_ARG);
        page = 0;
      }
      const int row = key % p.page_size;
      const size_t plane = static_cast<size_t>(page) * p.Hkv + kvh, at = plane * p.page_size + row;
      const size_t sc = plane * (p.page_size / p.block) + row / p.block;
      s = 0.f;
      for (int e = 0; e < D; ++e) s += s_q[e] * code_value(p.k_cache[at * D + e]);
      s *= p.k_scale[sc] * p.scale * 1.4426950408889634f;
      s_row[t] = at;
    }
    float mx = s;
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, x));
    if (t % 32 == 0) s_red[t / 32] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    const float now = fmaxf(m, mx), ref = now == -INFINITY ? 0.f : now, a = exp2f(m - ref);
    m = now;
    const float w = seen ? exp2f(s - ref) : 0.f;
    float sum = w;
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
    __syncthreads();
    if (t % 32 == 0) s_red[t / 32] = sum;
    s_p[t] = seen ? w : -1.f;
    __syncthreads();
    l = l * a + (s_red[0] + s_red[1]) + (s_red[2] + s_red[3]);
    o *= a;
    if (t < D)
      for (int j = 0; j < 128; ++j)
        if (!(s_p[j] < 0.f)) {
          const size_t at = s_row[j], plane = at / p.page_size;
          const float vs = p.v_scale[plane * (p.page_size / p.block) + at % p.page_size / p.block];
          o += s_p[j] * vs * code_value(p.v_cache[at * D + t]);
        }
  }
  const bool none = l == 0.f && m == -INFINITY;
  if (t < D) out[t] = static_cast<unsigned short>(at_pack(none ? 0.f : o / l, 0.f));
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
  p.page_size = page_size; p.num_pages = num_pages; p.max_pages = max_pages; p.block = scale_block;
  p.q = static_cast<const unsigned short*>(q);
  p.k_cache = static_cast<const unsigned char*>(k_cache);
  p.v_cache = static_cast<const unsigned char*>(v_cache);
  p.k_scale = k_scale; p.v_scale = v_scale;
  p.page_table = page_table; p.lens = lens; p.mask = mask; p.scale = scale;
  p.out = static_cast<unsigned short*>(out);
  WsHeader* hdr = static_cast<WsHeader*>(workspace);
  return d == 64 ? at_launch(paged_attn8_kernel<64>, B * n * Hq, 128, 0, stream, p, hdr)
                 : at_launch(paged_attn8_kernel<128>, B * n * Hq, 128, 0, stream, p, hdr);
}
