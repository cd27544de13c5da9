// dt_kv_append — new tokens' keys and values into a paged cache, rotated by their positions on the way.
//
// Rotary position embedding (Su et al., arXiv 2104.09864): a head's first `rot` elements are rot / 2 pairs, pair i
// turned by the angle position * f_i whose cosine and sine the caller's table holds (so any frequency schedule works):
//     (a, b) -> (a cos - b sin, b cos + a sin),
// the pairs being (x_i, x_{i + rot/2}) or, interleaved, (x_{2i}, x_{2i+1}). Everything is fp32 until the one rounding
// to bf16; elements past `rot` and the values are copied.
//
// Bound by memory: every input byte is read once and every output byte written once. One CTA takes a token at a time:
// an item is 32 bytes of one head (two groups of eight elements, paired so that a rotation never leaves the thread),
// and a thread's items all sit in the same columns of their heads, so it keeps its cosines and sines in registers
// across the token's heads. A (token, head) row is d contiguous elements in the cache, written in full 16-byte pieces.
// Measured (16384 tokens, 32/8 heads, d = 128, scattered slots, 445 MB): 72 us, 6.2 TB/s, 91% of the copy rate. Before
// its launch overlapped the kernel before: 74; a grid of exactly the resident CTAs 87, two heads' loads in flight a
// thread 84 (72 registers), fewer registers 80 to 90.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>

#include "append_shape.cuh"
#include "attn_common.cuh"
#include "rotate.cuh"

namespace dt {
namespace {

constexpr int kAppendPerSm = 2048;    // threads per SM that the grid is sized to: half again what fits (48 registers)

struct AppendParams {
  int N, Hq, Hkv, max_pos, half, interleaved, page_size;  // half = rot / 2
  long long slots_end;                                     // num_pages * page_size
  const unsigned short *q, *k, *v;
  long long q_stride, k_stride, v_stride;  // elements between tokens
  const int32_t *slots, *positions;
  const float* rope;  // [max_pos][2 half]: cosines, then sines
  unsigned short *out_q, *out_k, *k_cache, *v_cache;
};

// A head's part of a token: where its item comes from and goes to.
struct AppendHead {
  const unsigned short* src;
  unsigned short *dst, *dst2;  // dst2: the keys' dense copy, or null
  bool turned;
};
template <int D>
__device__ __forceinline__ AppendHead append_head(const AppendParams& p, int t, int h, size_t row) {
  AppendHead a;
  a.dst2 = nullptr;
  a.turned = true;
  if (h < p.Hq) {
    a.src = p.q + t * p.q_stride + h * D;
    a.dst = p.out_q + (static_cast<size_t>(t) * p.Hq + h) * D;
  } else {
    const bool is_k = h < p.Hq + p.Hkv;
    const int g = h - p.Hq - (is_k ? 0 : p.Hkv);
    a.src = (is_k ? p.k + t * p.k_stride : p.v + t * p.v_stride) + g * D;
    a.dst = (is_k ? p.k_cache : p.v_cache) + (row + static_cast<size_t>(g) * p.page_size) * D;
    if (is_k && p.out_k) a.dst2 = p.out_k + (static_cast<size_t>(t) * p.Hkv + g) * D;
    a.turned = is_k;
  }
  return a;
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(AppendParams p, WsHeader* hdr) {
  constexpr int kItems = D / 16;                                  // items per head
  const int step = static_cast<int>(blockDim.x) / kItems;         // heads a pass of the CTA covers
  const int item = threadIdx.x % kItems, head0 = threadIdx.x / kItems;
  const TurnCols cols = turn_cols(item, p.half, p.interleaved);
  const bool halves = cols.halves;
  const int ca = cols.ca, cb = cols.cb;
  const int heads = p.Hq + 2 * p.Hkv;
  at_launch_order();
  // a token's slot and position are read while the token before it is on its way
  int t = blockIdx.x;
  int slot_next = t < p.N ? p.slots[t] : -1, pos_next = p.half && t < p.N ? p.positions[t] : 0;
  for (; t < p.N; t += gridDim.x) {
    const int slot = slot_next, pos = pos_next;
    const long long after = static_cast<long long>(t) + gridDim.x;
    if (after < p.N) {
      slot_next = p.slots[after];
      if (p.half) pos_next = p.positions[after];
    }
    if (slot < 0) continue;  // a padding token: nothing of it is read or written
    if (slot >= p.slots_end || (p.half && (pos < 0 || pos >= p.max_pos))) {
      if (threadIdx.x == 0) record_error(hdr, DT_ERR_INVALID_ARG);
      continue;
    }
    Turn tu;
    if (p.half) load_turn(p.rope + static_cast<size_t>(pos) * (2 * p.half), item, p.half, p.interleaved, halves, tu);
    const size_t row = static_cast<size_t>(slot / p.page_size) * p.Hkv * p.page_size + slot % p.page_size;
    for (int h = head0; h < heads; h += step) {
      const AppendHead hd = append_head<D>(p, t, h, row);
      uint4 a = *reinterpret_cast<const uint4*>(hd.src + ca), b = *reinterpret_cast<const uint4*>(hd.src + cb);
      if (hd.turned) {
        if (halves) {
          turn_halves(a, b, tu);
        } else if (p.interleaved) {  // a group past rot is copied: its bits stay as they are
          if (ca < 2 * p.half) turn_pairs(a, tu.c, tu.s);
          if (cb < 2 * p.half) turn_pairs(b, tu.c + 4, tu.s + 4);
        }
      }
      *reinterpret_cast<uint4*>(hd.dst + ca) = a;
      *reinterpret_cast<uint4*>(hd.dst + cb) = b;
      if (hd.dst2) {
        *reinterpret_cast<uint4*>(hd.dst2 + ca) = a;
        *reinterpret_cast<uint4*>(hd.dst2 + cb) = b;
      }
    }
  }
}

}  // namespace
}  // namespace dt

extern "C" dt_status dt_kv_append(int N, int Hq, int Hkv, int d, const void* q, int64_t q_stride, const void* k,
                                  int64_t k_stride, const void* v, int64_t v_stride, dt_dtype dtype,
                                  const int32_t* slots, const int32_t* positions, const float* rope, int max_pos,
                                  int rot, int interleaved, void* out_q, void* out_k, void* k_cache, void* v_cache,
                                  int num_pages, int page_size, void* workspace, size_t workspace_bytes,
                                  cudaStream_t stream) {
  using namespace dt;
  if (N < 0 || Hq < 0 || Hkv < 1 || d < 1 || num_pages < 1 || page_size < 1 || rot < 0 || rot > d || rot % 2 != 0)
    return DT_ERR_INVALID_ARG;
  if (dtype != DT_F32 && dtype != DT_BF16) return DT_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return DT_ERR_INVALID_ARG;
  if (N == 0) return DT_OK;
  if ((Hq > 0) != (q != nullptr) || (Hq > 0) != (out_q != nullptr)) return DT_ERR_INVALID_ARG;
  if (rot > 0 && (!rope || !positions || max_pos < 1)) return DT_ERR_INVALID_ARG;
  const void* ptrs[] = {k, v, k_cache, v_cache, workspace};
  for (const void* x : ptrs)
    if (!x || !aligned16(x)) return DT_ERR_INVALID_ARG;
  const void* opts[] = {q, out_q, out_k, rope};
  for (const void* x : opts)
    if (!aligned16(x)) return DT_ERR_INVALID_ARG;
  if (!slots || (reinterpret_cast<uintptr_t>(slots) & 3u) || (reinterpret_cast<uintptr_t>(positions) & 3u))
    return DT_ERR_INVALID_ARG;
  if (workspace_bytes < sizeof(WsHeader)) return DT_ERR_INVALID_ARG;
  if (Hq > DT_MAX_HEADS || Hkv > DT_MAX_HEADS || N > INT_MAX / 2) return DT_ERR_UNSUPPORTED;
  const int64_t width[3] = {static_cast<int64_t>(Hq) * d, static_cast<int64_t>(Hkv) * d, static_cast<int64_t>(Hkv) * d};
  const int64_t stride[3] = {q_stride, k_stride, v_stride};
  for (int i = 0; i < 3; ++i)
    if ((i > 0 || Hq > 0) && (stride[i] < width[i] || stride[i] % 8 != 0 || stride[i] > INT_MAX))
      return DT_ERR_INVALID_ARG;
  if (dtype != DT_BF16 || (d != 64 && d != 128) || rot % 16 != 0) return DT_ERR_UNSUPPORTED;
  if (page_size < DT_MIN_PAGE || page_size > DT_MAX_PAGE || (page_size & (page_size - 1))) return DT_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_pages) * page_size > INT_MAX) return DT_ERR_UNSUPPORTED;
  DeviceInfo di{};
  if (current_device_info(&di) != cudaSuccess) return DT_ERR_CUDA;
  AppendParams p{};
  p.N = N; p.Hq = Hq; p.Hkv = Hkv; p.max_pos = max_pos; p.half = rot / 2; p.interleaved = interleaved;
  p.page_size = page_size;
  p.slots_end = static_cast<long long>(num_pages) * page_size;
  p.q = static_cast<const unsigned short*>(q);
  p.k = static_cast<const unsigned short*>(k);
  p.v = static_cast<const unsigned short*>(v);
  p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
  p.slots = slots; p.positions = positions; p.rope = rope;
  p.out_q = static_cast<unsigned short*>(out_q);
  p.out_k = static_cast<unsigned short*>(out_k);
  p.k_cache = static_cast<unsigned short*>(k_cache);
  p.v_cache = static_cast<unsigned short*>(v_cache);
  const int threads = append_threads(Hq + 2 * Hkv, d / 16);
  const int cap = kAppendPerSm / threads * di.sms, grid = N < cap ? N : cap;
  WsHeader* hdr = static_cast<WsHeader*>(workspace);
  return d == 64 ? at_launch(kv_append_kernel<64>, grid, threads, 0, stream, p, hdr)
                 : at_launch(kv_append_kernel<128>, grid, threads, 0, stream, p, hdr);
}
