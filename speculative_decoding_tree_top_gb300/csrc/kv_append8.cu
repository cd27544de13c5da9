// dt_kv_append8 — new tokens' keys and values into a paged cache in e4m3, a scale for each block of rows and head.
//
// A block of `block` rows of a page stores x as code * scale, scale = 2^e with the least e (from -48 to 48) that brings
// the block's largest finite element to 448 or less. Powers of two: a code's rounding is relative whatever the scale is,
// so a finer scale would gain nothing but the last bit of the range, and a block whose scale grows is coded again by a
// change of exponents, exactly but for codes that leave e4m3's normal range.
//
// The tokens of one block have to be seen together. A block is worked on where its lowest written row's token is (its
// leader): `who` holds the token of each of its rows, found by a look at all slots of the call when those are few, and
// otherwise through an index from slots to tokens that a launch before fills. An entry of the index counts if the token
// that it names has that slot, so the index needs no clearing, and what an earlier call left there does no harm.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>

#include "attn_common.cuh"
#include "rotate.cuh"

namespace dt {
namespace {

constexpr int kA8Threads = 256;
constexpr int kA8Warps = kA8Threads / 32;
constexpr int kA8Scan = 2048;    // up to so many tokens every CTA looks at all slots
constexpr int kA8Chunk = 16;     // tokens of a CTA that uses the index
constexpr int kE4m3Most = 448;
constexpr int kScaleLow = DT_SCALE_LOW, kScaleHigh = DT_SCALE_HIGH;

struct Append8Params {
  int N, Hq, Hkv, max_pos, half, interleaved, page_size, block;  // half = rot / 2
  int chunk, chunks;                                             // tokens a key/value CTA looks after; such CTAs
  long long slots_end;                                           // num_pages * page_size
  const unsigned short *q, *k, *v;
  long long q_stride, k_stride, v_stride;  // elements between tokens
  const int32_t *slots, *positions;
  const float* rope;  // [max_pos][2 half]: cosines, then sines
  unsigned short *out_q, *out_k;
  unsigned char *k_cache, *v_cache;
  float *k_scale, *v_scale;  // [num_pages][Hkv][page_size / block]
  int32_t* index;            // [slots_end], or null: look at all slots
};

// A token's slot, -1 for one that is left out.
__device__ __forceinline__ int a8_slot(const Append8Params& p, int t, bool* bad) {
  const int slot = p.slots[t];
  if (slot < 0) return -1;
  const int pos = p.half ? p.positions[t] : 0;
  if (slot >= p.slots_end || (p.half && (pos < 0 || pos >= p.max_pos))) {
    *bad = true;
    return -1;
  }
  return slot;
}

__global__ void __launch_bounds__(kA8Threads) append8_index_kernel(Append8Params p) {
  at_launch_order();
  const int t = blockIdx.x * kA8Threads + threadIdx.x;
  bool bad = false;
  const int slot = t < p.N ? a8_slot(p, t, &bad) : -1;
  if (slot >= 0) p.index[slot] = t;
}

// An item of 16 columns of one row in fp32, rotated. (No contraction: the largest element decides a scale, and should
// not depend on how a compiler pairs products and sums.)
struct Item {
  Eight a, b;
};
__device__ __forceinline__ void a8_turn(float& a, float& b, float c, float s) {
  const float u = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)), w = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = u;
  b = w;
}
__device__ __forceinline__ Item a8_item(const Append8Params& p, const unsigned short* src, const TurnCols& cols,
                                        int item, int pos, bool turned) {
  Item x;
  x.a = unpack8(*reinterpret_cast<const uint4*>(src + cols.ca));
  x.b = unpack8(*reinterpret_cast<const uint4*>(src + cols.cb));
  if (turned) {
    Turn tu;
    load_turn(p.rope + static_cast<size_t>(pos) * (2 * p.half), item, p.half, p.interleaved, cols.halves, tu);
    if (cols.halves) {
#pragma unroll
      for (int i = 0; i < 8; ++i) a8_turn(x.a.x[i], x.b.x[i], tu.c[i], tu.s[i]);
    } else if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (cols.ca < 2 * p.half) a8_turn(x.a.x[2 * i], x.a.x[2 * i + 1], tu.c[i], tu.s[i]);
        if (cols.cb < 2 * p.half) a8_turn(x.b.x[2 * i], x.b.x[2 * i + 1], tu.c[4 + i], tu.s[4 + i]);
      }
    }
  }
  return x;
}

// The bits of the largest |x| that a scale serves: they order as the values do. What is larger, infinite or no number is
// stored as NaN and leaves the block's scale alone.
constexpr unsigned kMostBits = (static_cast<unsigned>(kScaleHigh + 8 + 127) << 23) | 0x600000u;  // 448 2^kScaleHigh
__device__ __forceinline__ unsigned a8_most(const Eight& e, unsigned most) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const unsigned u = __float_as_uint(e.x[i]) & 0x7FFFFFFFu;
    if (u <= kMostBits && u > most) most = u;
  }
  return most;
}
// The least e within the limits with most <= 448 2^e.
__device__ __forceinline__ int a8_exponent(unsigned most) {
  const int k = static_cast<int>(most >> 23) - 127;  // most = m 2^k, 1 <= m < 2; 448 = 1.75 2^8
  const int e = (most & 0x7FFFFFu) > 0x600000u ? k - 7 : k - 8;
  return e < kScaleLow ? kScaleLow : e > kScaleHigh ? kScaleHigh : e;
}
__device__ __forceinline__ float a8_pow2(int e) { return __uint_as_float(static_cast<unsigned>(e + 127) << 23); }
// A stored scale's exponent; kScaleLow - 1 if it is none that this call gives.
__device__ __forceinline__ int a8_exponent_of(float scale) {
  const unsigned u = __float_as_uint(scale);
  const int e = static_cast<int>(u >> 23) - 127;  // a negative scale has e > kScaleHigh
  return (u & 0x7FFFFFu) == 0u && e >= kScaleLow && e <= kScaleHigh ? e : kScaleLow - 1;
}
__device__ __forceinline__ uint32_t a8_code2(float lo, float hi) {
  // what is not finite, or too large for the largest scale, is stored as NaN
  if (!(fabsf(lo) <= static_cast<float>(kE4m3Most))) lo = NAN;
  if (!(fabsf(hi) <= static_cast<float>(kE4m3Most))) hi = NAN;
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint2 a8_code8(const Eight& e, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = a8_code2(e.x[2 * i] * inv, e.x[2 * i + 1] * inv);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}
// Four codes under a scale 2^up times as large.
__device__ __forceinline__ uint32_t a8_again(uint32_t codes, float down) {
  uint32_t out = 0u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t two;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(static_cast<uint16_t>(codes >> (16 * h))));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
    out |= a8_code2(f.x * down, f.y * down) << (16 * h);
  }
  return out;
}

// One head's keys or values of a block, by a warp: D / 16 lanes a row.
template <int D>
__device__ __forceinline__ void a8_block(const Append8Params& p, const int* who, int low, int first_slot, int head,
                                         bool is_k) {
  constexpr int kItems = D / 16, kRows = 32 / kItems;
  const int lane = threadIdx.x & 31, item = lane % kItems, row0 = lane / kItems;
  const bool turned = is_k && p.half > 0;
  const TurnCols cols = turned ? turn_cols(item, p.half, p.interleaved) : TurnCols{16 * item, 16 * item + 8, false};
  const unsigned short* src = (is_k ? p.k : p.v) + head * D;
  const long long stride = is_k ? p.k_stride : p.v_stride;
  unsigned short* dense = is_k ? p.out_k : nullptr;
  const int page = first_slot / p.page_size, row_at = first_slot % p.page_size;
  const size_t plane = static_cast<size_t>(page) * p.Hkv + head;
  unsigned char* cache = (is_k ? p.k_cache : p.v_cache) + (plane * p.page_size + row_at) * D;
  float* scale = (is_k ? p.k_scale : p.v_scale) + plane * (p.page_size / p.block) + row_at / p.block;
  const int from = low / kRows * kRows;
  unsigned most = 0u;
  for (int r = from + row0; r < p.block; r += kRows) {
    const int t = who[r];
    if (t == INT_MAX) continue;
    const Item x = a8_item(p, src + t * stride, cols, item, turned ? p.positions[t] : 0, turned);
    most = a8_most(x.b, a8_most(x.a, most));
  }
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  int e = a8_exponent(most);
  const int was = low > 0 ? a8_exponent_of(*scale) : kScaleLow - 1;
  if (was > e) e = was;
  __syncwarp();  // every lane has read the scale
  if (lane == 0) *scale = a8_pow2(e);
  if (was >= kScaleLow && e > was) {  // the rows that are there already
    const float down = a8_pow2(was - e);
    for (int r = row0; r < low; r += kRows) {
      uint4* at = reinterpret_cast<uint4*>(cache + r * D + 16 * item);
      const uint4 c = *at;
      *at = make_uint4(a8_again(c.x, down), a8_again(c.y, down), a8_again(c.z, down), a8_again(c.w, down));
    }
  }
  const float inv = a8_pow2(-e);
  for (int r = from + row0; r < p.block; r += kRows) {
    const int t = who[r];
    if (t == INT_MAX) continue;
    const Item x = a8_item(p, src + t * stride, cols, item, turned ? p.positions[t] : 0, turned);
    *reinterpret_cast<uint2*>(cache + r * D + cols.ca) = a8_code8(x.a, inv);
    *reinterpret_cast<uint2*>(cache + r * D + cols.cb) = a8_code8(x.b, inv);
    if (dense) {
      unsigned short* o = dense + (static_cast<size_t>(t) * p.Hkv + head) * D;
      *reinterpret_cast<uint4*>(o + cols.ca) = pack8(x.a);
      *reinterpret_cast<uint4*>(o + cols.cb) = pack8(x.b);
    }
  }
}

// CTAs 0 .. chunks - 1: the keys and values of the blocks whose leaders are among the CTA's tokens. The others: queries.
template <int D>
__global__ void __launch_bounds__(kA8Threads) kv_append8_kernel(Append8Params p, WsHeader* hdr) {
  extern __shared__ int s_who[];  // [chunk][block]: the token of each row, INT_MAX for none
  __shared__ int s_low[kA8Chunk], s_first[kA8Chunk];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  at_launch_order();
  if (static_cast<int>(blockIdx.x) >= p.chunks) {
    constexpr int kItems = D / 16;
    const int item = t % kItems, head0 = t / kItems, step = kA8Threads / kItems;
    const TurnCols cols = p.half ? turn_cols(item, p.half, p.interleaved) : TurnCols{16 * item, 16 * item + 8, false};
    for (long long token = blockIdx.x - p.chunks; token < p.N; token += gridDim.x - p.chunks) {
      bool bad = false;
      if (a8_slot(p, static_cast<int>(token), &bad) < 0) continue;
      for (int h = head0; h < p.Hq; h += step) {
        const Item x = a8_item(p, p.q + token * p.q_stride + h * D, cols, item, p.half ? p.positions[token] : 0,
                               p.half > 0);
        unsigned short* o = p.out_q + (token * p.Hq + h) * D;
        *reinterpret_cast<uint4*>(o + cols.ca) = pack8(x.a);
        *reinterpret_cast<uint4*>(o + cols.cb) = pack8(x.b);
      }
    }
    return;
  }
  for (int i = t; i < p.chunk * p.block; i += kA8Threads) s_who[i] = INT_MAX;
  __syncthreads();
  const int token0 = blockIdx.x * p.chunk;
  for (int c = warp; c < p.chunk; c += kA8Warps) {  // a warp a token
    bool bad = false;
    const int token = token0 + c, slot = token < p.N ? a8_slot(p, token, &bad) : -1;
    if (bad && lane == 0) record_error(hdr, DT_ERR_INVALID_ARG);
    if (lane == 0) {
      s_low[c] = p.block;
      s_first[c] = slot < 0 ? -1 : slot / p.block * p.block;
    }
  }
  __syncthreads();
  if (p.index) {
    for (int c = warp; c < p.chunk; c += kA8Warps) {
      const int first = s_first[c];
      if (first < 0) continue;
      for (int r = lane; r < p.block; r += 32) {
        const int u = p.index[first + r];
        bool bad = false;
        if (u >= 0 && u < p.N && a8_slot(p, u, &bad) == first + r) {
          s_who[c * p.block + r] = u;
          atomicMin(&s_low[c], r);
        }
      }
    }
  } else {
    for (int u = t; u < p.N; u += kA8Threads) {
      bool bad = false;
      const int slot = a8_slot(p, u, &bad);
      if (slot < 0) continue;
      for (int c = 0; c < p.chunk; ++c)
        if (s_first[c] >= 0 && slot / p.block * p.block == s_first[c]) {
          atomicMin(&s_who[c * p.block + slot % p.block], u);
          atomicMin(&s_low[c], slot % p.block);
        }
    }
  }
  __syncthreads();
  for (int i = warp; i < p.chunk * 2 * p.Hkv; i += kA8Warps) {
    const int c = i / (2 * p.Hkv), part = i % (2 * p.Hkv);
    if (s_first[c] < 0 || s_low[c] >= p.block) continue;
    if (s_who[c * p.block + s_low[c]] != token0 + c) continue;  // another token leads
    a8_block<D>(p, s_who + c * p.block, s_low[c], s_first[c], part >> 1, (part & 1) == 0);
  }
}

inline size_t a8_bytes(int N, int num_pages, int page_size) {
  const size_t index = N > kA8Scan ? sizeof(int32_t) * static_cast<size_t>(num_pages) * page_size : 0;
  return align_up(align_up(sizeof(WsHeader)) + index);
}

}  // namespace
}  // namespace dt

extern "C" size_t dt_kv_append8_workspace_bytes(int N, int num_pages, int page_size) {
  if (N < 0 || num_pages < 1 || page_size < 1) return 0;
  return dt::a8_bytes(N, num_pages, page_size);
}

extern "C" dt_status dt_kv_append8(int N, int Hq, int Hkv, int d, const void* q, int64_t q_stride, const void* k,
                                   int64_t k_stride, const void* v, int64_t v_stride, dt_dtype dtype,
                                   const int32_t* slots, const int32_t* positions, const float* rope, int max_pos,
                                   int rot, int interleaved, void* out_q, void* out_k, void* k_cache, void* v_cache,
                                   float* k_scale, float* v_scale, int num_pages, int page_size, int scale_block,
                                   void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  using namespace dt;
  if (N < 0 || Hq < 0 || Hkv < 1 || d < 1 || num_pages < 1 || page_size < 1 || scale_block < 1 || rot < 0 || rot > d ||
      rot % 2 != 0)
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
  const void* words[] = {slots, k_scale, v_scale};
  for (const void* x : words)
    if (!x || (reinterpret_cast<uintptr_t>(x) & 3u)) return DT_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(positions) & 3u) return DT_ERR_INVALID_ARG;
  if (workspace_bytes < sizeof(WsHeader)) return DT_ERR_INVALID_ARG;
  if (Hq > DT_MAX_HEADS || Hkv > DT_MAX_HEADS || N > INT_MAX / 2) return DT_ERR_UNSUPPORTED;
  const int64_t width[3] = {static_cast<int64_t>(Hq) * d, static_cast<int64_t>(Hkv) * d, static_cast<int64_t>(Hkv) * d};
  const int64_t stride[3] = {q_stride, k_stride, v_stride};
  for (int i = 0; i < 3; ++i)
    if ((i > 0 || Hq > 0) && (stride[i] < width[i] || stride[i] % 8 != 0 || stride[i] > INT_MAX))
      return DT_ERR_INVALID_ARG;
  if (dtype != DT_BF16 || (d != 64 && d != 128) || rot % 16 != 0) return DT_ERR_UNSUPPORTED;
  if (page_size < DT_MIN_PAGE || page_size > DT_MAX_PAGE || (page_size & (page_size - 1))) return DT_ERR_UNSUPPORTED;
  if (scale_block < DT_MIN_PAGE || scale_block > page_size || (scale_block & (scale_block - 1)))
    return DT_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_pages) * page_size > INT_MAX || static_cast<long long>(num_pages) * Hkv > INT_MAX)
    return DT_ERR_UNSUPPORTED;
  if (workspace_bytes < a8_bytes(N, num_pages, page_size)) return DT_ERR_INVALID_ARG;
  DeviceInfo di{};
  if (current_device_info(&di) != cudaSuccess) return DT_ERR_CUDA;
  Append8Params p{};
  p.N = N; p.Hq = Hq; p.Hkv = Hkv; p.max_pos = max_pos; p.half = rot / 2; p.interleaved = interleaved;
  p.page_size = page_size; p.block = scale_block;
  p.slots_end = static_cast<long long>(num_pages) * page_size;
  p.q = static_cast<const unsigned short*>(q);
  p.k = static_cast<const unsigned short*>(k);
  p.v = static_cast<const unsigned short*>(v);
  p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
  p.slots = slots; p.positions = positions; p.rope = rope;
  p.out_q = static_cast<unsigned short*>(out_q);
  p.out_k = static_cast<unsigned short*>(out_k);
  p.k_cache = static_cast<unsigned char*>(k_cache);
  p.v_cache = static_cast<unsigned char*>(v_cache);
  p.k_scale = k_scale; p.v_scale = v_scale;
  const bool indexed = N > kA8Scan;
  p.index = indexed ? reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + align_up(sizeof(WsHeader))) : nullptr;
  p.chunk = indexed ? kA8Chunk : 1;
  p.chunks = (N + p.chunk - 1) / p.chunk;
  WsHeader* hdr = static_cast<WsHeader*>(workspace);
  if (indexed) {
    const dt_status s = at_launch(append8_index_kernel, (N + kA8Threads - 1) / kA8Threads, kA8Threads, 0, stream, p);
    if (s != DT_OK) return s;
  }
  const int cap = 16 * di.sms, grid = p.chunks + (Hq > 0 ? (N < cap ? N : cap) : 0);
  const size_t smem = sizeof(int) * static_cast<size_t>(p.chunk) * scale_block;
  return d == 64 ? at_launch(kv_append8_kernel<64>, grid, kA8Threads, smem, stream, p, hdr)
                 : at_launch(kv_append8_kernel<128>, grid, kA8Threads, smem, stream, p, hdr);
}
