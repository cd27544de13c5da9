// dt_kv_append8 — new tokens' keys and values into a paged cache in e4m3, a scale for each block of rows and head.
//
// A block of `block` rows of a page stores x as code * scale, scale = 2^e with the least e (from -48 to 48) that brings
// the block's largest finite element to 448 or less. Powers of two: a code's rounding is relative whatever the scale is,
// so a finer scale would gain nothing but the last bit of the range, and a block whose scale grows is coded again by a
// change of exponents, exactly but for codes that leave e4m3's normal range.
//
// The tokens of one block have to be seen together. A block is worked on where its lowest written row's token is (its
// leader), by a warp a head and side; `who` holds the token of each of its rows. It is found by a look at all slots of the
// call when those are few. Otherwise a launch before fills an index from slots to tokens, and a row's token is looked for
// first where it is when tokens are in order, then in the index. An entry of the index counts if the token that it names
// has that slot, so the index needs no clearing, and what an earlier call left there does no harm.
//
// Bound by memory when it is large: rows are read once, codes, scales and rotated queries written once. Measured (16384
// tokens, 32/8 heads, d = 128, 411 MB): 84 us, 4.9 TB/s, 72% of the copy rate; the queries' part alone 43, that of keys and
// values 48, whose CTAs are chains of loads (slots, index, rows) and hold the rest up: the two share the SMs, but not
// wholly. One kind of CTA for all took 90, rows kept in registers over both passes 189 (100 registers). 64 trees of 16
// nodes: 15 us, of which the index's launch is 3; one token: 4.4, a chain of loads (slot and position, rows, maximum, scale,
// codes) where the bf16 append takes 1.8.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>

#include "attn_common.cuh"
#include "rotate.cuh"

namespace dt {
namespace {

constexpr int kA8Threads = 256;
constexpr int kA8Warps = kA8Threads / 32;
constexpr int kA8PerSm = 5;      // CTAs: 48 registers a thread
// Up to so many tokens every CTA looks at all slots, past it a launch before makes an index. Measured (32/8 heads, d = 128,
// pages of 16), looks and index: 256 tokens 8.8 and 10.3 us, 512 11.3 and 12.3, 1024 15.5 and 14.5, 2048 21.1 and 18.0
// (since then 11.1 and, with the index, 11.8 at 513, 14.0, 17.6).
constexpr int kA8Scan = 512;
constexpr int kA8Chunk = 16;     // tokens that a CTA looks after, at most
constexpr int kA8TileBytes = 4096;  // of rows as they come, for each warp
constexpr size_t kA8Smem = kA8Warps * kA8TileBytes + kA8Chunk * DT_MAX_PAGE * sizeof(int2) +
                          2 * kA8TileBytes;  // at most
constexpr int kScaleLow = DT_SCALE_LOW, kScaleHigh = DT_SCALE_HIGH;

struct Append8Params {
  int N, Hq, Hkv, max_pos, half, interleaved;                    // half = rot / 2
  int page_shift, block_shift;                                   // log2 of a page's rows, of a block's
  int chunk, kv_ctas, q_ctas;                                    // tokens a key/value CTA looks after; CTAs of each kind
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

// A token as the arrays have it: its slot, -1 for one that is left out, and its position. Both are loaded at once, and
// several tokens' before any is looked at: a CTA's first microseconds are a chain of such loads.
struct A8Token {
  int slot, pos;
};
__device__ __forceinline__ A8Token a8_fetch(const Append8Params& p, int t, bool there) {
  A8Token x{-1, 0};
  if (there) {
    x.slot = p.slots[t];
    if (p.half) x.pos = p.positions[t];
  }
  return x;
}
__device__ __forceinline__ int a8_slot(const Append8Params& p, const A8Token& x, bool* bad) {
  if (x.slot < 0) return -1;
  if (x.slot >= p.slots_end || x.pos < 0 || (p.half && x.pos >= p.max_pos)) {
    *bad = true;
    return -1;
  }
  return x.slot;
}

__global__ void __launch_bounds__(kA8Threads) append8_index_kernel(Append8Params p) {
  at_launch_order();
  const int t = blockIdx.x * kA8Threads + threadIdx.x;
  bool bad = false;
  const int slot = a8_slot(p, a8_fetch(p, t, t < p.N), &bad);
  if (slot >= 0) p.index[slot] = t;
}

// Eight columns of one row in fp32, rotated: two groups of four, a half-split head's the two halves of four pairs. The
// products and sums are paired as written here, not as a compiler likes: the largest element decides a scale.
struct Cols {
  int a, b;     // the groups' first columns
  int pair;     // the first of their pairs, -1: not rotated
};
__device__ __forceinline__ Cols a8_cols(int item, int half, int interleaved) {
  if (interleaved || 4 * item >= half) {  // eight columns in a row; half is a multiple of 8, so they turn together
    const int at = interleaved ? 8 * item : 2 * half + 8 * (item - half / 4);
    return Cols{at, at + 4, interleaved && at < 2 * half ? 4 * item : -1};
  }
  return Cols{4 * item, 4 * item + half, 4 * item};
}
__device__ __forceinline__ uint64_t a8_mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Two pairs: (a, b) -> (a c - b s, b c + a s), each a product and a fused one.
__device__ __forceinline__ void a8_turn2(float& a0, float& a1, float& b0, float& b1, float c0, float c1, float s0,
                                         float s1) {
  const uint64_t a = at_pair(a0, a1), b = at_pair(b0, b1), c = at_pair(c0, c1);
  at_unpair(at_fma2(b, at_pair(-s0, -s1), a8_mul2(a, c)), a0, a1);
  at_unpair(at_fma2(a, at_pair(s0, s1), a8_mul2(b, c)), b0, b1);
}
__device__ __forceinline__ void a8_rotate(Eight& x, const float4& c, const float4& s, bool interleaved) {
  if (interleaved) {
    a8_turn2(x.x[0], x.x[2], x.x[1], x.x[3], c.x, c.y, s.x, s.y);
    a8_turn2(x.x[4], x.x[6], x.x[5], x.x[7], c.z, c.w, s.z, s.w);
  } else {
    a8_turn2(x.x[0], x.x[1], x.x[4], x.x[5], c.x, c.y, s.x, s.y);
    a8_turn2(x.x[2], x.x[3], x.x[6], x.x[7], c.z, c.w, s.z, s.w);
  }
}
__device__ __forceinline__ float4 a8_shared4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}

// The largest size that a scale serves, 448 2^kScaleHigh. What is larger, infinite or no number is stored as NaN and leaves
// the block's scale alone.
constexpr unsigned kMostBits = (static_cast<unsigned>(kScaleHigh + 8 + 127) << 23) | 0x600000u;
// The largest |x|, infinite ones among them.
__device__ __forceinline__ float a8_most(const Eight& e, float most) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) most = at_max3(most, fabsf(e.x[i]), fabsf(e.x[i + 1]));
  return most;
}
// The largest that a scale serves.
__device__ __forceinline__ float a8_most_served(const Eight& e, float most) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (fabsf(e.x[i]) <= __uint_as_float(kMostBits)) most = fmaxf(most, fabsf(e.x[i]));
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
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t a8_code4(const float* x, float inv) {
  const uint64_t by = at_pair(inv, inv);
  float a, b, c, d;
  at_unpair(a8_mul2(at_pair(x[0], x[1]), by), a, b);
  at_unpair(a8_mul2(at_pair(x[2], x[3]), by), c, d);
  return a8_code2(a, b) | a8_code2(c, d) << 16;
}
__device__ __forceinline__ void a8_drop(Eight& e) {  // what no scale serves
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (!(fabsf(e.x[i]) <= __uint_as_float(kMostBits))) e.x[i] = NAN;
}
// Four codes under a scale 1 / down times as large.
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

// One head's keys or values of a block, by a warp: D / 8 lanes a row. A tile of rows at a time comes to shared memory as they
// are and is read from there twice, for the scale and for the codes (kept in registers, they were either few loads in
// flight or spilled); a block of more rows is gone through twice.
template <int D>
struct A8 {
  static constexpr int kItems = D / 8, kRows = 32 / kItems, kTile = kA8TileBytes / (2 * D);
};
// A head's rows of a block, from r0 on, to the warp's tile.
template <int D>
__device__ __forceinline__ void a8_load(const Append8Params& p, const int2* who, int r0, int head, bool is_k,
                                        unsigned char* tile) {
  constexpr int kItems = A8<D>::kItems, kRows = A8<D>::kRows;
  const int lane = threadIdx.x & 31, item = lane % kItems, row0 = lane / kItems, block = 1 << p.block_shift;
  const unsigned short* src = (is_k ? p.k : p.v) + head * D + 8 * item;
  const long long stride = is_k ? p.k_stride : p.v_stride;
  const uint32_t to = smem_u32(tile) + (row0 * D + 8 * item) * 2;
#pragma unroll
  for (int u = 0; u < A8<D>::kTile; u += kRows) {
    const int r = r0 + u + row0, t = r < block ? who[r].x : INT_MAX;
    if (t != INT_MAX)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + u * D * 2), "l"(src + t * stride) : "memory");
  }
}
// kKind: values (or keys that are not rotated) 0; keys whose rows' parts of the rotation's table are in shared memory at
// `turns`, row by row, and whose first tile is there if `loaded`: 1; keys that read the table: 2.
template <int D, int kKind, bool kDense>
__device__ __forceinline__ void a8_block(const Append8Params& p, const int2* who, int low, int first_slot, int head,
                                         bool is_k, unsigned char* tile, uint32_t turns, bool loaded) {
  constexpr int kItems = A8<D>::kItems, kRows = A8<D>::kRows, kTile = A8<D>::kTile;
  const int lane = threadIdx.x & 31, item = lane % kItems, row0 = lane / kItems;
  const Cols cols = kKind ? a8_cols(item, p.half, p.interleaved) : Cols{8 * item, 8 * item + 4, -1};
  const bool turned = kKind && cols.pair >= 0;
  const int page = first_slot >> p.page_shift, row_at = first_slot & ((1 << p.page_shift) - 1);
  const size_t plane = static_cast<size_t>(page) * p.Hkv + head;
  unsigned char* cache = (is_k ? p.k_cache : p.v_cache) + ((plane << p.page_shift) + row_at) * D;
  float* scale = (is_k ? p.k_scale : p.v_scale) + (plane << (p.page_shift - p.block_shift)) + (row_at >> p.block_shift);
  const int block = 1 << p.block_shift, from = low & ~(kTile - 1), rot = 2 * p.half;
  const unsigned short* own = reinterpret_cast<const unsigned short*>(tile) + row0 * D;  // the lane's first row of a tile
  const int rows = block < kTile ? block : kTile;
  auto load = [&](int r0) {
    a8_load<D>(p, who, r0, head, is_k, tile);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
  };
  auto item_of = [&](int u, int pos) {  // of the tile's row u + row0
    Eight x;
    if constexpr (kKind == 0) {
      x = unpack8(*reinterpret_cast<const uint4*>(own + u * D + 8 * item));
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(own + u * D + cols.a);
      const uint2 b = *reinterpret_cast<const uint2*>(own + u * D + cols.b);
      x = unpack8(make_uint4(a.x, a.y, b.x, b.y));
      if (turned) {
        if constexpr (kKind == 1) {
          const uint32_t at = turns + ((u + row0) * rot + cols.pair) * 4;
          a8_rotate(x, a8_shared4(at), a8_shared4(at + 2 * rot), p.interleaved);
        } else {
          const float* at = p.rope + static_cast<size_t>(pos) * rot + cols.pair;
          a8_rotate(x, *reinterpret_cast<const float4*>(at), *reinterpret_cast<const float4*>(at + p.half), p.interleaved);
        }
      }
    }
    return x;
  };
  const float was_scale = low > 0 ? *scale : 0.f;
  float most = 0.f;
  bool odd = false;  // something that no scale serves
  unsigned bits;
#pragma unroll 1
  while (true) {
#pragma unroll 1
    for (int r0 = from; r0 < block; r0 += kTile) {
      if ((!odd && !loaded) || block > kTile) load(r0);
      const int2* w = who + r0 + row0;
#pragma unroll 4
      for (int u = 0; u < rows; u += kRows) {
        const int2 token = w[u];
        if (token.x == INT_MAX) continue;
        const Eight x = item_of(u, token.y);
        if (__builtin_expect(odd, 0)) most = a8_most_served(x, most);
        else most = a8_most(x, most);
      }
      if (block > kTile) __syncwarp();  // the tile is read before the next one comes
    }
    bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most));
    if (odd || bits <= kMostBits) break;
    odd = true;  // rare: once more, without what is not served
    most = 0.f;
  }
  int e = a8_exponent(bits);
  const int was = low > 0 ? a8_exponent_of(was_scale) : kScaleLow - 1;
  if (was > e) e = was;
  __syncwarp();  // every lane has read the scale
  if (lane == 0) *scale = a8_pow2(e);
  if (was >= kScaleLow && e > was) {  // the rows that are there already
    const float down = a8_pow2(was - e);
    for (int r = row0; r < low; r += kRows) {
      uint2* at = reinterpret_cast<uint2*>(cache + r * D + 8 * item);
      const uint2 c = *at;
      *at = make_uint2(a8_again(c.x, down), a8_again(c.y, down));
    }
  }
  const float inv = a8_pow2(-e);
#pragma unroll 1
  for (int r0 = from; r0 < block; r0 += kTile) {
    if (block > kTile) load(r0);
    const int2* w = who + r0 + row0;
    unsigned char* to = cache + (r0 + row0) * D;
#pragma unroll 4
    for (int u = 0; u < rows; u += kRows) {
      const int2 token = w[u];
      if (token.x == INT_MAX) continue;
      Eight x = item_of(u, token.y);
      if (kDense && is_k) {
        unsigned short* o = p.out_k + (static_cast<size_t>(token.x) * p.Hkv + head) * D;
        const uint4 y = pack8(x);
        *reinterpret_cast<uint2*>(o + cols.a) = make_uint2(y.x, y.y);
        *reinterpret_cast<uint2*>(o + cols.b) = make_uint2(y.z, y.w);
      }
      if (__builtin_expect(odd, 0)) a8_drop(x);
      if constexpr (kKind == 0) {
        *reinterpret_cast<uint2*>(to + u * D + 8 * item) = make_uint2(a8_code4(x.x, inv), a8_code4(x.x + 4, inv));
      } else {
        *reinterpret_cast<uint32_t*>(to + u * D + cols.a) = a8_code4(x.x, inv);
        *reinterpret_cast<uint32_t*>(to + u * D + cols.b) = a8_code4(x.x + 4, inv);
      }
    }
    __syncwarp();  // the tile is read before the next one comes
  }
}

// The dense row of a head's key whose token another one of the same slot keeps out of the cache: as a8_block writes the
// others'. Rare. A lane reads and writes the same columns: the row may be the key's own.
template <int D>
__device__ __noinline__ void a8_dense(const Append8Params& p, int token, int head) {
  const int item = threadIdx.x & 31;
  if (item >= A8<D>::kItems) return;
  const Cols cols = p.half ? a8_cols(item, p.half, p.interleaved) : Cols{8 * item, 8 * item + 4, -1};
  const unsigned short* src = p.k + token * p.k_stride + head * D;
  const uint2 a = *reinterpret_cast<const uint2*>(src + cols.a), b = *reinterpret_cast<const uint2*>(src + cols.b);
  Eight x = unpack8(make_uint4(a.x, a.y, b.x, b.y));
  if (cols.pair >= 0) {
    const float* at = p.rope + static_cast<size_t>(p.positions[token]) * (2 * p.half) + cols.pair;
    a8_rotate(x, *reinterpret_cast<const float4*>(at), *reinterpret_cast<const float4*>(at + p.half), p.interleaved);
  }
  unsigned short* o = p.out_k + (static_cast<size_t>(token) * p.Hkv + head) * D;
  const uint4 y = pack8(x);
  *reinterpret_cast<uint2*>(o + cols.a) = make_uint2(y.x, y.y);
  *reinterpret_cast<uint2*>(o + cols.b) = make_uint2(y.z, y.w);
}

// Two kinds of CTAs, in turn, so that they share the SMs: those of keys and values compute while those of queries wait for
// memory. Keys (the even ones of their kind) or values: of the blocks whose leaders are among the CTA's tokens. Queries: a
// token or several at a time, each thread in the same columns of its heads (as dt_kv_append). kDense: keys go to out_k as
// well (an instance for both spills more: trees without out_k 15.5 us where theirs takes 15.0; prompts with it 83.3, 83.4).
template <int D, bool kDense>
__global__ void __launch_bounds__(kA8Threads, kA8PerSm) kv_append8_kernel(Append8Params p, WsHeader* hdr) {
  extern __shared__ __align__(16) unsigned char s_tiles[];  // a tile a warp
  // [chunk][block]: the token of each row, INT_MAX for none, and its position
  int2* s_who = reinterpret_cast<int2*>(s_tiles + kA8Warps * kA8TileBytes);
  __shared__ int s_low[kA8Chunk], s_first[kA8Chunk], s_lead[kA8Chunk];
  __shared__ int s_slot[kA8Chunk], s_lost[kA8Chunk];  // kDense: the tokens' slots, and whether another of a slot is kept
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, block = 1 << p.block_shift;
  at_launch_order();
  const int both = 2 * (p.kv_ctas < p.q_ctas ? p.kv_ctas : p.q_ctas), b = blockIdx.x;
  const bool queries = b < both ? (b & 1) != 0 : p.q_ctas > p.kv_ctas;
  const int cta = b < both ? b >> 1 : b - both / 2;  // among its kind
  if (queries) {
    constexpr int kItems = D / 16, kStep = kA8Threads / kItems;
    const int item = t % kItems, tokens = p.Hq < kStep ? kStep / p.Hq : 1;
    const int mine = t / kItems / p.Hq;  // of the tokens of a pass
    if (mine >= tokens && p.Hq < kStep) return;
    const int head0 = p.Hq < kStep ? t / kItems % p.Hq : t / kItems;
    const TurnCols cols = p.half ? turn_cols(item, p.half, p.interleaved) : TurnCols{16 * item, 16 * item + 8, false};
    const long long stride = static_cast<long long>(p.q_ctas) * tokens;
    long long token = static_cast<long long>(cta) * tokens + (p.Hq < kStep ? mine : 0);
    int slot_next = token < p.N ? p.slots[token] : -1, pos_next = p.half && token < p.N ? p.positions[token] : 0;
    for (; token < p.N; token += stride) {
      const int slot = slot_next, pos = pos_next;
      const long long after = token + stride;
      if (after < p.N) {
        slot_next = p.slots[after];
        if (p.half) pos_next = p.positions[after];
      }
      if (slot < 0 || slot >= p.slots_end || (p.half && (pos < 0 || pos >= p.max_pos))) continue;
      Turn tu;
      if (p.half)
        load_turn(p.rope + static_cast<size_t>(pos) * (2 * p.half), item, p.half, p.interleaved, cols.halves, tu);
      for (int h = head0; h < p.Hq; h += kStep) {
        const unsigned short* src = p.q + token * p.q_stride + h * D;
        uint4 a = *reinterpret_cast<const uint4*>(src + cols.ca), b = *reinterpret_cast<const uint4*>(src + cols.cb);
        if (cols.halves) {
          turn_halves(a, b, tu);
        } else if (p.half && p.interleaved) {  // a group past rot is copied: its bits stay as they are
          if (cols.ca < 2 * p.half) turn_pairs(a, tu.c, tu.s);
          if (cols.cb < 2 * p.half) turn_pairs(b, tu.c + 4, tu.s + 4);
        }
        unsigned short* o = p.out_q + (static_cast<size_t>(token) * p.Hq + h) * D;
        *reinterpret_cast<uint4*>(o + cols.ca) = a;
        *reinterpret_cast<uint4*>(o + cols.cb) = b;
      }
    }
    return;
  }
  const int token0 = (cta >> 1) * p.chunk;
  const bool is_k = (cta & 1) == 0;
  // a look at all slots: under way before it is known what for
  constexpr int kLooks = kA8Scan / kA8Threads;
  int look[kLooks];
  if (!p.index) {
#pragma unroll
    for (int i = 0; i < kLooks; ++i) look[i] = t + i * kA8Threads < p.N ? p.slots[t + i * kA8Threads] : -1;
  }
  for (int i = t; i < p.chunk << p.block_shift; i += kA8Threads) s_who[i] = make_int2(INT_MAX, 0);
  if (t < p.chunk) {
    bool bad = false;
    const int token = token0 + t;
    const A8Token own = a8_fetch(p, token, token < p.N);
    const A8Token last = a8_fetch(p, token - 1, token > 0 && token <= p.N);
    const int slot = a8_slot(p, own, &bad);
    if (bad) record_error(hdr, DT_ERR_INVALID_ARG);
    // the token before it in the row before it: it does not lead, as most do not
    bool other = false;
    const bool follows = slot > 0 && (slot & (block - 1)) > 0 && a8_slot(p, last, &other) == slot - 1;
    s_low[t] = block;
    s_lead[t] = -1;
    s_slot[t] = slot;
    s_lost[t] = 0;
    s_first[t] = slot < 0 || follows ? -1 : slot;
  }
  __syncthreads();
  if (p.index) {
    // of tokens with one slot the index names the one that is kept: looked up by the last warp, used below
    const int own = t - (kA8Threads - 32);
    const bool looks = kDense && is_k && own >= 0 && own < p.chunk && s_slot[own] >= 0;
    const int kept = looks ? p.index[s_slot[own]] : -1;
    for (int c = warp; c < p.chunk; c += kA8Warps) {
      const int slot = s_first[c];
      if (slot < 0) continue;
      const int first = slot & ~(block - 1), token = token0 + c;
      int low = block, lead = -1;
      for (int r = lane; r < block; r += 32) {
        // the row's token where tokens are in order, else by the index
        const int named = p.index[first + r], near = token + first + r - slot;
        A8Token x = a8_fetch(p, near, near >= 0 && near < p.N);
        int u = near;
        bool bad = false, there = named == near && a8_slot(p, x, &bad) == first + r;
        if (!there) {
          u = named;
          x = a8_fetch(p, u, u >= 0 && u < p.N);
          there = a8_slot(p, x, &bad) == first + r;
        }
        if (there) {
          s_who[(c << p.block_shift) + r] = make_int2(u, x.pos);
          if (r < low) {
            low = r;
            lead = u;
          }
        }
      }
      const int lowest = __reduce_min_sync(0xFFFFFFFFu, low);
      if (low == lowest && low < block) {
        s_low[c] = low;
        s_lead[c] = lead;
      }
    }
    if (looks && kept != token0 + own) s_lost[own] = 1;
  } else {
#pragma unroll
    for (int i = 0; i < kLooks; ++i) {
      const int slot = look[i], u = t + i * kA8Threads;
#pragma unroll 1
      for (int c = 0; c < p.chunk; ++c)
        if (s_first[c] >= 0 && ((slot ^ s_first[c]) >> p.block_shift) == 0) {  // (a negative slot differs in its sign)
          const int pos = p.half ? p.positions[u] : 0, r = slot & (block - 1);
          if (p.half && (pos < 0 || pos >= p.max_pos)) continue;
          atomicMin(&s_who[(c << p.block_shift) + r].x, u);
          atomicMin(&s_low[c], r);
        }
    }
    if (kDense && is_k) {
#pragma unroll 1
      for (int c = 0; c < p.chunk; ++c)
#pragma unroll
        for (int i = 0; i < kLooks; ++i) {
          const int u = t + i * kA8Threads;
          if (look[i] == s_slot[c] && u < token0 + c && look[i] >= 0 &&  // the first token of a slot is kept
              (!p.half || static_cast<unsigned>(p.positions[u]) < static_cast<unsigned>(p.max_pos)))
            s_lost[c] = 1;
        }
    }
    __syncthreads();
    for (int i = t; i < p.chunk << p.block_shift; i += kA8Threads)
      if (p.half && s_who[i].x != INT_MAX) s_who[i].y = p.positions[s_who[i].x];
    if (t < p.chunk && s_low[t] < block) s_lead[t] = s_who[(t << p.block_shift) + s_low[t]].x;
  }
  __syncthreads();
  float* s_turns = reinterpret_cast<float*>(s_who + (p.chunk << p.block_shift));
  unsigned char* tile = s_tiles + warp * kA8TileBytes;
  // blocks of one tile: the rows' part of the rotation's table comes once for all heads
  const bool staged = is_k && p.half > 0 && block <= A8<D>::kTile;
  for (int c = 0; c < p.chunk; ++c) {
    if (s_lead[c] != token0 + c) continue;  // another token leads
    const int2* who = s_who + (c << p.block_shift);
    const int low = s_low[c], first = s_first[c] & ~(block - 1);
    if (staged) {
      __syncthreads();  // the block before is done
      if (warp < p.Hkv) a8_load<D>(p, who, low & ~(A8<D>::kTile - 1), warp, true, tile);
      const int quads = p.half / 2;  // 16-byte pieces of a position's row
      for (int i = t; i < quads << p.block_shift; i += kA8Threads) {
        const int r = i / quads, q = i - r * quads;
        if (who[r].x != INT_MAX)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(s_turns + r * 2 * p.half + 4 * q)),
                       "l"(p.rope + static_cast<size_t>(who[r].y) * (2 * p.half) + 4 * q)
                       : "memory");
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();
    }
    const uint32_t turns = smem_u32(s_turns);
    for (int head = warp; head < p.Hkv; head += kA8Warps) {
      if (staged) a8_block<D, 1, kDense>(p, who, low, first, head, true, tile, turns, head == warp);
      else if (is_k && p.half > 0) a8_block<D, 2, kDense>(p, who, low, first, head, true, tile, 0u, false);
      else a8_block<D, 0, kDense>(p, who, low, first, head, is_k, tile, 0u, false);
    }
  }
  if (kDense && is_k) {  // the tokens that the cache does not keep
    unsigned lost = __ballot_sync(0xFFFFFFFFu, lane < p.chunk && s_lost[lane] != 0);
    for (; __builtin_expect(lost != 0u, 0); lost &= lost - 1u)
      for (int head = warp; head < p.Hkv; head += kA8Warps) a8_dense<D>(p, token0 + __ffs(lost) - 1, head);
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
  while ((1 << p.page_shift) < page_size) ++p.page_shift;
  while ((1 << p.block_shift) < scale_block) ++p.block_shift;
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
  // as many CTAs as there is room for, but no more tokens than a CTA looks after
  const int each = 2 * N / (kA8PerSm * di.sms) + 1;
  p.chunk = each < kA8Chunk ? each : kA8Chunk;
  p.kv_ctas = 2 * ((N + p.chunk - 1) / p.chunk);
  const int cap = 8 * di.sms > N / 8 ? 8 * di.sms : N / 8;
  p.q_ctas = Hq == 0 ? 0 : N < cap ? N : cap;
  WsHeader* hdr = static_cast<WsHeader*>(workspace);
  if (indexed) {
    const dt_status s = at_launch(append8_index_kernel, (N + kA8Threads - 1) / kA8Threads, kA8Threads, 0, stream, p);
    if (s != DT_OK) return s;
  }
  const int grid = p.kv_ctas + p.q_ctas;
  const size_t smem = sizeof(int2) * static_cast<size_t>(p.chunk) * scale_block + kA8Warps * kA8TileBytes + 2 * kA8TileBytes;
  auto* kernel = d == 64 ? (out_k ? kv_append8_kernel<64, true> : kv_append8_kernel<64, false>)
                         : (out_k ? kv_append8_kernel<128, true> : kv_append8_kernel<128, false>);
  if (ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), kA8Smem) != cudaSuccess) return DT_ERR_CUDA;
  return at_launch(kernel, grid, kA8Threads, smem, stream, p, hdr);
}
