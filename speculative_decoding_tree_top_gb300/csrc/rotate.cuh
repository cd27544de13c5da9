// Rotary position embedding of bf16 heads, in fp32: what the appends to a paged cache share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace dt {
namespace {

struct Eight {  // eight bf16 as fp32
  float x[8];
};
__device__ __forceinline__ Eight unpack8(uint4 u) {
  Eight e;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e.x[2 * i] = __uint_as_float(w[i] << 16);
    e.x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return e;
}
__device__ __forceinline__ uint4 pack8(const Eight& e) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(e.x[2 * i], e.x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The cosines and sines of an item's columns, and its rotation. Half-split pairs: group A holds pairs c..c+7's first
// elements and group B their second ones. Interleaved: each group holds four whole pairs.
struct Turn {
  float c[8], s[8];
};
// The two groups of eight columns of a head's item (16 columns). Within the rotated part of a half-split head they are a
// pair's two halves; otherwise two neighbouring groups (half is a multiple of 8: a group is rotated as a whole or not
// at all).
struct TurnCols {
  int ca, cb;
  bool halves;
};
__device__ __forceinline__ TurnCols turn_cols(int item, int half, int interleaved) {
  TurnCols t;
  t.halves = !interleaved && 8 * item < half;
  if (interleaved) {
    t.ca = 16 * item;
    t.cb = t.ca + 8;
  } else if (t.halves) {
    t.ca = 8 * item;
    t.cb = t.ca + half;
  } else {  // the columns past rot = 2 half: items half / 8 on take 16 each
    t.ca = 2 * half + 16 * (item - half / 8);
    t.cb = t.ca + 8;
  }
  return t;
}
// An item's cosines and sines, from its position's row of the table.
__device__ __forceinline__ void load_turn(const float* row, int item, int half, int interleaved, bool halves, Turn& tu) {
  auto four = [](const float* from, float* to) {
    const float4 x = *reinterpret_cast<const float4*>(from);
    to[0] = x.x;
    to[1] = x.y;
    to[2] = x.z;
    to[3] = x.w;
  };
  if (interleaved) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {  // pairs 8 item + 4 g .. + 3 (half is a multiple of 8)
      const int pr = 8 * item + 4 * g;
      if (pr < half) {
        four(row + pr, tu.c + 4 * g);
        four(row + half + pr, tu.s + 4 * g);
      }
    }
  } else if (halves) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      four(row + 8 * item + 4 * g, tu.c + 4 * g);
      four(row + half + 8 * item + 4 * g, tu.s + 4 * g);
    }
  }
}
__device__ __forceinline__ void turn_halves(uint4& a, uint4& b, const Turn& t) {
  Eight x = unpack8(a), y = unpack8(b);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float u = x.x[i] * t.c[i] - y.x[i] * t.s[i], w = y.x[i] * t.c[i] + x.x[i] * t.s[i];
    x.x[i] = u;
    y.x[i] = w;
  }
  a = pack8(x);
  b = pack8(y);
}
__device__ __forceinline__ void turn_pairs(uint4& a, const float* c, const float* s) {
  Eight x = unpack8(a);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float u = x.x[2 * i] * c[i] - x.x[2 * i + 1] * s[i], w = x.x[2 * i + 1] * c[i] + x.x[2 * i] * s[i];
    x.x[2 * i] = u;
    x.x[2 * i + 1] = w;
  }
  a = pack8(x);
}

}  // namespace
}  // namespace dt
