// dt_page_plan — request lengths become pages, slots and positions on the device.
//
// A request that keeps len tokens and gets grow more holds want = ceil((len + grow) / page_size) pages afterwards: it
// gives back held - want or takes want - held. The free pages are a stack. First the pages given back are pushed, the
// last request's first and each request's from its last; then the takers pop, request by request in their order. With
// exclusive sums over the requests of what they give (G) and take (T) every page that moves knows its place without
// another's: the given page of rank a (ascending) lands at count + G_total - 1 - a, the taken one of rank k comes from
// count + G_total - 1 - k. Pages that are given and taken in one call move straight from table to table.
//
// Bound by latency: a few hundred bytes to a few hundred kilobytes. One CTA scans the requests (two a thread, all in
// shared memory), moves the pages and, for up to kPlanOwnRows rows, writes the slots too: one launch. More rows are
// written by a second launch over every SM, which finds the scans in the workspace.
#include <cuda_runtime.h>

#include <climits>

#include "attn_common.cuh"

namespace dt {
namespace {

constexpr int kPlanThreads = 1024;  // of the scanning CTA: two requests each
static_assert(2 * kPlanThreads >= DT_PAGED_MAX_BATCH, "every request has a thread");
constexpr int kPlanOwnRows = 8 * kPlanThreads;
constexpr int kPlanRowThreads = 256, kPlanRowsEach = 4;

struct PlanParams {
  int B, n, N, num_pages, max_pages, page_shift;
  const int32_t *lens, *grow;
  const int32_t *depth, *path;              // [B][n] or null
  int32_t *table, *held, *free_pages, *free_count;  // the last three null: no pool
  int32_t *out_lens, *cu, *slots, *positions;       // each may be null (slots and positions together)
  int32_t *rows, *base, *tokens;            // workspace of the second launch: [B + 1], [B], [B]
};

// Exclusive sums of two values over the CTA.
__device__ __forceinline__ void plan_scan(long long (&v)[2], long long (&total)[2], long long* s_part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  long long incl[2] = {v[0], v[1]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long y = __shfl_up_sync(0xFFFFFFFFu, incl[k], o);
      if (lane >= o) incl[k] += y;
    }
  if (lane == 31) {
    s_part[2 * warp] = incl[0];
    s_part[2 * warp + 1] = incl[1];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    long long before = 0, all = 0;
    const long long mine = lane < warps ? s_part[2 * lane + k] : 0;
    all = mine;
    before = lane < warp ? mine : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
      before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
    }
    total[k] = all;
    v[k] = before + incl[k] - v[k];
  }
  __syncthreads();
}

// The last b in [0, B) with start[b] <= x (start[0] <= x).
__device__ __forceinline__ int plan_find(const int* start, int B, int x) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Row t of the slot map. rows: the packed requests' first rows; base: tokens kept, -1 for a request that gets nothing;
// tokens: how many it gets.
__device__ __forceinline__ void plan_row(const PlanParams& p, int t, const int* rows, const int* base,
                                         const int* tokens, WsHeader* hdr) {
  int slot = -1, position = 0, b = 0, i = 0;
  bool live = true;
  if (p.n > 0) {
    b = t / p.n;
    i = t - b * p.n;
  } else if (t < rows[p.B]) {
    b = plan_find(rows, p.B, t);
    i = t - rows[b];
  } else {
    live = false;
  }
  if (live) {
    const int from = base[b], count = tokens[b];
    int j = i;
    if (p.path) {
      const int32_t* path = p.path + static_cast<size_t>(b) * p.n;
      j = 0;
      while (j < count && path[j] != i) ++j;
    }
    if (from >= 0 && j < count) {
      const int at = from + j;
      const int page = p.table[static_cast<size_t>(b) * p.max_pages + (at >> p.page_shift)];
      if (page < 0 || page >= p.num_pages) {
        record_error(hdr, DT_ERR_INVALID_ARG);
      } else {
        slot = (page << p.page_shift) + (at & ((1 << p.page_shift) - 1));
        // a depth of any size: the append looks at the position before it uses it
        position = p.depth ? static_cast<int>(static_cast<unsigned>(from) + static_cast<unsigned>(p.depth[t]) - 1u) : at;
      }
    }
  }
  p.slots[t] = slot;
  p.positions[t] = position;
}

__global__ void __launch_bounds__(kPlanThreads, 1) page_plan_kernel(PlanParams p, int own_rows, WsHeader* hdr) {
  __shared__ int s_rows[DT_PAGED_MAX_BATCH + 1], s_take[DT_PAGED_MAX_BATCH + 1], s_give[DT_PAGED_MAX_BATCH + 1];
  __shared__ int s_base[DT_PAGED_MAX_BATCH], s_tokens[DT_PAGED_MAX_BATCH];
  __shared__ long long s_part[2 * kPlanThreads / 32];
  __shared__ int s_taken;
  at_launch_order();
  const int t = threadIdx.x, page_size = 1 << p.page_shift;
  const bool pool = p.held != nullptr;
  if (t == 0) s_taken = 0;
  int len[2], tokens[2], held[2], want[2];
  bool bad[2] = {false, false};
  long long rows[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int b = 2 * t + k;
    len[k] = tokens[k] = held[k] = want[k] = 0;
    if (b >= p.B) continue;
    len[k] = p.lens[b];
    held[k] = pool ? p.held[b] : 0;
    const bool ended = len[k] < 0;  // holds nothing from here on
    tokens[k] = ended ? 0 : p.grow[b];
    if (ended) len[k] = 0;
    const long long end = static_cast<long long>(len[k]) + tokens[k];
    bad[k] = tokens[k] < 0 || (p.n > 0 && tokens[k] > p.n) || end > static_cast<long long>(p.max_pages) * page_size;
    if (pool) bad[k] = bad[k] || held[k] < 0 || held[k] > p.max_pages ||
                       (!ended && static_cast<long long>(held[k]) * page_size < len[k]);
    rows[k] = p.n > 0 ? p.n : tokens[k] > 0 ? tokens[k] : 0;
    want[k] = static_cast<int>((end + page_size - 1) >> p.page_shift);
  }
  // the rows' places; a packed request whose rows are not all there gets nothing
  long long v[2] = {rows[0] + rows[1], 0}, total[2];
  plan_scan(v, total, s_part);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int b = 2 * t + k;
    const long long at = v[0] + (k ? rows[0] : 0);
    if (b < p.B) {
      s_rows[b] = static_cast<int>(at < p.N ? at : p.N);
      if (p.slots && at + rows[k] > p.N) bad[k] = true;
      if (!p.slots) s_rows[b] = static_cast<int>(at < INT_MAX ? at : INT_MAX);
    }
  }
  const long long last = p.slots && total[0] > p.N ? p.N : total[0];
  if (t == 0) s_rows[p.B] = static_cast<int>(last < INT_MAX ? last : INT_MAX);
  // the pages that move
  long long give[2] = {0, 0}, take[2] = {0, 0};
  if (pool)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (2 * t + k < p.B && !bad[k]) (want[k] > held[k] ? take[k] = want[k] - held[k] : give[k] = held[k] - want[k]);
  long long moved[2] = {take[0] + take[1], give[0] + give[1]};
  plan_scan(moved, total, s_part);
  const long long count = pool ? p.free_count[0] : 0;
  const bool sound = count >= 0 && count + total[1] <= p.num_pages;  // else the pool's state contradicts itself
  const long long top = count + total[1];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int b = 2 * t + k;
    if (b >= p.B) continue;
    const long long before = moved[0] + (k ? take[0] : 0);
    const bool served = !bad[k] && (take[k] == 0 || (sound && before + take[k] <= top));
    if (bad[k] || !sound) record_error(hdr, DT_ERR_INVALID_ARG);
    else if (!served) record_error(hdr, DT_ERR_NO_PAGES);
    s_take[b] = static_cast<int>(before < INT_MAX ? before : INT_MAX);
    s_give[b] = sound ? static_cast<int>(moved[1] + (k ? give[0] : 0)) : 0;
    if (served && take[k] > 0) atomicMax(&s_taken, static_cast<int>(before + take[k]));
    s_base[b] = served ? len[k] : -1;
    s_tokens[b] = tokens[k];
    if (p.out_lens) p.out_lens[b] = served ? len[k] + tokens[k] : 0;
    if (p.cu) p.cu[b] = s_rows[b];
    if (own_rows == 0 && p.slots) {
      p.rows[b] = s_rows[b];
      p.base[b] = s_base[b];
      p.tokens[b] = tokens[k];
    }
  }
  if (t == 0) {
    s_give[p.B] = sound ? static_cast<int>(total[1]) : 0;
    if (p.cu) p.cu[p.B] = s_rows[p.B];
    if (own_rows == 0 && p.slots) p.rows[p.B] = s_rows[p.B];
  }
  __syncthreads();
  if (pool && sound) {
    const int taken = s_taken, given = s_give[p.B], at = static_cast<int>(count);
    auto given_page = [&](int a) {
      const int b = plan_find(s_give, p.B, a);
      const int left = p.held[b] - (s_give[b + 1] - s_give[b]);  // the pages that it keeps
      return p.table[static_cast<size_t>(b) * p.max_pages + left + a - s_give[b]];
    };
    for (int k = t; k < taken; k += blockDim.x) {
      const int b = plan_find(s_take, p.B, k), from = at + given - 1 - k;
      const int page = from < at ? p.free_pages[from] : given_page(given - 1 - (from - at));
      p.table[static_cast<size_t>(b) * p.max_pages + p.held[b] + k - s_take[b]] = page;
    }
    __syncthreads();  // the popped ones have been read: their places may be written
    for (int m = t; m < given && at + m < at + given - taken; m += blockDim.x)
      p.free_pages[at + m] = given_page(given - 1 - m);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (2 * t + k < p.B && s_base[2 * t + k] >= 0) p.held[2 * t + k] = want[k];
    if (t == 0) p.free_count[0] = at + given - taken;
  }
  for (int row = t; row < own_rows; row += blockDim.x) plan_row(p, row, s_rows, s_base, s_tokens, hdr);
}

__global__ void __launch_bounds__(kPlanRowThreads) page_rows_kernel(PlanParams p, WsHeader* hdr) {
  __shared__ int s_rows[DT_PAGED_MAX_BATCH + 1];
  at_launch_order();
  if (p.n == 0) {
    for (int b = threadIdx.x; b <= p.B; b += kPlanRowThreads) s_rows[b] = p.rows[b];
    __syncthreads();
  }
  const long long first = static_cast<long long>(blockIdx.x) * kPlanRowThreads * kPlanRowsEach + threadIdx.x;
#pragma unroll
  for (int u = 0; u < kPlanRowsEach; ++u) {
    const long long row = first + u * kPlanRowThreads;
    if (row < p.N) plan_row(p, static_cast<int>(row), s_rows, p.base, p.tokens, hdr);
  }
}

struct PlanLayout {
  size_t rows, base, tokens, bytes;
};
inline PlanLayout plan_layout(int B) {
  PlanLayout L{};
  L.rows = align_up(sizeof(WsHeader));
  L.base = align_up(L.rows + sizeof(int32_t) * (static_cast<size_t>(B) + 1));
  L.tokens = align_up(L.base + sizeof(int32_t) * static_cast<size_t>(B));
  L.bytes = align_up(L.tokens + sizeof(int32_t) * static_cast<size_t>(B));
  return L;
}

}  // namespace
}  // namespace dt

extern "C" size_t dt_page_plan_workspace_bytes(int B) {
  if (B < 1 || B > DT_PAGED_MAX_BATCH) return 0;
  return dt::plan_layout(B).bytes;
}

extern "C" dt_status dt_page_plan(int B, int n, int N, int page_size, int num_pages, int max_pages, const int32_t* lens,
                                  const int32_t* grow, const int32_t* depth, const int32_t* path, int32_t* page_table,
                                  int32_t* held, int32_t* free_pages, int32_t* free_count, int32_t* out_lens,
                                  int32_t* cu_seqlens, int32_t* slots, int32_t* positions, void* workspace,
                                  size_t workspace_bytes, cudaStream_t stream) {
  using namespace dt;
  if (B < 0 || n < 0 || N < 0 || page_size < 1 || num_pages < 1 || max_pages < 1) return DT_ERR_INVALID_ARG;
  if (n == 0 && (depth || path)) return DT_ERR_INVALID_ARG;
  if (depth && path) return DT_ERR_INVALID_ARG;
  if ((slots != nullptr) != (positions != nullptr)) return DT_ERR_INVALID_ARG;
  if (slots ? (n > 0 && N != static_cast<long long>(B) * n) : N != 0) return DT_ERR_INVALID_ARG;
  const bool pool = held || free_pages || free_count;
  if (pool && !(held && free_pages && free_count)) return DT_ERR_INVALID_ARG;
  if (B == 0 && N == 0) return DT_OK;
  const void* need[] = {lens, grow, page_table};
  for (const void* x : need)
    if (!x && B > 0) return DT_ERR_INVALID_ARG;
  const void* ints[] = {lens, grow, depth, path, page_table, held, free_pages, free_count, out_lens, cu_seqlens, slots,
                        positions};
  for (const void* x : ints)
    if (reinterpret_cast<uintptr_t>(x) & 3u) return DT_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace)) return DT_ERR_INVALID_ARG;
  if (B > DT_PAGED_MAX_BATCH || N > INT_MAX / 2) return DT_ERR_UNSUPPORTED;
  if (page_size < DT_MIN_PAGE || page_size > DT_MAX_PAGE || (page_size & (page_size - 1))) return DT_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_pages) * page_size > INT_MAX) return DT_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size > DT_PAGED_MAX_TOKENS) return DT_ERR_UNSUPPORTED;
  const PlanLayout L = plan_layout(B);
  if (workspace_bytes < L.bytes) return DT_ERR_INVALID_ARG;
  char* ws = static_cast<char*>(workspace);
  PlanParams p{};
  p.B = B; p.n = n; p.N = N; p.num_pages = num_pages; p.max_pages = max_pages;
  while ((1 << p.page_shift) < page_size) ++p.page_shift;
  p.lens = lens; p.grow = grow; p.depth = depth; p.path = path; p.table = page_table;
  p.held = held; p.free_pages = free_pages; p.free_count = free_count;
  p.out_lens = out_lens; p.cu = cu_seqlens; p.slots = slots; p.positions = positions;
  p.rows = reinterpret_cast<int32_t*>(ws + L.rows);
  p.base = reinterpret_cast<int32_t*>(ws + L.base);
  p.tokens = reinterpret_cast<int32_t*>(ws + L.tokens);
  WsHeader* hdr = reinterpret_cast<WsHeader*>(ws);
  const int own_rows = N <= kPlanOwnRows ? N : 0;
  const dt_status s = at_launch(page_plan_kernel, 1, kPlanThreads, 0, stream, p, own_rows, hdr);
  if (s != DT_OK || own_rows == N) return s;
  constexpr int kEach = kPlanRowThreads * kPlanRowsEach;
  return at_launch(page_rows_kernel, (N + kEach - 1) / kEach, kPlanRowThreads, 0, stream, p, hdr);
}
