// dt_page_plan — request lengths become pages, slots and positions on the device.
//
// A request that keeps len tokens and gets grow more holds want = ceil((len + grow) / page_size) pages afterwards: it
// gives back held - want or takes want - held. The free pages are a stack. First the pages given back are pushed, the
// last request's first and each request's from its last; then the takers pop, request by request in their order. With
// exclusive sums over the requests of what they give (G) and take (T) every page that moves knows its place without
// another's: the given page of rank a (ascending) lands at count + G_total - 1 - a, the taken one of rank k comes from
// count + G_total - 1 - k. Pages that are given and taken in one call move straight from table to table.
//
// A page that a row needs is therefore known from the sums too, before anyone has entered it in the table; and a call reads
// free pages (it takes more than is given) or writes them, never both.
//
// Bound by latency: a few hundred bytes to a few hundred kilobytes. Every CTA scans all requests (two a thread, all in
// shared memory) and does its part of the moves and of the rows; nothing that it reads is written by another, but for the
// lengths and the state's counts, which the last CTA to finish writes. Measured on the device, call behind call in a graph:
// a plan for one tree of 8 nodes 3.2 us, for 64 trees of 16 5.8; 256 prompts of up to 2500 tokens, in and out again, 19 for the
// two (in two launches each, one for the rows, the prompts alone took 32). A call costs the host 10.
#include <cuda_runtime.h>

#include <climits>

#include "attn_common.cuh"

namespace dt {
namespace {

constexpr int kPlanThreads = 1024;  // two requests each
static_assert(2 * kPlanThreads >= DT_PAGED_MAX_BATCH, "every request has a thread");
constexpr int kPlanMostCtas = 64;

struct PlanParams {
  int B, n, N, num_pages, max_pages, page_shift;
  const int32_t *lens, *grow;
  const int32_t *depth, *path;                      // [B][n] or null
  int32_t *table, *held, *free_pages, *free_count;  // the last three null: no pool
  int32_t *out_lens, *cu, *slots, *positions;       // each may be null (slots and positions together)
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

// What the scans leave, [B + 1] each: the packed requests' first rows; the pages taken and given before a request's; and by
// request: the pages it held, the tokens it keeps (-1: it gets nothing), those it gets.
struct PlanSums {
  int *rows, *take, *give, *held, *base, *tokens;
  int count, given;  // free pages, pages given back
};
__device__ __forceinline__ int plan_given(const PlanParams& p, const PlanSums& s, int a) {  // of rank a, ascending
  const int b = plan_find(s.give, p.B, a), of = s.give[b + 1] - s.give[b];
  return p.table[static_cast<size_t>(b) * p.max_pages + s.held[b] - of + a - s.give[b]];
}
__device__ __forceinline__ int plan_taken(const PlanParams& p, const PlanSums& s, int k) {  // of rank k
  const int from = s.count + s.given - 1 - k;
  return from < s.count ? p.free_pages[from] : plan_given(p, s, s.given - 1 - (from - s.count));
}

// Row t of the slot map.
__device__ __forceinline__ void plan_row(const PlanParams& p, const PlanSums& s, int t, WsHeader* hdr) {
  int slot = -1, position = 0, b = 0, i = 0;
  bool live = true;
  if (p.n > 0) {
    b = t / p.n;
    i = t - b * p.n;
  } else if (t < s.rows[p.B]) {
    b = plan_find(s.rows, p.B, t);
    i = t - s.rows[b];
  } else {
    live = false;
  }
  if (live) {
    const int from = s.base[b], count = s.tokens[b];
    int j = i;
    if (p.path && from >= 0) {  // (a served request has n tokens at most: the search ends within its path)
      const int32_t* path = p.path + static_cast<size_t>(b) * p.n;
      j = 0;
      while (j < count && path[j] != i) ++j;
    }
    if (from >= 0 && j < count) {
      const int at = from + j, index = at >> p.page_shift;
      const int page = p.held == nullptr || index < s.held[b] ? p.table[static_cast<size_t>(b) * p.max_pages + index]
                                                              : plan_taken(p, s, s.take[b] + index - s.held[b]);
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

__global__ void __launch_bounds__(kPlanThreads, 1) page_plan_kernel(PlanParams p, WsHeader* hdr) {
  extern __shared__ int s_sums[];
  __shared__ long long s_part[2 * kPlanThreads / 32];
  __shared__ int s_taken;
  __shared__ bool s_last;
  at_launch_order();
  const int t = threadIdx.x, page_size = 1 << p.page_shift;
  const bool pool = p.held != nullptr, first_cta = blockIdx.x == 0;
  PlanSums s;
  s.rows = s_sums;
  s.take = s.rows + p.B + 1;
  s.give = s.take + p.B + 1;
  s.held = s.give + p.B + 1;
  s.base = s.held + p.B + 1;
  s.tokens = s.base + p.B + 1;
  if (t == 0) s_taken = 0;
  const long long count = pool ? p.free_count[0] : 0;
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
  const long long most = p.slots ? p.N : INT_MAX;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int b = 2 * t + k;
    const long long at = v[0] + (k ? rows[0] : 0);
    if (b >= p.B) continue;
    s.rows[b] = static_cast<int>(at < most ? at : most);
    if (p.slots && at + rows[k] > p.N) bad[k] = true;
  }
  if (t == 0) s.rows[p.B] = static_cast<int>(total[0] < most ? total[0] : most);
  // the pages that move
  long long give[2] = {0, 0}, take[2] = {0, 0};
  if (pool)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (2 * t + k < p.B && !bad[k]) (want[k] > held[k] ? take[k] = want[k] - held[k] : give[k] = held[k] - want[k]);
  long long moved[2] = {take[0] + take[1], give[0] + give[1]};
  plan_scan(moved, total, s_part);
  const bool sound = count >= 0 && count + total[1] <= p.num_pages;  // else the pool's state contradicts itself
  s.count = sound ? static_cast<int>(count) : 0;
  s.given = sound ? static_cast<int>(total[1]) : 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int b = 2 * t + k;
    if (b >= p.B) continue;
    const long long before = moved[0] + (k ? take[0] : 0);
    const bool served = !bad[k] && (take[k] == 0 || (sound && before + take[k] <= count + total[1]));
    if (first_cta && (bad[k] || !sound)) record_error(hdr, DT_ERR_INVALID_ARG);
    else if (first_cta && !served) record_error(hdr, DT_ERR_NO_PAGES);
    s.take[b] = static_cast<int>(before < INT_MAX ? before : INT_MAX);
    s.give[b] = sound ? static_cast<int>(moved[1] + (k ? give[0] : 0)) : 0;
    if (served && take[k] > 0) atomicMax(&s_taken, static_cast<int>(before + take[k]));
    s.held[b] = held[k];
    s.base[b] = served ? len[k] : -1;
    s.tokens[b] = tokens[k];
    if (first_cta && p.cu) p.cu[b] = s.rows[b];
  }
  if (t == 0) {
    s.give[p.B] = s.given;
    if (first_cta && p.cu) p.cu[p.B] = s.rows[p.B];
  }
  __syncthreads();
  const int taken = s_taken, step = gridDim.x * blockDim.x, own = blockIdx.x * blockDim.x + t;
  if (pool && sound) {
    for (long long k = own; k < taken; k += step) {
      const int at = static_cast<int>(k), b = plan_find(s.take, p.B, at), page = plan_taken(p, s, at);
      if (page < 0 || page >= p.num_pages) record_error(hdr, DT_ERR_INVALID_ARG);
      p.table[static_cast<size_t>(b) * p.max_pages + s.held[b] + at - s.take[b]] = page;
    }
    for (long long m = own; m < s.given - taken; m += step) {
      const int page = plan_given(p, s, s.given - 1 - static_cast<int>(m));
      if (page < 0 || page >= p.num_pages) record_error(hdr, DT_ERR_INVALID_ARG);
      p.free_pages[s.count + m] = page;
    }
  }
  for (long long row = own; row < p.N; row += step) plan_row(p, s, static_cast<int>(row), hdr);
  // the lengths, which may take the old ones' place, and the state's counts, when every CTA has read them
  if (gridDim.x > 1) {
    __syncthreads();
    if (t == 0) s_last = atom_add_acq_rel_gpu(&hdr->deal_done, 1u) + 1u == gridDim.x;
    __syncthreads();
    if (!s_last) return;
    if (t == 0) hdr->deal_done = 0u;  // ready for the next call
  } else {
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int b = 2 * t + k;
    if (b >= p.B) continue;
    const bool served = s.base[b] >= 0;
    if (p.out_lens) p.out_lens[b] = served ? len[k] + tokens[k] : 0;
    if (pool && sound && served) p.held[b] = want[k];
  }
  if (t == 0 && pool && sound) p.free_count[0] = s.count + s.given - taken;
}

}  // namespace
}  // namespace dt

extern "C" size_t dt_page_plan_workspace_bytes(int B) {
  if (B < 1 || B > DT_PAGED_MAX_BATCH) return 0;
  return sizeof(dt::WsHeader);
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
  if (pool && !((held || B == 0) && free_pages && free_count)) return DT_ERR_INVALID_ARG;
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
  if (workspace_bytes < sizeof(WsHeader)) return DT_ERR_INVALID_ARG;
  PlanParams p{};
  p.B = B; p.n = n; p.N = N; p.num_pages = num_pages; p.max_pages = max_pages;
  while ((1 << p.page_shift) < page_size) ++p.page_shift;
  p.lens = lens; p.grow = grow; p.depth = depth; p.path = path; p.table = page_table;
  p.held = held; p.free_pages = free_pages; p.free_count = free_count;
  p.out_lens = out_lens; p.cu = cu_seqlens; p.slots = slots; p.positions = positions;
  // CTAs for the rows, and for the pages that may move: many when prompts come or requests end, few around a tree or a token
  // (call by call from the host, 64 trees of 16 nodes: 8.8 us with one CTA, 9.4 with five; 256 prompts: 12 us, with one CTA
  // and a second launch for the rows 32)
  const long long work = N / 2048 + (pool && n == 0 ? static_cast<long long>(B) * max_pages / 8192 : 0);
  const int grid = work < kPlanMostCtas ? 1 + static_cast<int>(work) : kPlanMostCtas;
  const size_t smem = 6 * sizeof(int) * (static_cast<size_t>(B) + 1);
  if (ensure_dynamic_smem(reinterpret_cast<const void*>(page_plan_kernel), 6 * sizeof(int) * (DT_PAGED_MAX_BATCH + 1)) !=
      cudaSuccess)
    return DT_ERR_CUDA;
  // few rows: fewer threads start, and meet, sooner. Measured in us (device, other kernels before and behind it), 256 and
  // 1024 threads: one tree of 8 nodes 2.7 and 4.0, 256 tokens 3.1 and 4.4, 512 3.8 and 4.6, 48 trees of 16 nodes 4.1 and 4.4,
  // 62 4.7 and 4.5, one prompt of 1000 tokens 3.9 and 4.1, of 2000 5.5 and 4.6. A thread has two requests.
  const int threads = N <= 768 && B <= 512 && grid == 1 ? 256 : kPlanThreads;
  return at_launch(page_plan_kernel, grid, threads, smem, stream, p, static_cast<WsHeader*>(workspace));
}
