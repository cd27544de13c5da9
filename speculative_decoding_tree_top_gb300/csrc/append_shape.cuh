// The shape of dt_kv_append's CTAs, in plain C++.
#pragma once

namespace dt {
namespace {

constexpr int kAppendThreads = 256;  // of a CTA, at most

// The CTA's threads: whole warps, the size whose passes over a token's heads leave the smallest share idle.
inline int append_threads(int heads, int items) {
  int best = kAppendThreads, best_idle = -1;  // none yet
  for (int threads = kAppendThreads; threads >= 64; threads -= 32) {
    const int step = threads / items, passes = (heads + step - 1) / step, idle = passes * step - heads;
    if (best_idle < 0 || idle * best < best_idle * threads) {
      best = threads;
      best_idle = idle;
    }
  }
  return best;
}

}  // namespace
}  // namespace dt
