// The search for a threshold among order keys that token_logprobs.cu's warps
// make, apart from how the keys are counted, so that the host can run it too.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define GH_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define GH_HOST_DEVICE inline
#endif

namespace gh {

// A value that k to `most` of more than k keys reach (*found), or the k-th
// largest key where ties leave no such value.  count(v): how many keys are >= v
// (it may count padding zeros at v = 0, but then more than `most`).  hi is the
// largest key.  32 keys reach lo, so it bounds the k-th from below for k <= 32;
// for larger k the search first steps down from there.
//
// The whole 32-bit range can occur: a NaN's key is the largest there is, and lo
// is 0 where some lanes of the warp hold no key.  The midpoint is therefore taken
// down from hi, where hi - lo + 1 would wrap to 0.  (step is at least 1 and wraps
// only once lo is at most step: count(0) >= k ends the descent there.)
template <typename Count>
GH_HOST_DEVICE uint32_t search_threshold(uint32_t lo, uint32_t hi, int k, int most, const Count& count, bool* found) {
  *found = false;
  if (k > 32) {
    uint32_t step = hi - lo + 1;
    int n;
    while ((n = count(lo)) < k) {
      hi = lo - 1;
      lo = lo > step ? lo - step : 0;
      step *= 2;
    }
    *found = n <= most;
  }
  while (lo < hi && !*found) {
    const uint32_t mid = hi - (hi - lo) / 2;  // lo < mid <= hi
    const int n = count(mid);
    if (n >= k) lo = mid;
    else hi = mid - 1;
    *found = n >= k && n <= most;
  }
  return lo;
}

}  // namespace gh
