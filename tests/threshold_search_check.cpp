// The threshold search of token_logprobs.cu on the host: every search ends, and
// its answer is a threshold that k to `most` keys reach, or the k-th largest
// key.  Built and run by tests/test_token_ops_host.py; prints one line and exits 0
// when every check holds.
#include <algorithm>
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>

#include "../lm_head_cross_gh_b200/csrc/threshold_search.h"

namespace {

constexpr uint32_t kNaNKey = 0xffffffffu;  // order key of the canonical NaN, above +inf's 0xff800000
constexpr uint32_t kNegInfKey = 0x007fffffu;
constexpr int kMostSteps = 200;  // 32 halvings and 32 doublings end any search

int searches = 0, failures = 0;

int most_listed(int k) { return k + k / 8 + 2; }

uint32_t key_of(float x) {
  uint32_t b;
  std::memcpy(&b, &x, 4);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

// As one warp searches: lane l holds keys l, l + 32, ..., and zeros up to a
// multiple of 256 (1024 from there on), which count(0) counts.
void check(const std::vector<uint32_t>& keys, int k, int shift, const char* what) {
  const size_t padded = keys.size() <= 256 ? 256 : 1024;
  uint32_t lane[32] = {};
  for (size_t i = 0; i < keys.size(); ++i) lane[i % 32] = std::max(lane[i % 32], keys[i]);
  const uint32_t lo = *std::min_element(lane, lane + 32) >> shift, hi = *std::max_element(lane, lane + 32) >> shift;
  int steps = 0;
  struct TooLong {};
  auto count = [&](uint32_t v) {
    if (++steps > kMostSteps) throw TooLong{};
    v <<= shift;
    int n = v == 0 ? static_cast<int>(padded - keys.size()) : 0;
    for (uint32_t q : keys) n += q >= v;
    return n;
  };
  ++searches;
  bool found = false;
  uint32_t v;
  try {
    v = gh::search_threshold(lo, hi, k, most_listed(k), count, &found);
  } catch (const TooLong&) {
    ++failures;
    std::fprintf(stderr, "%s: %zu keys, k %d, shift %d, [%08x, %08x]: no end after %d counts\n", what, keys.size(), k,
                 shift, lo, hi, kMostSteps);
    return;
  }
  std::vector<uint32_t> sorted(keys);
  std::sort(sorted.begin(), sorted.end(), [](uint32_t a, uint32_t b) { return a > b; });
  int n = 0;
  for (uint32_t q : keys) n += q >= (v << shift);
  const bool ok = found ? n >= k && n <= most_listed(k) : v == sorted[k - 1] >> shift;
  if (!ok) {
    ++failures;
    std::fprintf(stderr, "%s: %zu keys, k %d, shift %d: %08x (found %d), %d reach it\n", what, keys.size(), k, shift, v,
                 found, n);
  }
}

}  // namespace

int main() {
  std::mt19937 rng(1);
  std::normal_distribution<float> normal(0.0f, 3.0f);
  for (int shift : {0, 16}) {
    for (int k : {1, 2, 3, 5, 8, 12, 20, 26, 31, 32, 33, 40, 64, 100, 127, 128}) {
      for (int segs : {4, 5, 7, 9, 12, 16, 17, 24, 30, 31, 32, 33, 48, 63, 64, 65, 100, 146, 147, 200, 255, 256, 257, 700, 1024}) {
        if (segs <= most_listed(k)) continue;  // listed without a search
        for (int round = 0; round < 4; ++round) {
          std::vector<uint32_t> keys(segs);
          for (auto& q : keys) q = key_of(normal(rng));
          check(keys, k, shift, "finite");
          auto with = [&](uint32_t value, int n, const char* what) {
            std::vector<uint32_t> some(keys);
            for (int i = 0; i < n; ++i) some[rng() % some.size()] = value;
            check(some, k, shift, what);
            std::fill(some.begin(), some.end(), kNegInfKey);
            for (int i = 0; i < n; ++i) some[rng() % some.size()] = value;
            check(some, k, shift, what);
          };
          with(kNaNKey, 1, "a NaN");
          with(kNaNKey, k, "several NaN");
          with(kNaNKey, 4 * segs, "NaN throughout");
          with(key_of(1.0f), 2, "ties");
          with(key_of(3.3e38f), 1, "the largest");
          with(kNegInfKey, segs / 2, "masked");
          with(key_of(-3.3e38f), segs, "the lowest");
          // parts of a cluster that had fewer alternatives than places
          with(0, segs / 2, "empty places");
          std::vector<uint32_t> both(keys);
          for (int i = 0; i < segs; i += 3) both[i] = 0;
          both[segs / 2] = kNaNKey;
          check(both, k, shift, "empty places and a NaN");
        }
      }
    }
  }
  std::printf("%d searches, %d failed checks\n", searches, failures);
  return failures != 0;
}
