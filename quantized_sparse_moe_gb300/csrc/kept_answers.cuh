// Answers of a query that takes longer than a small product (how many clusters
// of a launch are resident at once), kept by what was asked.  Plain host code
// without allocation: a fixed table with open addressing, which holds kSlots
// answers (every row count from 1 to 32 with sixteen lengths of K makes about
// 2000) and replaces one per new answer beyond that.
#pragma once

#include <cstdint>

namespace qsm {
namespace mx4 {

class KeptAnswers {
 public:
  static constexpr unsigned kSlots = 4096;

  // Whether the answer to (device, kernel, CTAs per cluster, shared memory) is
  // kept; then *n is set.
  bool find(int dev, const void* kernel, int cs, int smem, int* n) const {
    const unsigned at = home(dev, kernel, cs, smem);
    for (unsigned i = 0; i < kSlots; ++i) {
      const Entry& e = table_[(at + i) % kSlots];
      if (e.kernel == nullptr) return false;
      if (e.dev == dev && e.kernel == kernel && e.cs == cs && e.smem == smem) {
        *n = e.n;
        return true;
      }
    }
    return false;
  }

  // Keeps an answer that find does not have; kernel is not null.
  void put(int dev, const void* kernel, int cs, int smem, int n) {
    unsigned at = home(dev, kernel, cs, smem);
    for (unsigned i = 0; i < kSlots && table_[at].kernel != nullptr; ++i) at = (at + 1) % kSlots;
    // full: every chain is unbroken whichever entry is replaced
    table_[at] = {kernel, dev, cs, smem, n};
  }

 private:
  struct Entry {
    const void* kernel;  // null: free
    int dev, cs, smem, n;
  };
  static unsigned home(int dev, const void* kernel, int cs, int smem) {
    uint64_t h = (uint64_t)reinterpret_cast<uintptr_t>(kernel) * 31 + (unsigned)dev;
    h = (h * 31 + (unsigned)cs) * 1000003 + (unsigned)smem;
    return (unsigned)((h * 0x9E3779B97F4A7C15ull) >> 40) % kSlots;
  }
  Entry table_[kSlots] = {};
};

}  // namespace mx4
}  // namespace qsm
