// Argument checks that the entry points of the operators over the ranks share.
#pragma once

#include <algorithm>
#include <memory>
#include <utility>
#include <vector>

#include "comm.hpp"
#include "hbmcoll.h"

namespace hbmc {

// Memory ranges of a call.  A range that is written may overlap no other;
// ranges that are only read may overlap each other.
class Ranges {
 public:
  // [p, p + bytes), checked for NULL, alignment and wrap-around; nothing to
  // check where it holds nothing.
  void add(const void* p, uint64_t bytes, uint32_t align, bool write) {
    if (bytes == 0) return;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (!a || a % align || a + bytes < a) bad_ = true;
    all_.push_back({a, a + bytes, write});
  }
  void read(const void* p, uint64_t bytes, uint32_t align) { add(p, bytes, align, false); }
  void write(const void* p, uint64_t bytes, uint32_t align) { add(p, bytes, align, true); }
  // An output that may be exactly the input `in`, which is then not added.
  void write_over(const void* p, const void* in, uint64_t bytes, uint32_t align) {
    write(p, bytes, align);
    if (in != p) read(in, bytes, align);
  }
  bool bad() const { return bad_; }
  bool ok() {
    if (bad_) return false;
    std::sort(all_.begin(), all_.end(), [](const Range& x, const Range& y) { return x.lo < y.lo; });
    uintptr_t any = 0, written = 0;  // ends of the ranges so far, of the written ones
    for (const Range& r : all_) {
      if (r.lo < written || (r.write && r.lo < any)) return false;
      any = std::max(any, r.hi);
      if (r.write) written = std::max(written, r.hi);
    }
    return true;
  }

 private:
  struct Range {
    uintptr_t lo, hi;
    bool write;
  };
  std::vector<Range> all_;
  bool bad_ = false;
};

// Element size of a type the operators take (0: they do not).
inline uint32_t float_bytes(int dtype) { return dtype == HBMC_FP32 || dtype == HBMC_FP16 || dtype == HBMC_BF16 ? elem_bytes(dtype) : 0; }

inline bool finite(float x) { return x - x == 0.0f; }

constexpr uint64_t kMaxRows = (uint64_t(1) << 31) - 1;

inline int ranks_of(hbmc_comm_t c) { return c && !c->topos.empty() ? c->topos[0].P : 0; }

// Bytes of a matrix, or false when they do not fit an address.
inline bool matrix_bytes(uint64_t rows, uint64_t width, uint32_t e, uint64_t* bytes) {
  return !__builtin_mul_overflow(rows, width, bytes) && !__builtin_mul_overflow(*bytes, uint64_t(e), bytes) &&
         *bytes <= uint64_t(PTRDIFF_MAX);
}

inline hbmc_status_t hip(hipError_t e) { return e == hipSuccess ? HBMC_OK : HBMC_ERR_HIP; }

}  // namespace hbmc
