// What the files of the C ABI share.
#pragma once

#include "../../include/scan.h"

#include <hip/hip_runtime.h>

#include "launch.hpp"

namespace sca {
namespace api {

// SCAN_OK, or SCAN_EHIP with the error kept for scan_last_hip_error().
scan_status hip_status(hipError_t e);

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int64_t kMaxN = 2147483647;        // INT32_MAX
constexpr int64_t kMaxChannels = 1ll << 22;
constexpr uint64_t kMaxBytes = 1ull << 47;   // a device address

inline bool activation_fmt(scan_dtype d, sca::Fmt* f, size_t* bytes) {
  switch (d) {
    case SCAN_F32: *f = sca::Fmt::F32; *bytes = 4; return true;
    case SCAN_F16: *f = sca::Fmt::F16; *bytes = 2; return true;
    case SCAN_BF16: *f = sca::Fmt::BF16; *bytes = 2; return true;
    default: return false;
  }
}

// The arrays of one call, checked as they are added: null (when required),
// alignment, size; then outputs against everything.
class Ranges {
 public:
  // A contiguous array of count elements.
  void add(const void* p, uint64_t count, size_t eb, bool output, bool required) {
    add_bytes(p, (unsigned __int128)count * eb, eb, output, required);
  }
  // dims[i] entries strides[i] elements apart, then `inner` contiguous ones.
  void add_strided(const void* p, const int64_t* dims, const int64_t* strides, int nd,
                   int64_t inner, size_t eb, bool required) {
    unsigned __int128 count = (unsigned __int128)inner;
    for (int i = 0; i < nd; ++i) {
      if (strides[i] < 0) {
        status_ = SCAN_EINVAL;
        return;
      }
      if (dims[i] == 0) count = 0;
    }
    if (count != 0)
      for (int i = 0; i < nd; ++i)
        count += (unsigned __int128)(dims[i] - 1) * (unsigned __int128)strides[i];
    add_bytes(p, count * eb, eb, false, required);
  }
  scan_status status() const {
    if (status_ != SCAN_OK) return status_;
    for (int i = 0; i < n_; ++i)
      for (int j = 0; j < n_; ++j)
        if (i != j && r_[i].output && r_[i].a < r_[j].e && r_[j].a < r_[i].e) return SCAN_EALIAS;
    return SCAN_OK;
  }

 private:
  struct Range {
    uintptr_t a, e;
    bool output;
  };
  void add_bytes(const void* p, unsigned __int128 bytes, size_t eb, bool output, bool required) {
    if (bytes >= kMaxBytes) {
      status_ = SCAN_EINVAL;
      return;
    }
    if (bytes == 0) return;
    if (p == nullptr) {
      if (required) status_ = SCAN_EINVAL;
      return;
    }
    if (!aligned(p, eb)) {
      status_ = SCAN_EINVAL;
      return;
    }
    r_[n_++] = Range{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, output};
  }
  Range r_[24];
  int n_ = 0;
  scan_status status_ = SCAN_OK;
};

// Whether [batch, length, channels] has a size below kMaxBytes.  (Its factors'
// product can pass 64 bits; below kMaxBytes, no product of a sequence operator's
// sizes does: a scan's rows of B and C and its kept states are at most 2^6 times as much,
// its state is at most 2^31 2^22 2^6 elements.)
inline bool activations_fit(int64_t batch, int64_t length, int64_t channels, size_t eb) {
  return (unsigned __int128)batch * (unsigned __int128)length * (unsigned __int128)channels * eb <
         kMaxBytes;
}

}  // namespace api
}  // namespace sca
