// Start of the workspaces of the attention sublayer's operators: the status word, then
// the tickets of split work.  Both are left as they were found, whatever the operator,
// so one workspace serves them all in stream order.
#pragma once

#include <algorithm>
#include <stddef.h>
#include <stdint.h>

#include "kernels.h"

namespace moe {

constexpr size_t kHdrBytes = 256;
constexpr size_t kTicketBytes = ((size_t)std::max(kLinMaxCtas, kAttMaxCtas) * sizeof(int) + 255) / 256 * 256;
constexpr size_t kDataAt = kHdrBytes + kTicketBytes;

struct Ws {
  int* status;
  int* tickets;
  uint8_t* data;
  explicit Ws(void* ws) {
    uint8_t* p = reinterpret_cast<uint8_t*>(ws);
    status = reinterpret_cast<int*>(p) + kHdrStatus;
    tickets = reinterpret_cast<int*>(p + kHdrBytes);
    data = p + kDataAt;
  }
};

inline bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace moe
