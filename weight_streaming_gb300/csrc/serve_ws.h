// The workspace of the served attention layer's calls (vp_linear_fp8_block, vp_paged_attention): the status
// word, then counters that are zero between calls, then data.  The counters' place does not depend on
// the call or its shape, so that one workspace serves them all in turn.
#pragma once
#include <cstddef>

namespace vp {

constexpr size_t kServeCounters = 256;                 // byte offset
constexpr size_t kServeMaxCounters = 65536;            // 32-bit words
constexpr size_t kServeData = kServeCounters + 4 * kServeMaxCounters;

}  // namespace vp
