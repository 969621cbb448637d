// Which keys a new token of a paged sequence sees.  Plain constexpr functions:
// the kernels run them, and a host test runs them over the ends of every range
// (tests/test_paged_keys.py).
#pragma once

#include <cstdint>

namespace sz {

constexpr uint32_t kMaxTokens = 1u << 30;       // of a batch, of a sequence: sums of two stay below 2^31

// A window as the kernels take it, 0: none.  Positions are below kMaxTokens,
// so a larger window hides nothing, and p - window + 1 stays above -2^31 for
// positions p down to -kMaxTokens (more new tokens than the cache has).
constexpr int32_t window_keys(uint32_t window)
{
    return (int32_t)(window < kMaxTokens ? window : kMaxTokens);
}

// The first key that position p sees; the last is p itself.
constexpr int32_t first_seen(int32_t p, int32_t window)
{
    return window > 0 && p - window + 1 > 0 ? p - window + 1 : 0;
}

}  // namespace sz
