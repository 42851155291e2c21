// Bounded waits of the head's kernels and of the attention over 4-bit rows, and what a kernel whose wait has expired does with its
// copies (internal header).
//
// The rule is that of mbar.cuh: the kernel that gives up has flagged MTPSD_STATUS_WAIT_TIMEOUT, stores nothing of the
// work that it could not finish, waits (bounded again) for its own copies in flight and returns.
#pragma once

#include "mbar.cuh"

// A test compiles the kernels with -DMTPSD_HEAD_ONE_PROBE: a wait that is not over at its first probe has expired.  It
// meets the same copies and arrivals in flight as a wait whose limit has passed.
#ifdef MTPSD_HEAD_ONE_PROBE
constexpr bool kHeadOneProbe = true;
#else
constexpr bool kHeadOneProbe = false;
#endif

namespace mtpsd {
namespace mbar {

// Like wait(), with the default limit.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_head(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  if constexpr (kHeadOneProbe) {
    if (test_wait(bar, parity)) return try_wait<CLUSTER>(bar, parity);     // over: the acquire
    *abort_flag = 1;
    flag_status(status, MTPSD_STATUS_WAIT_TIMEOUT);
    return false;
  }
  return wait<CLUSTER>(bar, parity, abort_flag, status, DEFAULT_LIMIT_NS);
}

// The wait of a kernel that gives up for what is still in flight.
template <bool CLUSTER>
__device__ __forceinline__ bool drain(uint64_t* bar, uint32_t parity, int32_t* status) {
  if (try_wait<CLUSTER>(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!try_wait_sleep<CLUSTER>(bar, parity, SLEEP_HINT_NS))
    if (globaltimer_ns() - t0 > DEFAULT_LIMIT_NS) {
      flag_status(status, MTPSD_STATUS_WAIT_TIMEOUT);
      return false;
    }
  return true;
}

}  // namespace mbar
}  // namespace mtpsd
