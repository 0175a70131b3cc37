// A wavefront of 64 lanes on the host, for the headers of csrc/ that use nothing of the GPU but lane
// exchanges: each lane is a coroutine that runs up to the next exchange, where all 64 meet.
#pragma once

#include <stdint.h>
#include <ucontext.h>

#define __device__
#define __forceinline__ inline

namespace wave {

constexpr int kLanes = 64, kStack = 1 << 16;
struct Lane {
  unsigned x;
};
inline Lane lane;            // threadIdx of the lane that runs
inline int64_t shown[2][kLanes];  // what the lanes brought to this exchange and to the one before
inline int turn[kLanes];     // exchanges each lane has been through
inline bool done[kLanes];
inline ucontext_t home, at[kLanes];
inline char stacks[kLanes][kStack];

// Every lane's value, once all have brought theirs.
inline const int64_t *exchange(int64_t v) {
  const int me = lane.x, t = turn[me]++ & 1;
  shown[t][me] = v;
  swapcontext(&at[me], &home);
  return shown[t];
}

inline void (*body)();
inline void start() {
  body();
  done[lane.x] = true;
}

// Runs f in all lanes; true if they went through the same number of exchanges.
inline bool run(void (*f)()) {
  body = f;
  for (int i = 0; i < kLanes; ++i) {
    turn[i] = 0;
    done[i] = false;
    getcontext(&at[i]);
    at[i].uc_stack.ss_sp = stacks[i];
    at[i].uc_stack.ss_size = kStack;
    at[i].uc_link = &home;
    makecontext(&at[i], start, 0);
  }
  for (bool left = true; left;) {
    left = false;
    for (unsigned i = 0; i < kLanes; ++i)
      if (!done[i]) {
        lane.x = i;
        swapcontext(&home, &at[i]);
        left |= !done[i];
      }
  }
  for (int i = 1; i < kLanes; ++i)
    if (turn[i] != turn[0]) return false;
  return true;
}

}  // namespace wave

#define threadIdx (::wave::lane)

inline int __shfl(int v, int from) { return (int)wave::exchange(v)[from & 63]; }
inline int __shfl_up(int v, int d) {
  const int me = wave::lane.x;
  const int64_t *all = wave::exchange(v);
  return (int)all[me >= d ? me - d : me];
}
inline uint64_t __ballot(bool v) {
  const int64_t *all = wave::exchange(v);
  uint64_t m = 0;
  for (int i = 0; i < wave::kLanes; ++i) m |= (uint64_t)(all[i] != 0) << i;
  return m;
}
inline int first_lane(int v) { return (int)wave::exchange(v)[0]; }
#define __builtin_amdgcn_readfirstlane(v) first_lane(v)
