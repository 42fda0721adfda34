// The order of a unit's items, apart from the work itself, so that it can be run on a CPU.
#pragma once

#ifdef __CUDACC__
#define KVARN_TEAM_CALL __device__ __forceinline__
#else
#define KVARN_TEAM_CALL inline
#endif

namespace kvarn {

// A team's threads go through a unit's items [ti, end) together: packed tiles below `last`, fresh ones behind
// them. Each thread calls this, and the items meet at barriers of the whole team, so that its threads have to take
// the same way through it: only answers that they have agreed on (at a barrier) steer it. A wait that ran out for one
// thread, and perhaps not for another whose limit ended a little later, is the team's own record, and
// counts from the next barrier that agrees on it. False: it ran out, and everyone leaves.
template <class Team>
KVARN_TEAM_CALL bool tree_unit(Team& team, int ti, int last, int end) {
  const bool rotated = ti < last;          // the accumulator will hold rotated channels
  for (; ti < last; ++ti)
    if (!team.packed_item(ti)) return false;
  if (rotated && !team.unrotate()) return false;
  for (; ti < end; ++ti)
    if (!team.fresh_item(ti)) return false;
  return team.agreed();
}

}  // namespace kvarn
