// Rules of the few-token layer's last launch (few.hip) that have to hold whatever the words
// of its workspace are, compiled into the kernel and into host code (tests/slices_host.cpp),
// where every order of arrival can be played.
//
// Tickets. A call that uses the workspace at the same time, against the rules, may have its
// scores or rows where this one counts tickets. Any word read there becomes the ticket of
// that number, or one past the last task: no task has a negative number, and a ticket times
// the tasks of a ticket stays an int.
//
// Slices of out: who writes a column tile whose K is cut into D slices that different
// workgroups hold. A slice whose wait for the up tasks ended well is handed over, and the one that arrives
// last adds all D up. A slice that gave the wait up has no sum to hand over: it writes NaN
// to out itself, and does not arrive. So the tile of a call that owns its workspace is NaN
// if one slice gave up, whoever arrives when; and where a call on the same workspace has
// cleared the arrivals, a slice that gave up does not leave out as it was either.
#pragma once

#if defined(__HIPCC__)
#define MOE_HD __host__ __device__
#else
#define MOE_HD
#endif

namespace moe {
namespace few {

// More than all up tasks of a call (units of 16 pairs x columns / 8) and small enough to be
// multiplied by the 8 tasks of a ticket.
constexpr unsigned kNoTicket = 1u << 27;
MOE_HD inline int ticket_number(unsigned word) { return (int)(word < kNoTicket ? word : kNoTicket); }

enum Slice { kStore, kHandOver, kGiveUp };

MOE_HD inline Slice slice_step(bool waited, int D) {
  return !waited ? kGiveUp : D > 1 ? kHandOver : kStore;
}

// before: slices that had arrived
MOE_HD inline bool adds_up(unsigned before, int D) { return before == (unsigned)(D - 1); }

}  // namespace few
}  // namespace moe
