// gdpa_cache_order.h -- the order in which a CTA's items are brought to it, free of
// CUDA: the kernel for many rows compiles it for the device, the tests as plain
// C++ for the host.
#pragma once

#include "gdpa_cache_index.h"

namespace gdpa {

// Brings every item that some row sees, in order.  `next` waits for the next item's
// record (false: there is none, or the wait has given up), `seen` says whether any
// row sees that item, `look` starts what its copies need, `take` keeps what the
// record and the look hold, `bring` issues the copies (false: a wait has given up).
//
// The look goes ahead of the copies by one record and no further.  Records pass
// through a ring, a record's place is free again once every warp has read it, and
// the warps that add up an item read on only when its copies are there: a search for
// the next item that is seen, with the present one's copies still to issue, would
// wait for ever where more unseen ones lie between than the ring holds.
template <class Next, class Seen, class Look, class Take, class Bring>
GDPA_HD bool bring_in_order(const Next& next, const Seen& seen, const Look& look, const Take& take, const Bring& bring) {
  bool more = next(), ahead = more && seen();
  if (ahead) look();
  while (more) {
    const bool present = ahead;
    if (present) take();
    more = next();
    ahead = more && seen();
    if (ahead) look();
    if (present && !bring()) return false;
  }
  return true;
}

// By how much a wait's limit (some seconds) is stretched: roles wait for whole items,
// and an item takes as long as its rows do (2^27 of them about a second) and as the
// search for it (2^26 sequences without rows 1.3 s).
inline uint64_t wait_stretch(int64_t rows, int64_t sequences) {
  return 1 + static_cast<uint64_t>(rows >> 27) + static_cast<uint64_t>(sequences >> 26);
}

}  // namespace gdpa
