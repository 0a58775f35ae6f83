// cq_status.h -- several status words read as one (host code without CUDA, so
// that a failing copy can be made on the host).
#pragma once

#include <stdint.h>

namespace cq {

// The bits of `n` words together in *status, and the words cleared. Every word is
// read before one is cleared: a call whose reads fail loses no bit, and one whose
// clearing fails has them all in *status (what it left uncleared comes again).
// read(i, words + i) enqueues a copy and wait() waits for those so far; `words`
// outlives the call, as copies may that no wait followed. clear(i) returns when it
// is done. All return 0 or an error, which is returned.
template <typename Read, typename Wait, typename Clear>
int collect_status(int n, uint32_t* words, Read read, Wait wait, Clear clear, uint32_t* status) {
  uint32_t all = 0;
  for (int i = 0; i < n; ++i)
    if (const int rc = read(i, words + i)) return rc;
  if (const int rc = wait()) return rc;
  for (int i = 0; i < n; ++i) all |= words[i];
  *status = all;
  int first = 0;
  for (int i = 0; i < n; ++i)
    if (words[i])
      if (const int rc = clear(i); rc && !first) first = rc;
  return first;
}

}  // namespace cq
