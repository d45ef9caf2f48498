// The words by which CTAs of the few-row attention hand over partial results of a
// shared item: one for each part, written by the CTA that leaves the part and by the one
// that joins them, each once a call.
//
// A word says by its value, of the call with number c (c ends in binary 01, no other call
// of the process has it): c, the part is there; c + 1, the part's CTA failed; c + 2, the
// joining CTA has given up.  Anything else, and so what memory happens to hold, is: not yet.
// A call captured in a graph has one number for all its replays, so both sides see to it that
// none of the three stays behind, in whichever order they come: the joining CTA clears what it
// has taken, and of a CTA that gives up and one that leaves a part, the second clears.
//
// W: a word with load (acquire), exchange (acquire and release) and store.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define KV4_READY_FN __host__ __device__ __forceinline__
#else
#define KV4_READY_FN inline
#endif

namespace sbsa {

enum Ready { kReadyNot, kReadyPart, kReadyFailed };

// By the part's CTA, when the part is written (or will not be: failed).
template <typename W>
KV4_READY_FN void ready_publish(const W& word, uint64_t call, bool failed) {
  if (word.exchange(failed ? call + 1 : call) == call + 2) word.store(0);
}

// By the joining CTA, until it is no longer kReadyNot.
template <typename W>
KV4_READY_FN Ready ready_look(const W& word, uint64_t call) {
  const uint64_t x = word.load();
  return x == call ? kReadyPart : x == call + 1 ? kReadyFailed : kReadyNot;
}

// By the joining CTA, once: behind a look that found something, or instead of one that may
// still (gave_up).
template <typename W>
KV4_READY_FN void ready_leave(const W& word, uint64_t call, bool gave_up) {
  if (gave_up) {
    const uint64_t x = word.exchange(call + 2);
    if (x != call && x != call + 1) return;
  }
  word.store(0);
}

}  // namespace sbsa
