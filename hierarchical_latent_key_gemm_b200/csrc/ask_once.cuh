// An answer of the driver that stays the same, asked for once.
#pragma once

#include <atomic>

namespace lsa {

// `known` is the answer + 1, or 0 before there is one.  ask() gives the answer
// (>= 0), or -1 where asking failed: that is 0 for this call, and the next call asks
// again.  Threads that ask at the same time get the same answer.
template <typename Ask>
int ask_once(std::atomic<int>& known, const Ask& ask) {
    int n = known.load(std::memory_order_relaxed) - 1;
    if (n >= 0) return n;
    n = ask();
    if (n < 0) return 0;
    known.store(n + 1, std::memory_order_relaxed);
    return n;
}

}  // namespace lsa
