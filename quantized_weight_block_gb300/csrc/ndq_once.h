// ndq_once.h -- what the host asks of a device once, for calls from several
// threads.  Not part of the public ABI.
#pragma once

#include <atomic>

namespace ndq {

// A positive number, asked for by the first calls (one or more at once, which
// find the same) and read by the later ones.  It is one word, so that a thread
// that sees it sees all of it: hosts with weakly ordered memory may show a
// second word's store before the first one's.
class Once {
   public:
    // ask(int*): 0, or an error code that is passed on (then the next call asks again)
    template <typename Ask>
    int get(Ask ask, int* value) {
        int v = value_.load(std::memory_order_relaxed);
        if (v == 0) {
            if (const int rc = ask(&v)) return rc;
            value_.store(v, std::memory_order_relaxed);
        }
        *value = v;
        return 0;
    }

   private:
    std::atomic<int> value_{0};
};

}  // namespace ndq
