// tq_memo.cuh -- answers of the runtime that do not change while the process lives (a kernel's
// registers, how many of its clusters a device holds), asked for once a key.  Host code only.
#pragma once

#include <atomic>

namespace tq {

// ask(&answer) tells whether there was an answer, of 0 or more.  One that could not be had is not
// kept: the next call asks again.  Threads may ask at once (they get the same answer).
template <int KEYS>
class Memo {
 public:
  template <class Ask>
  bool get(int key, Ask ask, int* answer) {
    int kept = kept_[key].load(std::memory_order_relaxed);
    if (kept == 0) {
      int a = 0;
      if (!ask(&a)) return false;
      kept = a + 1;
      kept_[key].store(kept, std::memory_order_relaxed);
    }
    *answer = kept - 1;
    return true;
  }

 private:
  std::atomic<int> kept_[KEYS] = {};          // answer + 1; 0: not known
};

}  // namespace tq
