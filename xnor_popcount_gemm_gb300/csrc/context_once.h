// What is set once per CUDA context: a kernel's attributes belong to the context (and device) that was current when they
// were set, so that a flag for the whole process would leave every other one without them. No CUDA header is needed here.
#pragma once

#include <atomic>

namespace bt {

class ContextOnce {
public:
    // id(unsigned long long *) tells the current context apart from every other one of the process, or returns false;
    // set() returns 0 on success. set runs unless it has last succeeded for this context.
    template <typename Id, typename Set> int run(Id id, Set set) {
        unsigned long long at = 0;
        if (id(&at) && done_.load(std::memory_order_acquire) == at + 1) return 0;
        const int e = static_cast<int>(set());
        // (set may have made a context current)
        if (e == 0 && id(&at)) done_.store(at + 1, std::memory_order_release);
        return e;
    }

private:
    std::atomic<unsigned long long> done_{0};  // the context's id + 1
};

}  // namespace bt
