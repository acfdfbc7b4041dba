// raise_limit.h -- a process-wide limit that only grows, raised by any thread.
// Plain C++ (no CUDA): tests compile it by itself.
#pragma once
#include <mutex>

namespace mnb {

inline std::mutex raise_limit_mutex;

// Makes the limit behind `known` at least `want`: set(want) is called where it is
// lower, and returns 0 or an error.  One thread at a time looks, sets and notes,
// so that no thread lowers what another has raised: threads that ask for 200 and
// 100 at once end with 200, and each finds its own in place on return.
template <typename Set>
int raise_limit(int *known, int want, Set set) {
    if (want <= __atomic_load_n(known, __ATOMIC_ACQUIRE))
        return 0;
    std::lock_guard<std::mutex> lock(raise_limit_mutex);
    if (want <= *known)
        return 0;
    const int e = set(want);
    if (e == 0)
        __atomic_store_n(known, want, __ATOMIC_RELEASE);
    return e;
}

}  // namespace mnb
