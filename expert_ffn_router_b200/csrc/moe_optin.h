// A limit that is raised for a kernel as larger launches ask for it (host only).
#pragma once

#include <cstddef>
#include <mutex>
#include <unordered_map>

namespace moe {

// Keeps what each key's limit was raised to.  raise(key, want, set) calls
// set(want) -- 0 for success -- unless the limit already reaches `want`.  The
// lock is held over the check, the call and the note: two callers at once
// could otherwise leave the smaller limit set and the larger noted.
class OptIn {
public:
    template <typename Set>
    auto raise(unsigned long long key, size_t want, Set set) -> decltype(set(want)) {
        std::lock_guard<std::mutex> lk(mu_);
        size_t& have = have_[key];
        if (have >= want) return {};
        const auto e = set(want);
        if (e == decltype(set(want)){}) have = want;
        return e;
    }

private:
    std::mutex mu_;
    std::unordered_map<unsigned long long, size_t> have_;
};

}  // namespace moe
