// Host-side row loops of the weight packers on a few threads.
#pragma once

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <thread>
#include <vector>

namespace {

// Runs rows [0, N) of `fn(n0, n1)` on up to 16 host threads.  No exception
// leaves it: a range whose thread cannot be started runs on the calling
// thread, and a range that throws (an allocation failure) is reported by the
// false return.
template <class F>
bool parallel_rows(int32_t N, F fn) {
    std::atomic<bool> ok{true};
    auto run = [&](int32_t n0, int32_t n1) {
        try {
            fn(n0, n1);
        } catch (...) {
            ok.store(false);
        }
    };
    unsigned nt = std::max(1u, std::min(16u, std::thread::hardware_concurrency()));
    nt = std::min<unsigned>(nt, unsigned(N));
    std::vector<std::thread> pool;
    try {
        pool.reserve(nt);
    } catch (...) {
        nt = 1;
    }
    const int32_t per = (N + int32_t(nt) - 1) / int32_t(nt);
    // range t = rows [t per, (t + 1) per); the calling thread takes range 0
    for (unsigned t = 1; t < nt; ++t) {
        const int32_t n0 = int32_t(t) * per, n1 = std::min(N, n0 + per);
        if (n0 >= n1) break;
        try {
            pool.emplace_back(run, n0, n1);
        } catch (...) {
            run(n0, n1);
        }
    }
    run(0, std::min(N, per));
    for (auto& th : pool) th.join();
    return ok.load();
}

}  // namespace
