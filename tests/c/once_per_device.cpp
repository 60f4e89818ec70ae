// Set-up that belongs to a device is done for each device, and a failure is
// not kept.
#include <cstdio>
#include <thread>
#include <vector>

#include "qmm_once.h"

static int bad = 0;
#define CHECK(x)                                             \
    do {                                                     \
        if (!(x)) std::printf("line %d: %s\n", __LINE__, #x), ++bad; \
    } while (0)

int main() {
    int calls[64] = {}, fails = 2;
    qmm::OncePerDevice once;
    auto set = [&](int dev, int status) { return once.run(dev, 0, [&] { return ++calls[dev], status; }); };
    CHECK(set(0, 0) == 0 && set(0, 0) == 0 && calls[0] == 1);
    CHECK(set(1, 0) == 0 && calls[1] == 1);          // another device is set up too
    CHECK(set(63, 7) == 7 && set(63, 7) == 7 && calls[63] == fails);  // a failure is tried again
    CHECK(set(63, 0) == 0 && set(63, 7) == 0 && calls[63] == 3);
    CHECK(set(0, 7) == 0 && calls[0] == 1);
    qmm::OncePerDevice other;                        // another kernel
    CHECK(other.run(0, 0, [] { return 3; }) == 3);
    std::atomic<int> ran{0};
    std::vector<std::thread> t;
    for (int i = 0; i < 8; ++i)
        t.emplace_back([&] {
            for (int d = 0; d < 64; ++d)
                if (other.run(d, 0, [&] { return ++ran, 0; }) != 0) ++bad;
        });
    for (auto &x : t) x.join();
    CHECK(ran >= 64 && ran <= 8 * 64);
    if (!bad) std::printf("all checks passed\n");
    return bad != 0;
}
