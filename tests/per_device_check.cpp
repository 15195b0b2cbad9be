// The first call of a device: an error is returned and not kept, a success is, for its device alone.
#include <cstdio>
#include "per_device.h"

int main()
{
    static std::atomic<int> slots[moe::kMaxDevices];
    int calls = 0, fail = 2, n = -1;
    auto get = [&](int dev) {
        return moe::per_device<int>(slots, dev, [&](int* v) {
            ++calls;
            if (fail > 0) { --fail; return 7; }
            *v = 100 + dev;
            return 0;
        }, &n);
    };
#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)
    CHECK(get(0) == 7 && n == -1 && get(1) == 7 && calls == 2);
    CHECK(get(0) == 0 && n == 100 && calls == 3);
    CHECK(get(0) == 0 && n == 100 && calls == 3);
    fail = 1;
    CHECK(get(1) == 7 && calls == 4);
    CHECK(get(0) == 0 && n == 100 && calls == 4);
    CHECK(get(1) == 0 && n == 101 && calls == 5);
    CHECK(get(moe::kMaxDevices) == 0 && get(moe::kMaxDevices) == 0 && n == 100 + moe::kMaxDevices && calls == 7);
    return 0;
}
