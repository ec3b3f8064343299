// The launch plans of w4a8_route over batches up to T * E next to 2^31, with
// UndefinedBehaviorSanitizer on the host code of route.hip.  Test
// infrastructure: only tests/test_selection_sanitizers.py builds and runs it.
#include <cstdio>
#include <initializer_list>

#include "launch.h"

int main() {
    int fails = 0;
    const long long limit = (1LL << 31) - 1;  // T * E < 2^31
    for (int E : {1, 2, 3, 8, 16, 17, 64, 100, 512})
        for (long long T : {1LL, 16LL, 64LL, 65LL, 2048LL, 2049LL, 16384LL, 16385LL, 1000003LL,
                            limit / 2, limit - (1LL << 22), limit - 1000, limit}) {
            if (T * E > limit) T = limit / E;
            const w4a8::RoutePlan p = w4a8::plan_route((int)T, E, 1);
            const bool ok = p.blocks >= 1 && p.blocks <= 512 && p.tokens >= 1 &&
                            (long long)p.blocks * p.tokens >= T &&
                            (long long)(p.blocks - 1) * p.tokens < T &&
                            p.workspace == (p.blocks == 1 ? 0 : (size_t)p.blocks * E * sizeof(int));
            if (!ok) {
                std::fprintf(stderr, "T %lld E %d: %d blocks of %d\n", T, E, p.blocks, p.tokens);
                ++fails;
            }
        }
    std::printf("route plans: %d failures\n", fails);
    return fails != 0;
}
