// The tile kernels' division of K (csrc/k_parts.h) over all row lengths and part
// counts that a plan can choose: every K-tile belongs to one part, and every
// K-tile whose weights a wave loads, on any of its steps, lies in the row.  Test
// infrastructure: only tests/test_layer_k_parts.py builds and runs it.
#include <algorithm>
#include <cstdio>
#include <vector>

#include "k_parts.h"

template <int KIN>
static int walk(int all, int splits) {
    int fails = 0;
    const int parts = splits * KIN;
    std::vector<int> seen(all, 0);
    for (int ks = 0; ks < splits; ++ks) {
        auto first = [&](int kp) { return w4a8::k_part_first(all, ks * KIN + kp, parts); };
        int steps = 0;
        for (int kp = 0; kp < KIN; ++kp) steps = std::max(steps, first(kp + 1) - first(kp));
        steps += steps & 1;
        for (int kp = 0; kp < KIN; ++kp) {
            const int kt0 = first(kp), tiles = first(kp + 1) - kt0;
            const int last = w4a8::k_last_step<KIN>(tiles);
            auto load = [&](int step) {  // K-tile of a step's weights
                const int kt = kt0 + step;
                if (kt < 0 || kt >= all || (tiles > 0 && (kt < kt0 || kt >= kt0 + tiles)))
                    if (fails++ < 5)
                        std::fprintf(stderr, "%d K-tiles, %d splits of %d: part %d loads K-tile %d\n",
                                     all, splits, KIN, ks * KIN + kp, kt);
            };
            load(0);
            load(std::min(1, last));
            for (int kt = 0; kt < steps; ++kt) load(std::min(kt + 2, last));
            for (int kt = 0; kt < tiles; ++kt) ++seen[kt0 + kt];
        }
    }
    for (int n : seen) fails += n != 1;
    return fails;
}

int main() {
    int fails = 0;
    for (int all = 1; all <= 1024; all += all < 130 ? 1 : 37)
        for (int splits = 1; splits <= 16 && splits <= all; ++splits) {
            fails += walk<1>(all, splits);
            fails += walk<2>(all, splits);
        }
    std::printf("K parts: %d failures\n", fails);
    return fails != 0;
}
