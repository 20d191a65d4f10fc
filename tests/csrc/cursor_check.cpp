// The sequence cursor on the CPU, under the address sanitizer: on ascending
// offsets it names each token's sequence; on any others it neither reads
// outside the array nor leaves [-1, S], and every walk ends.
#include "../../ternary_weight_linear_tern_amd/csrc/tern_cursor.h"

#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

using tern::Cursor;

static void need(bool ok, const char *what) {
    if (!ok) {
        std::printf("cursor: %s\n", what);
        std::exit(1);
    }
}

int main() {
    std::mt19937_64 rng(7);
    for (int rep = 0; rep < 4000; rep++) {
        const int64_t S = (int64_t)(rng() % 9), T = (int64_t)(rng() % 60) + 1;
        std::vector<int64_t> off((size_t)S + 1);
        const bool good = rep % 2 == 0;
        if (good) {
            off[0] = 0;
            for (int64_t i = 1; i <= S; i++) off[(size_t)i] = off[(size_t)i - 1] + (int64_t)(rng() % 3 ? rng() % 12 : 0);
        } else {
            for (auto &o : off) {
                const uint64_t k = rng();
                o = k % 4 == 0 ? INT64_MAX : k % 4 == 1 ? INT64_MIN : (int64_t)(rng() % 120) - 30;
            }
        }
        auto owner = [&](int64_t t) {   // last i with off[i] <= t
            int64_t c = -1;
            for (int64_t i = 0; i <= S; i++)
                if (off[(size_t)i] <= t) c = i;
            return c;
        };
        Cursor f{off.data(), S, T, 0}, b{off.data(), S, T, 0}, x{off.data(), S, T, 0};
        f.seek(0);
        b.seek(T - 1);
        for (int64_t t = 0; t < T; t++) {
            const int64_t u = T - 1 - t;
            if (t >= f.end()) f.forth(t);
            if (u < b.begin()) b.back(u);
            x.seek(t);
            for (const Cursor *c : {&f, &b, &x}) need(c->cur >= -1 && c->cur <= S, "left [-1, S]");
            if (good) {
                need(f.cur == owner(t), "forward walk");
                need(b.cur == owner(u), "backward walk");
                need(x.cur == owner(t), "search");
                need(f.begin() <= t && t < f.end(), "bounds of the sequence");
            }
        }
        Cursor one{nullptr, 1, T, 0};
        one.seek(T - 1);
        need(one.live() && one.begin() == 0 && one.end() == T, "one sequence");
        one.seek(T);
        need(!one.live(), "behind the one sequence");
    }
    std::puts("ok");
    return 0;
}
