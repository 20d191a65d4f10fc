// The sequence cursor over long runs of empty sequences, on the CPU: it names the
// same sequences as a walk one by one, and crosses a run in a few reads (one
// by one, the crossings below are 10^11 of them).
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
    std::mt19937_64 rng(11);
    for (int rep = 0; rep < 3000; rep++) {
        // runs of empty sequences of 0 to 300 between sequences of 1 to 5 tokens
        std::vector<int64_t> off{0};
        for (int k = 0; k < 12; k++) {
            for (uint64_t e = rng() % 3 ? rng() % 300 : 0; e; e--) off.push_back(off.back());
            off.push_back(off.back() + 1 + (int64_t)(rng() % 5));
        }
        for (uint64_t e = rng() % 40; e; e--) off.push_back(off.back());
        const int64_t S = (int64_t)off.size() - 1, T = off.back() + (int64_t)(rng() % 4);
        Cursor f{off.data(), S, T, 0}, b{off.data(), S, T, 0};
        f.seek(0);
        b.seek(T);
        // strides of 1 to 4 tokens: several sequences may be passed at once
        for (int64_t t = 0; t <= T; t += 1 + (int64_t)(rng() % 4)) {
            int64_t c = -1;
            for (int64_t i = 0; i <= S; i++)
                if (off[(size_t)i] <= t) c = i;
            f.forth(t);
            need(f.cur == c, "forward over empty sequences");
        }
        for (int64_t t = T; t >= -1; t -= 1 + (int64_t)(rng() % 4)) {
            int64_t c = -1;
            for (int64_t i = 0; i <= S; i++)
                if (off[(size_t)i] <= t) c = i;
            b.back(t);
            need(b.cur == c, "backward over empty sequences");
        }
    }
    const int64_t S = int64_t(1) << 21;   // all empty but the first and the last, of one token each
    std::vector<int64_t> off((size_t)S + 1, 1);
    off[0] = 0;
    off[(size_t)S] = 2;
    int64_t sum = 0;
    for (int rep = 0; rep < 50000; rep++) {
        Cursor c{off.data(), S, 2, 0};
        c.forth(1);
        sum += c.cur;
        c.back(0);
        sum += c.cur;
    }
    need(sum == 50000 * (S - 1), "across the long run");
    // offsets that break the rules: inside [-1, S], and every walk ends
    for (int rep = 0; rep < 20000; rep++) {
        const int64_t n = (int64_t)(rng() % 70);
        std::vector<int64_t> bad((size_t)n + 1);
        for (auto &o : bad) o = rng() % 5 == 0 ? INT64_MAX : rng() % 5 == 0 ? INT64_MIN : (int64_t)(rng() % 90) - 20;
        Cursor c{bad.data(), n, 50, (int64_t)(rng() % (uint64_t)(n + 2)) - 1};
        for (int k = 0; k < 60; k++) {
            const int64_t t = (int64_t)(rng() % 80) - 10;
            if (rng() % 2) c.forth(t);
            else c.back(t);
            need(c.cur >= -1 && c.cur <= n, "left [-1, S]");
        }
    }
    std::puts("ok");
    return 0;
}
