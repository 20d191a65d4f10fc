// tern_cursor.h -- where a token stands among packed sequences (host and
// device; no HIP headers, so that it is tested on the CPU).
#pragma once

#include <stdint.h>

#include "tern_plan.h"

namespace tern {

// cur is the last i in [0, S] with off[i] <= t (-1 before off[0]): the token
// belongs to sequence cur when 0 <= cur < S.  Offsets that do not ascend are
// only ever compared with t, so cur stays in [-1, S] and off is read at
// [0, S] whatever it holds.  off null: one sequence of T tokens.
struct Cursor {
    const int64_t *off;
    int64_t S, T, cur;

    TERN_HD int64_t at(int64_t i) const { return off ? off[i] : i * T; }
    TERN_HD bool live() const { return cur >= 0 && cur < S; }
    // first token of the sequence at the cursor, and of what follows it
    TERN_HD int64_t begin() const { return cur >= 0 ? at(cur) : INT64_MIN; }
    TERN_HD int64_t end() const { return cur < S ? at(cur + 1) : INT64_MAX; }

    TERN_HD void seek(int64_t t) {
        int64_t lo = -1, hi = S;
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) >> 1;
            if (at(mid) <= t) lo = mid;
            else hi = mid - 1;
        }
        cur = lo;
    }
    // To a later / an earlier token: one sequence on, and from there in steps that
    // double while they fall short and then halve.  A run of empty sequences takes
    // reads as its logarithm; one by one, a wave that crosses millions would be
    // waited for longer than the others wait.
    TERN_HD void forth(int64_t t) {
        if (cur >= S || at(cur + 1) > t) return;
        cur++;
        bool up = true;
        for (int64_t d = 1; d;) {
            if (d <= S - cur && at(cur + d) <= t) {
                cur += d;
                d = up ? 2 * d : d >> 1;
            } else {
                up = false;
                d >>= 1;
            }
        }
    }
    TERN_HD void back(int64_t t) {
        if (cur < 0 || at(cur) <= t) return;
        cur--;
        bool up = true;
        for (int64_t d = 1; d;) {
            if (d <= cur + 1 && at(cur - d + 1) > t) {
                cur -= d;
                d = up ? 2 * d : d >> 1;
            } else {
                up = false;
                d >>= 1;
            }
        }
    }
};

}  // namespace tern
