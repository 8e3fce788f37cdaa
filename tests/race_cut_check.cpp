// Every alignment of a row's logits and noise, and every short vocabulary: the loads that
// csrc/race_cut.h allows lie inside the row, and each token is taken once.
#include <cstdio>
#include <vector>

#include "race_cut.h"

static int fail(const char* what, int logits, int noise, int per, int vocab) {
    std::printf("%s: logits at %d of %d, noise at %d, %d tokens\n", what, logits, per, noise, vocab);
    return 1;
}

int main() {
    for (int per : {4, 8})  // logits per 16 bytes
        for (int logits = 0; logits < per; ++logits)
            for (int noise = 0; noise < 4; ++noise)  // places of the row's first elements
                for (int vocab = 1; vocab < 100; ++vocab) {
                    int head = logits ? per - logits : 0;
                    if (head > vocab) head = vocab;
                    const int chunks = (vocab - head) / 8, phase = (noise + head) % 4;
                    const z3::RaceCut c = z3::race_cut(head, chunks, phase, vocab);
                    std::vector<int> seen(vocab, 0);
                    for (int i = 0; i < c.chunks; ++i) {
                        const int first = c.head + 8 * i;
                        if ((logits + first) % per != 0) return fail("logits off a boundary", logits, noise, per, vocab);
                        if ((noise + first) % 4 != phase) return fail("another phase", logits, noise, per, vocab);
                        const int lo = first - phase, hi = lo + (phase ? 12 : 8);
                        if (lo < 0 || hi > vocab) return fail("outside the row", logits, noise, per, vocab);
                        for (int k = 0; k < 8; ++k) ++seen[first + k];
                    }
                    for (int lane = 0; lane < 32; ++lane) {
                        const int t = z3::end_token(lane, c.head, c.head + 8 * c.chunks, vocab);
                        if (t >= vocab) return fail("end outside", logits, noise, per, vocab);
                        if (t >= 0) ++seen[t];
                    }
                    for (int n : seen)
                        if (n != 1) return fail("not once", logits, noise, per, vocab);
                    if (chunks - c.chunks > 2) return fail("too few chunks", logits, noise, per, vocab);
                    // the word of a 16-bit logit whose row starts `logits` elements behind a boundary
                    if (per == 8)
                        for (int t = 0; t < vocab; ++t) {
                            const bool upper = (logits + t) % 2 != 0;
                            const int lo = upper ? t - 1 : t;
                            if (z3::word_in_row(upper, t, vocab) != (lo >= 0 && lo + 2 <= vocab))
                                return fail("word", logits, noise, per, vocab);
                        }
                }
    std::printf("ok\n");
    return 0;
}
