// Every K up to 2^22 and number of groups of waves: each group has a run, the runs are the
// whole of K, and copies of scales and activations stay inside them.
#include <stdio.h>
#include <stdlib.h>

#include "mxfp4_krun.h"

#define CHECK(c)                                                                               \
    do {                                                                                       \
        if (!(c)) {                                                                            \
            fprintf(stderr, "K %d, %d groups, run %d: %s\n", K, KG, g, #c);                    \
            exit(1);                                                                           \
        }                                                                                      \
    } while (0)

template <int KG>
static int runs(int nblk)
{
    using namespace gq;
    const int K = 32 * nblk, mode = scale_mode<KG>(K);
    int g = 0;
    if (mode < 0) { // refused: fewer chunks than groups
        CHECK(nblk <= 8 * (KG - 1));
        return 0;
    }
    // scales come 16 bytes or by dwords from where they start, so rows are whole such pieces
    CHECK(mode != kScale16 || nblk % 16 == 0);
    CHECK(mode != kScale4 || nblk % 4 == 0);
    int end = 0;
    for (; g < KG; ++g) {
        const KRun r = k_run<KG>(nblk, mode, g);
        CHECK(r.first == end && r.blocks >= 1 && r.blocks <= r.longest);
        // a run's stages of two blocks, chunks of eight and scales of sixteen begin with it
        CHECK(r.first % (mode == kScale16 ? 16 : 8) == 0);
        CHECK(mode == kScale1 || r.blocks % (mode == kScale16 ? 16 : 4) == 0);
        // the others keep its barriers: as many steps as the longest run has stages
        CHECK((r.blocks + 1) / 2 <= (r.longest + 1) / 2);
        end += r.blocks;
    }
    CHECK(end == nblk);
    return 1;
}

int main()
{
    int launched[3] = {0, 0, 0};
    for (int nblk = 1; nblk <= 1 << 17; ++nblk) {
        launched[0] += runs<1>(nblk);
        launched[1] += runs<2>(nblk);
        launched[2] += runs<4>(nblk);
    }
    if (launched[0] != 1 << 17 || launched[1] != (1 << 17) - 8 || launched[2] != (1 << 17) - 24)
        return fprintf(stderr, "launched %d %d %d\n", launched[0], launched[1], launched[2]), 1;
    puts("all checks passed");
    return 0;
}
