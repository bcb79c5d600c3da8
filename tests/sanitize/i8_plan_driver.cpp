// Answers, a line each: "grad PARTS M K N" with the tile (0: 256 x 256, 1: 256 x 128, 2: 128 x 64)
// and the number of runs of a gradient, "tile M K N PAIR CUS" with the tile of a product.
#include <stdio.h>

#include "i8_plan.h"

int main()
{
    char what[8];
    while (scanf("%7s", what) == 1) {
        long long a, b, c, d, e;
        if (what[0] == 'g' && scanf("%lld%lld%lld%lld", &a, &b, &c, &d) == 4) {
            const gq::GradPlan p = gq::grad_plan((int)a, b, c, d);
            printf("%d %d\n", p.tile, p.splits);
        } else if (what[0] == 't' && scanf("%lld%lld%lld%lld%lld", &a, &b, &c, &d, &e) == 5) {
            printf("%d 0\n", gq::i8_tile_choice(a, b, c, d != 0, e));
        } else {
            return 1;
        }
    }
    printf("all checks passed\n");
    return 0;
}
