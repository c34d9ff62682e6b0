// Which tile a product takes: for each line of the input (0 rows in out: 8-bit product;
// 1 rows experts in out layout: grouped forward; 2: grouped input gradient; 3: grouped
// weight gradient) the tile's kind and the pieces that the sums are cut into.
// Built with the entry points' own sources, whose plans are theirs, and launchers that
// do nothing.
#include "layers_grouped.cpp"
#include "layers_scaled.cpp"

#include <cstdio>

int main() {
    long long op, a, b, c, d, e;
    while (std::scanf("%lld %lld %lld %lld %lld %lld", &op, &a, &b, &c, &d, &e) == 6) {
        if (op == 0) {
            const ScaledPlan p = scaled_plan(a, c, b);
            std::printf("%d 1\n", (int)p.tile);
            continue;
        }
        // e: 0 [in, out], 1 [out, in]
        const GroupedPlan p = op == 1   ? rows_plan(a, b, d, c, e == 1)
                              : op == 2 ? rows_plan(a, b, c, d, e == 0)
                                        : weight_plan(a, b, e == 0 ? c : d, e == 0 ? d : c, false);
        std::printf("%d %d\n", (int)p.tile, p.pieces);
    }
    return 0;
}
