// How products are cut: for each line of the input (operation, tokens, in, out,
// weight layout, the byte offsets of the two operands' addresses from a 256-byte
// border, ld_x, ld_w and ld_y), the plan as
//   status, tile rows, tiles, whole tiles, pieces of each other tile, slices, rows read
//   as they are, first operand packed, second operand packed
// Built with layers.cpp itself, whose plans are its own, and launchers that do
// nothing.
#include "layers.cpp"

#include <cstdio>

int main() {
    long long op, t, i, o, lay, a, b, lx, lw, ly;
    while (std::scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld %lld", &op, &t, &i, &o, &lay, &a, &b, &lx, &lw,
                      &ly) == 10) {
        muon_linear d{};
        d.tokens = t;
        d.in_features = i;
        d.out_features = o;
        d.weight_layout = (int32_t)lay;
        d.ld_x = lx;
        d.ld_w = lw;
        d.ld_y = ly;
        Product P;
        // addresses that are only looked at
        const muon_status s = plan_product(d, (int)op, (void*)(uintptr_t)(4096 + a), (void*)(uintptr_t)(4096 + b), true, &P);
        const muon::GemmPlan& g = P.plan;
        std::printf("%d %d %d %d %d %d %d %d %d\n", (int)s, g.tile_m, g.tiles_m * g.tiles_n, g.whole, g.splits,
                    g.slices, (int)P.raw, (int)P.pack_a, (int)P.pack_b);
    }
    return 0;
}
