/* Which coincidences of a layer operator's output with its inputs are refused:
 * y / dx may be the very tensor of `add`, but not when another input lies there
 * too, since other workgroups still read that one while y is stored. Run on a
 * host without a GPU: a call that passes its checks stops at the device check.
 * Exit status 0 when every expectation holds. */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "libmuon.h"

static int fails = 0;
#define EXPECT(c)                                                \
    do {                                                         \
        if (!(c)) {                                              \
            fprintf(stderr, "FAIL line %d: %s\n", __LINE__, #c); \
            ++fails;                                             \
        }                                                        \
    } while (0)

/* addresses that are only compared, never read */
#define AT(n) ((void*)(uintptr_t)(0x100000000ull * (n)))

int main(void) {
    const muon_status reached = MUON_E_NO_DEVICE;
    char* const ws = AT(100);
    const size_t wsn = (size_t)1 << 31;

    /* tokens x features of few rows and many, of aligned rows and odd ones */
    const int64_t shape[][2] = {{1, 64}, {3, 64}, {64, 64}, {5, 7}, {1000, 1600}, {999, 1001}};
    for (size_t k = 0; k < sizeof(shape) / sizeof(shape[0]); ++k)
        for (int lay = 0; lay < 2; ++lay) {
            muon_linear d;
            muon_epilogue e;
            memset(&d, 0, sizeof(d));
            memset(&e, 0, sizeof(e));
            d.tokens = shape[k][0];
            d.in_features = d.out_features = shape[k][1];
            d.weight_layout = lay;
            e.add = AT(3);
            /* y over add alone */
            EXPECT(muon_linear_forward(&d, AT(1), AT(2), &e, AT(3), ws, wsn, NULL) == reached);
            EXPECT(muon_linear_grad_input(&d, AT(1), AT(2), &e, AT(3), ws, wsn, NULL) == reached);
            /* add may be an input where the output is elsewhere */
            EXPECT(muon_linear_forward(&d, AT(3), AT(2), &e, AT(4), ws, wsn, NULL) == reached);
            EXPECT(muon_linear_grad_input(&d, AT(3), AT(2), &e, AT(4), ws, wsn, NULL) == reached);
            /* y over add, which is x / dy too */
            EXPECT(muon_linear_forward(&d, AT(3), AT(2), &e, AT(3), ws, wsn, NULL) == MUON_E_INVALID_ARG);
            EXPECT(muon_linear_grad_input(&d, AT(3), AT(2), &e, AT(3), ws, wsn, NULL) == MUON_E_INVALID_ARG);
            /* y over add, which is w too (of as many rows, or fewer or more) */
            EXPECT(muon_linear_forward(&d, AT(1), AT(3), &e, AT(3), ws, wsn, NULL) == MUON_E_INVALID_ARG);
            EXPECT(muon_linear_grad_input(&d, AT(1), AT(3), &e, AT(3), ws, wsn, NULL) == MUON_E_INVALID_ARG);
            /* y over add, which holds the bias, or is the pre-activation too */
            e.bias = AT(3);
            EXPECT(muon_linear_forward(&d, AT(1), AT(2), &e, AT(3), ws, wsn, NULL) == MUON_E_INVALID_ARG);
            e.bias = NULL;
            e.z = AT(3);
            e.activation = MUON_ACT_GELU;
            EXPECT(muon_linear_forward(&d, AT(1), AT(2), &e, AT(3), ws, wsn, NULL) == MUON_E_INVALID_ARG);
            EXPECT(muon_linear_grad_input(&d, AT(1), AT(2), &e, AT(3), ws, wsn, NULL) == MUON_E_INVALID_ARG);
        }

    const int64_t rows[] = {1, 5, 1000}, cols[] = {8, 100, 1600, 9001};
    for (size_t r = 0; r < 3; ++r)
        for (size_t c = 0; c < 4; ++c)
            for (int type = 0; type < 3; ++type) {
                muon_layernorm m;
                memset(&m, 0, sizeof(m));
                m.rows = rows[r];
                m.cols = cols[c];
                m.dtype = type;
#define BACKWARD(dy, x, add, dx) \
    muon_layernorm_backward(&m, dy, x, NULL, AT(3), AT(4), add, dx, NULL, NULL, 0, NULL, 0, NULL)
                EXPECT(BACKWARD(AT(1), AT(2), AT(5), AT(5)) == reached);
                EXPECT(BACKWARD(AT(1), AT(2), AT(1), AT(5)) == reached);
                EXPECT(BACKWARD(AT(1), AT(2), AT(1), AT(1)) == MUON_E_INVALID_ARG);
                EXPECT(BACKWARD(AT(1), AT(2), AT(2), AT(2)) == MUON_E_INVALID_ARG);
            }

    if (fails) return 1;
    printf("all expectations hold\n");
    return 0;
}
