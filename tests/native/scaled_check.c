/* Host-side exercise of the C ABI of the RMS norm, the 8-bit and the grouped layer
 * operators for the sanitizer build: every refusal, sizes up to the limits, and (on a
 * host without a GPU) that a valid call stops at the device check. Exit status 0 when
 * every expectation holds. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "libmuon.h"

static int fails = 0;
#define EXPECT(c)                                                      \
    do {                                                               \
        if (!(c)) {                                                    \
            fprintf(stderr, "FAIL line %d: %s\n", __LINE__, #c);       \
            ++fails;                                                   \
        }                                                              \
    } while (0)

/* addresses that are only compared, never read */
#define AT(n) ((void*)(uintptr_t)(0x100000000ull * (n)))
#define reached MUON_E_NO_DEVICE
#define BAD_ARG MUON_E_INVALID_ARG

static muon_eight eight(void* data, void* scale) {
    muon_eight q;
    memset(&q, 0, sizeof(q));
    q.data = data;
    q.scale = scale;
    return q;
}

static void rms(void) {
    muon_rmsnorm d;
    memset(&d, 0, sizeof(d));
    d.rows = 5;
    d.cols = 100;
    d.eps = 1e-5f;
    size_t n = 7;
    EXPECT(muon_rmsnorm_workspace_bytes(NULL, &n) == BAD_ARG);
    EXPECT(muon_rmsnorm_workspace_bytes(&d, NULL) == BAD_ARG);
    EXPECT(muon_rmsnorm_workspace_bytes(&d, &n) == MUON_OK && n >= 8 * 100 * 4);
    muon_eight q = eight(AT(20), AT(21));
    for (int k = 0; k < 13; ++k) {
        muon_rmsnorm b = d;
        muon_status want = MUON_E_SHAPE;
        if (k == 0) b.rows = -1;
        if (k == 1) b.rows = (int64_t)1 << 24;
        if (k == 2) b.cols = 0;
        if (k == 3) b.cols = ((int64_t)1 << 21) + 1;
        if (k > 3) want = BAD_ARG;
        if (k == 4) b.dtype = 3;
        if (k == 5) b.eps = NAN;
        if (k == 6) b.eps = -1e-5f;
        if (k == 7) b.eps = INFINITY;
        if (k > 7) want = MUON_E_LAYOUT;
        if (k == 8) b.ld_x = 99;
        if (k == 9) b.ld_add = -1;
        if (k == 10) b.ld_sum = ((int64_t)1 << 21) + 1;
        if (k == 11) b.ld_y = 5;
        if (k == 12) b.ld_dx = 99;
        EXPECT(muon_rmsnorm_workspace_bytes(&b, &n) == want);
        EXPECT(muon_rmsnorm_forward(&b, AT(1), NULL, NULL, NULL, AT(2), NULL, AT(3), NULL) == want);
        EXPECT(muon_rmsnorm_backward(&b, AT(1), AT(2), NULL, AT(3), NULL, AT(4), NULL, 0, NULL, 0, NULL) == want);
        EXPECT(muon_op_last_error()[0] != 0);
    }
    EXPECT(muon_rmsnorm_forward(&d, AT(1), NULL, NULL, NULL, AT(2), NULL, AT(3), NULL) == reached);
    EXPECT(muon_rmsnorm_forward(&d, AT(1), NULL, NULL, NULL, NULL, &q, AT(3), NULL) == reached);
    EXPECT(muon_rmsnorm_forward(&d, AT(1), AT(4), AT(5), AT(6), AT(2), &q, AT(3), NULL) == reached);
    /* neither output; a residual without its sum and the other way round; nulls */
    EXPECT(muon_rmsnorm_forward(&d, AT(1), NULL, NULL, NULL, NULL, NULL, AT(3), NULL) == BAD_ARG);
    EXPECT(muon_rmsnorm_forward(&d, AT(1), AT(4), NULL, NULL, AT(2), NULL, AT(3), NULL) == BAD_ARG);
    EXPECT(muon_rmsnorm_forward(&d, AT(1), NULL, NULL, AT(6), AT(2), NULL, AT(3), NULL) == BAD_ARG);
    EXPECT(muon_rmsnorm_forward(&d, NULL, NULL, NULL, NULL, AT(2), NULL, AT(3), NULL) == BAD_ARG);
    EXPECT(muon_rmsnorm_forward(&d, AT(1), NULL, NULL, NULL, AT(2), NULL, NULL, NULL) == BAD_ARG);
    /* the sum may replace x or the residual, and nothing else overlaps */
    EXPECT(muon_rmsnorm_forward(&d, AT(1), AT(4), NULL, AT(1), AT(2), NULL, AT(3), NULL) == reached);
    EXPECT(muon_rmsnorm_forward(&d, AT(1), AT(4), NULL, AT(4), AT(2), NULL, AT(3), NULL) == reached);
    EXPECT(muon_rmsnorm_forward(&d, AT(1), AT(4), NULL, (char*)AT(4) + 2, AT(2), NULL, AT(3), NULL) == BAD_ARG);
    d.ld_sum = 128;
    EXPECT(muon_rmsnorm_forward(&d, AT(1), AT(4), NULL, AT(4), AT(2), NULL, AT(3), NULL) == BAD_ARG);
    d.ld_sum = 0;
    EXPECT(muon_rmsnorm_forward(&d, AT(1), NULL, NULL, NULL, AT(1), NULL, AT(3), NULL) == BAD_ARG);
    EXPECT(muon_rmsnorm_forward(&d, AT(1), AT(4), NULL, AT(6), AT(6), NULL, AT(3), NULL) == BAD_ARG);
    EXPECT(muon_rmsnorm_forward(&d, AT(1), NULL, AT(3), NULL, AT(2), NULL, AT(3), NULL) == BAD_ARG);
    q.data = AT(2);
    EXPECT(muon_rmsnorm_forward(&d, AT(1), NULL, NULL, NULL, AT(2), &q, AT(3), NULL) == BAD_ARG);
    q.data = AT(1);
    EXPECT(muon_rmsnorm_forward(&d, AT(1), NULL, NULL, NULL, AT(2), &q, AT(3), NULL) == BAD_ARG);
    q = eight(AT(20), AT(20));
    EXPECT(muon_rmsnorm_forward(&d, AT(1), NULL, NULL, NULL, NULL, &q, AT(3), NULL) == BAD_ARG);
    q = eight(AT(20), AT(3));
    EXPECT(muon_rmsnorm_forward(&d, AT(1), NULL, NULL, NULL, NULL, &q, AT(3), NULL) == BAD_ARG);
    EXPECT(muon_rmsnorm_forward(&d, (char*)AT(1) + 1, NULL, NULL, NULL, AT(2), NULL, AT(3), NULL) == MUON_E_LAYOUT);
    EXPECT(muon_rmsnorm_forward(&d, AT(1), NULL, NULL, NULL, AT(2), NULL, (float*)((char*)AT(3) + 2), NULL) ==
           MUON_E_LAYOUT);
    /* backward */
    char* const ws = AT(100);
    EXPECT(muon_rmsnorm_backward(&d, AT(1), AT(2), NULL, AT(3), NULL, AT(4), NULL, 0, NULL, 0, NULL) == reached);
    EXPECT(muon_rmsnorm_backward(&d, AT(1), AT(2), NULL, AT(3), AT(4), AT(4), NULL, 0, NULL, 0, NULL) == reached);
    EXPECT(muon_rmsnorm_backward(&d, AT(1), AT(2), NULL, AT(3), AT(1), AT(1), NULL, 0, NULL, 0, NULL) == BAD_ARG);
    EXPECT(muon_rmsnorm_backward(&d, AT(1), AT(2), NULL, AT(3), NULL, AT(2), NULL, 0, NULL, 0, NULL) == BAD_ARG);
    EXPECT(muon_rmsnorm_backward(&d, AT(1), AT(2), NULL, NULL, NULL, AT(4), NULL, 0, NULL, 0, NULL) == BAD_ARG);
    EXPECT(muon_rmsnorm_backward(&d, AT(1), AT(2), NULL, AT(3), NULL, AT(4), AT(5), 0, NULL, 0, NULL) ==
           MUON_E_WORKSPACE);
    EXPECT(muon_rmsnorm_workspace_bytes(&d, &n) == MUON_OK);
    EXPECT(muon_rmsnorm_backward(&d, AT(1), AT(2), NULL, AT(3), NULL, AT(4), AT(5), 0, ws, n - 1, NULL) ==
           MUON_E_WORKSPACE);
    EXPECT(muon_rmsnorm_backward(&d, AT(1), AT(2), NULL, AT(3), NULL, AT(4), AT(5), 0, ws + 16, n, NULL) ==
           MUON_E_WORKSPACE);
    EXPECT(muon_rmsnorm_backward(&d, ws, AT(2), NULL, AT(3), NULL, AT(4), AT(5), 0, ws, n, NULL) == BAD_ARG);
    EXPECT(muon_rmsnorm_backward(&d, AT(1), AT(2), AT(5), AT(3), NULL, AT(4), AT(5), 0, ws, n, NULL) == BAD_ARG);
    EXPECT(muon_rmsnorm_backward(&d, AT(1), AT(2), NULL, AT(3), NULL, AT(4), AT(5), 1, ws, n, NULL) == reached);
    d.rows = 0;
    EXPECT(muon_rmsnorm_forward(&d, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL) == MUON_OK);
    EXPECT(muon_rmsnorm_backward(&d, NULL, NULL, NULL, NULL, NULL, NULL, NULL, 0, NULL, 0, NULL) == MUON_OK);
    EXPECT(muon_rmsnorm_backward(&d, NULL, NULL, NULL, NULL, NULL, NULL, AT(5), 1, ws, 256, NULL) == MUON_OK);
    EXPECT(muon_rmsnorm_backward(&d, NULL, NULL, NULL, NULL, NULL, NULL, AT(5), 0, ws, 256, NULL) == reached);
}

static void quantize(void) {
    muon_eight q = eight(AT(2), AT(3)), t = eight(AT(4), AT(5));
    EXPECT(muon_quantize(9, 100, 0, MUON_TYPE_FP32, AT(1), &q, NULL) == reached);
    EXPECT(muon_quantize(0, 100, 0, MUON_TYPE_FP32, NULL, NULL, NULL) == MUON_OK);
    EXPECT(muon_quantize(-1, 100, 0, 0, AT(1), &q, NULL) == MUON_E_SHAPE);
    EXPECT(muon_quantize(9, 0, 0, 0, AT(1), &q, NULL) == MUON_E_SHAPE);
    EXPECT(muon_quantize((int64_t)1 << 23, (int64_t)1 << 21, 0, 0, AT(1), &q, NULL) == MUON_E_SHAPE);
    EXPECT(muon_quantize(9, 100, 99, 0, AT(1), &q, NULL) == MUON_E_LAYOUT);
    EXPECT(muon_quantize(9, 100, 0, 3, AT(1), &q, NULL) == BAD_ARG);
    EXPECT(muon_quantize(9, 100, 0, 0, NULL, &q, NULL) == BAD_ARG);
    EXPECT(muon_quantize(9, 100, 0, 0, AT(1), NULL, NULL) == BAD_ARG);
    EXPECT(muon_quantize(9, 100, 0, 0, (char*)AT(1) + 1, &q, NULL) == MUON_E_LAYOUT);
    EXPECT(muon_quantize(9, 100, 0, 0, AT(2), &q, NULL) == BAD_ARG);
    for (int k = 0; k < 8; ++k) {
        muon_eight b = q;
        muon_status want = k < 4 ? BAD_ARG : MUON_E_LAYOUT;
        if (k == 0) b.format = 2;
        if (k == 1) b.reserved = 1;
        if (k == 2) b.data = NULL;
        if (k == 3) b.scale = NULL;
        if (k == 4) b.data = (char*)AT(2) + 8;
        if (k == 5) b.ld = 120;
        if (k == 6) b.ld = 96;
        if (k == 7) b.scale = (float*)((char*)AT(3) + 2);
        EXPECT(muon_quantize(9, 100, 0, 0, AT(1), &b, NULL) == want);
        EXPECT(muon_quantize_weight(9, 100, 0, 0, AT(1), &b, NULL, NULL) == want);
        if (k != 6) EXPECT(muon_quantize_weight(100, 100, 0, 0, AT(1), NULL, &b, NULL) == want);
    }
    /* a row goes on to the next multiple of 16: 112 bytes, the last one too */
    q.scale = (float*)((char*)AT(2) + 9 * 112);
    EXPECT(muon_quantize(9, 100, 0, 0, AT(1), &q, NULL) == reached);
    q.scale = (float*)((char*)AT(2) + 9 * 112 - 4);
    EXPECT(muon_quantize(9, 100, 0, 0, AT(1), &q, NULL) == BAD_ARG);
    q = eight(AT(2), AT(3));
    EXPECT(muon_quantize_weight(300, 100, 0, 2, AT(1), &q, &t, NULL) == reached);
    EXPECT(muon_quantize_weight(300, 100, 0, 2, AT(1), NULL, NULL, NULL) == BAD_ARG);
    EXPECT(muon_quantize_weight(300, 100, 0, 2, NULL, &q, &t, NULL) == BAD_ARG);
    EXPECT(muon_quantize_weight(0, 100, 0, 2, AT(1), &q, &t, NULL) == MUON_E_SHAPE);
    EXPECT(muon_quantize_weight((int64_t)1 << 21, (int64_t)1 << 21, 0, 2, AT(1), &q, &t, NULL) == MUON_E_SHAPE);
    EXPECT(muon_quantize_weight(300, 100, 99, 2, AT(1), &q, &t, NULL) == MUON_E_LAYOUT);
    q.format = MUON_EIGHT_E5M2; /* rows have it, weights not */
    EXPECT(muon_quantize_weight(300, 100, 0, 2, AT(1), &q, NULL, NULL) == BAD_ARG);
    q.format = 0;
    t.data = AT(2);
    EXPECT(muon_quantize_weight(300, 100, 0, 2, AT(1), &q, &t, NULL) == BAD_ARG);
    t.data = AT(1);
    EXPECT(muon_quantize_weight(300, 100, 0, 2, AT(1), &q, &t, NULL) == BAD_ARG);
    t = eight(AT(4), AT(3));
    EXPECT(muon_quantize_weight(300, 100, 0, 2, AT(1), &q, &t, NULL) == BAD_ARG);
}

static void scaled(void) {
    muon_linear d;
    memset(&d, 0, sizeof(d));
    d.tokens = 64;
    d.in_features = 96;
    d.out_features = 128;
    d.weight_layout = MUON_WEIGHT_OUT_IN;
    muon_eight x = eight(AT(1), AT(2)), w = eight(AT(3), AT(4));
    muon_epilogue e;
    memset(&e, 0, sizeof(e));
    EXPECT(muon_linear_scaled_forward(&d, &x, &w, NULL, AT(5), NULL) == reached);
    EXPECT(muon_linear_scaled_forward(NULL, &x, &w, NULL, AT(5), NULL) == BAD_ARG);
    EXPECT(muon_linear_scaled_grad_input(&d, &x, &w, NULL, AT(5), NULL) == BAD_ARG); /* [out, in] */
    for (int k = 0; k < 10; ++k) {
        muon_linear b = d;
        muon_status want = MUON_E_SHAPE;
        if (k == 0) b.tokens = -1;
        if (k == 1) b.tokens = (int64_t)1 << 24;
        if (k == 2) b.in_features = 0;
        if (k == 3) b.out_features = INT64_MAX;
        if (k > 3) want = BAD_ARG;
        if (k == 4) b.dtype = MUON_TYPE_FP32;
        if (k == 5) b.weight_layout = MUON_WEIGHT_IN_OUT;
        if (k == 6) b.weight_layout = 7;
        if (k > 6) want = MUON_E_LAYOUT;
        if (k == 7) b.ld_x = 96;
        if (k == 8) b.ld_w = 96;
        if (k == 9) b.ld_y = 127;
        EXPECT(muon_linear_scaled_forward(&b, &x, &w, NULL, AT(5), NULL) == want);
    }
    EXPECT(muon_linear_scaled_forward(&d, NULL, &w, NULL, AT(5), NULL) == BAD_ARG);
    EXPECT(muon_linear_scaled_forward(&d, &x, NULL, NULL, AT(5), NULL) == BAD_ARG);
    EXPECT(muon_linear_scaled_forward(&d, &x, &w, NULL, NULL, NULL) == BAD_ARG);
    EXPECT(muon_linear_scaled_forward(&d, &x, &w, NULL, (char*)AT(5) + 1, NULL) == MUON_E_LAYOUT);
    x.format = MUON_EIGHT_E5M2;
    EXPECT(muon_linear_scaled_forward(&d, &x, &w, NULL, AT(5), NULL) == reached);
    w.format = MUON_EIGHT_E5M2;
    EXPECT(muon_linear_scaled_forward(&d, &x, &w, NULL, AT(5), NULL) == BAD_ARG);
    w.format = 0;
    x.ld = 104;
    EXPECT(muon_linear_scaled_forward(&d, &x, &w, NULL, AT(5), NULL) == MUON_E_LAYOUT);
    x.ld = 112;
    EXPECT(muon_linear_scaled_forward(&d, &x, &w, NULL, AT(5), NULL) == reached);
    /* outputs over operands or scales */
    EXPECT(muon_linear_scaled_forward(&d, &x, &w, NULL, AT(1), NULL) == BAD_ARG);
    EXPECT(muon_linear_scaled_forward(&d, &x, &w, NULL, AT(2), NULL) == BAD_ARG);
    EXPECT(muon_linear_scaled_forward(&d, &x, &w, NULL, (char*)AT(4) - 2, NULL) == BAD_ARG);
    e.add = AT(5);
    EXPECT(muon_linear_scaled_forward(&d, &x, &w, &e, AT(5), NULL) == reached);
    e.add = (char*)AT(5) + 2;
    EXPECT(muon_linear_scaled_forward(&d, &x, &w, &e, AT(5), NULL) == BAD_ARG);
    memset(&e, 0, sizeof(e));
    e.z = AT(5);
    EXPECT(muon_linear_scaled_forward(&d, &x, &w, &e, AT(5), NULL) == BAD_ARG);
    e.z = AT(6);
    e.ld_z = 127;
    EXPECT(muon_linear_scaled_forward(&d, &x, &w, &e, AT(5), NULL) == MUON_E_LAYOUT);
    memset(&e, 0, sizeof(e));
    e.activation = 6;
    EXPECT(muon_linear_scaled_forward(&d, &x, &w, &e, AT(5), NULL) == BAD_ARG);
    /* the way back: dy [64, 128], w [96, 128], dx [64, 96] */
    d.weight_layout = MUON_WEIGHT_IN_OUT;
    x.ld = 0;
    memset(&e, 0, sizeof(e));
    EXPECT(muon_linear_scaled_grad_input(&d, &x, &w, NULL, AT(5), NULL) == reached);
    e.activation = MUON_ACT_RELU;
    EXPECT(muon_linear_scaled_grad_input(&d, &x, &w, &e, AT(5), NULL) == BAD_ARG);
    e.z = AT(6);
    EXPECT(muon_linear_scaled_grad_input(&d, &x, &w, &e, AT(5), NULL) == reached);
    e.z = AT(5);
    EXPECT(muon_linear_scaled_grad_input(&d, &x, &w, &e, AT(5), NULL) == BAD_ARG);
    memset(&e, 0, sizeof(e));
    e.bias = AT(7);
    EXPECT(muon_linear_scaled_grad_input(&d, &x, &w, &e, AT(5), NULL) == BAD_ARG);
    d.ld_y = 128;
    EXPECT(muon_linear_scaled_grad_input(&d, &x, &w, NULL, AT(5), NULL) == MUON_E_LAYOUT);
    d.ld_y = 0;
    d.tokens = 0;
    EXPECT(muon_linear_scaled_grad_input(&d, NULL, NULL, NULL, NULL, NULL) == MUON_OK);
    /* sizes to the limits */
    const int64_t sizes[] = {1, 7, 33, 128, 257, 1600, 50304, (int64_t)1 << 21};
    const int64_t tokens[] = {1, 17, 33, 1000, 131072, ((int64_t)1 << 24) - 1};
    d.weight_layout = MUON_WEIGHT_OUT_IN;
    for (size_t a = 0; a < 8; ++a)
        for (size_t b = 0; b < 8; ++b)
            for (size_t t = 0; t < 6; ++t) {
                d.tokens = tokens[t];
                d.in_features = sizes[a];
                d.out_features = sizes[b];
                x = eight(AT(1 << 20), AT(2 << 20));
                w = eight(AT(3 << 20), AT(4 << 20));
                const muon_status s = muon_linear_scaled_forward(&d, &x, &w, NULL, AT(5 << 20), NULL);
                EXPECT(s == reached || s == MUON_E_SHAPE);
                if (tokens[t] <= 131072 && sizes[b] <= 50304) EXPECT(s == reached);
            }
}

static void grouped(void) {
    muon_grouped d;
    memset(&d, 0, sizeof(d));
    d.rows = 100;
    d.experts = 4;
    d.in_features = 96;
    d.out_features = 128;
    muon_epilogue e;
    memset(&e, 0, sizeof(e));
    int32_t* const off = AT(9);
    EXPECT(muon_grouped_linear_forward(&d, AT(1), AT(2), off, NULL, AT(3), NULL) == reached);
    EXPECT(muon_grouped_linear_grad_input(&d, AT(1), AT(2), off, NULL, AT(3), NULL) == reached);
    EXPECT(muon_grouped_linear_grad_weight(&d, AT(1), AT(2), off, AT(3), AT(4), 0, NULL, 0, NULL) == reached);
    for (int k = 0; k < 15; ++k) {
        muon_grouped b = d;
        muon_status want = MUON_E_SHAPE;
        if (k == 0) b.rows = -1;
        if (k == 1) b.rows = (int64_t)1 << 24;
        if (k == 2) b.experts = 0;
        if (k == 3) b.experts = 65537;
        if (k == 4) b.in_features = 7;
        if (k == 5) b.out_features = 7;
        if (k == 6) b.in_features = ((int64_t)1 << 21) + 1;
        if (k > 6) want = BAD_ARG;
        if (k == 7) b.dtype = MUON_TYPE_FP32;
        if (k == 8) b.weight_layout = 2;
        if (k > 8) want = MUON_E_LAYOUT;
        if (k == 9) b.ld_x = 95;
        if (k == 10) b.ld_w = 127;
        if (k == 11) b.ld_y = -128;
        if (k == 12) b.stride_w = 96 * 128 - 1;
        if (k == 13) b.stride_w = -1;
        if (k == 14) b.ld_w = 130, b.stride_w = 96 * 128;
        EXPECT(muon_grouped_linear_forward(&b, AT(1), AT(2), off, NULL, AT(3), NULL) == want);
        EXPECT(muon_grouped_linear_grad_input(&b, AT(1), AT(2), off, NULL, AT(3), NULL) == want);
        EXPECT(muon_grouped_linear_grad_weight(&b, AT(1), AT(2), off, AT(3), NULL, 0, NULL, 0, NULL) == want);
    }
    EXPECT(muon_grouped_linear_forward(NULL, AT(1), AT(2), off, NULL, AT(3), NULL) == BAD_ARG);
    EXPECT(muon_grouped_linear_forward(&d, NULL, AT(2), off, NULL, AT(3), NULL) == BAD_ARG);
    EXPECT(muon_grouped_linear_forward(&d, AT(1), NULL, off, NULL, AT(3), NULL) == BAD_ARG);
    EXPECT(muon_grouped_linear_forward(&d, AT(1), AT(2), NULL, NULL, AT(3), NULL) == BAD_ARG);
    EXPECT(muon_grouped_linear_forward(&d, AT(1), AT(2), off, NULL, NULL, NULL) == BAD_ARG);
    EXPECT(muon_grouped_linear_forward(&d, AT(1), AT(2), (int32_t*)((char*)off + 2), NULL, AT(3), NULL) ==
           MUON_E_LAYOUT);
    EXPECT(muon_grouped_linear_forward(&d, (char*)AT(1) + 1, AT(2), off, NULL, AT(3), NULL) == MUON_E_LAYOUT);
    /* y over x, over the last expert's last weight, over the offsets, over the last expert's bias */
    EXPECT(muon_grouped_linear_forward(&d, AT(1), AT(2), off, NULL, AT(1), NULL) == BAD_ARG);
    EXPECT(muon_grouped_linear_forward(&d, AT(1), AT(2), off, NULL, (char*)AT(2) + 4 * 96 * 128 * 2 - 2, NULL) ==
           BAD_ARG);
    EXPECT(muon_grouped_linear_forward(&d, AT(1), AT(2), off, NULL, (char*)AT(2) + 4 * 96 * 128 * 2, NULL) == reached);
    EXPECT(muon_grouped_linear_forward(&d, AT(1), AT(2), off, NULL, (char*)off + 16, NULL) == BAD_ARG);
    EXPECT(muon_grouped_linear_forward(&d, AT(1), AT(2), off, NULL, (char*)off + 20, NULL) == reached);
    e.bias = AT(4);
    EXPECT(muon_grouped_linear_forward(&d, AT(1), AT(2), off, &e, (char*)AT(4) + 4 * 128 * 4 - 4, NULL) == BAD_ARG);
    EXPECT(muon_grouped_linear_grad_input(&d, AT(1), AT(2), off, &e, AT(3), NULL) == BAD_ARG);
    memset(&e, 0, sizeof(e));
    e.add = AT(3);
    EXPECT(muon_grouped_linear_forward(&d, AT(1), AT(2), off, &e, AT(3), NULL) == reached);
    e.z = AT(3);
    EXPECT(muon_grouped_linear_forward(&d, AT(1), AT(2), off, &e, AT(3), NULL) == BAD_ARG);
    memset(&e, 0, sizeof(e));
    e.activation = MUON_ACT_SILU;
    EXPECT(muon_grouped_linear_grad_input(&d, AT(1), AT(2), off, &e, AT(3), NULL) == BAD_ARG);
    e.z = AT(5);
    EXPECT(muon_grouped_linear_grad_input(&d, AT(1), AT(2), off, &e, AT(3), NULL) == reached);
    EXPECT(muon_grouped_linear_grad_weight(&d, AT(1), AT(2), off, NULL, NULL, 0, NULL, 0, NULL) == BAD_ARG);
    EXPECT(muon_grouped_linear_grad_weight(&d, AT(1), AT(2), off, AT(3), AT(3), 0, NULL, 0, NULL) == BAD_ARG);
    EXPECT(muon_grouped_linear_grad_weight(&d, AT(1), AT(2), off, AT(2), NULL, 0, NULL, 0, NULL) == BAD_ARG);
    EXPECT(muon_grouped_linear_grad_weight(&d, AT(1), AT(2), off, AT(3), (float*)AT(9), 0, NULL, 0, NULL) == BAD_ARG);
    EXPECT(muon_grouped_linear_grad_weight(&d, AT(1), AT(2), off, (float*)((char*)AT(3) + 2), NULL, 0, NULL, 0, NULL) ==
           MUON_E_LAYOUT);
    /* many rows of few features: pieces of the rows, whose sums need a workspace */
    size_t n = 7;
    EXPECT(muon_grouped_linear_workspace_bytes(&d, AT(1), AT(2), &n) == MUON_OK && n == 0);
    EXPECT(muon_grouped_linear_workspace_bytes(&d, AT(1), AT(2), NULL) == BAD_ARG);
    EXPECT(muon_grouped_linear_workspace_bytes(NULL, AT(1), AT(2), &n) == BAD_ARG);
    d.rows = 100000;
    for (int odd = 0; odd < 2; ++odd) {
        void* x = (char*)AT(1) + 2 * odd;
        char* const ws = AT(100);
        EXPECT(muon_grouped_linear_workspace_bytes(&d, x, AT(2), &n) == MUON_OK && n >= 2 * 4 * 96 * 128 * 4);
        EXPECT(muon_grouped_linear_grad_weight(&d, x, AT(2), off, AT(3), AT(4), 1, NULL, 0, NULL) == MUON_E_WORKSPACE);
        EXPECT(muon_grouped_linear_grad_weight(&d, x, AT(2), off, AT(3), AT(4), 1, ws, n - 1, NULL) ==
               MUON_E_WORKSPACE);
        EXPECT(muon_grouped_linear_grad_weight(&d, x, AT(2), off, AT(3), AT(4), 1, ws + 16, n, NULL) ==
               MUON_E_WORKSPACE);
        EXPECT(muon_grouped_linear_grad_weight(&d, x, AT(2), off, AT(3), AT(4), 1, ws, n, NULL) == reached);
        EXPECT(muon_grouped_linear_grad_weight(&d, x, AT(2), off, (float*)(ws + n - 256), AT(4), 1, ws, n, NULL) ==
               BAD_ARG);
        EXPECT(muon_grouped_linear_grad_weight(&d, x, AT(2), off, AT(3), (float*)ws, 1, ws, n, NULL) == BAD_ARG);
        EXPECT(muon_grouped_linear_grad_weight(&d, x, ws, off, AT(3), AT(4), 1, ws, n, NULL) == BAD_ARG);
        EXPECT(muon_grouped_linear_grad_weight(&d, x, AT(2), (int32_t*)ws, AT(3), AT(4), 1, ws, n, NULL) == BAD_ARG);
    }
    d.rows = 0;
    EXPECT(muon_grouped_linear_forward(&d, NULL, NULL, NULL, NULL, NULL, NULL) == MUON_OK);
    EXPECT(muon_grouped_linear_grad_input(&d, NULL, NULL, NULL, NULL, NULL, NULL) == MUON_OK);
    EXPECT(muon_grouped_linear_grad_weight(&d, NULL, NULL, off, AT(3), NULL, 0, NULL, 0, NULL) == reached);
    EXPECT(muon_grouped_linear_grad_weight(&d, NULL, NULL, NULL, AT(3), NULL, 0, NULL, 0, NULL) == BAD_ARG);
    const int64_t sizes[] = {8, 33, 128, 1600, 50304, (int64_t)1 << 21};
    const int64_t rows[] = {1, 17, 1000, 131072, ((int64_t)1 << 24) - 1};
    const int64_t experts[] = {1, 3, 64, 1000, 65536};
    for (size_t a = 0; a < 6; ++a)
        for (size_t b = 0; b < 6; ++b)
            for (size_t r = 0; r < 5; ++r)
                for (size_t x = 0; x < 5; ++x)
                    for (int lay = 0; lay < 2; ++lay) {
                        memset(&d, 0, sizeof(d));
                        d.rows = rows[r];
                        d.experts = experts[x];
                        d.in_features = sizes[a];
                        d.out_features = sizes[b];
                        d.weight_layout = lay;
                        void *p = AT(1 << 22), *w = AT(1 << 23), *y = AT(3 << 22);
                        /* the largest reach over the next of these addresses */
                        const int huge = experts[x] * sizes[a] > ((int64_t)1 << 52) / sizes[b];
                        muon_status s = muon_grouped_linear_forward(&d, p, w, off, NULL, y, NULL);
                        EXPECT(s == reached || s == MUON_E_SHAPE || (huge && s == BAD_ARG));
                        if (rows[r] <= 131072 && experts[x] <= 64 && sizes[b] <= 1600) EXPECT(s == reached);
                        size_t n = 0;
                        EXPECT(muon_grouped_linear_workspace_bytes(&d, p, y, &n) == MUON_OK);
                        s = muon_grouped_linear_grad_weight(&d, p, y, off, w, NULL, 0, AT(1 << 24), n, NULL);
                        EXPECT(s == reached || s == MUON_E_SHAPE || (huge && s == BAD_ARG));
                        if (experts[x] <= 64 && sizes[a] <= 1600 && sizes[b] <= 1600) EXPECT(s == reached);
                    }
}

int main(void) {
    rms();
    quantize();
    scaled();
    grouped();
    if (fails) return 1;
    printf("all expectations hold\n");
    return 0;
}
