/* Host-side exercise of the layer operators' C ABI for the sanitizer build:
 * every refusal, workspace sizes over sizes from one element to the limits,
 * and (on a host without a GPU) that a valid call stops at the device check.
 * Exit status 0 when every expectation holds. */
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

static muon_linear lin(int64_t t, int64_t i, int64_t o) {
    muon_linear d;
    memset(&d, 0, sizeof(d));
    d.tokens = t;
    d.in_features = i;
    d.out_features = o;
    return d;
}

static muon_layernorm norm(int64_t r, int64_t c, int dtype) {
    muon_layernorm d;
    memset(&d, 0, sizeof(d));
    d.rows = r;
    d.cols = c;
    d.dtype = dtype;
    d.eps = 1e-5f;
    return d;
}

int main(int argc, char** argv) {
    const muon_status reached = argc > 1 && strcmp(argv[1], "gpu") == 0 ? MUON_OK : MUON_E_NO_DEVICE;
    size_t n = 7;
    muon_linear d = lin(64, 96, 128);
    muon_epilogue e;
    memset(&e, 0, sizeof(e));

    /* descriptors */
    EXPECT(muon_linear_workspace_bytes(NULL, 0, AT(1), AT(2), &n) == MUON_E_INVALID_ARG);
    EXPECT(muon_linear_workspace_bytes(&d, 0, AT(1), AT(2), NULL) == MUON_E_INVALID_ARG);
    EXPECT(muon_linear_workspace_bytes(&d, 3, AT(1), AT(2), &n) == MUON_E_INVALID_ARG);
    EXPECT(muon_linear_workspace_bytes(&d, -1, AT(1), AT(2), &n) == MUON_E_INVALID_ARG);
    EXPECT(muon_op_last_error()[0] != 0);
    for (int k = 0; k < 3; ++k) {
        muon_linear b = d;
        if (k == 0) b.tokens = -1;
        if (k == 1) b.in_features = 0;
        if (k == 2) b.out_features = INT64_MAX;
        EXPECT(muon_linear_workspace_bytes(&b, 0, AT(1), AT(2), &n) == MUON_E_SHAPE);
        EXPECT(muon_linear_forward(&b, AT(1), AT(2), NULL, AT(3), NULL, 0, NULL) == MUON_E_SHAPE);
        EXPECT(muon_linear_grad_input(&b, AT(1), AT(2), NULL, AT(3), NULL, 0, NULL) == MUON_E_SHAPE);
        EXPECT(muon_linear_grad_weight(&b, AT(1), AT(2), AT(3), NULL, 0, NULL, 0, NULL) == MUON_E_SHAPE);
    }
    {
        muon_linear b = d;
        b.tokens = (int64_t)1 << 24;
        EXPECT(muon_linear_workspace_bytes(&b, 0, AT(1), AT(2), &n) == MUON_E_SHAPE);
        b = d;
        b.dtype = MUON_TYPE_FP32;
        EXPECT(muon_linear_workspace_bytes(&b, 0, AT(1), AT(2), &n) == MUON_E_INVALID_ARG);
        b = d;
        b.weight_layout = 2;
        EXPECT(muon_linear_workspace_bytes(&b, 0, AT(1), AT(2), &n) == MUON_E_INVALID_ARG);
        b = d;
        b.ld_x = 95;
        EXPECT(muon_linear_workspace_bytes(&b, 0, AT(1), AT(2), &n) == MUON_E_LAYOUT);
        b = d;
        b.ld_w = 127;
        EXPECT(muon_linear_workspace_bytes(&b, 0, AT(1), AT(2), &n) == MUON_E_LAYOUT);
        b.weight_layout = MUON_WEIGHT_OUT_IN; /* rows of 96 then */
        EXPECT(muon_linear_workspace_bytes(&b, 0, AT(1), AT(2), &n) == MUON_OK);
        b = d;
        b.ld_y = -5;
        EXPECT(muon_linear_workspace_bytes(&b, 0, AT(1), AT(2), &n) == MUON_E_LAYOUT);
        b.ld_y = ((int64_t)1 << 21) + 8;
        EXPECT(muon_linear_workspace_bytes(&b, 0, AT(1), AT(2), &n) == MUON_E_LAYOUT);
    }

    /* the epilogue */
    e.activation = 6;
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), &e, AT(3), NULL, 0, NULL) == MUON_E_INVALID_ARG);
    e.activation = -1;
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), &e, AT(3), NULL, 0, NULL) == MUON_E_INVALID_ARG);
    memset(&e, 0, sizeof(e));
    e.reserved = 1;
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), &e, AT(3), NULL, 0, NULL) == MUON_E_INVALID_ARG);
    memset(&e, 0, sizeof(e));
    e.bias = AT(4);
    EXPECT(muon_linear_grad_input(&d, AT(1), AT(2), &e, AT(3), NULL, 0, NULL) == MUON_E_INVALID_ARG);
    memset(&e, 0, sizeof(e));
    e.activation = MUON_ACT_GELU; /* without its z */
    EXPECT(muon_linear_grad_input(&d, AT(1), AT(2), &e, AT(3), NULL, 0, NULL) == MUON_E_INVALID_ARG);
    memset(&e, 0, sizeof(e));
    e.add = AT(4);
    e.ld_add = 127;
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), &e, AT(3), NULL, 0, NULL) == MUON_E_LAYOUT);

    /* null, misaligned and overlapping tensors; enough workspace throughout */
    char* const ws = AT(100);
    const size_t wsn = (size_t)1 << 31;
    EXPECT(muon_linear_forward(&d, NULL, AT(2), NULL, AT(3), ws, wsn, NULL) == MUON_E_INVALID_ARG);
    EXPECT(muon_linear_forward(&d, AT(1), NULL, NULL, AT(3), ws, wsn, NULL) == MUON_E_INVALID_ARG);
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), NULL, NULL, ws, wsn, NULL) == MUON_E_INVALID_ARG);
    EXPECT(muon_linear_forward(&d, (char*)AT(1) + 1, AT(2), NULL, AT(3), ws, wsn, NULL) == MUON_E_LAYOUT);
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), NULL, AT(1), ws, wsn, NULL) == MUON_E_INVALID_ARG);
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), NULL, (char*)AT(2) + 96 * 128 * 2 - 2, ws, wsn, NULL) ==
           MUON_E_INVALID_ARG);
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), NULL, (char*)AT(2) + 96 * 128 * 2, ws, wsn, NULL) == reached);
    memset(&e, 0, sizeof(e));
    e.add = AT(3); /* the residual replaced by the sum */
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), &e, AT(3), ws, wsn, NULL) == reached);
    e.add = (char*)AT(3) + 2;
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), &e, AT(3), ws, wsn, NULL) == MUON_E_INVALID_ARG);
    e.add = AT(3);
    e.ld_add = 136; /* the same address, another stride */
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), &e, AT(3), ws, wsn, NULL) == MUON_E_INVALID_ARG);
    memset(&e, 0, sizeof(e));
    e.z = AT(3);
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), &e, AT(3), ws, wsn, NULL) == MUON_E_INVALID_ARG);
    e.z = AT(1);
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), &e, AT(3), ws, wsn, NULL) == MUON_E_INVALID_ARG);
    {
        /* column ranges of one buffer of rows of 512: side by side they are apart */
        muon_linear b = d;
        b.ld_x = b.ld_y = 512;
        char* const buf = AT(8);
        EXPECT(muon_linear_forward(&b, buf, AT(2), NULL, buf + 96 * 2, ws, wsn, NULL) == reached);
        EXPECT(muon_linear_forward(&b, buf + 128 * 2, AT(2), NULL, buf, ws, wsn, NULL) == reached);
        EXPECT(muon_linear_forward(&b, buf, AT(2), NULL, buf + 95 * 2, ws, wsn, NULL) == MUON_E_INVALID_ARG);
        EXPECT(muon_linear_forward(&b, buf + 127 * 2, AT(2), NULL, buf, ws, wsn, NULL) == MUON_E_INVALID_ARG);
        /* past the row's end the range goes on in the next row */
        EXPECT(muon_linear_forward(&b, buf, AT(2), NULL, buf + 400 * 2, ws, wsn, NULL) == MUON_E_INVALID_ARG);
        EXPECT(muon_linear_forward(&b, buf, AT(2), NULL, buf + 384 * 2, ws, wsn, NULL) == reached);
        EXPECT(muon_linear_forward(&b, buf + 512 * 2 * 3, AT(2), NULL, buf + 96 * 2, ws, wsn, NULL) == reached);
        b.ld_y = 520; /* another pitch: refused */
        EXPECT(muon_linear_forward(&b, buf, AT(2), NULL, buf + 96 * 2, ws, wsn, NULL) == MUON_E_INVALID_ARG);
    }
    EXPECT(muon_linear_grad_weight(&d, NULL, AT(2), AT(3), NULL, 0, ws, wsn, NULL) == MUON_E_INVALID_ARG);
    EXPECT(muon_linear_grad_weight(&d, AT(1), AT(2), NULL, NULL, 0, ws, wsn, NULL) == MUON_E_INVALID_ARG);
    EXPECT(muon_linear_grad_weight(&d, AT(1), AT(2), (float*)((char*)AT(3) + 2), NULL, 0, ws, wsn, NULL) ==
           MUON_E_LAYOUT);
    EXPECT(muon_linear_grad_weight(&d, AT(1), AT(2), AT(3), AT(3), 0, ws, wsn, NULL) == MUON_E_INVALID_ARG);
    EXPECT(muon_linear_grad_weight(&d, AT(1), AT(2), AT(3), AT(4), 1, ws, wsn, NULL) == reached);

    /* workspaces: rows shorter than a chunk need a packed copy */
    d = lin(24, 7, 128);
    EXPECT(muon_linear_workspace_bytes(&d, MUON_LINEAR_FORWARD, AT(1), AT(2), &n) == MUON_OK && n >= 24 * 8 * 2);
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), NULL, AT(3), NULL, 0, NULL) == MUON_E_WORKSPACE);
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), NULL, AT(3), ws, n - 1, NULL) == MUON_E_WORKSPACE);
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), NULL, AT(3), ws + 128, n, NULL) == MUON_E_WORKSPACE);
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), NULL, ws, ws, n, NULL) == MUON_E_INVALID_ARG);
    EXPECT(muon_linear_forward(&d, ws, AT(2), NULL, AT(3), ws, n, NULL) == MUON_E_INVALID_ARG);
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), NULL, AT(3), ws, n, NULL) == reached);
    /* aligned rows need none, and NULL is then accepted */
    d = lin(8, 96, 128);
    EXPECT(muon_linear_workspace_bytes(&d, MUON_LINEAR_FORWARD, AT(1), AT(2), &n) == MUON_OK && n == 0);
    EXPECT(muon_linear_forward(&d, AT(1), AT(2), NULL, AT(3), NULL, 0, NULL) == reached);
    EXPECT(muon_linear_workspace_bytes(&d, MUON_LINEAR_FORWARD, (char*)AT(1) + 2, AT(2), &n) == MUON_OK && n == 0);
    d = lin(16384, 1600, 1600);
    EXPECT(muon_linear_workspace_bytes(&d, MUON_LINEAR_FORWARD, (char*)AT(1) + 2, AT(2), &n) == MUON_OK &&
           n >= (size_t)16384 * 1600 * 2);

    /* no tokens: nothing to do, whatever the pointers; a weight gradient still is */
    d = lin(0, 96, 128);
    EXPECT(muon_linear_forward(&d, NULL, NULL, NULL, NULL, NULL, 0, NULL) == MUON_OK);
    EXPECT(muon_linear_grad_input(&d, NULL, NULL, NULL, NULL, NULL, 0, NULL) == MUON_OK);
    EXPECT(muon_linear_workspace_bytes(&d, MUON_LINEAR_GRAD_WEIGHT, NULL, NULL, &n) == MUON_OK);
    EXPECT(muon_linear_grad_weight(&d, NULL, NULL, AT(3), NULL, 0, ws, wsn, NULL) == reached);

    /* sizes: planning holds from one element to the limits */
    const int64_t sizes[] = {1, 7, 8, 33, 128, 257, 1600, 6400, 50304, (int64_t)1 << 21};
    const int64_t tokens[] = {0, 1, 17, 32, 33, 1000, 16384, 131072, ((int64_t)1 << 24) - 1};
    for (size_t a = 0; a < sizeof(sizes) / 8; ++a)
        for (size_t b = 0; b < sizeof(sizes) / 8; ++b)
            for (size_t t = 0; t < sizeof(tokens) / 8; ++t)
                for (int op = 0; op < 3; ++op)
                    for (int lay = 0; lay < 2; ++lay) {
                        d = lin(tokens[t], sizes[a], sizes[b]);
                        d.weight_layout = lay;
                        const muon_status s = muon_linear_workspace_bytes(&d, op, AT(1), AT(2), &n);
                        EXPECT(s == MUON_OK || s == MUON_E_SHAPE);
                        if (tokens[t] <= 131072 && sizes[a] <= 6400 && sizes[b] <= 6400) EXPECT(s == MUON_OK);
                        /* the workspace stays within the operands' copies and the pieces of at most 1024 tiles */
                        if (s == MUON_OK && sizes[b] % 8 == 0 && sizes[a] % 8 == 0)
                            EXPECT(n <= (size_t)1024 * (256 * 128 + 256) * 4 + 1024);
                    }

    /* layer norm */
    muon_layernorm m = norm(5, 100, MUON_TYPE_BF16);
    EXPECT(muon_layernorm_workspace_bytes(NULL, &n) == MUON_E_INVALID_ARG);
    EXPECT(muon_layernorm_workspace_bytes(&m, NULL) == MUON_E_INVALID_ARG);
    EXPECT(muon_layernorm_workspace_bytes(&m, &n) == MUON_OK && n > 0);
    for (int k = 0; k < 8; ++k) {
        muon_layernorm b = m;
        muon_status want = MUON_E_SHAPE;
        if (k == 0) b.rows = -1;
        if (k == 1) b.rows = (int64_t)1 << 24;
        if (k == 2) b.cols = 0;
        if (k == 3) b.cols = ((int64_t)1 << 21) + 1;
        if (k == 4) b.dtype = 3, want = MUON_E_INVALID_ARG;
        if (k == 5) b.eps = NAN, want = MUON_E_INVALID_ARG;
        if (k == 6) b.eps = -1e-5f, want = MUON_E_INVALID_ARG;
        if (k == 7) b.ld_x = 99, want = MUON_E_LAYOUT;
        EXPECT(muon_layernorm_workspace_bytes(&b, &n) == want);
        EXPECT(muon_layernorm_forward(&b, AT(1), NULL, NULL, AT(2), AT(3), AT(4), NULL) == want);
        EXPECT(muon_layernorm_backward(&b, AT(1), AT(2), NULL, AT(3), AT(4), NULL, AT(5), NULL, NULL, 0, NULL, 0,
                                       NULL) == want);
    }
    EXPECT(muon_layernorm_forward(&m, AT(1), NULL, NULL, AT(2), AT(3), AT(4), NULL) == reached);
    EXPECT(muon_layernorm_forward(&m, AT(1), NULL, NULL, AT(2), NULL, AT(4), NULL) == MUON_E_INVALID_ARG);
    EXPECT(muon_layernorm_forward(&m, AT(1), NULL, NULL, AT(1), AT(3), AT(4), NULL) == MUON_E_INVALID_ARG);
    EXPECT(muon_layernorm_forward(&m, AT(1), NULL, NULL, AT(2), AT(3), AT(3), NULL) == MUON_E_INVALID_ARG);
    EXPECT(muon_layernorm_forward(&m, AT(1), (float*)((char*)AT(6) + 1), NULL, AT(2), AT(3), AT(4), NULL) ==
           MUON_E_LAYOUT);
    EXPECT(muon_layernorm_backward(&m, AT(1), AT(2), NULL, AT(3), AT(4), NULL, AT(5), NULL, NULL, 0, NULL, 0, NULL) ==
           reached);
    EXPECT(muon_layernorm_backward(&m, AT(1), AT(2), NULL, AT(3), AT(4), AT(5), AT(5), NULL, NULL, 0, NULL, 0, NULL) ==
           reached);
    EXPECT(muon_layernorm_backward(&m, AT(1), AT(2), NULL, AT(3), AT(4), NULL, AT(1), NULL, NULL, 0, NULL, 0, NULL) ==
           MUON_E_INVALID_ARG);
    EXPECT(muon_layernorm_backward(&m, AT(1), AT(2), NULL, AT(3), AT(4), NULL, AT(5), AT(6), NULL, 0, NULL, 0, NULL) ==
           MUON_E_WORKSPACE);
    EXPECT(muon_layernorm_backward(&m, AT(1), AT(2), NULL, AT(3), AT(4), NULL, AT(5), AT(6), AT(6), 0, ws, wsn,
                                   NULL) == MUON_E_INVALID_ARG);
    m.rows = 0;
    EXPECT(muon_layernorm_forward(&m, NULL, NULL, NULL, NULL, NULL, NULL, NULL) == MUON_OK);
    EXPECT(muon_layernorm_backward(&m, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, 0, NULL, 0, NULL) ==
           MUON_OK);
    EXPECT(muon_layernorm_backward(&m, NULL, NULL, NULL, NULL, NULL, NULL, NULL, AT(6), AT(7), 1, ws, wsn, NULL) ==
           MUON_OK);
    EXPECT(muon_layernorm_backward(&m, NULL, NULL, NULL, NULL, NULL, NULL, NULL, AT(6), AT(7), 0, ws, wsn, NULL) ==
           reached);

    if (fails) return 1;
    printf("all expectations hold\n");
    return 0;
}
