/*
 * The step operators from plain C, through include/zpq.h and the HIP
 * runtime's C API only: a lookup, its gradient, the gradient's norm and one
 * AdamW step with 32- and 8-bit states, against loops in double.  Test
 * infrastructure.  Prints "c_step_check: ok" and exits 0, or names the first
 * failing check and exits 1.
 */
#include <hip/hip_runtime_api.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "zpq.h"

enum { ROWS = 37, DIM = 50, TOKENS = 700, N = ROWS * DIM, BLOCKS = (N + 255) / 256 };

static void fail(const char* what, long at, double got, double want) {
    printf("c_step_check: %s[%ld] is %.9g, not %.9g\n", what, at, got, want);
    exit(1);
}
static void hip_ok(hipError_t e, const char* what) {
    if (e != hipSuccess) {
        printf("c_step_check: %s: %s\n", what, hipGetErrorString(e));
        exit(1);
    }
}
static void zpq_ok(zpq_status s, const char* what) {
    if (s != ZPQ_OK) {
        printf("c_step_check: %s returned %d (%s)\n", what, (int)s, zpq_status_str(s));
        exit(1);
    }
}
static void* device(const void* host, size_t bytes) {
    void* p = NULL;
    hip_ok(hipMalloc(&p, bytes), "hipMalloc");
    if (host) hip_ok(hipMemcpy(p, host, bytes, hipMemcpyHostToDevice), "copy in");
    return p;
}
static void fetch(void* host, const void* dev, size_t bytes, hipStream_t st) {
    hip_ok(hipStreamSynchronize(st), "synchronize");
    hip_ok(hipMemcpy(host, dev, bytes, hipMemcpyDeviceToHost), "copy out");
}
/* small integers: sums and products below are exact */
static uint32_t state = 12345;
static float small(int most) {
    state = state * 1664525u + 1013904223u;
    return (float)((int)(state >> 16) % (2 * most + 1) - most);
}

int main(void) {
    static float table[N], dy[TOKENS * DIM], y[TOKENS * DIM], grad[N], p[N], m[N], v[N];
    static int32_t ids[TOKENS];
    static double want[N];
    hipStream_t st;
    hip_ok(hipStreamCreate(&st), "hipStreamCreate");
    for (int i = 0; i < N; ++i) table[i] = small(100);
    for (int i = 0; i < TOKENS * DIM; ++i) dy[i] = small(20);
    for (int t = 0; t < TOKENS; ++t) ids[t] = (int32_t)(fabsf(small(ROWS + 1))) - 1;   /* -1 and ROWS: outside */

    /* lookup */
    void *d_table = device(table, sizeof table), *d_ids = device(ids, sizeof ids), *d_y = device(NULL, sizeof y);
    zpq_ok(zpq_embedding(d_table, ZPQ_F32, ROWS, DIM, DIM, d_ids, 4, TOKENS, 0, 2.0f, d_y, ZPQ_F32, DIM, st),
           "zpq_embedding");
    fetch(y, d_y, sizeof y, st);
    for (int t = 0; t < TOKENS; ++t)
        for (int c = 0; c < DIM; ++c) {
            const int there = ids[t] >= 0 && ids[t] < ROWS;
            const double w = there ? 2.0 * table[ids[t] * DIM + c] : 0.0;
            if (y[t * DIM + c] != w) fail("lookup", t * DIM + c, y[t * DIM + c], w);
        }

    /* gradient */
    int64_t bytes = 0;
    zpq_ok(zpq_embedding_grad_bytes(TOKENS, ROWS, DIM, &bytes), "zpq_embedding_grad_bytes");
    void *d_dy = device(dy, sizeof dy), *d_grad = device(NULL, sizeof grad), *work = device(NULL, (size_t)bytes);
    zpq_ok(zpq_embedding_grad(d_dy, ZPQ_F32, DIM, d_ids, 4, TOKENS, 0, -1, ROWS, DIM, 0.5f, d_grad, ZPQ_F32, DIM, 0,
                              work, bytes, st), "zpq_embedding_grad");
    for (int t = 0; t < TOKENS; ++t)
        if (ids[t] >= 0 && ids[t] < ROWS)
            for (int c = 0; c < DIM; ++c) want[ids[t] * DIM + c] += 0.5 * dy[t * DIM + c];
    fetch(grad, d_grad, sizeof grad, st);
    double square = 0.0;
    for (int i = 0; i < N; ++i) {
        if (grad[i] != want[i]) fail("gradient", i, grad[i], want[i]);
        square += want[i] * want[i];
    }

    /* norm: sums of squares of halves below 2^53, exact */
    const void* ptr = d_grad;
    const int64_t size = N;
    zpq_list list;
    void* list_table = device(NULL, (size_t)ZPQ_LIST_BYTES(1));
    double* d_sum = (double*)device(NULL, 8);
    double sum = 0.0;
    zpq_ok(zpq_list_make(&ptr, &size, 1, ZPQ_F32, list_table, ZPQ_LIST_BYTES(1), &list, st), "zpq_list_make");
    for (int again = 0; again < 2; ++again) {
        zpq_ok(zpq_grad_sumsq(&list, d_sum, again, st), "zpq_grad_sumsq");
        fetch(&sum, d_sum, 8, st);
        if (sum != (again + 1) * square) fail("norm", again, sum, (again + 1) * square);
    }
    zpq_ok(zpq_grad_sumsq(&list, d_sum, 0, st), "zpq_grad_sumsq");

    /* AdamW, both state widths, from zero states */
    for (int bits = 32; bits >= 8; bits -= 24) {
        static uint8_t zeros[N * 4];
        zpq_adamw_tensor t = {device(table, sizeof table), d_grad, device(zeros, N * 4), device(zeros, N * 4),
                              bits == 8 ? (uint8_t*)device(zeros, BLOCKS) : NULL,
                              bits == 8 ? (uint8_t*)device(zeros, BLOCKS) : NULL, NULL, N, 0.1};
        zpq_adamw_plan plan;
        void* plan_table = device(NULL, (size_t)ZPQ_PLAN_BYTES(1));
        const zpq_adamw_hyper h = {1e-2, 0.9, 0.99, 1e-8, 1.0, 1.0, 1, 7};
        zpq_ok(zpq_adamw_plan_make(&t, 1, ZPQ_F32, ZPQ_F32, -1, bits, plan_table, ZPQ_PLAN_BYTES(1), &plan, st),
               "zpq_adamw_plan_make");
        zpq_ok(zpq_adamw_step(&plan, &h, d_sum, st), "zpq_adamw_step");
        fetch(p, t.p, sizeof p, st);
        const double c = 1.0 / (sqrt(square) + 1e-6);
        for (int i = 0; i < N; ++i) {
            const double g = want[i] * c, mm = 0.1 * g, vv = 0.01 * g * g;
            const double w = table[i] * (1 - 1e-2 * 0.1) - 1e-2 * (mm / 0.1) / (sqrt(vv / 0.01) + 1e-8);
            /* about 30 roundings of the step's 1e-2, 4 of the weight */
            if (fabs(p[i] - w) > 6e-8 * (30 * 1e-2 + 4 * fabs(w))) fail("step", i, p[i], w);
        }
        if (bits == 8) {
            void *fm = device(NULL, sizeof m), *fv = device(NULL, sizeof v);
            zpq_ok(zpq_state8_unpack((uint8_t*)t.m, t.m_exp, N, 1, fm, ZPQ_F32, st), "zpq_state8_unpack");
            zpq_ok(zpq_state8_unpack((uint8_t*)t.v, t.v_exp, N, 2, fv, ZPQ_F32, st), "zpq_state8_unpack");
            fetch(m, fm, sizeof m, st);
            fetch(v, fv, sizeof v, st);
            for (int i = 0; i < N; ++i) {      /* within a step of 3 fraction bits, or the smallest one */
                const double g = want[i] * c;
                if (fabs(m[i] - 0.1 * g) > 0.0125 * fabs(g) + 1e-7) fail("8-bit m", i, m[i], 0.1 * g);
                if (fabs(v[i] - 0.01 * g * g) > 0.00125 * g * g + 1e-12) fail("8-bit v", i, v[i], 0.01 * g * g);
            }
        } else {
            fetch(m, t.m, sizeof m, st);
            for (int i = 0; i < N; ++i)
                if (fabs(m[i] - 0.1 * want[i] * c) > 6e-7 * fabs(0.1 * want[i] * c)) fail("m", i, m[i], 0.1 * want[i] * c);
        }
    }
    printf("c_step_check: ok\n");
    return 0;
}
