/* The embedding, layer norm, dropout and the log probabilities with their
 * gradients from plain C, without Python or PyTorch: device memory from
 * cudaMalloc, results copied back.
 *
 * The rows of tokens 2, -1, 2 of a table that is twice the row's number are 4,
 * 0, 4 in every column, and gradients of 1 give its row 2 twice 1.  A row of
 * -1, 1, -1, 1 is its own layer norm.  Dropout of nothing is x, and of all of
 * it zero, plus the residual.  Logits (0, log 3) are probabilities 1/4 and 3/4.
 * Prints "c tokens ok" and exits 0 when all of it holds. */

#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <cuda_runtime.h>

#include "ddp_reducer.h"

static int fail(const char* what) {
    fprintf(stderr, "failed: %s\n", what);
    return 1;
}

static int near(float a, float b) { return fabsf(a - b) <= 1e-5f; }

static float host[64];

static const float* fetch(const float* from, int n) {
    return cudaMemcpy(host, from, n * sizeof(float), cudaMemcpyDeviceToHost) == cudaSuccess ? host : NULL;
}

int main(void) {
    const int32_t tokens[3] = {2, -1, 2};
    float values[24];
    float* d = NULL;
    void* space = NULL;
    const float* h;
    int i;
    if (cudaMalloc((void**)&d, 1024 * sizeof(float)) != cudaSuccess) return fail("malloc");
    cudaMemset(d, 0, 1024 * sizeof(float));
    float *table = d, *rows = d + 32, *grad = d + 64, *grad_table = d + 96, *x = d + 128, *y = d + 160, *stats = d + 192;
    int32_t* index = (int32_t*)(d + 224);
    for (i = 0; i < 24; ++i) values[i] = 2.0f * (i / 8);                 /* three rows of eight */
    cudaMemcpy(table, values, sizeof(values), cudaMemcpyHostToDevice);
    cudaMemcpy(index, tokens, sizeof(tokens), cudaMemcpyHostToDevice);

    ddp_embed_args e;
    memset(&e, 0, sizeof(e));
    e.tokens = 3;
    e.vocab = 3;
    e.dim = e.table_stride = e.row_stride = 8;
    e.scale = 1.0f;
    e.table_dtype = e.dtype = DDP_F32;
    e.index_bits = 16;
    if (ddp_embed(&e, table, index, rows, NULL) != DDP_ERR_INVALID_ARG) return fail("tokens of 16 bits");
    if (ddp_embed_workspace(&e) != DDP_ERR_INVALID_ARG) return fail("a workspace for them");
    e.index_bits = 32;
    if (ddp_embed(&e, table, index, rows, NULL) != DDP_OK) return fail("embed");
    if (!(h = fetch(rows, 24))) return fail("copy");
    for (i = 0; i < 24; ++i)
        if (h[i] != (i / 8 == 1 ? 0.0f : 4.0f)) return fail("rows");
    for (i = 0; i < 24; ++i) values[i] = 1.0f;
    cudaMemcpy(grad, values, sizeof(values), cudaMemcpyHostToDevice);
    const int64_t bytes = ddp_embed_workspace(&e);
    if (bytes < 0 || cudaMalloc(&space, (size_t)bytes + 1) != cudaSuccess) return fail("workspace");
    if (ddp_embed_backward(&e, grad, index, grad_table, 0, space, NULL) != DDP_OK) return fail("embed backward");
    if (ddp_embed_backward(&e, grad, index, grad_table, 1, space, NULL) != DDP_OK) return fail("embed backward, added");
    if (!(h = fetch(grad_table, 24))) return fail("copy");
    for (i = 0; i < 24; ++i)
        if (h[i] != (i / 8 == 2 ? 4.0f : 0.0f)) return fail("the table's gradient");
    cudaFree(space);

    for (i = 0; i < 4; ++i) values[i] = i % 2 ? 1.0f : -1.0f;
    cudaMemcpy(x, values, 4 * sizeof(float), cudaMemcpyHostToDevice);
    ddp_layer_norm_args l;
    memset(&l, 0, sizeof(l));
    l.rows = 1;
    l.dim = l.x_stride = l.out_stride = 4;
    l.dtype = l.param_dtype = DDP_F32;
    if (ddp_layer_norm(&l, x, NULL, NULL, y, stats, NULL) != DDP_OK) return fail("layer norm");
    if (!(h = fetch(y, 34))) return fail("copy");
    if (!near(h[0], -1.0f) || !near(h[3], 1.0f) || h[32] != 0.0f || !near(h[33], 1.0f)) return fail("norm");
    const int64_t more = ddp_layer_norm_workspace(&l);
    if (more < 0 || cudaMalloc(&space, (size_t)more + 1) != cudaSuccess) return fail("workspace");
    if (ddp_layer_norm_backward(&l, y, 4, x, stats, NULL, NULL, NULL, NULL, 0, space, NULL) != DDP_ERR_INVALID_ARG)
        return fail("a gradient of nothing");
    if (ddp_layer_norm_backward(&l, y, 4, x, stats, NULL, rows, grad, grad + 4, 0, space, NULL) != DDP_OK)
        return fail("layer norm backward");
    if (!(h = fetch(rows, 40))) return fail("copy");
    if (!near(h[0], 0.0f) || !near(h[32], 1.0f) || !near(h[36], -1.0f)) return fail("the norm's gradients");
    cudaFree(space);

    ddp_drop_args p;
    memset(&p, 0, sizeof(p));
    p.rows = 1;
    p.cols = p.x_stride = p.residual_stride = p.out_stride = 4;
    p.dtype = DDP_F32;
    p.p = 1.5;
    if (ddp_drop(&p, x, NULL, y, NULL) != DDP_ERR_INVALID_ARG) return fail("more than all");
    p.p = 0.0;
    if (ddp_drop(&p, x, x, y, NULL) != DDP_OK) return fail("drop");
    if (!(h = fetch(y, 4)) || h[0] != -2.0f || h[1] != 2.0f) return fail("nothing dropped");
    p.p = 1.0;
    if (ddp_drop(&p, x, x, y, NULL) != DDP_OK) return fail("drop");
    if (!(h = fetch(y, 4)) || h[0] != -1.0f || h[1] != 1.0f) return fail("all dropped");

    values[0] = 0.0f;
    values[1] = logf(3.0f);
    values[2] = 1.0f;
    cudaMemcpy(x, values, 3 * sizeof(float), cudaMemcpyHostToDevice);
    ddp_logprobs_args a;
    memset(&a, 0, sizeof(a));
    a.rows = 1;
    a.vocab = a.row_stride = 2;
    a.top = 1;
    a.index_bits = 32;
    a.scale = 1.0f;
    a.dtype = DDP_F32;
    const int32_t target = 0;
    cudaMemcpy(index, &target, sizeof(target), cudaMemcpyHostToDevice);
    if (ddp_logprobs(&a, x, index, y, y + 1, stats, index + 1, y + 2, NULL) != DDP_OK) return fail("log probabilities");
    if (!(h = fetch(y, 3))) return fail("copy");
    if (!near(h[0], -logf(4.0f)) || !near(h[1], logf(4.0f) - 0.75f * logf(3.0f)) || !near(h[2], logf(0.75f)))
        return fail("probabilities");
    int32_t best = -1;
    cudaMemcpy(&best, index + 1, sizeof(best), cudaMemcpyDeviceToHost);
    if (best != 1) return fail("the best");
    if (ddp_logprobs_backward(&a, x, index, stats, NULL, NULL, NULL, y, 2, NULL) != DDP_ERR_INVALID_ARG)
        return fail("a gradient from nothing");
    if (ddp_logprobs_backward(&a, x, index, stats, NULL, x + 2, NULL, y, 2, NULL) != DDP_OK)
        return fail("log probabilities backward");
    if (!(h = fetch(y, 2)) || !near(h[0], 0.75f) || !near(h[1], -0.75f)) return fail("the logits' gradient");
    cudaFree(d);
    printf("c tokens ok\n");
    return 0;
}
