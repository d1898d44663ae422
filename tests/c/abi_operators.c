/* The optimizer step, the gradient norm and the routing from plain C, without
 * Python or PyTorch: device memory from cudaMalloc, results copied back.
 *
 * Gradients (3, 0, 4) in two tensors have norm 5; the first step from zero
 * moments moves each weight by lr against its gradient's sign, and leaves one
 * without a gradient.  Logits (0, 1, 2, 2) choose experts 2 and 3 with weights
 * 1/2 each, whose gradient (1, 0) gives (0, 0, 1/4, -1/4).
 * Prints "c operators ok" and exits 0 when all of it holds. */

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

int main(void) {
    const int64_t numel[3] = {2, 0, 1};
    const float g[3] = {3.0f, 0.0f, -4.0f};
    float host[16];
    float* d = NULL;                       /* 0: gradients, 4: weights, 8: m, 12: v, 16: norm; 64 floats for routing after */
    if (cudaMalloc((void**)&d, 128 * sizeof(float)) != cudaSuccess) return fail("malloc");
    cudaMemset(d, 0, 128 * sizeof(float));
    cudaMemcpy(d, g, sizeof(g), cudaMemcpyHostToDevice);

    ddp_adamw* opt = NULL;
    if (ddp_adamw_create(numel, 3, DDP_F32, 16, &opt) != DDP_ERR_INVALID_ARG || opt) return fail("create 16");
    if (!strstr(ddp_adamw_last_error(NULL), "state_bits")) return fail("detail");
    if (ddp_adamw_create(numel, 3, DDP_F32, 32, &opt) != DDP_OK) return fail("create");
    const float* grads[3] = {d, NULL, d + 2};
    void* w[3] = {d + 4, NULL, d + 6};
    void* m[3] = {d + 8, NULL, d + 10};
    void* v[3] = {d + 12, NULL, d + 14};
    if (ddp_adamw_bind(opt, grads, w, NULL, m, v, NULL, NULL, NULL) != DDP_OK) return fail(ddp_adamw_last_error(opt));
    float* norm = d + 16;
    if (ddp_adamw_grad_norm(opt, NULL, norm, NULL) != DDP_OK) return fail(ddp_adamw_last_error(opt));
    ddp_adamw_args a;
    memset(&a, 0, sizeof(a));
    a.t = 1;
    a.lr = 0.5;
    a.beta1 = 0.9;
    a.beta2 = 0.999;
    a.eps = 1e-12;
    a.max_norm = 1.0;
    if (ddp_adamw_step(opt, &a, NULL) != DDP_ERR_INVALID_ARG) return fail("a norm to clip by is missing");
    a.norm = norm;
    if (ddp_adamw_step(opt, &a, NULL) != DDP_OK) return fail(ddp_adamw_last_error(opt));
    if (cudaMemcpy(host, d + 4, 13 * sizeof(float), cudaMemcpyDeviceToHost) != cudaSuccess) return fail("copy");
    if (host[12] != 5.0f) return fail("norm");
    if (!near(host[0], -0.5f) || host[1] != 0.0f || !near(host[2], 0.5f)) return fail("weights");
    if (!near(host[4], 0.1f * 0.6f) || !near(host[6], -0.1f * 0.8f)) return fail("first moments");
    ddp_adamw_destroy(opt);

    const float x[4] = {0.0f, 1.0f, 2.0f, 2.0f}, gw[2] = {1.0f, 0.0f};
    float *logits = d + 64, *weights = d + 72, *grad_w = d + 76, *grad_x = d + 80;
    int32_t *index = (int32_t*)(d + 84), *counts = (int32_t*)(d + 88), got[8];
    cudaMemcpy(logits, x, sizeof(x), cudaMemcpyHostToDevice);
    cudaMemcpy(grad_w, gw, sizeof(gw), cudaMemcpyHostToDevice);
    ddp_route_args r;
    memset(&r, 0, sizeof(r));
    r.tokens = 1;
    r.row_stride = 4;
    r.experts = 4;
    r.k = 2;
    r.score = DDP_SCORE_SOFTMAX;
    r.groups = r.top_groups = 1;
    r.renorm = 1;
    r.scale = 1.0f;
    r.dtype = DDP_F32;
    if (ddp_route(&r, logits, NULL, NULL, index, weights, counts, NULL) != DDP_OK) return fail("route");
    if (ddp_route_backward(&r, logits, index, weights, grad_w, grad_x, 4, NULL) != DDP_OK) return fail("backward");
    if (cudaMemcpy(got, index, 8 * sizeof(int32_t), cudaMemcpyDeviceToHost) != cudaSuccess) return fail("copy");
    if (got[0] != 2 || got[1] != 3) return fail("indices");
    if (got[4] != 0 || got[5] != 0 || got[6] != 1 || got[7] != 1) return fail("counts");
    cudaMemcpy(host, weights, 12 * sizeof(float), cudaMemcpyDeviceToHost);
    if (!near(host[0], 0.5f) || !near(host[1], 0.5f)) return fail("routing weights");
    if (host[8] != 0.0f || host[9] != 0.0f || !near(host[10], 0.25f) || !near(host[11], -0.25f)) return fail("gradient");
    cudaFree(d);
    printf("c operators ok\n");
    return 0;
}
