// sv_token.h -- types shared by the host library and the kernels of the token
// log-probability and distillation calls (not part of the public C ABI).
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "specverify.h"

namespace sv {

constexpr int kMaxAlternatives = SPECVERIFY_MAX_ALTERNATIVES;
constexpr int kMaxList = SPECVERIFY_MAX_LIST;

// A call over rows of logits. Row r is at logits + r * stride_bytes.
struct TokenParams {
    const char *logits;
    int64_t stride_bytes, rows;
    int32_t V;
    float c, c_lo;       // log2(e) / T; c_lo is 0, or (lists) more than 0
    float lag, near, far;  // 8 / c, 2^24 / c, about -2^25 / c (a bf16 number): see sv_token_math.cuh
    float inv_hi, inv_lo;  // 1 / T
    int32_t *status;
    uint64_t wait_ns;    // bound of a wait inside the kernel
    // entries: rows with a token (log-probabilities) or with a list (distillation)
    int64_t entries;
    int32_t B, M;        // sequences, and entries of one (log-probabilities)
    const int32_t *tokens;
    const int64_t *row_off;
    const int32_t *path;
    int32_t k;
    float *logprob, *entropy, *lse;
    int32_t *rank;
    float *top_logprob;
    int32_t *top_idx;
    // gradients
    char *grad;
    int64_t grad_stride_bytes;
    const float *g_logprob, *g_entropy;
    // distillation
    int32_t K;
    const int32_t *ids;
    const char *target;
    int32_t target_bf16, form, divergence;
    float beta;
    const float *weight;
    float *loss;
};

// What a handle knows of one of the kernels on its device, from its first call that takes it on: the clusters of 2^i CTAs that
// fit the GPU at once. (Calls on one handle may run beside one another: two that find nothing known write the same.)
struct TokenRoom {
    std::atomic<bool> known{false};
    std::atomic<int> clusters[5] = {};
};

struct TokenRooms {
    TokenRoom of[18];
};

cudaError_t launch_token_logprobs(const TokenParams &p, int dtype, TokenRooms &rooms, cudaStream_t s);
cudaError_t launch_token_logprobs_grad(const TokenParams &p, int dtype, TokenRooms &rooms, cudaStream_t s);
cudaError_t launch_distill(const TokenParams &p, int dtype, TokenRooms &rooms, cudaStream_t s);  // p.grad may be NULL

}  // namespace sv
