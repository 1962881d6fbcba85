// sv_logprobs_grad.cu -- the gradient of token log-probabilities and entropies.
#include "sv_token.cuh"

namespace sv {

namespace {

template <int DT, bool ENT>
using Grad = Kind<DT, false, true, ENT, false, false>;

}  // namespace

cudaError_t prepare_logprobs_grad() {
    cudaError_t e = prepare<Grad<SV_DT_FP32, false>>();
    if (e == cudaSuccess) e = prepare<Grad<SV_DT_BF16, false>>();
    if (e == cudaSuccess) e = prepare<Grad<SV_DT_FP32, true>>();
    if (e == cudaSuccess) e = prepare<Grad<SV_DT_BF16, true>>();
    return e;
}

cudaError_t launch_token_logprobs_grad(const TokenParams &P, int dtype, cudaStream_t s) {
    if (P.g_entropy || P.entropy)
        return dtype == SV_DT_FP32 ? launch<Grad<SV_DT_FP32, true>>(P, s) : launch<Grad<SV_DT_BF16, true>>(P, s);
    return dtype == SV_DT_FP32 ? launch<Grad<SV_DT_FP32, false>>(P, s) : launch<Grad<SV_DT_BF16, false>>(P, s);
}

}  // namespace sv
