// sv_logprobs_grad.cu -- the gradient of token log-probabilities and entropies.
#include "sv_token.cuh"

namespace sv {

namespace {

template <int DT, bool ENT>
using Grad = Kind<DT, false, true, ENT, false, false>;

}  // namespace

cudaError_t launch_token_logprobs_grad(const TokenParams &P, int dtype, TokenRooms &rooms, cudaStream_t s) {
    if (P.g_entropy || P.entropy)
        return dtype == SV_DT_FP32 ? launch<Grad<SV_DT_FP32, true>>(P, rooms, s) : launch<Grad<SV_DT_BF16, true>>(P, rooms, s);
    return dtype == SV_DT_FP32 ? launch<Grad<SV_DT_FP32, false>>(P, rooms, s) : launch<Grad<SV_DT_BF16, false>>(P, rooms, s);
}

}  // namespace sv
