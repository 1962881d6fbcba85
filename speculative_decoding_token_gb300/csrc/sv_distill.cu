// sv_distill.cu -- divergence of a draft's rows from its target's top tokens,
// alone and with its gradient.
#include "sv_token.cuh"

namespace sv {

namespace {

template <int DT, bool GRAD>
using List = Kind<DT, true, GRAD, false, false, false>;

}  // namespace

cudaError_t prepare_distill() {
    cudaError_t e = prepare<List<SV_DT_FP32, false>>();
    if (e == cudaSuccess) e = prepare<List<SV_DT_BF16, false>>();
    if (e == cudaSuccess) e = prepare<List<SV_DT_FP32, true>>();
    if (e == cudaSuccess) e = prepare<List<SV_DT_BF16, true>>();
    return e;
}

cudaError_t launch_distill(const TokenParams &P, int dtype, cudaStream_t s) {
    if (P.grad) return dtype == SV_DT_FP32 ? launch<List<SV_DT_FP32, true>>(P, s) : launch<List<SV_DT_BF16, true>>(P, s);
    return dtype == SV_DT_FP32 ? launch<List<SV_DT_FP32, false>>(P, s) : launch<List<SV_DT_BF16, false>>(P, s);
}

}  // namespace sv
