// sv_distill.cu -- divergence of a draft's rows from its target's top tokens,
// alone and with its gradient.
#include "sv_token.cuh"

namespace sv {

namespace {

template <int DT, bool GRAD>
using List = Kind<DT, true, GRAD, false, false, false>;

}  // namespace

cudaError_t launch_distill(const TokenParams &P, int dtype, TokenRooms &rooms, cudaStream_t s) {
    if (P.grad) return dtype == SV_DT_FP32 ? launch<List<SV_DT_FP32, true>>(P, rooms, s) : launch<List<SV_DT_BF16, true>>(P, rooms, s);
    return dtype == SV_DT_FP32 ? launch<List<SV_DT_FP32, false>>(P, rooms, s) : launch<List<SV_DT_BF16, false>>(P, rooms, s);
}

}  // namespace sv
