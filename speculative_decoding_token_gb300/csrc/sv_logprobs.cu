// sv_logprobs.cu -- log-probabilities of given tokens: the kernels without and
// with entropy, top tokens and rank.
#include "sv_token.cuh"

namespace sv {

namespace {

// entropy, top tokens, rank (with either of the last two the entropy comes along)
template <int DT>
using Plain = Kind<DT, false, false, false, false, false>;
template <int DT>
using Ent = Kind<DT, false, false, true, false, false>;
template <int DT>
using Top = Kind<DT, false, false, true, true, false>;
template <int DT>
using Rank = Kind<DT, false, false, true, false, true>;
template <int DT>
using Both = Kind<DT, false, false, true, true, true>;

template <int DT>
cudaError_t run(const TokenParams &P, TokenRooms &rooms, cudaStream_t s) {
    if (P.k > 0) return P.rank ? launch<Both<DT>>(P, rooms, s) : launch<Top<DT>>(P, rooms, s);
    if (P.rank) return launch<Rank<DT>>(P, rooms, s);
    return P.entropy ? launch<Ent<DT>>(P, rooms, s) : launch<Plain<DT>>(P, rooms, s);
}

}  // namespace

cudaError_t launch_token_logprobs(const TokenParams &P, int dtype, TokenRooms &rooms, cudaStream_t s) {
    return dtype == SV_DT_FP32 ? run<SV_DT_FP32>(P, rooms, s) : run<SV_DT_BF16>(P, rooms, s);
}

}  // namespace sv
