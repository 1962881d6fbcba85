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
cudaError_t run(const TokenParams &P, cudaStream_t s) {
    if (P.k > 0) return P.rank ? launch<Both<DT>>(P, s) : launch<Top<DT>>(P, s);
    if (P.rank) return launch<Rank<DT>>(P, s);
    return P.entropy ? launch<Ent<DT>>(P, s) : launch<Plain<DT>>(P, s);
}

}  // namespace

cudaError_t prepare_logprobs() {
    for (cudaError_t (*f)() : {prepare<Plain<SV_DT_FP32>>, prepare<Plain<SV_DT_BF16>>, prepare<Ent<SV_DT_FP32>>, prepare<Ent<SV_DT_BF16>>,
                               prepare<Top<SV_DT_FP32>>, prepare<Top<SV_DT_BF16>>, prepare<Rank<SV_DT_FP32>>, prepare<Rank<SV_DT_BF16>>,
                               prepare<Both<SV_DT_FP32>>, prepare<Both<SV_DT_BF16>>}) {
        const cudaError_t e = f();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_token_logprobs(const TokenParams &P, int dtype, cudaStream_t s) {
    return dtype == SV_DT_FP32 ? run<SV_DT_FP32>(P, s) : run<SV_DT_BF16>(P, s);
}

}  // namespace sv
