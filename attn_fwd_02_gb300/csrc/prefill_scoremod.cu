// prefill_scoremod.cu -- the prefill kernel with modified scores: s = cap tanh(scale q.k / cap) - slope
// |distance| on an interval of visible keys per query.
#include "prefill_kernel.cuh"

namespace attn {
namespace {

template <int D>
cudaError_t launch_scoremod_d(const PrefillArgs &a, cudaStream_t stream) {
    const bool cap = a.softcap > 0.f && a.scale / a.softcap > 0.f, bias = a.slopes != nullptr;
    if (cap) return bias ? launch_prefill_dm<D, kMod + 3>(a, stream) : launch_prefill_dm<D, kMod + 1>(a, stream);
    return bias ? launch_prefill_dm<D, kMod + 2>(a, stream) : launch_prefill_dm<D, kMod>(a, stream);
}

}  // namespace

cudaError_t launch_prefill_scoremod(const PrefillArgs &a, cudaStream_t stream) {
    switch (a.d) {
        case 32: return launch_scoremod_d<32>(a, stream);
        case 64: return launch_scoremod_d<64>(a, stream);
        case 80: return launch_scoremod_d<80>(a, stream);
        case 96: return launch_scoremod_d<96>(a, stream);
        case 128: return launch_scoremod_d<128>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace attn
