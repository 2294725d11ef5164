// prefill_scoremod.cu -- the prefill kernel with modified scores: s = cap tanh(scale q.k / cap) - slope
// |distance| on an interval of visible keys per query.
#include "prefill_kernel.cuh"

namespace attn {

cudaError_t launch_prefill_scoremod(const PrefillArgs &a, cudaStream_t stream) {
    switch (a.d) {
        case 32: return launch_prefill_dm<32, kContigMod>(a, stream);
        case 64: return launch_prefill_dm<64, kContigMod>(a, stream);
        case 80: return launch_prefill_dm<80, kContigMod>(a, stream);
        case 96: return launch_prefill_dm<96, kContigMod>(a, stream);
        case 128: return launch_prefill_dm<128, kContigMod>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace attn
