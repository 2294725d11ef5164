// backward_scoremod.cu -- the attention backward with modified scores and per-query key intervals.
#include "backward_kernel.cuh"

namespace attn {

cudaError_t launch_bwd_scoremod(const BwdArgs &a, cudaStream_t stream) {
    switch (a.d) {
        case 32: return launch_bwd_d<32, true>(a, stream);
        case 64: return launch_bwd_d<64, true>(a, stream);
        case 80: return launch_bwd_d<80, true>(a, stream);
        case 96: return launch_bwd_d<96, true>(a, stream);
        case 128: return launch_bwd_d<128, true>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

// The row term, then {lo, hi} of each query tile's keys.
size_t bwd_scoremod_workspace_bytes(int B, int Hq, int Nq) {
    const size_t dterm = bwd_workspace_bytes(B, Hq, Nq);
    return dterm == 0 ? 0 : dterm + (size_t)B * (((size_t)Nq + kT - 1) / kT) * sizeof(int2);
}

}  // namespace attn
