// backward.cu -- the attention backward with plain scores.
#include "backward_kernel.cuh"

namespace attn {

cudaError_t launch_bwd(const BwdArgs &a, cudaStream_t stream) {
    switch (a.d) {
        case 32: return launch_bwd_d<32, kPlain>(a, stream);
        case 64: return launch_bwd_d<64, kPlain>(a, stream);
        case 80: return launch_bwd_d<80, kPlain>(a, stream);
        case 96: return launch_bwd_d<96, kPlain>(a, stream);
        case 128: return launch_bwd_d<128, kPlain>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

size_t bwd_workspace_bytes(int B, int Hq, int Nq) {
    if (B <= 0 || Hq <= 0 || Nq <= 0) return 0;
    const size_t n = (size_t)B * (size_t)Hq * (size_t)Nq * sizeof(float);
    return (n + 255) & ~(size_t)255;
}

}  // namespace attn
