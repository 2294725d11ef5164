// backward_scoremod.cu -- the attention backward with modified scores and per-query key intervals.
#include "backward_kernel.cuh"

namespace attn {

namespace {

template <int D>
cudaError_t launch_scoremod_d(const BwdArgs &a, cudaStream_t stream) {
    const bool cap = a.softcap > 0.f && a.scale / a.softcap > 0.f, bias = a.slopes != nullptr;
    if (cap) return bias ? launch_bwd_d<D, kMod + 3>(a, stream) : launch_bwd_d<D, kMod + 1>(a, stream);
    return bias ? launch_bwd_d<D, kMod + 2>(a, stream) : launch_bwd_d<D, kMod>(a, stream);
}

}  // namespace

cudaError_t launch_bwd_scoremod(const BwdArgs &a, cudaStream_t stream) {
    switch (a.d) {
        case 32: return launch_scoremod_d<32>(a, stream);
        case 64: return launch_scoremod_d<64>(a, stream);
        case 80: return launch_scoremod_d<80>(a, stream);
        case 96: return launch_scoremod_d<96>(a, stream);
        case 128: return launch_scoremod_d<128>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

// The row term, then {lo, hi} of each query tile's keys, then the dK/dV sums of the splits.
size_t bwd_scoremod_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nkv, int d, size_t (&offsets)[2]) {
    const size_t dterm = bwd_workspace_bytes(B, Hq, Nq);
    if (dterm == 0 || Hkv <= 0 || Hq % Hkv != 0 || Nkv <= 0 || d <= 0) return 0;
    offsets[0] = dterm;
    offsets[1] = (dterm + (size_t)B * (((size_t)Nq + kT - 1) / kT) * sizeof(int2) + 255) & ~(size_t)255;
    const int causal = dkdv_plan(B, Hkv, Hq / Hkv, Nq, Nkv, true).most, dense = dkdv_plan(B, Hkv, Hq / Hkv, Nq, Nkv, false).most;
    const int splits = causal > dense ? causal : dense;
    return offsets[1] + (splits > 1 ? (size_t)splits * 2 * B * Hkv * Nkv * d * sizeof(float) : 0);
}

}  // namespace attn
