// prefill.cu -- the prefill kernel over contiguous K/V, bf16 pages and e4m3 pages.
#include "prefill_kernel.cuh"

namespace attn {
namespace {

template <int D>
cudaError_t launch_prefill_d(const PrefillArgs &a, cudaStream_t stream) {
    if (!a.paged) return launch_prefill_dm<D, kContig>(a, stream);
    if (a.kv_fp8) return launch_prefill_dm<D, kPagedE4m3>(a, stream);
    return launch_prefill_dm<D, kPagedBf16>(a, stream);
}

}  // namespace

cudaError_t launch_prefill(const PrefillArgs &a, cudaStream_t stream) {
    switch (a.d) {
        case 32: return launch_prefill_d<32>(a, stream);
        case 64: return launch_prefill_d<64>(a, stream);
        case 80: return launch_prefill_d<80>(a, stream);
        case 96: return launch_prefill_d<96>(a, stream);
        case 128: return launch_prefill_d<128>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace attn
