// decode_scoremod.cu -- paged decode with modified scores: s = cap tanh(scale q.k / cap) - slope (ctx - 1 -
// j) over the cached tokens key_begin <= j < ctx.  Pages before key_begin are not read.
#include "decode_rows.cuh"

namespace attn {
namespace {

// Pages per split: 64 (1024 tokens) where that fills the GPU several times over, down to 8 for small
// batches, whose latency is that of one split's pages.
int chunk_pages_for(int B, int H, int Hkv, int max_pages) {
    const int group = H / Hkv;
    const long long rows = (long long)B * Hkv * (group <= 8 ? 1 : (group + 15) / 16);
    int chunk = 64;
    while (chunk > 8 && rows * ((max_pages + chunk - 1) / chunk) < 4 * 152) chunk /= 2;
    return chunk;
}

template <int D>
cudaError_t launch_decode_scoremod_d(const DecodeMoreArgs &a, const RowsParams &p, cudaStream_t stream) {
    CUtensorMap tk, tv;
    if (!encode_rows_maps<D>(a.kv_fp8 != 0, a.k_pages, a.v_pages, a.num_pages * a.Hkv, tk, tv)) return cudaErrorInvalidValue;
    return launch_rows_d<D, true>(p, tk, tv, a.kv_fp8 != 0, false, stream);
}

}  // namespace

size_t decode_scoremod_workspace_bytes(int B, int H, int Hkv, int d, int max_pages, int page_size) {
    if (decode_workspace_bytes(B, H, Hkv, d, max_pages, page_size) == 0) return 0;  // unsupported sizes
    const size_t chunk = (size_t)chunk_pages_for(B, H, Hkv, max_pages);
    const size_t splits = ((size_t)max_pages + chunk - 1) / chunk;
    return (size_t)B * H * splits * (size_t)(d + 4) * sizeof(float);
}

cudaError_t launch_decode_scoremod(const DecodeMoreArgs &a, cudaStream_t stream) {
    RowsParams p{};
    p.q = a.q;
    p.page_table = a.page_table;
    p.ctx_lens = a.ctx_lens;
    p.o = a.o;
    p.lse = a.lse;
    p.ws = static_cast<float *>(a.workspace);
    p.status = a.status;
    p.B = a.B;
    p.H = a.H;
    p.Hkv = a.Hkv;
    p.group = a.H / a.Hkv;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.chunk_pages = chunk_pages_for(a.B, a.H, a.Hkv, a.max_pages);
    p.n_splits = p.ws_splits = (a.max_pages + p.chunk_pages - 1) / p.chunk_pages;
    p.cluster = cluster_splits(a.B, a.H, a.Hkv, a.d, a.max_pages, a.kv_fp8 != 0);
    const float kscale = a.scale * (a.kv_fp8 ? a.k_scale : 1.f);
    p.c = kscale * kRowLog2e;
    p.v_scale = a.v_scale;
    p.cap_in = a.softcap > 0.f ? kscale / a.softcap : 0.f;
    p.cap_out = a.softcap * kRowLog2e;
    p.slopes = a.slopes;
    p.key_begin = a.key_begin;
    switch (a.d) {
        case 32: return launch_decode_scoremod_d<32>(a, p, stream);
        case 64: return launch_decode_scoremod_d<64>(a, p, stream);
        case 80: return launch_decode_scoremod_d<80>(a, p, stream);
        case 96: return launch_decode_scoremod_d<96>(a, p, stream);
        case 128: return launch_decode_scoremod_d<128>(a, p, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace attn
