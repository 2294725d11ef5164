// decode_shared.cu -- paged decode of a batch whose groups of sequences share their first pages.
//
// Where the sequences' repeated reads of the shared pages would be many (shared_plan), they are read once
// per (group, key/value head): the query heads of all the group's sequences are the rows of the prefill
// kernel's 128-row tcgen05 tiles (a form without a causal mask), split along the keys so that the CTAs fill
// the GPU.  Each sequence's own pages go through the rows kernel, which may start as the first kernel's
// CTAs leave, and one merge joins the partial results.  Elsewhere the rows kernel reads the shared pages
// too.  Measured (32 query and 8 key/value heads, d 128): 32 sequences behind one prompt of 8192 tokens
// 28.9 us, of which the shared pages' kernel takes about 18 and the rows kernel 16, overlapping; 128 sequences
// in two groups behind documents of up to 16384 tokens over an e4m3 cache 70.5 us (47 and 31).  Both kernels are
// bound by latency, not bandwidth (15 to 52 % of it): a few key tiles per CTA in the first, a page's chain in the
// second.
#include "decode_rows.cuh"
#include "prefill_kernel.cuh"

namespace attn {
namespace {

constexpr int kSms = 152;

// How a batch is cut.  prefix_splits 0: the shared pages are read once per sequence by the rows kernel, as
// its own ones: groups of one sequence share nothing, groups of more than 128 query heads per key/value head
// do not fit a tile, and while the repeated reads are few they come from L2 and cost less than the first
// kernel's start and the merge of its parts; the more so where clusters merge the rows kernel's splits.  Repeated
// reads by the table's capacity, MB, and us once per group / once per sequence:
//   by clusters   97 15.6 / 12.7, 129 16.0 / 14.4, 140 15.1 / 16.1, 198 27.7 / 22.1, 192 18.4 / 18.8, e4m3 122
//                 23.7 / 21.8, 181 27.6 / 29.1, 239 31.7 / 40.5, 461 26.8 / 48.2
//   by workspace  34 12.4 / 10.8, 59 12.3 / 13.1, 67 15.7 / 15.3, 83 18.6 / 18.3, 91 16.2 / 17.0, 116 16.5 / 18.9,
//                 e4m3 87 21.7 / 19.0, 153 23.6 / 25.5
constexpr double kRepeatedBytesCluster = 180e6, kRepeatedBytes = 80e6;

struct SharedPlan {
    int group, seqs_per_tile, units, prefix_splits, own_splits;
};
SharedPlan shared_plan(int B, int H, int Hkv, int d, int max_pages, int S, bool fp8) {
    SharedPlan pl{};
    pl.group = H / Hkv;
    const double repeated = 2.0 * (B - B / S) * Hkv * max_pages * kPageTokens * d * (fp8 ? 1 : 2);
    const bool clusters = cluster_splits(B, H, Hkv, d, max_pages, fp8) > 0;
    if (pl.group <= 128 && repeated > (clusters ? kRepeatedBytesCluster : kRepeatedBytes)) {
        pl.seqs_per_tile = 128 / pl.group;
        const int qt = d <= 64 ? Cfg<64>::QT : Cfg<128>::QT;
        pl.units = (S + pl.seqs_per_tile * qt - 1) / (pl.seqs_per_tile * qt);
        // splits: whole waves of CTAs; a split costs about three key tiles on top of its share
        const long long ctas = (long long)(B / S) * Hkv * pl.units;
        const int bn = d <= 64 ? Cfg<64>::BN : Cfg<128>::BN, per_sm = d <= 64 ? 3 : 1;
        const int tiles = (max_pages * kPageTokens + bn - 1) / bn;
        const long long slots = (long long)kSms * per_sm;
        long long best = -1;
        for (long long waves = 1; waves <= 4; ++waves) {  // the most splits that fit this many waves
            long long n = waves * slots / ctas;
            if (n < 1) continue;
            n = n > 64 ? 64 : n;
            n = n > tiles ? tiles : n;
            const long long cost = waves * ((tiles + n - 1) / n + 3);
            if (best < 0 || cost < best) {
                best = cost;
                pl.prefix_splits = (int)n;
            }
        }
        if (best < 0) pl.prefix_splits = 1;
    }
    const int rgroups = pl.group <= 8 ? 1 : (pl.group + 15) / 16;
    const long long rows = (long long)B * Hkv * rgroups;
    const long long want = (4LL * kSms + rows - 1) / rows, most = (max_pages + 7) / 8;
    pl.own_splits = (int)(want < most ? want : most);
    return pl;
}

// Query heads [B, H, D] in boxes of 64 columns x `group` heads x `seqs` sequences.
template <int D, int M>
cudaError_t launch_shared_prefix(const DecodeMoreArgs &a, const SharedPlan &pl, const CUtensorMap &bf16_k,
                                 const CUtensorMap &bf16_v, cudaStream_t stream) {
    CUtensorMap tq, tk, tv;
    const int pool = a.num_pages * a.Hkv;
    bool ok = encode_q_heads_map(&tq, a.q, a.B, a.H, D, pl.group, pl.seqs_per_tile);
    if constexpr (kIsE4m3<M>) {
        ok = ok && encode_page_map_u8(&tk, a.k_pages, pool, kPageTokens, D, false) &&
             encode_page_map_u8(&tv, a.v_pages, pool, kPageTokens, D, false);
    } else {  // the page boxes of the rows kernel
        tk = bf16_k;
        tv = bf16_v;
    }
    if (!ok) return cudaErrorInvalidValue;
    cudaError_t e = check_register_split<D, M>();
    if (e != cudaSuccess) return e;
    PrefillSharedParams p{};
    p.status = a.status;
    p.B = a.B;
    p.H = a.H;
    p.Hkv = a.Hkv;
    p.group = pl.group;
    p.Nkv = a.max_pages * kPageTokens + 1;  // every page is a tile's own rows: a ragged end is always cleared
    p.n_units = pl.units;
    p.heads_per_chunk = a.B * a.H;
    p.page_table = a.page_table;
    p.ctx_lens = a.ctx_lens;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.scale_log2 = a.scale * kLog2e * (kIsE4m3<M> ? a.k_scale : 1.f);
    p.o_scale = kIsE4m3<M> ? a.v_scale : 1.f;
    p.shared_pages = a.shared_pages;
    p.S = a.group_size;
    p.seqs_per_tile = pl.seqs_per_tile;
    p.n_splits = pl.prefix_splits;
    p.ws_splits = pl.prefix_splits + pl.own_splits;
    p.ws = static_cast<float *>(a.workspace);
    const size_t smem = sizeof(PrefillSmem<D, M>) + 1024;
    e = ensure_max_dynamic_smem(reinterpret_cast<const void *>(prefill_kernel<D, M>), (int)smem);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((size_t)(a.B / a.group_size) * a.Hkv * pl.units * pl.prefix_splits);
    prefill_kernel<D, M><<<grid, Occ<D, M>::kThreads, smem, stream>>>(tq, tk, tv, tq, p);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_decode_shared_d(const DecodeMoreArgs &a, const SharedPlan &pl, const RowsParams &rows, cudaStream_t stream) {
    CUtensorMap tk, tv;
    if (!encode_rows_maps<D>(a.kv_fp8 != 0, a.k_pages, a.v_pages, a.num_pages * a.Hkv, tk, tv)) return cudaErrorInvalidValue;
    if (pl.prefix_splits > 0) {
        const cudaError_t e = a.kv_fp8 ? launch_shared_prefix<D, kSharedE4m3>(a, pl, tk, tv, stream)
                                       : launch_shared_prefix<D, kSharedBf16>(a, pl, tk, tv, stream);
        if (e != cudaSuccess) return e;
    }
    return launch_rows_d<D, false>(rows, tk, tv, a.kv_fp8 != 0, pl.prefix_splits > 0, stream);
}

}  // namespace

size_t decode_shared_workspace_bytes(int B, int H, int Hkv, int d, int max_pages, int S, int page_size) {
    if (S <= 0 || B % S != 0 || decode_workspace_bytes(B, H, Hkv, d, max_pages, page_size) == 0) return 0;
    // (the larger of the two cache types' plans)
    const SharedPlan a = shared_plan(B, H, Hkv, d, max_pages, S, false), b = shared_plan(B, H, Hkv, d, max_pages, S, true);
    const int parts = a.prefix_splits + a.own_splits, parts8 = b.prefix_splits + b.own_splits;
    return (size_t)B * H * (parts > parts8 ? parts : parts8) * (size_t)(d + 4) * sizeof(float);
}

cudaError_t launch_decode_shared(const DecodeMoreArgs &a, cudaStream_t stream) {
    const SharedPlan pl = shared_plan(a.B, a.H, a.Hkv, a.d, a.max_pages, a.group_size, a.kv_fp8 != 0);
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
    p.group = pl.group;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.n_splits = pl.own_splits;
    p.ws_first = pl.prefix_splits;
    p.ws_splits = pl.prefix_splits + pl.own_splits;
    p.c = a.scale * kRowLog2e * (a.kv_fp8 ? a.k_scale : 1.f);
    p.v_scale = a.v_scale;
    p.shared_pages = a.shared_pages;
    p.S = a.group_size;
    p.own_only = pl.prefix_splits > 0;
    if (!p.own_only) p.cluster = cluster_splits(a.B, a.H, a.Hkv, a.d, a.max_pages, a.kv_fp8 != 0);
    switch (a.d) {
        case 32: return launch_decode_shared_d<32>(a, pl, p, stream);
        case 64: return launch_decode_shared_d<64>(a, pl, p, stream);
        case 80: return launch_decode_shared_d<80>(a, pl, p, stream);
        case 96: return launch_decode_shared_d<96>(a, pl, p, stream);
        case 128: return launch_decode_shared_d<128>(a, pl, p, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace attn
