// launch.h -- internal interface between the C ABI (abi.cu) and the kernel
// translation units.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace attn {

struct PrefillArgs {
    const void *q, *k, *v;
    void *o;
    float *lse;              // may be null
    const int32_t *kv_lens;  // may be null
    int *status;             // device status word [2]
    int B, H, Nq, Nkv, d, causal;
    float scale;
    int Hkv;                 // key/value heads (H for multi-head; H % Hkv == 0)
    // paged mode: k, v are [num_pages, Hkv, 16, d] pages through page_table [B, max_pages];
    // ctx_lens[b] cached tokens, the queries being the last Nq of them; Nkv = capacity
    int paged = 0;
    const int32_t *page_table = nullptr, *ctx_lens = nullptr;
    int max_pages = 0, num_pages = 0;
    // paged mode over an e4m3 cache: k, v hold codes; value = e4m3(code) * k_scale / v_scale
    int kv_fp8 = 0;
    float k_scale = 1.f, v_scale = 1.f;
    // modified scores (launch_prefill_scoremod): cap (0: none), slopes [H] and intervals [B, Nq] (null: none)
    float softcap = 0.f;
    const float *slopes = nullptr;
    const int32_t *key_begin = nullptr, *key_end = nullptr;
};

struct DecodeArgs {
    const void *q, *k_pages, *v_pages;
    const int32_t *page_table, *ctx_lens;
    void *o;
    float *lse;  // may be null
    void *workspace;
    int *status;
    int B, H, d, page_size, max_pages, num_pages;
    float scale;
    int Hkv;  // key/value heads of the cache (H for multi-head; H % Hkv == 0)
    // e4m3 cache: pages hold FP8 codes, value = e4m3(code) * k_scale (keys) or * v_scale (values)
    int kv_fp8 = 0;
    float k_scale = 1.f, v_scale = 1.f;
};

// Of the further decode calls (apart from DecodeArgs, which is the decode kernels' parameter itself).
struct DecodeMoreArgs : DecodeArgs {
    // launch_decode_shared: groups of group_size sequences share their first shared_pages[b / group_size] pages
    const int32_t *shared_pages = nullptr;
    int group_size = 0;
    // launch_decode_scoremod: cap (0: none), slopes [H], first visible token [B] (null: none)
    float softcap = 0.f;
    const float *slopes = nullptr;
    const int32_t *key_begin = nullptr;
};

struct BwdArgs {
    const void *q, *k, *v, *o, *dout;  // q, o, dout [B,Hq,Nq,d]; k, v [B,Hkv,Nkv,d] (bf16)
    const float *lse;                  // [B,Hq,Nq], natural log, from the forward
    void *dq, *dk, *dv;                // bf16 outputs, shaped like q, k, v
    float *dterm;                      // workspace: the row term D [B,Hq,Nq]
    const int32_t *kv_lens;            // may be null
    int *status;
    int B, Hq, Hkv, Nq, Nkv, d, causal;
    float scale;
    // modified scores (launch_bwd_scoremod), as in PrefillArgs; spans: the rest of the workspace
    float softcap = 0.f;
    const float *slopes = nullptr;
    const int32_t *key_begin = nullptr, *key_end = nullptr;
    int2 *spans = nullptr;
    float *kv_parts = nullptr;
};

// Per-device facts looked up once (host-side caches shared by the launchers): the SM count
// of the current device, and a kernel's dynamic shared-memory opt-in (set once per
// function and device; cudaFuncSetAttribute is not free on every call).
cudaError_t current_sm_count(int *sms);
cudaError_t ensure_max_dynamic_smem(const void *kernel, int bytes);
// Allows clusters of more than 8 CTAs (once per kernel and device).
cudaError_t ensure_large_clusters(const void *kernel);
// Whether the current device can hold a cluster of n CTAs of this kernel (asked once per kernel, device and n).
bool cluster_fits(const void *kernel, int n, int threads, size_t smem);

// TMA descriptor of a bf16 [BH, N, D] tensor viewed as 3-D (innermost first) with boxes of
// 64 x box_rows x 1 and the 128-byte swizzle; rows past N read as zeros.
bool encode_qkv_map(CUtensorMap *m, const void *ptr, int BH, int N, int D, int box_rows = 128);
// [rows, page_rows, D] one-byte (e4m3) page blocks, one box of page_rows x 128 bytes per block,
// with the 128-byte swizzle or none; the bytes of a box past D are read as zeros.
bool encode_page_map_u8(CUtensorMap *m, const void *ptr, int rows, int page_rows, int D, bool swizzle = true);

// Launches a kernel that may start while the one before it on the stream drains (griddepcontrol.wait in
// the kernel orders it after that one's completion).
template <class K, class... A>
cudaError_t launch_dependent(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Query heads of a decode batch, [B, H, D] bf16, in swizzled boxes of 64 columns x heads x seqs rows.
bool encode_q_heads_map(CUtensorMap *m, const void *ptr, int B, int H, int D, int heads, int seqs);

// Encodes the TMA descriptors and launches the prefill kernel.
cudaError_t launch_prefill(const PrefillArgs &a, cudaStream_t stream);
// The same with modified scores and per-query key intervals (contiguous K/V only).
cudaError_t launch_prefill_scoremod(const PrefillArgs &a, cudaStream_t stream);

// Backward: the row term D, then the dK/dV kernel and the dQ kernel.
cudaError_t launch_bwd(const BwdArgs &a, cudaStream_t stream);
size_t bwd_workspace_bytes(int B, int Hq, int Nq);
cudaError_t launch_bwd_scoremod(const BwdArgs &a, cudaStream_t stream);
// Bytes of its workspace; offsets: where the query tiles' intervals and the dK/dV sums start in it.
size_t bwd_scoremod_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nkv, int d, size_t (&offsets)[2]);

// Writes new tokens' K/V into their pages (token t of sequence b goes to position
// start_pos[b] + t).  Positions past the table's capacity are skipped.
cudaError_t launch_kv_append(const void *k_new, const void *v_new, void *k_pages, void *v_pages,
                             const int32_t *page_table, const int32_t *start_pos, int B, int Hkv, int Nnew, int d,
                             int max_pages, int num_pages, cudaStream_t stream);

// FP8 (E4M3) cache conversion: codes = e4m3_rn_satfinite(fp32(x) * inv_scale).
//   kv_quantize_fp8: n contiguous bf16 elements -> n codes (n % 8 == 0).
//   kv_append_fp8: as launch_kv_append, converting each new element on the way into the pages.
cudaError_t launch_kv_quantize_fp8(const void *src, void *dst, size_t n, float inv_scale, cudaStream_t stream);
cudaError_t launch_kv_append_fp8(const void *k_new, const void *v_new, void *k_pages, void *v_pages,
                                 float k_inv_scale, float v_inv_scale, const int32_t *page_table,
                                 const int32_t *start_pos, int B, int Hkv, int Nnew, int d, int max_pages,
                                 int num_pages, cudaStream_t stream);

// Positions with several axes: pair i of a token turns by row positions[axis(i)][b][t] of the table.
constexpr int kMaxAxes = 4, kMaxRope = 128;
struct RopeAxes {
    const int32_t *positions = nullptr;  // null: none
    long long axis_stride = 0, batch_stride = 0;
    int axes = 0;
    uint64_t pair_axis[2] = {0, 0};  // two bits a pair
};

// As the append, with the queries and keys rotated to their positions on the way.
struct RopeAppendArgs {
    const void *q, *k_new, *v_new;                   // q may be null (keys and values only)
    int64_t q_strides[3], k_strides[3], v_strides[3];  // batch, head, token, in elements
    void *q_out, *k_pages, *v_pages;
    const float *cos_sin;  // [max_pos, rope_dim]
    int rope_dim, max_pos, interleaved;
    const int32_t *page_table, *start_pos, *new_lens;  // new_lens may be null
    int B, H, Hkv, Nnew, d, max_pages, num_pages;
    int kv_fp8 = 0;
    float k_scale = 1.f, v_scale = 1.f;
    RopeAxes axes;
};
cudaError_t launch_kv_append_rope(const RopeAppendArgs &a, cudaStream_t stream);
// Into the 4-bit cache (cos_sin may be null: no rotation, and no queries), and its pages as bf16.
cudaError_t launch_kv_append_fp4(const RopeAppendArgs &a, cudaStream_t stream);
cudaError_t launch_kv_unpack_fp4(const void *k_pages, const void *v_pages, float k_scale, float v_scale,
                                 const int32_t *page_ids, int n, void *k_out, void *v_out, int Hkv, int d, int num_pages,
                                 cudaStream_t stream);

// The rotation alone, of queries and keys (k may be null) in strided views; back: by the transposed rotation.
struct RopeArgs {
    const void *q, *k;
    void *q_out, *k_out;
    int64_t q_strides[3], k_strides[3], q_out_strides[3], k_out_strides[3];  // batch, head, token, in elements
    const float *cos_sin;
    int rope_dim, max_pos, interleaved, back;
    int B, H, Hkv, N, d;
    RopeAxes axes;
};
cudaError_t launch_rope_axes(const RopeArgs &a, cudaStream_t stream);

// Page tables and reference counts (see the header): forking, reserving, compacting, and copies of pages.
struct PagesArgs {
    const int32_t *page_table, *ctx_lens, *parents, *new_lens, *ref_counts;
    int32_t *page_table_out, *ctx_lens_out, *ref_counts_out, *reserved, *src, *dst, *count;
    int B, B_out, max_pages, num_pages;
    void *workspace;
};
cudaError_t launch_pages_fork(const PagesArgs &a, cudaStream_t stream);
cudaError_t launch_pages_reserve(const PagesArgs &a, cudaStream_t stream);
size_t pages_reserve_workspace_bytes(int B, int num_pages);
cudaError_t launch_pages_compact(const PagesArgs &a, cudaStream_t stream);
size_t pages_compact_workspace_bytes(int num_pages);
cudaError_t launch_pages_copy(void *const *pools, int n_pools, size_t page_bytes, const int32_t *src, const int32_t *dst,
                              const int32_t *count, int n, int num_pages, cudaStream_t stream);

// Launches the split kernel and the combine kernel.
cudaError_t launch_decode(const DecodeArgs &a, cudaStream_t stream);

// Workspace bytes the decode needs for H query heads over Hkv cache heads (0 if the sizes are
// unsupported).
size_t decode_workspace_bytes(int B, int H, int Hkv, int d, int max_pages, int page_size);

// Decode with modified scores, and decode of a batch whose groups share their first pages.
cudaError_t launch_decode_scoremod(const DecodeMoreArgs &a, cudaStream_t stream);
size_t decode_scoremod_workspace_bytes(int B, int H, int Hkv, int d, int max_pages, int page_size);
cudaError_t launch_decode_fp4(const DecodeMoreArgs &a, cudaStream_t stream);
size_t decode_fp4_workspace_bytes(int B, int H, int Hkv, int d, int max_pages, int page_size);
cudaError_t launch_decode_shared(const DecodeMoreArgs &a, cudaStream_t stream);
size_t decode_shared_workspace_bytes(int B, int H, int Hkv, int d, int max_pages, int S, int page_size);

// Same kernels with the chunk partials in the library's static scratch array
// (no workspace from the caller); see decode.cu.
cudaError_t launch_decode_noalloc(const DecodeArgs &a, cudaStream_t stream);
size_t decode_noalloc_scratch_bytes();

// One block that waits on an mbarrier nobody arrives on (exercises the bounded waits).
cudaError_t launch_selftest_wait(int *status, cudaStream_t stream);

// Tokens per split of the paged decode.
constexpr int kDecodeChunkTokens = 512;

}  // namespace attn
