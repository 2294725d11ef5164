// abi.cu -- the C ABI declared in include/attn_gb300.h: host-side argument
// checks, the device status word, and dispatch to the kernel launchers.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <mutex>

#include "attn_gb300.h"
#include "launch.h"

#define ATTN_API extern "C" __attribute__((visibility("default")))

namespace {

// Device status word (see sm103_ptx.cuh): [0] flags, [1] first failing site, [2..3] the address
// of this device's host-visible flag.
__device__ __align__(8) int g_status[4];

constexpr int kMaxDevices = 64;
int *g_status_ptr[kMaxDevices];
int g_arch_ok[kMaxDevices];  // 0 unknown, 1 sm_103, -1 other
std::mutex g_mu;

// Host-visible timeout flags, one per device (16 ints apart), in one page of the library's own
// static storage that is page-locked and mapped for the GPUs once per process.  A kernel whose
// bounded wait runs out stores 1 into its device's flag (and fences), so the host can see the
// timeout with a plain load, without synchronising any stream.
alignas(4096) volatile int g_host_flags[kMaxDevices * 16];
int g_host_flags_registered = 0;  // 0 not yet, 1 registered, -1 failed

int *host_flag_of(int dev) { return const_cast<int *>(&g_host_flags[dev * 16]); }

// Per-device set-up, done once per device by the first call on it (with the device current):
// architecture check, the status word's device address, registration of the flag page, and a
// copy of the flag's device-side address into the status word.  The copy is synchronous, so the
// first call on each device should come before any stream capture.
int device_setup_locked(int dev) {
    if (g_arch_ok[dev] == 0) {
        cudaDeviceProp prop;
        if (cudaGetDeviceProperties(&prop, dev) != cudaSuccess) return ATTN_ERR_CUDA;
        g_arch_ok[dev] = (prop.major == 10 && prop.minor == 3) ? 1 : -1;
    }
    if (g_arch_ok[dev] != 1) return ATTN_ERR_UNSUPPORTED;
    if (g_status_ptr[dev]) return ATTN_OK;
    if (g_host_flags_registered == 0) {
        const cudaError_t e = cudaHostRegister(const_cast<int *>(g_host_flags), sizeof(g_host_flags),
                                               cudaHostRegisterMapped | cudaHostRegisterPortable);
        g_host_flags_registered = (e == cudaSuccess) ? 1 : -1;
    }
    if (g_host_flags_registered != 1) return ATTN_ERR_CUDA;
    void *flag_dev = nullptr;
    if (cudaHostGetDevicePointer(&flag_dev, host_flag_of(dev), 0) != cudaSuccess || !flag_dev) return ATTN_ERR_CUDA;
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_status) != cudaSuccess || !p) return ATTN_ERR_CUDA;
    int init[4] = {0, 0, 0, 0};
    static_assert(sizeof(void *) == 2 * sizeof(int), "64-bit device addresses");
    memcpy(&init[2], &flag_dev, sizeof flag_dev);
    if (cudaMemcpy(p, init, sizeof init, cudaMemcpyHostToDevice) != cudaSuccess) return ATTN_ERR_CUDA;
    *host_flag_of(dev) = 0;
    g_status_ptr[dev] = static_cast<int *>(p);
    return ATTN_OK;
}

int current_device(int *dev) {
    if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= kMaxDevices) return ATTN_ERR_CUDA;
    return ATTN_OK;
}

// Set-up for a call that launches work: also refuses (ATTN_ERR_DEVICE_TIMEOUT, nothing
// launched) while a timeout recorded by an earlier call on this device is not yet cleared.
int device_setup(int **status_out) {
    int dev = -1;
    if (current_device(&dev) != ATTN_OK) return ATTN_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        const int st = device_setup_locked(dev);
        if (st != ATTN_OK) return st;
    }
    if (*host_flag_of(dev) != 0) return ATTN_ERR_DEVICE_TIMEOUT;
    *status_out = g_status_ptr[dev];
    return ATTN_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// Head dims of the prefill kernels (forward, paged prefill, KV append): the set the
// Kernel-Inference-Engine README instantiates its attention kernel for.  Decode and the
// backward take 64 and 128.
bool prefill_head_dim(int d) { return d == 32 || d == 64 || d == 80 || d == 96 || d == 128; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int prefill_checks(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H, int Hkv,
                   int Nq, int Nkv, int d, int causal, float scale, const int32_t *kv_lens) {
    if (!q || !k || !v || !o) return ATTN_ERR_INVALID_ARG;
    if (B <= 0 || H <= 0 || Nq <= 0 || Nkv <= 0 || d <= 0) return ATTN_ERR_INVALID_ARG;
    if (Hkv <= 0 || H % Hkv != 0) return ATTN_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !(scale < 3.0e38f)) return ATTN_ERR_INVALID_ARG;  // finite, positive
    if (!prefill_head_dim(d)) return ATTN_ERR_UNSUPPORTED;
    // grid = ceil(Nq/128) * B * H CTAs and 32-bit TMA coordinates
    const uint64_t bh = (uint64_t)B * (uint64_t)H;
    const uint64_t ctas = ((uint64_t)Nq + 127) / 128 * bh;
    if (bh > (1ull << 31) - 1 || ctas > (1ull << 31) - 1) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return ATTN_ERR_MISALIGNED;
    if ((lse && !aligned4(lse)) || (kv_lens && !aligned4(kv_lens))) return ATTN_ERR_MISALIGNED;
    return ATTN_OK;
}

}  // namespace

namespace attn {

cudaError_t current_sm_count(int *sms) {
    static int cache[kMaxDevices];  // 0 = unknown
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (cache[dev] == 0) {
        int n = 0;
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        cache[dev] = n;
    }
    *sms = cache[dev];
    return cudaSuccess;
}

cudaError_t ensure_max_dynamic_smem(const void *kernel, int bytes) {
    struct Entry {
        const void *fn;
        int dev;
        int bytes;
    };
    static Entry done[512];
    static int n_done = 0;
    static std::mutex mu;
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(mu);
    for (int i = 0; i < n_done; ++i)
        if (done[i].fn == kernel && done[i].dev == dev && done[i].bytes >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (n_done < 512) done[n_done++] = Entry{kernel, dev, bytes};
    return cudaSuccess;
}

cudaError_t ensure_large_clusters(const void *kernel) {
    struct Entry {
        const void *fn;
        int dev;
    };
    static Entry done[512];
    static int n_done = 0;
    static std::mutex mu;
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < n_done; ++i)
        if (done[i].fn == kernel && done[i].dev == dev) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (n_done < 512) done[n_done++] = Entry{kernel, dev};
    return cudaSuccess;
}

bool cluster_fits(const void *kernel, int n, int threads, size_t smem) {
    struct Entry {
        const void *fn;
        int dev, n;
        bool fits;
    };
    static Entry done[512];
    static int n_done = 0;
    static std::mutex mu;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < n_done; ++i)
        if (done[i].fn == kernel && done[i].dev == dev && done[i].n == n) return done[i].fits;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = n;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    const bool fits = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) == cudaSuccess && clusters > 0;
    if (!fits) (void)cudaGetLastError();
    if (n_done < 512) done[n_done++] = Entry{kernel, dev, n, fits};
    return fits;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn get_encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

// [BH, N, D] bf16 viewed as a 3-D tensor (innermost first), boxes of 64 x 128 x 1, 128-byte swizzle.
bool encode_qkv_map(CUtensorMap *m, const void *ptr, int BH, int N, int D, int box_rows) {
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)N, (cuuint64_t)BH};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)N * D * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

bool encode_q_heads_map(CUtensorMap *m, const void *ptr, int B, int H, int D, int heads, int seqs) {
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)B};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)seqs};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

bool encode_page_map_u8(CUtensorMap *m, const void *ptr, int rows, int page_rows, int D, bool swizzle) {
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)page_rows, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)page_rows * D};
    cuuint32_t box[3] = {128, (cuuint32_t)page_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(ptr), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

}  // namespace attn

ATTN_API int attn_fwd_gqa(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq,
                          int Hkv, int Nq, int Nkv, int d, int causal, float scale, const int32_t *kv_lens,
                          attn_stream_t stream) {
    int st = prefill_checks(q, k, v, o, lse, B, Hq, Hkv, Nq, Nkv, d, causal, scale, kv_lens);
    if (st != ATTN_OK) return st;
    int *status = nullptr;
    st = device_setup(&status);
    if (st != ATTN_OK) return st;
    attn::PrefillArgs a{q, k, v, o, lse, kv_lens, status, B, Hq, Nq, Nkv, d, causal, scale, Hkv};
    cudaError_t e = attn::launch_prefill(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

ATTN_API int attn_fwd_kvlen(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H,
                            int Nq, int Nkv, int d, int causal, float scale, const int32_t *kv_lens,
                            attn_stream_t stream) {
    return attn_fwd_gqa(q, k, v, o, lse, B, H, H, Nq, Nkv, d, causal, scale, kv_lens, stream);
}

ATTN_API int attn_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H, int Nq,
                      int Nkv, int d, int causal, float scale, attn_stream_t stream) {
    return attn_fwd_kvlen(q, k, v, o, lse, B, H, Nq, Nkv, d, causal, scale, nullptr, stream);
}

namespace {
// The score modification's arguments: softcap 0 (none), or positive with factors that fp32 holds (cap and
// score factor / cap at most 2^100, the factor at least 2^-100 with slopes; `factor` is the scale, times the
// key scale of an e4m3 cache); 4-byte aligned arrays.
int scoremod_checks(float factor, float softcap, const float *alibi_slopes, const int32_t *key_begin,
                    const int32_t *key_end) {
    constexpr float kMost = 1.2676506e30f;  // 2^100
    if (!(factor > 0.f) || !(factor < 3.0e38f)) return ATTN_ERR_INVALID_ARG;
    if (alibi_slopes && !(factor >= 1.f / kMost)) return ATTN_ERR_INVALID_ARG;  // slopes are divided by it
    if (!(softcap >= 0.f) || !(softcap <= kMost)) return ATTN_ERR_INVALID_ARG;
    if (softcap > 0.f && !(factor / softcap <= kMost)) return ATTN_ERR_INVALID_ARG;
    if (!aligned4(alibi_slopes) || !aligned4(key_begin) || !aligned4(key_end)) return ATTN_ERR_MISALIGNED;
    return ATTN_OK;
}
}  // namespace

ATTN_API int attn_fwd_scoremod(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq,
                               int Hkv, int Nq, int Nkv, int d, int causal, float scale, float softcap,
                               const float *alibi_slopes, const int32_t *key_begin, const int32_t *key_end,
                               const int32_t *kv_lens, attn_stream_t stream) {
    int st = prefill_checks(q, k, v, o, lse, B, Hq, Hkv, Nq, Nkv, d, causal, scale, kv_lens);
    if (st == ATTN_OK) st = scoremod_checks(scale, softcap, alibi_slopes, key_begin, key_end);
    if (st != ATTN_OK) return st;
    int *status = nullptr;
    st = device_setup(&status);
    if (st != ATTN_OK) return st;
    attn::PrefillArgs a{q, k, v, o, lse, kv_lens, status, B, Hq, Nq, Nkv, d, causal, scale, Hkv};
    a.softcap = softcap;
    a.slopes = alibi_slopes;
    a.key_begin = key_begin;
    a.key_end = key_end;
    cudaError_t e = attn::launch_prefill_scoremod(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

ATTN_API size_t attn_bwd_workspace_size(int B, int Hq, int Nq) { return attn::bwd_workspace_bytes(B, Hq, Nq); }

ATTN_API int attn_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse, const void *dout,
                      void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int Nq, int Nkv, int d, int causal,
                      float scale, const int32_t *kv_lens, void *workspace, size_t workspace_bytes,
                      attn_stream_t stream) {
    if (!o || !lse || !dout || !dk || !dv) return ATTN_ERR_INVALID_ARG;
    // q, k, v, dq and the sizes get the forward's checks (dq in the place of o)
    int st = prefill_checks(q, k, v, dq, nullptr, B, Hq, Hkv, Nq, Nkv, d, causal, scale, kv_lens);
    if (st != ATTN_OK) return st;
    if (d != 32 && d != 64 && d != 80 && d != 96 && d != 128) return ATTN_ERR_UNSUPPORTED;
    const uint64_t kv_ctas = ((uint64_t)Nkv + 127) / 128 * (uint64_t)B * (uint64_t)Hkv;
    if (kv_ctas > (1ull << 31) - 1) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(o) || !aligned16(dout) || !aligned16(dk) || !aligned16(dv) || !aligned4(lse))
        return ATTN_ERR_MISALIGNED;
    const size_t need = attn::bwd_workspace_bytes(B, Hq, Nq);
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
    int *status = nullptr;
    st = device_setup(&status);
    if (st != ATTN_OK) return st;
    attn::BwdArgs a{q,  k,  v,      o, dout, lse, dq, dk, dv, static_cast<float *>(workspace), kv_lens, status,
                    B,  Hq, Hkv, Nq, Nkv, d, causal, scale};
    cudaError_t e = attn::launch_bwd(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

ATTN_API int paged_attn_prefill(const void *q, const void *k_pages, const void *v_pages, const int32_t *page_table,
                                const int32_t *ctx_lens, int page_size, void *o, float *lse, int B, int H, int Hkv,
                                int Nq, int d, int max_pages_per_seq, int num_pages, int causal, float scale,
                                attn_stream_t stream) {
    if (!page_table || !ctx_lens || !k_pages || !v_pages) return ATTN_ERR_INVALID_ARG;
    if (page_size <= 0 || max_pages_per_seq <= 0 || num_pages <= 0) return ATTN_ERR_INVALID_ARG;
    if (page_size != 16) return ATTN_ERR_UNSUPPORTED;
    if ((uint64_t)max_pages_per_seq * 16 > (1ull << 30)) return ATTN_ERR_INVALID_ARG;
    if (Hkv <= 0 || (uint64_t)num_pages * (uint64_t)Hkv > (1ull << 31) - 1) return ATTN_ERR_INVALID_ARG;
    const int cap = max_pages_per_seq * 16;
    int st = prefill_checks(q, k_pages, v_pages, o, lse, B, H, Hkv, Nq, cap, d, causal, scale, nullptr);
    if (st != ATTN_OK) return st;
    if (!aligned4(page_table) || !aligned4(ctx_lens)) return ATTN_ERR_MISALIGNED;
    int *status = nullptr;
    st = device_setup(&status);
    if (st != ATTN_OK) return st;
    attn::PrefillArgs a{q, k_pages, v_pages, o, lse, nullptr, status, B, H, Nq, cap, d, causal, scale, Hkv};
    a.paged = 1;
    a.page_table = page_table;
    a.ctx_lens = ctx_lens;
    a.max_pages = max_pages_per_seq;
    a.num_pages = num_pages;
    cudaError_t e = attn::launch_prefill(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

ATTN_API int paged_attn_prefill_fp8(const void *q, const void *k_pages, const void *v_pages, float k_scale,
                                    float v_scale, const int32_t *page_table, const int32_t *ctx_lens, int page_size,
                                    void *o, float *lse, int B, int H, int Hkv, int Nq, int d, int max_pages_per_seq,
                                    int num_pages, int causal, float scale, attn_stream_t stream) {
    if (!page_table || !ctx_lens || !k_pages || !v_pages) return ATTN_ERR_INVALID_ARG;
    if (page_size <= 0 || max_pages_per_seq <= 0 || num_pages <= 0) return ATTN_ERR_INVALID_ARG;
    if (!(k_scale > 0.f) || !(k_scale < 3.0e38f) || !(v_scale > 0.f) || !(v_scale < 3.0e38f))
        return ATTN_ERR_INVALID_ARG;
    if (page_size != 16) return ATTN_ERR_UNSUPPORTED;
    if ((uint64_t)max_pages_per_seq * 16 > (1ull << 30)) return ATTN_ERR_INVALID_ARG;
    if (Hkv <= 0 || (uint64_t)num_pages * (uint64_t)Hkv > (1ull << 31) - 1) return ATTN_ERR_INVALID_ARG;
    const int cap = max_pages_per_seq * 16;
    int st = prefill_checks(q, k_pages, v_pages, o, lse, B, H, Hkv, Nq, cap, d, causal, scale, nullptr);
    if (st != ATTN_OK) return st;
    if (!aligned4(page_table) || !aligned4(ctx_lens)) return ATTN_ERR_MISALIGNED;
    int *status = nullptr;
    st = device_setup(&status);
    if (st != ATTN_OK) return st;
    attn::PrefillArgs a{q, k_pages, v_pages, o, lse, nullptr, status, B, H, Nq, cap, d, causal, scale, Hkv};
    a.paged = 1;
    a.page_table = page_table;
    a.ctx_lens = ctx_lens;
    a.max_pages = max_pages_per_seq;
    a.num_pages = num_pages;
    a.kv_fp8 = 1;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    cudaError_t e = attn::launch_prefill(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

ATTN_API int paged_kv_append(const void *k_new, const void *v_new, void *k_pages, void *v_pages,
                             const int32_t *page_table, const int32_t *start_pos, int page_size, int B, int Hkv,
                             int Nnew, int d, int max_pages_per_seq, int num_pages, attn_stream_t stream) {
    if (!k_new || !v_new || !k_pages || !v_pages || !page_table || !start_pos) return ATTN_ERR_INVALID_ARG;
    if (B <= 0 || Hkv <= 0 || Nnew <= 0 || d <= 0 || page_size <= 0 || max_pages_per_seq <= 0 || num_pages <= 0)
        return ATTN_ERR_INVALID_ARG;
    if (!prefill_head_dim(d)) return ATTN_ERR_UNSUPPORTED;
    if (page_size != 16) return ATTN_ERR_UNSUPPORTED;
    if ((uint64_t)max_pages_per_seq * 16 > (1ull << 30)) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pages) || !aligned16(v_pages))
        return ATTN_ERR_MISALIGNED;
    if (!aligned4(page_table) || !aligned4(start_pos)) return ATTN_ERR_MISALIGNED;
    int *status = nullptr;
    int st = device_setup(&status);
    if (st != ATTN_OK) return st;
    cudaError_t e = attn::launch_kv_append(k_new, v_new, k_pages, v_pages, page_table, start_pos, B, Hkv, Nnew, d,
                                           max_pages_per_seq, num_pages, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

ATTN_API size_t paged_attn_decode_workspace_size(int B, int H, int d, int max_pages_per_seq, int page_size) {
    return attn::decode_workspace_bytes(B, H, H, d, max_pages_per_seq, page_size);
}

ATTN_API size_t paged_attn_decode_workspace_size_ctx(int B, int H, int d, int max_ctx_len) {
    if (max_ctx_len <= 0) return 0;
    return attn::decode_workspace_bytes(B, H, H, d, (int)(((int64_t)max_ctx_len + 15) / 16), 16);
}

ATTN_API size_t paged_attn_decode_gqa_workspace_size(int B, int H, int Hkv, int d, int max_pages_per_seq,
                                                     int page_size) {
    return attn::decode_workspace_bytes(B, H, Hkv, d, max_pages_per_seq, page_size);
}

namespace {
bool finite_positive(float x) { return x > 0.f && x < 3.0e38f; }
// A tensor's scale of the 4-bit cache: it and its reciprocal are normal fp32 numbers.
bool fp4_scale(float x) { return x >= 1e-37f && x <= 1e37f; }
// Head dims of the decode kernels: the same five as the prefill.
bool decode_head_dim(int d) { return prefill_head_dim(d); }

// Checks shared by every decode entry point: everything but the caller's workspace.
int decode_arg_checks(const void *q, const void *k_pages, const void *v_pages, const int32_t *page_table,
                      const int32_t *ctx_lens, int page_size, void *o, float *lse, int B, int H, int Hkv, int d,
                      int max_pages_per_seq, int num_pages, float scale) {
    if (!q || !k_pages || !v_pages || !page_table || !ctx_lens || !o) return ATTN_ERR_INVALID_ARG;
    if (B <= 0 || H <= 0 || d <= 0 || page_size <= 0 || max_pages_per_seq <= 0 || num_pages <= 0)
        return ATTN_ERR_INVALID_ARG;
    if (Hkv <= 0 || H % Hkv != 0) return ATTN_ERR_INVALID_ARG;
    if ((uint64_t)num_pages * (uint64_t)Hkv > (1ull << 31) - 1) return ATTN_ERR_INVALID_ARG;  // TMA rows
    if (!finite_positive(scale)) return ATTN_ERR_INVALID_ARG;
    if (!decode_head_dim(d)) return ATTN_ERR_UNSUPPORTED;
    if (page_size != 16) return ATTN_ERR_UNSUPPORTED;
    if (B > 65535 || H > 65535) return ATTN_ERR_INVALID_ARG;  // grid y/z limits
    if ((uint64_t)max_pages_per_seq * (uint64_t)page_size > (1ull << 30)) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o)) return ATTN_ERR_MISALIGNED;
    if (!aligned4(page_table) || !aligned4(ctx_lens) || (lse && !aligned4(lse))) return ATTN_ERR_MISALIGNED;
    return ATTN_OK;
}

int decode_checks(const void *q, const void *k_pages, const void *v_pages, const int32_t *page_table,
                  const int32_t *ctx_lens, int page_size, void *o, float *lse, int B, int H, int Hkv, int d,
                  int max_pages_per_seq, int num_pages, float scale, void *workspace, size_t workspace_bytes) {
    const int st = decode_arg_checks(q, k_pages, v_pages, page_table, ctx_lens, page_size, o, lse, B, H, Hkv, d,
                                     max_pages_per_seq, num_pages, scale);
    if (st != ATTN_OK) return st;
    const size_t need = attn::decode_workspace_bytes(B, H, Hkv, d, max_pages_per_seq, page_size);
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
    return ATTN_OK;
}
}  // namespace

ATTN_API int paged_attn_decode_fp8(const void *q, const void *k_pages, const void *v_pages, float k_scale,
                                   float v_scale, const int32_t *page_table, const int32_t *ctx_lens, int page_size,
                                   void *o, float *lse, int B, int H, int Hkv, int d, int max_pages_per_seq,
                                   int num_pages, float scale, void *workspace, size_t workspace_bytes,
                                   attn_stream_t stream) {
    int st = decode_checks(q, k_pages, v_pages, page_table, ctx_lens, page_size, o, lse, B, H, Hkv, d,
                           max_pages_per_seq, num_pages, scale, workspace, workspace_bytes);
    if (st != ATTN_OK) return st;
    if (!finite_positive(k_scale) || !finite_positive(v_scale)) return ATTN_ERR_INVALID_ARG;
    int *status = nullptr;
    st = device_setup(&status);
    if (st != ATTN_OK) return st;
    attn::DecodeArgs a{q,  k_pages, v_pages, page_table, ctx_lens, o, lse, workspace, status, B, H, d, page_size,
                       max_pages_per_seq, num_pages, scale, Hkv};
    a.kv_fp8 = 1;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    cudaError_t e = attn::launch_decode(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

ATTN_API int kv_quantize_fp8(const void *src, void *dst, size_t n, float scale, attn_stream_t stream) {
    if (!src || !dst || n == 0 || n % 8 != 0 || n > (1ull << 40)) return ATTN_ERR_INVALID_ARG;
    if (!finite_positive(scale)) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(src) || !aligned16(dst)) return ATTN_ERR_MISALIGNED;
    int *status = nullptr;
    int st = device_setup(&status);
    if (st != ATTN_OK) return st;
    cudaError_t e = attn::launch_kv_quantize_fp8(src, dst, n, 1.0f / scale, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

ATTN_API int paged_kv_append_fp8(const void *k_new, const void *v_new, void *k_pages, void *v_pages, float k_scale,
                                 float v_scale, const int32_t *page_table, const int32_t *start_pos, int page_size,
                                 int B, int Hkv, int Nnew, int d, int max_pages_per_seq, int num_pages,
                                 attn_stream_t stream) {
    if (!k_new || !v_new || !k_pages || !v_pages || !page_table || !start_pos) return ATTN_ERR_INVALID_ARG;
    if (B <= 0 || Hkv <= 0 || Nnew <= 0 || d <= 0 || page_size <= 0 || max_pages_per_seq <= 0 || num_pages <= 0)
        return ATTN_ERR_INVALID_ARG;
    if (!finite_positive(k_scale) || !finite_positive(v_scale)) return ATTN_ERR_INVALID_ARG;
    if (!prefill_head_dim(d)) return ATTN_ERR_UNSUPPORTED;
    if (page_size != 16) return ATTN_ERR_UNSUPPORTED;
    if ((uint64_t)max_pages_per_seq * 16 > (1ull << 30)) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pages) || !aligned16(v_pages))
        return ATTN_ERR_MISALIGNED;
    if (!aligned4(page_table) || !aligned4(start_pos)) return ATTN_ERR_MISALIGNED;
    int *status = nullptr;
    int st = device_setup(&status);
    if (st != ATTN_OK) return st;
    cudaError_t e = attn::launch_kv_append_fp8(k_new, v_new, k_pages, v_pages, 1.0f / k_scale, 1.0f / v_scale,
                                               page_table, start_pos, B, Hkv, Nnew, d, max_pages_per_seq, num_pages,
                                               reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

ATTN_API size_t attn_bwd_scoremod_workspace_size(int B, int Hq, int Hkv, int Nq, int Nkv, int d) {
    size_t offsets[2];
    return attn::bwd_scoremod_workspace_bytes(B, Hq, Hkv, Nq, Nkv, d, offsets);
}

ATTN_API int attn_bwd_scoremod(const void *q, const void *k, const void *v, const void *o, const float *lse,
                               const void *dout, void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int Nq, int Nkv,
                               int d, int causal, float scale, float softcap, const float *alibi_slopes,
                               const int32_t *key_begin, const int32_t *key_end, const int32_t *kv_lens,
                               void *workspace, size_t workspace_bytes, attn_stream_t stream) {
    if (!o || !lse || !dout || !dk || !dv) return ATTN_ERR_INVALID_ARG;
    int st = prefill_checks(q, k, v, dq, nullptr, B, Hq, Hkv, Nq, Nkv, d, causal, scale, kv_lens);
    if (st == ATTN_OK) st = scoremod_checks(scale, softcap, alibi_slopes, key_begin, key_end);
    if (st != ATTN_OK) return st;
    const uint64_t kv_ctas = ((uint64_t)Nkv + 127) / 128 * (uint64_t)B * (uint64_t)Hkv;
    if (kv_ctas > (1ull << 31) - 1) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(o) || !aligned16(dout) || !aligned16(dk) || !aligned16(dv) || !aligned4(lse))
        return ATTN_ERR_MISALIGNED;
    size_t offsets[2];
    const size_t need = attn::bwd_scoremod_workspace_bytes(B, Hq, Hkv, Nq, Nkv, d, offsets);
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
    int *status = nullptr;
    st = device_setup(&status);
    if (st != ATTN_OK) return st;
    attn::BwdArgs a{q,  k,  v,      o, dout, lse, dq, dk, dv, static_cast<float *>(workspace), kv_lens, status,
                    B,  Hq, Hkv, Nq, Nkv, d, causal, scale};
    a.softcap = softcap;
    a.slopes = alibi_slopes;
    a.key_begin = key_begin;
    a.key_end = key_end;
    a.spans = reinterpret_cast<int2 *>(static_cast<char *>(workspace) + offsets[0]);
    a.kv_parts = reinterpret_cast<float *>(static_cast<char *>(workspace) + offsets[1]);
    cudaError_t e = attn::launch_bwd_scoremod(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

namespace {
// Strides {batch, head, token} of a [B, H, N, d] input, in elements: the caller's (dims of size one
// count as 0), or those of a contiguous tensor.  Rows are read as 16-byte vectors.
int input_strides(const int64_t *given, int B, int H, int N, int d, int64_t (&out)[3]) {
    const int64_t dense[3] = {(int64_t)H * N * d, (int64_t)N * d, d};
    const int size[3] = {B, H, N};
    for (int i = 0; i < 3; ++i) {
        out[i] = size[i] == 1 ? 0 : (given ? given[i] : dense[i]);
        if (out[i] < 0 || out[i] > (1ll << 40)) return ATTN_ERR_INVALID_ARG;
        if (out[i] % 8 != 0) return ATTN_ERR_MISALIGNED;
    }
    return ATTN_OK;
}

// Positions with several axes: [axes, B, N] (or [axes, 1, N] for all sequences), and the axis of each of the rope_dim / 2
// pairs, on the host.
int rope_axes_arg(const int32_t *positions, int n_axes, int positions_batch, const uint8_t *pair_axis, int rope_dim, int B,
                  int N, attn::RopeAxes &out) {
    if (!positions || !pair_axis || n_axes <= 0 || B <= 0 || N <= 0) return ATTN_ERR_INVALID_ARG;
    if (positions_batch != 1 && positions_batch != B) return ATTN_ERR_INVALID_ARG;
    if (n_axes > attn::kMaxAxes) return ATTN_ERR_UNSUPPORTED;
    if (rope_dim <= 0 || rope_dim > attn::kMaxRope || rope_dim % 16 != 0) return ATTN_ERR_UNSUPPORTED;
    if (!aligned4(positions)) return ATTN_ERR_MISALIGNED;
    out.positions = positions;
    out.batch_stride = positions_batch == 1 ? 0 : N;
    out.axis_stride = (long long)positions_batch * N;
    out.axes = n_axes;
    out.pair_axis[0] = out.pair_axis[1] = 0;
    for (int i = 0; i < rope_dim / 2; ++i) {
        if (pair_axis[i] >= n_axes) return ATTN_ERR_INVALID_ARG;
        out.pair_axis[i >> 5] |= (uint64_t)pair_axis[i] << (2 * (i & 31));
    }
    return ATTN_OK;
}

// fp4: into the 4-bit cache, where the rotation may be left out (cos_sin null, and then no queries).
int append_rope(attn::RopeAppendArgs a, const int64_t *q_strides, const int64_t *k_strides, const int64_t *v_strides,
                int page_size, attn_stream_t stream, bool fp4 = false) {
    if (!a.k_new || !a.v_new || !a.k_pages || !a.v_pages || !a.page_table || !a.start_pos) return ATTN_ERR_INVALID_ARG;
    const bool plain = fp4 && !a.cos_sin;
    if (!a.cos_sin && (!plain || a.q || a.axes.positions)) return ATTN_ERR_INVALID_ARG;
    if (plain) a.rope_dim = 16, a.max_pos = 1, a.interleaved = 0;
    if ((a.q == nullptr) != (a.q_out == nullptr)) return ATTN_ERR_INVALID_ARG;
    if (a.B <= 0 || a.Hkv <= 0 || a.Nnew <= 0 || a.d <= 0 || page_size <= 0 || a.max_pages <= 0 || a.num_pages <= 0 ||
        a.max_pos <= 0 || (a.q && a.H <= 0))
        return ATTN_ERR_INVALID_ARG;
    if (a.interleaved != 0 && a.interleaved != 1) return ATTN_ERR_INVALID_ARG;
    if (a.kv_fp8 && (!finite_positive(a.k_scale) || !finite_positive(a.v_scale))) return ATTN_ERR_INVALID_ARG;
    if (fp4 && (!fp4_scale(a.k_scale) || !fp4_scale(a.v_scale))) return ATTN_ERR_INVALID_ARG;
    if (!prefill_head_dim(a.d) || page_size != 16) return ATTN_ERR_UNSUPPORTED;
    if (a.rope_dim <= 0 || a.rope_dim > a.d || a.rope_dim % 16 != 0) return ATTN_ERR_UNSUPPORTED;
    if ((uint64_t)a.max_pages * 16 > (1ull << 30)) return ATTN_ERR_INVALID_ARG;
    if ((uint64_t)a.B * (uint64_t)a.Nnew > (1ull << 31) - 1) return ATTN_ERR_INVALID_ARG;
    if ((uint64_t)(a.q ? a.H : 0) + 2 * (uint64_t)a.Hkv > (1u << 24)) return ATTN_ERR_INVALID_ARG;
    if (!a.q) a.H = 0;
    int st = input_strides(a.q ? q_strides : nullptr, a.B, a.q ? a.H : 1, a.Nnew, a.d, a.q_strides);
    if (st == ATTN_OK) st = input_strides(k_strides, a.B, a.Hkv, a.Nnew, a.d, a.k_strides);
    if (st == ATTN_OK) st = input_strides(v_strides, a.B, a.Hkv, a.Nnew, a.d, a.v_strides);
    if (st != ATTN_OK) return st;
    if (!aligned16(a.q) || !aligned16(a.q_out) || !aligned16(a.k_new) || !aligned16(a.v_new) || !aligned16(a.k_pages) ||
        !aligned16(a.v_pages) || !aligned16(a.cos_sin))
        return ATTN_ERR_MISALIGNED;
    if (!aligned4(a.page_table) || !aligned4(a.start_pos) || !aligned4(a.new_lens)) return ATTN_ERR_MISALIGNED;
    int *status = nullptr;
    st = device_setup(&status);
    if (st != ATTN_OK) return st;
    const cudaError_t e = fp4 ? attn::launch_kv_append_fp4(a, reinterpret_cast<cudaStream_t>(stream))
                              : attn::launch_kv_append_rope(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
}  // namespace

ATTN_API int paged_kv_append_rope(const void *q, const int64_t *q_strides, const void *k_new, const int64_t *k_strides,
                                  const void *v_new, const int64_t *v_strides, void *q_out, void *k_pages,
                                  void *v_pages, const float *cos_sin, int rope_dim, int max_pos, int interleaved,
                                  const int32_t *page_table, const int32_t *start_pos, const int32_t *new_lens,
                                  int page_size, int B, int H, int Hkv, int Nnew, int d, int max_pages_per_seq,
                                  int num_pages, attn_stream_t stream) {
    attn::RopeAppendArgs a{q, k_new, v_new, {}, {}, {}, q_out, k_pages, v_pages, cos_sin, rope_dim, max_pos,
                           interleaved, page_table, start_pos, new_lens, B, H, Hkv, Nnew, d, max_pages_per_seq,
                           num_pages};
    return append_rope(a, q_strides, k_strides, v_strides, page_size, stream);
}

ATTN_API int paged_kv_append_rope_fp8(const void *q, const int64_t *q_strides, const void *k_new,
                                      const int64_t *k_strides, const void *v_new, const int64_t *v_strides,
                                      void *q_out, void *k_pages, void *v_pages, float k_scale, float v_scale,
                                      const float *cos_sin, int rope_dim, int max_pos, int interleaved,
                                      const int32_t *page_table, const int32_t *start_pos, const int32_t *new_lens,
                                      int page_size, int B, int H, int Hkv, int Nnew, int d, int max_pages_per_seq,
                                      int num_pages, attn_stream_t stream) {
    attn::RopeAppendArgs a{q, k_new, v_new, {}, {}, {}, q_out, k_pages, v_pages, cos_sin, rope_dim, max_pos,
                           interleaved, page_table, start_pos, new_lens, B, H, Hkv, Nnew, d, max_pages_per_seq,
                           num_pages, 1, k_scale, v_scale};
    return append_rope(a, q_strides, k_strides, v_strides, page_size, stream);
}

ATTN_API int paged_kv_append_rope_axes(const void *q, const int64_t *q_strides, const void *k_new, const int64_t *k_strides,
                                       const void *v_new, const int64_t *v_strides, void *q_out, void *k_pages,
                                       void *v_pages, const float *cos_sin, int rope_dim, int max_pos, int interleaved,
                                       const int32_t *positions, int n_axes, const uint8_t *pair_axis,
                                       const int32_t *page_table, const int32_t *start_pos, const int32_t *new_lens,
                                       int page_size, int B, int H, int Hkv, int Nnew, int d, int max_pages_per_seq,
                                       int num_pages, attn_stream_t stream) {
    attn::RopeAppendArgs a{q, k_new, v_new, {}, {}, {}, q_out, k_pages, v_pages, cos_sin, rope_dim, max_pos,
                           interleaved, page_table, start_pos, new_lens, B, H, Hkv, Nnew, d, max_pages_per_seq,
                           num_pages};
    const int st = rope_axes_arg(positions, n_axes, B, pair_axis, rope_dim, B, Nnew, a.axes);
    return st == ATTN_OK ? append_rope(a, q_strides, k_strides, v_strides, page_size, stream) : st;
}

ATTN_API int paged_kv_append_rope_axes_fp8(const void *q, const int64_t *q_strides, const void *k_new,
                                           const int64_t *k_strides, const void *v_new, const int64_t *v_strides,
                                           void *q_out, void *k_pages, void *v_pages, float k_scale, float v_scale,
                                           const float *cos_sin, int rope_dim, int max_pos, int interleaved,
                                           const int32_t *positions, int n_axes, const uint8_t *pair_axis,
                                           const int32_t *page_table, const int32_t *start_pos, const int32_t *new_lens,
                                           int page_size, int B, int H, int Hkv, int Nnew, int d, int max_pages_per_seq,
                                           int num_pages, attn_stream_t stream) {
    attn::RopeAppendArgs a{q, k_new, v_new, {}, {}, {}, q_out, k_pages, v_pages, cos_sin, rope_dim, max_pos,
                           interleaved, page_table, start_pos, new_lens, B, H, Hkv, Nnew, d, max_pages_per_seq,
                           num_pages, 1, k_scale, v_scale};
    const int st = rope_axes_arg(positions, n_axes, B, pair_axis, rope_dim, B, Nnew, a.axes);
    return st == ATTN_OK ? append_rope(a, q_strides, k_strides, v_strides, page_size, stream) : st;
}

ATTN_API int paged_kv_append_fp4(const void *q, const int64_t *q_strides, const void *k_new, const int64_t *k_strides,
                                 const void *v_new, const int64_t *v_strides, void *q_out, void *k_pages, void *v_pages,
                                 float k_scale, float v_scale, const float *cos_sin, int rope_dim, int max_pos,
                                 int interleaved, const int32_t *positions, int n_axes, const uint8_t *pair_axis,
                                 const int32_t *page_table, const int32_t *start_pos, const int32_t *new_lens, int page_size,
                                 int B, int H, int Hkv, int Nnew, int d, int max_pages_per_seq, int num_pages,
                                 attn_stream_t stream) {
    attn::RopeAppendArgs a{q, k_new, v_new, {}, {}, {}, q_out, k_pages, v_pages, cos_sin, rope_dim, max_pos,
                           interleaved, page_table, start_pos, new_lens, B, H, Hkv, Nnew, d, max_pages_per_seq,
                           num_pages, 0, k_scale, v_scale};
    if ((uint64_t)(B > 0 ? B : 0) * ((uint64_t)(Nnew > 0 ? Nnew : 0) / 2 + 1) > (1ull << 31) - 1) return ATTN_ERR_INVALID_ARG;
    int st = ATTN_OK;
    if (positions) st = rope_axes_arg(positions, n_axes, B, pair_axis, rope_dim, B, Nnew, a.axes);
    return st == ATTN_OK ? append_rope(a, q_strides, k_strides, v_strides, page_size, stream, true) : st;
}

ATTN_API int paged_kv_unpack_fp4(const void *k_pages, const void *v_pages, float k_scale, float v_scale,
                                 const int32_t *page_ids, int n, void *k_out, void *v_out, int page_size, int Hkv, int d,
                                 int num_pages, attn_stream_t stream) {
    if (!k_pages || !v_pages || !page_ids || !k_out || !v_out) return ATTN_ERR_INVALID_ARG;
    if (n <= 0 || Hkv <= 0 || d <= 0 || page_size <= 0 || num_pages <= 0) return ATTN_ERR_INVALID_ARG;
    if (!fp4_scale(k_scale) || !fp4_scale(v_scale)) return ATTN_ERR_INVALID_ARG;
    if (!prefill_head_dim(d) || page_size != 16) return ATTN_ERR_UNSUPPORTED;
    if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_out) || !aligned16(v_out) || !aligned4(page_ids))
        return ATTN_ERR_MISALIGNED;
    int *status = nullptr;
    const int st = device_setup(&status);
    if (st != ATTN_OK) return st;
    const cudaError_t e = attn::launch_kv_unpack_fp4(k_pages, v_pages, k_scale, v_scale, page_ids, n, k_out, v_out, Hkv, d,
                                                     num_pages, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

namespace {
// Whether no two of an output's rows of d elements overlap: in ascending order, each stride steps past all that the ones before
// it reach.  (Every stride is at most 2^40: what reaches past that is past every one.)
bool rows_apart(const int64_t (&strides)[3], int B, int H, int N, int d) {
    const int64_t size[3] = {B, H, N};
    bool seen[3] = {size[0] == 1, size[1] == 1, size[2] == 1};
    int64_t span = d;
    for (int n = 0; n < 3; ++n) {
        int at = -1;
        for (int i = 0; i < 3; ++i)
            if (!seen[i] && (at < 0 || strides[i] < strides[at])) at = i;
        if (at < 0) break;
        seen[at] = true;
        if (strides[at] < span) return false;
        constexpr int64_t kFar = 1ll << 41;
        span = size[at] - 1 > kFar / strides[at] ? kFar : span + (size[at] - 1) * strides[at];
    }
    return true;
}

int rope_axes(attn::RopeArgs a, const int64_t *q_strides, const int64_t *k_strides, const int64_t *q_out_strides,
              const int64_t *k_out_strides, const int32_t *positions, int n_axes, int positions_batch,
              const uint8_t *pair_axis, attn_stream_t stream) {
    if (!a.q || !a.q_out || !a.cos_sin || (a.k == nullptr) != (a.k_out == nullptr)) return ATTN_ERR_INVALID_ARG;
    if (a.B <= 0 || a.H <= 0 || a.N <= 0 || a.d <= 0 || a.max_pos <= 0 || (a.k && a.Hkv <= 0)) return ATTN_ERR_INVALID_ARG;
    if (a.interleaved != 0 && a.interleaved != 1) return ATTN_ERR_INVALID_ARG;
    if (!prefill_head_dim(a.d)) return ATTN_ERR_UNSUPPORTED;
    if (a.rope_dim <= 0 || a.rope_dim > a.d || a.rope_dim % 16 != 0) return ATTN_ERR_UNSUPPORTED;
    int st = rope_axes_arg(positions, n_axes, positions_batch, pair_axis, a.rope_dim, a.B, a.N, a.axes);
    if (st != ATTN_OK) return st;
    if ((uint64_t)a.B * (uint64_t)a.N > (1ull << 31) - 1) return ATTN_ERR_INVALID_ARG;
    if ((uint64_t)a.H + (uint64_t)(a.k ? a.Hkv : 0) > (1u << 24)) return ATTN_ERR_INVALID_ARG;
    st = input_strides(q_strides, a.B, a.H, a.N, a.d, a.q_strides);
    if (st == ATTN_OK) st = input_strides(q_out_strides, a.B, a.H, a.N, a.d, a.q_out_strides);
    if (st == ATTN_OK && a.k) st = input_strides(k_strides, a.B, a.Hkv, a.N, a.d, a.k_strides);
    if (st == ATTN_OK && a.k) st = input_strides(k_out_strides, a.B, a.Hkv, a.N, a.d, a.k_out_strides);
    if (st != ATTN_OK) return st;
    for (int i = 0; i < 3; ++i)  // in place: each row onto itself
        if ((a.q == a.q_out && a.q_strides[i] != a.q_out_strides[i]) ||
            (a.k && a.k == a.k_out && a.k_strides[i] != a.k_out_strides[i]))
            return ATTN_ERR_INVALID_ARG;
    if (!aligned16(a.q) || !aligned16(a.q_out) || !aligned16(a.k) || !aligned16(a.k_out) || !aligned16(a.cos_sin))
        return ATTN_ERR_MISALIGNED;
    // (each row is written by a block of its own)
    if (!rows_apart(a.q_out_strides, a.B, a.H, a.N, a.d) || (a.k && !rows_apart(a.k_out_strides, a.B, a.Hkv, a.N, a.d)) ||
        a.q_out == a.k_out)
        return ATTN_ERR_INVALID_ARG;
    int *status = nullptr;
    st = device_setup(&status);
    if (st != ATTN_OK) return st;
    const cudaError_t e = attn::launch_rope_axes(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
}  // namespace

ATTN_API int attn_rope_axes(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                            const float *cos_sin, int rope_dim, int max_pos, int interleaved, const int32_t *positions,
                            int n_axes, int positions_batch, const uint8_t *pair_axis, void *q_out,
                            const int64_t *q_out_strides, void *k_out, const int64_t *k_out_strides, int B, int H, int Hkv,
                            int N, int d, attn_stream_t stream) {
    const attn::RopeArgs a{q, k, q_out, k_out, {}, {}, {}, {}, cos_sin, rope_dim, max_pos, interleaved, 0, B, H, Hkv, N, d, {}};
    return rope_axes(a, q_strides, k_strides, q_out_strides, k_out_strides, positions, n_axes, positions_batch, pair_axis, stream);
}

ATTN_API int attn_rope_axes_bwd(const void *dq, const int64_t *dq_strides, const void *dk, const int64_t *dk_strides,
                                const float *cos_sin, int rope_dim, int max_pos, int interleaved, const int32_t *positions,
                                int n_axes, int positions_batch, const uint8_t *pair_axis, void *q_out,
                                const int64_t *q_out_strides, void *k_out, const int64_t *k_out_strides, int B, int H,
                                int Hkv, int N, int d, attn_stream_t stream) {
    const attn::RopeArgs a{dq, dk, q_out, k_out, {}, {}, {}, {}, cos_sin, rope_dim, max_pos, interleaved, 1, B, H, Hkv, N, d, {}};
    return rope_axes(a, dq_strides, dk_strides, q_out_strides, k_out_strides, positions, n_axes, positions_batch, pair_axis, stream);
}

// ---------------------------------------------------------------- page tables and reference counts
namespace {
int pages_sizes(int B, int max_pages, int num_pages, int page_size) {
    if (B <= 0 || max_pages <= 0 || num_pages <= 0 || page_size <= 0) return ATTN_ERR_INVALID_ARG;
    if (page_size != 16) return ATTN_ERR_UNSUPPORTED;
    if ((uint64_t)max_pages * 16 > (1ull << 30)) return ATTN_ERR_INVALID_ARG;
    // the kernels' sums over a table's entries and over the pool are 32 bits wide
    if ((uint64_t)B * (uint64_t)max_pages > (1ull << 30) || num_pages > (1 << 30)) return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}
}  // namespace

ATTN_API int paged_kv_fork(const int32_t *page_table, const int32_t *ctx_lens, const int32_t *parents,
                           const int32_t *ref_counts, int32_t *page_table_out, int32_t *ctx_lens_out,
                           int32_t *ref_counts_out, int page_size, int B, int B_out, int max_pages_per_seq, int num_pages,
                           attn_stream_t stream) {
    if (!page_table || !ctx_lens || !parents || !ref_counts || !page_table_out || !ctx_lens_out || !ref_counts_out)
        return ATTN_ERR_INVALID_ARG;
    int st = pages_sizes(B, max_pages_per_seq, num_pages, page_size);
    if (st != ATTN_OK) return st;
    if (B_out <= 0 || (uint64_t)B_out * (uint64_t)max_pages_per_seq > (1ull << 30) || page_table_out == page_table || ctx_lens_out == ctx_lens || ctx_lens_out == parents)
        return ATTN_ERR_INVALID_ARG;
    if (!aligned4(page_table) || !aligned4(ctx_lens) || !aligned4(parents) || !aligned4(ref_counts) ||
        !aligned4(page_table_out) || !aligned4(ctx_lens_out) || !aligned4(ref_counts_out))
        return ATTN_ERR_MISALIGNED;
    int *status = nullptr;
    st = device_setup(&status);
    if (st != ATTN_OK) return st;
    attn::PagesArgs a{};
    a.page_table = page_table;
    a.ctx_lens = ctx_lens;
    a.parents = parents;
    a.ref_counts = ref_counts;
    a.page_table_out = page_table_out;
    a.ctx_lens_out = ctx_lens_out;
    a.ref_counts_out = ref_counts_out;
    a.B = B;
    a.B_out = B_out;
    a.max_pages = max_pages_per_seq;
    a.num_pages = num_pages;
    const cudaError_t e = attn::launch_pages_fork(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

ATTN_API size_t paged_kv_reserve_workspace_size(int B, int num_pages) {
    return attn::pages_reserve_workspace_bytes(B, num_pages);
}

ATTN_API int paged_kv_reserve(const int32_t *page_table, const int32_t *ctx_lens, const int32_t *new_lens,
                              const int32_t *ref_counts, int32_t *page_table_out, int32_t *ref_counts_out,
                              int32_t *reserved, int32_t *src_pages, int32_t *dst_pages, int page_size, int B,
                              int max_pages_per_seq, int num_pages, void *workspace, size_t workspace_bytes,
                              attn_stream_t stream) {
    if (!page_table || !ctx_lens || !new_lens || !ref_counts || !page_table_out || !ref_counts_out || !reserved ||
        !src_pages || !dst_pages)
        return ATTN_ERR_INVALID_ARG;
    int st = pages_sizes(B, max_pages_per_seq, num_pages, page_size);
    if (st != ATTN_OK) return st;
    if (!aligned16(ref_counts) || !aligned16(ref_counts_out)) return ATTN_ERR_MISALIGNED;
    if (!aligned4(page_table) || !aligned4(ctx_lens) || !aligned4(new_lens) || !aligned4(page_table_out) ||
        !aligned4(reserved) || !aligned4(src_pages) || !aligned4(dst_pages))
        return ATTN_ERR_MISALIGNED;
    const size_t need = attn::pages_reserve_workspace_bytes(B, num_pages);
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
    int *status = nullptr;
    st = device_setup(&status);
    if (st != ATTN_OK) return st;
    attn::PagesArgs a{};
    a.page_table = page_table;
    a.ctx_lens = ctx_lens;
    a.new_lens = new_lens;
    a.ref_counts = ref_counts;
    a.page_table_out = page_table_out;
    a.ref_counts_out = ref_counts_out;
    a.reserved = reserved;
    a.src = src_pages;
    a.dst = dst_pages;
    a.B = a.B_out = B;
    a.max_pages = max_pages_per_seq;
    a.num_pages = num_pages;
    a.workspace = workspace;
    const cudaError_t e = attn::launch_pages_reserve(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

ATTN_API size_t paged_kv_compact_workspace_size(int num_pages) { return attn::pages_compact_workspace_bytes(num_pages); }

ATTN_API int paged_kv_compact(const int32_t *page_table, const int32_t *ref_counts, int32_t *page_table_out,
                              int32_t *ref_counts_out, int32_t *src_pages, int32_t *dst_pages, int32_t *count, int B,
                              int max_pages_per_seq, int num_pages, void *workspace, size_t workspace_bytes,
                              attn_stream_t stream) {
    if (!page_table || !ref_counts || !page_table_out || !ref_counts_out || !src_pages || !dst_pages || !count)
        return ATTN_ERR_INVALID_ARG;
    int st = pages_sizes(B, max_pages_per_seq, num_pages, 16);
    if (st != ATTN_OK) return st;
    if (ref_counts_out == ref_counts) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(ref_counts) || !aligned16(ref_counts_out)) return ATTN_ERR_MISALIGNED;
    if (!aligned4(page_table) || !aligned4(page_table_out) || !aligned4(src_pages) || !aligned4(dst_pages) || !aligned4(count))
        return ATTN_ERR_MISALIGNED;
    const size_t need = attn::pages_compact_workspace_bytes(num_pages);
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
    int *status = nullptr;
    st = device_setup(&status);
    if (st != ATTN_OK) return st;
    attn::PagesArgs a{};
    a.page_table = page_table;
    a.ref_counts = ref_counts;
    a.page_table_out = page_table_out;
    a.ref_counts_out = ref_counts_out;
    a.src = src_pages;
    a.dst = dst_pages;
    a.count = count;
    a.B = a.B_out = B;
    a.max_pages = max_pages_per_seq;
    a.num_pages = num_pages;
    a.workspace = workspace;
    const cudaError_t e = attn::launch_pages_compact(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

ATTN_API int paged_kv_copy_pages(void *const *pools, int n_pools, size_t page_bytes, const int32_t *src_pages,
                                 const int32_t *dst_pages, const int32_t *count, int n, int num_pages,
                                 attn_stream_t stream) {
    if (!pools || !src_pages || !dst_pages || n_pools <= 0 || n <= 0 || num_pages <= 0) return ATTN_ERR_INVALID_ARG;
    if (page_bytes == 0 || page_bytes > (1ull << 31) || page_bytes % 16 != 0) return ATTN_ERR_INVALID_ARG;
    for (int i = 0; i < n_pools; ++i) {
        if (!pools[i]) return ATTN_ERR_INVALID_ARG;
        if (!aligned16(pools[i])) return ATTN_ERR_MISALIGNED;
    }
    if (!aligned4(src_pages) || !aligned4(dst_pages) || !aligned4(count)) return ATTN_ERR_MISALIGNED;
    int *status = nullptr;
    const int st = device_setup(&status);
    if (st != ATTN_OK) return st;
    const cudaError_t e = attn::launch_pages_copy(pools, n_pools, page_bytes, src_pages, dst_pages, count, n, num_pages,
                                                  reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

ATTN_API int paged_attn_decode_gqa(const void *q, const void *k_pages, const void *v_pages,
                                   const int32_t *page_table, const int32_t *ctx_lens, int page_size, void *o,
                                   float *lse, int B, int H, int Hkv, int d, int max_pages_per_seq, int num_pages,
                                   float scale, void *workspace, size_t workspace_bytes, attn_stream_t stream) {
    int st = decode_checks(q, k_pages, v_pages, page_table, ctx_lens, page_size, o, lse, B, H, Hkv, d,
                           max_pages_per_seq, num_pages, scale, workspace, workspace_bytes);
    if (st != ATTN_OK) return st;
    int *status = nullptr;
    st = device_setup(&status);
    if (st != ATTN_OK) return st;
    attn::DecodeArgs a{q,  k_pages, v_pages, page_table, ctx_lens, o, lse, workspace, status, B, H, d, page_size,
                       max_pages_per_seq, num_pages, scale, Hkv};
    cudaError_t e = attn::launch_decode(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

ATTN_API size_t paged_attn_decode_scoremod_workspace_size(int B, int H, int Hkv, int d, int max_pages_per_seq,
                                                          int page_size) {
    return attn::decode_scoremod_workspace_bytes(B, H, Hkv, d, max_pages_per_seq, page_size);
}

ATTN_API size_t paged_attn_decode_shared_workspace_size(int B, int H, int Hkv, int d, int max_pages_per_seq,
                                                        int group_size, int page_size) {
    return attn::decode_shared_workspace_bytes(B, H, Hkv, d, max_pages_per_seq, group_size, page_size);
}

namespace {
// Decode with modified scores (k_scale, v_scale 1 for a bf16 cache); fp4: over the 4-bit cache.
int decode_scoremod(attn::DecodeMoreArgs a, size_t workspace_bytes, attn_stream_t stream, bool fp4 = false) {
    int st = decode_arg_checks(a.q, a.k_pages, a.v_pages, a.page_table, a.ctx_lens, a.page_size, a.o, a.lse, a.B, a.H,
                               a.Hkv, a.d, a.max_pages, a.num_pages, a.scale);
    if (st != ATTN_OK) return st;
    if ((uint64_t)a.B * (uint64_t)a.H > (1ull << 31) - 1) return ATTN_ERR_INVALID_ARG;
    if (!finite_positive(a.k_scale) || !finite_positive(a.v_scale)) return ATTN_ERR_INVALID_ARG;
    st = scoremod_checks(a.scale * a.k_scale, a.softcap, a.slopes, a.key_begin, nullptr);
    if (st != ATTN_OK) return st;
    const size_t need = (fp4 ? attn::decode_fp4_workspace_bytes : attn::decode_scoremod_workspace_bytes)(
        a.B, a.H, a.Hkv, a.d, a.max_pages, a.page_size);
    if (!a.workspace || !aligned16(a.workspace) || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
    st = device_setup(&a.status);
    if (st != ATTN_OK) return st;
    const cudaError_t e = (fp4 ? attn::launch_decode_fp4 : attn::launch_decode_scoremod)(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int decode_shared(attn::DecodeMoreArgs a, size_t workspace_bytes, attn_stream_t stream) {
    if (!a.shared_pages || a.group_size <= 0) return ATTN_ERR_INVALID_ARG;
    int st = decode_arg_checks(a.q, a.k_pages, a.v_pages, a.page_table, a.ctx_lens, a.page_size, a.o, a.lse, a.B, a.H,
                               a.Hkv, a.d, a.max_pages, a.num_pages, a.scale);
    if (st != ATTN_OK) return st;
    if (a.B % a.group_size != 0 || (uint64_t)a.B * (uint64_t)a.H > (1ull << 31) - 1) return ATTN_ERR_INVALID_ARG;
    if (!finite_positive(a.k_scale) || !finite_positive(a.v_scale) || !finite_positive(a.scale * a.k_scale))
        return ATTN_ERR_INVALID_ARG;
    if (!aligned4(a.shared_pages)) return ATTN_ERR_MISALIGNED;
    const size_t need = attn::decode_shared_workspace_bytes(a.B, a.H, a.Hkv, a.d, a.max_pages, a.group_size, a.page_size);
    if (!a.workspace || !aligned16(a.workspace) || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
    st = device_setup(&a.status);
    if (st != ATTN_OK) return st;
    const cudaError_t e = attn::launch_decode_shared(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
}  // namespace

ATTN_API int paged_attn_decode_scoremod(const void *q, const void *k_pages, const void *v_pages,
                                        const int32_t *page_table, const int32_t *ctx_lens, int page_size, void *o,
                                        float *lse, int B, int H, int Hkv, int d, int max_pages_per_seq, int num_pages,
                                        float scale, float softcap, const float *alibi_slopes,
                                        const int32_t *key_begin, void *workspace, size_t workspace_bytes,
                                        attn_stream_t stream) {
    attn::DecodeMoreArgs a{{q, k_pages, v_pages, page_table, ctx_lens, o, lse, workspace, nullptr, B, H, d, page_size,
                       max_pages_per_seq, num_pages, scale, Hkv}};
    a.softcap = softcap;
    a.slopes = alibi_slopes;
    a.key_begin = key_begin;
    return decode_scoremod(a, workspace_bytes, stream);
}

ATTN_API int paged_attn_decode_scoremod_fp8(const void *q, const void *k_pages, const void *v_pages, float k_scale,
                                            float v_scale, const int32_t *page_table, const int32_t *ctx_lens,
                                            int page_size, void *o, float *lse, int B, int H, int Hkv, int d,
                                            int max_pages_per_seq, int num_pages, float scale, float softcap,
                                            const float *alibi_slopes, const int32_t *key_begin, void *workspace,
                                            size_t workspace_bytes, attn_stream_t stream) {
    attn::DecodeMoreArgs a{{q, k_pages, v_pages, page_table, ctx_lens, o, lse, workspace, nullptr, B, H, d, page_size,
                       max_pages_per_seq, num_pages, scale, Hkv, 1, k_scale, v_scale}};
    a.softcap = softcap;
    a.slopes = alibi_slopes;
    a.key_begin = key_begin;
    return decode_scoremod(a, workspace_bytes, stream);
}

ATTN_API size_t paged_attn_decode_fp4_workspace_size(int B, int H, int Hkv, int d, int max_pages_per_seq, int page_size) {
    return attn::decode_fp4_workspace_bytes(B, H, Hkv, d, max_pages_per_seq, page_size);
}

ATTN_API int paged_attn_decode_fp4(const void *q, const void *k_pages, const void *v_pages, float k_scale, float v_scale,
                                   const int32_t *page_table, const int32_t *ctx_lens, int page_size, void *o, float *lse,
                                   int B, int H, int Hkv, int d, int max_pages_per_seq, int num_pages, float scale,
                                   float softcap, const float *alibi_slopes, const int32_t *key_begin, void *workspace,
                                   size_t workspace_bytes, attn_stream_t stream) {
    attn::DecodeMoreArgs a{{q, k_pages, v_pages, page_table, ctx_lens, o, lse, workspace, nullptr, B, H, d, page_size,
                       max_pages_per_seq, num_pages, scale, Hkv, 0, k_scale, v_scale}};
    a.softcap = softcap;
    a.slopes = alibi_slopes;
    a.key_begin = key_begin;
    // (their product is what a score's products are multiplied by: of 0, unseen scores of -inf would come to NaN)
    if (!fp4_scale(k_scale) || !fp4_scale(v_scale) || !fp4_scale(scale * k_scale)) return ATTN_ERR_INVALID_ARG;
    return decode_scoremod(a, workspace_bytes, stream, true);
}

ATTN_API int paged_attn_decode_shared(const void *q, const void *k_pages, const void *v_pages,
                                      const int32_t *page_table, const int32_t *ctx_lens,
                                      const int32_t *shared_pages, int group_size, int page_size, void *o, float *lse,
                                      int B, int H, int Hkv, int d, int max_pages_per_seq, int num_pages, float scale,
                                      void *workspace, size_t workspace_bytes, attn_stream_t stream) {
    attn::DecodeMoreArgs a{{q, k_pages, v_pages, page_table, ctx_lens, o, lse, workspace, nullptr, B, H, d, page_size,
                       max_pages_per_seq, num_pages, scale, Hkv}};
    a.shared_pages = shared_pages;
    a.group_size = group_size;
    return decode_shared(a, workspace_bytes, stream);
}

ATTN_API int paged_attn_decode_shared_fp8(const void *q, const void *k_pages, const void *v_pages, float k_scale,
                                          float v_scale, const int32_t *page_table, const int32_t *ctx_lens,
                                          const int32_t *shared_pages, int group_size, int page_size, void *o,
                                          float *lse, int B, int H, int Hkv, int d, int max_pages_per_seq,
                                          int num_pages, float scale, void *workspace, size_t workspace_bytes,
                                          attn_stream_t stream) {
    attn::DecodeMoreArgs a{{q, k_pages, v_pages, page_table, ctx_lens, o, lse, workspace, nullptr, B, H, d, page_size,
                       max_pages_per_seq, num_pages, scale, Hkv, 1, k_scale, v_scale}};
    a.shared_pages = shared_pages;
    a.group_size = group_size;
    return decode_shared(a, workspace_bytes, stream);
}

ATTN_API int paged_attn_decode(const void *q, const void *k_pages, const void *v_pages, const int32_t *page_table,
                               const int32_t *ctx_lens, int page_size, void *o, float *lse, int B, int H, int d,
                               int max_pages_per_seq, int num_pages, float scale, void *workspace,
                               size_t workspace_bytes, attn_stream_t stream) {
    return paged_attn_decode_gqa(q, k_pages, v_pages, page_table, ctx_lens, page_size, o, lse, B, H, H, d,
                                 max_pages_per_seq, num_pages, scale, workspace, workspace_bytes, stream);
}

// Decode with the chunk partials in the library's static scratch array (decode.cu);
// for callers that cannot allocate device memory.  Same checks as paged_attn_decode
// minus the workspace, plus the scratch capacity.
ATTN_API int paged_attn_decode_noalloc(const void *q, const void *k_pages, const void *v_pages,
                                       const int32_t *page_table, const int32_t *ctx_lens, int page_size, void *o,
                                       float *lse, int B, int H, int d, int max_pages_per_seq, int num_pages,
                                       float scale, attn_stream_t stream) {
    int st = decode_arg_checks(q, k_pages, v_pages, page_table, ctx_lens, page_size, o, lse, B, H, H, d,
                               max_pages_per_seq, num_pages, scale);
    if (st != ATTN_OK) return st;
    const size_t need = attn::decode_workspace_bytes(B, H, H, d, max_pages_per_seq, page_size);
    if (need == 0 || need > attn::decode_noalloc_scratch_bytes()) return ATTN_ERR_SCRATCH_LIMIT;
    int *status = nullptr;
    st = device_setup(&status);
    if (st != ATTN_OK) return st;
    attn::DecodeArgs a{q,  k_pages, v_pages, page_table, ctx_lens, o, lse, nullptr, status, B, H, d, page_size,
                       max_pages_per_seq, num_pages, scale, H};
    cudaError_t e = attn::launch_decode_noalloc(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

ATTN_API int attn_selftest_bounded_wait(attn_stream_t stream) {
    int *status = nullptr;
    int st = device_setup(&status);
    if (st != ATTN_OK) return st;
    return attn::launch_selftest_wait(status, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK
                                                                                                     : ATTN_ERR_CUDA;
}

ATTN_API int attn_check_device_status(attn_stream_t stream) {
    int dev = -1;
    if (current_device(&dev) != ATTN_OK) return ATTN_ERR_CUDA;
    int *status = nullptr;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        const int st = device_setup_locked(dev);
        if (st != ATTN_OK) return st;
        status = g_status_ptr[dev];
    }
    if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return ATTN_ERR_CUDA;
    int h[2] = {0, 0};
    if (cudaMemcpy(h, status, sizeof h, cudaMemcpyDeviceToHost) != cudaSuccess) return ATTN_ERR_CUDA;
    const bool timed_out = h[0] != 0 || *host_flag_of(dev) != 0;
    if (!timed_out) return ATTN_OK;
    const int zero[2] = {0, 0};  // flags and site; the flag address in [2..3] stays
    if (cudaMemcpy(status, zero, sizeof zero, cudaMemcpyHostToDevice) != cudaSuccess) return ATTN_ERR_CUDA;
    *host_flag_of(dev) = 0;
    return ATTN_ERR_DEVICE_TIMEOUT;
}

ATTN_API int attn_last_device_status(void) {
    int dev = -1;
    if (current_device(&dev) != ATTN_OK) return ATTN_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        const int st = device_setup_locked(dev);
        if (st != ATTN_OK) return st;
    }
    return *host_flag_of(dev) != 0 ? ATTN_ERR_DEVICE_TIMEOUT : ATTN_OK;
}

ATTN_API const char *attn_status_string(int status) {
    switch (status) {
        case ATTN_OK: return "ok";
        case ATTN_ERR_INVALID_ARG: return "invalid argument (null pointer, non-positive or oversized dimension, bad scale or cap)";
        case ATTN_ERR_UNSUPPORTED: return "unsupported (head dim 32, 64, 80, 96 or 128; page size 16; rotation of a multiple of 16 dims, at most the head dim, by at most 4 axes; device sm_103)";
        case ATTN_ERR_MISALIGNED: return "misaligned pointer (tensors need 16-byte alignment)";
        case ATTN_ERR_WORKSPACE: return "workspace missing, misaligned or smaller than the call's *_workspace_size() (paged_attn_decode_workspace_size(), attn_bwd_workspace_size() and so on)";
        case ATTN_ERR_CUDA: return "CUDA runtime error or launch failure";
        case ATTN_ERR_DEVICE_TIMEOUT: return "a bounded in-kernel wait ran out; results of the affected calls are invalid, and calls launch nothing until attn_check_device_status() clears it";
        case ATTN_ERR_SCRATCH_LIMIT: return "sizes need more decode scratch than the 12 MiB static array of paged_attn_decode_noalloc (use paged_attn_decode with a workspace)";
        default: return "unknown status";
    }
}

ATTN_API const char *attn_version(void) { return "0.1.0"; }
