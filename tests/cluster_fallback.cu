// The launches that the decode with modified scores makes where the device can, and cannot, place its clusters: run
// on the host, with fakes of the helpers and of the runtime's launch calls (--wrap), which print what they are given.
#include <cstdio>
#include <cstdlib>

#include "decode_scoremod.cu"

static bool room;
static cudaError_t pending = cudaSuccess;  // what the runtime's last error would be
namespace attn {
bool cluster_fits(const void *, int, int, size_t) { return room; }
cudaError_t ensure_large_clusters(const void *) { return pending = room ? cudaSuccess : cudaErrorInvalidValue; }
cudaError_t ensure_max_dynamic_smem(const void *, int) { return cudaSuccess; }
cudaError_t current_sm_count(int *n) { return *n = 152, cudaSuccess; }
bool encode_qkv_map(CUtensorMap *, const void *, int, int, int, int) { return true; }
bool encode_page_map_u8(CUtensorMap *, const void *, int, int, int, bool) { return true; }
size_t decode_workspace_bytes(int, int, int, int, int, int) { return 1; }
}  // namespace attn

static const attn::RowsParams &params(void **args, bool merge) {
    return *static_cast<const attn::RowsParams *>(args[merge ? 0 : 2]);
}
extern "C" cudaError_t __wrap_cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *, void **args) {
    const bool cluster = c->numAttrs == 1 && c->attrs[0].id == cudaLaunchAttributeClusterDimension;
    if (cluster && !room) return cudaErrorInvalidValue;  // as a launch would
    const attn::RowsParams &p = params(args, !cluster);
    printf("%s %u,%u,%u splits %d chunk %d cluster %d\n", cluster ? "cluster" : "dependent", c->gridDim.x, c->gridDim.y,
           c->gridDim.z, p.n_splits, p.chunk_pages, p.cluster ? 1 : 0);
    return cudaSuccess;
}
static cudaError_t plain(dim3 g, void **args) {
    const attn::RowsParams &p = params(args, false);
    printf("plain %u,%u,%u splits %d chunk %d cluster %d\n", g.x, g.y, g.z, p.n_splits, p.chunk_pages, p.cluster ? 1 : 0);
    return cudaSuccess;
}
// what <<<>>> calls (one of the two)
extern "C" cudaError_t __wrap_cudaLaunchKernel(const void *, dim3 g, dim3, void **args, size_t, cudaStream_t) {
    return plain(g, args);
}
extern "C" cudaError_t __wrap___cudaLaunchKernel(cudaKernel_t, dim3 g, dim3, void **args, size_t, cudaStream_t) {
    return plain(g, args);
}
extern "C" cudaError_t __wrap_cudaGetLastError() {
    const cudaError_t e = pending;
    pending = cudaSuccess;
    return e;
}

// room B H Hkv max_pages
int main(int, char **v) {
    room = atoi(v[1]) != 0;
    attn::DecodeMoreArgs a{};
    a.B = atoi(v[2]), a.H = atoi(v[3]), a.Hkv = atoi(v[4]), a.d = 32, a.max_pages = atoi(v[5]);
    a.num_pages = 100, a.scale = 0.1f, a.page_size = 16;
    const cudaError_t e = attn::launch_decode_scoremod(a, nullptr);
    printf("status %d\n", (int)e);
    return 0;
}
