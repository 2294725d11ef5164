// pages.cu -- page tables and reference counts of a paged cache: sequences that continue others, pages for new tokens,
// pages moved to the front of the pool; and the copies of pages that these ask for.
//
// A page's reference count is the number of table entries that name it (plus what the caller adds); a page is free iff its
// count is not positive.  Which free page goes where is fixed by the order of the rows and of the page numbers (prefix sums,
// no counters that race), so equal inputs give equal tables.  The counts' sums use integer atomics, whose order does not
// show in the result.
//
// The scans over the counts and over the rows are one cluster's work: each CTA takes an even part of the pool, the parts'
// totals are exchanged at a cluster barrier.  There is next to nothing to read and write, so the launches count: tables and
// pools of ordinary size are the work of one kernel a call, all of it by that cluster, and the kernels start while the ones
// before them drain (a fork, a reservation and the copies for 16 rows: 20.5 us in five kernels, 14.1 in three, which is the
// host's time for the three calls; a compaction of 400 pages with its copies 16.4 and 10.7).
#include "launch.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr int kPS = 16;
constexpr int kScanThreads = 1024;
constexpr int kScanCtas = 8;       // of the scanning cluster
constexpr int kScanTile = kScanThreads * 4;

__device__ __forceinline__ bool in_pool(int page, int num_pages) { return (unsigned)page < (unsigned)num_pages; }

// ---------------------------------------------------------------- fork
struct ForkParams {
    const int32_t *table, *ctx, *parents, *ref;
    int32_t *table_out, *ctx_out, *ref_out;
    int B, B_out, W, P;
};
// (Read through L2: the grid of a large table reads its inputs before it has waited itself.)
__device__ __forceinline__ int fork_entry(const ForkParams &p, int b, int c) {
    const int par = __ldcg(p.parents + b);
    if (par < 0 || par >= p.B) return -1;
    if (par != b) {
        const int n = min(max(__ldcg(p.ctx + par), 0), p.W * kPS);
        if (c >= (n + kPS - 1) / kPS) return -1;
    }
    return __ldcg(p.table + (size_t)par * p.W + c);
}
__device__ __forceinline__ void fork_lens(const ForkParams &p, long long i0, long long step) {
    for (long long i = i0; i < p.B_out; i += step) {
        const int par = __ldcg(p.parents + i);
        p.ctx_out[i] = par < 0 || par >= p.B ? 0 : __ldcg(p.ctx + par);
    }
}
// What a place of the table names now, and what it named.
__device__ __forceinline__ void fork_count(const ForkParams &p, int was, int is) {
    if (was == is) return;
    if (in_pool(was, p.P)) atomicSub(p.ref_out + was, 1);
    if (in_pool(is, p.P)) atomicAdd(p.ref_out + is, 1);
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
// One cluster: the rows, then the counts.
__global__ void __launch_bounds__(kScanThreads) pages_fork_cluster_kernel(const ForkParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const long long i0 = (long long)blockIdx.x * kScanThreads + threadIdx.x, step = (long long)gridDim.x * kScanThreads;
    const long long olds = (long long)p.B * p.W, news = (long long)p.B_out * p.W;
    for (long long i = i0; i < news; i += step) p.table_out[i] = fork_entry(p, (int)(i / p.W), (int)(i % p.W));
    for (long long i = i0; i < p.P; i += step) p.ref_out[i] = p.ref[i];
    fork_lens(p, i0, step);
    cluster_sync();
    for (long long i = i0; i < max(olds, news); i += step)
        fork_count(p, i < olds ? __ldcg(p.table + i) : -1, i < news ? __ldcg(p.table_out + i) : -1);
}
// Large tables: rows and counts by one grid, for which another has copied the counts where they are not changed in place.  That
// one lets it start when all before it has ended, so the rows are made while the counts are copied (fork, reservation and copies for
// 128 rows of 1024 entries: rows and counts by grids one after the other 27.0 us, so 25.1).
__global__ void __launch_bounds__(256) pages_fork_copy_kernel(const ForkParams p) {
    griddep_wait();
    griddep_launch_dependents();
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < p.P; i += (long long)gridDim.x * 256) p.ref_out[i] = p.ref[i];
}
__global__ void __launch_bounds__(256) pages_fork_kernel(const ForkParams p) {
    if (p.ref_out == p.ref) griddep_wait();
    griddep_launch_dependents();
    const long long i0 = (long long)blockIdx.x * 256 + threadIdx.x, step = (long long)gridDim.x * 256;
    const long long olds = (long long)p.B * p.W, news = (long long)p.B_out * p.W;
    fork_lens(p, i0, step);
    int was = -1, is = -1;
    auto entry = [&](long long i) {
        was = i < olds ? __ldcg(p.table + i) : -1;
        is = -1;
        if (i < news) p.table_out[i] = is = fork_entry(p, (int)(i / p.W), (int)(i % p.W));
    };
    entry(i0);
    griddep_wait();  // the counts are there
    for (long long i = i0; i < max(olds, news); i += step, entry(i)) fork_count(p, was, is);
}

// ---------------------------------------------------------------- scans
// Sum over the block's threads before this one, and over all of them (in `total`).
__device__ __forceinline__ int block_scan(int v, int (&warp_sums)[33], int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();  // the sums of a scan before this one have been read
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int s = warp_sums[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, off);
            if (lane >= off) s += y;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    total = warp_sums[31];
    return (warp ? warp_sums[warp - 1] : 0) + x - v;
}
// The four counts from page i on (past the end: `beyond`).
__device__ __forceinline__ int4 counts4(const int32_t *ref, int i, int end, int beyond) {
    if (i + 4 <= end) return *reinterpret_cast<const int4 *>(ref + i);
    int4 v = make_int4(beyond, beyond, beyond, beyond);
    if (i < end) v.x = ref[i];
    if (i + 1 < end) v.y = ref[i + 1];
    if (i + 2 < end) v.z = ref[i + 2];
    return v;
}
// The CTA's part [begin, end) of n pages, of which only the last may not be whole vectors.
__device__ __forceinline__ void scan_part(int n, int cta, int ctas, int &begin, int &end) {
    const long long per = ((long long)(n + ctas - 1) / ctas + 3) & ~3LL;
    begin = (int)min(per * cta, (long long)n);
    end = (int)min(per * (cta + 1), (long long)n);
}

// ---------------------------------------------------------------- reserve
struct ReserveParams {
    const int32_t *table, *ctx, *new_lens, *ref;
    int32_t *table_out, *ref_out, *reserved, *src, *dst;
    int32_t *frozen;  // a copy of the counts at the call's start, when they change in place
    int32_t *need;    // [B]
    int32_t *ids;     // [P]: free pages in order
    int32_t *parts;   // [kScanCtas]: free pages of each part
    int B, W, P, ctas, copy_table, copy_ref, copy_frozen;
    int counts_copied, table_apart;  // by a grid before; by the grid's other clusters
};
__device__ __forceinline__ void reserve_copy_counts(const ReserveParams &p, long long i0, long long step) {
    for (long long i = i0; i < p.P; i += step) {
        const int v = p.ref[i];
        if (p.copy_ref) p.ref_out[i] = v;
        if (p.copy_frozen) p.frozen[i] = v;
    }
}
__global__ void __launch_bounds__(256) pages_reserve_copy_kernel(const ReserveParams p) {
    griddep_launch_dependents();
    griddep_wait();
    reserve_copy_counts(p, (long long)blockIdx.x * 256 + threadIdx.x, (long long)gridDim.x * 256);
}
// Entries [from, to) of row b that cover its new tokens (to 0: none wanted, or more than the table holds).
__device__ __forceinline__ void reserve_range(const ReserveParams &p, int b, int &n, int &from, int &to) {
    const int add = p.new_lens[b];
    n = min(max(p.ctx[b], 0), p.W * kPS);
    const long long end = ((long long)n + add + kPS - 1) / kPS;
    from = n / kPS;
    to = add > 0 && end <= p.W ? (int)end : 0;
}
// The entries that no new token touches, of all rows: a warp takes 256 of a row.
constexpr int kCopyRun = 256;
__device__ __forceinline__ void reserve_copy_rows(const ReserveParams &p, int warp, int warps) {
    const int runs = (p.W + kCopyRun - 1) / kCopyRun, lane = threadIdx.x & 31;
    for (long long u = warp; u < (long long)p.B * runs; u += warps) {
        const int b = (int)(u / runs), c = (int)(u % runs) * kCopyRun + lane;
        int n, from, to, v[kCopyRun / 32];
        reserve_range(p, b, n, from, to);
        const int32_t *row = p.table + (size_t)b * p.W;
#pragma unroll
        for (int i = 0; i < kCopyRun / 32; ++i)
            if (c + 32 * i < p.W) v[i] = row[c + 32 * i];
#pragma unroll
        for (int i = 0; i < kCopyRun / 32; ++i)
            if (c + 32 * i < p.W && (c + 32 * i < from || c + 32 * i >= to)) p.table_out[(size_t)b * p.W + c + 32 * i] = v[i];
    }
}
// What waits on what: a row's lengths, its entries, their counts, the sums over the rows and over the pool, the free pages' ids.
// A warp's first row and a thread's first counts are read before anything waits and stay in registers, and the sums over the first
// kScanThreads rows in shared memory, so that nothing of an ordinary call is read twice.  The grid's first cluster does all but the
// copy of a large table, which is left to the others (fork, reservation and copies for 128 rows of 1024 entries: 28.8 us with that
// copy by a grid before, 27.0 so).
__global__ void __launch_bounds__(kScanThreads) pages_reserve_kernel(const ReserveParams p) {
    __shared__ int sums[33];
    __shared__ int offsets[kScanThreads];  // of a tile of rows: where their free pages begin (-1: more than there are)
    const int cta = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first_warp = cta * 32 + warp, all_warps = p.ctas * 32;
    griddep_launch_dependents();
    griddep_wait();
    if (cta >= p.ctas) {
        reserve_copy_rows(p, (cta - p.ctas) * 32 + warp, ((int)gridDim.x - p.ctas) * 32);
        return;
    }
    int begin, end, mine, total;
    scan_part(p.P, cta, p.ctas, begin, end);
    const int4 v0 = counts4(p.ref, begin + 4 * (int)threadIdx.x, end, 1);
    // an entry to be given a page: it has none, or shares it (by the counts at the call's start: the input's, which do not
    // change before the second barrier, and then its copy).  So what a row needs hangs on no other row's fate, and the rows' sums
    // are one scan; the price is one page more than needed where all that share one ask at once, free again at the next call.
    const int32_t *counts = p.ref;
    auto lacks = [&](int e) { return !in_pool(e, p.P) || __ldcg(counts + e) > 1; };
    // the first 32 entries of a row, one a lane: what they name, and which lack a page
    struct Head {
        int n, from, to, old;
        bool lack;
    };
    auto head_of = [&](int b) {
        Head r;
        reserve_range(p, b, r.n, r.from, r.to);
        r.old = r.from + lane < r.to ? p.table[(size_t)b * p.W + r.from + lane] : -1;
        return r;
    };
    auto lack_of = [&](Head &r) { r.lack = r.from + lane < r.to && lacks(r.old); };
    Head mine0{0, 0, 0, -1, false};
    if (first_warp < p.B) mine0 = head_of(first_warp);
    if (!p.counts_copied) reserve_copy_counts(p, (long long)cta * kScanThreads + threadIdx.x, (long long)p.ctas * kScanThreads);
    if (p.copy_table && !p.table_apart) reserve_copy_rows(p, first_warp, all_warps);
    if (first_warp < p.B) lack_of(mine0);
    mine = (v0.x <= 0) + (v0.y <= 0) + (v0.z <= 0) + (v0.w <= 0);
    for (int i = begin + kScanTile + 4 * (int)threadIdx.x; i < end; i += kScanTile) {
        const int4 v = counts4(p.ref, i, end, 1);
        mine += (v.x <= 0) + (v.y <= 0) + (v.z <= 0) + (v.w <= 0);
    }
    for (int b = first_warp; b < p.B; b += all_warps) {
        Head r = mine0;
        if (b != first_warp) r = head_of(b), lack_of(r);
        int need = __popc(__ballot_sync(0xffffffffu, r.lack));
        for (int c0 = r.from + 32; c0 < r.to; c0 += 32) {
            const bool lack = c0 + lane < r.to && lacks(p.table[(size_t)b * p.W + c0 + lane]);
            need += __popc(__ballot_sync(0xffffffffu, lack));
        }
        if (lane == 0) p.need[b] = need;
    }
    block_scan(mine, sums, total);
    if (threadIdx.x == 0) p.parts[cta] = total;
    cluster_sync();
    int before = 0, free_pages = 0;
    for (int i = 0; i < p.ctas; ++i) {
        const int v = __ldcg(p.parts + i);
        before += i < cta ? v : 0;
        free_pages += v;
    }
    // a tile of rows' offsets into the free pages; returns what they need together
    auto row_offsets = [&](int b0, long long base) {
        const int b = b0 + (int)threadIdx.x;
        const int need = b < p.B ? __ldcg(p.need + b) : 0;
        int sum;
        const long long off = base + block_scan(need, sums, sum);
        offsets[threadIdx.x] = need == 0 ? 0 : (off + need <= free_pages ? (int)off : -1);
        return sum;
    };
    // the free pages that are wanted at all, listed in order, each CTA those of its part
    const long long base1 = row_offsets(0, 0);  // (every CTA: of all rows)
    long long wanted = base1;
    for (int b0 = kScanThreads; b0 < p.B; b0 += kScanThreads) {
        const int b = b0 + (int)threadIdx.x;
        int sum;
        block_scan(b < p.B ? __ldcg(p.need + b) : 0, sums, sum);
        wanted += sum;
    }
    const int last = (int)min(wanted, (long long)free_pages);
    for (int i0 = begin; i0 < end && before < last; i0 += kScanTile) {
        const int i = i0 + 4 * (int)threadIdx.x;
        const int4 v = i0 == begin ? v0 : counts4(p.ref, i, end, 1);
        const bool f[4] = {v.x <= 0, v.y <= 0, v.z <= 0, v.w <= 0};
        int at = before + block_scan(f[0] + f[1] + f[2] + f[3], sums, total);
        before += total;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (f[j]) p.ids[at++] = i + j;
    }
    cluster_sync();
    if (p.copy_frozen) counts = p.frozen;
    // rows, a tile of kScanThreads at a time, a warp each
    long long base = 0;
    for (int b0 = 0; b0 < p.B; b0 += kScanThreads) {
        if (b0 > 0) {
            __syncthreads();  // the last tile's offsets have been read
            base += b0 == kScanThreads ? base1 : 0;
            base += row_offsets(b0, base);
            __syncthreads();
        }
        const int skip = (first_warp - b0 % all_warps + all_warps) % all_warps;  // (b mod all_warps is the warp, as above)
        for (int b = b0 + skip; b < min(b0 + kScanThreads, p.B); b += all_warps) {
            Head r = mine0;
            if (b != first_warp) r = head_of(b), lack_of(r);
            const int off = offsets[b - b0];
            const bool served = r.to > 0 && off >= 0;
            int src = -1, dst = -1, taken = 0;
            for (int c0 = r.from; c0 < r.to; c0 += 32) {
                const int c = c0 + lane;
                int old = r.old;
                bool lack = r.lack;
                if (c0 > r.from) {
                    old = c < r.to ? p.table[(size_t)b * p.W + c] : -1;
                    lack = c < r.to && lacks(old);
                }
                lack = lack && served;
                if (p.copy_table && c < r.to && !lack) p.table_out[(size_t)b * p.W + c] = old;
                const unsigned mask = __ballot_sync(0xffffffffu, lack);
                if (lack) {
                    const int page = __ldcg(p.ids + off + taken + __popc(mask & ((1u << lane) - 1)));
                    p.table_out[(size_t)b * p.W + c] = page;
                    p.ref_out[page] = 1;
                    if (in_pool(old, p.P)) {
                        atomicSub(p.ref_out + old, 1);
                        if (c == r.from && r.n % kPS != 0) src = old, dst = page;  // (lane 0: its tokens move along)
                    }
                }
                taken += __popc(mask);
            }
            if (lane == 0) {
                p.reserved[b] = served ? p.new_lens[b] : 0;
                p.src[b] = src;
                p.dst[b] = dst;
            }
        }
    }
}

// ---------------------------------------------------------------- compact
struct CompactParams {
    const int32_t *table, *ref;
    int32_t *table_out, *ref_out, *src, *dst, *count;
    int32_t *to;     // [P]: where a page goes (-1: it is not live)
    int32_t *back;   // [P]: the pages that move, the last one first
    int32_t *parts;  // [2 kScanCtas]
    int B, W, P, ctas, rename;  // rename: the table too
};
__device__ __forceinline__ void rename_entries(const CompactParams &p, long long i0, long long step) {
    for (long long i = i0; i < (long long)p.B * p.W; i += step) {
        const int e = p.table[i];
        p.table_out[i] = in_pool(e, p.P) ? __ldcg(p.to + e) : -1;
    }
}
__global__ void __launch_bounds__(kScanThreads) pages_compact_kernel(const CompactParams p) {
    __shared__ int sums[33];
    const int cta = blockIdx.x;
    griddep_launch_dependents();
    griddep_wait();
    int begin, end, total;
    scan_part(p.P, cta, p.ctas, begin, end);
    const int4 v0 = counts4(p.ref, begin + 4 * (int)threadIdx.x, end, 0);
    int mine = (v0.x > 0) + (v0.y > 0) + (v0.z > 0) + (v0.w > 0);
    for (int i = begin + kScanTile + 4 * (int)threadIdx.x; i < end; i += kScanTile) {
        const int4 v = counts4(p.ref, i, end, 0);
        mine += (v.x > 0) + (v.y > 0) + (v.z > 0) + (v.w > 0);
    }
    block_scan(mine, sums, total);
    if (threadIdx.x == 0) p.parts[cta] = total;
    cluster_sync();
    int before = 0, live = 0;  // live pages of the parts before, and of all
    for (int i = 0; i < p.ctas; ++i) {
        const int v = __ldcg(p.parts + i);
        before += i < cta ? v : 0;
        live += v;
    }
    // `stay` live pages lie below `live`; the others are `moves`, known after the next barrier, so those are listed from the last
    // one, in `back`, and the holes from the first
    int stays = 0;
    for (int i0 = begin; i0 < end; i0 += kScanTile) {
        const int i = i0 + 4 * (int)threadIdx.x;
        const int4 v = i0 == begin ? v0 : counts4(p.ref, i, end, 0);
        const int c[4] = {v.x, v.y, v.z, v.w};
        int at = before + block_scan((c[0] > 0) + (c[1] > 0) + (c[2] > 0) + (c[3] > 0), sums, total);  // live before i + j
        before += total;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int page = i + j;
            if (page >= end) break;
            if (page < live) {
                p.to[page] = c[j] > 0 ? page : -1;
                if (c[j] > 0) p.ref_out[page] = c[j], ++stays;
                else p.dst[page - at] = page;  // the holes, in order
            } else {
                p.ref_out[page] = 0;
                if (c[j] > 0) p.back[live - 1 - at] = page;
                else p.to[page] = -1;
            }
            at += c[j] > 0;
        }
    }
    block_scan(stays, sums, total);
    if (threadIdx.x == 0) p.parts[kScanCtas + cta] = total;
    cluster_sync();
    int moves = live;
    for (int i = 0; i < p.ctas; ++i) moves -= __ldcg(p.parts + kScanCtas + i);
    if (cta == 0 && threadIdx.x == 0) *p.count = moves;
    for (int i = cta * kScanThreads + (int)threadIdx.x; i < p.P; i += p.ctas * kScanThreads) {
        int s = -1;
        if (i < moves) {  // the pages that fill the holes, in order
            s = __ldcg(p.back + moves - 1 - i);
            const int d = __ldcg(p.dst + i);
            p.to[s] = d;
            p.ref_out[d] = p.ref[s];
        } else {
            p.dst[i] = -1;
        }
        p.src[i] = s;
    }
    if (!p.rename) return;
    cluster_sync();
    rename_entries(p, (long long)cta * kScanThreads + threadIdx.x, (long long)p.ctas * kScanThreads);
}
__global__ void __launch_bounds__(256) pages_compact_table_kernel(const CompactParams p) {
    griddep_launch_dependents();
    griddep_wait();
    rename_entries(p, (long long)blockIdx.x * 256 + threadIdx.x, (long long)gridDim.x * 256);
}

// ---------------------------------------------------------------- copies
// Bound by memory: 3930 pages of 32 KB in four pools take 155 us of the 178 with the compaction (6.6 TB/s read and written).
constexpr int kCopyPools = 256;  // pools of one launch
constexpr int kCopyChunk = 16384;  // bytes a block moves at a time

struct CopyParams {
    const int32_t *src, *dst, *count;  // count may be null
    size_t page_bytes;
    int n, num_pages, n_pools, chunks;
    uint8_t *pools[kCopyPools];
};
__global__ void __launch_bounds__(256) pages_copy_kernel(const __grid_constant__ CopyParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int n = p.count ? min(max(*p.count, 0), p.n) : p.n;
    const long long per_pair = (long long)p.n_pools * p.chunks, units = n * per_pair;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int i = (int)(u / per_pair), r = (int)(u % per_pair);
        const int src = p.src[i], dst = p.dst[i];
        if (!in_pool(src, p.num_pages) || !in_pool(dst, p.num_pages)) continue;
        const size_t from = (size_t)(r % p.chunks) * kCopyChunk;
        const int vectors = (int)(min((size_t)kCopyChunk, p.page_bytes - from) / 16);
        uint8_t *pool = p.pools[r / p.chunks];
        const uint4 *s = reinterpret_cast<const uint4 *>(pool + src * p.page_bytes + from);
        uint4 *d = reinterpret_cast<uint4 *>(pool + dst * p.page_bytes + from);
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if ((int)threadIdx.x + 256 * k < vectors) v[k] = s[threadIdx.x + 256 * k];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if ((int)threadIdx.x + 256 * k < vectors) d[threadIdx.x + 256 * k] = v[k];
    }
}

// Blocks of 256 threads for `work` items, at most `waves` on every SM.
int blocks_for(long long work, int waves) {
    int sms = 0;
    if (current_sm_count(&sms) != cudaSuccess || sms <= 0) sms = 1;
    const long long want = (work + 255) / 256, most = (long long)sms * waves;
    return (int)(want < 1 ? 1 : (want < most ? want : most));
}
// CTAs of the scanning cluster: one where it passes over the pool, and what else it reads and writes, in one step, or where
// the device (a part of a GPU) cannot place more.  Calls one after the other, us, one CTA / eight; entries and pages alike:
//             256           1024          2048          4096          8192
//   fork      3.6 / 3.5     4.2 / 4.2     5.4 / 4.1     7.6 / 4.3    12.6 / 4.3
//   reserve   7.1 / 7.6     7.1 / 7.6     7.1 / 7.3     9.0 / 8.4    12.4 / 8.5
//   compact   6.5 / 7.2     6.5 / 7.3     8.1 / 7.6    10.8 / 7.8    16.7 / 8.2
constexpr int kOneCta = 1024;
template <class K>
int scan_ctas(K kernel, long long items) {
    return items <= kOneCta || !cluster_fits(reinterpret_cast<const void *>(kernel), kScanCtas, kScanThreads, 0) ? 1 : kScanCtas;
}
// Table entries and pages that the cluster reads and writes itself; more take a grid of their own (the reservation's table: more
// clusters).  As above, all by the cluster of eight / the large steps apart:
//             2048          4096          8192          16384         32768         65536
//   fork      4.1 / 4.4     4.3 / 4.4     4.3 / 4.2     5.9 / 4.3     8.2 / 4.4    13.8 / 4.2
//   reserve   7.3 / 8.0     8.4 / 9.1     8.5 / 9.1     9.1 / 9.4     9.5 / 9.3    10.6 / 9.8
//   compact   7.6 / 8.1     7.8 / 8.2     8.2 / 8.5     9.0 / 8.7    11.5 / 10.2   18.0 / 15.3
constexpr long long kClusterItems = 1 << 13, kReserveItems = 1 << 15;

// A kernel of one cluster, or several, of `ctas` CTAs.
template <class K, class A>
cudaError_t launch_scan(K kernel, const A &p, int ctas, int clusters, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas * clusters);
    cfg.blockDim = dim3(kScanThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

size_t ints(size_t n) { return (n * sizeof(int32_t) + 15) & ~size_t(15); }

}  // namespace

cudaError_t launch_pages_fork(const PagesArgs &a, cudaStream_t stream) {
    const ForkParams p{a.page_table, a.ctx_lens, a.parents, a.ref_counts, a.page_table_out, a.ctx_lens_out,
                       a.ref_counts_out, a.B, a.B_out, a.max_pages, a.num_pages};
    const long long all = (long long)(a.B > a.B_out ? a.B : a.B_out) * a.max_pages, items = all > a.num_pages ? all : a.num_pages;
    if (items <= kClusterItems) return launch_scan(pages_fork_cluster_kernel, p, scan_ctas(pages_fork_cluster_kernel, items), 1, stream);
    if (p.ref_out != p.ref) {
        const cudaError_t e = launch_dependent(pages_fork_copy_kernel, dim3(blocks_for(a.num_pages, 8)), 256, 0, stream, p);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(pages_fork_kernel, dim3(blocks_for(all, 8)), 256, 0, stream, p);
}

size_t pages_reserve_workspace_bytes(int B, int num_pages) {
    return B <= 0 || num_pages <= 0 ? 0 : ints(B) + 2 * ints(num_pages) + ints(kScanCtas);
}
cudaError_t launch_pages_reserve(const PagesArgs &a, cudaStream_t stream) {
    ReserveParams p{};
    p.table = a.page_table;
    p.ctx = a.ctx_lens;
    p.new_lens = a.new_lens;
    p.ref = a.ref_counts;
    p.table_out = a.page_table_out;
    p.ref_out = a.ref_counts_out;
    p.reserved = a.reserved;
    p.src = a.src;
    p.dst = a.dst;
    char *ws = static_cast<char *>(a.workspace);
    p.need = reinterpret_cast<int32_t *>(ws);
    p.ids = reinterpret_cast<int32_t *>(ws += ints(a.B));
    p.copy_table = a.page_table_out != a.page_table;
    p.copy_ref = a.ref_counts_out != a.ref_counts;
    p.copy_frozen = !p.copy_ref;
    p.frozen = reinterpret_cast<int32_t *>(ws + ints(a.num_pages));
    p.parts = reinterpret_cast<int32_t *>(ws + 2 * ints(a.num_pages));
    p.B = a.B;
    p.W = a.max_pages;
    p.P = a.num_pages;
    const long long cells = p.copy_table ? (long long)a.B * a.max_pages : 0;
    p.table_apart = cells > kReserveItems;
    p.counts_copied = a.num_pages > kReserveItems;
    p.ctas = scan_ctas(pages_reserve_kernel, cells > a.num_pages ? cells : a.num_pages);
    if (p.counts_copied) {
        const cudaError_t e = launch_dependent(pages_reserve_copy_kernel, dim3(blocks_for(a.num_pages, 8)), 256, 0, stream, p);
        if (e != cudaSuccess) return e;
    }
    int clusters = 1;
    if (p.table_apart) {  // a run a warp, on at most 16 more clusters
        const long long runs = (long long)a.B * ((a.max_pages + kCopyRun - 1) / kCopyRun), want = (runs + 32 * p.ctas - 1) / (32 * p.ctas);
        clusters += (int)(want < 16 ? want : 16);
    }
    return launch_scan(pages_reserve_kernel, p, p.ctas, clusters, stream);
}

size_t pages_compact_workspace_bytes(int num_pages) {
    return num_pages <= 0 ? 0 : 2 * ints(num_pages) + ints(2 * kScanCtas);
}
cudaError_t launch_pages_compact(const PagesArgs &a, cudaStream_t stream) {
    const long long cells = (long long)a.B * a.max_pages, items = cells > a.num_pages ? cells : a.num_pages;
    char *ws = static_cast<char *>(a.workspace);
    const CompactParams p{a.page_table, a.ref_counts, a.page_table_out, a.ref_counts_out, a.src, a.dst, a.count,
                          reinterpret_cast<int32_t *>(ws), reinterpret_cast<int32_t *>(ws + ints(a.num_pages)),
                          reinterpret_cast<int32_t *>(ws + 2 * ints(a.num_pages)),
                          a.B, a.max_pages, a.num_pages, scan_ctas(pages_compact_kernel, items), cells <= kClusterItems};
    const cudaError_t e = launch_scan(pages_compact_kernel, p, p.ctas, 1, stream);
    if (e != cudaSuccess || p.rename) return e;
    return launch_dependent(pages_compact_table_kernel, dim3(blocks_for(cells, 8)), 256, 0, stream, p);
}

cudaError_t launch_pages_copy(void *const *pools, int n_pools, size_t page_bytes, const int32_t *src, const int32_t *dst,
                              const int32_t *count, int n, int num_pages, cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = current_sm_count(&sms);
    if (e != cudaSuccess) return e;
    for (int first = 0; first < n_pools; first += kCopyPools) {
        CopyParams p;
        p.src = src;
        p.dst = dst;
        p.count = count;
        p.page_bytes = page_bytes;
        p.n = n;
        p.num_pages = num_pages;
        p.n_pools = n_pools - first < kCopyPools ? n_pools - first : kCopyPools;
        p.chunks = (int)((page_bytes + kCopyChunk - 1) / kCopyChunk);
        for (int i = 0; i < kCopyPools; ++i) p.pools[i] = i < p.n_pools ? static_cast<uint8_t *>(pools[first + i]) : nullptr;
        const long long units = (long long)n * p.n_pools * p.chunks, most = (long long)sms * 8;
        e = launch_dependent(pages_copy_kernel, dim3((unsigned)(units < most ? units : most)), 256, 0, stream, p);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace attn
