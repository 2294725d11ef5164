// decode_fp4.cu -- paged decode over the 4-bit cache (fp4.cuh), with the modified scores of decode_scoremod.cu.
//
// The rows kernel's products (decode_rows.cuh: tokens as the rows, query heads as the columns), over pages of 9 d bytes a
// head that come by one bulk copy each:
//   S^T = K Q^T        a lane's codes of a token are neighbours in its row: 32 (d 128) or 16 dims, one or two blocks of the
//                     scales, read as one vector, and Q is held in that order of the dims;
//   O^T += V^T P^T    a block of 16 dims is one 8 x 8 matrix of ldmatrix, transposed: a lane gets four bytes, dims 2g and
//                     2g + 1 of token pairs (2t, 2t + 1) and (2t + 8, 2t + 9), the four registers of one operand.
// A byte of codes widens to one f16x2 register in one instruction and a product with the pair of block scales makes it the
// value (exact).  The scales of slots that are not seen are zeroed, so whatever they hold adds nothing.
//
// What the time goes by (32/8 heads, d 128, replayed graphs): 32 sequences of one length, 2048 / 4096 / 8192 / 16384 / 32768 tokens,
// take 23.6 / 34.9 / 57.9 / 104.8 / 198.2 us, which is 6.4 to 6.6 TB/s for every further byte, near a copy's rate, and 11 to 12 us at
// no bytes at all: the launch, then in a row the lengths of all sequences, the search for the share, page ids, the first pages, and
// the joining kernel.  (One sequence of 16384 to 262144: the same rate, and 10 to 11 us.)  A warp issues about 260 instructions a page
// (d 128), of which the widening takes 82 and the products with the scales 64, and it takes two pages at a step, which share the
// waiting, the vote on the maxima and the copies' issue.
//
// The pages of all rows (a sequence's heads that one CTA takes) are shared out over the CTAs that fit the GPU, by the lengths
// on the device: a CTA's share begins and ends anywhere in a row, rows that it has whole it writes itself, and the others'
// parts, two a CTA at most, are joined by a second kernel.  So uneven lengths cost nothing, and of the page table's width nothing is
// read that holds no token.  A small batch takes one cluster per row instead, which joins its CTAs' parts itself; the host
// chooses by the table's width, so short sequences in a wide table pay for the shares' start and join: 2 of up to 900, 12 heads of
// 64, with a distance bias, 5.6 us in a table of up to 1024 pages, 9.3 in a wider one (calls one after the other 6.1 and 11.3).
// Measured (32/8 heads, d 128): 64 sequences of up to 16000 tokens 116 us (5.6 TB/s), 32 of up to 8192 38.3 us (4.0 TB/s; 51
// with splits of the table's width), one of 103000 29.9 us (56).  More than 8 heads a group (a form that spills at d 128): 32 of
// up to 8192 over 8 key/value heads, 4 / 8 / 16 heads a group 38.0 / 40.6 / 71.0 us, with a cap 39.5 / 43.6 / 80.3; d 64, 8 / 16 25.1 / 35.2.
#include <type_traits>

#include "decode_rows.cuh"
#include "fp4.cuh"

namespace attn {
namespace {

constexpr int kFp4Slots = 2;  // steps in flight per warp
constexpr int kStep = 2;      // pages of a step (one: 47 -> 49 us on 32 sequences of up to 8192 tokens, 32/8 heads, d 128)
constexpr int kFp4Threads = kRowWarps * 32;

struct Fp4Params : RowsParams {
    int2 *row_ctas;  // [B, rows of a sequence]: the CTAs with a row's first and last page
};

// CTAs per SM, by registers (128 a thread for up to 8 heads, 168 for 16) and shared memory.  (Five of one page a step: 64 us.)  At
// d 128 the form of 16 heads spills under its 168: 268 bytes stored and 300 loaded (plain), 276 and 336 (modified); that of 8 heads 12 and 20.
template <int NT> constexpr int kFp4Ctas = NT == 1 ? 4 : 3;

// A CTA's part of a row.
struct Segment {
    int b, y, p0, p1, n;  // pages [p0, p1) of the n that its query sees
    int lo, hi, end;      // of their tokens it sees lo <= t < end, of the row's t < hi
    bool from_start, to_end;
};

template <int D, int NT>
struct Fp4Smem {
    alignas(128) uint8_t kv[kRowWarps][kFp4Slots][kStep][2][9 * D];
    RowsRed<D, NT> red;  // (not over the ring: the next row's pages arrive while this one's parts are joined)
    uint64_t full[kRowWarps][kFp4Slots];
    Segment seg[2];  // the part of a row that the CTA is at, and the next one
    int abort_flag;
};

// The dims of a lane's k-steps.  A row is cut into units of W dims, of which lane t takes W / 4 neighbours, 4 a k-step:
// one unit of 128, or units of 64 and one of the rest.
template <int D> constexpr int fp4_unit(int ks) { return D == 128 ? 128 : (D - ks / 4 * 64 >= 64 ? 64 : D % 64); }
template <int D> constexpr int fp4_base(int ks) { return D == 128 ? 0 : ks / 4 * 64; }
template <int D> constexpr int fp4_step(int ks) { return D == 128 ? ks : ks % 4; }

// A sequence's tokens lo <= t < hi that its query sees, on pages [p0, p1) of its row of the table.
__device__ __forceinline__ PageRange seen_pages(const RowsParams &a, int b) {
    PageRange r;
    r.hi = min(max(a.ctx_lens[b], 0), a.max_pages * kRowPS);
    r.lo = a.key_begin ? min(max(a.key_begin[b], 0), r.hi) : 0;
    r.p0 = r.lo / kRowPS;
    r.p1 = r.lo < r.hi ? (r.hi + kRowPS - 1) / kRowPS : r.p0;
    return r;
}
// Shares: a row of n pages counts as n + kRowCost (what its query's read, its end and its part's way through the workspace
// take, in pages), and a share takes the pages that lie between two marks, kLeast units apart at least.  kRowCost 4 / 8 / 16:
// 128 sequences of up to 110 tokens, 12 heads of 64, 20.5 / 18.5 / 16.4 us, of 1000 tokens 36.0 / 32.8 / 30.5; 32 of up to 8192,
// 32/8 heads of 128, 38.9 / 38.5 / 37.7.
constexpr int kRowCost = 16;
constexpr int kLeast = kRowWarps * kStep + kRowCost;

// The part of row y of sequence b from unit u0 of its cost on, of at most `left` units, which go down by what it takes.
__device__ __forceinline__ Segment segment_of(const PageRange &r, int b, int y, int u0, long long &left) {
    const int n = r.p1 - r.p0;
    const int u1 = (int)min((long long)(n + kRowCost), u0 + left);
    left -= u1 - u0;
    Segment s;
    s.b = b;
    s.y = y;
    s.lo = r.lo;
    s.hi = r.hi;
    s.n = n;
    s.p0 = r.p0 + max(0, u0 - kRowCost);
    s.p1 = r.p0 + max(0, u1 - kRowCost);
    s.end = min(r.hi, s.p1 * kRowPS);
    s.from_start = s.p0 == r.p0;
    s.to_end = s.p1 == r.p1;
    return s;
}
__device__ __forceinline__ long long cost_of(const PageRange &r) { return r.p0 < r.p1 ? r.p1 - r.p0 + kRowCost : 0; }

// Where share i of `shares` begins.  A full grid's CTAs i, i + 152, .. sit on one SM, whose schedulers let the ones that came
// first go ahead: with even shares they end after 92, 96, 101 and 108 us (64 sequences of up to 16000 tokens), so the first get
// more (97, 98, 101, 103).
constexpr int kSms = 152;
template <int NT>
__device__ __forceinline__ long long share_begin(long long total, int shares, int i) {
    constexpr int kCtas = kFp4Ctas<NT>, kUnits = 1024 * kCtas;  // weights of the CTAs of an SM, in 1024ths of an even share
    constexpr int kW[4] = {kCtas == 4 ? 1106 : 1070, kCtas == 4 ? 1060 : 1020, kCtas == 4 ? 1005 : 982, 925};
    if (shares < kSms * kCtas) return (long long)((unsigned)total * (unsigned)i / (unsigned)shares);  // (few pages)
    constexpr int kMarks = kUnits * kSms;
    const int at = i / kSms;
    int before = 0, w = 0;
#pragma unroll
    for (int c = 0; c < kCtas; ++c) {
        before += c < at ? kW[c] : 0;
        w = c == at ? kW[c] : w;
    }
    const int mark = before * kSms + w * (i - at * kSms);
    const long long q = total / kMarks;
    return q * mark + (total - q * kMarks) * mark / kMarks;
}

// The first part of share blockIdx.x of all rows, by one warp, and what is left of the share after it (false: no share).
template <int NT>
__device__ __forceinline__ bool first_segment(const RowsParams &a, Segment &s, long long &left) {
    const int lane = threadIdx.x & 31, R = a.Hkv * a.rgroups;
    const int per = (a.B + 31) / 32, b0 = min(lane * per, a.B), b1 = min(b0 + per, a.B);
    long long mine = 0;
#pragma unroll 8
    for (int b = b0; b < b1; ++b) mine += cost_of(seen_pages(a, b));
    long long upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += y;
    }
    const long long total = __shfl_sync(0xffffffffu, upto, 31) * R;
    const long long most = (total + kLeast - 1) / kLeast;
    const int shares = most < (int)gridDim.x ? (int)most : (int)gridDim.x;
    if ((int)blockIdx.x >= shares) return false;
    const long long x0 = share_begin<NT>(total, shares, blockIdx.x);
    left = share_begin<NT>(total, shares, blockIdx.x + 1) - x0;
    // the lane whose sequences hold x0 finds its sequence and row
    if (x0 >= (upto - mine) * R && x0 < upto * R) {
        long long off = x0 - (upto - mine) * R;
        int b = b0;
        PageRange r = seen_pages(a, b);
        for (long long n; off >= (n = cost_of(r) * R); off -= n) r = seen_pages(a, ++b);
        const int cost = (int)cost_of(r);
        const int y = off < (1ll << 32) ? (int)((unsigned)off / (unsigned)cost) : (int)(off / cost);
        s = segment_of(r, b, y, (int)(off - (long long)y * cost), left);
        return true;
    }
    return false;
}
// The part after s (b -1: the share ends there).
__device__ __forceinline__ Segment next_segment(const RowsParams &a, const Segment &s, long long &left) {
    int b = s.b, y = s.y + 1;
    PageRange r;
    if (left <= 0) {
        Segment none = s;
        none.b = -1;
        return none;
    }
    if (y == a.Hkv * a.rgroups) {
        y = 0;
        do r = seen_pages(a, ++b);
        while (r.p0 == r.p1);
    } else {
        r = seen_pages(a, b);
    }
    return segment_of(r, b, y, 0, left);
}

// The CTA's state of a part of a row: its warps' states joined, thread = four columns of a head, and written as a part or,
// where the CTA had the whole row, as its result.
template <int D, int NT>
__device__ __forceinline__ void write_part(RowsRed<D, NT> &red, const float (&o)[NT][D / 16][4], const float (&m_ref)[NT][2],
                                           const float (&l)[NT][2], const RowsParams &a, int rows, size_t row, float *part,
                                           bool whole) {
    constexpr int KS = D / 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 8 * nt + 2 * t + j;
            float ls = l[nt][j];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, off);
            if (g == 0) {
                // (a sum of NaN counts as seen, so that a query with NaN gives NaN)
                red.m[warp][r] = ls == ls ? m_ref[nt][j] : 0.f;
                red.l[warp][r] = ls;
            }
            if (r < rows) {
#pragma unroll
                for (int nd = 0; nd < KS; ++nd)  // rows g, g + 8 of the tile are dims 2g, 2g + 1
                    *reinterpret_cast<float2 *>(&red.o[warp][r][16 * nd + 2 * g]) = make_float2(o[nt][nd][j], o[nt][nd][j + 2]);
            }
        }
    __syncthreads();
    for (int e = threadIdx.x; e < rows * (D / 4); e += kFp4Threads) {
        const int r = e / (D / 4), x = e % (D / 4) * 4;
        const float M = fmaxf(fmaxf(red.m[0][r], red.m[1][r]), fmaxf(red.m[2][r], red.m[3][r]));
        float L = 0.f;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
        if (M != -INFINITY) {
#pragma unroll
            for (int w = 0; w < kRowWarps; ++w) {
                const float wt = ex2_approx(red.m[w][r] - M);
                const float4 v = *reinterpret_cast<const float4 *>(&red.o[w][r][x]);
                L = fmaf(red.l[w][r], wt, L);
                O.x = fmaf(v.x, wt, O.x);
                O.y = fmaf(v.y, wt, O.y);
                O.z = fmaf(v.z, wt, O.z);
                O.w = fmaf(v.w, wt, O.w);
            }
        }
        if (whole) {
            const bool any = L != 0.f;
            const OverSum over(a.v_scale, L, any);
            *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(a.o) + (row + r) * D + x) =
                make_uint2(pack_bf16x2(over(O.x), over(O.y)), pack_bf16x2(over(O.z), over(O.w)));
            if (x == 0 && a.lse) a.lse[row + r] = any ? kRowLn2 * (M + __log2f(L)) : -INFINITY;
        } else {
            *reinterpret_cast<float4 *>(part + (size_t)r * (D + 4) + x) = O;
            if (x == 0) *reinterpret_cast<float2 *>(part + (size_t)r * (D + 4) + D) = make_float2(M, L);
        }
    }
}

template <int D, int NT, bool MOD>
__global__ void __launch_bounds__(kFp4Threads, kFp4Ctas<NT>)
    decode_fp4_kernel(const uint8_t *__restrict__ k_pages, const uint8_t *__restrict__ v_pages, const Fp4Params a) {
    constexpr int kSl = kFp4Slots;
    constexpr uint32_t kBlock = 9 * D;
    constexpr int KS = D / 16;  // k-steps of S^T, and 16-dim tiles of O^T
    // A weight is 2^(score - reference), of which the reference moves when a score passes the last maximum by kThresh.  It lies
    // kLift under that maximum, so that the weights fill f16's range (at most 2^15) and those from 2^-21 of the largest on keep 11
    // bits: the values are often exactly 0 in 4 bits, and then a result is a sum over small weights alone.  Scores in the log2
    // domain are lifted up to kLifted, where the reference still has its bits; plain scores have the maximum taken off before
    // they come to that domain, so that no rounding of a large product is left in the exponent (one packed addition a pair of scores:
    // 32 sequences of up to 8192 tokens 38.0 -> 38.2 us).
    constexpr float kThresh = 8.0f, kLift = 7.0f, kLifted = 1048576.f;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    using Smem = Fp4Smem<D, NT>;
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int R = a.Hkv * a.rgroups;  // rows of a sequence

    if (threadIdx.x == 0) {
        for (int w = 0; w < kRowWarps; ++w)
            for (int s = 0; s < kSl; ++s) mbar_init(&sm.full[w][s], 1);
        sm.abort_flag = 0;
        fence_mbar_init();
    }

    griddep_launch_dependents();  // the joining kernel's CTAs come as this one's leave
    if (a.cluster) griddep_wait();  // as this one's may come as those of the kernel before leave
    long long left = 0;  // of the share, in units, after the segment that was found last (of the thread that finds them)
    if (a.cluster) {
        if (threadIdx.x == 0) {
            const PageRange r = seen_pages(a, blockIdx.z);
            const unsigned n = r.p1 - r.p0;  // (at most 2^26 pages, and 16 splits)
            Segment s;
            s.b = blockIdx.z;
            s.y = blockIdx.y;
            s.n = (int)n;
            s.p0 = r.p0 + (int)(n * blockIdx.x / (unsigned)a.n_splits);
            s.p1 = r.p0 + (int)(n * (blockIdx.x + 1) / (unsigned)a.n_splits);
            s.lo = r.lo;
            s.hi = r.hi;
            s.end = min(r.hi, s.p1 * kRowPS);
            s.from_start = s.to_end = false;
            sm.seg[0] = s;
        }
    } else if (warp == 0) {
        Segment s;
        const uint32_t found = __ballot_sync(0xffffffffu, first_segment<NT>(a, s, left));
        if (found) {
            if (lane == __ffs(found) - 1) sm.seg[0] = s;
            left = __shfl_sync(0xffffffffu, left, __ffs(found) - 1);
        } else if (lane == 0) {
            sm.seg[0].b = -1;
        }
    }
    __syncthreads();
    if (sm.seg[0].b < 0) return;
    int cur = 0;
    WaitCtx wc{&sm.abort_flag, a.status};

    // A warp takes a quarter of the segment's pages, [w0, w1), kStep of them a step.  Their ids are read 32 at a time, one a lane;
    // which of them do not lie in the pool (and hold no token) is kept for two such blocks, the one that is read and the one that
    // is issued.  Of a step's pages lane 2 j copies page j's keys into the ring, lane 2 j + 1 its values.
    constexpr int kIds = 32 / kStep;
    int my_pid = -1;
    uint32_t gaps[2] = {0, 0}, sent = 0, done = 0;  // sent, done: steps of this warp's ring that were issued, and consumed
    int w0 = 0, w1 = 0;
    auto quarter = [&] {
        const int p0 = sm.seg[cur].p0, n = sm.seg[cur].p1 - p0;
        const int unit = n < 4 * kRowWarps * kStep ? 1 : kStep;  // (whole steps where there are several)
        const int units = (n + unit - 1) / unit;  // (at most 2^26)
        w0 = p0 + unit * (units * warp / kRowWarps);
        w1 = min(p0 + unit * (units * (warp + 1) / kRowWarps), p0 + n);
        my_pid = w0 + lane < w1 ? a.page_table[(size_t)sm.seg[cur].b * a.max_pages + w0 + lane] : -1;  // the first ids
        return (w1 - w0 + kStep - 1) / kStep;
    };
    const uint8_t *const my_pages = (lane & 1) ? v_pages : k_pages;
    auto issue = [&](int kvh, int k) {
        if (k % kIds == 0) {
            const int p = w0 + kStep * k + lane;
            if (k > 0) my_pid = p < w1 ? a.page_table[(size_t)sm.seg[cur].b * a.max_pages + p] : -1;
            const uint32_t gap = __ballot_sync(0xffffffffu, p < w1 && (unsigned)my_pid >= (unsigned)a.num_pages);
            if ((k / kIds) & 1) gaps[1] = gap;
            else gaps[0] = gap;
        }
        const int pid = __shfl_sync(0xffffffffu, my_pid, kStep * (k % kIds) + ((lane >> 1) % kStep));
        const bool copies = lane < 2 * kStep && (unsigned)pid < (unsigned)a.num_pages;
        const uint32_t n = __popc(__ballot_sync(0xffffffffu, copies));
        uint64_t *bar = &sm.full[warp][sent % kSl];
        if (lane == 0) mbar_arrive_expect_tx(bar, n * kBlock);
        if (copies)
            bulk_load(sm.kv[warp][sent % kSl][lane >> 1][lane & 1],
                      my_pages + ((size_t)pid * a.Hkv + kvh) * kBlock, kBlock, bar);
        ++sent;
    };

    // Q as B fragments in the order of the codes: raw from load_q on, as f16 once the last row's products are done
    uint32_t qb[NT][KS][2];
    auto load_q = [&](int kvh) {
        const Segment &s = sm.seg[cur];
        const int row0 = (s.y - kvh * a.rgroups) * 8 * NT;
        const __nv_bfloat16 *q = reinterpret_cast<const __nv_bfloat16 *>(a.q) + ((size_t)s.b * a.H + kvh * a.group + row0) * D;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int x = fp4_base<D>(ks) + fp4_unit<D>(ks) / 4 * t + 4 * fp4_step<D>(ks);
                const uint2 u = 8 * nt + g < min(8 * NT, a.group - row0)
                                    ? *reinterpret_cast<const uint2 *>(q + (size_t)(8 * nt + g) * D + x) : make_uint2(0u, 0u);
                qb[nt][ks][0] = u.x;
                qb[nt][ks][1] = u.y;
            }
    };

    int kvh = sm.seg[0].y / a.rgroups, nk = quarter();
    load_q(kvh);
    for (int k = 0; k < min(nk, kSl); ++k) issue(kvh, k);
    bool failed = false;  // a wait ran out: this warp copies and reads nothing more, and only takes part in the barriers
    while (true) {
        // (the next part of the share is found meanwhile)
        if (threadIdx.x == 0 && !a.cluster) sm.seg[cur ^ 1] = next_segment(a, sm.seg[cur], left);
        const int lo = sm.seg[cur].lo, end = min(sm.seg[cur].end, w1 * kRowPS);
        // each head rounded to f16 after a 2^-sh of its own (query_shift); cc: per score column (heads 2t, 2t + 1 of an n-tile) the
        // factor of its products, to the cap's argument or, without a cap, to the log2 domain
        float cc[NT][2];
        {
            const float c = MOD && a.cap_in > 0.f ? a.cap_in : a.c;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float amax = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(qb[nt][ks][i] << 16)),
                                                 fabsf(__uint_as_float(qb[nt][ks][i] & 0xffff0000u))));
#pragma unroll
                for (int off = 1; off <= 2; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
                const int sh = query_shift(amax, a.q_low);
                const float f = __uint_as_float((uint32_t)(127 - sh) << 23), back = __uint_as_float((uint32_t)(127 + sh) << 23);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        qb[nt][ks][i] = pack_f16x2(__uint_as_float(qb[nt][ks][i] << 16) * f,
                                                   __uint_as_float(qb[nt][ks][i] & 0xffff0000u) * f);
#pragma unroll
                for (int j = 0; j < 2; ++j) cc[nt][j] = c * __shfl_sync(0xffffffffu, back, 4 * (2 * t + j));
            }
        }
        [[maybe_unused]] float slope2[NT][2];
        [[maybe_unused]] int last = 0;  // the row's last token
        if constexpr (MOD) {
            const int row0 = (sm.seg[cur].y - kvh * a.rgroups) * 8 * NT, h0 = kvh * a.group + row0;
            const int rows = min(8 * NT, a.group - row0);
            last = sm.seg[cur].hi - 1;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = 8 * nt + 2 * t + j;
                    slope2[nt][j] = a.slopes && r < rows ? bias_slope(a.slopes[h0 + r]) : 0.f;
                }
        }

        float o[NT][KS][4];
        // of heads 2t, 2t + 1: the reference (log2 domain), the score (as the products give it; MOD: in the log2 domain)
        // past which it moves, and as pairs what is added to a score (plain: less the maximum; MOD: less the reference; 0 before
        // the first) and this lane's tokens' part of the sum
        float m_ref[NT][2], edge[NT][2];
        uint64_t m_neg[NT], l[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int nd = 0; nd < KS; ++nd) o[nt][nd][0] = o[nt][nd][1] = o[nt][nd][2] = o[nt][nd][3] = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) m_ref[nt][j] = edge[nt][j] = -INFINITY;
            m_neg[nt] = l[nt] = 0;
        }

        int tok0 = w0 * kRowPS;
        for (int k = 0; k < nk; ++k, tok0 += kStep * kRowPS) {
            const uint32_t slot = done % kSl;
            if (!mbar_wait(&sm.full[warp][slot], (done / kSl) & 1, wc, 150 + warp)) {
                failed = true;
                break;
            }
            // slots that are not seen, and those of a page that is not there, may hold anything: their scales of the values become
            // 0, and so do their scores, which choose the form of the cap with the others, until they become -inf.  Steps with such
            // slots (PART) are a form of their own, which leaves out a second page past the end
            const bool ragged = tok0 + kStep * kRowPS > end || tok0 < lo || (gaps[0] | gaps[1]);
            auto step = [&](auto part) {
                constexpr bool PART = decltype(part)::value;
                uint8_t (*kv)[2][9 * D] = sm.kv[warp][slot];
                // rows (tokens) g, g + 8 of each page, columns (heads) 2t, 2t + 1
                float sc[kStep][NT][4];
#pragma unroll
                for (int j = 0; j < kStep; ++j) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) sc[j][nt][0] = sc[j][nt][1] = sc[j][nt][2] = sc[j][nt][3] = 0.f;
                    if (PART && j > 0 && tok0 + kRowPS * j >= end) continue;
                    const uint8_t *Kb = kv[j][0];
                    // one k-step: the f16 pairs of tokens g and g + 8 and their scales
                    auto k_step = [&](int ks, uint32_t x0, uint32_t x1, uint32_t y0, uint32_t y1, uint32_t s0, uint32_t s1) {
                        const uint32_t ka[4] = {f16x2_mul(x0, s0), f16x2_mul(y0, s1), f16x2_mul(x1, s0), f16x2_mul(y1, s1)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_16816_f16(sc[j][nt], ka, qb[nt][ks][0], qb[nt][ks][1]);
                    };
                    // two k-steps: a word of codes of each token
                    auto k_word = [&](int ks, uint32_t w0, uint32_t w1, uint32_t s0, uint32_t s1) {
                        uint32_t x[4], y[4];
                        e2m1x8_to_f16x2x4(w0, x);
                        e2m1x8_to_f16x2x4(w1, y);
                        k_step(ks, x[0], x[1], y[0], y[1], s0, s1);
                        k_step(ks + 1, x[2], x[3], y[2], y[3], s0, s1);
                    };
                    const uint8_t *k0 = Kb + fp4_k_codes(D, g, 0), *k1 = Kb + fp4_k_codes(D, g + 8, 0);
                    const uint8_t *s0 = Kb + fp4_k_scale(D, g, 0), *s1 = Kb + fp4_k_scale(D, g + 8, 0);
                    if constexpr (D == 128) {
                        const uint4 w0 = *reinterpret_cast<const uint4 *>(k0 + 16 * t), w1 = *reinterpret_cast<const uint4 *>(k1 + 16 * t);
                        const uint32_t p0 = e4m3_pair(*reinterpret_cast<const uint16_t *>(s0 + 2 * t));
                        const uint32_t p1 = e4m3_pair(*reinterpret_cast<const uint16_t *>(s1 + 2 * t));
                        const uint32_t a0 = prmt(p0, 0u, 0x1010u), a1 = prmt(p1, 0u, 0x1010u);
                        const uint32_t b0 = prmt(p0, 0u, 0x3232u), b1 = prmt(p1, 0u, 0x3232u);
                        k_word(0, w0.x, w1.x, a0, a1);
                        k_word(2, w0.y, w1.y, a0, a1);
                        k_word(4, w0.z, w1.z, b0, b1);
                        k_word(6, w0.w, w1.w, b0, b1);
                    } else {
#pragma unroll
                        for (int u = 0; u < D / 64; ++u) {
                            const uint2 w0 = *reinterpret_cast<const uint2 *>(k0 + 32 * u + 8 * t);
                            const uint2 w1 = *reinterpret_cast<const uint2 *>(k1 + 32 * u + 8 * t);
                            const uint32_t a0 = e4m3_pair(s0[4 * u + t] * 0x101u), a1 = e4m3_pair(s1[4 * u + t] * 0x101u);
                            k_word(4 * u, w0.x, w1.x, a0, a1);
                            k_word(4 * u + 2, w0.y, w1.y, a0, a1);
                        }
                        constexpr int x = D / 64 * 32, n = D / 64 * 4;  // the rest: its byte, its first k-step and block
                        if constexpr (D % 64 == 32) {
                            const uint32_t w0 = *reinterpret_cast<const uint32_t *>(k0 + x + 4 * t);
                            const uint32_t w1 = *reinterpret_cast<const uint32_t *>(k1 + x + 4 * t);
                            k_word(n, w0, w1, e4m3_pair(s0[n + (t >> 1)] * 0x101u), e4m3_pair(s1[n + (t >> 1)] * 0x101u));
                        } else if constexpr (D % 64 == 16) {
                            const uint32_t w0 = *reinterpret_cast<const uint16_t *>(k0 + x + 2 * t);
                            const uint32_t w1 = *reinterpret_cast<const uint16_t *>(k1 + x + 2 * t);
                            uint32_t z[4];
                            e2m1x8_to_f16x2x4(w0 | w1 << 16, z);
                            k_step(n, z[0], z[1], z[2], z[3], e4m3_pair(s0[n] * 0x101u), e4m3_pair(s1[n] * 0x101u));
                        }
                    }
                }
                auto seen = [&](int j, int i) {
                    const uint32_t gone = (((k / kIds) & 1) ? gaps[1] : gaps[0]) >> (kStep * (k % kIds));
                    const int x = tok0 + kRowPS * j + i;
                    return !((gone >> j) & 1u) && x >= lo && x < end;
                };
                auto unseen_to = [&](int j, float v) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!seen(j, g + (i < 2 ? 0 : 8)))
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) sc[j][nt][i] = v;
                };
                if constexpr (PART) {
#pragma unroll
                    for (int j = 0; j < kStep; ++j) {
                        for (int i = lane; i < kRowPS * KS; i += 32)
                            if (!seen(j, i & 15)) kv[j][1][fp4_v_scale(D, i & 15, i >> 4)] = 0;
                        unseen_to(j, MOD ? 0.f : -INFINITY);
                    }
                    fence_proxy_async_smem();  // before the next copy into these bytes
                    __syncwarp();
                }
                if constexpr (MOD) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint64_t c2 = f32x2_pack(cc[nt][0], cc[nt][1]);
                        uint64_t u[kStep][2];
#pragma unroll
                        for (int j = 0; j < kStep; ++j)
#pragma unroll
                            for (int i = 0; i < 2; ++i) u[j][i] = f32x2_mul(f32x2_pack(sc[j][nt][2 * i], sc[j][nt][2 * i + 1]), c2);
                        if (a.cap_in > 0.f) {
                            float big = 0.f;
#pragma unroll
                            for (int j = 0; j < kStep; ++j)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    float x, y;
                                    f32x2_unpack(u[j][i], x, y);
                                    big = fmax3_abs(big, x, y);
                                }
                            const int tier = !__any_sync(0xffffffffu, big > 0.25f) ? 0 : (__any_sync(0xffffffffu, big > 1.f) ? 2 : 1);
#pragma unroll
                            for (int j = 0; j < kStep; ++j)
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    u[j][i] = tier == 0 ? TanhCap::eval_u<0>(u[j][i], a.cap_out)
                                                        : (tier == 1 ? TanhCap::eval_u<1>(u[j][i], a.cap_out)
                                                                     : TanhCap::eval_u<2>(u[j][i], a.cap_out));
                        }
                        if (a.slopes) {
                            const uint64_t s2 = f32x2_pack(-slope2[nt][0], -slope2[nt][1]);
#pragma unroll
                            for (int j = 0; j < kStep; ++j)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {  // the distance of token g or g + 8
                                    const float far = (float)(last - tok0 - kRowPS * j - g - 8 * i);
                                    u[j][i] = f32x2_fma(s2, f32x2_pack(far, far), u[j][i]);
                                }
                        }
#pragma unroll
                        for (int j = 0; j < kStep; ++j)
#pragma unroll
                            for (int i = 0; i < 2; ++i) f32x2_unpack(u[j][i], sc[j][nt][2 * i], sc[j][nt][2 * i + 1]);
                    }
                }
                if constexpr (MOD && PART) {
#pragma unroll
                    for (int j = 0; j < kStep; ++j) unseen_to(j, -INFINITY);
                    __syncwarp();
                }
                auto most_of = [&](int nt, int i) {  // this lane's largest score of a head
                    const float m = fmaxf(sc[0][nt][i], sc[0][nt][i + 2]);
                    return kStep == 1 ? m : fmax3(m, sc[kStep - 1][nt][i], sc[kStep - 1][nt][i + 2]);
                };
                bool grow = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) grow = grow || most_of(nt, i) > edge[nt][i];
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float al[2], last_max[2];
                        f32x2_unpack(m_neg[nt] ^ 0x8000000080000000ull, last_max[0], last_max[1]);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float mx = most_of(nt, i);
#pragma unroll
                            for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                            al[i] = 1.f;
                            if (mx > edge[nt][i]) {
                                const float m = MOD ? mx : mx * cc[nt][i];
                                const float ref = !MOD || fabsf(m) < kLifted ? m - kLift : m;
                                const float past = MOD ? m_ref[nt][i] - ref : (last_max[i] - mx) * cc[nt][i];
                                al[i] = m_ref[nt][i] == -INFINITY ? 0.f : ex2_approx(past);
                                m_ref[nt][i] = ref;
                                edge[nt][i] = __fadd_rd(mx, MOD ? kThresh : kThresh / cc[nt][i]);
                                last_max[i] = mx;
                            }
                        }
                        l[nt] = f32x2_mul(l[nt], f32x2_pack(al[0], al[1]));
                        if constexpr (MOD)
                            m_neg[nt] = f32x2_pack(m_ref[nt][0] == -INFINITY ? 0.f : -m_ref[nt][0],
                                                   m_ref[nt][1] == -INFINITY ? 0.f : -m_ref[nt][1]);
                        else
                            m_neg[nt] = f32x2_pack(-last_max[0], -last_max[1]);
#pragma unroll
                        for (int nd = 0; nd < KS; ++nd) {
                            o[nt][nd][0] *= al[0];
                            o[nt][nd][1] *= al[1];
                            o[nt][nd][2] *= al[0];
                            o[nt][nd][3] *= al[1];
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < kStep; ++j) {
                    if (PART && j > 0 && tok0 + kRowPS * j >= end) continue;
                    uint32_t pb[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float p[4];
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {  // the two heads at once
                            const uint64_t x = f32x2_pack(sc[j][nt][i], sc[j][nt][i + 1]);
                            const uint64_t y = f32x2_add(x, m_neg[nt]);
                            f32x2_unpack(MOD ? y : f32x2_fma(y, f32x2_pack(cc[nt][0], cc[nt][1]), f32x2_pack(kLift, kLift)), p[i], p[i + 1]);
                            p[i] = ex2_approx(p[i]);
                            p[i + 1] = ex2_approx(p[i + 1]);
                            l[nt] = f32x2_add(l[nt], f32x2_pack(p[i], p[i + 1]));
                        }
                        // tokens from the rows into the pairs of the B operand.  The weights are rounded to f16 once
                        // (2^-11 of each at most, under 2^-21 of the largest 2^-32 of that; the sum takes them unrounded), as the product takes them: the rest in a
                        // second product would cost as much as the first, and the result, rounded to bf16, is off by
                        // 0.00168 of itself where fp32 weights give 0.00167.
                        pb[nt][0] = movmatrix_trans(pack_f16x2(p[0], p[1]));
                        pb[nt][1] = movmatrix_trans(pack_f16x2(p[2], p[3]));
                    }
                    const uint8_t *Vb = kv[j][1];
                    const uint32_t Vs = smem_u32(Vb);
                    uint32_t sv[(KS + 3) / 4 * 4];  // the scales of the lane's quad of tokens, 4 bytes a block
                    if constexpr (KS % 4 == 0) {
#pragma unroll
                        for (int n0 = 0; n0 < KS; n0 += 4) {
                            const uint4 w = *reinterpret_cast<const uint4 *>(Vb + fp4_v_scale(D, 2 * t, n0));
                            sv[n0] = w.x, sv[n0 + 1] = w.y, sv[n0 + 2] = w.z, sv[n0 + 3] = w.w;
                        }
                    } else {
#pragma unroll
                        for (int nd = 0; nd < KS; ++nd) sv[nd] = *reinterpret_cast<const uint32_t *>(Vb + fp4_v_scale(D, 2 * t, nd));
                    }
#pragma unroll
                    for (int n0 = 0; n0 < KS; n0 += 4) {
                        uint32_t w[4];  // lane l: row l & 7 of block n0 + (l >> 3); past the last block: that one again
                        ldsm_x4_trans(Vs + min(n0 + (lane >> 3), KS - 1) * 128 + (lane & 7) * 16, w);
#pragma unroll
                        for (int i = 0; i < 4 && n0 + i < KS; ++i) {
                            const int nd = n0 + i;
                            uint32_t sa, sb, va[4];
                            e4m3x4_to_f16x2x2(sv[nd], sa, sb);
                            e2m1x8_to_f16x2x4(w[i], va);
                            va[0] = f16x2_mul(va[0], sa);
                            va[1] = f16x2_mul(va[1], sa);
                            va[2] = f16x2_mul(va[2], sb);
                            va[3] = f16x2_mul(va[3], sb);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma_16816_f16(o[nt][nd], va, pb[nt][0], pb[nt][1]);
                        }
                    }
                }
            };
            if (ragged) step(std::true_type{});
            else step(std::false_type{});
            __syncwarp();  // the slot's reads are done
            ++done;
            if (k + kSl < nk) issue(kvh, k + kSl);
        }
        if (failed) {  // this warp's copies in flight land (bounded)
            WaitCtx drain{nullptr, a.status};
            for (; done != sent; ++done)
                if (lane == 0) (void)mbar_wait(&sm.full[warp][done % kSl], (done / kSl) & 1, drain, 198);
            __syncwarp();
        }

        float ls[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) f32x2_unpack(l[nt], ls[nt][0], ls[nt][1]);
        const Segment &was = sm.seg[cur];
        const int row0 = (was.y - kvh * a.rgroups) * 8 * NT, h0 = kvh * a.group + row0, rows = min(8 * NT, a.group - row0);
        if (a.cluster) {
            rows_finish<D, NT, true, true>(sm.red, &sm.abort_flag, a, o, m_ref, ls, rows, h0, was.b, blockIdx.x, nullptr, 0);
            return;
        }
        __syncthreads();  // the next part is there, and the last one's state has been read
        // its query and first pages may come already
        cur ^= 1;
        const bool more = sm.seg[cur].b >= 0;
        if (more) {
            kvh = sm.seg[cur].y / a.rgroups;
            nk = quarter();
            load_q(kvh);
            if (failed) nk = 0;
            for (int k = 0; k < min(nk, kSl); ++k) issue(kvh, k);
        }
        // a part of a row that begins in an earlier CTA goes to the CTA's first place, one that only begins here to its second
        write_part<D, NT>(sm.red, o, m_ref, ls, a, rows, (size_t)was.b * a.H + h0,
                          a.ws + (size_t)(2 * blockIdx.x + (was.from_start ? 1 : 0)) * (8 * NT) * (D + 4),
                          was.from_start && was.to_end);
        if (threadIdx.x == 0) {
            int2 *cta = a.row_ctas + (size_t)was.b * R + was.y;
            if (was.from_start && was.p0 < was.p1) cta->x = blockIdx.x;
            if (was.to_end) cta->y = blockIdx.x;
        }
        if (!more) return;
        __syncthreads();  // before that segment's place is taken by the one after the next
    }
}

// Joins the parts of a query head's row, where several CTAs had one: W warps a head, which take its parts in turn, lanes four
// columns each.  A sequence that sees nothing gets zeros.  One warp a head past kJoinHeads heads, four up to there, whose rows may
// have many parts (call with four / one: 32 sequences of 32 heads 37.9 / 39.0 us, 64 of 32 22.5 / 20.7, 128 of 12 29.7 / 28.9),
// sixteen up to a head an SM (call with four / sixteen, 32 heads: one sequence of 103000 tokens 31.5 / 29.9 us, of up to 40000
// 18.4 / 16.5, 4 of up to 30000 22.8 / 22.6; past that sixteen cost, 32 of up to 8192 38.3 / 43.0).
constexpr int kJoinHeads = 1024;
template <int W> constexpr int kJoinWarps = W > 4 ? W : 4;  // of a CTA
template <int D, int NT, int W>
__global__ void __launch_bounds__(kJoinWarps<W> * 32) decode_fp4_join_kernel(const Fp4Params a) {
    __shared__ float4 acc_s[kJoinWarps<W>][32];
    __shared__ float2 ml_s[kJoinWarps<W>];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row = (long long)blockIdx.x * (kJoinWarps<W> / W) + warp / W;  // (sequence, head)
    const bool there = row < (long long)a.B * a.H;
    const int b = there ? (int)(row / a.H) : 0, h = (int)(row - (long long)b * a.H);
    const int in_group = h % a.group, y = h / a.group * a.rgroups + in_group / (8 * NT);
    const PageRange r = seen_pages(a, b);
    const bool any_page = r.p0 < r.p1;
    griddep_launch_dependents();
    griddep_wait();  // (by every CTA, so that this grid does not end before the one that it depends on)
    if (!there) return;
    int2 ctas = make_int2(0, 0);
    if (any_page) {
        ctas = a.row_ctas[(size_t)b * a.Hkv * a.rgroups + y];
        if (ctas.x == ctas.y) return;  // written whole (uniform over the head's warps)
    }
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (any_page) {
        const size_t head = in_group % (8 * NT);
        for (int c = ctas.x + warp % W; c <= ctas.y; c += W * 4) {
            float2 ml[4];
            float4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // four parts in flight
                const int ci = c + W * i;
                ml[i] = make_float2(-INFINITY, 0.f);
                v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (ci <= ctas.y) {
                    const float *part = a.ws + ((size_t)(2 * ci + (ci == ctas.x ? 1 : 0)) * (8 * NT) + head) * (D + 4);
                    ml[i] = *reinterpret_cast<const float2 *>(part + D);
                    if (4 * lane < D) v[i] = *reinterpret_cast<const float4 *>(part + 4 * lane);
                }
            }
            const float m = fmaxf(fmax3(M, ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
            if (m == -INFINITY) continue;
            const float al = ex2_approx(M - m);
            M = m;
            L *= al;
            acc.x *= al, acc.y *= al, acc.z *= al, acc.w *= al;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float wt = ex2_approx(ml[i].x - M);  // 0 for an empty one, whose O is 0
                L = fmaf(ml[i].y, wt, L);
                acc.x = fmaf(v[i].x, wt, acc.x);
                acc.y = fmaf(v[i].y, wt, acc.y);
                acc.z = fmaf(v[i].z, wt, acc.z);
                acc.w = fmaf(v[i].w, wt, acc.w);
            }
        }
    }
    if constexpr (W > 1) {
        acc_s[warp][lane] = acc;  // (one head a CTA: its threads all come here)
        if (lane == 0) ml_s[warp] = make_float2(M, L);
        __syncthreads();
        if (warp != 0) return;
        M = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, ml_s[w].x);
        L = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (M != -INFINITY) {
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float wt = ex2_approx(ml_s[w].x - M);
                const float4 v = acc_s[w][lane];
                L = fmaf(ml_s[w].y, wt, L);
                acc.x = fmaf(v.x, wt, acc.x);
                acc.y = fmaf(v.y, wt, acc.y);
                acc.z = fmaf(v.z, wt, acc.z);
                acc.w = fmaf(v.w, wt, acc.w);
            }
        }
    }
    const bool any = L != 0.f;
    const OverSum over(a.v_scale, L, any);
    if (4 * lane < D)
        *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(a.o) + (size_t)row * D + 4 * lane) =
            make_uint2(pack_bf16x2(over(acc.x), over(acc.y)), pack_bf16x2(over(acc.z), over(acc.w)));
    if (lane == 0 && a.lse) a.lse[row] = any ? kRowLn2 * (M + __log2f(L)) : -INFINITY;
}

size_t fp4_parts_bytes(int group, int d) {
    return (size_t)kSms * (group <= 8 ? kFp4Ctas<1> * 8 : kFp4Ctas<2> * 16) * 2 * (size_t)(d + 4) * sizeof(float);
}

// Splits of a row for the form whose splits are one cluster (0: shares).  It takes one launch and no workspace, but as many CTAs for
// a short row as for a long one, and how many is the host's choice, by the table's width: for rows that are resident all at once
// with up to kClusterPages pages a CTA.  Both ways,
// us (cluster / shares; 32/8 heads, d 128 unless said):
//   2 sequences of up to 900, 12 heads of 64   6.1 / 11.3      32 of 1000 (32 pages a CTA)    14.4 / 16.4
//   1 of 16000 (63 pages a CTA)               13.4 / 14.3      64 of 200, 500, 1000 (63)      12.4 / 16.5, 16.4 / 18.5, 22.5 / 23.2
//   1 of 32000 (125)                          18.5 / 16.4      32 of 2000 (63), 4000 (125)    20.0 / 20.5, 29.9 / 26.6
//   not resident at once, one CTA a row: 128 of 110 and 600, 12 heads of 64, 17.5 / 16.4, 26.6 / 24.6; 256 of 100 32.6 / 28.7
constexpr int kClusterPages = 64;
int fp4_cluster(int B, int H, int Hkv, int max_pages) {
    const int group = H / Hkv;
    const long long rows = (long long)B * Hkv * (group <= 8 ? 1 : (group + 15) / 16);
    const long long slots = (long long)kSms * (group <= 8 ? kFp4Ctas<1> : kFp4Ctas<2>);
    // (clusters of more than 4 leave some slots unused)
    long long n = slots * 95 / 100 / rows;
    if (n > 4) n = slots * 85 / 100 / rows > 4 ? slots * 85 / 100 / rows : 4;
    if (n > kRowCluster) n = kRowCluster;
    if (n > (max_pages + kRowWarps - 1) / kRowWarps) n = (max_pages + kRowWarps - 1) / kRowWarps;
    return max_pages <= kClusterPages * n ? (int)n : 0;
}

template <int D, int NT, bool MOD>
cudaError_t launch_fp4_n(const DecodeMoreArgs &a, Fp4Params p, cudaStream_t stream) {
    const size_t smem = sizeof(Fp4Smem<D, NT>) + 128;
    auto kernel = decode_fp4_kernel<D, NT, MOD>;
    cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void *>(kernel), (int)smem);
    if (e != cudaSuccess) return e;
    const uint8_t *k = static_cast<const uint8_t *>(a.k_pages), *v = static_cast<const uint8_t *>(a.v_pages);
    if (p.cluster) {
        if (p.cluster > 8) e = ensure_large_clusters(reinterpret_cast<const void *>(kernel));
        if (e == cudaSuccess && cluster_fits(reinterpret_cast<const void *>(kernel), p.cluster, kFp4Threads, smem)) {
            Fp4Params c = p;
            c.n_splits = p.cluster;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(p.cluster, p.Hkv * p.rgroups, p.B);
            cfg.blockDim = dim3(kFp4Threads);
            cfg.dynamicSmemBytes = smem;
            cfg.stream = stream;
            cudaLaunchAttribute attr[2];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = p.cluster;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[1].val.programmaticStreamSerializationAllowed = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 2;
            return cudaLaunchKernelEx(&cfg, kernel, k, v, c);
        }
        (void)cudaGetLastError();
        p.cluster = 0;  // no room for the cluster (a part of a GPU): shares through the workspace
    }
    // (not as a dependent: one that comes while the last kernel's CTAs leave does not fill the SMs in turn, 37 -> 49 us)
    kernel<<<kSms * kFp4Ctas<NT>, kFp4Threads, smem, stream>>>(k, v, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long heads = (long long)p.B * p.H;
    auto join = [&](auto w) {
        constexpr int W = decltype(w)::value, kHeads = kJoinWarps<W> / W;
        return launch_dependent(decode_fp4_join_kernel<D, NT, W>, dim3((unsigned)((heads + kHeads - 1) / kHeads)), kJoinWarps<W> * 32, 0, stream, p);
    };
    if (heads <= kSms) return join(std::integral_constant<int, 16>{});
    return heads <= kJoinHeads ? join(std::integral_constant<int, 4>{}) : join(std::integral_constant<int, 1>{});
}

template <int D>
cudaError_t launch_fp4_d(const DecodeMoreArgs &a, Fp4Params p, cudaStream_t stream) {
    p.rgroups = p.group <= 8 ? 1 : (p.group + 15) / 16;
    const bool mod = a.softcap > 0.f || a.slopes;
    if (p.group <= 8) return mod ? launch_fp4_n<D, 1, true>(a, p, stream) : launch_fp4_n<D, 1, false>(a, p, stream);
    return mod ? launch_fp4_n<D, 2, true>(a, p, stream) : launch_fp4_n<D, 2, false>(a, p, stream);
}

}  // namespace

// Two parts of up to 8 or 16 heads for each CTA of the shares, and each row's first and last CTA.
size_t decode_fp4_workspace_bytes(int B, int H, int Hkv, int d, int max_pages, int page_size) {
    if (decode_workspace_bytes(B, H, Hkv, d, max_pages, page_size) == 0) return 0;  // unsupported sizes
    const size_t group = (size_t)(H / Hkv), rows = (size_t)B * Hkv * (group <= 8 ? 1 : (group + 15) / 16);
    return fp4_parts_bytes((int)group, d) + rows * sizeof(int2);
}

cudaError_t launch_decode_fp4(const DecodeMoreArgs &a, cudaStream_t stream) {
    Fp4Params p{};
    p.q = a.q;
    p.page_table = a.page_table;
    p.ctx_lens = a.ctx_lens;
    p.o = a.o;
    p.lse = a.lse;
    p.ws = static_cast<float *>(a.workspace);
    p.row_ctas = reinterpret_cast<int2 *>(static_cast<char *>(a.workspace) + fp4_parts_bytes(a.H / a.Hkv, a.d));
    p.status = a.status;
    p.B = a.B;
    p.H = a.H;
    p.Hkv = a.Hkv;
    p.group = a.H / a.Hkv;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.cluster = fp4_cluster(a.B, a.H, a.Hkv, a.max_pages);
    const float kscale = a.scale * a.k_scale;
    p.c = kscale * kRowLog2e;
    p.v_scale = a.v_scale;
    p.cap_in = a.softcap > 0.f ? kscale / a.softcap : 0.f;
    p.cap_out = a.softcap * kRowLog2e;
    p.q_low = query_low(p.cap_in > 0.f ? p.cap_in : p.c);
    p.slopes = a.slopes;
    p.key_begin = a.key_begin;
    switch (a.d) {
        case 32: return launch_fp4_d<32>(a, p, stream);
        case 64: return launch_fp4_d<64>(a, p, stream);
        case 80: return launch_fp4_d<80>(a, p, stream);
        case 96: return launch_fp4_d<96>(a, p, stream);
        case 128: return launch_fp4_d<128>(a, p, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace attn
