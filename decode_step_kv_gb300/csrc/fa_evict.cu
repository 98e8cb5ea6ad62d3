// fa_evict.cu -- eviction from a KV cache by accumulated attention weight, for
// sm_103a (GB300).
//
// For every sequence longer than the budget and each of its KV heads: keep the
// first n_sink tokens, the last n_recent, and of the tokens between them the
// ones with the largest running totals; move the kept rows, in order, to the
// front of the cache.
//
// A thread-block cluster per (sequence, KV head) selects and moves what needs an
// order; a second kernel moves the rest with every SM, unless there is little of it
// or the clusters fill the GPU: then they go on with it themselves.
//   Selection: a radix selection of the k-th largest total (11 + 11 + 10 bits
//   of the order-preserving integer), each CTA counting its share of the
//   tokens, the counts summed through distributed shared memory (one cluster
//   barrier per pass); then every
//   warp emits its tokens' kept indices at the rank that the warps before it
//   leave.  Ties go to the lowest index.  A CTA keeps its share of the totals in
//   shared memory when it fits (23424 tokens), so they are read once.
//   Move: rows go down in place (a kept row's new index is never above its old
//   one; those before the first dropped token stay).  A write to row j only
//   clobbers a source when token j itself is kept, so order matters only among
//   the kept tokens below the budget.  Those move first, in rounds: every CTA of the cluster reads its rows of the round into
//   shared memory, a cluster barrier, every CTA writes them (what a round
//   overwrites lies below the sources of all later rounds).  After them, the
//   kept tokens from the budget on move in any order.
// Bound by latency: of selecting (~18 us in the first case below, ~30 in the second), of the
// rounds' barriers, and of rows of 256 or 512 bytes read and written once from scattered
// places (DRAM 44% busy in the first case's kernel, 57% in the second's second one).  GPU time,
// cold L2, fp16, against the bytes of the totals and of the rows that change their place:
//   32 sequences of 1024 to 8192 tokens x 8 heads x 128, cut to 2048       119 us     67
//   32 of 2304 (cut again 256 tokens later)                                115 us     80
//   one of 131072 x 8 heads x 256, cut to 16384                             97 us     40
//   one of 16640 (again 256 later: 96% of the moved rows in order)          89 us     16
#include "fa_common.cuh"

namespace fa {
namespace ev {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int BINS = 2048;
constexpr int MAX_CTAS = 16;             // CTAs per cluster (8 are portable; fewer if they do not fit)
// Totals, then rows in flight, of a CTA: two CTAs per SM, or one when there are few units.
constexpr int STAGE_BYTES = 96 * 1024, STAGE_BYTES_1 = 200 * 1024;
constexpr int GROUPS = 64, GROUP_BINS = BINS / GROUPS;   // bins are summed over a cluster in groups
static_assert(GROUP_BINS == 32 && GROUPS == 64 && WARPS >= MAX_CTAS, "lanes and warps of the search");
constexpr int SCRATCH = 2 * GROUPS + THREADS + 32 * WARPS;      // words of it
constexpr int HELD = STAGE_BYTES / 4 - SCRATCH;                 // totals a CTA holds
constexpr int ROUND_ROWS = THREADS;      // most rows a CTA stages per round
constexpr double FUSED_BYTES = 4 << 20;  // rows to move up to which one kernel does it all

struct Args {
    char *a[4];          // K, V, K scales, V scales (NULL: none)
    int row_bytes[4];    // powers of two from 8
    float *acc;
    int *new_lens, *kept;
    int budget, sink, recent;
    int lg_page;         // log2 of page_size, or -1
    int rows;            // rows staged per CTA and round
    int fused;           // the cluster kernel also moves the rows from the budget on
};

// Totals as integers in the same order: NaN counts as -inf, -0 as 0.
__device__ __forceinline__ unsigned order_key(float x)
{
    unsigned b = __float_as_uint(x);
    if (x != x)
        b = 0xff800000u;
    else if (x == 0.f)
        b = 0u;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Cache row of token t of (b, kv); -1 for a block id out of range.
__device__ __forceinline__ long long row_of(const Params &p, const Args &x, int b, int kv, int t)
{
    if (!p.bt)
        return ((long long)b * p.Hkv + kv) * p.cap + t;
    const int page = x.lg_page >= 0 ? t >> x.lg_page : t / p.page_size;
    const int blk = __ldg(p.bt + (long long)b * p.max_blocks + page);
    if (blk < 0 || blk >= p.num_blocks)
        return -1;
    return ((long long)blk * p.Hkv + kv) * p.page_size + (t - page * p.page_size);
}

__device__ __forceinline__ unsigned ld_cluster(uint32_t a)
{
    unsigned v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// Places of up to ROUND_ROWS rows: src -1 where nothing is to be moved.
struct Places {
    long long src[ROUND_ROWS], dst[ROUND_ROWS];
};

// Rows pl.src -> pl.dst of the arrays first .. first + 1 (K and V, or the scales), by the
// whole CTA, in pieces, DEPTH of them in flight per thread over both arrays.  No
// source may be another row's destination.
template <typename Piece, int DEPTH>
__device__ __forceinline__ void copy_rows(const Args &x, int first, const Places &pl, int nr)
{
    char *a0 = x.a[first], *a1 = x.a[first + 1];
    const int l0 = a0 ? 31 - __clz(x.row_bytes[first] / static_cast<int>(sizeof(Piece))) : 0;
    const int l1 = a1 ? 31 - __clz(x.row_bytes[first + 1] / static_cast<int>(sizeof(Piece))) : 0;
    const int n0 = a0 ? nr << l0 : 0, total = n0 + (a1 ? nr << l1 : 0);
    // piece i: its row (-1: not moved) and its place in the row
    auto place = [&](int i, const long long *rows, Piece *&at) {
        const bool second = i >= n0;
        const int k = second ? i - n0 : i, lg = second ? l1 : l0;
        const long long r = rows[k >> lg];
        at = reinterpret_cast<Piece *>(second ? a1 : a0) + (r << lg) + (k & ((1 << lg) - 1));
        return r >= 0;
    };
    for (int i0 = threadIdx.x; i0 < total; i0 += DEPTH * blockDim.x) {
        Piece v[DEPTH];
#pragma unroll
        for (int q = 0; q < DEPTH; ++q) {
            const int i = i0 + q * blockDim.x;
            Piece *at;
            if (i < total && place(i, pl.src, at))
                v[q] = __ldcs(at);
        }
#pragma unroll
        for (int q = 0; q < DEPTH; ++q) {
            const int i = i0 + q * blockDim.x;
            Piece *at;
            if (i < total && place(i, pl.dst, at))
                *at = v[q];
        }
    }
}

// Kept rows r0 .. r0 + nr - 1 whose token lies at or above the budget.
template <int DEPTH>
__device__ __forceinline__ void move_far(const Params &p, const Args &x, int b, int kv,
                                         const int *kept, int r0, int nr, Places &pl)
{
    __syncthreads();                              // pl is free
    if (threadIdx.x < nr) {
        const int j = r0 + threadIdx.x, t = __ldcg(kept + j);
        const long long s = t >= x.budget ? row_of(p, x, b, kv, t) : -1;
        const long long d = s >= 0 ? row_of(p, x, b, kv, j) : -1;
        pl.src[threadIdx.x] = d >= 0 ? s : -1;
        pl.dst[threadIdx.x] = s >= 0 ? d : -1;
    }
    __syncthreads();
    copy_rows<uint4, DEPTH>(x, 0, pl, nr);
    if (x.a[3]) {
        if (x.row_bytes[3] >= 16)
            copy_rows<uint4, DEPTH>(x, 2, pl, nr);
        else
            copy_rows<uint2, DEPTH>(x, 2, pl, nr);
    }
}

// The totals of tokens t0, t0 + step, ... below n start again from zero.  Int holds n + 8
// steps: the second kernel's step is four times the budget, the first one's at most 8192.
template <typename Int>
__device__ __forceinline__ void clear_totals(const Params &p, const Args &x, int b, int kv, Int t0,
                                             Int step, int n)
{
    constexpr int U = 8;
    for (; t0 < n; t0 += U * step) {
        long long r[U];
#pragma unroll
        for (int q = 0; q < U; ++q)
            r[q] = t0 < n - q * step ? row_of(p, x, b, kv, static_cast<int>(t0 + q * step)) : -1;
#pragma unroll
        for (int q = 0; q < U; ++q)
            if (r[q] >= 0)
                x.acc[r[q]] = 0.f;
    }
}

constexpr int FAR_THREADS = 256;
constexpr int FAR_ROWS = 64;             // kept rows per CTA
__global__ void __launch_bounds__(FAR_THREADS, 4) evict_far_kernel(const Params p, const Args x)
{
    __shared__ Places pl;
    const int chunks = (x.budget + FAR_ROWS - 1) / FAR_ROWS;
    const int unit = blockIdx.x / chunks;
    const int b = unit / p.Hkv, kv = unit % p.Hkv;
    int lo, n;
    attended_range(p, b, lo, n, false);
    wait_for_previous();
    if (n <= x.budget)
        return;
    const int c = blockIdx.x % chunks, r0 = c * FAR_ROWS;
    clear_totals<long long>(p, x, b, kv, x.budget + (long long)c * FAR_THREADS + threadIdx.x,
                            (long long)chunks * FAR_THREADS, n);
    move_far<8>(p, x, b, kv, x.kept + (long long)unit * x.budget, r0, min(FAR_ROWS, x.budget - r0),
                pl);
}

template <int N>
__device__ __forceinline__ void cp(uint32_t dst, const void *src)
{
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// The sum of v over the lanes before this one.
__device__ __forceinline__ unsigned warp_above(unsigned v)
{
    unsigned incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, incl, off);
        if (static_cast<int>(threadIdx.x & 31) >= off)
            incl += y;
    }
    return incl - v;
}

__global__ void __launch_bounds__(THREADS, 2) evict_kernel(const Params p, const Args x)
{
    __shared__ __align__(16) unsigned hist[BINS];
    __shared__ unsigned cnt[WARPS][2];
    __shared__ unsigned wsum[WARPS];
    __shared__ unsigned found[2];
    __shared__ unsigned stay[2];             // this CTA's kept tokens: below the budget, at their places
    __shared__ __align__(16) Places pl;
    unsigned *hist2 = reinterpret_cast<unsigned *>(&pl);     // while selecting: every second pass's
    static_assert(sizeof(Places) >= BINS * sizeof(unsigned), "a histogram");
    extern __shared__ __align__(128) unsigned char stage[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int cs = p.cl_ctas;
    uint32_t rank = 0;
    if (cs > 1)
        asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const int unit = blockIdx.x / cs;
    const int b = unit / p.Hkv, kv = unit % p.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    int lo, n;
    attended_range(p, b, lo, n, kv == 0 && rank == 0 && tid == 0);
    int *kept = x.kept + (long long)unit * x.budget;
    if (kv == 0 && rank == 0 && tid == 0)
        x.new_lens[b] = min(n, x.budget);
    if (n <= x.budget) {
        for (long long j = rank * THREADS + tid; j < x.budget; j += cs * THREADS)
            kept[j] = j < n ? static_cast<int>(j) : -1;
        return;                                   // the whole cluster
    }

    // ---- the k-th largest total of the m tokens between sink and recent.  When one
    // CTA holds them all, every CTA of the cluster selects by itself: that costs
    // a few more passes over shared memory and saves six cluster barriers.
    const int m = n - x.sink - x.recent;
    const int k = x.budget - x.sink - x.recent;
    const bool solo = m <= HELD;
    const int sel = solo ? 1 : cs;                // CTAs that share the selection
    const int sr = solo ? 0 : rank;
    auto sync_sel = [&] {
        if (sel > 1)
            tc::cluster_sync();
        else
            __syncthreads();
    };
    auto sync_all = [&] {
        if (cs > 1)
            tc::cluster_sync();
        else
            __syncthreads();
    };
    const int gw = sr * WARPS + warp, nw = sel * WARPS;
    const int w0 = x.sink + static_cast<int>((long long)m * gw / nw);
    const int w1 = x.sink + static_cast<int>((long long)m * (gw + 1) / nw);
    auto total_at = [&](int t) -> float {
        const long long r = row_of(p, x, b, kv, t);
        if (r < 0) {
            flag(FA_STATUS_BAD_BLOCK);
            return -INFINITY;
        }
        return __ldcg(x.acc + r);
    };
    // this CTA's totals, as ordered integers, in shared memory, at the tokens' offsets
    // from its first
    const int c0 = x.sink + static_cast<int>((long long)m * (sr * WARPS) / nw);
    const int c1 = x.sink + static_cast<int>((long long)m * (sr * WARPS + WARPS) / nw);
    const bool held = c1 - c0 <= HELD;
    unsigned *tot = reinterpret_cast<unsigned *>(stage);          // and the selection's scratch
    if (held) {
        constexpr int U = 16;
        for (int t0 = w0 + lane; t0 < w1; t0 += 32 * U) {
            float v[U];
#pragma unroll
            for (int q = 0; q < U; ++q)
                v[q] = t0 + 32 * q < w1 ? total_at(t0 + 32 * q) : 0.f;
#pragma unroll
            for (int q = 0; q < U; ++q)
                if (t0 + 32 * q < w1)
                    tot[t0 + 32 * q - c0] = order_key(v[q]);
        }
        __syncwarp();                             // a warp reads its own tokens only
    }
    auto key_at = [&](int t) { return held ? tot[t - c0] : order_key(total_at(t)); };
    unsigned thr = 0xffffffffu;                   // keys above thr are kept ...
    unsigned rem = 0;                             // ... and the first rem equal to it
    if (k > 0) {
        thr = 0;
        rem = k;
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const int bits = pass == 2 ? 10 : 11;
            unsigned *h = pass == 1 && sel > 1 ? hist2 : hist;
            for (int i = tid; i < BINS; i += THREADS)
                h[i] = 0;
            __syncthreads();
#pragma unroll 4
            for (int t = w0 + lane; t < w1; t += 32) {
                const unsigned u = key_at(t);
                if (pass == 0 || ((u ^ thr) >> (shift + bits)) == 0)
                    atomicAdd(&h[(u >> shift) & ((1u << bits) - 1)], 1u);
            }
            __syncthreads();
            constexpr int PER = BINS / THREADS;
            if (sel > 1) {
                // One cluster barrier per pass: the sums of 64 groups of bins over the
                // cluster, then of the 32 bins of the group that holds the k-th.  What a
                // slower CTA still reads is written again only two passes later.
                unsigned *gsum = tot + HELD + (pass & 1) * GROUPS;
                unsigned *part = tot + HELD + 2 * GROUPS, *bins = part + THREADS;
                const uint4 q = *reinterpret_cast<const uint4 *>(h + PER * tid);
                unsigned v = q.x + q.y + q.z + q.w;
#pragma unroll
                for (int off = 1; off < GROUP_BINS / PER; off <<= 1)
                    v += __shfl_xor_sync(0xffffffffu, v, off);
                if (tid % (GROUP_BINS / PER) == 0)
                    gsum[tid / (GROUP_BINS / PER)] = v;
                tc::cluster_sync();
                const uint32_t ga = smem_u32(gsum + tid % GROUPS);
                v = 0;
                for (int r = tid / GROUPS; r < sel; r += THREADS / GROUPS)
                    v += ld_cluster(tc::cl_map(ga, r));
                part[tid] = v;
                __syncthreads();
                // every warp: lane l has the groups 2l and 2l + 1 from the top
                unsigned g0 = 0, g1 = 0;
#pragma unroll
                for (int r = 0; r < THREADS / GROUPS; ++r) {
                    g0 += part[r * GROUPS + GROUPS - 1 - 2 * lane];
                    g1 += part[r * GROUPS + GROUPS - 2 - 2 * lane];
                }
                unsigned above = warp_above(g0 + g1);
                const bool in0 = above < rem && rem <= above + g0;
                const bool in1 = above + g0 < rem && rem <= above + g0 + g1;
                int src = __ffs(__ballot_sync(0xffffffffu, in0 || in1)) - 1;
                const int group = __shfl_sync(0xffffffffu, GROUPS - 1 - 2 * lane - (in1 ? 1 : 0), src);
                rem -= __shfl_sync(0xffffffffu, above + (in1 ? g0 : 0u), src);
                // warp r fetches CTA r's bins; every warp: lane l has bin l from the top
                if (warp < sel)
                    bins[warp * 32 + lane] = ld_cluster(
                        tc::cl_map(smem_u32(h + group * GROUP_BINS + lane), warp));
                __syncthreads();
                v = 0;
                for (int r = 0; r < sel; ++r)
                    v += bins[r * 32 + 31 - lane];
                above = warp_above(v);
                src = __ffs(__ballot_sync(0xffffffffu, above < rem && rem <= above + v)) - 1;
                rem -= __shfl_sync(0xffffffffu, above, src);
                thr |= static_cast<unsigned>(group * GROUP_BINS + 31 - src) << shift;
            } else {
                unsigned c[PER], sum = 0;         // this thread's bins, from the top
#pragma unroll
                for (int q = 0; q < PER; ++q) {
                    c[q] = h[BINS - 1 - (tid * PER + q)];
                    sum += c[q];
                }
                unsigned above = warp_above(sum);
                if (lane == 31)
                    wsum[warp] = above + sum;
                __syncthreads();
                for (int i = 0; i < warp; ++i)
                    above += wsum[i];
#pragma unroll
                for (int q = 0; q < PER; ++q) {
                    if (above < rem && rem <= above + c[q]) {
                        found[0] = BINS - 1 - (tid * PER + q);
                        found[1] = above;
                    }
                    above += c[q];
                }
                __syncthreads();                  // the bins are read before they are cleared
                thr |= found[0] << shift;
                rem -= found[1];
            }
        }
    }
    // ---- ranks: what the warps before this one keep
    unsigned n_gt = 0, n_eq = 0;
#pragma unroll 4
    for (int t = w0 + lane; t < w1; t += 32) {    // per lane, then over the warp
        const unsigned u = key_at(t);
        n_gt += u > thr;
        n_eq += u == thr;
    }
    n_gt = __reduce_add_sync(0xffffffffu, n_gt);
    n_eq = __reduce_add_sync(0xffffffffu, n_eq);
    if (lane == 0) {
        cnt[warp][0] = n_gt;
        cnt[warp][1] = n_eq;
    }
    if (tid < 2)
        stay[tid] = 0;
    sync_sel();
    unsigned gt = 0, eq = 0;
    for (int i = lane; i < gw; i += 32) {
        const uint32_t a = smem_u32(&cnt[i % WARPS][0]);
        const uint32_t at = sel > 1 ? tc::cl_map(a, i / WARPS) : a;
        gt += ld_cluster(at);
        eq += ld_cluster(at + 4);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        gt += __shfl_xor_sync(0xffffffffu, gt, off);
        eq += __shfl_xor_sync(0xffffffffu, eq, off);
    }
    unsigned at = x.sink + gt + min(eq, rem), n_low = 0, n_fix = 0;
#pragma unroll 4
    for (int t0 = w0; t0 < w1; t0 += 32) {
        const int t = t0 + lane;
        const unsigned u = t < w1 ? key_at(t) : 0u;
        const unsigned eqm = __ballot_sync(0xffffffffu, t < w1 && u == thr);
        const unsigned below = (1u << lane) - 1u;
        const bool keep = t < w1 && (u > thr || (u == thr && eq + __popc(eqm & below) < rem));
        const unsigned km = __ballot_sync(0xffffffffu, keep);
        const unsigned to = at + __popc(km & below);
        if (keep && to < static_cast<unsigned>(x.budget))
            kept[to] = t;                         // solo: the same values by every CTA
        n_low += keep && t < x.budget;
        n_fix += keep && to == static_cast<unsigned>(t);
        at += __popc(km);
        eq += __popc(eqm);
    }
    n_low = __reduce_add_sync(0xffffffffu, n_low);
    n_fix = __reduce_add_sync(0xffffffffu, n_fix);
    if (lane == 0) {
        atomicAdd(&stay[0], n_low);
        atomicAdd(&stay[1], n_fix);
    }
    for (int j = sr * THREADS + tid; j < x.sink; j += sel * THREADS)
        kept[j] = j;
    for (int j = sr * THREADS + tid; j < x.recent; j += sel * THREADS)
        kept[x.budget - x.recent + j] = n - x.recent + j;
    sync_sel();                                   // kept[] is complete

    // kept[] ascends: its first n_fix entries are at their places, its first n_near
    // lie below the budget
    {
        const uint32_t a = smem_u32(stay);
        const bool mine = lane < sel;
        n_low = mine ? ld_cluster(sel > 1 ? tc::cl_map(a, lane) : a) : 0u;
        n_fix = mine ? ld_cluster((sel > 1 ? tc::cl_map(a, lane) : a) + 4) : 0u;
        n_low = __reduce_add_sync(0xffffffffu, n_low);
        n_fix = __reduce_add_sync(0xffffffffu, n_fix);
    }
    const int n_still = x.sink + n_fix;
    const int n_near = x.sink + n_low + min(max(x.budget - (n - x.recent), 0), x.recent);

    // ---- totals that move, in rounds: all of a round's reads before its writes (one
    // round at least: its barrier keeps the CTAs there until all have read the counts)
    for (int j0 = min(n_still, x.budget - 1); j0 < x.budget; j0 += cs * 4 * THREADS) {
        const int r0 = j0 + rank * 4 * THREADS + tid;
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int j = r0 + q * THREADS;
            long long src = -1;
            if (j < x.budget) {
                src = row_of(p, x, b, kv, __ldcg(kept + j));
                if (src < 0)                      // one of the last n_recent
                    flag(FA_STATUS_BAD_BLOCK);
            }
            v[q] = src >= 0 ? __ldcg(x.acc + src) : 0.f;
        }
        sync_all();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int j = r0 + q * THREADS;
            const long long dst = j < x.budget ? row_of(p, x, b, kv, j) : -1;
            if (dst >= 0)
                x.acc[dst] = v[q];
        }
    }
    if (x.fused)
        clear_totals<int>(p, x, b, kv, x.budget + rank * THREADS + tid, cs * THREADS, n);

    // ---- rows of kept tokens below the budget that change their place, in rounds of
    // cs * rows
    const int R = x.rows;
    for (int j0 = n_still; j0 < n_near; j0 += cs * R) {
        const int r0 = j0 + rank * R;
        const int nr = max(min(R, n_near - r0), 0);   // 0 for the last CTAs of the last round
        if (tid < nr) {
            const int j = r0 + tid, t = __ldcg(kept + j);
            const long long s = row_of(p, x, b, kv, t);
            const long long d = s >= 0 ? row_of(p, x, b, kv, j) : -1;
            pl.src[tid] = d >= 0 ? s : -1;
            pl.dst[tid] = d;
        }
        __syncthreads();
        uint32_t off = smem_u32(stage);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            if (!x.a[a])
                continue;
            const int rb = x.row_bytes[a];
            const int lg = 31 - __clz(rb >= 16 ? rb / 16 : 1);
            for (int i = tid; i < nr << lg; i += THREADS) {
                const long long src = pl.src[i >> lg];
                if (src < 0)
                    continue;
                if (rb >= 16)
                    cp<16>(off + i * 16, x.a[a] + src * rb + (i & ((1 << lg) - 1)) * 16);
                else
                    cp<8>(off + i * 8, x.a[a] + src * rb);
            }
            off += R * rb;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        sync_all();                               // every read of the round is done
        off = 0;
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            if (!x.a[a])
                continue;
            const int rb = x.row_bytes[a];
            const int lg = 31 - __clz(rb >= 16 ? rb / 16 : 1);
            for (int i = tid; i < nr << lg; i += THREADS) {
                if (pl.src[i >> lg] < 0)
                    continue;
                char *dst = x.a[a] + pl.dst[i >> lg] * rb;
                if (rb >= 16)
                    reinterpret_cast<uint4 *>(dst)[i & ((1 << lg) - 1)] =
                        *reinterpret_cast<const uint4 *>(stage + off + i * 16);
                else
                    *reinterpret_cast<uint2 *>(dst) =
                        *reinterpret_cast<const uint2 *>(stage + off + i * 8);
            }
            off += R * rb;
        }
        __syncthreads();                          // the stage and the places are free again
    }
    // ---- the others; their places may be sources of the rounds above, all read
    // before the last round's barrier
    if (x.fused) {
        // chunks as long as leave every CTA one: their places cost a chain of loads each
        // (32 ragged sequences, 64 rows at a time: a quarter slower)
        const int F = min(max((x.budget - n_near + cs - 1) / cs, FAR_ROWS), ROUND_ROWS);
        for (int r0 = n_near + rank * F; r0 < x.budget; r0 += cs * F)
            move_far<4>(p, x, b, kv, kept, r0, min(F, x.budget - r0), pl);
    }
}

// The kernel's shared memory and cluster sizes, allowed once per device.
static cudaError_t allow_attributes()
{
    static std::mutex mu;
    static bool done[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 64 && done[dev])
        return cudaSuccess;
    e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             STAGE_BYTES_1);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && dev < 64)
        done[dev] = true;
    return e;
}

// Clusters of cs CTAs with `stage` bytes each that the current device holds at once
// (0 if the query fails), cached per device.
static int cluster_capacity(int cs, int stage)
{
    static std::mutex mu;
    static int cache[64][2][5];
    static bool known[64][2][5] = {};
    int dev = 0;
    if (allow_attributes() != cudaSuccess || cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    const int si = stage == STAGE_BYTES ? 0 : 1, ci = __builtin_ctz(cs);
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 64 && known[dev][si][ci])
        return cache[dev][si][ci];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cs * 64);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = stage;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, evict_kernel, &cfg) != cudaSuccess) {
        n = 0;
        cudaGetLastError();
    }
    if (dev < 64) {
        cache[dev][si][ci] = n;
        known[dev][si][ci] = true;
    }
    return n;
}

}  // namespace ev

cudaError_t evict_take_status(unsigned int *v, cudaStream_t st)
{
    return take_status(v, st);
}

}  // namespace fa

using namespace fa;

extern "C" FA_API int fa_evict_kv(void *k_cache, void *v_cache, void *k_scales, void *v_scales,
                                  float *acc, const int32_t *block_table,
                                  const int32_t *seq_lens, int32_t *new_lens, int32_t *kept,
                                  int budget, int n_sink, int n_recent, int batch,
                                  int n_kv_heads, int head_dim, int page_size,
                                  int max_blocks_per_seq, int num_blocks, void *stream)
{
    const char *name = "fa_evict_kv";
    g_err[0] = 0;
    if (head_dim != 128 && head_dim != 256)
        return fail(FA_ERR_HEAD_DIM, "%s: head_dim %d not supported (128 or 256)", name, head_dim);
    if (n_kv_heads <= 0 || n_kv_heads > 4096)
        return fail(FA_ERR_HEADS, "%s: n_kv_heads %d", name, n_kv_heads);
    if (batch < 0 || batch > 65535)
        return fail(FA_ERR_LAYOUT, "%s: bad batch %d", name, batch);
    if (budget <= 0 || n_sink < 0 || n_recent < 0 || (long long)n_sink + n_recent > budget)
        return fail(FA_ERR_LAYOUT, "%s: budget %d must be positive and hold n_sink %d and "
                                   "n_recent %d", name, budget, n_sink, n_recent);
    if (batch == 0)                          // a no-op: empty arrays may have no pointer
        return 0;
    if (!k_cache || !v_cache || !acc || !seq_lens || !new_lens || !kept)
        return fail(FA_ERR_NULL, "%s: only block_table and the scales may be NULL", name);
    if (k_scales && !v_scales)
        return fail(FA_ERR_NULL, "%s: k_scales (a 4-bit cache) without v_scales", name);
    const bool paged = block_table != nullptr;
    if (max_blocks_per_seq <= 0 ||
        (paged && (page_size <= 0 || page_size % 16 || num_blocks <= 0)))
        return fail(FA_ERR_LAYOUT, "%s: bad capacity, page size or block count", name);
    const long long cap = paged ? (long long)max_blocks_per_seq * page_size
                                : (long long)max_blocks_per_seq;
    if (cap > (1ll << 30))
        return fail(FA_ERR_LAYOUT, "%s: capacity %lld tokens too large", name, cap);
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scales) ||
        !aligned16(v_scales) || !aligned_to(acc, 4) || !aligned_to(seq_lens, 4) ||
        !aligned_to(new_lens, 4) || !aligned_to(kept, 4) || !aligned_to(block_table, 4))
        return fail(FA_ERR_ALIGN, "%s: caches and scales must be 16-byte aligned, acc and int32 "
                                  "arrays 4-byte aligned", name);
    const size_t kv_rows = (paged ? (size_t)num_blocks * page_size : (size_t)batch * cap) *
                           n_kv_heads;
    const int D = head_dim;
    ev::Args x = {};
    x.a[0] = static_cast<char *>(k_cache);
    x.a[1] = static_cast<char *>(v_cache);
    x.a[2] = static_cast<char *>(k_scales);
    x.a[3] = static_cast<char *>(v_scales);
    x.row_bytes[0] = k_scales ? D / 2 : 2 * D;
    x.row_bytes[1] = k_scales ? D / 2 : v_scales ? D : 2 * D;
    x.row_bytes[2] = x.row_bytes[3] = D / 16;
    x.acc = acc;
    x.new_lens = new_lens;
    x.kept = kept;
    x.budget = budget;
    x.sink = n_sink;
    x.recent = n_recent;
    const struct { const void *p; size_t n; } io[] = {
        {x.a[0], kv_rows * x.row_bytes[0]}, {x.a[1], kv_rows * x.row_bytes[1]},
        {x.a[2], kv_rows * x.row_bytes[2]}, {x.a[3], kv_rows * x.row_bytes[3]},
        {acc, kv_rows * 4}, {new_lens, (size_t)batch * 4},
        {kept, (size_t)batch * n_kv_heads * budget * 4},
        {seq_lens, (size_t)batch * 4}, {block_table, (size_t)batch * max_blocks_per_seq * 4}};
    for (int i = 0; i < 9; ++i)
        for (int j = 0; j < i && j < 7; ++j)
            if (overlaps(io[i].p, io[i].n, io[j].p, io[j].n))
                return fail(FA_ERR_ALIAS, "%s: two arrays overlap", name);
    int total = 0;
    for (int a = 0; a < 4; ++a)
        total += x.a[a] ? x.row_bytes[a] : 0;
    x.lg_page = log2_of(page_size);
    Params p = {};
    p.bt = block_table;
    p.seq_lens = seq_lens;
    p.B = batch;
    p.Hkv = n_kv_heads;
    p.page_size = paged ? page_size : 16;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.cap = cap;
    const long long units = (long long)batch * n_kv_heads;
    // The largest cluster for which every unit's is resident at once, but none larger
    // than stages the whole budget in one round (more CTAs only add to the
    // barriers).  16 CTAs with the smaller stage come before 8 with the larger: the
    // same rows per round, and twice the CTAs to select with.
    int cs = 1, stage = ev::STAGE_BYTES;
    const long long round = ev::STAGE_BYTES / total;
    int most = ev::MAX_CTAS;
    while (most > 1 && round * (most / 2) >= budget)
        most /= 2;
    for (int c = most; c >= 2 && cs == 1; c /= 2)
        for (int st : {ev::STAGE_BYTES_1, ev::STAGE_BYTES})
            if (cs == 1 && (st == ev::STAGE_BYTES || c >= 8) &&
                units <= ev::cluster_capacity(c, st)) {
                cs = c;
                stage = st;
            }
    p.cl_ctas = cs;
    // One kernel when there is little to move, or when the clusters fill the GPU anyway:
    // 32 ragged sequences x 8 heads, a tenth slower with the far rows in a second.
    int sms = 0;
    if (const int rc = device_sms(&sms))
        return rc;
    // (A budget that no sequence can exceed moves nothing: the second kernel may rely on
    // budgets of less than 2^30.)
    x.fused = budget >= cap || (double)units * budget * total <= ev::FUSED_BYTES ||
              units * cs >= sms;
    x.rows = stage / total / 16 * 16;
    if (x.rows > ev::ROUND_ROWS)
        x.rows = ev::ROUND_ROWS;
    const long long far_chunks = (budget + (long long)ev::FAR_ROWS - 1) / ev::FAR_ROWS;
    if (units * cs > 0x7fffffffll || (!x.fused && units * far_chunks > 0x7fffffffll))
        return fail(FA_ERR_LAYOUT, "%s: too many rows", name);
    cudaError_t e = ev::allow_attributes();
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(units * cs));
        cfg.blockDim = dim3(ev::THREADS);
        cfg.dynamicSmemBytes = stage;
        cfg.stream = static_cast<cudaStream_t>(stream);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = cs;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, ev::evict_kernel, p, x);
        if (e == cudaSuccess)
            e = cudaGetLastError();
    }
    if (e == cudaSuccess && !x.fused) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(units * far_chunks));
        cfg.blockDim = dim3(ev::FAR_THREADS);
        cfg.stream = static_cast<cudaStream_t>(stream);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, ev::evict_far_kernel, p, x);
        if (e == cudaSuccess)
            e = cudaGetLastError();
    }
    if (e != cudaSuccess)
        return fail(FA_ERR_CUDA, "%s: launch failed: %s", name, cudaGetErrorString(e));
    return 0;
}
