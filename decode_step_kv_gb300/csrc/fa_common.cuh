// fa_common.cuh -- what the translation units of the library share: call
// parameters, PTX wrappers, ranges and paging, the walk over a step's tiles,
// the (query, head) columns of a unit, the log-sum-exp merge of split partials
// and the host checks.
#ifndef FA_COMMON_CUH
#define FA_COMMON_CUH

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <mutex>
#include <type_traits>
#include <utility>
#include <stdlib.h>

#include "../../include/fa_decode.h"

namespace fa {

constexpr unsigned long long WAIT_NS = 1000000000ull;  // ~1 s bound on any wait

// Device-side status bits of this translation unit's kernels
// (fa_decode_device_status collects every unit's).
static __device__ unsigned int g_status;

struct Params {
    const __half *q;
    const char *k;
    const char *v;
    const char *vs;
    const char *ks;   // 4-bit cache: K scales
    const int *bt;
    const int *seq_lens;
    const int *window;
    float *out;
    float *ws_o;      // [B*Hq][max_splits][D]
    float2 *ws_ml;    // [B*Hq][max_splits] (m, l), m in log2 units
    int B, Hq, Hkv, G, n_hg, hpg;
    int page_size, max_blocks, num_blocks;
    long long cap;    // tokens per sequence
    float c2;         // scale * log2(e)
    int tile;         // tokens per tile
    int tps;          // tiles per split (split kernels)
    int max_splits;
    int ring;         // contiguous ring cache: token t at row t % cap, lengths unbounded
    int tq;           // queries per sequence (multi-query decode); 1 = one
    int W;            // stream-K workers (warps) in the grid
    int U_b;          // units per sequence: kv heads x head groups
    int sh;           // heads stored per workspace slot (stream-K)
    long long *pref;  // stream-K, more than 32*SCAN_REG sequences: [B+1] flattened
                      // start tile of each sequence (last entry: all tiles)
    int cpu;          // tensor-core kernel: (query, head) columns per unit, 8 or 16
    int chunk;        // batch-invariant plan: tiles per chunk (0: stream-K plan)
    int max_chunks;   // batch-invariant plan: chunk slots per unit
    const int *slot;  // contiguous / ring caches: sequence b's cache is slot slot[b] of
                      // [n_slots][Hkv][cap][D]; NULL: slot b
    int n_slots;
    int cl_ctas;      // cluster plan: CTAs per cluster (1, 2, 4 or 8)
    float *lse;       // recorded weights: [B*tq*Hq] log2-sum-exp2 of each row (-inf: no key)
    float *ws_s;      // recorded weights: scores in log2 units, of units of up to 16 columns
                      // [B*units][cap16][sh], of wider ones [B*units][cap16/16][sh][16 keys]
    float *acc;       // recorded weights: the running total of every cache row
    long long cap16;  // recorded weights: capacity rounded up to whole tiles
    int lg_page;      // recorded weights: log2 of page_size, or -1
    int w_rounds;     // recorded weights: rounds of WEIGHT_KEYS keys per item
};

// ------------------------------------------------------------ PTX wrappers
__device__ __forceinline__ uint32_t smem_u32(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint32_t bar, unsigned count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ unsigned long long global_ns()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Warp-uniform bounded wait on a stage's phase.  Returns false after ~1 s.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
        return true;
    const unsigned long long t0 = global_ns();
    for (;;) {
        for (int i = 0; i < 256; ++i)
            if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
                return true;
        if (global_ns() - t0 > WAIT_NS)
            return false;
    }
}

__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void *src, uint32_t bytes,
                                         uint32_t bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1], %2, [%3], %4;" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

__device__ __forceinline__ uint64_t evict_first_policy()
{
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float ex2_ftz(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Of a kernel launched while the one before it may still run: waits until that one has
// finished and its writes can be read.  Every CTA of such a kernel gets here before it ends,
// those without anything to read too: what follows on the stream waits for this kernel alone,
// and must find both done.
__device__ __forceinline__ void wait_for_previous()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void flag(unsigned bit)
{
    atomicOr(&g_status, bit);
}

// --------------------------------------------------------- range and paging
// Attended key range [lo, hi) of sequence b (length clamped to capacity).
__device__ __forceinline__ void attended_range(const Params &p, int b, int &lo, int &hi,
                                               bool report)
{
    long long L = p.seq_lens[b];
    if (L < 0 || (!p.ring && L > p.cap) || L > 0x7fffffffll) {
        if (report)
            flag(FA_STATUS_LEN_CLAMPED);
        L = L < 0 ? 0 : (p.ring ? 0x7fffffffll : p.cap);
    }
    const int W = p.window ? p.window[b] : 0;
    hi = static_cast<int>(L);
    // with tq queries (the last tq tokens) the window of the first one starts
    // earliest; each query's own range is masked inside the kernel
    const int first_end = hi - (p.tq > 1 ? p.tq - 1 : 0);
    lo = (W > 0 && first_end > W) ? first_end - W : 0;
    // a ring cache holds only the last cap tokens (live length min(N, cap))
    if (p.ring && (long long)hi - p.cap > lo)
        lo = static_cast<int>(hi - p.cap);
    // a slot id that names no cache slot: nothing to attend (a zero row)
    if (p.slot) {
        const int s = p.slot[b];
        if (s < 0 || s >= p.n_slots) {
            if (report)
                flag(FA_STATUS_BAD_SLOT);
            lo = hi = 0;
        }
    }
}

// Cache slot of sequence b in a contiguous or ring cache (the slot map, or b).
__device__ __forceinline__ long long cache_slot(const Params &p, int b)
{
    return p.slot ? p.slot[b] : b;
}

template <int TILE>
__device__ __forceinline__ int tiles_in(int lo, int hi)
{
    return hi > lo ? (hi - 1) / TILE - lo / TILE + 1 : 0;
}

// Byte offset of token `tok` (a tile start) of (b, kv) in a cache whose rows
// hold `row_bytes`; -1 when the block id is out of range.
__device__ __forceinline__ long long row_offset(const Params &p, int b, int kv, int tok,
                                                int row_bytes)
{
    if (p.bt) {
        const long long blk = p.bt[(long long)b * p.max_blocks + tok / p.page_size];
        if (blk < 0 || blk >= p.num_blocks)
            return -1;
        return ((blk * p.Hkv + kv) * p.page_size + tok % p.page_size) * (long long)row_bytes;
    }
    const long long r = p.ring ? tok % p.cap : tok;
    return ((cache_slot(p, b) * p.Hkv + kv) * p.cap + r) * (long long)row_bytes;
}

namespace tc {

constexpr int TILE = 16;
constexpr int GPH = 8;          // heads per unit (the mma N dimension)

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            uint32_t bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2,
                                        uint32_t &r3)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t &r0, uint32_t &r1,
                                          uint32_t &r2, uint32_t &r3)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Four int8 codes -> two half2 of code * scale.  Each biased byte u = code +
// 128 becomes the fp16 1024 + u by placing it under the exponent byte 0x64;
// subtracting 1152 gives the code exactly, and one fp16 multiply by the scale
// rounds the product once (code * scale has at most 18 significant bits).
__device__ __forceinline__ void dequant4(uint32_t w, __half2 s2, uint32_t &lo, uint32_t &hi)
{
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140);
    const uint32_t b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 bias = __half2half2(__ushort_as_half((unsigned short)0x6480));   // 1152
    __half2 ha = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&a), bias), s2);
    __half2 hb = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&b), bias), s2);
    lo = *reinterpret_cast<const uint32_t *>(&ha);
    hi = *reinterpret_cast<const uint32_t *>(&hb);
}

// Shared address of 16-byte chunk `chunk` (0..D/8-1) of tile row `row` in a
// tile of BOXES swizzled 64-column boxes.
__device__ __forceinline__ uint32_t swz(uint32_t base, int row, int chunk)
{
    const int box = chunk >> 3;
    const int c = (chunk & 7) ^ (row & 7);
    return base + box * (TILE * 128) + row * 128 + c * 16;
}

// Distributed shared memory: the address of shared location `local` (an
// address in this CTA's window) in cluster CTA `rank`, and loads from it.
__device__ __forceinline__ uint32_t cl_map(uint32_t local, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
__device__ __forceinline__ float2 cl_ld2(uint32_t a)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a)
                 : "memory");
    return v;
}
__device__ __forceinline__ float4 cl_ld4(uint32_t a)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
// Every thread of every CTA of the cluster: writes before the barrier are
// visible to the cluster's reads after it.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Tile row coordinate (the tensor maps view K and V as [rows][D]); -1 for a
// block id out of range.
__device__ __forceinline__ long long tile_row(const Params &p, int b, int kv, int tok)
{
    if (p.bt) {
        const long long blk = p.bt[(long long)b * p.max_blocks + tok / p.page_size];
        if (blk < 0 || blk >= p.num_blocks)
            return -1;
        return (blk * p.Hkv + kv) * p.page_size + tok % p.page_size;
    }
    return (cache_slot(p, b) * p.Hkv + kv) * p.cap + (p.ring ? tok % p.cap : tok);
}

// Per-sequence walk over the flattened tile space.  Units (one KV head and
// head group of one sequence) are ordered by (sequence, unit); the tiles of
// a unit are its 16-token tiles intersecting the attended range [lo, hi).
//
// The stream-K plan charges each unit's start UNIT_COST tiles of work (the
// query load and the partial write a worker pays on entering a new unit):
// a unit takes n + UNIT_COST positions of the flattened space that workers
// split evenly, UNIT_COST empty ones then its n tiles, so a worker whose
// range crosses into a new unit gets that many fewer tiles.  Position of
// tile k of unit j of sequence b: P_b + j*(n_b + c) + c + k, with c =
// UNIT_COST (stream-K plan) or 0 (batch-invariant plan, which cuts real
// tiles).
#ifndef FA_UNIT_COST
#define FA_UNIT_COST 2
#endif
constexpr int UNIT_COST = FA_UNIT_COST;

// Flattened positions sequence b takes in the stream-K plan: its units x
// (n + UNIT_COST), none when it has no tiles.
__device__ __forceinline__ long long seq_span(const Params &p, int n)
{
    return n > 0 ? (long long)(n + UNIT_COST) * p.U_b : 0;
}

struct Walk {
    int b, j, k, n, lo, hi;   // sequence, unit in sequence, tile in unit, tiles per unit
    int c;                    // empty positions before each unit's tiles
    long long P;              // flattened position of sequence b's first unit

    __device__ __forceinline__ void load(const Params &p)
    {
        attended_range(p, b, lo, hi, false);
        n = tiles_in<TILE>(lo, hi);
    }
    // position at the first tile at or after flattened position t of
    // sequence b_ (whose first unit starts at P_)
    __device__ __forceinline__ void init(const Params &p, int b_, long long P_, long long t,
                                         int c_)
    {
        b = b_;
        P = P_;
        c = c_;
        load(p);
        const long long off = t - P;
        j = static_cast<int>(off / (n + c));
        const int r = static_cast<int>(off % (n + c));
        k = r < c ? 0 : r - c;
    }
    __device__ __forceinline__ void next(const Params &p)
    {
        if (++k < n)
            return;
        k = 0;
        if (++j < p.U_b)
            return;
        j = 0;
        do {
            if (n > 0)
                P += (long long)p.U_b * (n + c);
            ++b;
            if (b >= p.B)
                return;
            load(p);
        } while (n == 0);
    }
    __device__ __forceinline__ int tok() const { return (lo / TILE + k) * TILE; }
    __device__ __forceinline__ long long unit(const Params &p) const
    {
        return (long long)b * p.U_b + j;
    }
    // flattened position of the unit's first tile, and of the current tile
    __device__ __forceinline__ long long unit_start() const
    {
        return P + (long long)j * (n + c) + c;
    }
    __device__ __forceinline__ long long pos() const { return unit_start() + k; }
};

// Warp-cooperative scan over the sequences: T = the flattened positions of
// the step (tiles plus UNIT_COST per unit); when target >= 0 also the
// sequence holding position `target` and that sequence's first position;
// when want >= 0 also sequence want's first position and tile count.
// Every lane returns the same values.
__device__ __forceinline__ long long flat_scan(const Params &p, long long target, int &b_at,
                                               long long &P_at, bool report = false,
                                               long long *pref = nullptr, int want = -1,
                                               long long *P_want = nullptr,
                                               int *n_want = nullptr)
{
    const int lane = threadIdx.x & 31;
    long long run = 0;
    b_at = -1;
    P_at = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        long long c = 0;
        int nt = 0;
        if (b < p.B) {
            int lo, hi;
            attended_range(p, b, lo, hi, report);
            nt = tiles_in<TILE>(lo, hi);
            c = seq_span(p, nt);
        }
        long long x = c;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off)
                x += y;
        }
        const long long excl = run + x - c;
        if (pref && b < p.B)
            pref[b] = excl;
        if (want >= b0 && want < b0 + 32) {       // warp-uniform
            *P_want = __shfl_sync(0xffffffffu, excl, want - b0);
            *n_want = __shfl_sync(0xffffffffu, nt, want - b0);
        }
        if (target >= 0 && b_at < 0) {
            const unsigned hit = __ballot_sync(0xffffffffu, b < p.B && target >= excl &&
                                                                target < excl + c);
            if (hit) {
                const int src = __ffs(hit) - 1;
                b_at = b0 + src;
                P_at = __shfl_sync(0xffffffffu, excl, src);
            }
        }
        run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (pref && lane == 0)
        pref[p.B] = run;
    return run;
}

// Batch-invariant plan: each unit's tiles are cut into chunks of p.chunk
// tiles counted from its first attended tile, and workers take equal
// contiguous ranges of whole chunks in (sequence, unit, chunk) order, so what
// each chunk computes depends on its own sequence alone.  Warp-cooperative
// scan over the sequences: returns the step's chunks and, through *tiles, its
// tiles; when target >= 0 also the sequence holding flattened chunk `target`
// (b_at), that sequence's first flattened tile (P_at) and first flattened
// chunk (Pc_at).  Every lane returns the same values.
__device__ __forceinline__ long long chunk_scan(const Params &p, long long target,
                                                long long *tiles, int &b_at, long long &P_at,
                                                long long &Pc_at, bool report)
{
    const int lane = threadIdx.x & 31;
    long long run_t = 0, run_c = 0;
    b_at = -1;
    P_at = 0;
    Pc_at = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        long long ct = 0, cc = 0;
        if (b < p.B) {
            int lo, hi;
            attended_range(p, b, lo, hi, report);
            const int n = tiles_in<TILE>(lo, hi);
            ct = (long long)n * p.U_b;
            cc = (long long)((n + p.chunk - 1) / p.chunk) * p.U_b;
        }
        long long xt = ct, xc = cc;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long yt = __shfl_up_sync(0xffffffffu, xt, off);
            const long long yc = __shfl_up_sync(0xffffffffu, xc, off);
            if (lane >= off) {
                xt += yt;
                xc += yc;
            }
        }
        const long long et = run_t + xt - ct, ec = run_c + xc - cc;
        if (target >= 0 && b_at < 0) {
            const unsigned hit =
                __ballot_sync(0xffffffffu, b < p.B && target >= ec && target < ec + cc);
            if (hit) {
                const int src = __ffs(hit) - 1;
                b_at = b0 + src;
                P_at = __shfl_sync(0xffffffffu, et, src);
                Pc_at = __shfl_sync(0xffffffffu, ec, src);
            }
        }
        run_t += __shfl_sync(0xffffffffu, xt, 31);
        run_c += __shfl_sync(0xffffffffu, xc, 31);
    }
    if (tiles)
        *tiles = run_t;
    return run_c;
}

// Flattened tile index of chunk `off` of sequence b (whose first tile is P).
__device__ __forceinline__ long long chunk_tile(const Params &p, int b, long long P, long long off)
{
    int lo, hi;
    attended_range(p, b, lo, hi, false);
    const int n = tiles_in<TILE>(lo, hi);
    const int nch = (n + p.chunk - 1) / p.chunk;
    const long long j = off / nch;
    return P + j * n + (off - j * nch) * p.chunk;
}

// Workers actually used for T tiles (at least MIN_TPW tiles each), and the
// worker whose contiguous range holds flattened tile t.
#ifndef FA_MIN_TPW
#define FA_MIN_TPW 1
#endif
constexpr int MIN_TPW = FA_MIN_TPW;   // fewest tiles a stream-K worker is given
constexpr int SCAN_REG = 4;     // sequences per lane kept in registers by the one-pass scan
__device__ __forceinline__ int workers_for(const Params &p, long long T)
{
    long long w = T / MIN_TPW;
    if (w < 1)
        w = 1;
    return static_cast<int>(w < p.W ? w : p.W);
}
__device__ __forceinline__ long long range_start(long long w, long long T, int We)
{
    return w * T / We;
}
__device__ __forceinline__ int worker_of(long long t, long long T, int We)
{
    return static_cast<int>(((t + 1) * We - 1) / T);
}

// Stream-K plan: worker w's flattened positions [t0, t1), with T and We of the
// step and the sequence holding t0 (b_at) and its first position (P_at).
// Warp-cooperative; false when the worker has nothing to do.
__device__ __forceinline__ bool stream_range(const Params &p, int w, long long &T, int &We,
                                             long long &t0, long long &t1, int &b_at,
                                             long long &P_at)
{
    const int lane = threadIdx.x & 31;
    if (p.B <= 32 * SCAN_REG) {
        // one pass: each lane keeps the tile counts of its sequences
        // (b = lane + 32 i) in registers, then locates t0 from them
        long long c[SCAN_REG], x[SCAN_REG], base[SCAN_REG];
        long long run = 0;
        const int nblk = (p.B + 31) / 32;       // blocks of 32 sequences in use
#pragma unroll
        for (int i = 0; i < SCAN_REG; ++i) {
            const int b = lane + 32 * i;
            c[i] = 0;
            x[i] = 0;
            base[i] = run;
            if (i >= nblk)                       // warp-uniform: nothing left to scan
                continue;
            if (b < p.B) {
                int lo, hi;
                attended_range(p, b, lo, hi, w == 0);   // worker 0 reports clamped lengths
                c[i] = seq_span(p, tiles_in<TILE>(lo, hi));
            }
            x[i] = c[i];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x[i], off);
                if (lane >= off)
                    x[i] += y;
            }
            run += __shfl_sync(0xffffffffu, x[i], 31);
        }
        T = run;
        if (T == 0)
            return false;
        We = workers_for(p, T);
        if (w >= We)
            return false;
        t0 = range_start(w, T, We);
        t1 = range_start(w + 1, T, We);
#pragma unroll
        for (int i = 0; i < SCAN_REG; ++i) {
            if (i >= nblk || b_at >= 0)
                continue;
            const long long excl = base[i] + x[i] - c[i];
            const unsigned hit =
                __ballot_sync(0xffffffffu, c[i] > 0 && t0 >= excl && t0 < excl + c[i]);
            if (hit) {
                const int src = __ffs(hit) - 1;
                b_at = 32 * i + src;
                P_at = __shfl_sync(0xffffffffu, excl, src);
            }
        }
    } else {
        // worker 0 also publishes each sequence's flattened start for the merge
        T = flat_scan(p, -1, b_at, P_at, w == 0, w == 0 ? p.pref : nullptr);
        if (T == 0)
            return false;
        We = workers_for(p, T);
        if (w >= We)
            return false;
        t0 = range_start(w, T, We);
        t1 = range_start(w + 1, T, We);
        flat_scan(p, t0, b_at, P_at);
    }
    return true;
}

// Column c (0..cpu-1) of column group cg of KV head kv, with cpu columns per
// unit: the (query j, head h) pair x = cg*cpu + c = j*G + g (head-fastest);
// live while x < tq*G.  With one query the columns are the KV head's query
// heads.
struct Col {
    bool live;
    int j;    // query index within the sequence
    int h;    // query head
};
__device__ __forceinline__ Col column(const Params &p, int kv, int cg, int c, int cpu)
{
    const int tq = p.tq > 1 ? p.tq : 1;
    const int x = cg * cpu + c;
    Col r;
    r.live = x < tq * p.G;
    r.j = x / p.G;
    r.h = kv * p.G + x % p.G;
    return r;
}

// Keys [lo, hi) column (query j) of sequence b attends: up to and including
// its own position L - tq + j, the window counted back from there.
__device__ __forceinline__ void column_range(const Params &p, int b, int L, int j, int &lo,
                                             int &hi)
{
    const int tq = p.tq > 1 ? p.tq : 1;
    hi = max(L - (tq - 1 - j), 0);
    const int W = p.window ? p.window[b] : 0;
    lo = (W > 0 && hi > W) ? hi - W : 0;
    if (p.ring && (long long)L - p.cap > lo)
        lo = static_cast<int>(L - p.cap);
}

// Log-sum-exp merge for the stream-K kernel: one CTA of MERGE_THREADS per
// (sequence, query head) row folds the partial slots of the workers that
// covered the row's unit (or writes the zero row of an empty range).  The
// slots are spread over the threads: each thread owns one float4 column of
// D and a strided subset of the slots, so the loads of many slots are in
// flight at once; the per-slot weights ex2(m - M) are computed once into
// shared memory.
constexpr int MERGE_THREADS = 256;
// rows per SM from which the stream-K merge takes a warp per row
#ifndef FA_MERGE_WARP_ROWS_PER_SM
#define FA_MERGE_WARP_ROWS_PER_SM 4
#endif
// slots per row whose partial O the merge loads into registers up front
#ifndef FA_MERGE_REG_SLOTS_128
#define FA_MERGE_REG_SLOTS_128 32
#endif
#ifndef FA_MERGE_REG_SLOTS_256
#define FA_MERGE_REG_SLOTS_256 64
#endif
constexpr int MERGE_MAX_SLOTS = 512;   // per pass over the slots

// Four consecutive output values, as fp32 or rounded to fp16.
__device__ __forceinline__ void store4(float *dst, float4 v)
{
    *reinterpret_cast<float4 *>(dst) = v;
}
__device__ __forceinline__ void store4(__half *dst, float4 v)
{
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_half2(v.x, v.y), pack_half2(v.z, v.w));
}

// One output row, by a CTA of MERGE_THREADS.  OutT: float, or __half for the entry
// points whose output is fp16.
template <int D, bool BI, typename OutT>
__device__ __forceinline__ void merge_row(const Params &p, const long long row)
{
    constexpr int CH = D / 4;                    // float4 columns
    constexpr int SG = MERGE_THREADS / CH;       // slot groups
    __shared__ float wgt[MERGE_MAX_SLOTS];
    __shared__ float red[MERGE_THREADS / 32];
    __shared__ float4 part[SG][CH];

    // row = (b * tq + query) * Hq + head; its column x = query * G + head % G
    const int tq = p.tq > 1 ? p.tq : 1;
    const int b = static_cast<int>(row / ((long long)tq * p.Hq));
    const int qj = static_cast<int>((row / p.Hq) % tq);
    const int h = static_cast<int>(row % p.Hq);
    const int kv = h / p.G;
    const int x = qj * p.G + h % p.G;
    const int j = kv * p.n_hg + x / p.cpu;
    const int hh = x % p.cpu;
    const int tid = threadIdx.x;
    const int lane = tid & 31, wid = tid >> 5;

    const long long u = (long long)b * p.U_b + j;
    long long sb;    // workspace slot of the row's first partial
    int ns;          // partials to fold, in slot order
    int n;           // tiles of the row's sequence
    auto zero_row = [&] {
        if (tid < CH)
            store4(reinterpret_cast<OutT *>(p.out) + row * D + 4 * tid,
                   make_float4(0.f, 0.f, 0.f, 0.f));
    };
    if constexpr (BI) {
        int lo, hi;
        attended_range(p, b, lo, hi, false);
        n = tiles_in<TILE>(lo, hi);
        if (n == 0) {
            zero_row();
            return wait_for_previous();
        }
        // batch-invariant plan: the unit's chunks, one slot each
        ns = (n + p.chunk - 1) / p.chunk;
        wait_for_previous();
        if (ns == 1)
            return;                               // written by the split kernel
        sb = u * p.max_chunks;
    } else {
        // T, and the flattened start and tiles of sequence b: one warp's
        // single pass over the lengths for up to 32*SCAN_REG sequences
        // (before the dependency wait, so it overlaps the split kernel's tail
        // where the CTA is resident by then), else published by the split
        // kernel's worker 0
        __shared__ long long sh_T, sh_P;
        __shared__ int sh_n;
        const bool scan_here = p.B <= 32 * SCAN_REG;
        if (scan_here) {
            if (wid == 0) {
                int b_at, nb = 0;
                long long P_at, Pb = 0;
                const long long T = flat_scan(p, -1, b_at, P_at, false, nullptr, b, &Pb, &nb);
                if (lane == 0) {
                    sh_T = T;
                    sh_P = Pb;
                    sh_n = nb;
                }
            }
            __syncthreads();
            n = sh_n;
        } else {
            int lo, hi;
            attended_range(p, b, lo, hi, false);
            n = tiles_in<TILE>(lo, hi);
        }
        if (n == 0) {                             // uniform over the CTA
            zero_row();
            return wait_for_previous();
        }
        if (!scan_here) {
            wait_for_previous();
            if (tid == 0) {
                sh_T = p.pref[p.B];
                sh_P = p.pref[b];
            }
            __syncthreads();
        }
        const long long T = sh_T;
        const int We = workers_for(p, T);
        const long long us = sh_P + (long long)j * (n + UNIT_COST) + UNIT_COST;   // first tile
        const int wf = worker_of(us, T, We);
        const int wl = worker_of(us + n - 1, T, We);
        if (scan_here)
            wait_for_previous();
        if (wf == wl)
            return;                               // written by the split kernel
        sb = wf + u;
        ns = wl - wf + 1;
    }

    const int c = tid % CH;
    const int sg = tid / CH;
    // this thread's O columns of its slots (sg, sg + SG, ...): when they fit
    // in registers they are loaded before the (m, l) pairs, so both loads are
    // in flight together and the weights arrive to find them there
    constexpr int OR = (D == 128 ? FA_MERGE_REG_SLOTS_128 : FA_MERGE_REG_SLOTS_256) / SG;
    const bool in_regs = OR > 0 && ns <= SG * OR;
    float4 ov[OR > 0 ? OR : 1];
    if (in_regs) {
#pragma unroll
        for (int k = 0; k < OR; ++k) {
            const int s = sg + k * SG;
            ov[k] = s < ns ? reinterpret_cast<const float4 *>(
                                 p.ws_o + ((sb + s) * p.sh + hh) * D)[c]
                           : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    // (m, l) of the slots: loaded once per thread (one slot per thread per
    // pass of MERGE_THREADS), reduced to M, turned into weights in shared memory
    float L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY;
    float2 mine = make_float2(-INFINITY, 0.f);
    if (ns <= MERGE_THREADS) {
        if (tid < ns)
            mine = p.ws_ml[(sb + tid) * p.sh + hh];
        M = mine.x;
    } else {
        for (int s = tid; s < ns; s += MERGE_THREADS)
            M = fmaxf(M, p.ws_ml[(sb + s) * p.sh + hh].x);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    if (lane == 0)
        red[wid] = M;
    __syncthreads();
    M = red[0];
#pragma unroll
    for (int i = 1; i < MERGE_THREADS / 32; ++i)
        M = fmaxf(M, red[i]);
    __syncthreads();

    for (int s0 = 0; s0 < ns; s0 += MERGE_MAX_SLOTS) {
        const int cnt = min(MERGE_MAX_SLOTS, ns - s0);
        float Lp = 0.f;
        for (int s = tid; s < cnt; s += MERGE_THREADS) {
            const float2 v = (ns <= MERGE_THREADS) ? mine : p.ws_ml[(sb + s0 + s) * p.sh + hh];
            const float a = (v.x == -INFINITY) ? 0.f : ex2(v.x - M);
            wgt[s] = a;
            Lp = fmaf(v.y, a, Lp);
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            Lp += __shfl_xor_sync(0xffffffffu, Lp, off);
        if (lane == 0)
            red[wid] = Lp;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MERGE_THREADS / 32; ++i)
            L += red[i];
        if (in_regs) {
#pragma unroll
            for (int k = 0; k < OR; ++k) {
                const int s = sg + k * SG;
                if (s < cnt) {
                    const float a = wgt[s];
                    o.x = fmaf(ov[k].x, a, o.x);
                    o.y = fmaf(ov[k].y, a, o.y);
                    o.z = fmaf(ov[k].z, a, o.z);
                    o.w = fmaf(ov[k].w, a, o.w);
                }
            }
        } else
#pragma unroll 4
        for (int s = sg; s < cnt; s += SG) {
            const long long slot = sb + s0 + s;
            const float4 x =
                reinterpret_cast<const float4 *>(p.ws_o + (slot * p.sh + hh) * D)[c];
            const float a = wgt[s];
            o.x = fmaf(x.x, a, o.x);
            o.y = fmaf(x.y, a, o.y);
            o.z = fmaf(x.z, a, o.z);
            o.w = fmaf(x.w, a, o.w);
        }
        __syncthreads();
    }
    part[sg][c] = o;
    __syncthreads();
    if (sg == 0) {
#pragma unroll
        for (int g = 1; g < SG; ++g) {
            const float4 y = part[g][c];
            o.x += y.x;
            o.y += y.y;
            o.z += y.z;
            o.w += y.w;
        }
        const float inv = L > 0.f ? 1.f / L : 0.f;
        store4(reinterpret_cast<OutT *>(p.out) + row * D + 4 * c,
               make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    }
}

template <int D, bool BI, typename OutT = float>
__global__ void __launch_bounds__(MERGE_THREADS) fa_stream_merge_kernel(const Params p)
{
    merge_row<D, BI, OutT>(p, blockIdx.x);
}

// Warp-per-row form of the stream-K merge, for steps with many rows (the
// host picks it at four or more rows per SM): eight rows per CTA, so the
// grid runs in fewer, fuller waves and every row's length scan is one warp's
// work.  Each lane owns D/128 float4 columns of the row; the slots' weights
// are computed 32 at a time, one per lane, and broadcast by shuffles while
// the partial O columns stream in.  The fold runs in slot order.
constexpr int MERGE_ROWS_PER_CTA = 8;

template <int D, typename OutT>
__device__ __forceinline__ void merge_rows(const Params &p, const int cta)
{
    constexpr int CPL = D / 128;                 // float4 columns per lane
    const int lane = threadIdx.x & 31;
    const int tq = p.tq > 1 ? p.tq : 1;
    const long long rows = (long long)p.B * tq * p.Hq;
    const long long row = (long long)cta * MERGE_ROWS_PER_CTA + (threadIdx.x >> 5);
    if (row >= rows)
        return wait_for_previous();
    // row = (b * tq + query) * Hq + head; its column x = query * G + head % G
    const int b = static_cast<int>(row / ((long long)tq * p.Hq));
    const int qj = static_cast<int>((row / p.Hq) % tq);
    const int h = static_cast<int>(row % p.Hq);
    const int kv = h / p.G;
    const int x = qj * p.G + h % p.G;
    const int j = kv * p.n_hg + x / p.cpu;
    const int hh = x % p.cpu;
    OutT *dst = reinterpret_cast<OutT *>(p.out) + row * D;

    // T, and the flattened start and tiles of sequence b (as in
    // fa_stream_merge_kernel)
    long long T = 0, P = 0;
    int n = 0;
    const bool scan_here = p.B <= 32 * SCAN_REG;
    if (scan_here) {
        int b_at;
        long long P_at;
        T = flat_scan(p, -1, b_at, P_at, false, nullptr, b, &P, &n);
    } else {
        int lo, hi;
        attended_range(p, b, lo, hi, false);
        n = tiles_in<TILE>(lo, hi);
    }
    if (n == 0) {
#pragma unroll
        for (int c = 0; c < CPL; ++c)
            store4(dst + 4 * (lane + 32 * c), make_float4(0.f, 0.f, 0.f, 0.f));
        return wait_for_previous();
    }
    if (!scan_here) {
        wait_for_previous();
        T = p.pref[p.B];
        P = p.pref[b];
    }
    const int We = workers_for(p, T);
    const long long us = P + (long long)j * (n + UNIT_COST) + UNIT_COST;   // first tile
    const int wf = worker_of(us, T, We);
    const int wl = worker_of(us + n - 1, T, We);
    if (scan_here)
        wait_for_previous();
    if (wf == wl)
        return;                                   // written by the split kernel
    const long long sb = (long long)wf + (long long)b * p.U_b + j;
    const int ns = wl - wf + 1;
    const float2 *ml = p.ws_ml + sb * p.sh + hh;
    const float4 *po = reinterpret_cast<const float4 *>(p.ws_o + (sb * p.sh + hh) * D) + lane;
    const long long stride = (long long)p.sh * (D / 4);   // float4 per slot

    float M = -INFINITY;
    for (int s = lane; s < ns; s += 32)
        M = fmaxf(M, ml[(long long)s * p.sh].x);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float L = 0.f;
    float4 o[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c)
        o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < ns; s0 += 32) {
        const int cnt = min(32, ns - s0);
        const float2 v = lane < cnt ? ml[(long long)(s0 + lane) * p.sh]
                                    : make_float2(-INFINITY, 0.f);
        const float a = v.x == -INFINITY ? 0.f : ex2(v.x - M);
        L = fmaf(v.y, a, L);
#pragma unroll 8
        for (int k = 0; k < cnt; ++k) {
            const float ak = __shfl_sync(0xffffffffu, a, k);
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                const float4 y = po[(long long)(s0 + k) * stride + 32 * c];
                o[c].x = fmaf(y.x, ak, o[c].x);
                o[c].y = fmaf(y.y, ak, o[c].y);
                o[c].z = fmaf(y.z, ak, o[c].z);
                o[c].w = fmaf(y.w, ak, o[c].w);
            }
        }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        L += __shfl_xor_sync(0xffffffffu, L, off);
    const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
    for (int c = 0; c < CPL; ++c)
        store4(dst + 4 * (lane + 32 * c),
               make_float4(o[c].x * inv, o[c].y * inv, o[c].z * inv, o[c].w * inv));
}

template <int D, typename OutT = float>
__global__ void __launch_bounds__(MERGE_ROWS_PER_CTA * 32) fa_stream_merge_rows_kernel(
    const Params p)
{
    merge_rows<D, OutT>(p, blockIdx.x);
}

// Recorded weights: every key of sequence b and KV head kv adds
//     sum over the KV head's (query, head) columns of ex2(score - lse)
// to its cache row's running total.  The split kernel left the scores (log2
// units, -inf where a column does not attend the key) and, for units one worker
// covered, the rows' log2-sum-exp2; of the other units' it is reduced here from
// their partials' (m, l), so this needs no merged row and runs beside the merge.
// An item is w_rounds * 1024 keys of one (b, kv): its rows' log-sum-exps once, then
// four keys per thread and round, so that their loads overlap.  (With items of
// one round and page divisions, 16 sequences of 16384 keys took 41 us instead of
// their bytes' 8.)  One fp32 reduction per key, atomic because two sequences'
// tables may name the same block (a prefix they share).
constexpr int WEIGHT_THREADS = MERGE_THREADS;
constexpr int WEIGHT_KPT = 4;                              // keys per thread
constexpr int WEIGHT_KEYS = WEIGHT_THREADS * WEIGHT_KPT;   // keys per round
constexpr int WEIGHT_COLS = 512;                           // columns at a time

// Cache row of token t of (b, kv); -1 for a block id out of range (caches here have
// fewer than 2^31 rows).
__device__ __forceinline__ int weight_row(const Params &p, int b, int kv, int t)
{
    if (!p.bt)
        return (b * p.Hkv + kv) * static_cast<int>(p.cap) + t;
    const int page = p.lg_page >= 0 ? t >> p.lg_page : t / p.page_size;
    const int blk = p.bt[(long long)b * p.max_blocks + page];
    if (blk < 0 || blk >= p.num_blocks)
        return -1;
    return (blk * p.Hkv + kv) * p.page_size + (t - page * p.page_size);
}

__device__ __forceinline__ void add_weights(const Params &p, const int cta, const int ctas)
{
    __shared__ __align__(16) float lse[WEIGHT_COLS];
    const int tq = p.tq > 1 ? p.tq : 1;
    const int cols = tq * p.G;
    const int item_keys = WEIGHT_KEYS * p.w_rounds;
    const int chunks = static_cast<int>((p.cap16 + item_keys - 1) / item_keys);
    const long long items = (long long)chunks * p.B * p.Hkv;
    bool waited = false;
    long long T = 0, P = 0;
    int have_b = -1, n = 0;
    for (long long it = cta; it < items; it += ctas) {
        const int u = static_cast<int>(it / chunks);       // (b, kv)
        const int b = u / p.Hkv, kv = u - b * p.Hkv;
        int lo, hi;
        attended_range(p, b, lo, hi, false);
        const long long t0 = (lo / TILE) * TILE + (it - (long long)u * chunks) * item_keys;
        if (t0 >= hi)
            continue;
        const int end = static_cast<int>(t0 + item_keys < hi ? t0 + item_keys : hi);
        if (b != have_b && p.B <= 32 * SCAN_REG) {         // every warp for itself
            int b_at;
            long long P_at;
            T = flat_scan(p, -1, b_at, P_at, false, nullptr, b, &P, &n);
            have_b = b;
        }
        if (!waited)
            wait_for_previous();
        waited = true;
        if (b != have_b) {                                 // published by the split kernel
            T = p.pref[p.B];
            P = p.pref[b];
            n = tiles_in<TILE>(lo, hi);
            have_b = b;
        }
        const int We = workers_for(p, T);
        for (int x0 = 0; x0 < cols; x0 += WEIGHT_COLS) {
            const int nx = min(WEIGHT_COLS, cols - x0);
            __syncthreads();
            // 32 lanes per column, or 4 when there are many: its row's log-sum-exp, +inf
            // where it has no key
            const int lpc = nx > 8 ? 4 : 32;
            for (int i0 = 0; i0 < nx; i0 += WEIGHT_THREADS / lpc) {
                const int i = min(i0 + static_cast<int>(threadIdx.x) / lpc, nx - 1);
                const int x = x0 + i, j = kv * p.n_hg + x / p.cpu;
                const long long us = P + (long long)j * (n + UNIT_COST) + UNIT_COST;
                const int wf = worker_of(us, T, We), wl = worker_of(us + n - 1, T, We);
                float M = -INFINITY, L = 0.f;
                if (wf < wl) {
                    const float2 *ml = p.ws_ml + ((long long)wf + (long long)b * p.U_b + j) * p.sh +
                                       x % p.cpu;
                    for (int s = threadIdx.x % lpc; s <= wl - wf; s += lpc) {
                        const float2 y = ml[(long long)s * p.sh];
                        if (y.x == -INFINITY)
                            continue;
                        const float m = fmaxf(M, y.x);
                        L = L * ex2(M - m) + y.y * ex2(y.x - m);
                        M = m;
                    }
                }
                float Mw = M;
                for (int off = lpc / 2; off >= 1; off >>= 1)
                    Mw = fmaxf(Mw, __shfl_xor_sync(0xffffffffu, Mw, off));
                L = M == -INFINITY ? 0.f : L * ex2(M - Mw);
                for (int off = lpc / 2; off >= 1; off >>= 1)
                    L += __shfl_xor_sync(0xffffffffu, L, off);
                float v = L > 0.f ? Mw + log2f(L) : -INFINITY;
                if (wf == wl)
                    v = p.lse[((long long)b * tq + x / p.G) * p.Hq + kv * p.G + x % p.G];
                lse[i] = v == -INFINITY ? INFINITY : v;    // the same value by all its lanes
            }
            __syncthreads();
            const long long group = p.cap16 * p.sh;        // one column group's scores
            const float *at = p.ws_s + ((long long)b * p.U_b + kv * p.n_hg + x0 / p.cpu) * group;
            // (more than WEIGHT_COLS columns add to a key once per pass)
            for (int tr = static_cast<int>(t0) + threadIdx.x; tr < end; tr += WEIGHT_KEYS) {
                int row[WEIGHT_KPT];
                float sum[WEIGHT_KPT] = {};
#pragma unroll
                for (int q = 0; q < WEIGHT_KPT; ++q) {
                    const int t = tr + q * WEIGHT_THREADS;
                    row[q] = t >= lo && t < end ? weight_row(p, b, kv, t) : -1;
                }
                if (p.cpu > 2 * GPH) {
                    // key t's scores lie 16 floats from column to column, keys side by side
                    const float *s = at + (long long)(tr / TILE) * p.sh * TILE + tr % TILE;
                    for (int i = 0; i < nx; i += p.cpu, s += group) {
                        const int nc = min(p.cpu, nx - i);
#pragma unroll 4
                        for (int c = 0; c < nc; ++c) {
                            const float z = lse[i + c];
#pragma unroll
                            for (int q = 0; q < WEIGHT_KPT; ++q)
                                if (row[q] >= 0)
                                    sum[q] += ex2_ftz(__ldcs(s + c * TILE +
                                                             q * (WEIGHT_THREADS * p.sh)) - z);
                        }
                    }
                } else if (p.sh % 4 == 0) {                // a key's scores in 16-byte loads
                    const float *s = at + (long long)tr * p.sh;
                    for (int x = 0, c = 0; x < nx; x += 4) {
                        float4 v[WEIGHT_KPT];
#pragma unroll
                        for (int q = 0; q < WEIGHT_KPT; ++q)
                            if (row[q] >= 0)
                                v[q] = __ldcs(reinterpret_cast<const float4 *>(
                                    s + c + q * WEIGHT_THREADS * p.sh));
                        const float4 z = *reinterpret_cast<const float4 *>(lse + x);
#pragma unroll
                        for (int q = 0; q < WEIGHT_KPT; ++q)
                            if (row[q] >= 0) {
                                sum[q] += ex2_ftz(v[q].x - z.x);
                                sum[q] += x + 1 < nx ? ex2_ftz(v[q].y - z.y) : 0.f;
                                sum[q] += x + 2 < nx ? ex2_ftz(v[q].z - z.z) : 0.f;
                                sum[q] += x + 3 < nx ? ex2_ftz(v[q].w - z.w) : 0.f;
                            }
                        if ((c += 4) == p.sh) {            // on to the next column group
                            c = 0;
                            s += group;
                        }
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < WEIGHT_KPT; ++q)
                        if (row[q] >= 0)
                            for (int x = 0; x < nx; ++x)
                                sum[q] += ex2_ftz(at[x / p.cpu * group + x % p.cpu +
                                                     (long long)(tr + q * WEIGHT_THREADS) * p.sh] -
                                                  lse[x]);
                }
#pragma unroll
                for (int q = 0; q < WEIGHT_KPT; ++q)
                    if (row[q] >= 0)
                        atomicAdd(p.acc + row[q], sum[q]);
            }
        }
    }
    if (!waited)
        wait_for_previous();
}

// The same in the cluster plan, whose warps have their own keys' scores at hand (`unit`:
// the scores of the unit's row of columns; tokens t0 .. t1 - 1 are this warp's) and the
// partials (m, l) of every warp r and column c: ml(r, c).
template <typename Ml>
__device__ __forceinline__ void add_cluster_weights(const Params &p, int b, int kv, int t0, int t1,
                                                    int nh, const float *unit, int R, Ml ml)
{
    const int lane = threadIdx.x & 31;
    float lse[GPH];
#pragma unroll
    for (int c = 0; c < GPH; ++c) {
        lse[c] = INFINITY;
        if (c >= nh)
            continue;
        float M = -INFINITY, L = 0.f;
        for (int r = lane; r < R; r += 32) {
            const float2 y = ml(r, c);
            if (y.x == -INFINITY)
                continue;
            const float m = fmaxf(M, y.x);
            L = L * ex2(M - m) + y.y * ex2(y.x - m);
            M = m;
        }
        float Mw = M;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            Mw = fmaxf(Mw, __shfl_xor_sync(0xffffffffu, Mw, off));
        L = M == -INFINITY ? 0.f : L * ex2(M - Mw);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            L += __shfl_xor_sync(0xffffffffu, L, off);
        if (L > 0.f)
            lse[c] = Mw + log2f(L);
    }
    for (int t = t0 + lane; t < t1; t += 32) {
        const int row = weight_row(p, b, kv, t);
        if (row < 0)
            continue;
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < GPH; ++c)
            if (c < nh)
                sum += ex2_ftz(unit[(long long)t * p.sh + c] - lse[c]);
        atomicAdd(p.acc + row, sum);
    }
}

// The merge (fp16 output) and the recorded weights in one launch: the first
// merge_ctas CTAs merge, BY_WARP as fa_stream_merge_rows_kernel.
template <int D, bool BY_WARP>
__global__ void __launch_bounds__(MERGE_THREADS, D == 128 ? 4 : 2) fa_merge_weights_kernel(const Params p,
                                                                         const int merge_ctas)
{
    if (static_cast<int>(blockIdx.x) >= merge_ctas)
        add_weights(p, blockIdx.x - merge_ctas, gridDim.x - merge_ctas);
    else if constexpr (BY_WARP)
        merge_rows<D, __half>(p, blockIdx.x);
    else
        merge_row<D, false, __half>(p, blockIdx.x);
}
static_assert(MERGE_THREADS == MERGE_ROWS_PER_CTA * 32, "one block size for both merges");

// Scores of keys ka and kb of a unit of up to 16 columns for this lane's columns c0 = 2 t4
// and c0 + 1, of nh live ones.
__device__ __forceinline__ void store_scores(float *unit, int sh, int ka, int kb, int c0, int nh,
                                             const float (&sc)[4])
{
    if (c0 >= nh)
        return;
    float *a = unit + (long long)ka * sh + c0;
    float *b = unit + (long long)kb * sh + c0;
    if ((sh & 1) == 0 && c0 + 1 < nh) {
        *reinterpret_cast<float2 *>(a) = make_float2(sc[0], sc[1]);
        *reinterpret_cast<float2 *>(b) = make_float2(sc[2], sc[3]);
        return;
    }
    a[0] = sc[0];
    b[0] = sc[2];
    if (c0 + 1 < nh) {
        a[1] = sc[1];
        b[1] = sc[3];
    }
}

}  // namespace tc

// ================================================================ host side
inline thread_local char g_err[512] = "";

static int fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
static int fail(int code, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return code;
}

// Reads and clears this translation unit's status bits (asynchronous on st;
// *v holds them once st has been waited for).
static cudaError_t take_status(unsigned int *v, cudaStream_t st)
{
    static const unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(v, g_status, sizeof(*v), 0, cudaMemcpyDeviceToHost,
                                              st);
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbolAsync(g_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st);
    return e;
}
// the other translation units' take_status
cudaError_t int4_take_status(unsigned int *v, cudaStream_t st);
cudaError_t evict_take_status(unsigned int *v, cudaStream_t st);

static int device_sms(int *out)
{
    static std::mutex mu;
    static int cache[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return fail(FA_ERR_CUDA, "cudaGetDevice failed");
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 64 && cache[dev] > 0) {
        *out = cache[dev];
        return 0;
    }
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        return fail(FA_ERR_CUDA, "cannot read the SM count of device %d", dev);
    if (dev < 64)
        cache[dev] = n;
    *out = n;
    return 0;
}

// Workspace of the recorded weights behind a plan's own `base` bytes: the
// rows' log-sum-exps, then the scores.  false when the bytes overflow.
struct WeightSpace {
    size_t lse, scores, total;   // offsets of the two parts; bytes in all
};
static bool weight_space(size_t base, int B, int tq, int Hq, int units, int sh, long long cap,
                         WeightSpace *w)
{
    const size_t cap16 = (size_t)(cap + 15) / 16 * 16;
    w->lse = (base + 15) / 16 * 16;
    w->scores = w->lse + ((size_t)B * tq * Hq * sizeof(float) + 15) / 16 * 16;
    size_t n = (size_t)B * units;
    if (__builtin_mul_overflow(n, cap16, &n) ||
        __builtin_mul_overflow(n, sh * sizeof(float), &n) ||
        __builtin_add_overflow(n, w->scores, &w->total))
        return false;
    return true;
}

static int log2_of(int x)               // -1 when x is not a power of two
{
    return x <= 0 || (x & (x - 1)) ? -1 : __builtin_ctz(x);
}

// The merge of an fp16 output, with the recorded weights when p.acc is set; as the
// fp32 merge, a warp per row from MERGE_WARP_ROWS_PER_SM rows per SM.  Beside the
// recorded weights from one row per SM, which leaves their items more of the first
// wave of CTAs (16 sequences of 16384 keys, 512 rows: 206 us with a CTA per row, 203).
constexpr int MERGE_WARP_ROWS_PER_SM = 4;
template <int D>
static cudaError_t launch_merge_half(const Params &p0, int sms, cudaStream_t st)
{
    Params p = p0;
    const long long rows = (long long)p.B * (p.tq > 1 ? p.tq : 1) * p.Hq;
    const bool by_warp = rows >= (p.acc ? 1ll : MERGE_WARP_ROWS_PER_SM) * sms;
    const long long merge = by_warp ? (rows + tc::MERGE_ROWS_PER_CTA - 1) / tc::MERGE_ROWS_PER_CTA
                                    : rows;
    long long ctas = merge;
    if (p.acc) {
        // items of up to 8 rounds, while the capacity leaves two for every SM; of one
        // with many columns, whose rounds are long enough
        const long long most = (long long)sms * 4;
        const long long rounds = (p.cap16 + tc::WEIGHT_KEYS - 1) / tc::WEIGHT_KEYS;
        const long long units = (long long)p.B * p.Hkv;
        p.w_rounds = p.cpu > 2 * tc::GPH ? 1 : 8;
        while (p.w_rounds > 1 && (rounds + p.w_rounds - 1) / p.w_rounds * units < 2ll * sms)
            p.w_rounds /= 2;
        const long long items = (rounds + p.w_rounds - 1) / p.w_rounds * units;
        ctas += items < most ? items : most;
    }
    if (ctas > 0x7fffffffll)
        return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(tc::MERGE_THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int m = static_cast<int>(merge);
    const cudaError_t e =
        p.acc ? (by_warp ? cudaLaunchKernelEx(&cfg, tc::fa_merge_weights_kernel<D, true>, p, m)
                         : cudaLaunchKernelEx(&cfg, tc::fa_merge_weights_kernel<D, false>, p, m))
              : (by_warp ? cudaLaunchKernelEx(&cfg, tc::fa_stream_merge_rows_kernel<D, __half>, p)
                         : cudaLaunchKernelEx(&cfg, tc::fa_stream_merge_kernel<D, false, __half>, p));
    return e == cudaSuccess ? cudaGetLastError() : e;
}

static bool overlaps(const void *a, size_t na, const void *b, size_t nb)
{
    if (!a || !b || na == 0 || nb == 0)
        return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + nb && b0 < a0 + na;
}

static bool aligned16(const void *x)
{
    return ((uintptr_t)x & 15u) == 0;
}

// natural alignment of an element of `bytes` bytes (a null pointer passes)
static bool aligned_to(const void *x, unsigned bytes)
{
    return ((uintptr_t)x & (bytes - 1u)) == 0;
}

}  // namespace fa

#endif
