// fa_int4.cu -- the KV cache held in 4 bits: the rows' writer and reader, and
// decode attention over it, for sm_103a (GB300).
//
// A row of head_dim elements is cut into blocks of 32; block j holds
//     s_j = fp16_rn(max|x| / 7),   c = clamp(rint(x / s_j), -7, 7),   x ~ c * s_j
// as D/2 bytes of codes (nibble u = c + 8) and D/32 fp16 scales.  The codes of
// a row are D/8 32-bit words of 8 consecutive elements each; word (o, j),
// octet o = 0..3 of block j, is stored at word o * (D/32) + j, its element n
// in bits 4n..4n+3.  So the 16 (D = 128) or 32 (D = 256) bytes of one octet
// hold the same octet of every block, which is what one lane of the attention
// kernel wants of a row in one load.
#include "fa_common.cuh"

namespace fa {
namespace i4 {

using tc::GPH;
using tc::TILE;

// ------------------------------------------------------------------- codec
constexpr float X_MAX = 7.f * 65504.f;     // beyond it the scale saturates

// The scale of a block whose largest magnitude is amax (<= X_MAX): amax / 7
// rounded once to fp16.  The fp32 quotient is truncated with a sticky last
// bit, so the second rounding sees which side of a midpoint the exact one is.
__device__ __forceinline__ __half block_scale(float amax)
{
    float q = __fdiv_rz(amax, 7.f);
    if (fmaf(-q, 7.f, amax) != 0.f)
        q = __uint_as_float(__float_as_uint(q) | 1u);
    return __float2half_rn(q);
}

// rint(x / s) clamped to [-7, 7], of the exact quotient (ties to even): the
// product with 1/s is at most one off, and x - c*s is exact where it decides.
__device__ __forceinline__ int block_code(float x, float s, float inv)
{
    float c = rintf(x * inv);
    c = fminf(fmaxf(c, -7.f), 7.f);
    const float e2 = 2.f * fmaf(-c, s, x);
    const bool tie = fabsf(e2) == s && (static_cast<int>(c) & 1);
    if (fabsf(e2) > s || tie)
        c += copysignf(1.f, e2);
    return static_cast<int>(fminf(fmaxf(c, -7.f), 7.f));
}

// Where the token of row (b, i) of an append or gather lives: cache row of
// KV head kv, or -1 (flagged when `report`).
__device__ __forceinline__ long long token_row(const Params &p, int b, long long i, int kv,
                                               bool report)
{
    const long long t = p.seq_lens[b] + i;                // positions
    if (p.seq_lens[b] < 0 || t >= p.cap) {
        if (report)
            flag(FA_STATUS_POS_RANGE);
        return -1;
    }
    const long long row = tc::tile_row(p, b, kv, static_cast<int>(t / TILE * TILE));
    if (row < 0) {
        if (report)
            flag(FA_STATUS_BAD_BLOCK);
        return -1;
    }
    return row + t % TILE;
}

// One thread per word (8 elements), 4 neighbouring lanes per block; y = 0
// writes K, y = 1 writes V.  Reads each element once and writes whole rows;
// bound by HBM.
__global__ void __launch_bounds__(256) append_kernel(const Params p, const float *k_new,
                                                     const float *v_new, unsigned *k_codes,
                                                     __half *k_scales, unsigned *v_codes,
                                                     __half *v_scales, const int *n_new, int T,
                                                     int words, long long total)
{
    const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (idx >= total)                       // whole groups of 4 lanes: words is a multiple of 4
        return;
    const int w = static_cast<int>(idx % words);
    const long long r = idx / words;        // (b, i, kv)
    const int kv = static_cast<int>(r % p.Hkv);
    const long long bi = r / p.Hkv;
    const int b = static_cast<int>(bi / T);
    const int i = static_cast<int>(bi % T);
    if (n_new && i >= n_new[b])
        return;
    const bool isv = blockIdx.y != 0;
    const long long row = token_row(p, b, i, kv, !isv && w == 0);
    if (row < 0)
        return;
    const float4 *src = reinterpret_cast<const float4 *>((isv ? v_new : k_new) + idx * 8);
    float x[8];
    {
        const float4 a = __ldcs(src), c = __ldcs(src + 1);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = c.x; x[5] = c.y; x[6] = c.z; x[7] = c.w;
    }
    float amax = 0.f;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        x[n] = x[n] == x[n] ? fminf(fmaxf(x[n], -X_MAX), X_MAX) : 0.f;
        amax = fmaxf(amax, fabsf(x[n]));
    }
    const unsigned quad = 0xfu << (threadIdx.x & 28);     // the block's 4 lanes took this path
    amax = fmaxf(amax, __shfl_xor_sync(quad, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(quad, amax, 2));
    const __half sh = block_scale(amax);
    const float s = __half2float(sh);
    unsigned word = 0x88888888u;
    if (s > 0.f) {
        const float inv = 1.f / s;
        word = 0;
#pragma unroll
        for (int n = 0; n < 8; ++n)
            word |= static_cast<unsigned>(block_code(x[n], s, inv) + 8) << (4 * n);
    }
    const int j = w >> 2, o = w & 3, nj = words >> 2;
    (isv ? v_codes : k_codes)[row * words + o * nj + j] = word;
    if (o == 0)
        (isv ? v_scales : k_scales)[row * nj + j] = sh;
}

// The inverse: rows back as fp16 values c * s (each product rounded once).  A
// token outside the cache or in an unmapped block reads as zeros; rows i >=
// n_rows[b] are left as they were.
__global__ void __launch_bounds__(256) gather_kernel(const Params p, const unsigned *k_codes,
                                                     const __half *k_scales,
                                                     const unsigned *v_codes,
                                                     const __half *v_scales, const int *n_rows,
                                                     __half *k_out, __half *v_out, int T,
                                                     int words, long long total)
{
    const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (idx >= total)
        return;
    const int w = static_cast<int>(idx % words);
    const long long r = idx / words;
    const int kv = static_cast<int>(r % p.Hkv);
    const long long bi = r / p.Hkv;
    const int b = static_cast<int>(bi / T);
    const int i = static_cast<int>(bi % T);
    if (n_rows && i >= n_rows[b])
        return;
    const bool isv = blockIdx.y != 0;
    const long long row = token_row(p, b, i, kv, !isv && w == 0);
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (row >= 0) {
        const int j = w >> 2, o = w & 3, nj = words >> 2;
        const unsigned word = __ldg((isv ? v_codes : k_codes) + row * words + o * nj + j);
        const float s = __half2float(__ldg((isv ? v_scales : k_scales) + row * nj + j));
        unsigned h[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int c0 = static_cast<int>((word >> (8 * n)) & 15u) - 8;
            const int c1 = static_cast<int>((word >> (8 * n + 4)) & 15u) - 8;
            h[n] = tc::pack_half2(c0 * s, c1 * s);
        }
        v = make_uint4(h[0], h[1], h[2], h[3]);
    }
    reinterpret_cast<uint4 *>(isv ? v_out : k_out)[idx] = v;
}

// --------------------------------------------------------------- attention
// Per 16-key tile and per warp, as in the fp16 kernel,
//   S[16 keys x 8 columns] = K . Q^T,   O^T[D x 8] += V^T . P^T
// on mma.sync m16n8k16, with the codes going from shared memory straight into
// the A fragments: no dequantised tile is ever written.
//   K: fp16 bits 0x000u and 0x00u0 are the subnormals u 2^-24 and u 2^-20, so
//      an AND makes two codes into a half2 (the queries of odd elements are
//      held divided by 16).  The codes' offset of 8 is folded into the
//      accumulator's first value, -8 sum(q) per block, and each block's sum is
//      multiplied by the key's scale in fp32.
//   V: the pair of a half2 runs over two keys (the contraction), so the words
//      of two keys are interleaved by a byte permute; the offset is taken off
//      exactly in fp16 (1024 + u - 1032, 64 + u - 72), because left in the sum
//      it would be hundreds of times the result.  A key's scale multiplies its
//      weight instead of its 32 codes: P s_j is the B operand of block j.
// P and P s are rounded to fp16 (2^-11 each); everything else is fp32.
// The running maximum moves only when a score passes it by 8 (log2 units), so
// weights reach 2^8 and most tiles need no shuffles.  V scales outside
// [2^-12, 2^7] are carried times 2^-e, a power of two per warp, so that P s
// stays within fp16 whatever the scales.
//
// HBM-bound in bytes (144 B per key and KV head at D = 128, against 512 in
// fp16) but close to the issue rate: ~280 instructions per tile, and the copy
// rate leaves a warp scheduler ~390 cycles for it.
#ifndef FA_I4_NW
#define FA_I4_NW 4
#endif
#ifndef FA_I4_STAGES_128
#define FA_I4_STAGES_128 4
#endif
#ifndef FA_I4_CTAS_128
#define FA_I4_CTAS_128 4
#endif
#ifndef FA_I4_STAGES_256
#define FA_I4_STAGES_256 4
#endif
#ifndef FA_I4_CTAS_256
#define FA_I4_CTAS_256 2
#endif

template <int D>
struct Cfg {
    static constexpr int NW = FA_I4_NW;
    static constexpr int STAGES = D == 128 ? FA_I4_STAGES_128 : FA_I4_STAGES_256;
    static constexpr int CTAS_PER_SM = D == 128 ? FA_I4_CTAS_128 : FA_I4_CTAS_256;
    static constexpr int NJ = D / 32;                  // blocks per row
    static constexpr int RB = D / 2;                   // code bytes per row
    static constexpr int SB = D / 16;                  // scale bytes per row
    static constexpr int K_OFF = 0;
    static constexpr int V_OFF = TILE * RB;
    static constexpr int KS_OFF = 2 * TILE * RB;
    static constexpr int VS_OFF = KS_OFF + TILE * SB;
    static constexpr int STAGE_BYTES = VS_OFF + TILE * SB;
    static constexpr int SMEM = NW * STAGES * STAGE_BYTES;
    static_assert(CTAS_PER_SM * (SMEM + 1024) <= 228 * 1024, "shared memory per SM");
};

constexpr float NO_MAX = -3e38f;       // running maximum of a column that has no key yet
constexpr float MAX_SLACK = 8.f;       // log2 units a score may pass the running maximum by

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes, uint64_t policy)
{
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
                 "l"(src), "r"(bytes), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ __half2 as_half2(uint32_t x)
{
    return *reinterpret_cast<__half2 *>(&x);
}
__device__ __forceinline__ uint32_t as_u32(__half2 x)
{
    return *reinterpret_cast<uint32_t *>(&x);
}
__device__ __forceinline__ float pow2(int e)      // 2^e, e in [-126, 127]
{
    return __uint_as_float(static_cast<unsigned>(e + 127) << 23);
}
// D = A . B + C with C apart from D
__device__ __forceinline__ void mma_c(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%10, %11, %10, %11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

// Producer's place: the tile to issue next, as a cache row.  The block id of a
// page is fetched when the page is entered, an iteration before it is used.
struct Feed {
    int ti, off, blk;            // tile index in the sequence, tile in page, page's block
    const int *bt;               // the sequence's table row
    long long row0;              // contiguous: the sequence and head's first row
};

// Swizzled offset of 16-byte chunk c of code row r: the 8 lanes of every
// shared-memory phase of the K and V reads fall into different banks.
template <int D>
__device__ __forceinline__ int code_off(int r, int c)
{
    return D == 128 ? r * 64 + ((c ^ ((r >> 1) & 3)) << 4) : r * 128 + ((c ^ (r & 7)) << 4);
}

template <int D, bool WT>
__global__ void __launch_bounds__(Cfg<D>::NW * 32, Cfg<D>::CTAS_PER_SM) decode_kernel(const Params p)
{
    using C = Cfg<D>;
    constexpr int NJ = C::NJ, S = C::STAGES;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2;         // mma row group: a key of K, a 4-element group of V
    const int t = lane & 3;          // mma column pair: an octet of K, a key pair of V
    const int w = blockIdx.x * C::NW + warp;
    int b_at = -1, We = 0;
    long long P_at = 0, T = 0, t0 = 0, t1 = 0;
    if (!tc::stream_range(p, w, T, We, t0, t1, b_at, P_at))
        return;

    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t ring = smem_u32(smem) + warp * (S * C::STAGE_BYTES);
    const uint64_t policy = evict_first_policy();

    tc::Walk pw;
    pw.init(p, b_at, P_at, t0, tc::UNIT_COST);
    tc::Walk cw = pw;
    int n_my = 0;                    // tiles in [t0, t1)
    {
        tc::Walk e = pw;
        while (e.pos() < t1) {
            const long long us = e.unit_start();
            const long long end = us + e.n < t1 ? us + e.n : t1;
            n_my += static_cast<int>(end - e.pos());
            if (us + e.n >= t1)
                break;
            e.k = e.n - 1;
            e.next(p);
        }
    }

    const int tpp = p.page_size / TILE;          // tiles per page
    Feed f = {};
    auto feed_unit = [&] {                       // pw stands in a new unit (or at its start)
        f.ti = pw.lo / TILE + pw.k;
        const int kv = pw.j / p.n_hg;
        if (p.bt) {
            f.bt = p.bt + (long long)pw.b * p.max_blocks;
            f.off = f.ti % tpp;
            f.blk = f.bt[f.ti / tpp];
        } else {
            f.row0 = ((long long)pw.b * p.Hkv + kv) * p.cap;
        }
    };
    // per-lane copy places: code chunks lane, lane + 32, ... and one scale chunk
    constexpr int CPR = C::RB / 16;              // code chunks per row
    constexpr int NCP = TILE * CPR / 32;         // code chunks per lane, K and V each
    constexpr int NSC = TILE * C::SB / 16;       // scale chunks, K and V each
    auto issue = [&](int s) -> bool {            // false: the block id is out of range
        const int kv = pw.j / p.n_hg;
        long long row;
        if (p.bt) {
            if (f.blk < 0 || f.blk >= p.num_blocks) {
                if (lane == 0)
                    flag(FA_STATUS_BAD_BLOCK);
                return false;
            }
            row = ((long long)f.blk * p.Hkv + kv) * p.page_size + f.off * TILE;
        } else {
            row = f.row0 + (long long)f.ti * TILE;
        }
        const uint32_t st = ring + s * C::STAGE_BYTES;
        const int live = pw.hi - f.ti * TILE;    // rows from here on are zero-filled
#pragma unroll
        for (int i = 0; i < NCP; ++i) {
            const int id = lane + 32 * i, r = id / CPR, c = id % CPR;
            const int bytes = r < live ? 16 : 0;
            const long long at = row * C::RB + id * 16;
            cp16(st + C::K_OFF + code_off<D>(r, c), p.k + at, bytes, policy);
            cp16(st + C::V_OFF + code_off<D>(r, c), p.v + at, bytes, policy);
        }
        if (lane < 2 * NSC) {
            const int c = lane % NSC;
            const int bytes = min(max(live * C::SB - c * 16, 0), 16);
            cp16(st + (lane < NSC ? C::KS_OFF : C::VS_OFF) + c * 16,
                 (lane < NSC ? p.ks : p.vs) + row * C::SB + c * 16, bytes, policy);
        }
        return true;
    };
    auto feed_next = [&] {                       // pw to the tile after this one
        pw.next(p);
        if (pw.k == 0) {
            if (pw.b < p.B)
                feed_unit();
            return;
        }
        ++f.ti;
        if (p.bt && ++f.off == tpp) {
            f.off = 0;
            f.blk = f.bt[f.ti / tpp];
        }
    };
    unsigned ok = 0;                             // bit s: stage s holds a tile
    auto put = [&](int i) {                      // issue tile i (an empty group past the end)
        const int s = i % S;
        if (i < n_my) {
            ok = issue(s) ? ok | (1u << s) : ok & ~(1u << s);
            if (i + 1 < n_my)
                feed_next();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (n_my > 0)
        feed_unit();
    for (int i = 0; i < S - 1; ++i)
        put(i);

    // The unit's queries: column g's elements (n, n+4) of octet t of block j as
    // half2, odd n divided by 16; and per column pair the block's offset term.
    const int tq = p.tq > 1 ? p.tq : 1;
    uint32_t qb[NJ][4];
    float c0[NJ], c1[NJ];
    int nh = 0, clo[2], chi[2], all_lo = 0, all_hi = 0;
    auto load_q = [&] {
        const int kv = cw.j / p.n_hg, cg = cw.j % p.n_hg;
        nh = min(GPH, tq * p.G - cg * GPH);
        const tc::Col cq = tc::column(p, kv, cg, g, GPH);
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.q + (((long long)cw.b * tq + cq.j) * p.Hq + cq.h) * D);
        const __half2 sixteenth = __float2half2_rn(0.0625f);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const uint4 x = cq.live ? __ldg(src + j * 4 + t) : make_uint4(0u, 0u, 0u, 0u);
            qb[j][0] = __byte_perm(x.x, x.z, 0x5410);                              // 0, 4
            qb[j][1] = as_u32(__hmul2(as_half2(__byte_perm(x.x, x.z, 0x7632)), sixteenth));
            qb[j][2] = __byte_perm(x.y, x.w, 0x5410);                              // 2, 6
            qb[j][3] = as_u32(__hmul2(as_half2(__byte_perm(x.y, x.w, 0x7632)), sixteenth));
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float2 v = __half22float2(as_half2(qb[j][n]));
                sum += (v.x + v.y) * (n & 1 ? 16.f : 1.f);
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            sum *= -8.f / 16777216.f;
            c0[j] = __shfl_sync(0xffffffffu, sum, 8 * t);          // column 2t
            c1[j] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);      // column 2t + 1
        }
        const tc::Col a = tc::column(p, kv, cg, 2 * t, GPH);
        const tc::Col b = tc::column(p, kv, cg, 2 * t + 1, GPH);
        tc::column_range(p, cw.b, cw.hi, a.live ? a.j : tq - 1, clo[0], chi[0]);
        tc::column_range(p, cw.b, cw.hi, b.live ? b.j : tq - 1, clo[1], chi[1]);
        int x;
        tc::column_range(p, cw.b, cw.hi, tq - 1, all_lo, x);   // keys every query attends
        tc::column_range(p, cw.b, cw.hi, 0, x, all_hi);
    };

    float acc[2 * NJ][4];     // [2j + h]: elements 32j + 4g + 2h (0, 1) and + 1 (2, 3); columns 2t, 2t+1
    float mr[2], l[2];
    int e = 0;                // O is held times 2^-e
    __half vlim = __float2half_rn(0.f);     // V scales above it call for another e
    auto reset = [&] {
#pragma unroll
        for (int i = 0; i < 2 * NJ; ++i)
            acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        mr[0] = mr[1] = NO_MAX;
        l[0] = l[1] = 0.f;
        e = 0;
        vlim = __float2half_rn(0.f);
    };
    if (n_my > 0)
        load_q();
    reset();
    const float c2 = p.c2 * 16777216.f;

    for (int i = 0; i < n_my; ++i) {
        const int s = i % S;
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        __syncwarp();                 // tile i has landed; every lane is done with tile i - 1
        const bool tile_ok = (ok >> s) & 1u;
        put(i + S - 1);
        const uint32_t st = ring + s * C::STAGE_BYTES;
        const int base = cw.tok();

        if (tile_ok) {
            // ---- scores: rows are keys g and g + 8, columns 2t and 2t + 1
            float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int jj = 0; jj < NJ; jj += 4) {
                const int ch = D == 128 ? t : 2 * t + jj / 4;
                const uint4 wa = lds128(st + C::K_OFF + code_off<D>(g, ch));
                const uint4 wb = lds128(st + C::K_OFF + code_off<D>(g + 8, ch));
                const uint2 sa = lds64(st + C::KS_OFF + g * C::SB + jj * 2);
                const uint2 sb = lds64(st + C::KS_OFF + (g + 8) * C::SB + jj * 2);
                const uint32_t a[4] = {wa.x, wa.y, wa.z, wa.w};
                const uint32_t b[4] = {wb.x, wb.y, wb.z, wb.w};
                const float2 fa[2] = {__half22float2(as_half2(sa.x)), __half22float2(as_half2(sa.y))};
                const float2 fb[2] = {__half22float2(as_half2(sb.x)), __half22float2(as_half2(sb.y))};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int j = jj + q;
                    float d[4];
                    mma_c(d, a[q] & 0x000f000fu, b[q] & 0x000f000fu, a[q] & 0x00f000f0u,
                          b[q] & 0x00f000f0u, qb[j][0], qb[j][1], c0[j], c1[j]);
                    const uint32_t ah = a[q] >> 8, bh = b[q] >> 8;
                    tc::mma16816(d, ah & 0x000f000fu, bh & 0x000f000fu, ah & 0x00f000f0u,
                                 bh & 0x00f000f0u, qb[j][2], qb[j][3]);
                    const float ka = q & 1 ? fa[q / 2].y : fa[q / 2].x;
                    const float kb = q & 1 ? fb[q / 2].y : fb[q / 2].x;
                    sc[0] = fmaf(d[0], ka, sc[0]);
                    sc[1] = fmaf(d[1], ka, sc[1]);
                    sc[2] = fmaf(d[2], kb, sc[2]);
                    sc[3] = fmaf(d[3], kb, sc[3]);
                }
            }
            // ---- V scales as half2 over the key pairs (2t, 2t+1), (2t+8, 2t+9)
            __half2 sv[2][NJ];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t x[NJ];       // the two keys' scales: NJ / 2 words each
#pragma unroll
                for (int q = 0; q < NJ / 4; ++q) {
                    const uint4 v = lds128(st + C::VS_OFF + (2 * t + 8 * h) * C::SB + q * 16);
                    x[4 * q] = v.x; x[4 * q + 1] = v.y; x[4 * q + 2] = v.z; x[4 * q + 3] = v.w;
                }
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    sv[h][j] = as_half2(__byte_perm(x[j / 2], x[NJ / 2 + j / 2],
                                                    j & 1 ? 0x7632 : 0x5410));
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                sc[q] *= c2;                  // log2 units
            // ---- tile edges, and the ranges of several queries
            if (base < all_lo || base + TILE > all_hi) {
                const int ka = base + g, kb = base + g + 8;
                if (ka < clo[0] || ka >= chi[0])
                    sc[0] = -INFINITY;
                if (ka < clo[1] || ka >= chi[1])
                    sc[1] = -INFINITY;
                if (kb < clo[0] || kb >= chi[0])
                    sc[2] = -INFINITY;
                if (kb < clo[1] || kb >= chi[1])
                    sc[3] = -INFINITY;
                // rows before the window hold other data: their scales must not
                // turn a zero weight into NaN (rows after the end are zero-filled)
                const int r0 = cw.lo - base;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const uint32_t m = (2 * t + 8 * h >= r0 ? 0x0000ffffu : 0u) |
                                           (2 * t + 8 * h + 1 >= r0 ? 0xffff0000u : 0u);
                        sv[h][j] = as_half2(as_u32(sv[h][j]) & m);
                    }
            }
            if constexpr (WT)
                tc::store_scores(p, cw.unit(p), base + g, base + g + 8, 2 * t, nh, sc);
            // ---- online softmax
            float d[4] = {sc[0] - mr[0], sc[1] - mr[1], sc[2] - mr[0], sc[3] - mr[1]};
            __half2 vm = sv[0][0];
#pragma unroll
            for (int j = 1; j < 2 * NJ; ++j)
                vm = __hmax2(vm, sv[j / NJ][j % NJ]);
            const __half vmx = __hmax(__low2half(vm), __high2half(vm));
            const bool over = fmaxf(fmaxf(d[0], d[1]), fmaxf(d[2], d[3])) > MAX_SLACK;
            if (__any_sync(0xffffffffu, over || __hgt(vmx, vlim))) {
                float x0 = fmaxf(sc[0], sc[2]), x1 = fmaxf(sc[1], sc[3]);
                float vx = __half2float(vmx);
#pragma unroll
                for (int mask = 4; mask <= 16; mask <<= 1) {
                    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, mask));
                    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, mask));
                }
                vx = fmaxf(vx, __shfl_xor_sync(0xffffffffu, vx, 1));
                vx = fmaxf(vx, __shfl_xor_sync(0xffffffffu, vx, 2));
                const float n0 = fmaxf(mr[0], x0), n1 = fmaxf(mr[1], x1);
                int en = e;
                if (vx > __half2float(vlim)) {
                    // the largest scale so far: carried as it is from 2^-12 to
                    // 2^7, else brought to [1/2, 1) (at most 2^14 up)
                    const int ex = static_cast<int>((__float_as_uint(vx) >> 23) & 255u) - 126;
                    en = (ex >= -11 && ex <= 7) ? 0 : max(ex, -14);
                    vlim = __float2half_rn(en == 0 ? 128.f : fminf(pow2(en + 2), 65504.f));
                }
                const float r0 = ex2(mr[0] - n0) * pow2(e - en);
                const float r1 = ex2(mr[1] - n1) * pow2(e - en);
#pragma unroll
                for (int ii = 0; ii < 2 * NJ; ++ii) {
                    acc[ii][0] *= r0;
                    acc[ii][1] *= r1;
                    acc[ii][2] *= r0;
                    acc[ii][3] *= r1;
                }
                l[0] *= ex2(mr[0] - n0);
                l[1] *= ex2(mr[1] - n1);
                mr[0] = n0;
                mr[1] = n1;
                e = en;
                d[0] = sc[0] - n0;
                d[1] = sc[1] - n1;
                d[2] = sc[2] - n0;
                d[3] = sc[3] - n1;
            }
            if (e != 0) {
                const __half2 f2 = __float2half2_rn(pow2(-e));
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        sv[h][j] = __hmul2(sv[h][j], f2);
            }
            const float p0 = ex2(d[0]), p1 = ex2(d[1]), p2 = ex2(d[2]), p3 = ex2(d[3]);
            l[0] += p0 + p2;
            l[1] += p1 + p3;
            // P^T as the B operand: keys (2t, 2t+1) and (2t+8, 2t+9), column g
            const __half2 pa = as_half2(tc::movmatrix_t(tc::pack_half2(p0, p1)));
            const __half2 pb = as_half2(tc::movmatrix_t(tc::pack_half2(p2, p3)));
            // ---- O^T += V^T . (P s)^T: rows are elements, 4 per block and lane
            const uint32_t half_sel = g & 1 ? 0x7632 : 0x5410;
            const __half2 b1032 = __float2half2_rn(1032.f), b72 = __float2half2_rn(72.f);
#pragma unroll
            for (int jj = 0; jj < NJ; jj += 4) {
                uint32_t v[4][4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int key = 2 * t + (q & 1) + 8 * (q >> 1);
                    const int ch = D == 128 ? g >> 1 : 2 * (g >> 1) + jj / 4;
                    const uint4 x = lds128(st + C::V_OFF + code_off<D>(key, ch));
                    v[q][0] = x.x; v[q][1] = x.y; v[q][2] = x.z; v[q][3] = x.w;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int j = jj + q;
                    const uint32_t x = __byte_perm(v[0][q], v[1][q], half_sel);
                    const uint32_t y = __byte_perm(v[2][q], v[3][q], half_sel);
                    const uint32_t xh = x >> 8, yh = y >> 8;
                    auto even = [&](uint32_t z) {
                        return as_u32(__hsub2(as_half2((z & 0x000f000fu) | 0x64006400u), b1032));
                    };
                    auto odd = [&](uint32_t z) {
                        return as_u32(__hsub2(as_half2((z & 0x00f000f0u) | 0x54005400u), b72));
                    };
                    const uint32_t s0 = as_u32(__hmul2(pa, sv[0][j]));
                    const uint32_t s1 = as_u32(__hmul2(pb, sv[1][j]));
                    tc::mma16816(acc[2 * j], even(x), odd(x), even(y), odd(y), s0, s1);
                    tc::mma16816(acc[2 * j + 1], even(xh), odd(xh), even(yh), odd(yh), s0, s1);
                }
            }
        }

        const bool unit_end = cw.k == cw.n - 1;
        if (unit_end || i + 1 == n_my) {
            // ---- end of this worker's segment of the unit
#pragma unroll
            for (int mask = 4; mask <= 16; mask <<= 1) {
                l[0] += __shfl_xor_sync(0xffffffffu, l[0], mask);
                l[1] += __shfl_xor_sync(0xffffffffu, l[1], mask);
            }
            const long long us = cw.unit_start();
            const bool whole = tc::worker_of(us, T, We) == tc::worker_of(us + cw.n - 1, T, We);
            const int kv = cw.j / p.n_hg, cg = cw.j % p.n_hg;
            const float up = pow2(e);
            const long long slot = w + cw.unit(p);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int h = 2 * t + x;
                if (h >= nh)
                    continue;
                const float mx = mr[x] == NO_MAX ? -INFINITY : mr[x];
                if (whole) {
                    const tc::Col cc = tc::column(p, kv, cg, h, GPH);
                    const long long r = ((long long)cw.b * tq + cc.j) * p.Hq + cc.h;
                    const float inv = l[x] > 0.f ? up / l[x] : 0.f;
                    __half *o = reinterpret_cast<__half *>(p.out) + r * D + 4 * g;
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        tc::store4(o + 32 * j,
                                   make_float4(acc[2 * j][x] * inv, acc[2 * j][x + 2] * inv,
                                               acc[2 * j + 1][x] * inv, acc[2 * j + 1][x + 2] * inv));
                    if (WT && g == 0)
                        p.lse[r] = l[x] > 0.f ? mx + log2f(l[x]) : -INFINITY;
                } else {
                    float *o = p.ws_o + (slot * p.sh + h) * D + 4 * g;
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        tc::store4(o + 32 * j,
                                   make_float4(acc[2 * j][x] * up, acc[2 * j][x + 2] * up,
                                               acc[2 * j + 1][x] * up, acc[2 * j + 1][x + 2] * up));
                    if (g == 0)
                        p.ws_ml[slot * p.sh + h] = make_float2(mx, l[x]);
                }
            }
            reset();
            if (i + 1 < n_my) {
                cw.next(p);
                load_q();
            }
        } else {
            cw.next(p);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---------------------------------------------------------------- host side
struct Plan {
    int ctas, W, n_hg, units, sh;
    size_t bytes;                // partial slots and prefix
};

static Plan make_plan(int B, int tq, int Hq, int Hkv, int D, long long cap, int sms)
{
    Plan pl = {};
    const int cols = tq * (Hq / Hkv);
    pl.n_hg = (cols + GPH - 1) / GPH;
    pl.sh = cols < GPH ? cols : GPH;
    pl.units = Hkv * pl.n_hg;
    const int nw = D == 128 ? Cfg<128>::NW : Cfg<256>::NW;
    const int cps = D == 128 ? Cfg<128>::CTAS_PER_SM : Cfg<256>::CTAS_PER_SM;
    // one persistent wave, capped at a warp per position the capacity allows
    const long long most = ((long long)B * pl.units * ((cap + TILE - 1) / TILE + tc::UNIT_COST) +
                            nw - 1) / nw;
    const long long wave = (long long)sms * cps;
    pl.ctas = static_cast<int>(most < wave ? (most > 0 ? most : 1) : wave);
    pl.W = pl.ctas * nw;
    const size_t slots = (size_t)pl.W + (size_t)B * pl.units;
    pl.bytes = slots * pl.sh * (D * sizeof(float) + sizeof(float2)) +
               (size_t)(B + 1) * sizeof(long long);
    return pl;
}

static bool sizes_ok(int batch, int tq, int Hq, int Hkv, int D)
{
    return batch >= 0 && batch <= 65535 && tq >= 1 && tq <= 256 && Hq > 0 && Hkv > 0 &&
           Hkv <= 4096 && Hq % Hkv == 0 && Hq / Hkv <= 64 && (D == 128 || D == 256);
}

template <int D, bool WT>
static cudaError_t launch(const Params &p, int ctas, int sms, cudaStream_t st)
{
    static std::mutex mu;
    static bool done[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev >= 64 || !done[dev]) {
            e = cudaFuncSetAttribute(decode_kernel<D, WT>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
            if (e != cudaSuccess)
                return e;
            if (dev < 64)
                done[dev] = true;
        }
    }
    decode_kernel<D, WT><<<ctas, Cfg<D>::NW * 32, Cfg<D>::SMEM, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    const long long rows = (long long)p.B * p.tq * p.Hq;
    const bool by_warp = rows >= 4ll * sms;      // as the fp16 kernel's merge
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(
        by_warp ? (rows + tc::MERGE_ROWS_PER_CTA - 1) / tc::MERGE_ROWS_PER_CTA : rows));
    cfg.blockDim = dim3(by_warp ? tc::MERGE_ROWS_PER_CTA * 32 : tc::MERGE_THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = by_warp ? cudaLaunchKernelEx(&cfg, tc::fa_stream_merge_rows_kernel<D, __half, WT>, p)
                : cudaLaunchKernelEx(&cfg, tc::fa_stream_merge_kernel<D, false, __half, WT>, p);
    if (e == cudaSuccess)
        e = cudaGetLastError();
    if (WT && e == cudaSuccess)
        e = launch_weights(p, sms, st);
    return e;
}

// The checks of a cache's layout that append, gather and decode share.
static int check_cache(const char *name, int head_dim, int n_kv_heads, bool paged, int batch,
                       int page_size, int max_blocks, int num_blocks, long long *cap,
                       size_t *kv_rows)
{
    if (head_dim != 128 && head_dim != 256)
        return fail(FA_ERR_HEAD_DIM, "%s: head_dim %d not supported (128 or 256)", name, head_dim);
    if (n_kv_heads <= 0 || n_kv_heads > 4096)
        return fail(FA_ERR_HEADS, "%s: n_kv_heads %d", name, n_kv_heads);
    if (batch < 0 || batch > 65535 || max_blocks <= 0)
        return fail(FA_ERR_LAYOUT, "%s: bad batch %d or max_blocks_per_seq %d", name, batch,
                    max_blocks);
    if (paged) {
        if (page_size <= 0 || page_size % 16 || num_blocks <= 0)
            return fail(FA_ERR_LAYOUT, "%s: page_size %d must be a positive multiple of 16 and "
                                       "num_blocks %d positive", name, page_size, num_blocks);
        *cap = (long long)max_blocks * page_size;
    } else {
        *cap = max_blocks;
        if (*cap % 16)
            return fail(FA_ERR_LAYOUT, "%s: contiguous capacity %lld must be a multiple of 16",
                        name, *cap);
    }
    if (*cap > (1ll << 30))
        return fail(FA_ERR_LAYOUT, "%s: capacity %lld tokens too large", name, *cap);
    *kv_rows = (paged ? (size_t)num_blocks * page_size : (size_t)batch * *cap) * n_kv_heads;
    return 0;
}

struct Span {
    const void *p;
    size_t n;
};

// What append and gather share: the rows' side (`wide`, bytes per element) and
// the cache's side.
static int check_rows(const char *name, const Span *outs, int n_outs, const Span *ins, int n_ins)
{
    for (int i = 0; i < n_outs; ++i) {
        for (int j = 0; j < n_ins; ++j)
            if (overlaps(outs[i].p, outs[i].n, ins[j].p, ins[j].n))
                return fail(FA_ERR_ALIAS, "%s: an output overlaps an input", name);
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return fail(FA_ERR_ALIAS, "%s: two outputs overlap", name);
    }
    return 0;
}

static Params row_params(const int32_t *block_table, const int32_t *positions, int batch,
                         int n_kv_heads, int page_size, int max_blocks, int num_blocks,
                         long long cap)
{
    Params p = {};
    p.bt = block_table;
    p.seq_lens = positions;
    p.B = batch;
    p.Hkv = n_kv_heads;
    p.page_size = block_table ? page_size : 16;
    p.max_blocks = max_blocks;
    p.num_blocks = num_blocks;
    p.cap = cap;
    return p;
}

}  // namespace i4

cudaError_t int4_take_status(unsigned int *v, cudaStream_t st)
{
    return take_status(v, st);
}

}  // namespace fa

using namespace fa;

extern "C" {

FA_API int fa_append_kv_int4(const float *k_new, const float *v_new, void *k_codes,
                             void *k_scales, void *v_codes, void *v_scales,
                             const int32_t *block_table, const int32_t *positions,
                             const int32_t *n_new, int batch, int n_tokens, int n_kv_heads,
                             int head_dim, int page_size, int max_blocks_per_seq, int num_blocks,
                             void *stream)
{
    const char *name = "fa_append_kv_int4";
    g_err[0] = 0;
    if (!k_new || !v_new || !k_codes || !k_scales || !v_codes || !v_scales || !positions)
        return fail(FA_ERR_NULL, "%s: only block_table and n_new may be NULL", name);
    long long cap;
    size_t kv_rows;
    int rc = i4::check_cache(name, head_dim, n_kv_heads, block_table != nullptr, batch, page_size,
                             max_blocks_per_seq, num_blocks, &cap, &kv_rows);
    if (rc)
        return rc;
    if (n_tokens < 0)
        return fail(FA_ERR_LAYOUT, "%s: n_tokens %d", name, n_tokens);
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_codes) || !aligned16(v_codes) ||
        !aligned16(k_scales) || !aligned16(v_scales) || !aligned_to(positions, 4) ||
        !aligned_to(block_table, 4) || !aligned_to(n_new, 4))
        return fail(FA_ERR_ALIGN, "%s: rows, codes and scales must be 16-byte aligned, int32 "
                                  "arrays 4-byte aligned", name);
    const size_t rows = (size_t)batch * n_tokens * n_kv_heads;
    const size_t cb = kv_rows * (head_dim / 2), sb = kv_rows * (head_dim / 16);
    const i4::Span outs[] = {{k_codes, cb}, {k_scales, sb}, {v_codes, cb}, {v_scales, sb}};
    const i4::Span ins[] = {{k_new, rows * head_dim * 4}, {v_new, rows * head_dim * 4},
                            {positions, (size_t)batch * 4}, {n_new, (size_t)batch * 4},
                            {block_table, (size_t)batch * max_blocks_per_seq * 4}};
    if ((rc = i4::check_rows(name, outs, 4, ins, 5)))
        return rc;
    if (rows == 0)
        return 0;
    const int words = head_dim / 8;
    const long long total = (long long)rows * words;
    const long long ctas = (total + 255) / 256;
    if (ctas > 0x7fffffffll)
        return fail(FA_ERR_LAYOUT, "%s: too many rows", name);
    const Params p = i4::row_params(block_table, positions, batch, n_kv_heads, page_size,
                                    max_blocks_per_seq, num_blocks, cap);
    i4::append_kernel<<<dim3((unsigned)ctas, 2), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        p, k_new, v_new, static_cast<unsigned *>(k_codes), static_cast<__half *>(k_scales),
        static_cast<unsigned *>(v_codes), static_cast<__half *>(v_scales), n_new, n_tokens, words,
        total);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(FA_ERR_CUDA, "%s: launch failed: %s", name, cudaGetErrorString(e));
    return 0;
}

FA_API int fa_gather_kv_int4(const void *k_codes, const void *k_scales, const void *v_codes,
                             const void *v_scales, const int32_t *block_table,
                             const int32_t *positions, const int32_t *n_rows, void *k_out,
                             void *v_out, int batch, int n_tokens, int n_kv_heads, int head_dim,
                             int page_size, int max_blocks_per_seq, int num_blocks, void *stream)
{
    const char *name = "fa_gather_kv_int4";
    g_err[0] = 0;
    if (!k_codes || !k_scales || !v_codes || !v_scales || !positions || !k_out || !v_out)
        return fail(FA_ERR_NULL, "%s: only block_table and n_rows may be NULL", name);
    long long cap;
    size_t kv_rows;
    int rc = i4::check_cache(name, head_dim, n_kv_heads, block_table != nullptr, batch, page_size,
                             max_blocks_per_seq, num_blocks, &cap, &kv_rows);
    if (rc)
        return rc;
    if (n_tokens < 0)
        return fail(FA_ERR_LAYOUT, "%s: n_tokens %d", name, n_tokens);
    if (!aligned16(k_out) || !aligned16(v_out) || !aligned16(k_codes) || !aligned16(v_codes) ||
        !aligned16(k_scales) || !aligned16(v_scales) || !aligned_to(positions, 4) ||
        !aligned_to(block_table, 4) || !aligned_to(n_rows, 4))
        return fail(FA_ERR_ALIGN, "%s: rows, codes and scales must be 16-byte aligned, int32 "
                                  "arrays 4-byte aligned", name);
    const size_t rows = (size_t)batch * n_tokens * n_kv_heads;
    const size_t cb = kv_rows * (head_dim / 2), sb = kv_rows * (head_dim / 16);
    const i4::Span outs[] = {{k_out, rows * head_dim * 2}, {v_out, rows * head_dim * 2}};
    const i4::Span ins[] = {{k_codes, cb}, {k_scales, sb}, {v_codes, cb}, {v_scales, sb},
                            {positions, (size_t)batch * 4}, {n_rows, (size_t)batch * 4},
                            {block_table, (size_t)batch * max_blocks_per_seq * 4}};
    if ((rc = i4::check_rows(name, outs, 2, ins, 7)))
        return rc;
    if (rows == 0)
        return 0;
    const int words = head_dim / 8;
    const long long total = (long long)rows * words;
    const long long ctas = (total + 255) / 256;
    if (ctas > 0x7fffffffll)
        return fail(FA_ERR_LAYOUT, "%s: too many rows", name);
    const Params p = i4::row_params(block_table, positions, batch, n_kv_heads, page_size,
                                    max_blocks_per_seq, num_blocks, cap);
    i4::gather_kernel<<<dim3((unsigned)ctas, 2), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        p, static_cast<const unsigned *>(k_codes), static_cast<const __half *>(k_scales),
        static_cast<const unsigned *>(v_codes), static_cast<const __half *>(v_scales), n_rows,
        static_cast<__half *>(k_out), static_cast<__half *>(v_out), n_tokens, words, total);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(FA_ERR_CUDA, "%s: launch failed: %s", name, cudaGetErrorString(e));
    return 0;
}

FA_API size_t fa_decode_int4_workspace_size(int batch, int n_queries, int n_q_heads,
                                            int n_kv_heads, int head_dim, int max_kv_len,
                                            int with_weights, int num_sms)
{
    if (!i4::sizes_ok(batch, n_queries, n_q_heads, n_kv_heads, head_dim) || max_kv_len < 0 ||
        batch == 0)
        return 0;
    if (num_sms <= 0 && device_sms(&num_sms) != 0)
        return 0;
    const i4::Plan pl = i4::make_plan(batch, n_queries, n_q_heads, n_kv_heads, head_dim,
                                      max_kv_len, num_sms);
    if (!with_weights)
        return pl.bytes;
    WeightSpace ws;
    return weight_space(pl.bytes, batch, n_queries, n_q_heads, pl.units, pl.sh, max_kv_len, &ws)
               ? ws.total
               : 0;
}

FA_API int fa_decode_int4(const void *q, const void *k_codes, const void *k_scales,
                          const void *v_codes, const void *v_scales, const int32_t *block_table,
                          const int32_t *seq_lens, int n_queries, int n_q_heads, int n_kv_heads,
                          int head_dim, float scale, const int32_t *window, void *out, float *acc,
                          int batch, int page_size, int max_blocks_per_seq, int num_blocks,
                          void *workspace, size_t workspace_bytes, void *stream)
{
    const char *name = "fa_decode_int4";
    g_err[0] = 0;
    if (!q || !k_codes || !k_scales || !v_codes || !v_scales || !seq_lens || !out)
        return fail(FA_ERR_NULL, "%s: only block_table, window and acc may be NULL", name);
    long long cap;
    size_t kv_rows;
    int rc = i4::check_cache(name, head_dim, n_kv_heads, block_table != nullptr, batch, page_size,
                             max_blocks_per_seq, num_blocks, &cap, &kv_rows);
    if (rc)
        return rc;
    if (n_q_heads <= 0 || n_q_heads % n_kv_heads || n_q_heads / n_kv_heads > 64)
        return fail(FA_ERR_HEADS, "%s: bad heads (q %d, kv %d)", name, n_q_heads, n_kv_heads);
    if (n_queries <= 0 || n_queries > 256)
        return fail(FA_ERR_LAYOUT, "%s: n_queries %d must be in [1, 256]", name, n_queries);
    if (!isfinite(scale))
        return fail(FA_ERR_SCALE, "%s: scale is not finite", name);
    if (!aligned16(q) || !aligned16(k_codes) || !aligned16(k_scales) || !aligned16(v_codes) ||
        !aligned16(v_scales) || !aligned16(out) || !aligned16(workspace))
        return fail(FA_ERR_ALIGN, "%s: q, codes, scales, out and workspace must be 16-byte "
                                  "aligned", name);
    if (!aligned_to(seq_lens, 4) || !aligned_to(block_table, 4) || !aligned_to(window, 4) ||
        !aligned_to(acc, 4))
        return fail(FA_ERR_ALIGN, "%s: seq_lens, block_table, window and acc must be 4-byte "
                                  "aligned", name);
    const size_t q_bytes = (size_t)batch * n_queries * n_q_heads * head_dim * 2;
    const size_t cb = kv_rows * (head_dim / 2), sb = kv_rows * (head_dim / 16);
    const i4::Span outs[] = {{out, q_bytes}, {acc, kv_rows * sizeof(float)}};
    const i4::Span ins[] = {{q, q_bytes}, {k_codes, cb}, {k_scales, sb}, {v_codes, cb},
                            {v_scales, sb}, {seq_lens, (size_t)batch * 4},
                            {window, (size_t)batch * 4},
                            {block_table, (size_t)batch * max_blocks_per_seq * 4}};
    if ((rc = i4::check_rows(name, outs, 2, ins, 8)))
        return rc;
    if (batch == 0)
        return 0;
    int sms = 0;
    if ((rc = device_sms(&sms)))
        return rc;
    const i4::Plan pl = i4::make_plan(batch, n_queries, n_q_heads, n_kv_heads, head_dim, cap, sms);
    size_t need = pl.bytes;
    WeightSpace wsp = {};
    if (acc) {
        if (!weight_space(pl.bytes, batch, n_queries, n_q_heads, pl.units, pl.sh, cap, &wsp))
            return fail(FA_ERR_WORKSPACE, "%s: the workspace for these sizes exceeds 2^64 bytes",
                        name);
        need = wsp.total;
    }
    if (!workspace || workspace_bytes < need)
        return fail(FA_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", name, workspace_bytes,
                    need);
    const i4::Span ws[] = {{workspace, need}};
    if ((rc = i4::check_rows(name, ws, 1, ins, 8)) || (rc = i4::check_rows(name, ws, 1, outs, 2)))
        return rc;

    Params p = {};
    p.q = static_cast<const __half *>(q);
    p.k = static_cast<const char *>(k_codes);
    p.ks = static_cast<const char *>(k_scales);
    p.v = static_cast<const char *>(v_codes);
    p.vs = static_cast<const char *>(v_scales);
    p.bt = block_table;
    p.seq_lens = seq_lens;
    p.window = window;
    p.out = static_cast<float *>(out);
    p.ws_o = static_cast<float *>(workspace);
    const size_t slots = (size_t)pl.W + (size_t)batch * pl.units;
    p.ws_ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) +
                                         slots * pl.sh * head_dim * sizeof(float));
    p.pref = reinterpret_cast<long long *>(p.ws_ml + slots * pl.sh);
    p.B = batch;
    p.Hq = n_q_heads;
    p.Hkv = n_kv_heads;
    p.G = n_q_heads / n_kv_heads;
    p.n_hg = pl.n_hg;
    p.page_size = block_table ? page_size : 16;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.cap = cap;
    p.c2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    p.tile = i4::TILE;
    p.tq = n_queries;
    p.W = pl.W;
    p.U_b = pl.units;
    p.sh = pl.sh;
    p.cpu = i4::GPH;
    if (acc) {
        p.acc = acc;
        p.lse = reinterpret_cast<float *>(static_cast<char *>(workspace) + wsp.lse);
        p.ws_s = reinterpret_cast<float *>(static_cast<char *>(workspace) + wsp.scores);
        p.cap16 = (cap + 15) / 16 * 16;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        acc ? (head_dim == 128 ? i4::launch<128, true>(p, pl.ctas, sms, st)
                               : i4::launch<256, true>(p, pl.ctas, sms, st))
            : (head_dim == 128 ? i4::launch<128, false>(p, pl.ctas, sms, st)
                               : i4::launch<256, false>(p, pl.ctas, sms, st));
    if (e != cudaSuccess)
        return fail(FA_ERR_CUDA, "%s: launch failed: %s", name, cudaGetErrorString(e));
    return 0;
}

}  // extern "C"
