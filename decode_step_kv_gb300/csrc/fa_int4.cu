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
// rounded once to fp16.  The rounded product with 1/7 is it whenever amax - 7 h
// (exact) stays clear of the midpoint, 7/2 units of h's last place away (of the
// place below when h is a power of two); else the fp32 quotient is truncated with
// a sticky last bit, so that rounding it sees which side of the midpoint the exact
// one is on.
__device__ __forceinline__ __half block_scale(float amax)
{
    const __half h = __float2half_rn(amax * (1.f / 7.f));
    const float f = __half2float(h);
    const float binade = __uint_as_float((max(__float_as_uint(f), 1u) - 1u) & 0x7f800000u);
    if (fabsf(fmaf(-7.f, f, amax)) < binade * (7.f / 2048.f * 0.999f))
        return h;
    float q = __fdiv_rz(amax, 7.f);
    if (fmaf(-q, 7.f, amax) != 0.f)
        q = __uint_as_float(__float_as_uint(q) | 1u);
    return __float2half_rn(q);
}

// rint(x / s) clamped to [-7, 7], of the exact quotient (ties to even); 0 for a
// NaN.  The product with 1/s is at most one off, and x - c*s is exact where it
// decides.
__device__ __forceinline__ int block_code(float x, float s, float inv)
{
    if (x != x)
        return 0;
    float c = rintf(x * inv);
    c = fminf(fmaxf(c, -7.f), 7.f);
    const float e2 = 2.f * fmaf(-c, s, x);
    const bool tie = fabsf(e2) == s && (static_cast<int>(c) & 1);
    if (fabsf(e2) > s || tie)
        c += copysignf(1.f, e2);
    return static_cast<int>(fminf(fmaxf(c, -7.f), 7.f));
}

// Where row i of sequence b of an append or gather lives: the cache row of KV head
// kv, or -1 (flagged when `report`).  lg_page: log2 of the page size, or -1.
__device__ __forceinline__ long long token_row(const Params &p, int lg_page, int b, int i, int kv,
                                               bool report)
{
    const int pos = p.seq_lens[b];                        // positions
    const long long t = (long long)pos + i;
    if (pos < 0 || t >= p.cap) {
        if (report)
            flag(FA_STATUS_POS_RANGE);
        return -1;
    }
    const int tok = static_cast<int>(t);
    if (!p.bt)
        return ((long long)b * p.Hkv + kv) * p.cap + tok;
    const int page = lg_page >= 0 ? tok >> lg_page : tok / p.page_size;
    const int blk = p.bt[(long long)b * p.max_blocks + page];
    if (blk < 0 || blk >= p.num_blocks) {
        if (report)
            flag(FA_STATUS_BAD_BLOCK);
        return -1;
    }
    return ((long long)blk * p.Hkv + kv) * p.page_size + (tok - page * p.page_size);
}

// A call's rows: sequence b = blockIdx.y, K or V = blockIdx.z, and along x one
// thread per half block (16 elements, two words), so two neighbouring lanes hold a
// block: what a row costs (its place, the scale) is shared by 16 elements.
struct RowArgs {
    int T, n_half;        // rows per sequence; half blocks per sequence (T * Hkv * D / 16)
    int lg_page, lg_hkv;  // log2 of the page size and of the KV heads, or -1
    const int *count;     // real rows per sequence, or NULL
};

// (row i, KV head kv, half block y of the row) of thread idx
template <int D>
__device__ __forceinline__ void row_place(const Params &p, const RowArgs &a, unsigned idx, int &i,
                                          int &kv, int &y)
{
    constexpr unsigned H = D / 16;
    const unsigned r = idx / H;
    y = idx % H;
    i = a.lg_hkv >= 0 ? r >> a.lg_hkv : r / p.Hkv;
    kv = r - i * p.Hkv;
}

// Reads each element once and writes whole rows, in few instructions per element: the
// code comes from one fused multiply-add: with 1.5 * 2^23 + 8 added, the sum's low four
// bits are the nibble of the rounded x / s; where x - c*s does not confirm it (a tie, a
// quotient next to one, a NaN, a scale rounded so far down that codes are cut off) the
// thread takes the exact form.  2 x 16384 rows of 8 heads x 128: 33 us, 23 for the bytes;
// nothing is full (DRAM 52%, ALU 56%, issue 64%), the loads of 16 bytes that lie 64 apart
// wait longest.  (One word per thread and a division per scale: 38 us.)
template <int D>
__global__ void __launch_bounds__(256) append_kernel(const Params p, const RowArgs a,
                                                     const float *k_new, const float *v_new,
                                                     unsigned *k_codes, __half *k_scales,
                                                     unsigned *v_codes, __half *v_scales)
{
    constexpr int W = D / 8, NJ = D / 32;
    const unsigned idx = blockIdx.x * blockDim.x + threadIdx.x;
    if (idx >= a.n_half)                    // whole pairs of lanes
        return;
    const int b = blockIdx.y;
    int i, kv, y;
    row_place<D>(p, a, idx, i, kv, y);
    if (a.count && i >= a.count[b])
        return;
    const bool isv = blockIdx.z != 0;
    const float4 *src = reinterpret_cast<const float4 *>(
        (isv ? v_new : k_new) + ((long long)b * a.n_half + idx) * 16);
    float x[16];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float4 z = __ldcs(src + q);
        x[4 * q] = z.x; x[4 * q + 1] = z.y; x[4 * q + 2] = z.z; x[4 * q + 3] = z.w;
    }
    const long long row = token_row(p, a.lg_page, b, i, kv, !isv && y == 0);
    if (row < 0)
        return;
    float amax = 0.f;
#pragma unroll
    for (int n = 0; n < 16; ++n)
        amax = fmaxf(amax, fabsf(x[n]));    // a NaN is passed over
    const unsigned pair = 3u << (threadIdx.x & 30);       // the block's 2 lanes took this path
    amax = fmaxf(amax, __shfl_xor_sync(pair, amax, 1));
    const __half sh = block_scale(fminf(amax, X_MAX));
    const float s = __half2float(sh);
    unsigned word[2] = {0x88888888u, 0x88888888u};
    if (s > 0.f) {
        const float inv = __fdividef(1.f, s), hs = 0.5f * s;
        constexpr float MAGIC = 12582920.f;               // 1.5 * 2^23 + 8
        float worst = 0.f;                                // largest |x - c*s|; NaN sticks
        word[0] = word[1] = 0;
#pragma unroll
        for (int n = 0; n < 16; ++n) {
            const float v = fmaf(x[n], inv, MAGIC);
            const float e = fabsf(fmaf(MAGIC - v, s, x[n]));
            worst = e >= worst || e != e ? e : worst;
            word[n / 8] |= (__float_as_uint(v) & 15u) << (4 * (n % 8));
        }
        if (!(worst < hs && amax * inv < 7.4f)) {
            word[0] = word[1] = 0;
#pragma unroll
            for (int n = 0; n < 16; ++n)
                word[n / 8] |= static_cast<unsigned>(block_code(x[n], s, inv) + 8) << (4 * (n % 8));
        }
    }
    const int j = y >> 1, o = (y & 1) * 2;
    unsigned *codes = (isv ? v_codes : k_codes) + row * W + o * NJ + j;
    codes[0] = word[0];
    codes[NJ] = word[1];
    if (o == 0)
        (isv ? v_scales : k_scales)[row * NJ + j] = sh;
}

// The inverse: rows back as fp16 values c * s (each product rounded once).  Bound by
// the latency of its two short reads per thread: 16384 rows of 8 heads x 128 in 20
// us, 13 for the bytes.  A token outside the cache or in an unmapped block reads as zeros; rows behind the
// count are left as they were.
template <int D>
__global__ void __launch_bounds__(256) gather_kernel(const Params p, const RowArgs a,
                                                     const unsigned *k_codes,
                                                     const __half *k_scales,
                                                     const unsigned *v_codes,
                                                     const __half *v_scales, __half *k_out,
                                                     __half *v_out)
{
    constexpr int W = D / 8, NJ = D / 32;
    const unsigned idx = blockIdx.x * blockDim.x + threadIdx.x;
    if (idx >= a.n_half)
        return;
    const int b = blockIdx.y;
    int i, kv, y;
    row_place<D>(p, a, idx, i, kv, y);
    if (a.count && i >= a.count[b])
        return;
    const bool isv = blockIdx.z != 0;
    const long long row = token_row(p, a.lg_page, b, i, kv, !isv && y == 0);
    uint4 out[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if (row >= 0) {
        const int j = y >> 1, o = (y & 1) * 2;
        const unsigned *codes = (isv ? v_codes : k_codes) + row * W + o * NJ + j;
        const unsigned word[2] = {__ldg(codes), __ldg(codes + NJ)};
        const __half2 s2 = __half2half2(__ldg((isv ? v_scales : k_scales) + row * NJ + j));
        // elements (n, n+4) as 1024 + u or 64 + u, less 1032 or 72 exactly, times the scale
        const __half2 b1032 = __float2half2_rn(1032.f), b72 = __float2half2_rn(72.f);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t h[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const uint32_t z = n < 2 ? word[q] : word[q] >> 8;
                const uint32_t u = n & 1 ? (z & 0x00f000f0u) | 0x54005400u
                                         : (z & 0x000f000fu) | 0x64006400u;
                const __half2 c = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&u),
                                                  n & 1 ? b72 : b1032), s2);
                h[n] = *reinterpret_cast<const uint32_t *>(&c);
            }
            out[q] = make_uint4(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410),
                                __byte_perm(h[0], h[1], 0x7632), __byte_perm(h[2], h[3], 0x7632));
        }
    }
    uint4 *to = reinterpret_cast<uint4 *>(isv ? v_out : k_out) + ((long long)b * a.n_half + idx) * 2;
    __stcs(to, out[0]);
    __stcs(to + 1, out[1]);
}

// --------------------------------------------------------------- attention
// Per 16-key tile and per warp, as in the fp16 kernel,
//   S[16 keys x 8 columns] = K . Q^T,   O^T[D x 8] += V^T . P^T
// on mma.sync m16n8k16, with the codes going from shared memory straight into
// the A fragments: no dequantised tile is ever written.  The fp16 bits 0x000u
// and 0x00u0 are the subnormals u 2^-24 and u 2^-20, so an AND makes two codes
// into a half2.
//   K: the queries of even elements are held times 16, and each block's sum is multiplied
//      by the key's scale in fp32.  (In a column with an even element of 4096 or more, those of
//      odd elements are held divided by 16 instead: exactly, but for 2^-33 of the largest.)
//      The codes' offset of 8 adds -8 sum_j s_j sum(q_j) to a score: one tf32 mma per tile,
//      scales by block sums (in two tf32 parts, 21 bits: 2^-21 of the offset, which is at most
//      a few times the sum of the score's absolute terms).
//   V: the pair of a half2 runs over two keys (the contraction), so the words
//      of two keys are interleaved by a byte permute; the accumulators of odd
//      elements hold 2^-20, the even ones 2^-24.  The offset is taken off in fp16,
//      exactly (u - 8 at either exponent): left in the sum it would be hundreds of
//      times the result, and a second mma with a constant -8 as its A fragment kept
//      the tensor pipe busy longer than it saved instructions (226 us against 214
//      for 32 x 32768 keys of 8 heads x 128).  A key's scale multiplies its weight
//      instead of its 32 codes: P s_j is the B operand of block j.
// P and P s are rounded to fp16, by 2^-11 of their value where that is a normal fp16;
// everything else is fp32.  Both are kept as high in fp16's range as they may go, because the
// keys behind a dominant one (an attention sink) have weights of 2^-10 to 2^-20 and scales of any
// size, and their sum still counts:
//   P is taken against a reference 2^P_SHIFT below the largest score, which moves only when a
//      score passes that maximum by MAX_SLACK (log2 units), so most tiles need no shuffles: P
//      reaches 2^14, and is a normal fp16 from 2^-24 of the largest weight on.
//   The V scales of block j are carried times 2^-e_j, which brings the largest so far to
//      [1/2, 1) and lets it grow to 2, so that P s stays below 2^16 and is a normal fp16 while
//      weight times scale is at least 2^-24 of their largest values.
// So the result is off by 3.0-3.8e-4 of its norm, 2.1e-4 of them its own rounding, also behind a
// sink that takes half the weight (32768 keys, V of 0.02: 3.1e-4; with weights up to 2^8 and
// the scales as they are it was 2.9e-2, with V of 0.1 5.6e-3).  P in two fp16 parts would take
// off one of the two roundings and cost 5% (226 us against 214 for 32 x 32768 keys).
// Tiles are copied in batches of up to BT of one unit (cp.async, a ring of
// batches per warp); the lanes look their cache rows up side by side, so a tile's
// share of the addressing is a shuffle and three multiply-adds.  They are
// worked on two at a time.
// Warps per CTA, tiles per batch, batches in the ring, CTAs per SM: measured best of
// the configurations whose rings fit, at D = 128 on 32 x 32768 keys (213 us): 2 CTAs x 3
// batches took 226-238 then, 4 CTAs of 128 registers x batches of 2 267-289, one CTA of 14
// warps 308; the tile loop unrolled by two 219 and more.  Two column groups per warp (NG = 2,
// D = 128) take the registers of two CTAs per SM.
template <int D, int NG>
struct Cfg {
    static constexpr int NW = 4;
    static constexpr int BT = D == 128 ? 4 : 2;
    static constexpr int STAGES = D == 128 && NG == 1 ? 2 : 3;
    static constexpr int CTAS_PER_SM = D == 128 && NG == 1 ? 3 : 2;
    static constexpr int NJ = D / 32;                  // blocks per row
    static constexpr int RB = D / 2;                   // code bytes per row
    static constexpr int SB = D / 16;                  // scale bytes per row
    static constexpr int K_OFF = 0;
    static constexpr int V_OFF = BT * TILE * RB;
    static constexpr int KS_OFF = 2 * BT * TILE * RB;
    static constexpr int VS_OFF = KS_OFF + BT * TILE * SB;
    static constexpr int STAGE_BYTES = VS_OFF + BT * TILE * SB;
    static constexpr int SMEM = NW * STAGES * STAGE_BYTES;
    static_assert(BT % 2 == 0 && BT <= 32, "tiles are worked on in pairs");
    static_assert(STAGES * BT <= 32, "a bit per tile of the ring");
    static_assert(CTAS_PER_SM * (SMEM + 1024) <= 228 * 1024, "shared memory per SM");
};

constexpr float NO_MAX = -3e38f;       // reference of a column that has no key yet
constexpr float P_SHIFT = 10.f;        // log2 units from the reference up to the running maximum
constexpr float MAX_SLACK = 4.f;       // ... a score may pass that maximum by

// The reference for scores up to `top`, at least `mr`.  Beside a score of 2^27 a step of 32 bits is
// 2^4, and P_SHIFT below it would be rounded to 16 below: P of 2^16, an infinity in fp16.
__device__ __forceinline__ float reference(float top, float mr)
{
    const float y = top - P_SHIFT;
    return fmaxf(top - y > P_SHIFT + MAX_SLACK ? top : y, mr);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint64_t policy)
{
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(src), "l"(policy)
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
__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v)
{
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}
__device__ __forceinline__ float lds_half(uint32_t a)
{
    unsigned short v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return __half2float(__ushort_as_half(v));
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
__device__ __forceinline__ float inv_pow2(float x)       // 1 / x of a power of two
{
    return __uint_as_float((254u << 23) - __float_as_uint(x));
}

// The V scales' powers of two.  Lane `lane` keeps those of the two blocks that its scale words
// hold (words lane, lane + 32, ... of rows of NJ / 2 words: blocks 2 (lane % (NJ / 2)) and the
// next), the same in every lane of these blocks.
template <int NJ>
struct Carry {
    __half2 f;       // 2^-e: the scales are used times this
    __half2 limit;   // a scale above it calls for another
    __device__ __forceinline__ void reset()
    {
        f = __float2half2_rn(1.f);
        limit = __float2half2_rn(0.f);
    }
    // 2^-e for a largest scale of x > 0: x * 2^-e in [1/2, 1), or less from 2^-14 down
    static __device__ __forceinline__ float factor(float x)
    {
        const int ex = static_cast<int>((__float_as_uint(x) >> 23) & 255u) - 126;
        return pow2(-min(max(ex, -14), 16));
    }
    // vm: the largest of this lane's words.  Takes the new powers and gives each block's
    // rescale(j, new / old), by all lanes.
    template <typename F>
    __device__ __forceinline__ void grow(__half2 vm, F rescale)
    {
#pragma unroll
        for (int mask = NJ / 2; mask <= 16; mask <<= 1)
            vm = __hmax2(vm, as_half2(__shfl_xor_sync(0xffffffffu, as_u32(vm), mask)));
        const float2 x = __half22float2(vm), lim = __half22float2(limit);
        const float2 old = __half22float2(f);
        float2 to = old, top = lim;
        if (x.x > lim.x) {
            to.x = factor(x.x);
            top.x = fminf(2.f * inv_pow2(to.x), 65504.f);
        }
        if (x.y > lim.y) {
            to.y = factor(x.y);
            top.y = fminf(2.f * inv_pow2(to.y), 65504.f);
        }
        f = __floats2half2_rn(to.x, to.y);
        limit = __floats2half2_rn(top.x, top.y);
        const float r0 = to.x * inv_pow2(old.x), r1 = to.y * inv_pow2(old.y);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            rescale(j, __shfl_sync(0xffffffffu, j & 1 ? r1 : r0, j / 2));
    }
    // 2^e of block j, by all lanes
    __device__ __forceinline__ float undo(int j) const
    {
        const float2 x = __half22float2(f);
        return inv_pow2(__shfl_sync(0xffffffffu, j & 1 ? x.y : x.x, j / 2));
    }
};
// C = A . B, fp16 operands
__device__ __forceinline__ void mma_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// C += A . B, tf32 operands (fp32 values of which 10 fraction bits count)
__device__ __forceinline__ void mma_tf32(float (&d)[4], float a0, float a1, float a2, float a3,
                                         float b0, float b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)),
          "r"(__float_as_uint(a3)), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

// Swizzled offset of 16-byte chunk c of code row r: the 8 lanes of every
// shared-memory phase of the K and V reads fall into different banks.
template <int D>
__device__ __forceinline__ int code_off(int r, int c)
{
    return D == 128 ? r * 64 + ((c ^ ((r >> 1) & 3)) << 4) : r * 128 + ((c ^ (r & 7)) << 4);
}

// A producer's cache rows.  The lanes of a warp look up 32 tiles of pw's unit side by
// side (lane x: tile k + x), with the next 32 tiles' block ids already on their way.
struct Feed {
    int tpp;                     // tiles per page
    int k = 0, row = -1, blk = 0;
    unsigned have = 0;           // bit x: tile k + x is mapped

    __device__ __forceinline__ Feed(const Params &p) : tpp(p.page_size / TILE) {}
    __device__ __forceinline__ int block_of(const Params &p, const tc::Walk &pw, int x) const
    {
        const int ti = pw.lo / TILE + x;
        return x < pw.n ? p.bt[(long long)pw.b * p.max_blocks + (tpp == 1 ? ti : ti / tpp)] : 0;
    }
    // tiles pw.k .. pw.k + 31; `next`: they follow the window before
    __device__ __forceinline__ void window(const Params &p, const tc::Walk &pw, int left, bool next)
    {
        const int lane = threadIdx.x & 31;
        const int kv = pw.j / p.n_hg, x = pw.k + lane, ti = pw.lo / TILE + x;
        k = pw.k;
        row = -1;
        if (!p.bt) {
            if (x < pw.n)
                row = static_cast<int>(((long long)pw.b * p.Hkv + kv) * p.cap + ti * TILE);
        } else {
            const int id = next ? blk : block_of(p, pw, x);
            blk = block_of(p, pw, x + 32);
            if (x < pw.n && id >= 0 && id < p.num_blocks)
                row = (id * p.Hkv + kv) * p.page_size + (tpp == 1 ? 0 : ti % tpp * TILE);
            else if (lane < left && x < pw.n)    // a tile of this worker's
                flag(FA_STATUS_BAD_BLOCK);
        }
        have = __ballot_sync(0xffffffffu, row >= 0);
    }
    // the lane that holds tile pw.k, with the N - 1 tiles after it in the next lanes
    // (units are walked in steps of N from a window's start)
    template <int N>
    __device__ __forceinline__ int at(const Params &p, const tc::Walk &pw, int left)
    {
        if (pw.k - k > 32 - N)
            window(p, pw, left, pw.k - k == 32);
        return pw.k - k;
    }
};

// NG: groups of 8 columns per warp.  With two, a tile is unpacked once for 16
// columns (speculative verify).
// CL, the plan of small steps: one thread-block cluster of p.cl_ctas CTAs per unit,
// its warps sharing the unit's tiles evenly and folding their partials through
// distributed shared memory, which saves the merge kernel.
template <int D, int NG, bool WT, bool CL>
__global__ void __launch_bounds__(Cfg<D, NG>::NW * 32, Cfg<D, NG>::CTAS_PER_SM)
    decode_kernel(const Params p)
{
    using C = Cfg<D, NG>;
    constexpr int NJ = C::NJ, S = C::STAGES, COLS = GPH * NG;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2;         // mma row group: a key of K, a 4-element group of V
    const int t = lane & 3;          // mma column pair: an octet of K, a key pair of V
    const int w = blockIdx.x * C::NW + warp;
    int b_at = -1, We = 0;
    long long P_at = 0, T = 0, t0 = 0, t1 = 0;
    uint32_t rank = 0;               // in the cluster
    if constexpr (CL)
        asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    else if (!tc::stream_range(p, w, T, We, t0, t1, b_at, P_at))
        return;

    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t ring = smem_u32(smem) + warp * (S * C::STAGE_BYTES);
    const uint64_t policy = evict_first_policy();

    tc::Walk pw;
    int n_my = 0;                    // tiles in [t0, t1)
    if constexpr (CL) {
        const int unit = blockIdx.x / p.cl_ctas, R = p.cl_ctas * C::NW, r = rank * C::NW + warp;
        pw.b = unit / p.U_b;
        pw.j = unit % p.U_b;
        pw.c = 0;
        pw.P = 0;
        attended_range(p, pw.b, pw.lo, pw.hi, pw.j == 0 && r == 0);
        pw.n = tiles_in<TILE>(pw.lo, pw.hi);
        pw.k = static_cast<int>((long long)pw.n * r / R);
        n_my = static_cast<int>((long long)pw.n * (r + 1) / R) - pw.k;
    } else {
        pw.init(p, b_at, P_at, t0, tc::UNIT_COST);
    }
    tc::Walk cw = pw;
    if constexpr (!CL) {
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

    // ---- producer: the next batch, pw.k .. pw.k + n - 1 of pw's unit
    constexpr int BT = C::BT;
    int left = n_my;
    Feed f(p);
    constexpr int CPR = C::RB / 16;              // code chunks per row
    constexpr int NCP = TILE * CPR / 32;         // code chunks per lane and tile, K or V
    constexpr int NSC = TILE * C::SB / 16;       // scale chunks per tile, K or V
    const uint32_t d_code = code_off<D>(lane / CPR, lane % CPR);
    const uint32_t d_scale = (lane >= NSC ? C::VS_OFF : C::KS_OFF) + lane % NSC * 16;
    const char *k_src = p.k + lane * 16, *v_src = p.v + lane * 16;
    const char *s_src = (lane >= NSC ? p.vs : p.ks) + lane % NSC * 16;
    unsigned loaded = 0;                         // BT bits per stage: the tiles it holds
    int s_put = 0;                               // stage of the next batch
    auto copy_tile = [&](uint32_t st, int x, int r) {
        const char *kp = k_src + (long long)r * C::RB;
        const char *vp = v_src + (long long)r * C::RB;
        const uint32_t dst = st + d_code + x * TILE * C::RB;
#pragma unroll
        for (int i = 0; i < NCP; ++i) {
            // at D = 256 every second chunk flips the swizzle's bit 2
            const uint32_t at = D == 256 && (i & 1) ? (dst ^ 64u) : dst;
            cp16(at + C::K_OFF + i * 512, kp + i * 512, policy);
            cp16(at + C::V_OFF + i * 512, vp + i * 512, policy);
        }
        if (lane < 2 * NSC)
            cp16(st + d_scale + x * TILE * C::SB, s_src + (long long)r * C::SB, policy);
    };
    auto put = [&] {                             // an empty group past the end
        if (left > 0) {
            const int n = min(min(BT, pw.n - pw.k), left);
            const int x0 = f.at<BT>(p, pw, left);
            const unsigned have = (f.have >> x0) & ((1u << n) - 1u);
            loaded = (loaded & ~(((1u << BT) - 1u) << (s_put * BT))) | have << (s_put * BT);
            const uint32_t st = ring + s_put * C::STAGE_BYTES;
            if (have == (1u << BT) - 1u) {
#pragma unroll
                for (int x = 0; x < BT; ++x)
                    copy_tile(st, x, __shfl_sync(0xffffffffu, f.row, x0 + x));
            } else {
#pragma unroll 1
                for (int x = 0; x < n; ++x)
                    if ((have >> x) & 1u)
                        copy_tile(st, x, __shfl_sync(0xffffffffu, f.row, x0 + x));
            }
            left -= n;
            pw.k += n;
            if (pw.k == pw.n && left > 0) {
                --pw.k;
                pw.next(p);
                f.window(p, pw, left, false);
            }
            s_put = s_put + 1 == S ? 0 : s_put + 1;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (n_my > 0)
        f.window(p, pw, left, false);
#pragma unroll 1
    for (int i = 0; i < S - 1; ++i)
        put();

    // ---- the unit's queries: column g's elements (n, n+4) of octet t of block j
    // as half2, odd n a 16th of even ones; and column g's offset terms in two tf32 parts
    const int tq = p.tq > 1 ? p.tq : 1;
    uint32_t qb[NG][NJ][4];
    float ct[NG][NJ / 4][2];         // of block 4i + t
    int nh = 0, clo[NG][2], chi[NG][2], all_lo = 0, all_hi = 0, base = 0;
    float *scores = nullptr;         // WT: the unit's
    float c2[NG][2];                 // a sum's log2 units: columns 2t, 2t + 1
    auto load_q = [&] {
        base = cw.tok();
        if constexpr (WT)
            scores = p.ws_s + cw.unit(p) * p.cap16 * p.sh;
        const int kv = cw.j / p.n_hg, cg = cw.j % p.n_hg;
        nh = min(COLS, tq * p.G - cg * COLS);
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
            const tc::Col cq = tc::column(p, kv, cg, gi * GPH + g, COLS);
            const uint4 *src = reinterpret_cast<const uint4 *>(
                p.q + (((long long)cw.b * tq + cq.j) * p.Hq + cq.h) * D);
            // even elements times 16 / down, odd ones over down; whether every block's sum is
            // finite
            auto hold = [&](auto any, const bool low) {
                constexpr bool ANY = decltype(any)::value;       // a column may be held low
                const float down = ANY && low ? 16.f : 1.f;
                const __half2 even = __float2half2_rn(ANY && low ? 1.f : 16.f);
                const __half2 odd = __float2half2_rn(ANY && low ? 0.0625f : 1.f);
                uint4 x[NJ];
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    x[j] = cq.live ? __ldg(src + j * 4 + t) : make_uint4(0u, 0u, 0u, 0u);
                bool finite = true;
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    uint32_t *q = qb[gi][j];
                    q[0] = as_u32(__hmul2(as_half2(__byte_perm(x[j].x, x[j].z, 0x5410)), even));
                    q[1] = __byte_perm(x[j].x, x[j].z, 0x7632);                        // 1, 5
                    q[2] = as_u32(__hmul2(as_half2(__byte_perm(x[j].y, x[j].w, 0x5410)), even));
                    q[3] = __byte_perm(x[j].y, x[j].w, 0x7632);                        // 3, 7
                    if constexpr (ANY) {
                        q[1] = as_u32(__hmul2(as_half2(q[1]), odd));
                        q[3] = as_u32(__hmul2(as_half2(q[3]), odd));
                    }
                    float sum = 0.f;
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const float2 v = __half22float2(as_half2(q[n]));
                        sum += (v.x + v.y) * (n & 1 ? 16.f : 1.f);
                    }
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    finite = finite && fabsf(sum) < INFINITY;
                    if (j % 4 == t) {
                        sum *= -0.5f * down * p.c2;                    // log2 units
                        ct[gi][j / 4][0] = __uint_as_float(__float_as_uint(sum) & 0xffffe000u);
                        ct[gi][j / 4][1] = sum - ct[gi][j / 4][0];
                    }
                }
                return finite;
            };
            const bool low = !hold(std::false_type(), false);    // of all four lanes of a column
            const unsigned lows = __ballot_sync(0xffffffffu, low);
            if (lows)
                hold(std::true_type(), low);
            c2[gi][0] = p.c2 * ((lows >> (8 * t)) & 1u ? 16777216.f : 1048576.f);
            c2[gi][1] = p.c2 * ((lows >> (8 * t + 4)) & 1u ? 16777216.f : 1048576.f);
#pragma unroll
            for (int x1 = 0; x1 < 2; ++x1) {
                const tc::Col c = tc::column(p, kv, cg, gi * GPH + 2 * t + x1, COLS);
                tc::column_range(p, cw.b, cw.hi, c.live ? c.j : tq - 1, clo[gi][x1], chi[gi][x1]);
            }
        }
        int x0;
        tc::column_range(p, cw.b, cw.hi, tq - 1, all_lo, x0);   // keys every query attends
        tc::column_range(p, cw.b, cw.hi, 0, x0, all_hi);
    };

    // [2j + i]: elements 32j + 4g + 2i (0, 1: columns 2t, 2t+1; times 2^-24) and
    // + 1 (2, 3; times 2^-20)
    float acc[NG][2 * NJ][4];
    float mr[NG][2], l[NG][2];       // reference (the running maximum less P_SHIFT), sum of P
    Carry<NJ> cv;                    // block j of O is held times 2^-e_j
    auto reset = [&] {
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
#pragma unroll
            for (int i = 0; i < 2 * NJ; ++i)
                acc[gi][i][0] = acc[gi][i][1] = acc[gi][i][2] = acc[gi][i][3] = 0.f;
            mr[gi][0] = mr[gi][1] = NO_MAX;
            l[gi][0] = l[gi][1] = 0.f;
        }
        cv.reset();
    };
    if (n_my > 0)
        load_q();
    reset();
    const uint32_t half_sel = g & 1 ? 0x7632 : 0x5410;
    // lane's places in a stage: K rows g, V rows 2t, scales
    uint32_t kc[NJ / 4], vc[2][NJ / 4];
#pragma unroll
    for (int q = 0; q < NJ / 4; ++q) {
        kc[q] = C::K_OFF + code_off<D>(g, D == 128 ? t : 2 * t + q);
        vc[0][q] = C::V_OFF + code_off<D>(2 * t, D == 128 ? g >> 1 : 2 * (g >> 1) + q);
        vc[1][q] = C::V_OFF + code_off<D>(2 * t + 1, D == 128 ? g >> 1 : 2 * (g >> 1) + q);
    }

    int s = 0;
    for (int i = 0; i < n_my;) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        __syncwarp();                 // the batch has landed; every lane is done with the last
        const unsigned have_all = loaded >> (s * BT);
        const int nb = min(min(BT, cw.n - cw.k), n_my - i);
        const uint32_t stage = ring + s * C::STAGE_BYTES;
        s = s + 1 == S ? 0 : s + 1;
        put();

#pragma unroll 1
        for (int hh = 0; hh < nb; hh += 2) {
        const uint32_t st = stage + hh * TILE * C::RB;       // codes and scales of this pair
        const uint32_t ss = stage + hh * TILE * C::SB;
        const unsigned have = (have_all >> hh) & 3u;
        // ---- scores of tile h: rows are keys g and g + 8, columns 2t and 2t + 1
        float sc[NG][2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float a4[NG][4], off[NG][4];
#pragma unroll
            for (int gi = 0; gi < NG; ++gi)
                off[gi][0] = off[gi][1] = off[gi][2] = off[gi][3] = 0.f;
#pragma unroll
            for (int jj = 0; jj < NJ; jj += 4) {
                const uint32_t row = st + h * TILE * C::RB;
                const uint32_t srow = ss + C::KS_OFF + (h * TILE + g) * C::SB + jj * 2;
                // 8 rows down the swizzle is the same
                const uint4 wa = lds128(row + kc[jj / 4]);
                const uint4 wb = lds128(row + kc[jj / 4] + 8 * C::RB);
                const uint2 sa = lds64(srow);
                const uint2 sb = lds64(srow + 8 * C::SB);
                const float ta = lds_half(srow + 2 * t), tb = lds_half(srow + 8 * C::SB + 2 * t);
#pragma unroll
                for (int gi = 0; gi < NG; ++gi)
                    mma_tf32(off[gi], ta, tb, ta, tb, ct[gi][jj / 4][0], ct[gi][jj / 4][1]);
                const uint32_t a[4] = {wa.x, wa.y, wa.z, wa.w};
                const uint32_t b[4] = {wb.x, wb.y, wb.z, wb.w};
                const float2 fa[2] = {__half22float2(as_half2(sa.x)), __half22float2(as_half2(sa.y))};
                const float2 fb[2] = {__half22float2(as_half2(sb.x)), __half22float2(as_half2(sb.y))};
                float d[NG][4][4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int gi = 0; gi < NG; ++gi)
                        mma_zero(d[gi][q], a[q] & 0x000f000fu, b[q] & 0x000f000fu,
                                 a[q] & 0x00f000f0u, b[q] & 0x00f000f0u, qb[gi][jj + q][0],
                                 qb[gi][jj + q][1]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t ah = a[q] >> 8, bh = b[q] >> 8;
#pragma unroll
                    for (int gi = 0; gi < NG; ++gi)
                        tc::mma16816(d[gi][q], ah & 0x000f000fu, bh & 0x000f000fu,
                                     ah & 0x00f000f0u, bh & 0x00f000f0u, qb[gi][jj + q][2],
                                     qb[gi][jj + q][3]);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float ka = q & 1 ? fa[q / 2].y : fa[q / 2].x;
                    const float kb = q & 1 ? fb[q / 2].y : fb[q / 2].x;
#pragma unroll
                    for (int gi = 0; gi < NG; ++gi) {
                        const float *x = d[gi][q];
                        float *y = a4[gi];
                        y[0] = jj + q ? fmaf(x[0], ka, y[0]) : x[0] * ka;
                        y[1] = jj + q ? fmaf(x[1], ka, y[1]) : x[1] * ka;
                        y[2] = jj + q ? fmaf(x[2], kb, y[2]) : x[2] * kb;
                        y[3] = jj + q ? fmaf(x[3], kb, y[3]) : x[3] * kb;
                    }
                }
            }
#pragma unroll
            for (int gi = 0; gi < NG; ++gi)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    sc[gi][h][q] = fmaf(a4[gi][q], c2[gi][q & 1], off[gi][q]);   // log2 units
        }
        // the pair's V scales, a few words per lane, against the limit
        constexpr int NVW = 2 * TILE * NJ / 2 / 32;
        uint32_t vw[NVW];
#pragma unroll
        for (int q = 0; q < NVW; ++q)
            vw[q] = lds32(ss + C::VS_OFF + (lane + 32 * q) * 4);
        // ---- tile edges, and the ranges of several queries
        const bool edge = base < all_lo || base + 2 * TILE > all_hi || have != 3u;
        // the pair's keys that are there at all; other rows hold anything
        auto there = [&](int k) {
            return k >= cw.lo - base && k < cw.hi - base && ((have >> (k / TILE)) & 1u);
        };
        if (edge) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int ka = base + h * TILE + g, kb = ka + 8;
                const bool un = !((have >> h) & 1u);
#pragma unroll
                for (int gi = 0; gi < NG; ++gi)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (un || ka < clo[gi][x] || ka >= chi[gi][x])
                            sc[gi][h][x] = -INFINITY;
                        if (un || kb < clo[gi][x] || kb >= chi[gi][x])
                            sc[gi][h][2 + x] = -INFINITY;
                    }
            }
            // other rows must not turn a zero weight into NaN
#pragma unroll
            for (int q = 0; q < NVW; ++q)
                if (!there((lane + 32 * q) / (NJ / 2)))
                    vw[q] = 0u;
        }
        if constexpr (WT) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if ((have >> h) & 1u)
#pragma unroll
                    for (int gi = 0; gi < NG; ++gi)
                        tc::store_scores(scores, p.sh, base + h * TILE + g, base + h * TILE + g + 8,
                                         gi * GPH + 2 * t, nh, sc[gi][h]);
        }
        // ---- online softmax
        __half2 vm = as_half2(vw[0]);
#pragma unroll
        for (int q = 1; q < NVW; ++q)
            vm = __hmax2(vm, as_half2(vw[q]));
        float top[NG][2];
        const bool big = !__hble2(vm, cv.limit);
        bool over = big;
#pragma unroll
        for (int gi = 0; gi < NG; ++gi)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                top[gi][x] = fmaxf(fmaxf(sc[gi][0][x], sc[gi][0][2 + x]),
                                   fmaxf(sc[gi][1][x], sc[gi][1][2 + x]));
                over = over || top[gi][x] - mr[gi][x] > P_SHIFT + MAX_SLACK;
            }
        if (__any_sync(0xffffffffu, over)) {
            if (__any_sync(0xffffffffu, big))
                cv.grow(vm, [&](int j, float r) {
#pragma unroll
                    for (int gi = 0; gi < NG; ++gi)
#pragma unroll
                        for (int ii = 2 * j; ii < 2 * j + 2; ++ii) {
                            acc[gi][ii][0] *= r;
                            acc[gi][ii][1] *= r;
                            acc[gi][ii][2] *= r;
                            acc[gi][ii][3] *= r;
                        }
                });
#pragma unroll
            for (int gi = 0; gi < NG; ++gi)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float y = top[gi][x];
#pragma unroll
                    for (int mask = 4; mask <= 16; mask <<= 1)
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, mask));
                    y = reference(y, mr[gi][x]);
                    const float a = ex2_ftz(mr[gi][x] - y);
                    l[gi][x] *= a;
                    mr[gi][x] = y;
#pragma unroll
                    for (int ii = 0; ii < 2 * NJ; ++ii) {
                        acc[gi][ii][x] *= a;
                        acc[gi][ii][2 + x] *= a;
                    }
                }
        }
#pragma unroll
        for (int q = 0; q < NVW; ++q)
            sts32(ss + C::VS_OFF + (lane + 32 * q) * 4, as_u32(__hmul2(as_half2(vw[q]), cv.f)));
        __syncwarp();
        // ---- O^T += V^T . (P s)^T: rows are elements, 4 per block and lane
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // P^T as the B operand: keys (2t, 2t+1) and (2t+8, 2t+9), column g
            __half2 pa[NG], pb[NG];
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
                const float *x = sc[gi][h];
                const float p0 = ex2_ftz(x[0] - mr[gi][0]), p1 = ex2_ftz(x[1] - mr[gi][1]);
                const float p2 = ex2_ftz(x[2] - mr[gi][0]), p3 = ex2_ftz(x[3] - mr[gi][1]);
                l[gi][0] += p0 + p2;
                l[gi][1] += p1 + p3;
                pa[gi] = as_half2(tc::movmatrix_t(tc::pack_half2(p0, p1)));
                pb[gi] = as_half2(tc::movmatrix_t(tc::pack_half2(p2, p3)));
            }
            // V scales as half2 over the same key pairs
            __half2 sv[2][NJ];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t u[NJ];       // the two keys' scales: NJ / 2 words each
#pragma unroll
                for (int q = 0; q < NJ / 4; ++q) {
                    const uint4 v = lds128(ss + C::VS_OFF + (h * TILE + 2 * t + 8 * x) * C::SB +
                                           q * 16);
                    u[4 * q] = v.x; u[4 * q + 1] = v.y; u[4 * q + 2] = v.z; u[4 * q + 3] = v.w;
                }
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    sv[x][j] = as_half2(__byte_perm(u[j / 2], u[NJ / 2 + j / 2],
                                                    j & 1 ? 0x7632 : 0x5410));
            }
#pragma unroll
            for (int jj = 0; jj < NJ; jj += 4) {
                const uint32_t row = st + h * TILE * C::RB;
                uint32_t v[4][4];     // keys 2t, 2t+1, 2t+8, 2t+9
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint4 x = lds128(row + vc[q & 1][jj / 4] + (q >> 1) * 8 * C::RB);
                    v[q][0] = x.x; v[q][1] = x.y; v[q][2] = x.z; v[q][3] = x.w;
                }
                auto even = [](uint32_t z) {
                    return as_u32(__hsub2(as_half2(z & 0x000f000fu), as_half2(0x00080008u)));
                };
                auto odd = [](uint32_t z) {
                    return as_u32(__hsub2(as_half2(z & 0x00f000f0u), as_half2(0x00800080u)));
                };
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int j = jj + q;
                    const uint32_t x = __byte_perm(v[0][q], v[1][q], half_sel);
                    const uint32_t y = __byte_perm(v[2][q], v[3][q], half_sel);
                    const uint32_t xh = x >> 8, yh = y >> 8;
                    const uint32_t a[4] = {even(x), odd(x), even(y), odd(y)};
                    const uint32_t b[4] = {even(xh), odd(xh), even(yh), odd(yh)};
#pragma unroll
                    for (int gi = 0; gi < NG; ++gi) {
                        const uint32_t s0 = as_u32(__hmul2(pa[gi], sv[0][j]));
                        const uint32_t s1 = as_u32(__hmul2(pb[gi], sv[1][j]));
                        tc::mma16816(acc[gi][2 * j], a[0], a[1], a[2], a[3], s0, s1);
                        tc::mma16816(acc[gi][2 * j + 1], b[0], b[1], b[2], b[3], s0, s1);
                    }
                }
            }
        }

        base += 2 * TILE;
        }   // pairs of the batch

        i += nb;
        cw.k += nb;
        if constexpr (CL)
            continue;                // one segment, folded below
        if (cw.k == cw.n || i == n_my) {
            // ---- end of this worker's segment of the unit
            const long long us = cw.unit_start();
            const bool whole = tc::worker_of(us, T, We) == tc::worker_of(us + cw.n - 1, T, We);
            const int kv = cw.j / p.n_hg, cg = cw.j % p.n_hg;
            const long long slot = w + cw.unit(p);
            float un[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                un[j] = cv.undo(j);
#pragma unroll
            for (int gi = 0; gi < NG; ++gi)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float lx = l[gi][x];
#pragma unroll
                    for (int mask = 4; mask <= 16; mask <<= 1)
                        lx += __shfl_xor_sync(0xffffffffu, lx, mask);
                    const int h = gi * GPH + 2 * t + x;
                    if (h >= nh)
                        continue;
                    const float mx = mr[gi][x] == NO_MAX ? -INFINITY : mr[gi][x];
                    // 2^24 and 2^20 as the accumulators hold them; l = 0 only without keys
                    const float up0 = whole && lx > 0.f ? pow2(20) / lx : pow2(20);
                    auto four = [&](int j) {
                        const float up = up0 * un[j], up16 = up * 16.f;
                        return make_float4(acc[gi][2 * j][x] * up16, acc[gi][2 * j][x + 2] * up,
                                           acc[gi][2 * j + 1][x] * up16,
                                           acc[gi][2 * j + 1][x + 2] * up);
                    };
                    if (whole) {
                        const tc::Col cc = tc::column(p, kv, cg, h, COLS);
                        const long long r = ((long long)cw.b * tq + cc.j) * p.Hq + cc.h;
                        __half *o = reinterpret_cast<__half *>(p.out) + r * D + 4 * g;
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
                            tc::store4(o + 32 * j, four(j));
                        if (WT && g == 0)
                            p.lse[r] = lx > 0.f ? mx + log2f(lx) : -INFINITY;
                    } else {
                        float *o = p.ws_o + (slot * p.sh + h) * D + 4 * g;
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
                            tc::store4(o + 32 * j, four(j));
                        if (g == 0)
                            p.ws_ml[slot * p.sh + h] = make_float2(mx, lx);
                    }
                }
            reset();
            if (i < n_my) {
                --cw.k;
                cw.next(p);
                load_q();
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if constexpr (CL) {
        // ---- the unit's partials: of every warp (m, l) of 8 columns, then O [8][D], in
        // its ring; folded by all threads of the cluster, 32 elements of a column per warp
        __syncwarp();
        float un[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            un[j] = cv.undo(j) * pow2(20);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float lx = l[0][x];
#pragma unroll
            for (int mask = 4; mask <= 16; mask <<= 1)
                lx += __shfl_xor_sync(0xffffffffu, lx, mask);
            const int h = 2 * t + x;
            const uint32_t o = ring + 64 + (h * D + 4 * g) * 4;
            if (g == 0) {
                sts32(ring + h * 8, __float_as_uint(mr[0][x] == NO_MAX ? -INFINITY : mr[0][x]));
                sts32(ring + h * 8 + 4, __float_as_uint(lx));
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                sts128(o + j * 128, __float_as_uint(acc[0][2 * j][x] * (16.f * un[j])),
                       __float_as_uint(acc[0][2 * j][x + 2] * un[j]),
                       __float_as_uint(acc[0][2 * j + 1][x] * (16.f * un[j])),
                       __float_as_uint(acc[0][2 * j + 1][x + 2] * un[j]));
        }
        tc::cluster_sync();
        const int R = p.cl_ctas * C::NW, kv = pw.j / p.n_hg, cg = pw.j % p.n_hg;
        const int live = min(GPH, tq * p.G - cg * GPH);
        const uint32_t rings = smem_u32(smem);
        for (int i = rank * C::NW + warp; i < live * (D / 32); i += R) {
            const int h = i / (D / 32), d = i % (D / 32) * 32 + lane;
            // lane r has warp r's (m, l)
            const uint32_t mine = tc::cl_map(rings + lane % C::NW * (S * C::STAGE_BYTES), lane / C::NW);
            const float2 ml = lane < R ? tc::cl_ld2(mine + h * 8) : make_float2(-INFINITY, 0.f);
            float M = ml.x;
#pragma unroll
            for (int mask = 16; mask >= 1; mask >>= 1)
                M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, mask));
            const float a = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
            float L = a * ml.y;
#pragma unroll
            for (int mask = 16; mask >= 1; mask >>= 1)
                L += __shfl_xor_sync(0xffffffffu, L, mask);
            float sum = 0.f;
#pragma unroll 8
            for (int r = 0; r < R; ++r) {
                const uint32_t at = tc::cl_map(rings + r % C::NW * (S * C::STAGE_BYTES), r / C::NW);
                float y;
                asm volatile("ld.shared::cluster.f32 %0, [%1];"
                             : "=f"(y)
                             : "r"(at + 64 + (h * D + d) * 4)
                             : "memory");
                const float ar = __shfl_sync(0xffffffffu, a, r);
                sum = ar > 0.f ? fmaf(y, ar, sum) : sum;
            }
            const tc::Col cc = tc::column(p, kv, cg, h, GPH);
            reinterpret_cast<__half *>(p.out)[(((long long)pw.b * tq + cc.j) * p.Hq + cc.h) * D + d] =
                __float2half_rn(L == 0.f ? 0.f : sum / L);
        }
        if constexpr (WT)            // the plan gives one column group per KV head
            if (n_my > 0) {
                const int first = pw.lo / TILE + static_cast<int>((long long)pw.n * (rank * C::NW + warp) / R);
                tc::add_cluster_weights(
                    p, pw.b, pw.j, max(pw.lo, first * TILE), min(pw.hi, (first + n_my) * TILE), live,
                    p.ws_s + cw.unit(p) * p.cap16 * p.sh, R, [&](int r, int c) {
                        return tc::cl_ld2(tc::cl_map(rings + r % C::NW * (S * C::STAGE_BYTES),
                                                     r / C::NW) + c * 8);
                    });
            }
        tc::cluster_sync();          // no CTA leaves while its partials are read
    }
}

// ------------------------------------------------- attention, many columns
// 64 (query, head) columns per unit, for calls with many of them: a CTA of four
// warps unpacks a tile of KT keys once into shared memory as fp16 codes, and its
// warps share it, 16 columns each (the mma's M: S[16 columns x keys] = Q . K^T,
// whose accumulators are the A operand of O[16 x D] += (P s) . V without a
// transpose).  Scales are used as above, K's in fp32 after each block's mma, V's on
// the weights.  Work is split as above with CTAs as workers.
// Bound by the instructions between its two barriers per tile; see WIDE_GROUPS for
// where it wins.  (Deeper prefetch and tiles of 128 keys changed nothing; 32 columns
// with the keys in two slices lost to the kernel above.)
template <int D>
struct WideCfg {
    static constexpr int KT = D == 128 ? 64 : 32;      // keys per tile
    static constexpr int SUB = KT / TILE;              // 16-key subtiles per tile
    static constexpr int CK = 32;                      // keys per softmax step
    static constexpr int COLS = 64;
    static constexpr int NJ = D / 32, RB = D / 2, SB = D / 16;
    static constexpr int RAW_K = 0, RAW_V = KT * RB;   // codes as copied (swizzled rows)
    static constexpr int SC = 2 * KT * RB;             // two stages of K scales, V scales
    static constexpr int SC_STAGE = 2 * KT * SB;
    static constexpr int F16_K = SC + 2 * SC_STAGE;    // codes as fp16, rows of 2 D bytes
    static constexpr int F16_V = F16_K + KT * D * 2;
    static constexpr int Q = F16_V + KT * D * 2;       // the unit's queries
    static constexpr int VS = Q + COLS * D * 2;        // the tile's V scales as they are used
    static constexpr int SMEM = VS + KT * SB;
    static constexpr int CTAS_PER_SM = D == 128 ? 3 : 2;
    static_assert(F16_K % 128 == 0 && Q % 128 == 0, "swizzled rows");
    static_assert(KT * SB / 4 == 128, "a word of V scales per thread");
    static_assert(CTAS_PER_SM * (SMEM + 1024) <= 228 * 1024, "shared memory per SM");
};

// Byte offset of 16-byte chunk c of row r in rows of D fp16 values.
template <int D>
__device__ __forceinline__ int f16_off(int r, int c)
{
    return r * (2 * D) + ((c ^ (r & 7)) << 4);
}

template <int D, bool WT>
__global__ void __launch_bounds__(128, WideCfg<D>::CTAS_PER_SM) wide_kernel(const Params p)
{
    using C = WideCfg<D>;
    constexpr int NJ = C::NJ, KT = C::KT, SUB = C::SUB, CK = C::CK, NT = CK / 8;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int cwi = warp;                          // this warp's 16 columns
    const int w = blockIdx.x;
    int b_at = -1, We = 0;
    long long P_at = 0, T = 0, t0 = 0, t1 = 0;
    if (!tc::stream_range(p, w, T, We, t0, t1, b_at, P_at))
        return;                                    // the whole CTA: the range is the worker's

    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t sm = smem_u32(smem);
    const uint64_t policy = evict_first_policy();

    tc::Walk cw;
    cw.init(p, b_at, P_at, t0, tc::UNIT_COST);
    tc::Walk pw = cw;
    int n_my = 0;                                  // 16-key tiles in [t0, t1)
    {
        tc::Walk e = cw;
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
    if (n_my == 0)
        return;
    // ---- copies: warp x takes subtile x % SUB (at D = 256 its K with warps 0 and 1,
    // its V with 2 and 3)
    const int sub = warp % SUB;
    const bool does_k = warp < SUB, does_v = SUB == 4 || warp >= SUB;
    constexpr int CPR = C::RB / 16, NCP = TILE * CPR / 32, NSC = TILE * C::SB / 16;
    int left = n_my;
    unsigned mapped = 0;                           // SUB bits per stage: its mapped subtiles
    Feed f(p);
    uint32_t c_dst[NCP];
#pragma unroll
    for (int i = 0; i < NCP; ++i)
        c_dst[i] = sm + sub * TILE * C::RB + code_off<D>((lane + 32 * i) / CPR, (lane + 32 * i) % CPR);
    auto copy = [&](int stage) {                   // the next tile of pw's unit
        const int nb = min(min(SUB, pw.n - pw.k), left);
        const int x0 = f.at<SUB>(p, pw, left);
        const unsigned have = (f.have >> x0) & ((1u << nb) - 1u);
        mapped = (mapped & ~(((1u << SUB) - 1u) << (stage * SUB))) | have << (stage * SUB);
        const long long row = __shfl_sync(0xffffffffu, f.row, x0 + sub);
        if ((have >> sub) & 1u) {
            const char *kp = p.k + row * C::RB + lane * 16, *vp = p.v + row * C::RB + lane * 16;
#pragma unroll
            for (int i = 0; i < NCP; ++i) {
                if (does_k)
                    cp16(c_dst[i] + C::RAW_K, kp + i * 512, policy);
                if (does_v)
                    cp16(c_dst[i] + C::RAW_V, vp + i * 512, policy);
            }
            const uint32_t sc = sm + C::SC + stage * C::SC_STAGE + sub * TILE * C::SB;
            if (does_k && lane < NSC)
                cp16(sc + lane * 16, p.ks + row * C::SB + lane * 16, policy);
            if (does_v && lane >= 16 && lane < 16 + NSC)
                cp16(sc + KT * C::SB + (lane - 16) * 16, p.vs + row * C::SB + (lane - 16) * 16,
                     policy);
        }
        left -= nb;
        pw.k += nb;
        if (pw.k == pw.n && left > 0) {
            --pw.k;
            pw.next(p);
            f.window(p, pw, left, false);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    f.window(p, pw, left, false);

    // ---- the unit's queries in shared memory; every 8 elements in the order 0, 4,
    // 1, 5, 2, 6, 3, 7 that unpacking a word of codes gives
    const int tq = p.tq > 1 ? p.tq : 1;
    int nh = 0, clo[2], chi[2], all_lo = 0, all_hi = 0, base = 0;
    auto load_q = [&] {
        base = cw.tok();
        const int kv = cw.j / p.n_hg, cg = cw.j % p.n_hg;
        nh = min(C::COLS, tq * p.G - cg * C::COLS);
        for (int i = tid; i < C::COLS * (D / 8); i += 128) {
            const int r = i / (D / 8), c = i % (D / 8);
            const tc::Col q = tc::column(p, kv, cg, r, C::COLS);
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (q.live)
                x = __ldg(reinterpret_cast<const uint4 *>(
                              p.q + (((long long)cw.b * tq + q.j) * p.Hq + q.h) * D) + c);
            const uint4 y = make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                                       __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
            *reinterpret_cast<uint4 *>(smem + C::Q + f16_off<D>(r, c)) = y;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const tc::Col c = tc::column(p, kv, cg, cwi * 16 + g + 8 * x, C::COLS);
            tc::column_range(p, cw.b, cw.hi, c.live ? c.j : tq - 1, clo[x], chi[x]);
        }
        int x0;
        tc::column_range(p, cw.b, cw.hi, tq - 1, all_lo, x0);   // keys every query attends
        tc::column_range(p, cw.b, cw.hi, 0, x0, all_hi);
    };

    // [n]: columns g (0, 1) and g + 8 (2, 3), elements 8n + t (0, 2) and 8n + t + 4
    float acc[D / 8][4];
    float mr[2], l[2];
    Carry<NJ> cv;             // as above; every warp sees the same scales and keeps the same powers
    auto reset = [&] {
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        mr[0] = mr[1] = NO_MAX;
        l[0] = l[1] = 0.f;
        cv.reset();
    };
    // ---- this lane's places.  Chunk c of row r lies at (c ^ (r & 7)) * 16, so a lane
    // needs one address per value of c's low three bits; the rest are constants.
    // Unpacking: two code chunks of one key, K's and V's alike.
    uint32_t raw_a[2], f16_a[2][2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int key = tid % KT, c = tid / KT + x * (128 / KT);
        const int o = D == 128 ? c : c / 2;         // octet of the chunk's four words
        raw_a[x] = sm + C::RAW_K + code_off<D>(key, c);
#pragma unroll
        for (int z = 0; z < 2; ++z)
            f16_a[x][z] = sm + C::F16_K + f16_off<D>(key, 4 * z + o) +
                          (D == 256 ? (c & 1) * 256 : 0);
    }
    // ldmatrix: queries (16 rows, two chunks), K (8 rows, four chunks), V (16 rows, two)
    uint32_t q_a[4], k_a[2], v_a[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        q_a[x] = sm + C::Q + f16_off<D>(cwi * 16 + (lane & 15), 2 * x + (lane >> 4));
        v_a[x] = sm + C::F16_V + f16_off<D>(lane & 15, 2 * x + (lane >> 4));
        k_a[x & 1] = sm + C::F16_K + f16_off<D>(lane & 7, 4 * (x & 1) + (lane >> 3));
    }
    copy(0);
    load_q();
    reset();

    int stage = 0;
    for (int i = 0; i < n_my;) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();      // the tile has landed; every warp is done with the one before
        const int nb = min(min(SUB, cw.n - cw.k), n_my - i);
        const unsigned have = (mapped >> (stage * SUB)) & ((1u << SUB) - 1u);
        const uint32_t sc = sm + C::SC + stage * C::SC_STAGE;
        const bool edge = base < all_lo || base + KT > all_hi || have != (1u << SUB) - 1u;
        auto there = [&](int k) {                  // key k of the tile is attended by someone
            return k >= cw.lo - base && k < cw.hi - base && ((have >> (k / TILE)) & 1u);
        };
        {
            // V scales: every warp looks at all of them, a thread writes one word as it is used
            constexpr int NVW = KT * NJ / 2 / 32;
            uint32_t mine = 0;
            __half2 vm = __float2half2_rn(0.f);
#pragma unroll
            for (int q = 0; q < NVW; ++q) {
                const int x = lane + 32 * q;
                uint32_t v = lds32(sc + KT * C::SB + x * 4);
                // other rows must not turn a zero weight into NaN
                if (edge && !there(x / (NJ / 2))) {
                    v = 0u;
                    if (q == warp)
                        sts32(sc + x * 4, 0u);               // their K scales
                }
                vm = __hmax2(vm, as_half2(v));
                mine = q == warp ? v : mine;
            }
            if (__any_sync(0xffffffffu, !__hble2(vm, cv.limit)))
                cv.grow(vm, [&](int j, float r) {
#pragma unroll
                    for (int ii = 4 * j; ii < 4 * j + 4; ++ii) {
                        acc[ii][0] *= r;
                        acc[ii][1] *= r;
                        acc[ii][2] *= r;
                        acc[ii][3] *= r;
                    }
                });
            sts32(sm + C::VS + tid * 4, as_u32(__hmul2(as_half2(mine), cv.f)));
        }
        // ---- unpack: a word of codes is one 16-byte chunk of fp16 values.  8 lanes
        // take the same octet of 8 keys, so reads and writes meet no bank twice.
        {
            const __half2 b1032 = __float2half2_rn(1032.f), b72 = __float2half2_rn(72.f);
#pragma unroll
            for (int x = 0; x < 4; ++x) {                   // K, K, V, V
                const uint4 v = lds128(raw_a[x & 1] + (x >> 1) * (C::RAW_V - C::RAW_K));
                const uint32_t wds[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t a = wds[q], h = wds[q] >> 8;
                    auto even = [&](uint32_t z) {
                        return as_u32(__hsub2(as_half2((z & 0x000f000fu) | 0x64006400u), b1032));
                    };
                    auto odd = [&](uint32_t z) {
                        return as_u32(__hsub2(as_half2((z & 0x00f000f0u) | 0x54005400u), b72));
                    };
                    sts128(f16_a[x & 1][q & 1] + (x >> 1) * (C::F16_V - C::F16_K) + (q >> 1) * 128,
                           even(a), odd(a), even(h), odd(h));
                }
            }
        }
        __syncthreads();
        i += nb;
        const bool seg_end = cw.k + nb == cw.n || i == n_my;
        if (i < n_my)
            copy(stage ^ 1);

#pragma unroll 1
        for (int kk = 0; kk < nb * TILE; kk += CK) {
            // ---- scores: 8 keys per mma, blocks of 32 elements scaled in fp32
            float sc4[NT][4];
            float kscale[NT][2][4];
#pragma unroll
            for (int jj = 0; jj < NJ; jj += 4) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint2 u = lds64(sc + (kk + 8 * n + 2 * t + x) * C::SB + jj * 2);
                        const float2 f0 = __half22float2(as_half2(u.x));
                        const float2 f1 = __half22float2(as_half2(u.y));
                        kscale[n][x][0] = f0.x; kscale[n][x][1] = f0.y;
                        kscale[n][x][2] = f1.x; kscale[n][x][3] = f1.y;
                    }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int j = jj + q;
                    // A: 16 columns x 32 elements (chunks 4j .. 4j+3)
                    uint32_t a[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        tc::ldsm_x4(q_a[(2 * j + h) & 3] + (j >> 1) * 128, a[h][0], a[h][1], a[h][2],
                                    a[h][3]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        // B: 8 keys x 32 elements
                        uint32_t k0, k1, k2, k3;
                        tc::ldsm_x4(k_a[j & 1] + kk * (2 * D) + n * (16 * D) + (j >> 1) * 128, k0,
                                    k1, k2, k3);
                        float d[4];
                        mma_zero(d, a[0][0], a[0][1], a[0][2], a[0][3], k0, k1);
                        tc::mma16816(d, a[1][0], a[1][1], a[1][2], a[1][3], k2, k3);
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            sc4[n][x] = j ? fmaf(d[x], kscale[n][x & 1][q], sc4[n][x])
                                          : d[x] * kscale[n][x & 1][q];
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    sc4[n][x] *= p.c2;                     // log2 units
            if (edge) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int kt = kk + 8 * n + 2 * t + (x & 1), k = base + kt;
                        if (k < clo[x >> 1] || k >= chi[x >> 1] || !((have >> (kt / TILE)) & 1u))
                            sc4[n][x] = -INFINITY;
                    }
            }
            if constexpr (WT) {
                // of every column, 4 lanes write 8 neighbouring keys
                const int col = cwi * 16 + g;
                float *at = p.ws_s + ((cw.unit(p) * (p.cap16 / TILE) + (base + kk) / TILE) * p.sh +
                                      col) * TILE + 2 * t;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (!((have >> ((kk + 8 * n) / TILE)) & 1u))
                        continue;
                    float *a = at + (n / 2) * (p.sh * TILE) + (n & 1) * 8;
                    if (col < nh)
                        *reinterpret_cast<float2 *>(a) = make_float2(sc4[n][0], sc4[n][1]);
                    if (col + 8 < nh)
                        *reinterpret_cast<float2 *>(a + 8 * TILE) = make_float2(sc4[n][2], sc4[n][3]);
                }
            }
            // ---- online softmax (as above)
            float x0 = sc4[0][0], x1 = sc4[0][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                x0 = fmaxf(x0, fmaxf(sc4[n][0], sc4[n][1]));
                x1 = fmaxf(x1, fmaxf(sc4[n][2], sc4[n][3]));
            }
            const bool over = fmaxf(x0 - mr[0], x1 - mr[1]) > P_SHIFT + MAX_SLACK;
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int mask = 1; mask <= 2; mask <<= 1) {
                    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, mask));
                    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, mask));
                }
                const float n0 = reference(x0, mr[0]), n1 = reference(x1, mr[1]);
                const float a0 = ex2_ftz(mr[0] - n0), a1 = ex2_ftz(mr[1] - n1);
                l[0] *= a0;
                l[1] *= a1;
#pragma unroll
                for (int ii = 0; ii < D / 8; ++ii) {
                    acc[ii][0] *= a0;
                    acc[ii][1] *= a0;
                    acc[ii][2] *= a1;
                    acc[ii][3] *= a1;
                }
                mr[0] = n0;
                mr[1] = n1;
            }
            // ---- O += (P s) . V, 16 keys at a time
#pragma unroll
            for (int m = 0; m < CK / 16; ++m) {
                uint32_t pa[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float *s = sc4[2 * m + h];
                    const float p0 = ex2_ftz(s[0] - mr[0]), p1 = ex2_ftz(s[1] - mr[0]);
                    const float p2 = ex2_ftz(s[2] - mr[1]), p3 = ex2_ftz(s[3] - mr[1]);
                    l[0] += p0 + p1;
                    l[1] += p2 + p3;
                    pa[2 * h] = tc::pack_half2(p0, p1);
                    pa[2 * h + 1] = tc::pack_half2(p2, p3);
                }
                // V scales as half2 over the key pairs (2t, 2t+1) and (2t+8, 2t+9)
                __half2 sv[2][NJ];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t u[NJ];
#pragma unroll
                    for (int q = 0; q < NJ / 4; ++q) {
                        const uint4 v = lds128(sm + C::VS +
                                               (kk + 16 * m + 8 * x + 2 * t) * C::SB + q * 16);
                        u[4 * q] = v.x; u[4 * q + 1] = v.y; u[4 * q + 2] = v.z; u[4 * q + 3] = v.w;
                    }
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        sv[x][j] = as_half2(__byte_perm(u[j / 2], u[NJ / 2 + j / 2],
                                                        j & 1 ? 0x7632 : 0x5410));
                }
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const uint32_t a0 = as_u32(__hmul2(as_half2(pa[0]), sv[0][j]));
                    const uint32_t a1 = as_u32(__hmul2(as_half2(pa[1]), sv[0][j]));
                    const uint32_t a2 = as_u32(__hmul2(as_half2(pa[2]), sv[1][j]));
                    const uint32_t a3 = as_u32(__hmul2(as_half2(pa[3]), sv[1][j]));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // B: 16 keys x elements 32j + 16h .. + 15
                        uint32_t v0, v1, v2, v3;
                        tc::ldsm_x4_t(v_a[(2 * j + h) & 3] + kk * (2 * D) + m * (32 * D) +
                                          (j >> 1) * 128,
                                      v0, v1, v2, v3);
                        tc::mma16816(acc[4 * j + 2 * h], a0, a1, a2, a3, v0, v1);
                        tc::mma16816(acc[4 * j + 2 * h + 1], a0, a1, a2, a3, v2, v3);
                    }
                }
            }
        }
        stage ^= 1;
        cw.k += nb;
        base += nb * TILE;
        if (!seg_end)
            continue;

        // ---- end of this worker's segment of the unit
#pragma unroll
        for (int mask = 1; mask <= 2; mask <<= 1) {
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], mask);
            l[1] += __shfl_xor_sync(0xffffffffu, l[1], mask);
        }
        float un[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            un[j] = cv.undo(j);
        {
            const long long us = cw.unit_start();
            const bool whole = tc::worker_of(us, T, We) == tc::worker_of(us + cw.n - 1, T, We);
            const int kv = cw.j / p.n_hg, cg = cw.j % p.n_hg;
            const long long slot = w + cw.unit(p);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int c = cwi * 16 + g + 8 * x;
                if (c >= nh)
                    continue;
                const float mx = mr[x] == NO_MAX ? -INFINITY : mr[x];
                if (whole) {
                    const tc::Col cc = tc::column(p, kv, cg, c, C::COLS);
                    const long long r = ((long long)cw.b * tq + cc.j) * p.Hq + cc.h;
                    const float inv = l[x] > 0.f ? 1.f / l[x] : 0.f;
                    __half *o = reinterpret_cast<__half *>(p.out) + r * D + t;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[8 * n] = __float2half_rn(acc[n][2 * x] * (inv * un[n / 4]));
                        o[8 * n + 4] = __float2half_rn(acc[n][2 * x + 1] * (inv * un[n / 4]));
                    }
                    if (WT && t == 0)
                        p.lse[r] = l[x] > 0.f ? mx + log2f(l[x]) : -INFINITY;
                } else {
                    float *o = p.ws_o + (slot * p.sh + c) * D + t;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[8 * n] = acc[n][2 * x] * un[n / 4];
                        o[8 * n + 4] = acc[n][2 * x + 1] * un[n / 4];
                    }
                    if (t == 0)
                        p.ws_ml[slot * p.sh + c] = make_float2(mx, l[x]);
                }
            }
        }
        reset();
        if (i < n_my) {
            if (cw.k == cw.n) {
                --cw.k;
                cw.next(p);
            }
            __syncthreads();                       // every warp is done with the queries
            load_q();                              // read after the next barriers
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---------------------------------------------------------------- host side
// Groups of 8 columns beyond which a unit of 64 columns is taken.  16 x 4096 keys of 4 heads,
// us with units of 64 columns against units of 8: 56 columns 51.9 / 51.7 at D = 128 and 103 /
// 99 at 256, 64 columns 53.0 / 51.9 and 105 / 112: seven or eight groups cost what a unit does;
// 72 columns, two units, would lose.
constexpr int WIDE_GROUPS = 6;
// Tiles per warp (at full capacity, with units of 8 columns) from which a unit of 16
// columns is taken at D = 128: fewer, larger units cost parallelism first.  16 columns
// on 16 sequences x 4 heads: 512 keys (2 tiles) 17.3 us against 14.7, 4096 (18) 25.2 and
// 26.6, 32768 (144) 87 against 114.  Not with recorded weights, whose passes over the
// scores outweigh it (24 columns, 32768 keys: 324 us against 253).
constexpr double TWO_GROUP_MIN_TILES = 20.0;

// The plan of small steps: a cluster of up to 8 CTAs per unit while every cluster is
// resident at once and a warp has at most so many tiles (at full capacity).  us with
// clusters against the split and merge, 4 query heads per KV head:
//                          1 x 2 heads       1 x 8        4 x 8        8 x 8
//   D = 128,  512 keys     7.1 /  8.0     7.2 /  8.1   7.0 /  9.1   7.8 / 10.3
//            2048          7.8 / 10.5     7.8 / 11.1   9.2 / 11.9  11.9 / 13.1
//            8192         11.8 / 18.3    11.9 / 14.9  17.1 / 16.7  28.2 / 23.8
//   D = 256, 2048          9.9 / 12.4     9.9 / 13.6  12.8 / 13.7  17.8 / 16.9
//            8192         16.3 / 22.4    16.4 / 16.5  25.8 / 22.5  44.4 / 36.4
// Equal lengths; the split also balances ragged ones, so the limit is half of where
// it breaks even.
constexpr int CL_MAX_CTAS = 8;
constexpr int CL_MAX_TILES_128 = 16, CL_MAX_TILES_256 = 8;      // per warp

struct Plan {
    int cl_ctas;                 // the plan of small steps: CTAs per cluster; else 0
    int ctas, W, n_hg, units, sh, cpu;
    size_t bytes;                // partial slots and prefix
};

static bool two_groups_pay(int B, int Hkv, int D, int groups, long long cap, int sms)
{
    const double per_warp = (double)B * Hkv * groups * ((cap + TILE - 1) / TILE) /
                            ((double)sms * Cfg<128, 1>::CTAS_PER_SM * Cfg<128, 1>::NW);
    return D == 128 && groups > 1 && per_warp >= TWO_GROUP_MIN_TILES;
}

// cpu: the columns per unit; 0: what the rules above give.
static Plan make_plan(int B, int tq, int Hq, int Hkv, int D, long long cap, int sms,
                      bool weights, int cpu = 0)
{
    Plan pl = {};
    const int cols = tq * (Hq / Hkv);
    const int groups = (cols + GPH - 1) / GPH;
    pl.cpu = cpu                                                               ? cpu
             : groups > WIDE_GROUPS * ((cols + 63) / 64)                       ? 64
             : !weights && two_groups_pay(B, Hkv, D, groups, cap, sms)         ? 2 * GPH
                                                                               : GPH;
    pl.n_hg = (cols + pl.cpu - 1) / pl.cpu;
    pl.sh = cols < pl.cpu ? cols : pl.cpu;
    pl.units = Hkv * pl.n_hg;
    int nw, cps;                 // workers per CTA, CTAs per SM
    if (pl.cpu == 64) {
        nw = 1;
        cps = D == 128 ? WideCfg<128>::CTAS_PER_SM : WideCfg<256>::CTAS_PER_SM;
    } else if (pl.cpu == 16) {
        nw = Cfg<128, 2>::NW;
        cps = Cfg<128, 2>::CTAS_PER_SM;
    } else {
        nw = D == 128 ? Cfg<128, 1>::NW : Cfg<256, 1>::NW;
        cps = D == 128 ? Cfg<128, 1>::CTAS_PER_SM : Cfg<256, 1>::CTAS_PER_SM;
    }
    // one persistent wave, capped at a worker per position the capacity allows
    const double most = (double)B * pl.units * ((cap + TILE - 1) / TILE + tc::UNIT_COST);
    const long long wave = (long long)sms * cps;
    pl.ctas = static_cast<int>(most < (double)wave * nw ? ((long long)most + nw - 1) / nw : wave);
    if (pl.ctas == 0)
        pl.ctas = 1;
    pl.W = pl.ctas * nw;
    const long long units = (long long)B * pl.units, tiles = (cap + TILE - 1) / TILE;
    const int most_tiles = D == 128 ? CL_MAX_TILES_128 : CL_MAX_TILES_256;
    if (pl.cpu == GPH && !(weights && groups > 1))       // one addition per key and call
        for (int c = CL_MAX_CTAS; c >= 2 && !pl.cl_ctas; c /= 2)
            if (units * c <= sms && tiles <= (long long)most_tiles * c * nw)
                pl.cl_ctas = c;
    const size_t slots = (size_t)pl.W + (size_t)B * pl.units;
    pl.bytes = slots * pl.sh * (D * sizeof(float) + sizeof(float2)) +
               (size_t)(B + 1) * sizeof(long long);
    return pl;
}

// Bytes of partial slots and prefix that serve these sizes and any smaller batch, number of
// queries or capacity, whose units may be of another width with more slots: the largest over
// the widths that one of them may take (each width's bytes grow with every size).
static size_t plan_bytes(int B, int tq, int Hq, int Hkv, int D, long long cap, int sms)
{
    const int cols = tq * (Hq / Hkv), groups = (cols + GPH - 1) / GPH;
    size_t n = make_plan(B, tq, Hq, Hkv, D, cap, sms, false, GPH).bytes;
    if (two_groups_pay(B, Hkv, D, groups, cap, sms)) {
        const size_t m = make_plan(B, tq, Hq, Hkv, D, cap, sms, false, 2 * GPH).bytes;
        n = m > n ? m : n;
    }
    if (groups > WIDE_GROUPS) {
        const size_t m = make_plan(B, tq, Hq, Hkv, D, cap, sms, false, 64).bytes;
        n = m > n ? m : n;
    }
    return n;
}

static bool sizes_ok(int batch, int tq, int Hq, int Hkv, int D)
{
    return batch >= 0 && batch <= 65535 && tq >= 1 && tq <= 256 && Hq > 0 && Hkv > 0 &&
           Hkv <= 4096 && Hq % Hkv == 0 && Hq / Hkv <= 64 && (D == 128 || D == 256);
}

// Launches `kernel` after letting it use `smem` bytes of shared memory (once per
// device).
template <typename K>
static cudaError_t launch_split(K kernel, bool (&done)[64], const Params &p, int ctas, int threads,
                                int smem, cudaStream_t st, int cluster = 1)
{
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev >= 64 || !done[dev]) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess)
                return e;
            if (dev < 64)
                done[dev] = true;
        }
    }
    if (cluster == 1) {
        kernel<<<ctas, threads, smem, st>>>(p);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int D, bool WT>
static cudaError_t launch(const Params &p, int ctas, int sms, cudaStream_t st)
{
    static bool done[4][64] = {};
    cudaError_t e;
    if (p.cpu == 64) {
        e = launch_split(wide_kernel<D, WT>, done[0], p, ctas, 128, WideCfg<D>::SMEM, st);
    } else if (p.cl_ctas) {
        using C = Cfg<D, 1>;
        return launch_split(decode_kernel<D, 1, WT, true>, done[3], p, p.B * p.U_b * p.cl_ctas,
                            C::NW * 32, C::SMEM, st, p.cl_ctas);
    } else if (p.cpu == GPH) {
        using C = Cfg<D, 1>;
        e = launch_split(decode_kernel<D, 1, WT, false>, done[1], p, ctas, C::NW * 32, C::SMEM, st);
    } else {
        using C = Cfg<128, 2>;       // the plan gives 16 columns at D = 128, without weights
        e = launch_split(decode_kernel<128, 2, false, false>, done[2], p, ctas, C::NW * 32, C::SMEM,
                         st);
    }
    return e == cudaSuccess ? launch_merge_half<D>(p, sms, st) : e;
}

// Whether a call has anything to do: 0 (a no-op, whatever its pointers: empty arrays may have
// none), an error of its sizes, or NOT_EMPTY.
constexpr int NOT_EMPTY = 1;
static int check_empty(const char *name, int head_dim, int n_kv_heads, int batch, int n_tokens)
{
    if (head_dim != 128 && head_dim != 256)
        return fail(FA_ERR_HEAD_DIM, "%s: head_dim %d not supported (128 or 256)", name, head_dim);
    if (n_kv_heads <= 0 || n_kv_heads > 4096)
        return fail(FA_ERR_HEADS, "%s: n_kv_heads %d", name, n_kv_heads);
    if (batch < 0 || batch > 65535 || n_tokens < 0)
        return fail(FA_ERR_LAYOUT, "%s: bad batch %d or n_tokens %d", name, batch, n_tokens);
    return batch == 0 || n_tokens == 0 ? 0 : NOT_EMPTY;
}

// The checks of a cache's layout that append, gather and decode share.
static int check_cache(const char *name, int n_kv_heads, bool paged, int batch, int page_size,
                       int max_blocks, int num_blocks, long long *cap, size_t *kv_rows)
{
    if (max_blocks <= 0)
        return fail(FA_ERR_LAYOUT, "%s: bad max_blocks_per_seq %d", name, max_blocks);
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

static bool row_args(int T, int Hkv, int D, int page_size, const int *count, RowArgs *a)
{
    const long long half = (long long)T * Hkv * (D / 16);
    if (half > 0x7fffffffll - 255)          // row_grid rounds up to whole CTAs
        return false;
    a->T = T;
    a->n_half = static_cast<int>(half);
    a->lg_page = log2_of(page_size);
    a->lg_hkv = log2_of(Hkv);
    a->count = count;
    return true;
}

static dim3 row_grid(const RowArgs &a, int batch)
{
    return dim3((a.n_half + 255) / 256, batch, 2);
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
    long long cap;
    size_t kv_rows;
    int rc = i4::check_empty(name, head_dim, n_kv_heads, batch, n_tokens);
    if (rc != i4::NOT_EMPTY)
        return rc;
    if (!k_new || !v_new || !k_codes || !k_scales || !v_codes || !v_scales || !positions)
        return fail(FA_ERR_NULL, "%s: only block_table and n_new may be NULL", name);
    rc = i4::check_cache(name, n_kv_heads, block_table != nullptr, batch, page_size,
                         max_blocks_per_seq, num_blocks, &cap, &kv_rows);
    if (rc)
        return rc;
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
    i4::RowArgs a = {};
    if (!i4::row_args(n_tokens, n_kv_heads, head_dim, page_size, n_new, &a))
        return fail(FA_ERR_LAYOUT, "%s: too many rows per sequence", name);
    const Params p = i4::row_params(block_table, positions, batch, n_kv_heads, page_size,
                                    max_blocks_per_seq, num_blocks, cap);
    const auto kernel = head_dim == 128 ? i4::append_kernel<128> : i4::append_kernel<256>;
    kernel<<<i4::row_grid(a, batch), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        p, a, k_new, v_new, static_cast<unsigned *>(k_codes), static_cast<__half *>(k_scales),
        static_cast<unsigned *>(v_codes), static_cast<__half *>(v_scales));
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
    long long cap;
    size_t kv_rows;
    int rc = i4::check_empty(name, head_dim, n_kv_heads, batch, n_tokens);
    if (rc != i4::NOT_EMPTY)
        return rc;
    if (!k_codes || !k_scales || !v_codes || !v_scales || !positions || !k_out || !v_out)
        return fail(FA_ERR_NULL, "%s: only block_table and n_rows may be NULL", name);
    rc = i4::check_cache(name, n_kv_heads, block_table != nullptr, batch, page_size,
                         max_blocks_per_seq, num_blocks, &cap, &kv_rows);
    if (rc)
        return rc;
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
    i4::RowArgs a = {};
    if (!i4::row_args(n_tokens, n_kv_heads, head_dim, page_size, n_rows, &a))
        return fail(FA_ERR_LAYOUT, "%s: too many rows per sequence", name);
    const Params p = i4::row_params(block_table, positions, batch, n_kv_heads, page_size,
                                    max_blocks_per_seq, num_blocks, cap);
    const auto kernel = head_dim == 128 ? i4::gather_kernel<128> : i4::gather_kernel<256>;
    kernel<<<i4::row_grid(a, batch), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        p, a, static_cast<const unsigned *>(k_codes), static_cast<const __half *>(k_scales),
        static_cast<const unsigned *>(v_codes), static_cast<const __half *>(v_scales),
        static_cast<__half *>(k_out), static_cast<__half *>(v_out));
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
    const size_t bytes = i4::plan_bytes(batch, n_queries, n_q_heads, n_kv_heads, head_dim,
                                        max_kv_len, num_sms);
    if (!with_weights)
        return bytes;
    // (the scores of a plan with weights grow with every size)
    const i4::Plan pl = i4::make_plan(batch, n_queries, n_q_heads, n_kv_heads, head_dim,
                                      max_kv_len, num_sms, true);
    WeightSpace ws;
    return weight_space(bytes, batch, n_queries, n_q_heads, pl.units, pl.sh, max_kv_len, &ws)
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
    long long cap;
    size_t kv_rows;
    int rc = i4::check_empty(name, head_dim, n_kv_heads, batch, 1);
    if (rc != i4::NOT_EMPTY)
        return rc;
    if (!q || !k_codes || !k_scales || !v_codes || !v_scales || !seq_lens || !out)
        return fail(FA_ERR_NULL, "%s: only block_table, window and acc may be NULL", name);
    rc = i4::check_cache(name, n_kv_heads, block_table != nullptr, batch, page_size,
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
    if (kv_rows >= (1ull << 31))
        return fail(FA_ERR_LAYOUT, "%s: caches of 2^31 rows or more are not supported", name);
    const size_t q_bytes = (size_t)batch * n_queries * n_q_heads * head_dim * 2;
    const size_t cb = kv_rows * (head_dim / 2), sb = kv_rows * (head_dim / 16);
    const i4::Span outs[] = {{out, q_bytes}, {acc, kv_rows * sizeof(float)}};
    const i4::Span ins[] = {{q, q_bytes}, {k_codes, cb}, {k_scales, sb}, {v_codes, cb},
                            {v_scales, sb}, {seq_lens, (size_t)batch * 4},
                            {window, (size_t)batch * 4},
                            {block_table, (size_t)batch * max_blocks_per_seq * 4}};
    if ((rc = i4::check_rows(name, outs, 2, ins, 8)))
        return rc;
    int sms = 0;
    if ((rc = device_sms(&sms)))
        return rc;
    const i4::Plan pl = i4::make_plan(batch, n_queries, n_q_heads, n_kv_heads, head_dim, cap, sms,
                                      acc != nullptr);
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
    p.cpu = pl.cpu;
    p.cl_ctas = pl.cl_ctas;
    if (acc) {
        p.acc = acc;
        p.lse = reinterpret_cast<float *>(static_cast<char *>(workspace) + wsp.lse);
        p.ws_s = reinterpret_cast<float *>(static_cast<char *>(workspace) + wsp.scores);
        p.cap16 = (cap + 15) / 16 * 16;
        p.lg_page = block_table ? log2_of(page_size) : -1;
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
