// fa_rope.cu -- the pass between a projection and attention: each head's RMS
// norm, its rotation to the token's position, and the rows' way into the
// cache.
//
//     y = x * rsqrt(mean(x^2) + eps) * w                  (with a weight)
//     (a, b) -> (a cos - b sin, a sin + b cos) * magnitude, angle = pos * rate_j
//
// for the pairs j < rot_dim / 2 of a head: elements (j, j + rot_dim / 2), or
// (2 j, 2 j + 1) interleaved; elements from rot_dim on pass through.
//
// Angles.  A rate is held as a 64-bit fraction of a turn, f = rate / 2 pi *
// 2^64, so pos * f mod 2^64 is the angle's fraction of a turn at any 32-bit
// position: two integer multiplications, which add no error, and no 64-bit floating
// point, whose rate on this GPU is 1/60 of the 32-bit one.  The rates themselves come
// from 64-bit floats on the host, off by under 2^-54 turns each, so an angle by
// pos * 2^-54 (2^-34 turns at position 2^20, 2^-23 at 2^31).  Its top 32 bits go to
// sincospif.
//
// What bounds it: HBM, then latency.  A row of D elements is held by D / 16 threads,
// 16 elements each in two chunks of 8 that hold whole pairs, so that a rotation
// needs no exchange; the norm takes log2(D / 16) shuffles.  A thread's 8 pairs are
// the same ones in every head, so its sines and cosines are computed once for all
// the rows of a token that it takes.  Measured: 5 prompts of 1K-5K tokens, 64 + 16
// heads x 128 in bf16, 617 MB, 123 us (5.0 TB/s); 8 x 2048 tokens of 16 heads x 256 in
// bf16, 268 MB, 55.6 us (4.8 TB/s); 64 single tokens 5 and 7 us on the GPU.
#include <cuda_bf16.h>

#include "fa_common.cuh"

namespace fa {
namespace rope {

constexpr int THREADS = 256;
// Rows of a thread in flight together in the append kernel, which is held to 80 registers
// (three CTAs per SM): 123 us for the 5 prompts above; one row 149, two rows at the 106
// registers they would take 150.  The rotation alone keeps one row at 64 registers, four
// CTAs: 55.6 us against 59.4-63.7 with two rows at two and three CTAs.  Both limits spill: the
// rotation with norm 14 bytes (bf16) and 24 (fp32), the append with norm from fp32 104, with
// int8 V 8-116 in all kinds but fp16 with norm at D = 256.
constexpr int ROWS = 2;

struct Turn {                       // the rotation, the same for every row of a call
    const unsigned long long *freqs;    // [rot_dim / 2] turns per position, 2^64 = one turn
    int rot;
    int inter;
    float magnitude;
    float eps;
};

// 8 consecutive elements as they lie in memory, and as floats.
template <typename T>
struct Raw {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *src)
    {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
            v[i] = reinterpret_cast<const uint4 *>(src)[i];
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
            v[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
#pragma unroll
        for (int k = 0; k < static_cast<int>(sizeof(T) / 2); ++k) {
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 4) {
                    x[4 * k + i] = __uint_as_float(w[i]);
                } else {
                    float2 f;
                    if constexpr (std::is_same<T, __half>::value)
                        f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                    else
                        f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
                    x[2 * i] = f.x;
                    x[2 * i + 1] = f.y;
                }
            }
        }
    }
};

template <typename T>
__device__ __forceinline__ void store8(T *dst, const float (&x)[8])
{
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4 *>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<T, __half>::value) {
                w[i] = tc::pack_half2(x[2 * i], x[2 * i + 1]);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// What thread c of a row's D / 16 holds: elements a .. a + 7 and b .. b + 7, both 16 bytes
// (of a 16-bit type) from its neighbours', so that a warp reads and writes whole lines.
template <int D>
struct Chunks {
    int a, b;
    bool turned, turned_b;          // (of two halves: one is the other's partner)
    __device__ __forceinline__ Chunks(const Turn &t, int c)
    {
        const int pairs = t.rot / 16;
        if (t.inter) {                  // pairs lie within 8 elements
            a = 8 * c;
            b = a + D / 2;
            turned = a < t.rot;
            turned_b = b < t.rot;
        } else {
            turned = turned_b = c < pairs;
            a = turned ? 8 * c : t.rot + 8 * (c - pairs);
            b = a + (turned ? t.rot : D - t.rot) / 2;
        }
    }
};

// Sines and cosines of the thread's pairs at position pos: 8 c .. 8 c + 7 of two halves, or
// interleaved a / 2 .. a / 2 + 3 and b / 2 .. b / 2 + 3.
struct Angles {
    float cs[8], sn[8];
    template <int D>
    __device__ __forceinline__ void set(const Turn &t, const Chunks<D> &at, int pos)
    {
        if (!at.turned)
            return;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= 4 && !at.turned_b)
                return;
            const int j = !t.inter ? at.a + i : i < 4 ? at.a / 2 + i : at.b / 2 + i - 4;
            const unsigned long long f = __ldg(t.freqs + j);
            const unsigned long long turn = (unsigned long long)(long long)pos * f;
            // a signed fraction of a half turn, in [-1, 1)
            const float x = static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f;
            sincospif(x, &sn[i], &cs[i]);
            sn[i] *= t.magnitude;
            cs[i] *= t.magnitude;
        }
    }
};

// One row's chunks x, y normed and turned, in place.  w, v: the weight's chunks; a row
// with `plain` set has none and is only turned.  Every lane of the row's D / 16 takes part.
template <int D, bool NORM, typename In>
__device__ __forceinline__ void norm_turn(const Turn &t, const Chunks<D> &at, const Angles &g,
                                          float (&x)[8], float (&y)[8], const Raw<In> &w, const Raw<In> &v,
                                          bool plain, bool still = false)
{
    if constexpr (NORM) {
        uint64_t q[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const uint64_t a = pair2(x[i], x[i + 1]), b = pair2(y[i], y[i + 1]);
            q[0] = fma2(a, a, q[0]);
            q[1] = fma2(b, b, q[1]);
        }
        float s, s1;
        split2(add2(q[0], q[1]), s, s1);
        s += s1;
#pragma unroll
        for (int m = D / 32; m >= 1; m >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, m);
        if (!plain) {
            const float r = rsqrtf(s * (1.f / D) + t.eps);
            float a[8], b[8];
            w.get(a);
            v.get(b);
            const uint64_t r2 = pair2(r, r);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                split2(mul2(pair2(x[i], x[i + 1]), mul2(r2, pair2(a[i], a[i + 1]))), x[i], x[i + 1]);
                split2(mul2(pair2(y[i], y[i + 1]), mul2(r2, pair2(b[i], b[i + 1]))), y[i], y[i + 1]);
            }
        }
    }
    if (!at.turned || still)
        return;
    if (t.inter) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * g.cs[i] - b * g.sn[i];
            x[2 * i + 1] = a * g.sn[i] + b * g.cs[i];
        }
        if (at.turned_b) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = y[2 * i], b = y[2 * i + 1];
                y[2 * i] = a * g.cs[i + 4] - b * g.sn[i + 4];
                y[2 * i + 1] = a * g.sn[i + 4] + b * g.cs[i + 4];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const uint64_t a = pair2(x[i], x[i + 1]), b = pair2(y[i], y[i + 1]);
            const uint64_t c = pair2(g.cs[i], g.cs[i + 1]), d = pair2(g.sn[i], g.sn[i + 1]);
            split2(sub2(mul2(a, c), mul2(b, d)), x[i], x[i + 1]);
            split2(fma2(a, d, mul2(b, c)), y[i], y[i + 1]);
        }
    }
}

// ------------------------------------------------------------ one array of heads
struct RopeArgs {
    Turn turn;
    const void *x, *w;
    void *out;
    const int *positions;
    long long tokens, x_stride, out_stride;
    int heads, per;                 // heads of a token, and how many of them a group takes
};

// A group of D / 16 threads takes `per` consecutive heads of one token.
template <int D, typename In, typename Out, bool NORM>
__global__ void __launch_bounds__(THREADS, 4) rope_kernel(const RopeArgs p)
{
    constexpr int L = D / 16;
    const int c = threadIdx.x % L;
    const long long group = (long long)blockIdx.x * (THREADS / L) + threadIdx.x / L;
    const int parts = (p.heads + p.per - 1) / p.per;
    const long long n = group / parts;
    const bool live = n < p.tokens;
    const int h0 = static_cast<int>(group % parts) * p.per;
    const int h1 = live ? min(h0 + p.per, p.heads) : h0;
    const Chunks<D> at(p.turn, c);
    Angles g;
    if (live)
        g.set(p.turn, at, p.turn.rot ? p.positions[n] : 0);
    Raw<In> w, v;
    if constexpr (NORM) {
        w.load(static_cast<const In *>(p.w) + at.a);
        v.load(static_cast<const In *>(p.w) + at.b);
    }
    const In *src = static_cast<const In *>(p.x) + n * p.x_stride;
    Out *dst = static_cast<Out *>(p.out) + n * p.out_stride;
    for (int h = h0; h < h0 + p.per; ++h) {     // the same count in every lane: the norm's shuffles
        Raw<In> a, b;
        a.zero();
        b.zero();
        if (h < h1) {
            a.load(src + h * D + at.a);
            b.load(src + h * D + at.b);
        }
        float x[8], y[8];
        a.get(x);
        b.get(y);
        norm_turn<D, NORM, In>(p.turn, at, g, x, y, w, v, false);
        if (h < h1) {
            store8(dst + h * D + at.a, x);
            store8(dst + h * D + at.b, y);
        }
    }
}

// ------------------------------------------------------------ q, k, v into the cache
struct AppendArgs {
    Turn turn;
    Params cache;                   // paging only: bt, Hkv, page_size, max_blocks, num_blocks, cap, B
    const void *q, *k, *v, *qw, *kw;
    __half *q_out, *k_cache;
    void *v_cache;
    __half *v_scales;
    const int *starts, *positions, *rope_pos;
    long long q_stride, k_stride, v_stride;
    int tokens, hq, per;
};

// Sequence of token n: the last b with starts[b] <= n, -1 for a row of no sequence.
__device__ __forceinline__ int sequence_of(const int *starts, int B, int n)
{
    if (!starts)
        return n < B ? n : -1;
    int lo = 0, hi = B;             // starts[lo] <= n < starts[hi]
    if (n < __ldg(starts) || n >= __ldg(starts + B))
        return -1;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (__ldg(starts + m) <= n)
            lo = m;
        else
            hi = m;
    }
    return lo;
}

// 32 consecutive elements, 8 in each of four neighbouring lanes, as int8 codes and
// one fp16 scale: s = fp16(max|x| / 127) of the exact quotient, code = the exact
// quotient x / s rounded half to even.  The 32-bit quotient of an element lies on
// the wrong side of a tie only when it equals the tie k + 1/2 itself; then the sign
// of x - (k + 1/2) s, exact in one fma (a product of 9 by 11 bits), decides.
__device__ __forceinline__ uint2 quantize8(const float (&x)[8], __half &scale)
{
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        top = fmaxf(top, fabsf(x[i]));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    scale = __double2half(static_cast<double>(top) / 127.0);
    const float s = __half2float(scale);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float r = 0.f;
        if (s != 0.f) {
            const float t = __fdiv_rn(x[i], s);
            r = rintf(t);
            const float tie = floorf(t) + 0.5f;
            if (t == tie) {
                const float e = fmaf(-tie, s, x[i]);
                r = e > 0.f ? tie + 0.5f : e < 0.f ? tie - 0.5f : r;
            }
            r = fminf(fmaxf(r, -127.f), 127.f);
        }
        w[i / 4] |= (static_cast<uint32_t>(static_cast<int>(r)) & 0xffu) << (8 * (i % 4));
    }
    return make_uint2(w[0], w[1]);
}

// A group of D / 16 threads takes `per` consecutive rows of one token, whose rows
// are its query heads, then its key heads, then its value heads.
template <int D, typename In, bool NORM, bool VI8>
__global__ void __launch_bounds__(THREADS, 3) rope_append_kernel(const AppendArgs p)
{
    constexpr int L = D / 16;
    const int c = threadIdx.x % L;
    const int hkv = p.cache.Hkv, keys = p.hq + hkv, rows = keys + hkv;
    const long long group = (long long)blockIdx.x * (THREADS / L) + threadIdx.x / L;
    const int parts = (rows + p.per - 1) / p.per;
    const long long n = group / parts;
    const int r0 = static_cast<int>(group % parts) * p.per;
    const int b = n < p.tokens ? sequence_of(p.starts, p.cache.B, static_cast<int>(n)) : -1;
    const int r1 = b >= 0 ? min(r0 + p.per, rows) : r0;
    const Chunks<D> at(p.turn, c);
    Angles g;
    long long cache_row = -1;       // of KV head 0; heads are `step` rows apart
    int step = 0;
    if (b >= 0) {
        const int i = static_cast<int>(n) - (p.starts ? __ldg(p.starts + b) : b);
        const int first_at = p.positions[b];
        const long long t = (long long)first_at + i;
        if (r0 < keys && p.turn.rot)
            g.set(p.turn, at, p.rope_pos ? p.rope_pos[b] + i : static_cast<int>(t));
        if (r1 > p.hq) {
            const bool first = c == 0 && r0 <= p.hq;    // one report per token
            if (t >= p.cache.cap || first_at < 0) {
                if (first)
                    flag(FA_STATUS_POS_RANGE);
            } else {
                cache_row = row_offset(p.cache, b, 0, static_cast<int>(t), 1);
                if (cache_row < 0 && first)
                    flag(FA_STATUS_BAD_BLOCK);
                step = p.cache.bt ? p.cache.page_size : static_cast<int>(p.cache.cap);
            }
        }
    }
    const In *const q = static_cast<const In *>(p.q) + n * p.q_stride;
    const In *const k = static_cast<const In *>(p.k) + n * p.k_stride - (long long)p.hq * D;
    const In *const v = static_cast<const In *>(p.v) + n * p.v_stride - (long long)keys * D;
    for (int i = 0; i < p.per; i += ROWS) {     // the same count in every lane: the shuffles
        Raw<In> ra[ROWS], rb[ROWS];
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            const int r = r0 + i + u;
            ra[u].zero();
            rb[u].zero();
            if (r < r1) {
                const In *src = (r < p.hq ? q : r < keys ? k : v) + r * D;
                ra[u].load(src + (r < keys ? at.a : 8 * c));
                rb[u].load(src + (r < keys ? at.b : 8 * c + D / 2));
            }
        }
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            const int r = r0 + i + u;
            const bool is_q = r < p.hq, is_v = r >= keys, live = r < r1;
            float x[8], y[8];
            ra[u].get(x);
            rb[u].get(y);
            Raw<In> w, z;
            bool plain = true;
            if constexpr (NORM) {
                const void *weight = is_q ? p.qw : is_v ? nullptr : p.kw;
                plain = !weight;
                w.zero();
                z.zero();
                if (weight && live) {
                    w.load(static_cast<const In *>(weight) + at.a);
                    z.load(static_cast<const In *>(weight) + at.b);
                }
            }
            norm_turn<D, NORM, In>(p.turn, at, g, x, y, w, z, plain, is_v);
            const long long row = cache_row + (long long)(r - (is_v ? keys : p.hq)) * step;
            if constexpr (VI8) {
                if (__any_sync(0xffffffffu, live && is_v)) {
                    __half s0, s1;
                    const uint2 c0 = quantize8(x, s0), c1 = quantize8(y, s1);
                    if (live && is_v && cache_row >= 0) {
                        int8_t *dst = static_cast<int8_t *>(p.v_cache) + row * D + 8 * c;
                        *reinterpret_cast<uint2 *>(dst) = c0;
                        *reinterpret_cast<uint2 *>(dst + D / 2) = c1;
                        if (c % 4 == 0) {
                            p.v_scales[row * (D / 32) + c / 4] = s0;
                            p.v_scales[row * (D / 32) + D / 64 + c / 4] = s1;
                        }
                    }
                }
            }
            if (live && (is_q || (cache_row >= 0 && !(VI8 && is_v)))) {
                __half *dst = is_q ? p.q_out + (n * p.hq + r) * D
                                   : (is_v ? static_cast<__half *>(p.v_cache) : p.k_cache) + row * D;
                store8(dst + (is_v ? 8 * c : at.a), x);
                store8(dst + (is_v ? 8 * c + D / 2 : at.b), y);
            }
        }
    }
}

// Rows per group: as many as leave every SM four CTAs' worth of groups, 8 at most
// (the angles of a token are then computed once for 8 heads).
static int rows_per_group(long long tokens, int rows, int groups_per_cta, int sms)
{
    int per = 1;
    while (per < 8 && tokens * ((rows + 2 * per - 1) / (2 * per)) >= 4ll * sms * groups_per_cta)
        per *= 2;
    return per;
}

static int size_of(int dtype)
{
    return dtype == FA_DTYPE_F32 ? 4 : 2;
}

static bool dtype_ok(int dtype)
{
    return dtype == FA_DTYPE_F32 || dtype == FA_DTYPE_F16 || dtype == FA_DTYPE_BF16;
}

// Bytes that n rows of `row` elements at a stride span.
static size_t span(long long n, long long stride, long long row, int size)
{
    return n <= 0 ? 0 : static_cast<size_t>((n - 1) * stride + row) * size;
}

template <int D, typename In, typename Out>
static cudaError_t launch_rope(const RopeArgs &p, unsigned ctas, cudaStream_t st)
{
    if (p.w)
        rope_kernel<D, In, Out, true><<<ctas, THREADS, 0, st>>>(p);
    else
        rope_kernel<D, In, Out, false><<<ctas, THREADS, 0, st>>>(p);
    return cudaGetLastError();
}

template <int D, typename In>
static cudaError_t launch_rope(const RopeArgs &p, int out_dtype, unsigned ctas, cudaStream_t st)
{
    switch (out_dtype) {
    case FA_DTYPE_F32: return launch_rope<D, In, float>(p, ctas, st);
    case FA_DTYPE_F16: return launch_rope<D, In, __half>(p, ctas, st);
    default: return launch_rope<D, In, __nv_bfloat16>(p, ctas, st);
    }
}

template <int D>
static cudaError_t launch_rope(const RopeArgs &p, int dtype, int out_dtype, unsigned ctas,
                               cudaStream_t st)
{
    switch (dtype) {
    case FA_DTYPE_F32: return launch_rope<D, float>(p, out_dtype, ctas, st);
    case FA_DTYPE_F16: return launch_rope<D, __half>(p, out_dtype, ctas, st);
    default: return launch_rope<D, __nv_bfloat16>(p, out_dtype, ctas, st);
    }
}

template <int D, typename In>
static cudaError_t launch_append(const AppendArgs &p, unsigned ctas, cudaStream_t st)
{
    const bool norm = p.qw || p.kw;
    if (norm && p.v_scales)
        rope_append_kernel<D, In, true, true><<<ctas, THREADS, 0, st>>>(p);
    else if (norm)
        rope_append_kernel<D, In, true, false><<<ctas, THREADS, 0, st>>>(p);
    else if (p.v_scales)
        rope_append_kernel<D, In, false, true><<<ctas, THREADS, 0, st>>>(p);
    else
        rope_append_kernel<D, In, false, false><<<ctas, THREADS, 0, st>>>(p);
    return cudaGetLastError();
}

template <int D>
static cudaError_t launch_append(const AppendArgs &p, int dtype, unsigned ctas, cudaStream_t st)
{
    switch (dtype) {
    case FA_DTYPE_F32: return launch_append<D, float>(p, ctas, st);
    case FA_DTYPE_F16: return launch_append<D, __half>(p, ctas, st);
    default: return launch_append<D, __nv_bfloat16>(p, ctas, st);
    }
}

// The checks that both calls share; 0 or an error already reported.
static int check_turn(const char *name, int head_dim, int dtype, int rot_dim, const void *freqs,
                      float magnitude, float eps)
{
    if (head_dim != 128 && head_dim != 256)
        return fail(FA_ERR_HEAD_DIM, "%s: head_dim %d not supported (128 or 256)", name, head_dim);
    if (!dtype_ok(dtype))
        return fail(FA_ERR_LAYOUT, "%s: unknown dtype %d", name, dtype);
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16)
        return fail(FA_ERR_LAYOUT, "%s: rot_dim %d must be a multiple of 16 in [0, head_dim]", name,
                    rot_dim);
    if (!isfinite(magnitude) || !isfinite(eps) || eps < 0.f)
        return fail(FA_ERR_SCALE, "%s: magnitude must be finite and eps finite and not negative",
                    name);
    if (rot_dim && !freqs)
        return fail(FA_ERR_NULL, "%s: freqs is required when rot_dim > 0", name);
    if (!aligned_to(freqs, 8))
        return fail(FA_ERR_ALIGN, "%s: freqs must be 8-byte aligned", name);
    return 0;
}

}  // namespace rope

cudaError_t rope_take_status(unsigned int *v, cudaStream_t st)
{
    return take_status(v, st);
}

}  // namespace fa

using namespace fa;
using namespace fa::rope;

extern "C" {

FA_API int fa_rope_freqs(int rot_dim, double base, int scaling, double factor, double original_len,
                         uint64_t *freqs, float *magnitude)
{
    g_err[0] = 0;
    if (!freqs || !magnitude)
        return fail(FA_ERR_NULL, "fa_rope_freqs: freqs and magnitude are required");
    if (rot_dim < 2 || rot_dim % 2 || rot_dim > 65536)
        return fail(FA_ERR_LAYOUT, "fa_rope_freqs: rot_dim %d must be even, in [2, 65536]", rot_dim);
    if (!(base > 1.0) || !isfinite(base) || !(factor >= 1.0) || !isfinite(factor))
        return fail(FA_ERR_SCALE, "fa_rope_freqs: base must be above 1 and factor at least 1");
    if (scaling < FA_ROPE_NONE || scaling > FA_ROPE_YARN)
        return fail(FA_ERR_LAYOUT, "fa_rope_freqs: unknown scaling %d", scaling);
    if (scaling == FA_ROPE_YARN && (!(original_len >= 1.0) || !isfinite(original_len)))
        return fail(FA_ERR_SCALE, "fa_rope_freqs: original_len must be at least 1");
    const double two_pi = 6.283185307179586476925;
    if (scaling == FA_ROPE_NTK && rot_dim > 2)
        base *= pow(factor, (double)rot_dim / (rot_dim - 2));
    // YaRN's ramp between the pair that turns 32 times in original_len positions
    // and the one that turns once
    auto pair_of = [&](double turns) {
        return rot_dim * log(original_len / (turns * two_pi)) / (2.0 * log(base));
    };
    double lo = 0.0, hi = 0.0;
    if (scaling == FA_ROPE_YARN) {
        lo = fmax(floor(pair_of(32.0)), 0.0);
        hi = fmin(ceil(pair_of(1.0)), rot_dim - 1.0);
    }
    for (int j = 0; j < rot_dim / 2; ++j) {
        double r = pow(base, -2.0 * j / rot_dim);
        if (scaling == FA_ROPE_LINEAR)
            r /= factor;
        if (scaling == FA_ROPE_YARN) {
            const double slow = fmin(fmax((j - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
            r = r * (1.0 - slow) + r / factor * slow;
        }
        freqs[j] = static_cast<uint64_t>(r / two_pi * 18446744073709551616.0);   // r <= 1 rad
    }
    *magnitude = scaling == FA_ROPE_YARN ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.f;
    return 0;
}

FA_API int fa_rope(const void *x, int dtype, void *out, int out_dtype, const void *weight,
                   float eps, const int32_t *positions, const uint64_t *freqs, int rot_dim,
                   int interleaved, float magnitude, long long n_tokens, int n_heads, int head_dim,
                   long long x_stride, long long out_stride, void *stream)
{
    g_err[0] = 0;
    const int rc = check_turn("fa_rope", head_dim, dtype, rot_dim, freqs, magnitude, eps);
    if (rc)
        return rc;
    if (!dtype_ok(out_dtype))
        return fail(FA_ERR_LAYOUT, "fa_rope: unknown out_dtype %d", out_dtype);
    if (n_heads <= 0 || n_heads > 65536)
        return fail(FA_ERR_HEADS, "fa_rope: n_heads %d", n_heads);
    const long long row = (long long)n_heads * head_dim;
    const int sx = size_of(dtype), so = size_of(out_dtype);
    if (n_tokens < 0 || n_tokens > 0x7fffffffll || x_stride < row || out_stride < row ||
        x_stride > (1ll << 40) || out_stride > (1ll << 40))
        return fail(FA_ERR_LAYOUT, "fa_rope: bad n_tokens %lld or strides %lld, %lld (at least "
                                   "n_heads * head_dim)", n_tokens, x_stride, out_stride);
    if (n_tokens == 0)
        return 0;
    if (!x || !out || (rot_dim && !positions))
        return fail(FA_ERR_NULL, "fa_rope: x, out and positions are required");
    if (!aligned16(x) || !aligned16(out) || !aligned16(weight) || !aligned_to(positions, 4) ||
        x_stride * sx % 16 || out_stride * so % 16)
        return fail(FA_ERR_ALIGN, "fa_rope: x, out, weight and their rows must be 16-byte and "
                                  "positions 4-byte aligned");
    const size_t nx = span(n_tokens, x_stride, row, sx), no = span(n_tokens, out_stride, row, so);
    const bool in_place = x == out && x_stride == out_stride && dtype == out_dtype;
    if ((!in_place && overlaps(out, no, x, nx)) ||
        overlaps(out, no, weight, (size_t)head_dim * sx) ||
        overlaps(out, no, positions, (size_t)n_tokens * 4) ||
        overlaps(out, no, freqs, (size_t)rot_dim / 2 * 8))
        return fail(FA_ERR_ALIAS, "fa_rope: out overlaps an input (it may only be x itself)");
    int sms = 0;
    if (const int e = device_sms(&sms))
        return e;
    RopeArgs p = {};
    p.turn = {reinterpret_cast<const unsigned long long *>(freqs), rot_dim, interleaved != 0,
              magnitude, eps};
    p.x = x;
    p.w = weight;
    p.out = out;
    p.positions = positions;
    p.tokens = n_tokens;
    p.x_stride = x_stride;
    p.out_stride = out_stride;
    p.heads = n_heads;
    const int groups = THREADS / (head_dim / 16);
    p.per = rows_per_group(n_tokens, n_heads, groups, sms);
    const long long all = n_tokens * ((n_heads + p.per - 1) / p.per);
    const long long ctas = (all + groups - 1) / groups;
    if (ctas > 0x7fffffffll)
        return fail(FA_ERR_LAYOUT, "fa_rope: too many rows");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = head_dim == 128
                              ? launch_rope<128>(p, dtype, out_dtype, (unsigned)ctas, st)
                              : launch_rope<256>(p, dtype, out_dtype, (unsigned)ctas, st);
    if (e != cudaSuccess)
        return fail(FA_ERR_CUDA, "fa_rope: launch failed: %s", cudaGetErrorString(e));
    return 0;
}

FA_API int fa_rope_append_kv(const void *q, const void *k, const void *v, int dtype,
                             long long q_stride, long long k_stride, long long v_stride,
                             const void *q_weight, const void *k_weight, float eps,
                             const uint64_t *freqs, int rot_dim, int interleaved, float magnitude,
                             void *q_out, void *k_cache, void *v_cache, void *v_scales,
                             const int32_t *block_table, const int32_t *starts,
                             const int32_t *positions, const int32_t *rope_positions, int batch,
                             int n_tokens, int n_q_heads, int n_kv_heads, int head_dim,
                             int page_size, int max_blocks_per_seq, int num_blocks, void *stream)
{
    g_err[0] = 0;
    const char *name = "fa_rope_append_kv";
    const int rc = check_turn(name, head_dim, dtype, rot_dim, freqs, magnitude, eps);
    if (rc)
        return rc;
    if (n_q_heads < 0 || n_kv_heads <= 0 || n_q_heads > 65536 || n_kv_heads > 4096)
        return fail(FA_ERR_HEADS, "%s: bad heads (q %d, kv %d)", name, n_q_heads, n_kv_heads);
    const bool paged = block_table != nullptr;
    if (batch < 0 || n_tokens < 0 || max_blocks_per_seq <= 0 ||
        (paged && (page_size <= 0 || page_size % 16 || num_blocks <= 0)))
        return fail(FA_ERR_LAYOUT, "%s: bad batch, n_tokens, capacity, page size or block count",
                    name);
    if (!starts && n_tokens != batch)
        return fail(FA_ERR_LAYOUT, "%s: without starts every sequence has one token (n_tokens %d, "
                                   "batch %d)", name, n_tokens, batch);
    const long long cap = paged ? (long long)max_blocks_per_seq * page_size : max_blocks_per_seq;
    if (cap > (1ll << 30))
        return fail(FA_ERR_LAYOUT, "%s: capacity %lld tokens too large", name, cap);
    const int D = head_dim, sx = size_of(dtype);
    const long long qrow = (long long)n_q_heads * D, krow = (long long)n_kv_heads * D;
    if ((n_q_heads && (q_stride < qrow || q_stride > (1ll << 40))) || k_stride < krow ||
        v_stride < krow || k_stride > (1ll << 40) || v_stride > (1ll << 40))
        return fail(FA_ERR_LAYOUT, "%s: a token's stride is below heads * head_dim", name);
    if (n_tokens == 0 || batch == 0)
        return 0;
    if ((n_q_heads && (!q || !q_out)) || !k || !v || !k_cache || !v_cache || !positions)
        return fail(FA_ERR_NULL, "%s: q, k, v, q_out, caches and positions are required", name);
    if ((n_q_heads && (!aligned16(q) || !aligned16(q_out) || q_stride * sx % 16)) ||
        !aligned16(k) || !aligned16(v) || k_stride * sx % 16 || v_stride * sx % 16 ||
        !aligned16(q_weight) || !aligned16(k_weight) || !aligned16(k_cache) ||
        !aligned16(v_cache) || !aligned_to(v_scales, 2) || !aligned_to(block_table, 4) ||
        !aligned_to(starts, 4) || !aligned_to(positions, 4) || !aligned_to(rope_positions, 4))
        return fail(FA_ERR_ALIGN, "%s: q, k, v, their rows, the weights, q_out and the caches must "
                                  "be 16-byte aligned, scales 2-byte, int32 arrays 4-byte", name);
    const size_t rows = (paged ? (size_t)num_blocks * page_size : (size_t)batch * cap) * n_kv_heads;
    const struct { const void *p; size_t n; } outs[] = {
        {q_out, (size_t)n_tokens * qrow * 2}, {k_cache, rows * D * 2},
        {v_cache, rows * D * (v_scales ? 1 : 2)}, {v_scales, rows * (D / 32) * 2}};
    const struct { const void *p; size_t n; } ins[] = {
        {n_q_heads ? q : nullptr, span(n_tokens, q_stride, qrow, sx)},
        {k, span(n_tokens, k_stride, krow, sx)}, {v, span(n_tokens, v_stride, krow, sx)},
        {q_weight, (size_t)D * sx}, {k_weight, (size_t)D * sx}, {freqs, (size_t)rot_dim / 2 * 8},
        {block_table, (size_t)batch * max_blocks_per_seq * 4},
        {starts, ((size_t)batch + 1) * 4}, {positions, (size_t)batch * 4},
        {rope_positions, (size_t)batch * 4}};
    for (int i = 0; i < 4; ++i) {
        for (const auto &in : ins)
            if (overlaps(outs[i].p, outs[i].n, in.p, in.n))
                return fail(FA_ERR_ALIAS, "%s: q_out or a cache overlaps an input", name);
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return fail(FA_ERR_ALIAS, "%s: q_out and the caches overlap", name);
    }
    int sms = 0;
    if (const int e = device_sms(&sms))
        return e;
    AppendArgs p = {};
    p.turn = {reinterpret_cast<const unsigned long long *>(freqs), rot_dim, interleaved != 0,
              magnitude, eps};
    p.cache.bt = block_table;
    p.cache.B = batch;
    p.cache.Hkv = n_kv_heads;
    p.cache.page_size = paged ? page_size : 16;
    p.cache.max_blocks = max_blocks_per_seq;
    p.cache.num_blocks = num_blocks;
    p.cache.cap = cap;
    p.q = q;
    p.k = k;
    p.v = v;
    p.qw = q_weight;
    p.kw = k_weight;
    p.q_out = static_cast<__half *>(q_out);
    p.k_cache = static_cast<__half *>(k_cache);
    p.v_cache = v_cache;
    p.v_scales = static_cast<__half *>(v_scales);
    p.starts = starts;
    p.positions = positions;
    p.rope_pos = rope_positions;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.tokens = n_tokens;
    p.hq = n_q_heads;
    const int all_rows = n_q_heads + 2 * n_kv_heads, groups = THREADS / (D / 16);
    p.per = rows_per_group(n_tokens, all_rows, groups, sms);
    const long long all = (long long)n_tokens * ((all_rows + p.per - 1) / p.per);
    const long long ctas = (all + groups - 1) / groups;
    if (ctas > 0x7fffffffll)
        return fail(FA_ERR_LAYOUT, "%s: too many rows", name);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = D == 128 ? launch_append<128>(p, dtype, (unsigned)ctas, st)
                                   : launch_append<256>(p, dtype, (unsigned)ctas, st);
    if (e != cudaSuccess)
        return fail(FA_ERR_CUDA, "%s: launch failed: %s", name, cudaGetErrorString(e));
    return 0;
}

}  // extern "C"
