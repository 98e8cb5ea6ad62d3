// fa_prefill.cu -- attention of a chunk of new tokens per sequence over its
// cache: row (token i of sequence b, query head h) at position
// at = L_b - n_b + i sees the keys t <= at and, with a window W, of those the
// last W and the first n_sink.
#include "fa_common.cuh"

namespace fa {
namespace prefill {

struct Args {
    Params cache;            // paging: bt, Hkv, page_size, max_blocks, num_blocks, cap, B, seq_lens
    const __half *q;
    const __half *k, *v;
    const int *starts, *window;
    __half *out;
    int tokens, hq, group, sink;
    float c2;                // scale * log2(e)
};

// A warp per (token, query head) row, a key at a time.
template <int D>
__global__ void __launch_bounds__(256) rows_kernel(const Args p)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= (long long)p.tokens * p.hq)
        return;
    const int n = static_cast<int>(row / p.hq), h = static_cast<int>(row % p.hq);
    int b = 0;
    if (p.starts) {
        if (n < p.starts[0] || n >= p.starts[p.cache.B])
            return;
        while (p.starts[b + 1] <= n)
            ++b;
    } else {
        b = n;
    }
    const int first = p.starts ? p.starts[b] : b, count = p.starts ? p.starts[b + 1] - first : 1;
    long long len = p.cache.seq_lens[b];
    if (len < 0 || len > p.cache.cap) {
        flag(FA_STATUS_LEN_CLAMPED);
        len = len < 0 ? 0 : p.cache.cap;
    }
    const int at = static_cast<int>(len) - count + n - first;
    const int w = p.window ? p.window[b] : 0;
    float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
        q[e] = __half2float(p.q[row * D + lane + 32 * e]);
    for (int t = 0; t <= at; ++t) {
        if (w > 0 && t <= at - w && t >= p.sink) {
            t = at - w;
            continue;
        }
        const long long r = row_offset(p.cache, b, h / p.group, t, 1);
        if (r < 0) {
            flag(FA_STATUS_BAD_BLOCK);
            continue;
        }
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            s = fmaf(q[e], __half2float(p.k[r * D + lane + 32 * e]), s);
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= p.c2;
        const float top = fmaxf(m, s), ref = top == -INFINITY ? 0.f : top;
        const float a = ex2(m - ref), x = ex2(s - ref);
        m = top;
        l = l * a + x;
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = o[e] * a + x * __half2float(p.v[r * D + lane + 32 * e]);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
        p.out[row * D + lane + 32 * e] = __float2half_rn(o[e] * inv);
}

}  // namespace prefill

cudaError_t prefill_take_status(unsigned int *v, cudaStream_t st)
{
    return take_status(v, st);
}

}  // namespace fa

using namespace fa;
using namespace fa::prefill;

extern "C" {

FA_API size_t fa_prefill_workspace_size(int batch, int n_tokens, int n_q_heads, int n_kv_heads,
                                        int head_dim, int max_kv_len, int num_sms)
{
    if (batch <= 0 || n_tokens <= 0 || n_q_heads <= 0 || n_kv_heads <= 0 ||
        n_q_heads % n_kv_heads || n_q_heads / n_kv_heads > 64 ||
        (head_dim != 128 && head_dim != 256) || max_kv_len < 0)
        return 0;
    if (num_sms <= 0 && device_sms(&num_sms) != 0)
        return 0;
    return 16;
}

FA_API int fa_prefill(const void *q, const void *k_cache, const void *v_cache,
                      const void *v_scales, const int32_t *block_table, const int32_t *starts,
                      const int32_t *seq_lens, int n_q_heads, int n_kv_heads, int head_dim,
                      float scale, const int32_t *window, int n_sink, void *out, int batch,
                      int n_tokens, int page_size, int max_blocks_per_seq, int num_blocks,
                      void *workspace, size_t workspace_bytes, void *stream)
{
    g_err[0] = 0;
    const int D = head_dim;
    if (D != 128 && D != 256)
        return fail(FA_ERR_HEAD_DIM, "fa_prefill: head_dim %d not supported (128 or 256)", D);
    if (n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads % n_kv_heads ||
        n_q_heads / n_kv_heads > 64 || n_kv_heads > 4096)
        return fail(FA_ERR_HEADS, "fa_prefill: bad heads (q %d, kv %d)", n_q_heads, n_kv_heads);
    if (!isfinite(scale))
        return fail(FA_ERR_SCALE, "fa_prefill: scale is not finite");
    const bool paged = block_table != nullptr;
    if (batch < 0 || batch > 65535 || n_tokens < 0 || max_blocks_per_seq <= 0 ||
        (paged && (page_size <= 0 || page_size % 16 || num_blocks <= 0)))
        return fail(FA_ERR_LAYOUT, "fa_prefill: bad batch %d, n_tokens %d, capacity, page size or "
                                   "block count", batch, n_tokens);
    if (n_sink < 0 || n_sink > (1 << 30))
        return fail(FA_ERR_LAYOUT, "fa_prefill: n_sink %d must be in [0, 2^30]", n_sink);
    if (!starts && n_tokens != batch)
        return fail(FA_ERR_LAYOUT, "fa_prefill: without starts every sequence has one token "
                                   "(n_tokens %d, batch %d)", n_tokens, batch);
    if (v_scales)
        return fail(FA_ERR_LAYOUT, "fa_prefill: int8 V is not supported (fa_decode_multi takes up "
                                   "to 256 queries over it)");
    const long long cap = paged ? (long long)max_blocks_per_seq * page_size : max_blocks_per_seq;
    if (cap > (1ll << 30))
        return fail(FA_ERR_LAYOUT, "fa_prefill: capacity %lld tokens too large", cap);
    const size_t rows = (paged ? (size_t)num_blocks * page_size : (size_t)batch * cap) * n_kv_heads;
    if (rows >= (1ull << 31))
        return fail(FA_ERR_LAYOUT, "fa_prefill: caches of 2^31 rows or more are not supported");
    if (batch == 0 || n_tokens == 0)
        return 0;
    if (!q || !k_cache || !v_cache || !seq_lens || !out)
        return fail(FA_ERR_NULL, "fa_prefill: q, k_cache, v_cache, seq_lens and out are required");
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
        !aligned16(workspace) || !aligned_to(seq_lens, 4) || !aligned_to(block_table, 4) ||
        !aligned_to(window, 4) || !aligned_to(starts, 4))
        return fail(FA_ERR_ALIGN, "fa_prefill: q, caches, out and workspace must be 16-byte, int32 "
                                  "arrays 4-byte aligned");
    const size_t need = fa_prefill_workspace_size(batch, n_tokens, n_q_heads, n_kv_heads, D,
                                                  static_cast<int>(cap), 0);
    if (!need)
        return fail(FA_ERR_WORKSPACE, "fa_prefill: no workspace size for these sizes");
    if (!workspace || workspace_bytes < need)
        return fail(FA_ERR_WORKSPACE, "fa_prefill: workspace %zu bytes, need %zu", workspace_bytes,
                    need);
    const size_t qn = (size_t)n_tokens * n_q_heads * D * 2;
    const struct { const void *p; size_t n; } in[] = {
        {q, qn}, {k_cache, rows * D * 2}, {v_cache, rows * D * 2}, {seq_lens, (size_t)batch * 4},
        {starts, ((size_t)batch + 1) * 4}, {block_table, (size_t)batch * max_blocks_per_seq * 4},
        {window, (size_t)batch * 4}};
    for (const auto &x : in)
        if (overlaps(out, qn, x.p, x.n) || overlaps(workspace, need, x.p, x.n))
            return fail(FA_ERR_ALIAS, "fa_prefill: out or the workspace overlaps an input");
    if (overlaps(out, qn, workspace, need))
        return fail(FA_ERR_ALIAS, "fa_prefill: out overlaps the workspace");
    Args p = {};
    p.cache.bt = block_table;
    p.cache.seq_lens = seq_lens;
    p.cache.B = batch;
    p.cache.Hkv = n_kv_heads;
    p.cache.page_size = paged ? page_size : 16;
    p.cache.max_blocks = max_blocks_per_seq;
    p.cache.num_blocks = num_blocks;
    p.cache.cap = cap;
    p.q = static_cast<const __half *>(q);
    p.k = static_cast<const __half *>(k_cache);
    p.v = static_cast<const __half *>(v_cache);
    p.starts = starts;
    p.window = window;
    p.out = static_cast<__half *>(out);
    p.tokens = n_tokens;
    p.hq = n_q_heads;
    p.group = n_q_heads / n_kv_heads;
    p.sink = n_sink;
    p.c2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    const long long ctas = ((long long)n_tokens * n_q_heads + 7) / 8;
    if (ctas > 0x7fffffffll)
        return fail(FA_ERR_LAYOUT, "fa_prefill: too many rows");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (D == 128)
        rows_kernel<128><<<(unsigned)ctas, 256, 0, st>>>(p);
    else
        rows_kernel<256><<<(unsigned)ctas, 256, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(FA_ERR_CUDA, "fa_prefill: launch failed: %s", cudaGetErrorString(e));
    return 0;
}

}  // extern "C"
