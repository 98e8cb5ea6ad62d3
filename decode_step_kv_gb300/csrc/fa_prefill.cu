// fa_prefill.cu -- attention of a chunk of new tokens per sequence over its
// cache: row (token i of sequence b, query head h) at position
// at = L_b - n_b + i sees the keys t <= at and, with a window W, of those the
// last W and the first n_sink.
//
//     O = sum_t 2^(c2 q.k_t - m) v_t / sum_t 2^(c2 q.k_t - m),  c2 = scale log2(e)
//
// Rows.  The G query heads of a KV head share its keys, so a tile of 128 rows
// holds floor(128 / G) tokens with their G heads; a unit of work is one KV head
// of one row tile (two tiles of 128 rows at head_dim 128, one at 256) and walks
// the keys its rows see in tiles of 128.
//
// Matrix products.  S = Q K^T and O += P V are tcgen05 products of 128 x 128 x
// 16 steps: Q, K and V from shared memory (TMA, 128-byte swizzle), S and O in
// TMEM, P written over S in TMEM as fp16.  One softmax thread owns a row: its
// running maximum and sum never leave it.  O is rescaled only when a row's
// maximum has grown by more than 2^5, so the usual tile does not touch O.
//
// What bounds it: 128 keys cost a row tile 4 x 128 x 128 x D operations, at D = 128
// 1024 tensor cycles, so whole prompts are bound by the products and the softmax
// (64 exponentials per 64 keys and thread at four cycles a warp, and as much again
// around them), chunks of few rows by K and V.  Each stream has two S buffers, so
// that its products run ahead of its softmax.  At D = 128 these hold 64 keys: a
// 128 x 64 x 16 step takes 52-76 cycles where a 128 x 128 x 16 one takes 64, but TMEM
// has no room for two of 128 keys beside O, and one buffer a stream, whose Q K^T
// waits for its P V, took 1943 us for a prompt of 16384 tokens (32 / 8 heads) against
// 1657.  As it stands: 1526-1570 us (1.40-1.44 PFLOP/s of the 1.91 that a library
// product reaches; the power cap holds the clocks at 1.65-1.75 GHz), 512 tokens over
// 131072 keys 827-839 us, 4 prompts of 1K-8K at D = 256 913-930 us.
//
// Every CTA fetches its own K and V tiles.  At D = 256 its 128 rows take 128 KB per
// 2048 tensor cycles and the ring has room for 160 KB on their way: the loads' latency
// bounds it (tensor pipe 45% busy, L2 and DRAM 34%).  A load into two CTAs of a cluster
// halves what is fetched (4 prompts at D = 256 704 us, 512 tokens over 131072 keys 760),
// but it must stay off memory that another GPU serves, which a pointer does not tell,
// and the library is the same for every rank of a run on several GPUs.
//
// Work over the GPU.  A one-CTA kernel lists the units' tiles as positions of one
// axis (as the decode plan: UNIT_COST positions per unit beside its tiles), every
// CTA takes an equal stretch of it, and a unit that a stretch cuts leaves fp32
// partials that a merge kernel joins in a fixed order.
#include <cfloat>

#include "fa_common.cuh"

namespace fa {
namespace prefill {

constexpr int BM = 128;             // rows of a stream
constexpr int BN = 128;             // keys of a tile
constexpr int STAGES = 5;           // ring of K / V parts of 128 keys x 128 dims
constexpr int STAGE_BYTES = 32768;
constexpr int SLAB = 16384;         // 128 rows x 64 columns
// Positions charged for a unit's start (its Q, the pipeline's filling, its epilogue).  1, 2, 3,
// 4: the 16384-token prompt, 13 units per CTA, 1694, 1602, 1525, 1531 us; others within 2%
constexpr int UNIT_COST = 3;
constexpr int MIN_POS = 4;          // fewest positions a CTA is given
// Few and short units (at most this many positions on average, their start included) go to
// a CTA each, more of them where they take most CTAs anyway: a merge of split units costs
// what two or three tiles in a row do.  64 tokens over 512 keys, 2 units of 4 tiles: 17.1 us
// whole, 18.4 split; over 1024 keys 23.1 and 19.5; 16 single tokens over 1000 keys, 128
// units of 8 tiles: 20.6 and 23.8
constexpr int WHOLE = 8, WHOLE_BUSY = 11;
constexpr int BITS = 8;             // key tiles whose unmapped groups are remembered
// Weights are taken 2^UP above the reference's 1, so that the keys behind a dominant one
// (2^-10 to 2^-20 of it each: an attention sink's companions) keep their bits in fp16, and
// the reference follows a row's maximum when that has outgrown it by 2^GROW: P < 2^15.
constexpr float UP = 10.f, GROW = 5.f;
// A score in log2 units beyond FAR (its steps in 32 bits are 2^-7 there, and 2^4 at 2^27) is taken as a
// difference from the row's largest before it meets c2 and UP, which would be rounded to its steps.
constexpr float FAR = 65536.f;

// The most key tiles of a piece.  The tensor cores' 32-bit sums drop what an addition leaves below
// their last bit: a sum of one sign loses 4e-9 of itself (6e-9 at D = 256) with every key, 5e-3 over
// 2^20 keys.  So O is begun anew with every piece and added to what came before in fp32: a piece of
// 16384 keys loses 2^-13 at most.  512 tokens over 131072 keys, three cuts per CTA, 818 -> 830 us.
constexpr int SPAN = 128;

// VI8: int8 V.  Its tiles arrive raw and are turned into fp16 stages by a warpgroup of
// their own, in a ring of four whose odd (at D = 256 last two) stages only V uses, so
// that every stage has one producer.  Code times scale is rounded to fp16, as fa_decode
// rounds it: a factor per 32 dims cannot ride on the weight, which one product takes
// against all dims.  8192-token prompt, 32 / 8 heads x 128: 500 us against 406 with
// fp16 V; 4 x 4096 tokens, 16 / 8 heads x 256, 970 against 627 (the ring then holds one
// K tile).  These kernels spill: 164 bytes at D = 128, 168 at D = 256.
constexpr int RAW_BYTES = BN * 128;
template <int D, bool VI8 = false>
struct Cfg {
    static constexpr int NS = D == 128 ? 2 : 1;             // streams of 128 rows
    static constexpr int DS = D / 128;                      // ring stages per K or V tile
    static constexpr int SW = D == 128 ? 64 : 128;          // keys of an S buffer
    static constexpr int STG = VI8 ? 4 : STAGES;
    static constexpr int THREADS = 128 + 128 * NS + (VI8 ? 128 : 0);
    static constexpr int Q_BYTES = NS * BM * D * 2;
    static constexpr int RAW_OFF = Q_BYTES + STG * STAGE_BYTES;
    static constexpr int BAR_OFF = RAW_OFF + (VI8 ? 2 * RAW_BYTES : 0);
    static constexpr int SMEM = BAR_OFF + 512 + 1024;       // barriers, alignment slack
    static constexpr int ROWS = NS * BM;                    // of a partial slot
    static constexpr size_t SLOT_BYTES = (size_t)ROWS * D * sizeof(float);
    // registers of the warps around (VI8; 65536 in all) and of the rows' warps
    static constexpr int FEW = D == 128 ? 80 : 96, MANY = D == 128 ? 168 : 240;
    __host__ __device__ static constexpr bool v_stage(int i) { return VI8 && (D == 128 ? i % 2 == 1 : i >= 2); }
};

// A row tile of a sequence.
struct Ent {
    int b, tok;                     // sequence; first row of q
    int ntok, at;                   // tokens; position of the first
    int lo, hi;                     // keys [lo, hi) some row's window holds
    int n, ns, kt0;                 // key tiles; those before kt0 that hold sinks; first of [lo, hi)
    int window;
    int pad[2];
};

struct Args {
    Params cache;                   // paging: bt, Hkv, page_size, max_blocks, num_blocks, cap, B, seq_lens
    const int *starts, *window;
    const __half *v_scales;         // int8 V
    __half *out;
    int tokens, hq, group, tpt, sink;
    int lg_br;                      // log2 of the rows of a K / V box
    int oob_row;                    // a cache row beyond the tensor: reads as zeros
    float c2;
    uint32_t idesc_qk;
    int W;                          // CTAs of the main kernel
    int max_ents;
    // workspace
    Ent *ents;
    long long *pos;                 // [max_ents + 1] first position of each entry
    int *ebase;                     // [B + 1] first entry of each sequence
    int4 *split;                    // [W] the unit that a CTA leaves to its successors: entry, kv, parts
    float *part;                    // [2 W] slots of [D / 4][ROWS] float4
    float2 *ml;                     // [2 W][ROWS]
};

// ------------------------------------------------------------ the plan
// Row tiles of every sequence and the positions of their units, by one CTA.
constexpr int PLAN_THREADS = 1024;

__device__ __forceinline__ long long block_scan(long long x, long long *sh, long long &total)
{
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    long long s = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off)
            s += y;
    }
    if (lane == 31)
        sh[wid] = s;
    __syncthreads();
    if (wid == 0) {
        long long v = sh[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, v, off);
            if (lane >= off)
                v += y;
        }
        sh[lane] = v;
    }
    __syncthreads();
    const long long before = wid ? sh[wid - 1] : 0;
    total = sh[31];
    __syncthreads();
    return before + s - x;
}

__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const Args p, int per)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ long long sh[32];
    const int B = p.cache.B;
    auto rows_of = [&](int b, int &first) {         // a sequence's rows, within q whatever starts says
        first = p.starts ? min(max(p.starts[b], 0), p.tokens) : b;
        const int end = p.starts ? min(max(p.starts[b + 1], first), p.tokens) : b + 1;
        return end - first;
    };
    long long run = 0, total;
    for (int b0 = 0; b0 < B; b0 += PLAN_THREADS) {
        const int b = b0 + threadIdx.x;
        int first;
        const long long n = b < B ? (rows_of(b, first) + per - 1) / per : 0;
        const long long at = block_scan(n, sh, total);
        if (b < B)
            p.ebase[b] = static_cast<int>(min(run + at, (long long)p.max_ents));
        run += total;
    }
    const int E = static_cast<int>(min(run, (long long)p.max_ents));
    if (threadIdx.x == 0)
        p.ebase[B] = E;
    __syncthreads();
    run = 0;
    for (int e0 = 0; e0 < E; e0 += PLAN_THREADS) {
        const int e = e0 + threadIdx.x;
        long long span = 0;
        if (e < E) {
            int lo = 0, hi = B;                     // ebase[lo] <= e < ebase[hi]
            while (hi - lo > 1) {
                const int m = (lo + hi) >> 1;
                if (p.ebase[m] <= e)
                    lo = m;
                else
                    hi = m;
            }
            const int b = lo, rt = e - p.ebase[b];
            int first;
            const int nb = rows_of(b, first);
            long long len = p.cache.seq_lens[b];
            if (len < 0 || len > p.cache.cap) {
                flag(FA_STATUS_LEN_CLAMPED);
                len = len < 0 ? 0 : p.cache.cap;
            }
            Ent x = {};
            x.b = b;
            x.tok = first + rt * per;
            x.ntok = min(per, nb - rt * per);
            x.at = static_cast<int>(len) - nb + rt * per;
            x.window = p.window ? max(p.window[b], 0) : 0;
            x.hi = max(x.at + x.ntok, 0);
            const int at0 = max(x.at, 0);
            x.lo = x.window > 0 && at0 >= x.window ? at0 - x.window + 1 : 0;
            x.kt0 = x.lo / BN;
            x.ns = x.hi > 0 ? min((p.sink + BN - 1) / BN, x.kt0) : 0;
            x.n = x.hi > 0 ? x.ns + (x.hi - 1) / BN - x.kt0 + 1 : 0;
            p.ents[e] = x;
            span = (long long)p.cache.Hkv * (x.n + UNIT_COST);
        }
        const long long at = block_scan(span, sh, total);
        if (e < E)
            p.pos[e] = run + at;
        run += total;
    }
    if (threadIdx.x == 0)
        p.pos[E] = run;
}

// ------------------------------------------------------------ a CTA's stretch
__device__ __forceinline__ int ctas_for(const Args &p, long long T)
{
    const long long w = T / MIN_POS;
    return w < 1 ? 1 : static_cast<int>(w < p.W ? w : p.W);
}

struct Piece {
    Ent x;
    int e, kv, k0, k1;              // key tiles [k0, k1) of unit (e, kv)
    int slot;                       // partial slot, -1: the whole unit
    bool first_part;                // a partial from the unit's first tile
    bool begins, ends;              // the first, the last piece of the unit's tiles in this stretch
    long long last;                 // the unit's last tile, counted from the stretch's first position
    __device__ __forceinline__ int key_tile(int k) const { return k < x.ns ? k : x.kt0 + k - x.ns; }
};

// The pieces of a stretch of `len` positions, in order.
struct Pieces {
    int e, kv;
    int done;                       // tiles of the current unit before the next piece, 0: at its first
    long long us, len;              // us: the current unit's first tile, counted from the stretch's start
    __device__ __forceinline__ void start(const Args &p, int e_, long long t0, long long t1)
    {
        e = e_;
        done = 0;
        const int unit = p.ents[e].n + UNIT_COST;
        const long long off = t0 - p.pos[e];
        kv = static_cast<int>(off / unit);
        us = kv * (long long)unit + UNIT_COST - off;
        len = t1 - t0;
    }
    __device__ __forceinline__ bool next(const Args &p, Piece &q)
    {
        while (us - UNIT_COST < len) {      // the last unit ends where the last stretch does
            if (e != q.e)               // kept over its KV heads
                q.x = p.ents[e];
            const int n = q.x.n;
            const bool empty = n == 0 && us >= UNIT_COST;       // zero rows
            q.k0 = empty || us > 0 ? 0 : static_cast<int>(-us);
            q.k1 = empty ? 0 : len - us < n ? static_cast<int>(len - us) : n;
            q.e = e;
            q.kv = kv;
            const bool whole = q.k0 == 0 && q.k1 == n;
            q.slot = whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (q.k0 == 0);
            q.first_part = !whole && q.k0 == 0;
            q.last = us + n - 1;
            q.begins = done == 0;
            q.k0 = q.begins ? q.k0 : done;
            q.ends = q.k1 - q.k0 <= SPAN;
            if (!q.ends) {
                done = q.k1 = q.k0 + SPAN;
                return true;
            }
            done = 0;
            us += n + UNIT_COST;
            if (++kv == p.cache.Hkv) {
                kv = 0;
                ++e;
            }
            if (empty || q.k1 > q.k0)
                return true;
        }
        return false;
    }
};

// ------------------------------------------------------------ tcgen05 wrappers
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                            uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Arrives on bar when the products issued so far by this thread are done.
__device__ __forceinline__ void mma_commit(uint32_t lead, uint32_t bar)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
                 "r"(lead)
                 : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// A matrix in shared memory under the 128-byte swizzle, version 1.  K-major (Q, K):
// rows of 128 bytes, 8-row groups 1024 bytes apart.  MN-major (V): a row is 64
// columns of one key, 8-key groups 1024 bytes apart, the next 64 columns a slab
// further.  The high word is the same for all; the low one is the address (in
// units of 16 bytes) and the slab distance, so a step adds to it.
constexpr uint32_t DESC_HI = 1024 >> 4 | 1u << 14 | 2u << 29;
constexpr uint32_t DESC_V = (SLAB >> 4) << 16;
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return addr >> 4; }

// `lead` is set in one lane; the others run along, so that the warp never
// diverges around the products and their operands stay in uniform registers.
__device__ __forceinline__ uint32_t elect()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}

__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "setp.ne.u32 q, %5, 0;\n\tmov.b64 da, {%1, %6};\n\tmov.b64 db, {%2, %6};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(lead), "r"(DESC_HI)
                 : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "setp.ne.u32 q, %5, 0;\n\tmov.b64 db, {%2, %6};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(lead), "r"(DESC_HI)
                 : "memory");
}

#define FA_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), \
                    "=r"(r[i + 6]), "=r"(r[i + 7])
#define FA_W8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), \
                    "r"(r[i + 6]), "r"(r[i + 7])

// 32 columns of this warp's 32 TMEM lanes, one lane per thread.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
                 "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
                 "%28, %29, %30, %31}, [%32];"
                 : FA_R8(r, 0), FA_R8(r, 8), FA_R8(r, 16), FA_R8(r, 24)
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
                 "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
                 "%28, %29, %30, %31, %32};" ::"r"(addr),
                 FA_W8(r, 0), FA_W8(r, 8), FA_W8(r, 16), FA_W8(r, 24)
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
                 "%11, %12, %13, %14, %15, %16};" ::"r"(addr),
                 FA_W8(r, 0), FA_W8(r, 8)
                 : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The factor on weights whose reference moves from score a to score b >= a (q . k, before c2).
// The weights of scores that are not far are taken against the rounded product of reference and c2,
// so that their factor is that of the products.
__device__ __forceinline__ float rescale(float a, float b, float c2)
{
    const float y = __fmul_rn(b, c2);
    return ex2(fabsf(y) > FAR ? (a - b) * c2 : __fmul_rn(a, c2) - y);
}

// The low n bits, n of any sign and size.
__device__ __forceinline__ uint32_t below(int n)
{
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// V rows of key tile k that no row sees may hold anything: zero them, so that a
// weight of 0 leaves nothing.  `part` is the tile's 128 dims in shared memory.
__device__ __forceinline__ void clean(const Args &p, const Piece &pc, int k, uint32_t part, int lane)
{
    const int kb = pc.key_tile(k) * BN, hi = pc.x.hi - kb, lo = pc.x.lo - kb, sk = p.sink - kb;
    if (hi >= BN && (lo <= 0 || sk >= min(lo, BN)))
        return;
    for (int i = lane; i < BN * 8; i += 32) {
        const int r = i >> 3;
        if (r < hi && (r >= lo || r < sk))
            continue;
#pragma unroll
        for (int c = 0; c < 2; ++c)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(part + c * SLAB + i * 16), "r"(0)
                         : "memory");
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

// ------------------------------------------------------------ the main kernel
// Warp 0 loads, warps 1 and 3 issue the products of streams 0 and 1, warps 4-7 and
// 8-11 own their rows.  Every stream has two S buffers of SW keys, so that its
// products run ahead of its softmax: Q K^T of part i + 2 of the keys follows P V of
// part i, whose columns it takes over.  A piece whose tokens do not reach a stream
// leaves it out: it waits for none of its barriers.
struct Bars {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t q_full, q_empty;
    uint64_t s_full[2][2], p_full[2][2];    // S, P of [stream][buffer]
    uint64_t pv[2];                         // a P V of the stream done
    uint64_t o_full[2], o_empty[2];         // the unit's O complete; read out
    uint64_t raw_full[2], raw_empty[2];     // int8 V: a raw part has arrived, has been read
    uint64_t end;
    uint32_t tmem;
    uint32_t bits[BITS];                    // per key tile: groups in unmapped blocks
    int e0;
};

template <int D, bool VI8>
__global__ void __launch_bounds__(Cfg<D, VI8>::THREADS, 1)
    attend_kernel(const Args p, const __grid_constant__ CUtensorMap tmQ,
                  const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV)
{
    using C = Cfg<D, VI8>;
    constexpr int NS = C::NS, DS = C::DS, SW = C::SW, PARTS = BN / SW, STG = C::STG;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars &bars = *reinterpret_cast<Bars *>(smem + C::BAR_OFF);
    static_assert(sizeof(Bars) <= 512, "barriers fit their space");
    const uint32_t sQ = smem_u32(smem), ring = sQ + C::Q_BYTES;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int w = blockIdx.x;

    if (warp == 0 && lane == 0) {
        for (int i = 0; i < STG; ++i) {
            // (an int8 V stage is filled by four warps)
            mbar_init(smem_u32(&bars.full[i]), C::v_stage(i) ? 4 : 1);
            mbar_init(smem_u32(&bars.empty[i]), NS);
        }
        mbar_init(smem_u32(&bars.q_full), 1);
        mbar_init(smem_u32(&bars.q_empty), NS);
        for (int i = 0; i < 2; ++i) {
            for (int b = 0; b < 2; ++b) {
                mbar_init(smem_u32(&bars.s_full[i][b]), 1);
                mbar_init(smem_u32(&bars.p_full[i][b]), 4);
            }
            mbar_init(smem_u32(&bars.pv[i]), 1);
            mbar_init(smem_u32(&bars.o_full[i]), 1);
            mbar_init(smem_u32(&bars.o_empty[i]), 4);
            mbar_init(smem_u32(&bars.raw_full[i]), 1);
            mbar_init(smem_u32(&bars.raw_empty[i]), 4);
        }
        mbar_init(smem_u32(&bars.end), NS);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmQ)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmK)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmV)) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_u32(&bars.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        fence_before();
    }
    wait_for_previous();
    const int E = p.ebase[p.cache.B];
    const long long T = E > 0 ? p.pos[E] : 0;
    const long long units = (long long)E * p.cache.Hkv;
    const bool whole = units <= p.W && T <= units * (2 * units > p.W ? WHOLE_BUSY : WHOLE);
    const int We = T > 0 ? whole ? static_cast<int>(units) : ctas_for(p, T) : 0;
    const bool working = w < We;
    auto unit_at = [&](int u) {
        const int e = u / p.cache.Hkv;
        return e < E ? p.pos[e] + (long long)(u % p.cache.Hkv) * (p.ents[e].n + UNIT_COST) : T;
    };
    const long long t0 = !working ? 0 : whole ? unit_at(w) : T * w / We;
    const long long t1 = !working ? 0 : whole ? unit_at(w + 1) : T * (w + 1) / We;
    if (warp == 0 && working) {
        // the entry that holds position t0, 32 ways at a time
        int lo = 0, hi = E;                         // pos[lo] <= t0 < pos[hi]
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32;
            const int at = min(lo + step * lane, hi);
            const unsigned le = __ballot_sync(0xffffffffu, at < hi && p.pos[at] <= t0);
            const int last = 31 - __clz(le);
            hi = min(lo + step * (last + 1), hi);
            lo = lo + step * last;
        }
        if (lane == 0)
            bars.e0 = lo;
    }
    if (threadIdx.x == 0)
        p.split[w] = make_int4(-1, 0, 0, 0);
    __syncthreads();
    fence_after();
    const uint32_t tmem = bars.tmem;
    constexpr uint32_t O_COL = 256;

    Pieces walk;
    Piece pc;
    pc.e = -1;
    bool ok = working;
    if (working)
        walk.start(p, bars.e0, t0, t1);
    auto wait = [&](uint64_t &bar, uint32_t count) {      // the bar's phase number `count`
        if (mbar_wait_warp(smem_u32(&bar), count & 1))
            return true;
        if (lane == 0)
            flag(FA_STATUS_WAIT_TIMEOUT);
        return false;
    };
    // the piece has rows of stream s (of the first it always has)
    auto takes = [&](int s) { return NS == 1 || s == 0 || pc.x.ntok > p.tpt; };

    // key tiles that Q K^T runs ahead of P V by
    constexpr int LEAD = 2 / PARTS;
    // VI8 moves registers from the other warps to the rows'.  (8192-token prompt 511 us; 560 with
    // the roles of the first four warps in a branch of their own behind their setmaxnreg.)
    if (VI8 && warp < 4)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::FEW));
    if (warp == 0) {
        // ---------------------------------------------------------- loads
        uint32_t stage = 0, phase = 1, it = 0, qn = 0, tiles = 0;   // (stages filled, Q tiles, key tiles)
        uint32_t raw = 0;                                           // VI8: raw parts
        const int br = 1 << p.lg_br, groups = BN >> p.lg_br;
        const int g = lane % groups, slab = lane / groups;      // a lane per group of rows and 64 dims
        const uint32_t to = ring + slab * SLAB + g * br * 128;
        // a K or V tile: DS stages of 128 dims
        auto tile = [&](const CUtensorMap *map, int row) {
            const int y = row < 0 ? p.oob_row : row;
#pragma unroll
            for (int ds = 0; ds < DS; ++ds) {
                if constexpr (VI8) {
                    // K's stages: 0 and 2 in turn, or 0 and 1 for the two parts
                    stage = DS == 1 ? it % 2 * 2 : ds;
                    phase = (DS == 1 ? it / 2 : it / DS) + 1;
                }
                // (the first round of stages: the phase before a barrier's first counts as done)
                if (!wait(bars.empty[stage], phase))
                    return false;
                const uint32_t bar = smem_u32(&bars.full[stage]);
                if (lane == 0)
                    mbar_expect_tx(bar, STAGE_BYTES);
                __syncwarp();
                if (slab < 2)
                    tma_load(to + stage * STAGE_BYTES, map, ds * 128 + slab * 64, y, bar);
                ++it;
                if (!VI8 && ++stage == STG) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            return true;
        };
        // VI8: a V tile's raw parts
        auto raw_tile = [&](int row) {
            const int y = row < 0 ? p.oob_row : row;
#pragma unroll
            for (int ds = 0; ds < DS; ++ds) {
                const uint32_t b = raw % 2;
                if (!wait(bars.raw_empty[b], raw / 2 + 1))
                    return false;
                const uint32_t bar = smem_u32(&bars.raw_full[b]);
                if (lane == 0)
                    mbar_expect_tx(bar, RAW_BYTES);
                __syncwarp();
                if (slab == 0)
                    tma_load(sQ + C::RAW_OFF + b * RAW_BYTES + g * br * 128, &tmV, ds * 128, y, bar);
                ++raw;
            }
            return true;
        };
        while (ok && walk.next(p, pc)) {
            const int n = pc.k1 - pc.k0;
            if (n == 0)
                continue;
            // This lane's group of key tile j lies in block `look(j)` of the table, which is read
            // a tile before it is needed; its cache row is row_of(j, block): oob_row for groups
            // that no row sees, -1 for an unmapped block
            auto token = [&](int j) {
                const int t = j < n ? pc.key_tile(pc.k0 + j) * BN + g * br : pc.x.hi;
                return t < pc.x.hi && (t + br > pc.x.lo || t < p.sink) ? t : -1;
            };
            auto look = [&](int j) {
                const int t = token(j);
                return p.cache.bt && t >= 0
                           ? p.cache.bt[(long long)pc.x.b * p.cache.max_blocks + t / p.cache.page_size]
                           : 0;
            };
            auto row_of = [&](int j, int block) {
                const int t = token(j);
                if (t < 0)
                    return p.oob_row;
                if (!p.cache.bt)
                    return static_cast<int>(((long long)pc.x.b * p.cache.Hkv + pc.kv) * p.cache.cap + t);
                if (block < 0 || block >= p.cache.num_blocks)
                    return -1;
                return static_cast<int>(((long long)block * p.cache.Hkv + pc.kv) * p.cache.page_size +
                                        t % p.cache.page_size);
            };
            auto k_tile = [&](int row) {
                const uint32_t bits = __ballot_sync(0xffffffffu, row < 0 && slab == 0);
                if (lane == 0) {
                    if (bits)
                        flag(FA_STATUS_BAD_BLOCK);
                    bars.bits[tiles % BITS] = bits;
                }
                ++tiles;
                return tile(&tmK, row);
            };
            // in the order of their products: K0 (K1), then V(j), K(j + LEAD)
            const int block0 = look(0), block1 = look(1);
            int ahead = look(2);
            int row0 = row_of(0, block0), row1 = row_of(1, block1);
            ok = k_tile(row0);
            if (ok && qn > 0)
                ok = wait(bars.q_empty, qn - 1);
            if (!ok)
                break;
            if (lane == 0) {
                const uint32_t bar = smem_u32(&bars.q_full);
                const int box = p.group * p.tpt * 128, streams = NS == 2 && takes(1) ? 2 : 1;
                mbar_expect_tx(bar, streams * (D / 64) * box);
                for (int s = 0; s < streams; ++s)
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_3d(sQ + s * BM * D * 2 + c * SLAB, &tmQ, c * 64, pc.kv * p.group,
                                    pc.x.tok + s * p.tpt, bar);
            }
            ++qn;
            __syncwarp();
            if (LEAD == 2 && n > 1)
                ok = k_tile(row1);
            for (int j = 0; ok && j < n; ++j) {
                const int row2 = row_of(j + 2, ahead);
                ahead = look(j + 3);
                ok = VI8 ? raw_tile(row0) : tile(&tmV, row0);
                if (ok && j + LEAD < n)
                    ok = k_tile(LEAD == 1 ? row1 : row2);
                row0 = row1;
                row1 = row2;
            }
        }
        // no copy is left in flight when the CTA ends
        constexpr uint32_t LAST = VI8 ? 2 : STG;    // fills that may still be on their way
        for (uint32_t i = it > LAST ? it - LAST : 0; i < it; ++i) {
            const uint32_t st = !VI8 ? i % STG : DS == 1 ? i % 2 * 2 : i % 2;
            const uint32_t ph = (!VI8 ? i / STG : i / 2) & 1;
            mbar_wait_warp(smem_u32(&bars.full[st]), ph);
        }
        for (uint32_t i = raw > 2 ? raw - 2 : 0; i < raw; ++i)
            mbar_wait_warp(smem_u32(&bars.raw_full[i % 2]), i / 2 & 1);
        if (qn > 0)
            mbar_wait_warp(smem_u32(&bars.q_full), (qn - 1) & 1);
    } else if (warp == 1 || (NS == 2 && warp == 3)) {
        // ------------------------------------- products: a warp per stream
        // Each waits for every stage in turn and gives every stage back, also of
        // the pieces it sits out, so that neither loses count of the phases.
        const int s = warp >> 1;
        uint32_t stage = 0, phase = 0, qn = 0, on = 0, used[2] = {0, 0};
        constexpr uint32_t idesc_pv = 1u << 4 | 1u << 16 | (128u >> 3) << 17 | (128u >> 4) << 24;
        const uint32_t lead = elect();
        const uint32_t q_lo = desc_lo(sQ) + s * (BM * D * 2 >> 4), ring_lo = desc_lo(ring);
        const uint32_t s_col = tmem + s * 128, o_col = tmem + O_COL + s * 128;
        bool mine = true;
        auto full = [&](uint32_t st, uint32_t ph) {     // stage st has arrived
            if (mbar_wait_warp(smem_u32(&bars.full[st]), ph))
                return true;
            if (lane == 0)
                flag(FA_STATUS_WAIT_TIMEOUT);
            return false;
        };
        auto advance = [&] {
            if (++stage == STG) {
                stage = 0;
                phase ^= 1;
            }
        };
        uint32_t done = 0;                              // VI8 with two parts: tiles before the piece
        auto release = [&](uint32_t st) {               // refilled when the products are done
            mma_commit(lead, smem_u32(&bars.empty[st]));
        };
        // S of buffer b <- Q K^T: dims 128 ds .. of the keys from row 64 * half of stage st
        auto qk = [&](int b, int half, int ds, uint32_t st) {
            if (!mine)
                return;
            const uint32_t k = ring_lo + st * (STAGE_BYTES >> 4) + half * (64 * 128 >> 4);
            const uint32_t q = q_lo + ds * (2 * SLAB >> 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t off = ((i / 4) * SLAB + (i % 4) * 32) >> 4;
                mma_ss(lead, s_col + b * SW, q + off, k + off, p.idesc_qk, ds > 0 || i > 0);
            }
        };
        // O's columns 128 ds .. (+)= P of buffer b . the keys from row 64 * half of stage st
        auto pv = [&](int b, int half, int ds, uint32_t st, bool add) {
            if (!mine)
                return;
            const uint32_t v = ring_lo + DESC_V + st * (STAGE_BYTES >> 4) + half * (64 * 128 >> 4);
#pragma unroll
            for (int i = 0; i < SW / 16; ++i)
                mma_ts(lead, o_col + ds * 128, s_col + b * SW + i * 8, v + i * (2048 >> 4), idesc_pv, add || i > 0);
        };
        auto commit = [&](uint64_t &bar) {
            if (mine)
                mma_commit(lead, smem_u32(&bar));
        };
        // P of part i is there (and, first, O has been read out)
        auto p_ready = [&](int i) {
            if (!mine)
                return true;
            if (!wait(bars.p_full[s][i & 1], used[i & 1] + i / 2) ||
                (i == 0 && on > 0 && !wait(bars.o_empty[s], on - 1)))
                return false;
            fence_after();
            return true;
        };
        auto dirty = [&](int k) {       // only a range's ends hold keys that no row sees
            return mine && (k == pc.x.n - 1 || k == pc.x.ns || k == pc.x.ns - 1);
        };
        while (ok && walk.next(p, pc)) {
            const int n = __shfl_sync(0xffffffffu, pc.k1 - pc.k0, 0);
            if (n == 0)
                continue;
            mine = NS == 1 || __shfl_sync(0xffffffffu, takes(s), 0);
            ok = wait(bars.q_full, qn);
            ++qn;
            if constexpr (PARTS == 2) {
                // parts 2 j and 2 j + 1 are the halves of tile j
                ok = ok && full(stage, phase);
                if (ok) {
                    for (int b = 0; b < 2; ++b) {
                        qk(b, b, 0, stage);
                        commit(bars.s_full[s][b]);
                    }
                    release(stage);
                    if (n == 1)
                        mma_commit(lead, smem_u32(&bars.q_empty));
                    advance();
                }
                for (int j = 0; ok && j < n; ++j) {
                    const uint32_t v = stage, vp = phase;
                    advance();
                    const uint32_t k = stage, kp = phase;
                    ok = full(v, vp);
                    if (!VI8 && ok && dirty(pc.k0 + j))
                        clean(p, pc, pc.k0 + j, ring + v * STAGE_BYTES, lane);
                    for (int b = 0; ok && b < 2; ++b) {
                        ok = p_ready(2 * j + b);
                        if (!ok)
                            break;
                        pv(b, b, 0, v, 2 * j + b > 0);
                        commit(bars.pv[s]);
                        if (b == 1)
                            release(v);
                        if (j + 1 < n) {
                            if (b == 0)
                                ok = full(k, kp);
                            if (ok) {
                                qk(b, b, 0, k);
                                commit(bars.s_full[s][b]);
                            }
                        }
                    }
                    if (ok && j + 1 < n) {
                        release(k);
                        advance();
                        if (j + 2 == n)
                            mma_commit(lead, smem_u32(&bars.q_empty));
                    }
                }
            } else {
                auto k_tile = [&](int j) {
                    for (int ds = 0; ds < DS; ++ds) {
                        const uint32_t st = VI8 ? ds : stage;
                        if (!full(st, VI8 ? done + j & 1 : phase))
                            return false;
                        qk(j & 1, 0, ds, st);
                        release(st);
                        if (!VI8)
                            advance();
                    }
                    commit(bars.s_full[s][j & 1]);
                    if (j == n - 1)
                        mma_commit(lead, smem_u32(&bars.q_empty));
                    return true;
                };
                ok = ok && k_tile(0) && (n == 1 || k_tile(1));
                for (int j = 0; ok && j < n; ++j) {
                    for (int ds = 0; ok && ds < DS; ++ds) {
                        const uint32_t st = VI8 ? 2 + ds : stage;
                        ok = full(st, VI8 ? done + j & 1 : phase);
                        if (!VI8 && ok && dirty(pc.k0 + j))
                            clean(p, pc, pc.k0 + j, ring + st * STAGE_BYTES, lane);
                        if (ok && ds == 0)
                            ok = p_ready(j);
                        if (!ok)
                            break;
                        pv(j & 1, 0, ds, st, j > 0);
                        release(st);
                        if (!VI8)
                            advance();
                    }
                    if (ok) {
                        commit(bars.pv[s]);
                        if (j + 2 < n)
                            ok = k_tile(j + 2);
                    }
                }
            }
            done += n;
            if (ok && mine) {
                commit(bars.o_full[s]);
                ++on;
                used[0] += (n * PARTS + 1) / 2;
                used[1] += n * PARTS / 2;
            }
        }
        // no product is left running when the TMEM goes back
        mma_commit(lead, smem_u32(&bars.end));
        mbar_wait_warp(smem_u32(&bars.end), 0);
    } else if (warp >= 4 && (!VI8 || warp < 4 + 4 * NS)) {
        if constexpr (VI8)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::MANY));
        // ---------------------------------------------------------- softmax
        const int s = (warp - 4) >> 2;              // stream
        const int r = threadIdx.x & 127;            // row of the stream
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
        const uint32_t s_col = lanes + s * 128, o_col = lanes + O_COL + s * 128;
        uint32_t tiles = 0, on = 0, pv_n = 0, used[2] = {0, 0};
        float m, l;                     // a unit's reference (a score before c2), sum of its weights
        float kept;                     // the reference of O in the slot
        bool far;                       // some row of the warp has one beyond FAR
        while (ok && walk.next(p, pc)) {
            const int n = pc.k1 - pc.k0, m_parts = n * PARTS;
            if (pc.begins) {
                m = kept = -INFINITY;
                l = 0.f;
                far = false;
            }
            if (takes(s)) {
                const int i_tok = s * p.tpt + r / p.group;
                const int at = pc.x.at + i_tok;
                // positions of this stream's first and last row
                const int at_lo = pc.x.at + s * p.tpt;
                const int at_hi = pc.x.at + min((s + 1) * p.tpt, pc.x.ntok) - 1;
                for (int i = 0; ok && i < m_parts; ++i) {
                    const int b = i & 1, half = PARTS == 2 ? b : 0;
                    ok = wait(bars.s_full[s][b], used[b] + i / 2);
                    if (!ok)
                        break;
                    fence_after();
                    uint32_t x[SW];
#pragma unroll
                    for (int c = 0; c < SW / 32; ++c)
                        tmem_ld32(s_col + b * SW + c * 32, x + c * 32);
                    const int kb = pc.key_tile(pc.k0 + i / PARTS) * BN + half * SW;
                    const uint32_t bits =
                        *reinterpret_cast<volatile uint32_t *>(&bars.bits[(tiles + i / PARTS) % BITS]);
                    const bool edge = kb + SW - 1 > at_lo || bits ||
                                      (pc.x.window > 0 && kb <= at_hi - pc.x.window && kb + SW > p.sink);
                    tmem_ld_wait();
                    // a bit per column of 32 that the row sees
                    auto seen = [&](int c) {
                        const int hi = at - kb, lo = pc.x.window > 0 ? hi - pc.x.window + 1 : -1;
                        const int sk = p.sink - kb;
                        uint32_t see = below(hi + 1 - c * 32) & (~below(lo - c * 32) | below(sk - c * 32));
                        if (bits)
                            for (int t = 0; t < 32; t += 16)
                                if (bits >> ((half * SW + c * 32 + t) >> p.lg_br) & 1)
                                    see &= ~(0xffffu << t);
                        return see;
                    };
                    if (edge) {
#pragma unroll
                        for (int c = 0; c < SW / 32; ++c) {
                            const uint32_t see = seen(c);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(see >> e & 1))
                                    x[c * 32 + e] = 0xff800000u;        // -infinity
                        }
                    }
                    float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};   // chains of their own
#pragma unroll
                    for (int e = 0; e < SW; e += 2)
                        tops[e / 2 & 3] = max3(tops[e / 2 & 3], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                    const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                    const bool grow = (top - m) * p.c2 > GROW;      // also from -infinity
                    if (__any_sync(0xffffffffu, grow)) {
                        // a row's reference follows its own scores alone: its bits depend neither on
                        // its neighbours nor on the rows behind the last token, which hold anything
                        const float a = grow ? rescale(m, top, p.c2) : 1.f;
                        m = grow ? top : m;
                        l *= a;
                        far = __any_sync(0xffffffffu, m != -INFINITY && fabsf(m * p.c2) > FAR);
                        if (i > 0) {
                            // the P V before must have landed
                            ok = wait(bars.pv[s], pv_n + i - 1);
                            if (!ok)
                                break;
                            fence_after();
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t o[32];
                                tmem_ld32(o_col + c * 32, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                                tmem_st32(o_col + c * 32, o);
                            }
                        }
                    }
                    const float ref = m == -INFINITY ? 0.f : __fmul_rn(m, p.c2) - UP;
                    const uint64_t c22 = pair2(p.c2, p.c2), ref2 = pair2(-ref, -ref);
                    uint64_t sums[4] = {0, 0, 0, 0};
                    if (far) {                  // (uniform over the warp; the scores are read again)
                        const bool mine = m != -INFINITY && fabsf(m * p.c2) > FAR;
                        const float from = mine ? m : 0.f, up = mine ? UP : -ref;
#pragma unroll 1
                        for (int c = 0; c < SW / 32; ++c) {
                            uint32_t y[32], h[16];
                            tmem_ld32(s_col + b * SW + c * 32, y);
                            const uint32_t see = seen(c);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float w[2];
#pragma unroll
                                for (int k = 0; k < 2; ++k)
                                    w[k] = see >> (2 * e + k) & 1
                                               ? ex2_ftz(fmaf(__uint_as_float(y[2 * e + k]) - from, p.c2, up))
                                               : 0.f;
                                h[e] = tc::pack_half2(w[0], w[1]);
                                sums[e & 3] = add2(sums[e & 3], pair2(w[0], w[1]));
                            }
                            tmem_st16(s_col + b * SW + c * 16, h);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < SW / 32; ++c) {
                            // a step for all 32 before the next: a dozen exponentials in flight
                            uint32_t h[16];
                            float w[32];
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                split2(fma2(pair2(__uint_as_float(x[c * 32 + 2 * e]),
                                                  __uint_as_float(x[c * 32 + 2 * e + 1])), c22, ref2),
                                       w[2 * e], w[2 * e + 1]);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                w[e] = ex2_ftz(w[e]);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                h[e] = tc::pack_half2(w[2 * e], w[2 * e + 1]);
                                sums[e & 3] = add2(sums[e & 3], pair2(w[2 * e], w[2 * e + 1]));
                            }
                            tmem_st16(s_col + b * SW + c * 16, h);
                        }
                    }
                    tmem_st_wait();
                    fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_u32(&bars.p_full[s][b]));
                    {
                        float a, d;
                        split2(add2(add2(sums[0], sums[1]), add2(sums[2], sums[3])), a, d);
                        l += a + d;
                    }
                }
                if (ok && n > 0) {
                    ok = wait(bars.o_full[s], on);
                    ++on;
                }
                if (!ok)
                    break;
                fence_after();
                // ---- the unit's rows, or this piece's partial of them
                const bool live = r < p.tpt * p.group && i_tok < pc.x.ntok;
                const float inv = l > 0.f ? 1.f / l : 0.f;
                __half *dst = p.out + ((long long)(pc.x.tok + i_tok) * p.hq + pc.kv * p.group + r % p.group) * D;
                // (a whole unit may take the slot of the CTA's last piece, which comes after it)
                float4 *part = reinterpret_cast<float4 *>(p.part) +
                               (size_t)(pc.slot >= 0 ? pc.slot : 2 * w + 1) * (D / 4) * C::ROWS + s * BM + r;
                const float f = kept == -INFINITY ? 0.f : rescale(kept, m, p.c2);
                kept = m;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    if (n > 0) {
                        tmem_ld32(o_col + c * 32, o);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = 0;
                    }
                    if (!live)
                        continue;
                    if (!pc.begins) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float4 was = part[(size_t)(c * 8 + e) * C::ROWS];
                            o[4 * e] = __float_as_uint(fmaf(was.x, f, __uint_as_float(o[4 * e])));
                            o[4 * e + 1] = __float_as_uint(fmaf(was.y, f, __uint_as_float(o[4 * e + 1])));
                            o[4 * e + 2] = __float_as_uint(fmaf(was.z, f, __uint_as_float(o[4 * e + 2])));
                            o[4 * e + 3] = __float_as_uint(fmaf(was.w, f, __uint_as_float(o[4 * e + 3])));
                        }
                    }
                    if (pc.slot >= 0 || !pc.ends) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            part[(size_t)(c * 8 + e) * C::ROWS] =
                                make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                            __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t h[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                h[k] = tc::pack_half2(__uint_as_float(o[8 * e + 2 * k]) * inv,
                                                      __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
                            *reinterpret_cast<uint4 *>(dst + c * 32 + e * 8) = make_uint4(h[0], h[1], h[2], h[3]);
                        }
                    }
                }
                if (pc.slot >= 0 && live)
                    p.ml[(size_t)pc.slot * C::ROWS + s * BM + r] = make_float2(m, l);
                if (n > 0) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_u32(&bars.o_empty[s]));
                }
                if (pc.first_part && s == 0 && r == 0)
                    p.split[w] = make_int4(pc.e, pc.kv,
                                           static_cast<int>(((t0 + pc.last + 1) * We - 1) / T) - w + 1, 0);
                used[0] += (m_parts + 1) / 2;
                used[1] += m_parts / 2;
                pv_n += m_parts;
            }
            tiles += n;
        }
    } else if (VI8 && warp >= 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::FEW));
        // ---------------------------------------------------------- int8 V
        // A thread per row of a tile: its codes times its scales, rounded to fp16, into
        // the swizzled stage; zeros for rows that no row of q sees or whose block is
        // unmapped.  The lanes' 16-byte chunks are rotated by the row, so that both the
        // reads and the writes of eight lanes fall into different banks.
        const int r = threadIdx.x & 127;
        uint32_t raw = 0, tiles = 0;
        while (ok && walk.next(p, pc)) {
            const int n = pc.k1 - pc.k0;
            // the scales of this thread's row of key tile j, on their way a tile early
            auto look = [&](int j, uint2 (&sc)[DS]) {
                const int t = j < n ? pc.key_tile(pc.k0 + j) * BN + r : pc.x.hi;
                long long row = -1;
                if (t < pc.x.hi && (t >= pc.x.lo || t < p.sink))
                    row = tc::tile_row(p.cache, pc.x.b, pc.kv, t);
#pragma unroll
                for (int ds = 0; ds < DS; ++ds)
                    sc[ds] = row < 0 ? make_uint2(0u, 0u)
                                     : __ldg(reinterpret_cast<const uint2 *>(p.v_scales + row * (D / 32)) + ds);
                return row >= 0;
            };
            uint2 next[DS];
            bool next_live = look(0, next);
            for (int j = 0; ok && j < n; ++j) {
                uint2 sc[DS];
                const bool live = next_live;
#pragma unroll
                for (int ds = 0; ds < DS; ++ds)
                    sc[ds] = next[ds];
                next_live = look(j + 1, next);
#pragma unroll
                for (int ds = 0; ds < DS; ++ds) {
                    const uint32_t b = raw % 2, st = DS == 1 ? 1 + tiles % 2 * 2 : 2 + ds;
                    ok = ok && wait(bars.raw_full[b], raw / 2) &&
                         wait(bars.empty[st], (DS == 1 ? tiles / 2 : tiles) + 1);
                    if (!ok)
                        break;
                    const uint32_t src = sQ + C::RAW_OFF + b * RAW_BYTES + r * 128;
                    const uint32_t dst = ring + st * STAGE_BYTES + r * 128;
#pragma unroll 4
                    for (int i = 0; i < 8; ++i) {
                        const int c = (i + r) & 7;
                        uint32_t w[4], o[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                     : "r"(src + c * 16));
                        if (live) {
                            const uint32_t two = c & 4 ? sc[ds].y : sc[ds].x;
                            const __half2 s2 = __half2half2(
                                __ushort_as_half(static_cast<unsigned short>(c & 2 ? two >> 16 : two)));
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc::dequant4(w[k], s2, o[2 * k], o[2 * k + 1]);
                        }
                        const uint32_t to = dst + (c >> 2) * SLAB;
                        const int q = 2 * c & 7;
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                             to + (((q + k) ^ (r & 7)) * 16)),
                                         "r"(o[4 * k]), "r"(o[4 * k + 1]), "r"(o[4 * k + 2]), "r"(o[4 * k + 3])
                                         : "memory");
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_u32(&bars.full[st]));
                        mbar_arrive(smem_u32(&bars.raw_empty[b]));
                    }
                    ++raw;
                }
                ++tiles;
            }
        }
    }
    __syncthreads();
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ------------------------------------------------------------ the merge
// CTA (x, w): 256 of the (row, 16 columns) of the unit that CTA w of the main kernel
// began and left to the next ones: their partials in order, weighed by 2^(c2 (m - M)).
template <int D>
__global__ void __launch_bounds__(256) merge_kernel(const Args p)
{
    using C = Cfg<D>;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    wait_for_previous();
    const int w = blockIdx.y;
    const int4 u = p.split[w];
    if (u.x < 0)
        return;
    const Ent x = p.ents[u.x];
    const int idx = blockIdx.x * 256 + threadIdx.x;
    const int row = idx % C::ROWS, c16 = idx / C::ROWS;
    const int s = row / BM, r = row % BM;
    const int i_tok = s * p.tpt + r / p.group;
    if (r >= p.tpt * p.group || i_tok >= x.ntok)
        return;
    auto slot = [&](int i) { return (size_t)(i == 0 ? 2 * w + 1 : 2 * (w + i)); };
    float M = -INFINITY;
    for (int i = 0; i < u.z; ++i)
        M = fmaxf(M, p.ml[slot(i) * C::ROWS + row].x);
    float4 o[4] = {};
    float L = 0.f;
    for (int i = 0; i < u.z; ++i) {
        const float2 v = p.ml[slot(i) * C::ROWS + row];
        const float a = v.x == -INFINITY ? 0.f : rescale(v.x, M, p.c2);
        L = fmaf(v.y, a, L);
        const float4 *src = reinterpret_cast<const float4 *>(p.part) + slot(i) * (D / 4) * C::ROWS +
                            (size_t)c16 * 4 * C::ROWS + row;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float4 y = src[(size_t)c * C::ROWS];
            o[c].x = fmaf(y.x, a, o[c].x);
            o[c].y = fmaf(y.y, a, o[c].y);
            o[c].z = fmaf(y.z, a, o[c].z);
            o[c].w = fmaf(y.w, a, o[c].w);
        }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    __half *dst = p.out + ((long long)(x.tok + i_tok) * p.hq + u.y * p.group + r % p.group) * D + c16 * 16;
#pragma unroll
    for (int c = 0; c < 2; ++c)
        *reinterpret_cast<uint4 *>(dst + 8 * c) =
            make_uint4(tc::pack_half2(o[2 * c].x * inv, o[2 * c].y * inv),
                       tc::pack_half2(o[2 * c].z * inv, o[2 * c].w * inv),
                       tc::pack_half2(o[2 * c + 1].x * inv, o[2 * c + 1].y * inv),
                       tc::pack_half2(o[2 * c + 1].z * inv, o[2 * c + 1].w * inv));
}

// Sizes of a call and the layout of its workspace.
struct Space {
    int tpt, per, max_ents, W;
    size_t ents, pos, ebase, split, ml, part, total;    // offsets, and the bytes in all
};

static Space space_of(int batch, int n_tokens, int hq, int hkv, int D, long long cap, int sms)
{
    Space s = {};
    const int ns = D == 128 ? Cfg<128>::NS : Cfg<256>::NS;
    const int rows = D == 128 ? Cfg<128>::ROWS : Cfg<256>::ROWS;
    const size_t slot = D == 128 ? Cfg<128>::SLOT_BYTES : Cfg<256>::SLOT_BYTES;
    s.tpt = BM / (hq / hkv);
    s.per = ns * s.tpt;
    s.max_ents = n_tokens / s.per + (batch < n_tokens ? batch : n_tokens);
    const double most = (double)s.max_ents * hkv * ((cap + BN - 1) / BN + UNIT_COST) / MIN_POS;
    s.W = most < 1 ? 1 : most < sms ? static_cast<int>(most) : sms;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += (n + 127) / 128 * 128;
        return here;
    };
    s.ents = take((size_t)s.max_ents * sizeof(Ent));
    s.pos = take(((size_t)s.max_ents + 1) * sizeof(long long));
    s.ebase = take(((size_t)batch + 1) * sizeof(int));
    s.split = take((size_t)s.W * sizeof(int4));
    s.ml = take((size_t)2 * s.W * rows * sizeof(float2));
    s.part = take((size_t)2 * s.W * slot);
    s.total = at;
    return s;
}

// [rows][D] of fp16 in boxes of `br` rows x 64 columns, 128-byte swizzle; q as
// [tokens][heads][D] in boxes of tpt tokens x G heads x 64 columns; bytes: int8 V in
// boxes of `br` rows x 128 columns as they lie.
static int encode_map(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims,
                      const cuuint64_t *strides, const cuuint32_t *box, bool bytes = false)
{
    auto enc = tensor_map_encoder();
    if (!enc)
        return fail(FA_ERR_CUDA, "fa_prefill: cuTensorMapEncodeTiled unavailable");
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                           const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           bytes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(FA_ERR_CUDA, "fa_prefill: cuTensorMapEncodeTiled failed (%d)", (int)r);
    return 0;
}

template <int D, bool VI8>
static cudaError_t launch(const Args &p, const CUtensorMap &tmQ, const CUtensorMap &tmK,
                          const CUtensorMap &tmV, int per, cudaStream_t st)
{
    using C = Cfg<D, VI8>;
    static std::mutex mu;
    static bool done[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev >= 64 || !done[dev]) {
            e = cudaFuncSetAttribute(attend_kernel<D, VI8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
            if (e != cudaSuccess)
                return e;
            if (dev < 64)
                done[dev] = true;
        }
    }
    plan_kernel<<<1, PLAN_THREADS, 0, st>>>(p, per);
    e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(p.W);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    e = cudaLaunchKernelEx(&cfg, attend_kernel<D, VI8>, p, tmQ, tmK, tmV);
    if (e != cudaSuccess)
        return e;
    cfg.gridDim = dim3(C::ROWS * (D / 16) / 256, p.W);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, merge_kernel<D>, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
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
    return space_of(batch, n_tokens, n_q_heads, n_kv_heads, head_dim, max_kv_len, num_sms).total;
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
    const bool vi8 = v_scales != nullptr;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(v_scales) || !aligned16(out) ||
        !aligned16(workspace) || !aligned_to(seq_lens, 4) || !aligned_to(block_table, 4) ||
        !aligned_to(window, 4) || !aligned_to(starts, 4))
        return fail(FA_ERR_ALIGN, "fa_prefill: q, caches, out and workspace must be 16-byte, int32 "
                                  "arrays 4-byte aligned");
    int sms = 0;
    if (const int rc = device_sms(&sms))
        return rc;
    const Space sp = space_of(batch, n_tokens, n_q_heads, n_kv_heads, D, cap, sms);
    const size_t need = sp.total;
    if (!workspace || workspace_bytes < need)
        return fail(FA_ERR_WORKSPACE, "fa_prefill: workspace %zu bytes, need %zu", workspace_bytes,
                    need);
    const size_t qn = (size_t)n_tokens * n_q_heads * D * 2;
    const struct { const void *p; size_t n; } in[] = {
        {q, qn}, {k_cache, rows * D * 2}, {v_cache, rows * D * (vi8 ? 1 : 2)},
        {v_scales, rows * (D / 32) * 2}, {seq_lens, (size_t)batch * 4},
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
    p.starts = starts;
    p.window = window;
    p.v_scales = static_cast<const __half *>(v_scales);
    p.out = static_cast<__half *>(out);
    p.tokens = n_tokens;
    p.hq = n_q_heads;
    p.group = n_q_heads / n_kv_heads;
    p.tpt = sp.tpt;
    p.sink = n_sink;
    // boxes of as many rows as always lie together, the largest power of two in a page; at most
    // half a tile, so that half of a tile that no row sees is not read
    const int br = paged && (page_size & -page_size) < 64 ? (page_size & -page_size) : 64;
    p.lg_br = log2_of(br);
    p.oob_row = static_cast<int>(rows);
    // a negative scale: the product negates Q; the running maximum wants c2 > 0, and 0
    // weighs every key alike, as this does
    const double c2 = fabs(static_cast<double>(scale)) * 1.4426950408889634;
    p.c2 = static_cast<float>(fmin(fmax(c2, 1e-37), static_cast<double>(FLT_MAX)));
    const uint32_t sw = D == 128 ? Cfg<128>::SW : Cfg<256>::SW;
    p.idesc_qk = 1u << 4 | (scale < 0.f ? 1u << 13 : 0u) | (sw >> 3) << 17 | (BM >> 4) << 24;
    p.W = sp.W;
    p.max_ents = sp.max_ents;
    char *ws = static_cast<char *>(workspace);
    p.ents = reinterpret_cast<Ent *>(ws + sp.ents);
    p.pos = reinterpret_cast<long long *>(ws + sp.pos);
    p.ebase = reinterpret_cast<int *>(ws + sp.ebase);
    p.split = reinterpret_cast<int4 *>(ws + sp.split);
    p.ml = reinterpret_cast<float2 *>(ws + sp.ml);
    p.part = reinterpret_cast<float *>(ws + sp.part);
    CUtensorMap tmQ, tmK, tmV;
    const cuuint64_t qd[3] = {(cuuint64_t)D, (cuuint64_t)n_q_heads, (cuuint64_t)n_tokens};
    const cuuint64_t qs[2] = {(cuuint64_t)D * 2, (cuuint64_t)n_q_heads * D * 2};
    const cuuint32_t qb[3] = {64, (cuuint32_t)p.group, (cuuint32_t)p.tpt};
    const cuuint64_t kd[2] = {(cuuint64_t)D, (cuuint64_t)rows};
    const cuuint64_t ks[1] = {(cuuint64_t)D * 2};
    const cuuint32_t kb[2] = {64, (cuuint32_t)br};
    int rc = encode_map(&tmQ, q, 3, qd, qs, qb);
    if (!rc)
        rc = encode_map(&tmK, k_cache, 2, kd, ks, kb);
    const cuuint64_t vs[1] = {(cuuint64_t)D};
    const cuuint32_t vb[2] = {128, (cuuint32_t)br};
    if (!rc)
        rc = vi8 ? encode_map(&tmV, v_cache, 2, kd, vs, vb, true) : encode_map(&tmV, v_cache, 2, kd, ks, kb);
    if (rc)
        return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto go = [&](auto int8) {
        constexpr bool I = decltype(int8)::value;
        return D == 128 ? launch<128, I>(p, tmQ, tmK, tmV, sp.per, st) : launch<256, I>(p, tmQ, tmK, tmV, sp.per, st);
    };
    const cudaError_t e = vi8 ? go(std::true_type()) : go(std::false_type());
    if (e != cudaSuccess)
        return fail(FA_ERR_CUDA, "fa_prefill: launch failed: %s", cudaGetErrorString(e));
    return 0;
}

}  // extern "C"
