// paged_attn.cuh -- attention of one new token per request over a paged key-value cache.
//
// For request b, query head i of key head h = i / G, and keys n in [lo_b, len_b):
//     o = sum_n 2^(s_n - m) v_n / sum_n 2^(s_n - m),   s_n = (scale log2 e) q . k_n
// for any reference m; a range of keys is summed up by (m, l = sum 2^(s_n - m),
// o = sum 2^(s_n - m) v_n), and ranges join as m' = max m_i, l' = sum l_i 2^(m_i - m'),
// o' likewise.
//
// What bounds it: HBM.  A cached token costs 4 G flops per key and value element pair of 4
// bytes (2 in q8), which the matrix instructions do at a fraction of their rate; the design
// keeps enough bytes in flight and few instructions per byte.  GB300, against the measured
// copy rate of 6782 GB/s: 64 requests of 1000 to 32768 tokens, 8 key heads of 128 in fp16 (2.42
// GB), 350 to 363 us on different machines, 6.7 to 6.9 TB/s; one request of 131071 tokens (537 MB) 85.1 us, 6.3 TB/s; 16 ragged
// requests (62 MB) 17.1 us, of which 2.3 us pass before the first keys arrive and 3.5 us join the
// split items.  q8 is bound by its arithmetic: 533 instructions per 16 keys and warp to widen,
// scale and multiply 4 KB (48 requests of 500 to 16000 tokens, 476 MB, 100.4 us, 4.7 TB/s).  Few
// tokens cost a chain of trips to memory, lengths -> pages -> keys -> output: 3.75 us for 17.
//
// Work: a unit is TK consecutive keys of one (request, key head, block of query heads).
// The units of all requests, in that order, are dealt out evenly over one resident grid, so
// a batch of any mix of lengths keeps every SM streaming to the end; a CTA computes its
// share from `lens` by itself.  An item's own cost counts as a unit or two: equal units alone
// gave CTAs with many short items up to 1.6 times the mean time (25 requests of 30 to 6667 tokens,
// 32 heads of 80: 94 us, with it 64 us).  A share may begin and end inside a (request, head) item:
// such pieces go to the workspace as (m, l, o) in fp32 and the last CTA to arrive at the
// item joins them in the order of the keys, so results do not depend on the order of
// arrival.  (Large pieces of few items are joined by a second kernel, see paged_attn_splits.)
//
// CTA: NW warps, four or one.  WH warps work on the same keys for 8 NH query heads each,
// NW / WH such groups on neighbouring keys; each group has its own ring of S stages in
// shared memory, filled by cp.async 16 bytes at a time (rows of any page size and stride;
// rows past the range are filled with zeros, so what lies there is never read) and waits
// for nobody else.  Page ids are read one unit ahead, and an item's queries travel with its
// first unit.
//
// Products run on mma.sync m16n8k16 with the keys as the 16 rows and the query heads as the
// 8 columns (scores), then the value columns as rows (outputs), so that 8 query heads, the
// common case, waste nothing; tcgen05.mma would want 128 rows with 8 columns and a trip
// through tensor memory for a softmax over every column.  The weights turn from a result
// into an operand by movmatrix.
//
// Numbers: scores, maxima, sums and outputs stay in fp32.  The reference m moves only when
// a score passes it by kAttnSlack, so most units rescale nothing; weights are then at most
// 2^kAttnSlack.  What enters the products in fewer bits:
//   16-bit caches: weights as the sum of two 16-bit values (the rounded weight and the rounded rest,
//     2^-16 of a weight in bf16, 2^-22 in fp16): one rounding to 8 bits would cost as much accuracy as
//     the output's own, and the matrix unit has the time.  fp16 ends at 2^-24, where the tokens of a
//     long context beside one that outweighs them all would be rounded to few bits or to zero
//     (131071 tokens 16.3 below: their sum 7 % short with the heavy one in one warp of four).  The
//     reference therefore stays 2^kAttnLower below the largest score: weights reach 2^15 and keep
//     2^-32 of the largest one.
//   q8: weight times value scale in fp16, two parts for fp16 queries (2^-22).  One part for bf16
//     queries: 2^-11 of a weight, an eighth of the output's rounding, where two would cost 5 to 18 %
//     (48 requests of 4096 tokens, 8 heads of 128 a request: 77 and 84 us head by head, 16 query heads
//     a key head 101 and 120).  Below fp16's range 2^-31 of a group's largest scale is kept (v_top).
//   q8 with bf16 queries: queries in fp16, scaled by a power of two per head: what is 2^-25 of the
//     head's largest element is lost (load_q).
// The second part of a weight may be 0 or negative, so an infinite value makes its column NaN.
#pragma once

#include <type_traits>

#include "paged.cuh"
#include "ptx.cuh"

namespace sdt {

constexpr float kAttnSlack = 8.f;  // log2 by which a score may pass the largest before it: rarely passed
constexpr float kAttnLower = 7.f;  // log2 of an fp16 cache's weights at the largest score: with the slack 2^15 of fp16's 65504
constexpr int kAttnSplitValues = 2048;  // least values of a piece's o that a second kernel joins
constexpr int kAttnFlat = 256;     // most pieces x query heads that are joined in one level

struct PagedAttnArgs {
    const char *q;             // strides in bytes
    char *out;
    float *lse;                // [batch][q_heads], or null
    int64_t q_batch, q_head, o_batch, o_head;
    KvRows k, v;
    ScaleRows ks, vs;
    const int *table;
    int64_t table_stride;
    const int *lens;
    int batch, kv_heads, group, head_blocks;  // group: query heads per key head
    int head_dim, max_pages, num_pages, window;
    int whole_pages;           // 1: any 16 consecutive keys of a unit lie in one page, fewer than 2^31 bytes apart
    FastDiv page;
    float scale_log2;          // scale * log2(e)
    int q_rows;                // query rows that a CTA keeps in shared memory: min(group, 8 NH WH)
    float *partials;           // 2 slots per CTA: [rows][DP] o, [rows] m, [rows] l
    unsigned *counters;        // 3 per CTA, zero between calls
    int2 *split;               // null: the last CTA to arrive joins an item's pieces; else [items]: the first
                               // CTA with a piece of an item writes (that CTA, pieces), 0 pieces if it is whole,
                               // and a kernel of its own joins them
    int *status;
};

template <int DP, int NH, int WH, int NW, bool Q8>
struct AttnCfg {
    static constexpr int THREADS = NW * 32;
    static constexpr int ROWB = DP * (Q8 ? 1 : 2);        // bytes of a cached row in shared memory
    // Keys per warp of a unit: about 8 KB of keys and values, and room for the warp's o (8 NH x DP
    // fp32), which passes through the stage at an item's end.  Smaller units cost more instructions a key
    // (q8 of 128, 48 requests of 4096: 16 keys a warp 96.4 us, 32 keys 75.8 at the time, 76.4 now).
    static constexpr int KW = Q8 ? (DP == 256 && NH == 1 ? 16 : 32) : (DP == 64 ? 32 : 16);
    static constexpr int TK = KW * NW;                    // keys of a unit
    static constexpr int WK = NW / WH;                    // groups of warps with keys of their own
    static constexpr int KS = TK / WK;                    // keys of one group
    static constexpr int RW = KW;                         // rows that one warp loads
    static constexpr int SCB = Q8 ? DP / 16 : 0;          // bytes of a row's scales
    static constexpr int STAGE = TK * 2 * (ROWB + SCB);
    static constexpr int HEADS = 8 * NH;                  // query heads of a warp
    static constexpr int ROWS = HEADS * WH;               // query heads of a CTA
    static constexpr int SLOT = ROWS * (DP + 2);          // floats of a partial
    static constexpr int QROW = DP * 2;                   // bytes of a query row in shared memory
    // Whether a call may have its pieces joined by the second kernel (paged_attn_splits).
    static constexpr bool SPLITS = ROWS * DP >= kAttnSplitValues;
    // The warps of an SM hide each other's latency, so stages beyond two are worth less than another CTA
    // where one fits: one-warp CTAs, heads of 64 and q8 of 128 take two (that: 48 requests of 500 to 16000
    // tokens 100 us with three CTAs an SM, 108 with three stages and two CTAs).  Four warps of 16-bit heads of
    // 128 have three stages, two CTAs an SM (one request of 8192 tokens 16.0 us; two stages, three CTAs and their pieces 21.0; 2.42 GB of
    // cache the same within 2 %); wider heads have the SM to themselves.
    static constexpr bool fits(int s, int bytes) { return s * (STAGE + ROWS * QROW) + 2048 <= bytes; }
    static constexpr int S = NW == 1 || DP == 64 || (Q8 && DP == 128) ? 2 : fits(3, 113 * 1024) || (!fits(2, 113 * 1024) && fits(3, 227 * 1024)) ? 3 : 2;
    // What an item costs besides its units (queries, join of the warps, output), in units: measured 1.5 to
    // 2.3 us an item against 0.9 to 1.4 us a unit, and 3 us a unit in q8 of 128.
    static constexpr int COST = NW == 1 || Q8 ? 1 : 2;
    static constexpr int smem(int q_rows) { return S * (STAGE + q_rows * QROW); }
    static_assert(fits(S, 227 * 1024), "shared memory of an SM");
    static_assert(STAGE >= NW * HEADS * DP * 4, "the stage must hold every warp's o");
    static_assert(RW <= 32, "a lane describes one row");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// An 8 x 8 matrix of 16-bit elements, row lane / 4 and columns 2 (lane % 4) + {0, 1} a lane, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// d (16 x 8, fp32) = a (16 x 16) . b (16 x 8) + c
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const float (&c)[4]) {
    if constexpr (std::is_same_v<T, __half>)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float x, float y) {  // x in the low half
    if constexpr (std::is_same_v<T, __half>) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
    if constexpr (std::is_same_v<T, __half>) return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v));
}
// Two fp32 -> packed 16-bit pair (x in the low half), and the pair of what the rounding left.
template <typename T>
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack2<T>(x, y);
    const float2 f = unpack2<T>(hi);
    lo = pack2<T>(x - f.x, y - f.y);
}
// Bytes 0 and 2 of t, int8 with their sign bits flipped (bytes 1 and 3 are ignored) -> two
// fp16 values, exact: 0x64 in front of a byte u reads 1024 + u, and u = value + 128.
__device__ __forceinline__ uint32_t widen_u8(uint32_t t) {
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&t), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&d);
}
// 2^x within 2^-22 (below 2^-126: 0); 2^-inf = 0.
__device__ __forceinline__ float pow2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// 1 / x within 2^-23, for normal x
__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Lengths and page ids come from the kernel before this one in the stream, which may still run when this one
// starts: an ordinary load, volatile so that it stays behind the wait (not __ldg, whose data nobody may
// write while the kernel lives).
__device__ __forceinline__ int load_int(const int *p) {
    int v;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

// 16-byte piece c of row r of a tile lies at piece c ^ swizzle(r) of its row, which spreads the
// reads over the banks: 8 rows at one piece (16 bits); in q8, whose pieces move in pairs (32
// values, one group), 8-byte reads of rows r .. r + 3 and 4-byte reads of rows r, r + 2, r + 4,
// r + 6.  swizzle(a + b) = swizzle(a) ^ swizzle(b) where a and b share no bit.
template <int DP, bool Q8>
__host__ __device__ constexpr uint32_t swizzle(uint32_t r) {
    return !Q8 ? r & 7 : DP >= 128 ? ((r & 3) ^ ((r >> 2) & 1)) << 1 : ((r >> 1) & 1) << 1;
}

// Where in the work a reader stands: the unit that begins with key `key` of the keys [lo, len) of
// one item (request b, key head h, block hb of its query heads), and the unit's place, where an
// item takes `cost` places and then one for each unit, counted from the CTA's first.
struct AttnWalk {
    int b, h, hb, key, lo, len, at;
};
// What a CTA has computed of an item that it does not have whole.  An item's pieces lie with the
// CTAs first .. first + n - 1, the first one's in its second slot, the others' in their first.  The
// last CTA to arrive joins them; with many pieces, the last of a group of per_group joins the
// group's over the group's first piece, and the last group's those.
struct AttnPiece {
    int b, h, hb;
    int first, n, per_group;
};

// a / b for 0 <= a, 0 < b: in 32 bits where they do
__device__ __forceinline__ long long div_small(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}
// Adds 1 and returns what was there; writes of this thread, and of those that it has met at a
// barrier, are seen by whoever reads a later value here the same way.
__device__ __forceinline__ unsigned add_acq_rel(unsigned *p) {
    unsigned v;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
    return v;
}

template <typename T, int DP, int NH, int WH, int NW, bool Q8>
__global__ void __launch_bounds__(NW * 32) paged_attn_kernel(const PagedAttnArgs p) {
    using C = AttnCfg<DP, NH, WH, NW, Q8>;
    constexpr int TK = C::TK, KS = C::KS, RW = C::RW, ROWB = C::ROWB, S = C::S, NTH = C::THREADS;
    constexpr int MT = DP / 16;       // 16-wide row tiles of o
    // keys between two looks at the running maximum: 32, but 16 where the registers would not do
    constexpr int SUB = KS < 32 || (DP == 256 && NH == 2) ? 16 : 32;
    using PT = std::conditional_t<Q8, __half, T>;            // operand type of both products
    constexpr float LOWER = !Q8 && std::is_same_v<T, __half> ? kAttnLower : 0.f;  // (q8: see v_top)
    constexpr bool LOW = !Q8 || std::is_same_v<T, __half>;   // weights in two parts (see Numbers above)
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ float st_m[NW][C::HEADS], st_l[NW][C::HEADS];
    __shared__ long long sh_sum[NW], sh_rest;
    __shared__ int sh_b, sh_last;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int wk = warp / WH, hw = warp % WH;
    const int g = lane >> 2, c = lane & 3;
    const uint32_t smem0 = smem_u32(smem);
    const uint32_t q_smem = smem0 + S * C::STAGE, q_slot = p.q_rows * C::QROW;  // the stages' queries
    const int q_own = min(max(p.q_rows - hw * C::HEADS, 0), C::HEADS);           // rows of them that are this warp's
    auto cta_sync = [] {
        if constexpr (NW == 1) __syncwarp();
        else __syncthreads();
    };

    griddep_launch_dependents();
    // The chain lengths -> pages -> keys is three trips to memory: the tables set out for L2 with the
    // lengths (all of them, spread over the grid; L2 is where memory is coherent, so before the wait).
    {
        const int64_t line = static_cast<int64_t>(blockIdx.x) * NTH + tid;
        const int64_t bytes = ((p.batch - 1) * p.table_stride + p.max_pages) * 4;
        if (p.max_pages > 0 && line * 128 < bytes) asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char *>(p.table) + line * 128));
    }
    griddep_wait();

    // ---- this CTA's share ----
    const int cap = p.max_pages * static_cast<int>(p.page.d);  // < 2^31: checked on the host
    auto range_of = [&](int b, int &lo, int &len) {
        const int n = load_int(p.lens + b);
        len = min(max(n, 0), cap);
        lo = p.window > 0 && len > p.window ? len - p.window : 0;
        return n > cap;
    };
    auto units_in = [&](int lo, int len) { return max((len - lo + TK - 1) / TK, 1); };  // (a request without keys has zeros to write)
    // a thread's requests are consecutive: one scan over the threads' sums finds everything
    const int per = (p.batch + NTH - 1) / NTH;
    const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
    long long mine = 0;  // units of this thread's requests, one head
#pragma unroll 4
    for (int b = b0; b < b1; ++b) {
        int lo, len;
        if (range_of(b, lo, len) && blockIdx.x == 0) paged_status(p.status, kSiteLength);
        mine += units_in(lo, len);
    }
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
    }
    if (lane == 31) sh_sum[warp] = inc;
    cta_sync();
    long long U = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (w < warp) inc += sh_sum[w];
        U += sh_sum[w];
    }
    const long long H = static_cast<long long>(p.kv_heads) * p.head_blocks;
    // An item's own cost counts where CTAs have several units; where they have one or two it would only
    // leave some without any.
    const int cost = U * H >= 4ll * gridDim.x ? C::COST : 0;
    const long long V = (U + static_cast<long long>(p.batch) * cost) * H;  // places
    U *= H;                                                                // units
    // CTAs with work: one for a unit while there are few, then two units each, which halves the pieces to
    // join (one request of 4096 tokens and 8 key heads: 11.3 instead of 12.6 us)
    const long long P = U <= 128 ? min(U, static_cast<long long>(gridDim.x)) : min(max(U / 2, 128ll), static_cast<long long>(gridDim.x));
    const long long cta = blockIdx.x;
    if (cta >= P) return;
    const long long v0 = div_small(V * cta, P), v1 = div_small(V * (cta + 1), P);
    // The CTA i with place v, floor(V i / P) <= v < floor(V (i + 1) / P): V i < (v + 1) P <= V (i + 1).  In
    // floats, with P < 2^12, the guess is off by one at most.
    const float per_place = static_cast<float>(P) / static_cast<float>(V);
    auto cta_of = [&](long long v) {
        int i = static_cast<int>(static_cast<float>(v + 1) * per_place);
        if (V * i >= (v + 1) * P) --i;
        else if (V * (i + 1) < (v + 1) * P) ++i;
        return i;
    };
    long long at = (inc - mine + static_cast<long long>(b0) * cost) * H;
    if (v0 >= at && v0 < (inc + static_cast<long long>(b1) * cost) * H) {  // place v0 is in one of this thread's requests
        int b = b0;
        for (; b < b1; ++b) {
            int lo, len;
            range_of(b, lo, len);
            const long long n = static_cast<long long>(units_in(lo, len) + cost) * H;
            if (v0 < at + n) break;
            at += n;
        }
        sh_b = b;
        sh_rest = v0 - at;
    }
    cta_sync();
    const int places = static_cast<int>(v1 - v0);
    auto advance = [&](AttnWalk &w) {
        ++w.at;
        w.key += TK;
        if (w.key >= w.len) {
            w.at += cost;
            if (++w.hb == p.head_blocks) {
                w.hb = 0;
                if (++w.h == p.kv_heads) {
                    w.h = 0;
                    if (++w.b < p.batch) range_of(w.b, w.lo, w.len);
                }
            }
            w.key = w.lo;
        }
    };
    AttnWalk pw;  // the loads' place
    pw.b = sh_b;
    const int *pw_pages = p.table + pw.b * p.table_stride;  // its request's pages
    range_of(pw.b, pw.lo, pw.len);
    {
        const int n = units_in(pw.lo, pw.len) + cost, item = static_cast<int>(div_small(sh_rest, n));
        const int at = static_cast<int>(sh_rest - static_cast<long long>(item) * n), j = max(at - cost, 0);
        pw.h = item / p.head_blocks;
        pw.hb = item - pw.h * p.head_blocks;
        pw.key = pw.lo + j * TK;
        pw.at = j + cost - at;
    }
    if (pw.at >= places) return;  // a share without units
    AttnWalk cw = pw;             // the products' place

    // ---- loads: lane r < RW describes row warp * RW + r of the unit ----
    int pg_id = -1, pg_off = 0;
    bool pg_ok = false;
    auto load_next = [&] {  // the loads' place moves on
        const int b = pw.b;
        advance(pw);
        if (pw.b != b) pw_pages += p.table_stride;
    };
    auto look_up = [&] {
        const int key = pw.key + warp * RW + lane;
        pg_ok = lane < RW && key < pw.len;
        if (pg_ok) {
            const int pi = static_cast<int>(p.page.div(key));
            pg_off = key - pi * static_cast<int>(p.page.d);
            pg_id = load_int(pw_pages + pi);
        }
    };
    const int pieces = p.head_dim * (Q8 ? 1 : 2) / 16;  // 16-byte pieces of a row that exist
    bool first_unit_of_cta = true;
    auto issue = [&](int stage) {
        const uint32_t lost = __ballot_sync(0xffffffffu, pg_ok && static_cast<uint32_t>(pg_id) >= static_cast<uint32_t>(p.num_pages));
        if (__builtin_expect(lost != 0, 0)) {
            paged_status(p.status, kSitePage);
            if (lost >> lane & 1) pg_ok = false;
        }
        constexpr int CPR = ROWB / 16, RPI = 32 / CPR;  // pieces per row, rows per instruction
        const int cc = lane % CPR, rr = lane / CPR;
        const uint32_t dst = smem0 + stage * C::STAGE + (warp * RW + rr) * ROWB + ((cc ^ swizzle<DP, Q8>(rr)) << 4);
        // (r, a multiple of RPI known at compile time, shares no bit with rr; rows start at multiples of ROWB)
        auto place = [&](int r) { return (dst ^ (swizzle<DP, Q8>(r) << 4)) + r * ROWB; };
        if (p.whole_pages) {
            // 16 rows at a time lie in one page, token after token: one address and steps from it.  (A row
            // past the range has zeros copied, but its address is still one of the page, or of page 0.)
#pragma unroll
            for (int r0 = 0; r0 < RW; r0 += 16) {
                const int id = __shfl_sync(0xffffffffu, pg_ok ? pg_id : -1, r0), off = __shfl_sync(0xffffffffu, pg_off, r0);
                const int have = id >= 0 && cc < pieces ? pw.len - (pw.key + warp * RW + r0) - rr : 0;
                const int col = cc < pieces ? cc * 16 : 0;
                const char *ka = p.k.at(max(id, 0), id >= 0 ? off + rr : rr, pw.h) + col;
                const char *va = p.v.at(max(id, 0), id >= 0 ? off + rr : rr, pw.h) + col;
                const int k_step = static_cast<int>(p.k.token) * 16, v_step = static_cast<int>(p.v.token) * 16;
#pragma unroll
                for (int it = 0; it < 16 / RPI; ++it) {
                    const uint32_t to = place(r0 + it * RPI);
                    const int n = it * RPI < have ? 16 : 0;
                    cp_async16(to, ka + static_cast<int64_t>(k_step) * (it * RPI), n);
                    cp_async16(to + TK * ROWB, va + static_cast<int64_t>(v_step) * (it * RPI), n);
                }
            }
        } else {
            const int64_t ko = pg_ok ? p.k.at(pg_id, pg_off, pw.h) - p.k.base : -1;
            const int64_t vo = pg_ok ? p.v.at(pg_id, pg_off, pw.h) - p.v.base : -1;
#pragma unroll
            for (int it = 0; it < RW / RPI; ++it) {
                const int r = it * RPI + rr;
                const int64_t ka = __shfl_sync(0xffffffffu, ko, r), va = __shfl_sync(0xffffffffu, vo, r);
                const uint32_t to = place(it * RPI);
                const int n = ka >= 0 && cc < pieces ? 16 : 0;
                cp_async16(to, n ? p.k.base + ka + cc * 16 : p.k.base, n);
                cp_async16(to + TK * ROWB, n ? p.v.base + va + cc * 16 : p.v.base, n);
            }
        }
        if constexpr (Q8) {
            if (lane < RW) {
                const uint32_t sdst = smem0 + stage * C::STAGE + 2 * TK * ROWB + (warp * RW + lane) * C::SCB;
                const char *ks = pg_ok ? p.ks.at(pg_id, pg_off, pw.h) : p.ks.base;
                const char *vs = pg_ok ? p.vs.at(pg_id, pg_off, pw.h) : p.vs.base;
                if constexpr (DP == 128) {  // four scales, aligned to their size
                    cp_async8(sdst, ks, pg_ok ? 8 : 0);
                    cp_async8(sdst + TK * C::SCB, vs, pg_ok ? 8 : 0);
                } else {
#pragma unroll
                    for (int i = 0; i < DP / 64; ++i) {
                        const int n = pg_ok && i * 64 < p.head_dim ? 4 : 0;
                        cp_async4(sdst + i * 4, ks + (n ? i * 4 : 0), n);
                        cp_async4(sdst + TK * C::SCB + i * 4, vs + (n ? i * 4 : 0), n);
                    }
                }
            }
        }
        if (__builtin_expect(lost != 0, 0)) {
            // a key of a page that does not exist scores NaN, and so does its request: zeros would be a key that
            // looks like any other.  (After the zeros that were copied to its row.)
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
            const uint32_t row = smem0 + stage * C::STAGE + (Q8 ? 2 * TK * ROWB + (warp * RW + lane) * C::SCB : (warp * RW + lane) * ROWB);
            if (lost >> lane & 1) asm volatile("st.shared.b32 [%0], %1;" ::"r"(row), "r"(0x7fff7fffu) : "memory");  // (NaN in fp16 and bf16)
        }
        if (pw.key == pw.lo || first_unit_of_cta) {  // the item's queries
            first_unit_of_cta = false;
            const int h0 = pw.hb * C::ROWS + hw * C::HEADS;
            const char *q = p.q + pw.b * p.q_batch + static_cast<int64_t>(pw.h * p.group + h0) * p.q_head;
            constexpr int QP = DP / 8;  // 16-byte pieces of a padded row
            for (int e = wk * 32 + lane; e < q_own * QP; e += C::WK * 32) {
                const int r = e / QP, x = e % QP;
                const int n = h0 + r < p.group && x * 8 < p.head_dim ? 16 : 0;
                cp_async16(q_smem + stage * q_slot + (hw * C::HEADS + r) * C::QROW + ((x ^ (r & 7)) << 4),
                           n ? q + r * p.q_head + x * 16 : p.q, n);
            }
        }
    };
    auto group_sync = [&] {
        if constexpr (WH == 1) __syncwarp();
        else if constexpr (WH == NW) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + wk), "n"(WH * 32) : "memory");
    };

    // ---- per item state: tile t of o holds value columns 16 t + {g, g + 8}, query heads 2c, 2c + 1 ----
    uint32_t qf[MT][NH][2];
    float o[MT][NH][4];
    float m[NH][2], l[NH][2];  // running reference and this thread's part of the sum, heads 2c, 2c + 1
    float q_unit[NH][2];       // q8: what one unit of a head's staged query stands for
    // q8: the largest value scale so far of each group of 32 columns, its fp16 exponent field in place, two
    // groups a word.  With e that field's number (scales < 2^(e - 14)) o holds sum w v 2^(21 - e), so that a
    // weight (at most 2^kAttnSlack) times a scale stays below 2^15 and keeps 2^-31 of the group's largest.
    uint32_t v_top[Q8 ? DP / 64 : 1];
    static_assert(kAttnSlack + 7 == 15, "2^kAttnSlack 2^(e - 14) 2^(21 - e) must lie in fp16's range");
    auto v_top_of = [&](int gr) { return gr & 1 ? v_top[gr >> 1] >> 16 : v_top[gr >> 1] & 0xffffu; };  // e << 10
    auto v_up = [&](int gr) { return __uint_as_float(((127u + 21u) << 23) - (v_top_of(gr) << 13)); };     // 2^(21 - e)
    auto load_q = [&](int stage) {
#pragma unroll
        for (int nt = 0; nt < NH; ++nt) {
            const int r = nt * 8 + g;
            const bool ok = r < q_own;
            const uint32_t row = q_smem + stage * q_slot + (hw * C::HEADS + r) * C::QROW;
#pragma unroll
            for (int kk = 0; kk < MT; ++kk) {
                // this thread's two pairs of columns (any order of d does, the keys' operand has the same)
                if constexpr (!Q8) {
                    qf[kk][nt][0] = ok ? lds32(row + (((2 * kk) ^ g) << 4) + c * 4) : 0u;
                    qf[kk][nt][1] = ok ? lds32(row + (((2 * kk + 1) ^ g) << 4) + c * 4) : 0u;
                } else {  // 8 values of a group are two k-steps' share
                    const uint2 x = ok ? lds64(row + ((((kk >> 1) * 4 + c) ^ g) << 4) + (kk & 1) * 8) : make_uint2(0, 0);
                    qf[kk][nt][0] = x.x;
                    qf[kk][nt][1] = x.y;
                }
            }
            if constexpr (Q8 && !std::is_same_v<T, __half>) {
                // bf16 queries as fp16: scaled by a power of two so that the head's largest lies in [1, 2);
                // what falls below fp16's range is 2^-24 of it
                float top = 0.f;
#pragma unroll
                for (int kk = 0; kk < MT; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 f = unpack2<T>(qf[kk][nt][i]);
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // exponent field of the largest, kept where its inverse is a normal number too
                const uint32_t ex = min(max(__float_as_uint(top) >> 23, 1u), 252u);
                const float down = __uint_as_float((254u - ex) << 23), up = __uint_as_float(ex << 23);
#pragma unroll
                for (int kk = 0; kk < MT; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 f = unpack2<T>(qf[kk][nt][i]);
                        qf[kk][nt][i] = pack2<__half>(f.x * down, f.y * down);
                    }
                q_unit[nt][0] = __shfl_sync(0xffffffffu, up, 8 * c);      // heads 2c and 2c + 1 lie in lane groups
                q_unit[nt][1] = __shfl_sync(0xffffffffu, up, 8 * c + 4);  // 2c and 2c + 1
            } else {
                q_unit[nt][0] = q_unit[nt][1] = 1.f;
            }
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int t = 0; t < MT; ++t) o[t][nt][0] = o[t][nt][1] = o[t][nt][2] = o[t][nt][3] = 0.f;
        }
        if constexpr (Q8) {
#pragma unroll
            for (int x = 0; x < DP / 64; ++x) v_top[x] = 0;
        }
    };

    // ---- prologue: S - 1 units in flight, the page ids of the next ----
    look_up();
#pragma unroll
    for (int s = 0; s < S - 1; ++s) {
        if (pw.at < places) {
            issue(s);
            load_next();
            if (pw.at < places) look_up();
        }
        cp_async_commit();
    }

    // ---- an item's end ----
    auto heads_of = [&](int hb) { return min(p.group - hb * C::ROWS, C::ROWS); };  // query heads of the block
    auto store = [&](int b, int h, int hb, int r, int col, const float4 &v, float M, float L) {
        const int head = h * p.group + hb * C::ROWS + r;
        const float inv = L > 0.f ? reciprocal(L) : L == 0.f ? 0.f : L;  // no key: zeros; a NaN sum stays NaN
        if (col < p.head_dim)
            *reinterpret_cast<uint2 *>(p.out + b * p.o_batch + static_cast<int64_t>(head) * p.o_head + col * 2) =
                make_uint2(pack2<T>(v.x * inv, v.y * inv), pack2<T>(v.z * inv, v.w * inv));
        if (p.lse && col == 0)
            p.lse[static_cast<int64_t>(b) * p.kv_heads * p.group + head] = L == 0.f ? -INFINITY : M * 0.6931471805599453f + logf(L);
    };
    // The item of the walk: n units, the first at place `at`.
    auto piece_of = [&](const AttnWalk &w, int at, int n) {
        AttnPiece i;
        i.b = w.b;
        i.h = w.h;
        i.hb = w.hb;
        i.first = cta_of(v0 + at);
        i.n = cta_of(v0 + at + n - 1) - i.first + 1;
        i.per_group = i.n;
        if (i.n > 16 && i.n * heads_of(w.hb) > kAttnFlat) {
            i.per_group = 16;
            while (i.per_group * i.per_group < i.n) i.per_group += 4;
        }
        return i;
    };
    // The counter of this CTA's group.  An item's first group counts at its first CTA, the others at
    // theirs in a field of their own, where no other item has a group that is not its first; a second
    // level counts in a third field.
    auto counter_of = [&](const AttnPiece &i) {
        const int at = static_cast<int>(cta) - i.first;
        return p.counters + (at < i.per_group ? i.first : static_cast<int>(gridDim.x) + i.first + at / i.per_group * i.per_group);
    };
    // Joins `count` pieces i0, i0 + step, ... of the item, to the output or over piece i0.  The ring is
    // free by now: EB float4 of o per thread and piece come through it, as many pieces at once as it
    // holds, so that a join costs a trip to L2 or two and not one per few pieces.  (EB is as small as the
    // rows allow: few warps run here, and instructions that do nothing cost as much as others.  CTAs of one
    // warp have the largest alone: with all three, 256 requests of 1 to 500 tokens, 16 heads of 64, took 23.9
    // us for 23.0, and of 500 to 4000 tokens 294 for 291.)
    auto join_wide = [&](auto eb, const AttnPiece &item, int i0, int step, int count, bool final) {
        constexpr int EB = decltype(eb)::value, BLOCK = EB * NTH;  // float4 of o at a time
        constexpr int HELD = BLOCK * 16 + 2 * C::ROWS * 4;  // bytes of a piece in the ring: o, m, l
        constexpr int AT_ONCE = S * C::STAGE / HELD;
        static_assert(AT_ONCE >= 2, "a join makes progress");
        const float *base = p.partials + static_cast<size_t>(2 * item.first) * C::SLOT;
        auto at = [&](int i) { return base + static_cast<size_t>(i == 0 ? 1 : 2 * i) * C::SLOT; };
        const int all = heads_of(item.hb) * (DP / 4);
        for (int e0 = 0; e0 < all; e0 += BLOCK) {
            const int block = min(BLOCK, all - e0);
            float M[EB], L[EB];
            float4 acc[EB];
#pragma unroll
            for (int x = 0; x < EB; ++x) {
                M[x] = -INFINITY;
                L[x] = 0.f;
                acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            for (int c0 = 0; c0 < count; c0 += AT_ONCE) {
                const int n = min(AT_ONCE, count - c0);
                for (int i = 0; i < n; ++i) {
                    const float *src = at(i0 + (c0 + i) * step);
                    const uint32_t dst = smem0 + i * HELD;
#pragma unroll
                    for (int x = 0; x < EB; ++x)
                        if (x * NTH + tid < block) cp_async16(dst + (x * NTH + tid) * 16, src + (e0 + x * NTH + tid) * 4, 16);
                    for (int x = tid; x < C::ROWS / 2; x += NTH) cp_async16(dst + BLOCK * 16 + x * 16, src + C::ROWS * DP + x * 4, 16);
                }
                cp_async_commit();
                cp_async_wait<0>();
                cta_sync();
#pragma unroll
                for (int x = 0; x < EB; ++x) {
                    const int e = x * NTH + tid, r = (e0 + e) / (DP / 4);
                    if (e >= block) break;
                    auto held = [&](int i) { return reinterpret_cast<const float *>(smem + i * HELD); };
                    float top = M[x];
#pragma unroll 4
                    for (int i = 0; i < n; ++i) top = fmaxf(top, held(i)[BLOCK * 4 + r]);
                    const float f = M[x] == top ? 1.f : pow2(M[x] - top);
                    M[x] = top;
                    L[x] *= f;
                    acc[x].x *= f;
                    acc[x].y *= f;
                    acc[x].z *= f;
                    acc[x].w *= f;
#pragma unroll 4
                    for (int i = 0; i < n; ++i) {
                        const float mi = held(i)[BLOCK * 4 + r];
                        const float w = mi == top ? 1.f : pow2(mi - top);  // (both -inf: zeros either way)
                        const float4 v = *reinterpret_cast<const float4 *>(held(i) + e * 4);
                        L[x] += held(i)[BLOCK * 4 + C::ROWS + r] * w;
                        acc[x].x += v.x * w;
                        acc[x].y += v.y * w;
                        acc[x].z += v.z * w;
                        acc[x].w += v.w * w;
                    }
                }
                cta_sync();
            }
#pragma unroll
            for (int x = 0; x < EB; ++x) {
                const int e = e0 + x * NTH + tid, r = e / (DP / 4), col = (e % (DP / 4)) * 4;
                if (e >= e0 + block) break;
                if (final) {
                    store(item.b, item.h, item.hb, r, col, acc[x], M[x], L[x]);
                } else {  // (the piece's own m and l are still read for the next block: they change at the end)
                    *reinterpret_cast<float4 *>(const_cast<float *>(at(i0)) + e * 4) = acc[x];
                    if (col == 0) {
                        st_m[r / C::HEADS][r % C::HEADS] = M[x];
                        st_l[r / C::HEADS][r % C::HEADS] = L[x];
                    }
                }
            }
        }
        if (!final) {
            cta_sync();
            for (int r = tid; r < heads_of(item.hb); r += NTH) {
                const_cast<float *>(at(i0))[C::ROWS * DP + r] = st_m[r / C::HEADS][r % C::HEADS];
                const_cast<float *>(at(i0))[C::ROWS * (DP + 1) + r] = st_l[r / C::HEADS][r % C::HEADS];
            }
            cta_sync();
        }
    };

    auto join = [&](const AttnPiece &item, int i0, int step, int count, bool final) {
        const int all = heads_of(item.hb) * (DP / 4);
        if (all * 2 <= NTH && final) {
            // few float4: groups of threads take every so many-th piece, straight from L2, and meet at the end
            const int groups = NTH / all, mine = tid / all, e = tid - mine * all, r = e / (DP / 4);
            float M = -INFINITY, L = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            if (mine < groups)
#pragma unroll 4
                for (int i = mine; i < count; i += groups) {
                    const int y = i0 + i * step;
                    const float *src = p.partials + static_cast<size_t>(2 * item.first + (y == 0 ? 1 : 2 * y)) * C::SLOT;
                    const float mi = __ldcg(src + C::ROWS * DP + r), li = __ldcg(src + C::ROWS * (DP + 1) + r);
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(src + e * 4));
                    const float top = fmaxf(M, mi);
                    const float f = M == top ? 1.f : pow2(M - top), w = mi == top ? 1.f : pow2(mi - top);  // (both -inf: zeros either way)
                    M = top;
                    L = L * f + li * w;
                    acc = make_float4(acc.x * f + v.x * w, acc.y * f + v.y * w, acc.z * f + v.z * w, acc.w * f + v.w * w);
                }
            float4 *o4 = reinterpret_cast<float4 *>(smem);
            float2 *ml = reinterpret_cast<float2 *>(smem + NTH * 16);
            o4[tid] = acc;
            ml[tid] = make_float2(M, L);
            cta_sync();
            if (mine == 0) {
#pragma unroll 1
                for (int i = 1; i < groups; ++i) {
                    const float2 y = ml[i * all + e];
                    const float4 v = o4[i * all + e];
                    const float top = fmaxf(M, y.x);
                    const float f = M == top ? 1.f : pow2(M - top), w = y.x == top ? 1.f : pow2(y.x - top);
                    M = top;
                    L = L * f + y.y * w;
                    acc = make_float4(acc.x * f + v.x * w, acc.y * f + v.y * w, acc.z * f + v.z * w, acc.w * f + v.w * w);
                }
                store(item.b, item.h, item.hb, r, (e % (DP / 4)) * 4, acc, M, L);
            }
            cta_sync();
        } else if (NW > 1 && all <= NTH) {
            join_wide(std::integral_constant<int, 1>{}, item, i0, step, count, final);
        } else if (NW > 1 && all <= 2 * NTH) {
            join_wide(std::integral_constant<int, 2>{}, item, i0, step, count, final);
        } else {
            join_wide(std::integral_constant<int, 4>{}, item, i0, step, count, final);
        }
    };

    int stage = 0;
    bool fresh = true;
    // Pieces that this CTA shares with others: of the item that its share begins inside, and of the one
    // that it ends inside.  Whether they are complete is asked at the end, when the answer has come.
    AttnPiece begun{}, left_open{};
    unsigned begun_ticket = 0, left_ticket = 0;  // thread 0's
    bool has_begun = false, has_left = false;
    int item_at = 0, item_n = 0;  // place and number of the item's units
    while (cw.at < places) {
        if (fresh) {  // (while the unit is on its way)
            item_n = units_in(cw.lo, cw.len);
            item_at = cw.at - (cw.key - cw.lo) / TK;
            if (item_at < 0) {
                has_begun = true;
                begun = piece_of(cw, item_at, item_n);
            } else if (item_at + item_n > places) {
                has_left = true;
                left_open = piece_of(cw, item_at, item_n);
            }
        }
        cp_async_wait<S - 2>();
        group_sync();
        {
            const int st = stage == 0 ? S - 1 : stage - 1;  // consumed in the previous round
            if (pw.at < places) {
                issue(st);
                load_next();
                if (pw.at < places) look_up();
            }
            cp_async_commit();
        }
        if (fresh) {
            if constexpr (C::WK > 1) __syncthreads();  // the groups load shares of the queries
            load_q(stage);
            if constexpr (NW > 1) __syncthreads();     // ... and may load others over them
            else __syncwarp();
            fresh = false;
        }
        const uint32_t kt = smem0 + stage * C::STAGE + wk * KS * ROWB, vt = kt + TK * ROWB;
        const uint32_t kst = smem0 + stage * C::STAGE + 2 * TK * ROWB + wk * KS * C::SCB, vst = kst + TK * C::SCB;
        const int left = cw.len - (cw.key + wk * KS);  // valid keys from this group's first on
#pragma unroll 1
        for (int k0 = 0; k0 < KS; k0 += SUB) {
            if (k0 >= left) break;
            constexpr int KT = SUB / 16;  // 16-key tiles: keys 16 kt + g and + 8 are this thread's
            float s[KT][NH][4];
            // scores: SUB keys x 8 NH query heads
            if constexpr (!Q8) {
#pragma unroll
                for (int i = 0; i < KT; ++i)
#pragma unroll
                    for (int nt = 0; nt < NH; ++nt) s[i][nt][0] = s[i][nt][1] = s[i][nt][2] = s[i][nt][3] = 0.f;
                // (rows start at multiples of ROWB: the piece is bits of the address alone)
                const uint32_t row = kt + (k0 + (lane & 15)) * ROWB + (((lane >> 4) ^ (lane & 7)) << 4);
#pragma unroll
                for (int kk = 0; kk < MT; ++kk)
#pragma unroll
                    for (int i = 0; i < KT; ++i) {
                        uint32_t a[4];
                        ldsm_x4((row ^ (kk << 5)) + i * 16 * ROWB, a);
#pragma unroll
                        for (int nt = 0; nt < NH; ++nt) mma16816<PT>(s[i][nt], a, qf[kk][nt][0], qf[kk][nt][1], s[i][nt]);
                    }
            } else {
                const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                const uint32_t row = kt + (k0 + g) * ROWB + ((c >> 1) ^ swizzle<DP, true>(g)) * 16 + (c & 1) * 8;
                const uint32_t row_sc = kst + (k0 + g) * C::SCB;
#pragma unroll
                for (int i = 0; i < KT; ++i) {
                    float2 sc0[DP / 64], sc1[DP / 64];  // the scales of this thread's two keys, 8 apart
#pragma unroll
                    for (int x = 0; x < DP / 64; ++x) {
                        sc0[x] = unpack2<__half>(lds32(row_sc + i * 16 * C::SCB + x * 4));
                        sc1[x] = unpack2<__half>(lds32(row_sc + (i * 16 + 8) * C::SCB + x * 4));
                    }
#pragma unroll
                    for (int gr = 0; gr < DP / 32; ++gr) {
                        uint2 w0 = lds64((row ^ (gr << 5)) + i * 16 * ROWB);
                        uint2 w1 = lds64((row ^ (gr << 5)) + (i * 16 + 8) * ROWB);
                        w0.x ^= 0x80808080u;
                        w0.y ^= 0x80808080u;
                        w1.x ^= 0x80808080u;
                        w1.y ^= 0x80808080u;
                        const uint32_t front = 0x64646464u;
                        const uint32_t a0[4] = {widen_u8(__byte_perm(w0.x, front, 0x4140)), widen_u8(__byte_perm(w1.x, front, 0x4140)),
                                                widen_u8(__byte_perm(w0.x, front, 0x4342)), widen_u8(__byte_perm(w1.x, front, 0x4342))};
                        const uint32_t a1[4] = {widen_u8(__byte_perm(w0.y, front, 0x4140)), widen_u8(__byte_perm(w1.y, front, 0x4140)),
                                                widen_u8(__byte_perm(w0.y, front, 0x4342)), widen_u8(__byte_perm(w1.y, front, 0x4342))};
                        const float f0 = gr & 1 ? sc0[gr >> 1].y : sc0[gr >> 1].x, f1 = gr & 1 ? sc1[gr >> 1].y : sc1[gr >> 1].x;
#pragma unroll
                        for (int nt = 0; nt < NH; ++nt) {
                            float t[4];
                            mma16816<PT>(t, a0, qf[2 * gr][nt][0], qf[2 * gr][nt][1], zero);
                            mma16816<PT>(t, a1, qf[2 * gr + 1][nt][0], qf[2 * gr + 1][nt][1], t);
                            s[i][nt][0] = gr ? s[i][nt][0] + t[0] * f0 : t[0] * f0;
                            s[i][nt][1] = gr ? s[i][nt][1] + t[1] * f0 : t[1] * f0;
                            s[i][nt][2] = gr ? s[i][nt][2] + t[2] * f1 : t[2] * f1;
                            s[i][nt][3] = gr ? s[i][nt][3] + t[3] * f1 : t[3] * f1;
                        }
                    }
                }
            }
            // scaled scores; keys past the range drop out; the largest of this thread's
            bool past = false;
            float x[NH][2];
#pragma unroll
            for (int nt = 0; nt < NH; ++nt) {
                const float sc0 = Q8 ? p.scale_log2 * q_unit[nt][0] : p.scale_log2, sc1 = Q8 ? p.scale_log2 * q_unit[nt][1] : p.scale_log2;
                x[nt][0] = x[nt][1] = -INFINITY;
#pragma unroll
                for (int i = 0; i < KT; ++i) {
                    s[i][nt][0] *= sc0;
                    s[i][nt][1] *= sc1;
                    s[i][nt][2] *= sc0;
                    s[i][nt][3] *= sc1;
                    if (k0 + SUB > left) {
                        const int n = k0 + i * 16 + g;
                        if (n >= left) s[i][nt][0] = s[i][nt][1] = -INFINITY;
                        if (n + 8 >= left) s[i][nt][2] = s[i][nt][3] = -INFINITY;
                    }
                    x[nt][0] = fmaxf(x[nt][0], fmaxf(s[i][nt][0], s[i][nt][2]));
                    x[nt][1] = fmaxf(x[nt][1], fmaxf(s[i][nt][1], s[i][nt][3]));
                }
                past = past || x[nt][0] > m[nt][0] + (kAttnSlack + LOWER) || x[nt][1] > m[nt][1] + (kAttnSlack + LOWER);
            }
            if (__any_sync(0xffffffffu, past)) {  // the reference moves to LOWER below the largest score so far
#pragma unroll
                for (int nt = 0; nt < NH; ++nt) {
                    float a[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float y = x[nt][i];
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
                        y = fmaxf(y - LOWER, m[nt][i]);
                        a[i] = y == m[nt][i] ? 1.f : pow2(m[nt][i] - y);
                        m[nt][i] = y;
                        l[nt][i] *= a[i];
                    }
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        o[t][nt][0] *= a[0];
                        o[t][nt][1] *= a[1];
                        o[t][nt][2] *= a[0];
                        o[t][nt][3] *= a[1];
                    }
                }
            }
            // weights (a head that has seen only -inf keeps its weights at zero)
#pragma unroll
            for (int nt = 0; nt < NH; ++nt) {
                const float e0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], e1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
                for (int i = 0; i < KT; ++i) {
                    s[i][nt][0] = pow2(s[i][nt][0] - e0);
                    s[i][nt][1] = pow2(s[i][nt][1] - e1);
                    s[i][nt][2] = pow2(s[i][nt][2] - e0);
                    s[i][nt][3] = pow2(s[i][nt][3] - e1);
                    l[nt][0] += s[i][nt][0] + s[i][nt][2];
                    l[nt][1] += s[i][nt][1] + s[i][nt][3];
                }
            }
            // o += values . weights
            if constexpr (!Q8) {
#pragma unroll
                for (int i = 0; i < KT; ++i) {
                    uint32_t hi[NH][2], lo[NH][2];
#pragma unroll
                    for (int nt = 0; nt < NH; ++nt)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            split2<PT>(s[i][nt][2 * y], s[i][nt][2 * y + 1], hi[nt][y], lo[nt][y]);
                            hi[nt][y] = transpose8x8(hi[nt][y]);
                            lo[nt][y] = transpose8x8(lo[nt][y]);
                        }
                    // values stored key by key: transposed on the way into registers
                    const uint32_t row = vt + (k0 + (lane & 7) + ((lane >> 4) << 3)) * ROWB + ((((lane >> 3) & 1) ^ (lane & 7)) << 4);
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        uint32_t a[4];
                        ldsm_x4_t((row ^ (t << 5)) + i * 16 * ROWB, a);
#pragma unroll
                        for (int nt = 0; nt < NH; ++nt) {
                            mma16816<PT>(o[t][nt], a, hi[nt][0], hi[nt][1], o[t][nt]);
                            mma16816<PT>(o[t][nt], a, lo[nt][0], lo[nt][1], o[t][nt]);
                        }
                    }
                }
            } else {
                // this thread's keys in the values: 2c, 2c + 1 and 8 further on
                const uint32_t v_row[2] = {vt + (k0 + 2 * c) * ROWB + ((g >> 2) ^ swizzle<DP, true>(2 * c)) * 16 + (g & 3) * 4,
                                           vt + (k0 + 2 * c + 1) * ROWB + ((g >> 2) ^ swizzle<DP, true>(2 * c + 1)) * 16 + (g & 3) * 4};
                // this block's value scales, and whether one has a larger exponent than its group's so far
                uint32_t xs[KT][2][DP / 64], top[DP / 64];
                bool grows = false;
#pragma unroll
                for (int x = 0; x < DP / 64; ++x) {
                    top[x] = v_top[x];
#pragma unroll
                    for (int i = 0; i < KT; ++i)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            xs[i][y][x] = lds32(vst + (k0 + g) * C::SCB + (i * 16 + 8 * y) * C::SCB + x * 4);
                            top[x] = __vmaxu2(top[x], xs[i][y][x] & 0x7c007c00u);
                        }
                    grows = grows || top[x] != v_top[x];
                }
                if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                    for (int gr = 0; gr < DP / 32; ++gr) {
                        const uint32_t was = v_top_of(gr), mine = gr & 1 ? top[gr >> 1] >> 16 : top[gr >> 1] & 0xffffu;
                        const uint32_t now = __reduce_max_sync(0xffffffffu, mine);
                        const float f = __uint_as_float((127u << 23) - ((now - was) << 13));
#pragma unroll
                        for (int t = 2 * gr; t < 2 * gr + 2; ++t)  // (a group's columns are two tiles of o)
#pragma unroll
                            for (int nt = 0; nt < NH; ++nt)
#pragma unroll
                                for (int y = 0; y < 4; ++y) o[t][nt][y] *= f;
                        v_top[gr >> 1] = gr & 1 ? (v_top[gr >> 1] & 0xffffu) | now << 16 : (v_top[gr >> 1] & 0xffff0000u) | now;
                    }
                }
#pragma unroll
                for (int i = 0; i < KT; ++i) {
#pragma unroll
                    for (int gr = 0; gr < DP / 32; ++gr) {
                        uint32_t w[4];
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            w[t] = lds32((v_row[t & 1] ^ (gr << 5)) + (i * 16 + (t >> 1) * 8) * ROWB) ^ 0x80808080u;
                        }
                        const float2 y0 = unpack2<__half>(xs[i][0][gr >> 1]), y1 = unpack2<__half>(xs[i][1][gr >> 1]);
                        const float f0 = (gr & 1 ? y0.y : y0.x) * v_up(gr), f1 = (gr & 1 ? y1.y : y1.x) * v_up(gr);
                        uint32_t hi[NH][2], lo[NH][2];
#pragma unroll
                        for (int nt = 0; nt < NH; ++nt)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const float wx = s[i][nt][2 * y] * (y ? f1 : f0), wy = s[i][nt][2 * y + 1] * (y ? f1 : f0);
                                if constexpr (LOW) {
                                    split2<PT>(wx, wy, hi[nt][y], lo[nt][y]);
                                    lo[nt][y] = transpose8x8(lo[nt][y]);
                                } else {
                                    hi[nt][y] = pack2<PT>(wx, wy);
                                }
                                hi[nt][y] = transpose8x8(hi[nt][y]);
                            }
#pragma unroll
                        for (int t = 0; t < 2; ++t) {  // rows g and g + 8 of the tile: values 4 g + 2 t and + 1 of the group
                            uint32_t a[4];
#pragma unroll
                            for (int y = 0; y < 2; ++y) {  // bytes 2 t and 2 t + 1 of two neighbouring keys, interleaved
                                const uint32_t x = __byte_perm(w[2 * y], w[2 * y + 1], t ? 0x7362 : 0x5140);
                                a[2 * y] = widen_u8(__byte_perm(x, 0x64646464u, 0x4140));
                                a[2 * y + 1] = widen_u8(__byte_perm(x, 0x64646464u, 0x4342));
                            }
#pragma unroll
                            for (int nt = 0; nt < NH; ++nt) {
                                mma16816<PT>(o[2 * gr + t][nt], a, hi[nt][0], hi[nt][1], o[2 * gr + t][nt]);
                                if constexpr (LOW) mma16816<PT>(o[2 * gr + t][nt], a, lo[nt][0], lo[nt][1], o[2 * gr + t][nt]);
                            }
                        }
                    }
                }
            }
        }

        if (cw.key + TK >= cw.len || cw.at == places - 1) {
            // ---- the CTA's piece of the item: join the warps through the stage just read ----
#pragma unroll
            for (int nt = 0; nt < NH; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 4);
                    l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 8);
                    l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 16);
                }
            const bool begun_here = item_at >= 0, whole = begun_here && item_at + item_n <= places;
            cta_sync();  // every warp has read the stage
            float *ob = reinterpret_cast<float *>(smem + stage * C::STAGE);
            const int valid = heads_of(cw.hb);
#pragma unroll
            for (int nt = 0; nt < NH; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = nt * 8 + 2 * c + i;
                    if (g == 0) {
                        st_m[warp][r] = m[nt][i];
                        st_l[warp][r] = l[nt][i];
                    }
                    if (hw * C::HEADS + r >= valid) continue;
                    float *row = ob + (warp * C::HEADS + r) * DP;
                    const int sw = c << 3;  // 32-byte pieces of a row swapped by head: no bank conflicts
                    if constexpr (!Q8) {
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            row[(t * 16 + g) ^ sw] = o[t][nt][i];
                            row[(t * 16 + g + 8) ^ sw] = o[t][nt][2 + i];
                        }
                    } else {
#pragma unroll
                        for (int gr = 0; gr < DP / 32; ++gr) {
                            const float back = __uint_as_float(((127u - 21u) << 23) + (v_top_of(gr) << 13));  // 2^(e - 21)
                            *reinterpret_cast<float4 *>(row + ((gr * 32 + g * 4) ^ sw)) =
                                make_float4(o[2 * gr][nt][i] * back, o[2 * gr][nt][2 + i] * back, o[2 * gr + 1][nt][i] * back,
                                            o[2 * gr + 1][nt][2 + i] * back);
                        }
                    }
                }
            cta_sync();

            float *slot = p.partials + static_cast<size_t>(2 * cta + (begun_here ? 1 : 0)) * C::SLOT;
            for (int e = tid; e < valid * (DP / 4); e += NTH) {
                const int r = e / (DP / 4), col = (e % (DP / 4)) * 4, rw = r / C::HEADS, rr = r % C::HEADS;
                float M = st_m[rw][rr];
#pragma unroll
                for (int w = 1; w < C::WK; ++w) M = fmaxf(M, st_m[w * WH + rw][rr]);
                float L = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < C::WK; ++w) {
                    const float mw = st_m[w * WH + rw][rr];
                    const float f = mw == M ? 1.f : pow2(mw - M);  // (both -inf: zeros either way)
                    const float4 v = *reinterpret_cast<const float4 *>(ob + ((w * WH + rw) * C::HEADS + rr) * DP + (col ^ (((rr >> 1) & 3) << 3)));
                    L += st_l[w * WH + rw][rr] * f;
                    acc.x += v.x * f;
                    acc.y += v.y * f;
                    acc.z += v.z * f;
                    acc.w += v.w * f;
                }
                if (whole) {
                    store(cw.b, cw.h, cw.hb, r, col, acc, M, L);
                } else {
                    *reinterpret_cast<float4 *>(slot + r * DP + col) = acc;
                    if (col == 0) {
                        slot[C::ROWS * DP + r] = M;
                        slot[C::ROWS * (DP + 1) + r] = L;
                    }
                }
            }
            cta_sync();  // the stage and the statistics may be written again; a piece is whole in the workspace
            if (C::SPLITS && p.split) {
                if (begun_here && tid == 0)
                    p.split[(cw.b * p.kv_heads + cw.h) * p.head_blocks + cw.hb] = whole ? make_int2(0, 0) : make_int2(left_open.first, left_open.n);
            } else if (!whole && tid == 0) {
                if (begun_here) left_ticket = add_acq_rel(counter_of(left_open));
                else begun_ticket = add_acq_rel(counter_of(begun));
            }
            fresh = true;
        }
        advance(cw);
        if (++stage == S) stage = 0;
    }
#pragma unroll 1
    for (int x = 0; x < 2; ++x) {
        if ((C::SPLITS && p.split) || !(x == 0 ? has_begun : has_left)) continue;
        const AttnPiece item = x == 0 ? begun : left_open;
        unsigned t = x == 0 ? begun_ticket : left_ticket;
        unsigned *counter = counter_of(item);
        int i0 = (static_cast<int>(cta) - item.first) / item.per_group * item.per_group, step = 1, count = min(item.per_group, item.n - i0);
#pragma unroll 1
        while (true) {
            if (tid == 0) {
                sh_last = t == static_cast<unsigned>(count - 1);
                if (sh_last) *counter = 0;
            }
            cta_sync();
            if (!sh_last) break;
            const bool final = step > 1 || item.per_group == item.n;
            join(item, i0, step, count, final);
            if (final) break;
            counter = p.counters + 2 * gridDim.x + item.first;
            if (tid == 0) t = add_acq_rel(counter);
            i0 = 0;
            step = item.per_group;
            count = (item.n + item.per_group - 1) / item.per_group;
        }
        cta_sync();  // sh_last is written again
    }
}

}  // namespace sdt
