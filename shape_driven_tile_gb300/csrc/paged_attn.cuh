// paged_attn.cuh -- attention of one new token per request over a paged key-value cache.
//
// For request b, query head i of key head h = i / G, and keys n in [lo_b, len_b):
//     o = sum_n 2^(s_n - m) v_n / sum_n 2^(s_n - m),   s_n = (scale log2 e) q . k_n
// for any reference m; a range of keys is summed up by (m, l = sum 2^(s_n - m),
// o = sum 2^(s_n - m) v_n), and two ranges join as m' = max(m1, m2),
// l' = l1 2^(m1 - m') + l2 2^(m2 - m'), o' likewise.
//
// What bounds it: HBM.  A cached token costs 4 G flops per key and value element pair of 4
// bytes (2 in q8), so with up to 16 query heads per key head the matrix instructions need
// to run at a fraction of their rate; the design keeps enough bytes in flight.
//
// Work: a unit is TK consecutive keys of one (request, key head, block of 16 WH query
// heads).  The units of all requests, in that order, are dealt out evenly over one
// resident grid, so a batch of any mix of lengths keeps every SM streaming to the end; a
// CTA computes its share from `lens` by itself.  A share may begin and end inside a
// (request, head) item: such pieces go to the workspace as (m, l, o) in fp32 and the last
// CTA to arrive at the item joins them in the order of the keys, so results do not depend
// on the order of arrival.
//
// CTA: four warps.  WH warps work on the same keys for 16 query heads each, WK = 4 / WH
// such groups on neighbouring keys; each has its own ring of S stages in shared memory,
// filled by cp.async 16 bytes at a time (rows of any page size and stride; rows past the
// range are filled with zeros, so what lies there is never read) and waits for nobody
// else.  Page ids are read one unit ahead.  Products run on mma.sync m16n8k16 (16 query
// heads x 8 keys, then 16 query heads x 8 value columns): the accumulators of one product
// are the operand of the next without leaving their registers.  (tcgen05.mma wants 64 or
// more rows of queries; one new token has G.)
//
// Numbers: scores, maxima, sums and outputs stay in fp32.  The weights 2^(s - m) enter the
// second product as the sum of two 16-bit values (the rounded weight and the rounded
// rest): one rounding to 8 bits would cost as much accuracy as the output's own, and the
// matrix unit has the time.
#pragma once

#include <type_traits>

#include "paged.cuh"
#include "ptx.cuh"

namespace sdt {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = kAttnWarps * 32;

struct PagedAttnArgs {
    const char *q;             // strides in bytes
    char *out;
    float *lse;                // [batch][q_heads], or null
    int64_t q_batch, q_head, o_batch, o_head;
    PagedRows k, v, ks, vs;
    const int *table;
    int64_t table_stride;
    const int *lens;
    int batch, kv_heads, group, head_blocks;  // group: query heads per key head
    int head_dim, max_pages, num_pages, window;
    FastDiv page;
    float scale_log2;          // scale * log2(e)
    float *partials;           // 2 slots per CTA: [rows][DP] o, [rows] m, [rows] l
    unsigned *counters;        // one per CTA, zero between calls
    int *status;
};

template <int DP, int WH, bool Q8>
struct AttnCfg {
    static constexpr int ROWB = DP * (Q8 ? 1 : 2);       // bytes of a cached row in shared memory
    static constexpr int TK = ROWB >= 256 && !Q8 ? 64 : 128;  // keys of a unit: the stage also holds the warps' o (fp32)
    static constexpr int WK = kAttnWarps / WH;
    static constexpr int KS = TK / WK;                    // keys of one group of warps
    static constexpr int RW = TK / kAttnWarps;            // rows that one warp loads
    static constexpr int SCB = Q8 ? DP / 16 : 0;          // bytes of a row's scales
    static constexpr int STAGE = TK * 2 * (ROWB + SCB);
    static constexpr int S = 3;
    static constexpr int ROWS = 16 * WH;                  // query heads of a CTA
    static constexpr int SLOT = ROWS * (DP + 2);          // floats of a partial
    static constexpr int SMEM = S * STAGE;
    static constexpr int CTAS = SMEM <= 112 * 1024 ? 2 : 1;
    static_assert(STAGE >= ROWS * WK * DP * 4, "the stage must hold every warp's o");
    static_assert(RW <= 32, "a lane describes one row");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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
// d (16 x 8, fp32) += a (16 x 16) . b (16 x 8)
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same_v<T, __half>)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two fp32 -> packed 16-bit pair (x in the low half), and the pair of what the rounding left.
template <typename T>
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    if constexpr (std::is_same_v<T, __half>) {
        const __half2 h = __floats2half2_rn(x, y);
        const float2 f = __half22float2(h);
        const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        const float2 f = __bfloat1622float2(h);
        const __nv_bfloat162 l = __floats2bfloat162_rn(x - f.x, y - f.y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    }
}
// int8 bytes in the low and third byte of t (others anything) -> two exact bf16 (T =
// __nv_bfloat16) or fp16 values.  bf16: 0x43 in front of seven bits b reads 128 + b, and in
// front of the sign bit alone 128 or 256: the difference is the signed value.  fp16: 0x64 in
// front of the byte with its sign bit flipped reads 1024 + 128 + value.
template <typename T>
__device__ __forceinline__ uint32_t widen_s8(uint32_t t) {
    uint32_t r;
    if constexpr (std::is_same_v<T, __half>) {
        const uint32_t x = ((t ^ 0x00800080u) & 0x00ff00ffu) | 0x64006400u;
        const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&x), __half2half2(__ushort_as_half(0x6480)));
        r = *reinterpret_cast<const uint32_t *>(&d);
    } else {
        const uint32_t x = (t & 0x007f007fu) | 0x43004300u, y = (t & 0x00800080u) | 0x43004300u;
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&x), *reinterpret_cast<const __nv_bfloat162 *>(&y));
        r = *reinterpret_cast<const uint32_t *>(&d);
    }
    return r;
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

// Position of 16-byte piece c of row r in a q8 tile: pairs of pieces (32 values, one group)
// move together, so that both access patterns below spread over the banks: 8-byte reads of
// rows r .. r+3 and 4-byte reads of rows r, r+2, r+4, r+6.
template <int DP>
__device__ __forceinline__ uint32_t q8_piece(uint32_t r, uint32_t c) {
    return DP >= 128 ? c ^ (((r & 3) ^ ((r >> 2) & 1)) << 1) : c ^ (((r >> 1) & 1) << 1);
}

// Where in the work a reader stands: unit j of n of item (b, h), keys [lo, len).
struct AttnWalk {
    int b, h, j, n, lo, len;
};

template <typename T, int DP, int WH, bool Q8>
__global__ void __launch_bounds__(kAttnThreads, (AttnCfg<DP, WH, Q8>::CTAS)) paged_attn_kernel(const PagedAttnArgs p) {
    using C = AttnCfg<DP, WH, Q8>;
    constexpr int TK = C::TK, KS = C::KS, RW = C::RW, ROWB = C::ROWB, S = C::S;
    constexpr int NT = DP / 8;        // 8-wide column tiles of o
    constexpr int SUB = KS < 32 ? KS : 32;  // keys between two looks at the running maximum
    using PT = std::conditional_t<Q8, __nv_bfloat16, T>;  // type of the second product: a q8 weight times its
                                                          // scale needs bf16's range
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float st_m[kAttnWarps][16], st_l[kAttnWarps][16];
    __shared__ long long sh_sum[kAttnWarps];
    __shared__ int sh_b;
    __shared__ long long sh_rest;
    __shared__ unsigned sh_last;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int wk = warp / WH, hw = warp % WH;
    const int g = lane >> 2, c = lane & 3;
    const uint32_t smem0 = smem_u32(smem);
    const int H = p.kv_heads * p.head_blocks;

    griddep_launch_dependents();
    griddep_wait();

    // ---- this CTA's share ----
    auto range_of = [&](int b, int &lo, int &len) {
        const int cap = p.max_pages * static_cast<int>(p.page.d);  // < 2^31: checked on the host
        int n = __ldg(p.lens + b);
        n = n < 0 ? 0 : n;
        len = n > cap ? cap : n;
        lo = p.window > 0 && len > p.window ? len - p.window : 0;
        return n > cap;
    };
    auto units_of = [&](int b) {
        int lo, len;
        range_of(b, lo, len);
        const int n = (len - lo + TK - 1) / TK;
        return n < 1 ? 1 : n;  // a request without keys still has zeros to write
    };
    long long mine = 0;
    for (int b = tid; b < p.batch; b += kAttnThreads) {
        mine += units_of(b);
        int lo, len;
        if (range_of(b, lo, len) && blockIdx.x == 0) paged_status(p.status, kSiteLength);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) sh_sum[warp] = mine;
    __syncthreads();
    long long U = 0;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) U += sh_sum[w];
    U *= H;
    const long long P = U < gridDim.x ? U : gridDim.x;  // CTAs with work
    const long long cta = blockIdx.x;
    if (cta >= P) return;
    const long long u0 = U * cta / P, u1 = U * (cta + 1) / P;
    // the request of unit u0: scan the requests 128 at a time
    {
        long long before = 0;
        for (int b0 = 0; b0 < p.batch; b0 += kAttnThreads) {
            const int b = b0 + tid;
            const long long n = b < p.batch ? static_cast<long long>(units_of(b)) * H : 0;
            long long inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long t = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += t;
            }
            __syncthreads();
            if (lane == 31) sh_sum[warp] = inc;
            __syncthreads();
            long long off = before;
            for (int w = 0; w < warp; ++w) off += sh_sum[w];
            inc += off;
            if (u0 < inc && u0 >= inc - n) {
                sh_b = b;
                sh_rest = u0 - (inc - n);
            }
            for (int w = 0; w < kAttnWarps; ++w) before += sh_sum[w];
            if (before > u0) break;
        }
        __syncthreads();
    }
    auto enter = [&](AttnWalk &w) {  // the walk stands on request w.b
        if (w.b >= p.batch) return;
        range_of(w.b, w.lo, w.len);
        const int n = (w.len - w.lo + TK - 1) / TK;
        w.n = n < 1 ? 1 : n;
    };
    auto advance = [&](AttnWalk &w) {
        if (++w.j == w.n) {
            w.j = 0;
            if (++w.h == H) {
                w.h = 0;
                ++w.b;
                enter(w);
            }
        }
    };
    AttnWalk pw;  // the loads' place
    pw.b = sh_b;
    enter(pw);
    pw.h = static_cast<int>(sh_rest / pw.n);
    pw.j = static_cast<int>(sh_rest - static_cast<long long>(pw.h) * pw.n);
    AttnWalk cw = pw;  // the products' place

    // ---- loads: lane r < RW describes row warp * RW + r of the unit ----
    int pg_id = -1, pg_off = 0, pg_head = 0;
    bool pg_ok = false;
    auto look_up = [&] {
        const int key = pw.lo + pw.j * TK + warp * RW + lane;
        pg_ok = lane < RW && key < pw.len;
        pg_head = pw.h / p.head_blocks;
        if (pg_ok) {
            const int pi = static_cast<int>(p.page.div(key));
            pg_off = key - pi * static_cast<int>(p.page.d);
            pg_id = __ldg(p.table + pw.b * p.table_stride + pi);
        }
    };
    const int pieces = p.head_dim * (Q8 ? 1 : 2) / 16;  // 16-byte pieces of a row that exist
    auto issue = [&](int stage) {
        if (pg_ok && (pg_id < 0 || pg_id >= p.num_pages)) {
            paged_status(p.status, kSitePage);
            pg_ok = false;
        }
        const int64_t ko = pg_ok ? p.k.at(pg_id, pg_off, pg_head) : -1;
        const int64_t vo = pg_ok ? p.v.at(pg_id, pg_off, pg_head) : -1;
        constexpr int CPR = ROWB / 16, RPI = 32 / CPR;  // pieces per row, rows per instruction
        const uint32_t kdst = smem0 + stage * C::STAGE + warp * RW * ROWB, vdst = kdst + TK * ROWB;
        const int cc = lane % CPR, rr = lane / CPR;
#pragma unroll
        for (int it = 0; it < RW / RPI; ++it) {
            const int r = it * RPI + rr;
            const int64_t ka = __shfl_sync(0xffffffffu, ko, r), va = __shfl_sync(0xffffffffu, vo, r);
            const uint32_t pos = r * ROWB + (Q8 ? q8_piece<DP>(r, cc) : static_cast<uint32_t>(cc ^ (r & 7))) * 16u;
            const int n = ka >= 0 && cc < pieces ? 16 : 0;
            cp_async16(kdst + pos, n ? p.k.base + ka + cc * 16 : p.k.base, n);
            cp_async16(vdst + pos, n ? p.v.base + va + cc * 16 : p.v.base, n);
        }
        if constexpr (Q8) {
            if (lane < RW) {
                const uint32_t sdst = smem0 + stage * C::STAGE + 2 * TK * ROWB + (warp * RW + lane) * C::SCB;
                const char *ks = pg_ok ? p.ks.base + p.ks.at(pg_id, pg_off, pg_head) : p.ks.base;
                const char *vs = pg_ok ? p.vs.base + p.vs.at(pg_id, pg_off, pg_head) : p.vs.base;
#pragma unroll
                for (int i = 0; i < DP / 64; ++i) {
                    const int n = pg_ok && i * 64 < p.head_dim ? 4 : 0;
                    cp_async4(sdst + i * 4, ks + (n ? i * 4 : 0), n);
                    cp_async4(sdst + TK * C::SCB + i * 4, vs + (n ? i * 4 : 0), n);
                }
            }
        }
    };
    auto group_sync = [&] {
        if constexpr (WH == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + wk), "n"(WH * 32) : "memory");
    };

    // ---- per item state ----
    uint32_t qf[DP / 16][4];
    float o[NT][4];
    float m0, m1, l0, l1;  // rows g and g + 8: running reference and this thread's part of the sum
    auto load_q = [&] {
        const int hb = cw.h % p.head_blocks, kvh = cw.h / p.head_blocks;
        const int r0 = hb * C::ROWS + hw * 16 + g, r1 = r0 + 8;
        const char *q0 = p.q + cw.b * p.q_batch + static_cast<int64_t>(kvh * p.group + r0) * p.q_head;
        const char *q1 = q0 + 8 * p.q_head;
        const bool ok0 = r0 < p.group, ok1 = r1 < p.group;
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
            // columns of this thread's two pairs (any order of d does, the keys' operand has the same)
            const int d0 = Q8 ? (kk >> 1) * 32 + c * 8 + (kk & 1) * 4 : kk * 16 + c * 2, d1 = Q8 ? d0 + 2 : d0 + 8;
            const bool in0 = d0 < p.head_dim, in1 = d1 < p.head_dim;
            qf[kk][0] = ok0 && in0 ? __ldg(reinterpret_cast<const unsigned *>(q0 + d0 * 2)) : 0u;
            qf[kk][1] = ok1 && in0 ? __ldg(reinterpret_cast<const unsigned *>(q1 + d0 * 2)) : 0u;
            qf[kk][2] = ok0 && in1 ? __ldg(reinterpret_cast<const unsigned *>(q0 + d1 * 2)) : 0u;
            qf[kk][3] = ok1 && in1 ? __ldg(reinterpret_cast<const unsigned *>(q1 + d1 * 2)) : 0u;
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
    };

    // ---- prologue: S - 1 units in flight, the page ids of the next ----
    look_up();
    long long issued = u0;
#pragma unroll
    for (int s = 0; s < S - 1; ++s) {
        if (issued < u1) {
            issue(s);
            ++issued;
            advance(pw);
            if (issued < u1) look_up();
        }
        cp_async_commit();
    }

    int stage = 0;
    bool fresh = true;
    for (long long u = u0; u < u1; ++u) {
        cp_async_wait<S - 2>();
        group_sync();
        {
            const int st = stage == 0 ? S - 1 : stage - 1;  // consumed in the previous round
            if (issued < u1) {
                issue(st);
                ++issued;
                advance(pw);
                if (issued < u1) look_up();
            }
            cp_async_commit();
        }
        if (fresh) {
            load_q();
            fresh = false;
        }
        const uint32_t kt = smem0 + stage * C::STAGE + wk * KS * ROWB, vt = kt + TK * ROWB;
        const uint32_t kst = smem0 + stage * C::STAGE + 2 * TK * ROWB + wk * KS * C::SCB, vst = kst + TK * C::SCB;
        const int left = cw.len - (cw.lo + cw.j * TK + wk * KS);  // valid keys from this group's first on
#pragma unroll 1
        for (int k0 = 0; k0 < KS; k0 += SUB) {
            if (k0 >= left) break;
            float s[SUB / 8][4];
#pragma unroll
            for (int i = 0; i < SUB / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
            // scores: 16 query heads x SUB keys
            if constexpr (!Q8) {
                const uint32_t row = kt + (k0 + (lane & 7) + ((lane >> 4) << 3)) * ROWB;
                const uint32_t sw = (((lane >> 3) & 1) ^ (lane & 7)) << 4;
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk) {
#pragma unroll
                    for (int i = 0; i < SUB / 16; ++i) {
                        uint32_t b[4];
                        ldsm_x4(row + i * 16 * ROWB + ((kk << 5) ^ sw), b);
                        mma16816<T>(s[2 * i], qf[kk], b[0], b[1]);
                        mma16816<T>(s[2 * i + 1], qf[kk], b[2], b[3]);
                    }
                }
            } else {
#pragma unroll
                for (int gr = 0; gr < DP / 32; ++gr) {
#pragma unroll
                    for (int i = 0; i < SUB / 8; ++i) {
                        const uint32_t r = k0 + i * 8 + g;
                        const uint2 w = lds64(kt + r * ROWB + q8_piece<DP>(r, gr * 2 + (c >> 1)) * 16 + (c & 1) * 8);
                        float t[4] = {0.f, 0.f, 0.f, 0.f};
                        mma16816<T>(t, qf[2 * gr], widen_s8<T>(__byte_perm(w.x, 0, 0x4140)), widen_s8<T>(__byte_perm(w.x, 0, 0x4342)));
                        mma16816<T>(t, qf[2 * gr + 1], widen_s8<T>(__byte_perm(w.y, 0, 0x4140)), widen_s8<T>(__byte_perm(w.y, 0, 0x4342)));
                        // columns 2c, 2c + 1 of the tile are keys with scales of their own
                        const uint32_t sa = kst + (k0 + i * 8 + 2 * c) * C::SCB + gr * 2;
                        unsigned short x0, x1;
                        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x0) : "r"(sa) : "memory");
                        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x1) : "r"(sa + C::SCB) : "memory");
                        const float f0 = __half2float(__ushort_as_half(x0)), f1 = __half2float(__ushort_as_half(x1));
                        s[i][0] += t[0] * f0;
                        s[i][1] += t[1] * f1;
                        s[i][2] += t[2] * f0;
                        s[i][3] += t[3] * f1;
                    }
                }
            }
            // running maximum; keys past the range drop out
            float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
            for (int i = 0; i < SUB / 8; ++i) {
                const int n = k0 + i * 8 + 2 * c;
                s[i][0] = n < left ? s[i][0] * p.scale_log2 : -INFINITY;
                s[i][1] = n + 1 < left ? s[i][1] * p.scale_log2 : -INFINITY;
                s[i][2] = n < left ? s[i][2] * p.scale_log2 : -INFINITY;
                s[i][3] = n + 1 < left ? s[i][3] * p.scale_log2 : -INFINITY;
                x0 = fmaxf(x0, fmaxf(s[i][0], s[i][1]));
                x1 = fmaxf(x1, fmaxf(s[i][2], s[i][3]));
            }
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
            if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
                const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
                const float a0 = m0 == n0 ? 1.f : exp2f(m0 - n0), a1 = m1 == n1 ? 1.f : exp2f(m1 - n1);
                m0 = n0;
                m1 = n1;
                l0 *= a0;
                l1 *= a1;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    o[i][0] *= a0;
                    o[i][1] *= a0;
                    o[i][2] *= a1;
                    o[i][3] *= a1;
                }
            }
            // weights (a row that has seen only -inf keeps its weights at zero)
            const float e0 = m0 == -INFINITY ? 0.f : m0, e1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
            for (int i = 0; i < SUB / 8; ++i) {
                s[i][0] = exp2f(s[i][0] - e0);
                s[i][1] = exp2f(s[i][1] - e0);
                s[i][2] = exp2f(s[i][2] - e1);
                s[i][3] = exp2f(s[i][3] - e1);
                l0 += s[i][0] + s[i][1];
                l1 += s[i][2] + s[i][3];
            }
            // o += weights . values
#pragma unroll
            for (int kb = 0; kb < SUB / 16; ++kb) {
                if constexpr (!Q8) {
                    uint32_t hi[4], lo[4];
                    split2<PT>(s[2 * kb][0], s[2 * kb][1], hi[0], lo[0]);
                    split2<PT>(s[2 * kb][2], s[2 * kb][3], hi[1], lo[1]);
                    split2<PT>(s[2 * kb + 1][0], s[2 * kb + 1][1], hi[2], lo[2]);
                    split2<PT>(s[2 * kb + 1][2], s[2 * kb + 1][3], hi[3], lo[3]);
                    const uint32_t row = vt + (k0 + kb * 16 + (lane & 15)) * ROWB;
                    const uint32_t sw = ((lane >> 4) ^ (lane & 7)) << 4;
#pragma unroll
                    for (int i = 0; i < NT / 2; ++i) {
                        uint32_t b[4];
                        ldsm_x4_t(row + ((i << 5) ^ sw), b);
                        mma16816<PT>(o[2 * i], hi, b[0], b[1]);
                        mma16816<PT>(o[2 * i], lo, b[0], b[1]);
                        mma16816<PT>(o[2 * i + 1], hi, b[2], b[3]);
                        mma16816<PT>(o[2 * i + 1], lo, b[2], b[3]);
                    }
                } else {
                    const uint32_t r = k0 + kb * 16 + 2 * c;  // this thread's keys: r, r+1, r+8, r+9
#pragma unroll
                    for (int gr = 0; gr < DP / 32; ++gr) {
                        float f[4];
                        uint32_t w[4];
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const uint32_t rt = r + (t & 1) + (t >> 1) * 8;
                            unsigned short x;
                            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(vst + rt * C::SCB + gr * 2) : "memory");
                            f[t] = __half2float(__ushort_as_half(x));
                            w[t] = lds32(vt + rt * ROWB + q8_piece<DP>(rt, gr * 2 + (g >> 2)) * 16 + (g & 3) * 4);
                        }
                        uint32_t hi[4], lo[4];
                        split2<PT>(s[2 * kb][0] * f[0], s[2 * kb][1] * f[1], hi[0], lo[0]);
                        split2<PT>(s[2 * kb][2] * f[0], s[2 * kb][3] * f[1], hi[1], lo[1]);
                        split2<PT>(s[2 * kb + 1][0] * f[2], s[2 * kb + 1][1] * f[3], hi[2], lo[2]);
                        split2<PT>(s[2 * kb + 1][2] * f[2], s[2 * kb + 1][3] * f[3], hi[3], lo[3]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {  // column tile j: value g * 4 + j of the group
                            const uint32_t sel = static_cast<uint32_t>(j) | (static_cast<uint32_t>(4 + j) << 8);
                            const uint32_t b0 = widen_s8<PT>(__byte_perm(w[0], w[1], sel));
                            const uint32_t b1 = widen_s8<PT>(__byte_perm(w[2], w[3], sel));
                            mma16816<PT>(o[gr * 4 + j], hi, b0, b1);
                            mma16816<PT>(o[gr * 4 + j], lo, b0, b1);
                        }
                    }
                }
            }
        }

        const bool item_done = cw.j == cw.n - 1;
        if (item_done || u == u1 - 1) {
            // ---- the CTA's piece of the item: join the warps through the stage just read ----
            l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
            l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
            __syncthreads();  // every warp has read the stage
            if (c == 0) {
                st_m[warp][g] = m0;
                st_m[warp][g + 8] = m1;
                st_l[warp][g] = l0;
                st_l[warp][g + 8] = l1;
            }
            float *ob = reinterpret_cast<float *>(smem + stage * C::STAGE);
            const int valid = min(p.group - (cw.h % p.head_blocks) * C::ROWS, C::ROWS);  // query heads of this block
            const int sw = (g & 3) << 3;  // 32-byte pieces of a row swapped by row: no bank conflicts
            float *w0 = ob + (warp * 16 + g) * DP, *w1 = w0 + 8 * DP;
            if constexpr (!Q8) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    if (hw * 16 + g < valid) *reinterpret_cast<float2 *>(w0 + ((i * 8 + 2 * c) ^ sw)) = make_float2(o[i][0], o[i][1]);
                    if (hw * 16 + g + 8 < valid) *reinterpret_cast<float2 *>(w1 + ((i * 8 + 2 * c) ^ sw)) = make_float2(o[i][2], o[i][3]);
                }
            } else {  // column n of tile j of a group is its value 4 n + j
#pragma unroll
                for (int gr = 0; gr < DP / 32; ++gr) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int at = (gr * 32 + c * 8 + x * 4) ^ sw;
                        if (hw * 16 + g < valid)
                            *reinterpret_cast<float4 *>(w0 + at) = make_float4(o[gr * 4][x], o[gr * 4 + 1][x], o[gr * 4 + 2][x], o[gr * 4 + 3][x]);
                        if (hw * 16 + g + 8 < valid)
                            *reinterpret_cast<float4 *>(w1 + at) = make_float4(o[gr * 4][2 + x], o[gr * 4 + 1][2 + x], o[gr * 4 + 2][2 + x], o[gr * 4 + 3][2 + x]);
                    }
                }
            }
            __syncthreads();

            const long long first_unit = u - cw.j, end_unit = first_unit + cw.n;
            const bool whole = first_unit >= u0 && end_unit <= u1;
            const int head0 = (cw.h / p.head_blocks) * p.group + (cw.h % p.head_blocks) * C::ROWS;
            auto store = [&](int r, int col, const float4 &v, float M, float L) {
                const float inv = L > 0.f ? 1.f / L : L == 0.f ? 0.f : L;  // no key: zeros; a NaN sum stays NaN
                if (col < p.head_dim) {
                    uint2 b;
                    if constexpr (std::is_same_v<T, __half>) {
                        const __half2 a0 = __floats2half2_rn(v.x * inv, v.y * inv), a1 = __floats2half2_rn(v.z * inv, v.w * inv);
                        b = make_uint2(*reinterpret_cast<const uint32_t *>(&a0), *reinterpret_cast<const uint32_t *>(&a1));
                    } else {
                        const __nv_bfloat162 a0 = __floats2bfloat162_rn(v.x * inv, v.y * inv), a1 = __floats2bfloat162_rn(v.z * inv, v.w * inv);
                        b = make_uint2(*reinterpret_cast<const uint32_t *>(&a0), *reinterpret_cast<const uint32_t *>(&a1));
                    }
                    *reinterpret_cast<uint2 *>(p.out + cw.b * p.o_batch + static_cast<int64_t>(head0 + r) * p.o_head + col * 2) = b;
                }
                if (p.lse && col == 0)
                    p.lse[static_cast<int64_t>(cw.b) * p.kv_heads * p.group + head0 + r] =
                        L == 0.f ? -INFINITY : M * 0.6931471805599453f + logf(L);
            };
            float *slot = p.partials + static_cast<size_t>(2 * cta + (first_unit >= u0 ? 1 : 0)) * C::SLOT;
            for (int e = tid; e < valid * (DP / 4); e += kAttnThreads) {
                const int r = e / (DP / 4), col = (e % (DP / 4)) * 4, rw = r >> 4, rr = r & 15;
                float M = st_m[rw][rr];
#pragma unroll
                for (int w = 1; w < C::WK; ++w) M = fmaxf(M, st_m[w * WH + rw][rr]);
                float L = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < C::WK; ++w) {
                    const float mw = st_m[w * WH + rw][rr];
                    const float f = mw == M ? 1.f : exp2f(mw - M);  // (both -inf: zeros either way)
                    const float4 v = *reinterpret_cast<const float4 *>(ob + ((w * WH + rw) * 16 + rr) * DP + (col ^ ((rr & 3) << 3)));
                    L += st_l[w * WH + rw][rr] * f;
                    acc.x += v.x * f;
                    acc.y += v.y * f;
                    acc.z += v.z * f;
                    acc.w += v.w * f;
                }
                if (whole) {
                    store(r, col, acc, M, L);
                } else {
                    *reinterpret_cast<float4 *>(slot + r * DP + col) = acc;
                    if (col == 0) {
                        slot[C::ROWS * DP + r] = M;
                        slot[C::ROWS * (DP + 1) + r] = L;
                    }
                }
            }
            if (!whole) {
                // ---- the item's pieces: the last CTA to arrive joins them ----
                const long long first_cta = ((first_unit + 1) * P - 1) / U, last_cta = (end_unit * P - 1) / U;
                const int pieces_n = static_cast<int>(last_cta - first_cta) + 1;
                __threadfence();
                __syncthreads();
                if (tid == 0) sh_last = atomicAdd(p.counters + first_cta, 1u) == static_cast<unsigned>(pieces_n - 1);
                __syncthreads();
                if (sh_last) {
                    __threadfence();
                    // piece 0 lies in its CTA's second slot, the others in their first
                    auto piece = [&](int i) { return p.partials + static_cast<size_t>(2 * (first_cta + i) + (i == 0 ? 1 : 0)) * C::SLOT; };
                    for (int e = tid; e < valid * (DP / 4); e += kAttnThreads) {
                        const int r = e / (DP / 4), col = (e % (DP / 4)) * 4;
                        float M = -INFINITY;
                        for (int i = 0; i < pieces_n; ++i) M = fmaxf(M, __ldcg(piece(i) + C::ROWS * DP + r));
                        float L = 0.f;
                        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                        for (int i = 0; i < pieces_n; ++i) {
                            const float *s = piece(i);
                            const float mi = __ldcg(s + C::ROWS * DP + r);
                            const float f = mi == M ? 1.f : exp2f(mi - M);
                            const float4 v = __ldcg(reinterpret_cast<const float4 *>(s + r * DP + col));
                            L += __ldcg(s + C::ROWS * (DP + 1) + r) * f;
                            acc.x += v.x * f;
                            acc.y += v.y * f;
                            acc.z += v.z * f;
                            acc.w += v.w * f;
                        }
                        store(r, col, acc, M, L);
                    }
                    if (tid == 0) p.counters[first_cta] = 0;
                }
            }
            __syncthreads();  // the stage may be loaded again, the statistics written again
            fresh = true;
        }
        advance(cw);
        if (++stage == S) stage = 0;
    }
    cp_async_wait<0>();
}

}  // namespace sdt
