// fp8_rows.cu -- rows of 16-bit values to fp8 with a scale per 128: rms_norm_fp8 (with the
// residual's addition) and quant_fp8 (as they are, or act(gate) * x).
//
// Quantisation of one block of 128 values y (the last block of a row may be shorter):
// top = max(max|y|, 2^-100), scale = top * fl(1/448), q = e4m3(y * 448 / top), rounded to nearest
// even.  With 16-bit values on both sides of the quotient exact ties are common (0.5 % of normally
// distributed bf16 values), and a factor 448 / top of 24 bits puts a fifth of them on the wrong
// side: without a gate it is held in two parts, so that the quotient is off by 2^-45 before its
// rounding to fp32 and a tie stays one.  What a gate or the norm makes is itself off by some steps
// of fp32 and takes one factor, rounded once.  (The norm's ties can be kept too, as a row's factor divides
// out of the quotients and value times weight is exact; 8191 x 8128 then took 96.4 us in place of 94.5,
// 16384 x 4096 in fp16 without a residual 48.8 in place of 45.9.)
// The floor keeps the factor finite for rows of zeros.  A NaN stays a NaN of its
// own; an infinity makes the scale infinite, so that its whole block stands for NaN.
//
// A thread moves 16-byte pieces of 8 values; 16 neighbouring threads hold a block and find its
// largest value by shuffles.  The norm holds a row in registers between the sum of squares and
// the scaling, so each value is read once and written once.
//
// What bounds it: memory for prompts (quant_fp8 of 8192 x 14336: 55 us, 97 % of the measured copy rate, 53.7 with
// a factor in one part; gated by silu 91 us, 96 %; by gelu 101 us, 87 %, where instructions count; rms_norm_fp8 of
// 8191 x 8128 with a residual and 16-bit output 94.5 us, 95 %; 16384 x 4096 with a residual 79 us, 89 %), the
// launch for a decode step's rows (1.5 to 2.5 us).
#include <cuda_fp8.h>

#include <cstring>
#include <type_traits>

#include "launch.cuh"
#include "overlap.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace sdt {

constexpr float kE4m3Max = 448.0f;
constexpr float kTinyTop = 7.888609052210118e-31f;  // 2^-100
constexpr int64_t kMaxQuantWidth = 65536, kMaxNormWidth = 32768;

enum : int { kGateNone = 0, kGateSilu = 1, kGateGelu = 2 };

// Eight values as four pairs: one instruction multiplies or adds both of a pair.
template <typename T>
__device__ __forceinline__ void to_f32(const uint4 &v, float2 (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same_v<T, __half>) {
            __half2 h;
            memcpy(&h, &w[i], 4);
            f[i] = __half22float2(h);
        } else {
            f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        }
    }
}

template <typename T>
__device__ __forceinline__ uint4 from_f32(const float2 (&f)[4]) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same_v<T, __half>) {
            const __half2 v = __float22half2_rn(f[i]);
            memcpy(&h[i], &v, 4);
        } else {
            const __nv_bfloat162 v = __float22bfloat162_rn(f[i]);
            memcpy(&h[i], &v, 4);
        }
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

// max(|a|, |b|, |c|); a NaN counts only if all are.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float d;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float top_of(const float2 (&f)[4]) {
    const float t = max3_abs(f[0].x, f[0].y, f[1].x), u = max3_abs(f[1].y, f[2].x, f[2].y);
    return max3_abs(max3_abs(t, u, f[3].x), f[3].y, kTinyTop);
}

// 1 / x to a step, for x of 2^-126 to 2^126.
__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 448 / top as hi + lo, for a top whose scale (top / 448, to some steps) is s.  hi is off by some steps, and
// what it lacks is known: 448 - hi * top is exact but for one rounding.  (By way of s no top, up to the
// largest fp32 value, takes the quotient out of the range of normal numbers.)  In one part it is rounded once.
struct Factor {
    float hi, lo;
};
template <bool TWO>
__device__ __forceinline__ Factor factor_of(float top, float s) {
    const float r = reciprocal(s), lacks = fmaf(-r, top, kE4m3Max), unit = r * (1.0f / kE4m3Max);
    if (TWO) return {r, lacks * unit};
    return {fmaf(lacks, unit, r), 0.0f};
}

template <bool TWO>
__device__ __forceinline__ uint2 to_e4m3(const float2 (&f)[4], Factor k) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 hi = make_float2(k.hi, k.hi), lo = make_float2(k.lo, k.lo);
        const float2 v = TWO ? __ffma2_rn(f[i], hi, __fmul2_rn(f[i], lo)) : __fmul2_rn(f[i], hi);
        w[i] = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
}

struct RowsOut {
    uint8_t *q;
    float *scales;
    int64_t q_row, s_row, s_block;
};

// The block's scale and the piece's fp8 values; `group` lanes (16, or a row's 8) hold the block.
// TWO: a factor in two parts.  q and scale: where they go, used only if `write`.
template <bool TWO>
__device__ __forceinline__ void quantise_piece(uint8_t *q, float *scale, int piece, const float2 (&f)[4], int group, bool write) {
    float top = top_of(f);
#pragma unroll
    for (int x = 1; x < 16; x <<= 1)
        if (x < group) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float s = top * (1.0f / kE4m3Max);
    if (!write) return;
    *reinterpret_cast<uint2 *>(q) = to_e4m3<TWO>(f, factor_of<TWO>(top, s));
    if ((piece & 15) == 0) *scale = s;
}

// 1 / (1 + exp(-t)) of two values, to some 1.5 steps of fp32 whatever t: with n = -t and x the rounded n / ln 2,
// exp(n) = 2^x * exp(n - x ln 2), and the rest in brackets (at most 1e-5, so that 1 + rest is its exponential) is
// taken with ln 2 in two parts; the reciprocal gets a Newton step.  (Values next to a border of the fp8 grid
// fall on its other side as often as such errors reach it; with a rounded argument alone, which is off by |t|
// steps, and no Newton step twice as many did.)  Past +-87.5 it is 1 or 0; a NaN counts as infinity here.
__device__ __forceinline__ float2 sigmoid(float2 t) {
    constexpr float kLn2Hi = 0.693147182f, kLn2Lo = -1.90465421e-9f;  // together ln 2 to 2^-53
    const float2 n = make_float2(fminf(fmaxf(-t.x, -87.5f), 87.5f), fminf(fmaxf(-t.y, -87.5f), 87.5f));
    const float2 x = __fmul2_rn(n, make_float2(1.44269504f, 1.44269504f));
    const float2 rest = __ffma2_rn(x, make_float2(-kLn2Lo, -kLn2Lo), __ffma2_rn(x, make_float2(-kLn2Hi, -kLn2Hi), n));
    float2 e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(x.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(x.y));
    e = __ffma2_rn(e, rest, e);
    const float2 minus_one = make_float2(-1.0f, -1.0f), minus_d = __ffma2_rn(e, minus_one, minus_one);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(-minus_d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(-minus_d.y));
    return __ffma2_rn(__ffma2_rn(minus_d, r, make_float2(1.0f, 1.0f)), r, r);
}

// ---- quant_fp8 ----------------------------------------------------------------------------

// Two pieces a thread: with four, silu takes 97 us (8192 x 14336) and 16 rows of it 2.45 us instead of
// 2.0; with one, 108 us; with CTAs of 128 threads rows without a gate take 59 us instead of 53.
constexpr int kQuantThreads = 256;
constexpr int kQuantUnroll = 2;

struct QuantArgs {
    const char *x, *gate;
    int64_t x_row, gate_row;  // bytes
    RowsOut out;
    uint32_t total;   // padded pieces of all rows
    int pieces;       // 16-byte pieces of a row
    FastDiv padded;   // pieces of a row rounded up to whole blocks of 16
};

// CTAs an SM holds, and so the registers of a thread: 8 of 32 registers are full SMs (silu without a bound: 38
// registers and 106 us for 8192 x 14336, 91 with it); gelu's instructions are better off with 47 and five CTAs
// (100.7 us; six 110, seven and eight 104.7, unbounded, 52 registers, 102.4).
constexpr int quant_resident(int gate) { return gate == kGateGelu ? 5 : 8; }

template <typename T, int GATE>
__global__ void __launch_bounds__(kQuantThreads, quant_resident(GATE)) quant_fp8_kernel(const QuantArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t base = blockIdx.x * (kQuantThreads * kQuantUnroll) + threadIdx.x;
    uint4 x[kQuantUnroll], g[kQuantUnroll];
    uint32_t row[kQuantUnroll];
    int piece[kQuantUnroll];
    bool have[kQuantUnroll];
#pragma unroll
    for (int u = 0; u < kQuantUnroll; ++u) {
        const uint32_t i = base + u * kQuantThreads;
        row[u] = a.padded.div(i);
        piece[u] = static_cast<int>(i - row[u] * a.padded.d);
        have[u] = i < a.total && piece[u] < a.pieces;
        x[u] = g[u] = make_uint4(0, 0, 0, 0);
        if (have[u]) {
            x[u] = *reinterpret_cast<const uint4 *>(a.x + row[u] * a.x_row + piece[u] * 16);
            if (GATE) g[u] = *reinterpret_cast<const uint4 *>(a.gate + row[u] * a.gate_row + piece[u] * 16);
        }
    }
#pragma unroll
    for (int u = 0; u < kQuantUnroll; ++u) {
        float2 f[4];
        to_f32<T>(x[u], f);
        if constexpr (GATE != kGateNone) {
            float2 h[4];
            to_f32<T>(g[u], h);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // g * sigmoid(t): silu has t = g; gelu's tanh form is 0.5 g (1 + tanh(t / 2))
                float2 t = h[i];
                if (GATE == kGateGelu) {
                    const float2 c1 = make_float2(1.59576912160573f, 1.59576912160573f), c3 = make_float2(0.0713548162726f, 0.0713548162726f);
                    t = __fmul2_rn(h[i], __ffma2_rn(c3, __fmul2_rn(h[i], h[i]), c1));
                }
                f[i] = __fmul2_rn(f[i], __fmul2_rn(h[i], sigmoid(t)));
            }
        }
        quantise_piece<GATE == kGateNone>(a.out.q + row[u] * a.out.q_row + piece[u] * 8, a.out.scales + row[u] * a.out.s_row + (piece[u] >> 4) * a.out.s_block, piece[u], f, 16, have[u]);
    }
}

// ---- rms_norm_fp8 -------------------------------------------------------------------------

struct NormArgs {
    const char *x;
    char *residual;       // NULL: none
    const char *weight;
    char *out16;          // NULL: not wanted
    int64_t x_row, r_row, o_row;  // bytes
    RowsOut out;
    int rows, pieces, per_row;    // per_row: threads of a row, 8, 16, 32 or the whole CTA
    float inv_width, eps;
    int weight_f32;
};

// A CTA walks over its rows (or groups of short rows), the next ones on their way into registers
// while it works on the present ones; the weights stay in registers.  VPT pieces a thread; rows of
// more than 16384 values (VPT 8) have no registers for a second row and load one after another.
constexpr int kNormThreads = 512;  // at most

// Registers of a thread, and how many threads an SM then holds: without a residual half as much is
// on its way per thread, so it takes more of them (16384 rows of 2880: 38.9 us with 768, 43.1 with 512).
constexpr int norm_registers(int vpt, bool residual) { return vpt <= 2 ? 64 : vpt == 4 && !residual ? 80 : 128; }
constexpr int norm_resident(int vpt, bool residual) { return vpt <= 2 ? 1024 : vpt == 4 && !residual ? 768 : 512; }

template <typename T, int VPT, bool RES>
__global__ void __maxnreg__(norm_registers(VPT, RES)) rms_norm_fp8_kernel(const NormArgs a) {
    constexpr bool kAhead = VPT <= 4;
    __shared__ float part[2][32];
    griddep_launch_dependents();
    const int per = a.per_row, whole = blockDim.x;
    const int r = threadIdx.x % per, step = gridDim.x * (whole / per);
    int row = blockIdx.x * (whole / per) + threadIdx.x / per;
    griddep_wait();
    uint4 x[VPT], res[RES ? VPT : 1], w[VPT];
    const auto load = [&](int at) {
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int piece = r + u * per;
            x[u] = make_uint4(0, 0, 0, 0);
            if (RES) res[u] = make_uint4(0, 0, 0, 0);
            if (at < a.rows && piece < a.pieces) {
                x[u] = *reinterpret_cast<const uint4 *>(a.x + at * a.x_row + piece * 16);
                if (RES) res[u] = *reinterpret_cast<const uint4 *>(a.residual + at * a.r_row + piece * 16);
            }
        }
    };
    load(row);
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        w[u] = make_uint4(0, 0, 0, 0);
        if (kAhead && !a.weight_f32 && r + u * per < a.pieces) w[u] = *reinterpret_cast<const uint4 *>(a.weight + (r + u * per) * 16);
    }
    // (every thread of a CTA takes as many turns: they meet in them)
    for (int first = blockIdx.x * (whole / per), turn = 0; first < a.rows; first += step, row += step, turn ^= 1) {
        const bool live = row < a.rows;
        uint4 v[VPT];
        float2 sums = make_float2(0.f, 0.f);
        char *res_row = a.residual + row * a.r_row + r * 16;
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            v[u] = x[u];
            float2 f[4];
            to_f32<T>(x[u], f);
            if constexpr (RES) {
                float2 h[4];
                to_f32<T>(res[u], h);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = __fadd2_rn(f[i], h[i]);
                v[u] = from_f32<T>(f);  // the norm is of the sum as it is kept
                to_f32<T>(v[u], f);
                if (live && r + u * per < a.pieces) *reinterpret_cast<uint4 *>(res_row + u * per * 16) = v[u];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sums = __ffma2_rn(f[i], f[i], sums);
        }
        if (kAhead) load(row + step);
        float sum = sums.x + sums.y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
            if (o < per) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (per > 32) {  // (a row is the whole CTA; two places, so that one meeting a row is enough)
            if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = sum;
            __syncthreads();
            sum = (threadIdx.x & 31) < (whole >> 5) ? part[turn][threadIdx.x & 31] : 0.f;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        const float k = rsqrtf(fmaf(sum, a.inv_width, a.eps));
        uint8_t *q = a.out.q + row * a.out.q_row + r * 8;
        float *scale = a.out.scales + row * a.out.s_row + (r >> 4) * a.out.s_block;
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int piece = r + u * per;
            const bool have = live && piece < a.pieces;
            float2 f[4], h[4];
            to_f32<T>(v[u], f);
            if (a.weight_f32) {
                float4 lo = make_float4(0, 0, 0, 0), hi = lo;
                if (piece < a.pieces) {
                    lo = *reinterpret_cast<const float4 *>(a.weight + piece * 32);
                    hi = *reinterpret_cast<const float4 *>(a.weight + piece * 32 + 16);
                }
                h[0] = make_float2(lo.x, lo.y); h[1] = make_float2(lo.z, lo.w); h[2] = make_float2(hi.x, hi.y); h[3] = make_float2(hi.z, hi.w);
            } else {
                if (!kAhead && piece < a.pieces) w[u] = *reinterpret_cast<const uint4 *>(a.weight + piece * 16);
                to_f32<T>(w[u], h);
            }
            // (pieces past the row are zeros throughout)
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = __fmul2_rn(__fmul2_rn(f[i], make_float2(k, k)), h[i]);
            if (a.out16 && have) *reinterpret_cast<uint4 *>(a.out16 + row * a.o_row + piece * 16) = from_f32<T>(f);
            quantise_piece<false>(q + u * per * 8, scale + (u * per >> 4) * a.out.s_block, piece, f, per < 16 ? per : 16, have);
        }
        if (!kAhead) load(row + step);
    }
}

template <typename T, bool RES>
static auto norm_kernel(int vpt) {
    return vpt == 1   ? rms_norm_fp8_kernel<T, 1, RES>
           : vpt == 2 ? rms_norm_fp8_kernel<T, 2, RES>
           : vpt == 4 ? rms_norm_fp8_kernel<T, 4, RES>
                      : rms_norm_fp8_kernel<T, 8, RES>;
}
template <typename T>
static auto norm_kernel(int vpt, bool residual) {
    return residual ? norm_kernel<T, true>(vpt) : norm_kernel<T, false>(vpt);
}

static int check_out(const char *who, void *q, float *scales, int64_t tokens, int64_t width, int64_t q_row, int64_t s_row,
                     int64_t s_block) {
    if (!q || !scales) return fail(SDT_ERR_NULL, "%s: q or scales is NULL", who);
    if (!aligned(q, 8) || !aligned(scales, 4)) return fail(SDT_ERR_ALIGN, "%s: q must be 8-byte aligned, scales 4-byte", who);
    if (tokens > 1 && (q_row < width || q_row % 8)) return fail(SDT_ERR_ARG, "%s: q's row stride must be a multiple of 8, at least the width", who);
    const int64_t blocks = (width + 127) / 128;
    if (tokens == 1) s_row = q_row = 0;  // (a dimension of one never steps)
    if (blocks == 1) s_block = 0;
    constexpr int64_t most = int64_t(1) << 32;
    if (s_row < 0 || s_block < 0 || s_row > most || s_block > most || q_row > most) return fail(SDT_ERR_ARG, "%s: strides must be in 0 .. 2^32", who);
    const bool rows_out = tokens == 1 || s_row >= (blocks == 1 ? 1 : (blocks - 1) * s_block + 1);
    const bool blocks_out = blocks == 1 || s_block >= (tokens == 1 ? 1 : (tokens - 1) * s_row + 1);
    if (!((rows_out && (blocks == 1 || s_block > 0)) || (blocks_out && (tokens == 1 || s_row > 0))))
        return fail(SDT_ERR_ARG, "%s: scales must not overlap one another", who);
    return SDT_OK;
}

static int check_in(const char *who, const char *what, const void *p, int64_t tokens, int64_t row, int64_t width, bool out = false) {
    if (!p) return fail(SDT_ERR_NULL, "%s: %s is NULL", who, what);
    if (!aligned(p, 16)) return fail(SDT_ERR_ALIGN, "%s: %s must be 16-byte aligned", who, what);
    if (tokens > 1 && (row < (out ? width : 0) || row % 8 || row > (int64_t(1) << 32)))
        return fail(SDT_ERR_ARG, "%s: the row stride of %s must be a multiple of 8 elements%s", who, what, out ? ", at least the width" : "");
    return SDT_OK;
}

static int check_size(const char *who, int64_t tokens, int64_t width, int64_t widest, int dtype) {
    if (width < 0 || width > widest || width % 8) return fail(SDT_ERR_SHAPE, "%s: width must be a multiple of 8 up to %lld (got %lld)", who, (long long)widest, (long long)width);
    if (tokens < 0 || (width > 0 && tokens > (INT32_MAX - kQuantThreads * kQuantUnroll) / ((width + 127) / 128 * 16)))
        return fail(SDT_ERR_SHAPE, "%s: tokens times the width in whole blocks of 128 must be below 2^34 - 2^12 (got %lld tokens)", who, (long long)tokens);
    if (dtype != SDT_DTYPE_F16 && dtype != SDT_DTYPE_BF16) return fail(SDT_ERR_ARG, "%s: dtype must be fp16 or bf16 (got %d)", who, dtype);
    return SDT_OK;
}

// The tensors of a call, outputs first: no output may share a byte with another of them.
struct Tensor {
    const char *name;
    Stretches at;
};
template <int N>
static int check_apart(const char *who, const Tensor (&all)[N], int outputs) {
    for (int i = 0; i < outputs; ++i)
        for (int j = i + 1; j < N; ++j)
            if (overlap(all[i].at, all[j].at)) return fail(SDT_ERR_ARG, "%s: %s and %s overlap", who, all[i].name, all[j].name);
    return SDT_OK;
}
static Stretches scales_of(const float *p, int64_t tokens, int64_t width, int64_t s_row, int64_t s_block) {
    const int64_t blocks = (width + 127) / 128;
    return {p, tokens, step_bytes(tokens, s_row, 4), blocks, step_bytes(blocks, s_block, 4), 4};
}

}  // namespace sdt

using namespace sdt;

extern "C" {

int quant_fp8(const sdt_quant_fp8 *call, sdt_stream_t stream) {
    clear_error();
    if (!call) return fail(SDT_ERR_NULL, "quant_fp8: NULL call");
    sdt_quant_fp8 c;
    memcpy(&c, call, sizeof c);
    int rc = check_size("quant_fp8", c.tokens, c.width, kMaxQuantWidth, c.dtype);
    if (rc) return rc;
    if (c.activation < 0 || c.activation > 2 || (c.activation != 0) != (c.gate != nullptr))
        return fail(SDT_ERR_ARG, "quant_fp8: an activation (1 silu, 2 gelu) goes with a gate, and only with one");
    if (c.tokens == 0 || c.width == 0) return SDT_OK;
    rc = check_in("quant_fp8", "x", c.x, c.tokens, c.x_row, c.width);
    if (!rc && c.gate) rc = check_in("quant_fp8", "gate", c.gate, c.tokens, c.gate_row, c.width);
    if (!rc) rc = check_out("quant_fp8", c.q, c.scales, c.tokens, c.width, c.q_row, c.s_row, c.s_block);
    if (rc) return rc;
    rc = check_apart("quant_fp8", {{"q", rows_of(c.q, c.tokens, c.q_row, c.width)}, {"scales", scales_of(c.scales, c.tokens, c.width, c.s_row, c.s_block)},
                                   {"x", rows_of(c.x, c.tokens, step_bytes(c.tokens, c.x_row, 2), 2 * c.width)}, {"gate", rows_of(c.gate, c.tokens, step_bytes(c.tokens, c.gate_row, 2), 2 * c.width)}}, 2);
    if (rc) return rc;
    rc = current_device(nullptr);
    if (rc) return rc;
    const uint32_t padded = static_cast<uint32_t>((c.width + 127) / 128 * 16);
    QuantArgs a{static_cast<const char *>(c.x), static_cast<const char *>(c.gate), step_bytes(c.tokens, c.x_row, 2), step_bytes(c.tokens, c.gate_row, 2),
                {static_cast<uint8_t *>(c.q), c.scales, c.q_row, c.s_row, c.s_block},
                static_cast<uint32_t>(c.tokens) * padded, static_cast<int>(c.width / 8), FastDiv::of(padded)};
    constexpr uint32_t per_cta = kQuantThreads * kQuantUnroll;
    const dim3 grid((a.total + per_cta - 1) / per_cta);
    const bool half = c.dtype == SDT_DTYPE_F16;
    auto kern = c.activation == kGateNone   ? (half ? quant_fp8_kernel<__half, 0> : quant_fp8_kernel<__nv_bfloat16, 0>)
                : c.activation == kGateSilu ? (half ? quant_fp8_kernel<__half, 1> : quant_fp8_kernel<__nv_bfloat16, 1>)
                                            : (half ? quant_fp8_kernel<__half, 2> : quant_fp8_kernel<__nv_bfloat16, 2>);
    const cudaError_t e = launch_kernel(kern, grid, dim3(kQuantThreads), 0, reinterpret_cast<cudaStream_t>(stream), 1, a);
    if (e != cudaSuccess) return fail(SDT_ERR_LAUNCH, "quant_fp8 launch failed: %s", cudaGetErrorString(e));
    return SDT_OK;
}

int rms_norm_fp8(const sdt_rms_norm_fp8 *call, sdt_stream_t stream) {
    clear_error();
    if (!call) return fail(SDT_ERR_NULL, "rms_norm_fp8: NULL call");
    sdt_rms_norm_fp8 c;
    memcpy(&c, call, sizeof c);
    int rc = check_size("rms_norm_fp8", c.tokens, c.width, kMaxNormWidth, c.dtype);
    if (rc) return rc;
    if (c.weight_dtype != c.dtype && c.weight_dtype != SDT_DTYPE_F32)
        return fail(SDT_ERR_ARG, "rms_norm_fp8: weight must have x's type or fp32 (dtype %d)", c.weight_dtype);
    if (!(c.eps >= 0.0f)) return fail(SDT_ERR_ARG, "rms_norm_fp8: eps must not be negative or NaN");
    if (c.tokens == 0 || c.width == 0) return SDT_OK;
    rc = check_in("rms_norm_fp8", "x", c.x, c.tokens, c.x_row, c.width);
    if (!rc) rc = check_in("rms_norm_fp8", "weight", c.weight, 1, 0, c.width);
    if (!rc && c.residual) rc = check_in("rms_norm_fp8", "residual", c.residual, c.tokens, c.r_row, c.width, true);
    if (!rc && c.out) rc = check_in("rms_norm_fp8", "out", c.out, c.tokens, c.o_row, c.width, true);
    if (!rc) rc = check_out("rms_norm_fp8", c.q, c.scales, c.tokens, c.width, c.q_row, c.s_row, c.s_block);
    if (rc) return rc;
    rc = check_apart("rms_norm_fp8", {{"q", rows_of(c.q, c.tokens, c.q_row, c.width)}, {"scales", scales_of(c.scales, c.tokens, c.width, c.s_row, c.s_block)},
                                      {"residual", rows_of(c.residual, c.tokens, step_bytes(c.tokens, c.r_row, 2), 2 * c.width)}, {"out", rows_of(c.out, c.tokens, step_bytes(c.tokens, c.o_row, 2), 2 * c.width)},
                                      {"x", rows_of(c.x, c.tokens, step_bytes(c.tokens, c.x_row, 2), 2 * c.width)},
                                      {"weight", rows_of(c.weight, 1, 0, (c.weight_dtype == SDT_DTYPE_F32 ? 4 : 2) * c.width)}}, 4);
    if (rc) return rc;
    NormArgs a{static_cast<const char *>(c.x), static_cast<char *>(c.residual), static_cast<const char *>(c.weight),
               static_cast<char *>(c.out), step_bytes(c.tokens, c.x_row, 2), step_bytes(c.tokens, c.r_row, 2), step_bytes(c.tokens, c.o_row, 2),
               {static_cast<uint8_t *>(c.q), c.scales, c.q_row, c.s_row, c.s_block},
               static_cast<int>(c.tokens), static_cast<int>(c.width / 8), 0, 1.0f / static_cast<float>(c.width), c.eps,
               c.weight_dtype == SDT_DTYPE_F32};
    // Few rows are spread over as many threads as they have pieces; many rows take four pieces a
    // thread, so that each has several loads on their way.  Rows of few threads share a CTA, a power
    // of two of threads each.
    DeviceInfo dev;
    rc = current_device(&dev);
    if (rc) return rc;
    const bool many = c.tokens >= 4 * dev.sm_count;
    int vpt = many ? 4 : 1, threads = 128;
    while (vpt < 8 && a.pieces > vpt * kNormThreads) vpt *= 2;
    while (vpt > 1 && a.pieces <= vpt * 8) vpt /= 2;  // a block's 16 pieces stay with 16 neighbours
    const int per = (a.pieces + vpt - 1) / vpt;
    if (per <= 32) a.per_row = a.pieces <= 8 ? 8 : per <= 16 ? 16 : 32;
    else a.per_row = threads = (per + 31) / 32 * 32;
    const int per_cta = threads / a.per_row;
    const int64_t groups = (c.tokens + per_cta - 1) / per_cta;
    const int resident = dev.sm_count * (norm_resident(vpt, c.residual != nullptr) / threads);
    const dim3 grid(static_cast<unsigned>(groups < resident ? groups : resident));
    auto kern = c.dtype == SDT_DTYPE_F16 ? norm_kernel<__half>(vpt, c.residual != nullptr) : norm_kernel<__nv_bfloat16>(vpt, c.residual != nullptr);
    const cudaError_t e = launch_kernel(kern, grid, dim3(threads), 0, reinterpret_cast<cudaStream_t>(stream), 1, a);
    if (e != cudaSuccess) return fail(SDT_ERR_LAUNCH, "rms_norm_fp8 launch failed: %s", cudaGetErrorString(e));
    return SDT_OK;
}

}  // extern "C"
