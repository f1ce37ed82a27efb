// rope.cu -- rotary positions: each pair (x, y) of a head's first `rotary` values turns by
// position * frequency of its pair, and is multiplied by a magnitude.
//
// The angle in turns is position * f modulo 1, f = frequency / (2 pi) as a 64-bit binary
// fraction: the product of two 64-bit integers wraps modulo one turn by itself, so a position
// of a million turns as exactly as position one (fp32 angles are off by 0.06 rad there).  The
// fraction is cut to 32 bits and rounded to fp32 (together at most 2^-25 turns off), and sine
// and cosine of it are taken once per pair and token and used for several heads.
//
// What bounds it: memory (each value is read and written once) for prompts, the launch for a
// decode step.  A thread turns V pairs, V values (at most 16 bytes) at a time from each place;
// V is what the width and the caller's alignment allow.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>
#include <type_traits>

#include "launch.cuh"
#include "overlap.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace sdt {

constexpr int kRopeThreads = 128;
constexpr int kRopeHeads = 4;  // heads a thread turns by the same angles

struct RopeArgs {
    const char *in[2];   // queries, keys
    char *out[2];
    int64_t in_token[2], in_head[2], out_token[2], out_head[2];  // bytes
    const void *positions;
    const uint64_t *turns;   // per pair: turns per position, as a fraction of 2^64
    int heads[2];
    int groups[2];           // groups of HP heads
    int rotary, pairs_items, items;  // items of a head: V pairs each, then V-pairs to copy
    int pos64;
    uint32_t total;          // tokens * groups * items
    FastDiv per_token, per_group;
    float magnitude, direction;
};

template <int V>
struct Vec {
    using type = std::conditional_t<V == 8, uint4, std::conditional_t<V == 4, uint2, std::conditional_t<V == 2, uint32_t, uint16_t>>>;
};

template <typename T>
__device__ __forceinline__ float value_of16(uint16_t b) {
    if constexpr (std::is_same_v<T, __half>) return __half2float(__ushort_as_half(b));
    else return __uint_as_float(static_cast<uint32_t>(b) << 16);
}
template <typename T>
__device__ __forceinline__ uint16_t bits_of16(float f) {
    if constexpr (std::is_same_v<T, __half>) return __half_as_ushort(__float2half_rn(f));
    else return __bfloat16_as_ushort(__float2bfloat16_rn(f));
}

template <typename T, int V, int HP, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
    using Vt = typename Vec<V>::type;
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t i = blockIdx.x * kRopeThreads + threadIdx.x;
    if (i >= a.total) return;
    const uint32_t token = a.per_token.div(i);
    const uint32_t rest = i - token * a.per_token.d;
    uint32_t group = a.per_group.div(rest);
    const int item = static_cast<int>(rest - group * a.per_group.d);
    const int side = group >= static_cast<uint32_t>(a.groups[0]) ? 1 : 0;
    if (side) group -= a.groups[0];
    const int h0 = static_cast<int>(group) * HP;
    const bool turn = item < a.pairs_items;
    // where the item's two vectors lie in a head
    int at0, at1;
    if (!turn) {
        at0 = a.rotary + (item - a.pairs_items) * 2 * V;
        at1 = at0 + V;
    } else if (INTERLEAVED) {
        at0 = item * 2 * V;
        at1 = at0 + V;
    } else {
        at0 = item * V;
        at1 = a.rotary / 2 + item * V;
    }
    const char *in = a.in[side] + token * a.in_token[side] + h0 * a.in_head[side];
    char *out = a.out[side] + token * a.out_token[side] + h0 * a.out_head[side];
    Vt x[HP], y[HP];
#pragma unroll
    for (int h = 0; h < HP; ++h)
        if (h0 + h < a.heads[side]) {
            x[h] = *reinterpret_cast<const Vt *>(in + h * a.in_head[side] + at0 * 2);
            y[h] = *reinterpret_cast<const Vt *>(in + h * a.in_head[side] + at1 * 2);
        }
    if (turn) {
        const int64_t pos = a.pos64 ? static_cast<const int64_t *>(a.positions)[token] : static_cast<const int32_t *>(a.positions)[token];
        float c[V], s[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint64_t t = static_cast<uint64_t>(pos) * a.turns[item * V + j];
            // in half turns, -1 .. 1
            const float half_turns = static_cast<float>(static_cast<int32_t>(t >> 32)) * 4.656612873077393e-10f;
            sincospif(half_turns, &s[j], &c[j]);
            c[j] *= a.magnitude;
            s[j] *= a.magnitude * a.direction;
        }
#pragma unroll
        for (int h = 0; h < HP; ++h) {
            uint16_t e[2 * V];
            memcpy(e, &x[h], 2 * V);
            memcpy(e + V, &y[h], 2 * V);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int p = INTERLEAVED ? 2 * j : j, r = INTERLEAVED ? 2 * j + 1 : V + j;
                const float u = value_of16<T>(e[p]), v = value_of16<T>(e[r]);
                e[p] = bits_of16<T>(fmaf(u, c[j], -(v * s[j])));
                e[r] = bits_of16<T>(fmaf(v, c[j], u * s[j]));
            }
            memcpy(&x[h], e, 2 * V);
            memcpy(&y[h], e + V, 2 * V);
        }
    }
#pragma unroll
    for (int h = 0; h < HP; ++h)
        if (h0 + h < a.heads[side]) {
            *reinterpret_cast<Vt *>(out + h * a.out_head[side] + at0 * 2) = x[h];
            *reinterpret_cast<Vt *>(out + h * a.out_head[side] + at1 * 2) = y[h];
        }
}

template <typename T, int V>
static auto kernel_for(bool interleaved) {
    return interleaved ? rope_kernel<T, V, kRopeHeads, true> : rope_kernel<T, V, kRopeHeads, false>;
}
template <typename T>
static auto kernel_for(int v, bool interleaved) {
    return v == 8   ? kernel_for<T, 8>(interleaved)
           : v == 4 ? kernel_for<T, 4>(interleaved)
           : v == 2 ? kernel_for<T, 2>(interleaved)
                    : kernel_for<T, 1>(interleaved);
}

constexpr int64_t kRopeMaxHeads = 65535, kRopeMaxDim = 65536, kRopeMaxStride = int64_t(1) << 32;

// An output whose tokens and heads do not overlap one another.
static bool apart(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t d) {
    if (n0 <= 1) return n1 <= 1 || s1 >= d;
    if (n1 <= 1) return s0 >= d;
    if (s0 < s1) return s0 >= d && s1 >= (n0 - 1) * s0 + d;
    return s1 >= d && s0 >= (n1 - 1) * s1 + d;
}

static int check_rope_side(const char *what, const void *in, const void *out, int64_t tokens, int64_t heads, int64_t d, int64_t it,
                           int64_t ih, int64_t ot, int64_t oh) {
    if (!in || !out) return fail(SDT_ERR_NULL, "rope_qk: %s or its output is NULL", what);
    if (!aligned(in, 2) || !aligned(out, 2)) return fail(SDT_ERR_ALIGN, "rope_qk: %s and its output must be 2-byte aligned", what);
    for (int64_t s : {it, ih, ot, oh})
        if (s < 0 || s > kRopeMaxStride) return fail(SDT_ERR_ARG, "rope_qk: strides of %s must be in 0 .. 2^32", what);
    if (!apart(tokens, ot, heads, oh, d)) return fail(SDT_ERR_ARG, "rope_qk: tokens and heads of the output of %s must not overlap", what);
    const bool itself = in == out && it == ot && ih == oh;
    if (!itself && overlap({in, tokens, 2 * it, heads, 2 * ih, 2 * d}, {out, tokens, 2 * ot, heads, 2 * oh, 2 * d}))
        return fail(SDT_ERR_ARG, "rope_qk: the output of %s must be %s itself or lie apart from it", what, what);
    return SDT_OK;
}

}  // namespace sdt

using namespace sdt;

extern "C" int rope_qk(const sdt_rope_qk *call, sdt_stream_t stream) {
    clear_error();
    if (!call) return fail(SDT_ERR_NULL, "rope_qk: NULL call");
    sdt_rope_qk c;
    memcpy(&c, call, sizeof c);
    if (c.dtype != SDT_DTYPE_F16 && c.dtype != SDT_DTYPE_BF16) return fail(SDT_ERR_ARG, "rope_qk: dtype must be fp16 or bf16 (got %d)", c.dtype);
    if (c.head_dim < 0 || c.head_dim > kRopeMaxDim || c.rotary < 0 || c.rotary > c.head_dim || c.rotary % 2 || (c.head_dim - c.rotary) % 2)
        return fail(SDT_ERR_SHAPE, "rope_qk: head_dim and rotary must be even, rotary at most head_dim (got %lld and %lld)",
                    (long long)c.head_dim, (long long)c.rotary);
    if (c.tokens < 0 || c.q_heads < 0 || c.k_heads < 0 || c.q_heads > kRopeMaxHeads || c.k_heads > kRopeMaxHeads)
        return fail(SDT_ERR_SHAPE, "rope_qk: tokens and heads must not be negative, heads at most %lld", (long long)kRopeMaxHeads);
    if (c.position_bytes != 4 && c.position_bytes != 8) return fail(SDT_ERR_ARG, "rope_qk: positions must be 32 or 64 bits wide");
    const int64_t heads = c.q_heads + c.k_heads;
    if (c.tokens == 0 || heads == 0 || c.head_dim == 0) return SDT_OK;
    if (c.tokens > INT32_MAX / (heads * c.head_dim)) return fail(SDT_ERR_SHAPE, "rope_qk: tokens * heads * head_dim must be below 2^31");
    int64_t step[8] = {c.q_token, c.q_head, c.k_token, c.k_head, c.qo_token, c.qo_head, c.ko_token, c.ko_head};
    for (int i = 0; i < 8; ++i)  // a dimension of one never steps: its stride may be anything
        if ((i % 2 ? (i % 4 == 1 ? c.q_heads : c.k_heads) : c.tokens) == 1) step[i] = 0;
    int rc = c.q_heads ? check_rope_side("q", c.q, c.q_out, c.tokens, c.q_heads, c.head_dim, step[0], step[1], step[4], step[5]) : SDT_OK;
    if (!rc && c.k_heads) rc = check_rope_side("k", c.k, c.k_out, c.tokens, c.k_heads, c.head_dim, step[2], step[3], step[6], step[7]);
    const auto side = [&](const void *p, int64_t heads, int i) {
        return Stretches{p, c.tokens, 2 * step[i], heads, 2 * step[i + 1], 2 * c.head_dim};
    };
    const Stretches qo = side(c.q_out, c.q_heads, 4), ko = side(c.k_out, c.k_heads, 6);
    if (!rc && c.q_heads && c.k_heads && (overlap(qo, ko) || overlap(qo, side(c.k, c.k_heads, 2)) || overlap(ko, side(c.q, c.q_heads, 0))))
        rc = fail(SDT_ERR_ARG, "rope_qk: the output of one side must not overlap the other side's tensors");
    if (rc) return rc;
    if (c.rotary && (!c.positions || !c.turns)) return fail(SDT_ERR_NULL, "rope_qk: positions or turns is NULL");
    if (!aligned(c.positions, static_cast<uintptr_t>(c.position_bytes)) || !aligned(c.turns, 8))
        return fail(SDT_ERR_ALIGN, "rope_qk: positions and turns must be aligned to their elements");
    for (const Stretches &in : {rows_of(c.positions, 1, 0, c.tokens * c.position_bytes), rows_of(c.turns, 1, 0, c.rotary / 2 * 8)})
        if ((c.q_heads && overlap(qo, in)) || (c.k_heads && overlap(ko, in))) return fail(SDT_ERR_ARG, "rope_qk: an output overlaps positions or turns");
    rc = current_device(nullptr);
    if (rc) return rc;
    const bool in_place = (!c.q_heads || c.q == c.q_out) && (!c.k_heads || c.k == c.k_out);  // then the rest of a head stays as it is
    RopeArgs a;
    memset(&a, 0, sizeof a);
    const void *in[2] = {c.q, c.k};
    void *out[2] = {c.q_out, c.k_out};
    const int64_t count[2] = {c.q_heads, c.k_heads};
    int v = 8;
    const auto fits = [&](int64_t s) { while (s % v) v /= 2; };
    fits(c.rotary / 2);
    if (!in_place) fits((c.head_dim - c.rotary) / 2);
    for (int s = 0; s < 2; ++s) {
        a.in[s] = static_cast<const char *>(in[s]);
        a.out[s] = static_cast<char *>(out[s]);
        a.heads[s] = static_cast<int>(count[s]);
        if (!count[s]) continue;
        a.in_token[s] = step[2 * s] * 2;
        a.in_head[s] = step[2 * s + 1] * 2;
        a.out_token[s] = step[4 + 2 * s] * 2;
        a.out_head[s] = step[5 + 2 * s] * 2;
        for (int64_t x : {step[2 * s], step[2 * s + 1], step[4 + 2 * s], step[5 + 2 * s]}) fits(x);
        fits(static_cast<int64_t>(reinterpret_cast<uintptr_t>(in[s]) / 2));
        fits(static_cast<int64_t>(reinterpret_cast<uintptr_t>(out[s]) / 2));
    }
    a.positions = c.positions;
    a.turns = c.turns;
    a.pos64 = c.position_bytes == 8;
    a.rotary = static_cast<int>(c.rotary);
    a.pairs_items = static_cast<int>(c.rotary / 2 / v);
    a.items = a.pairs_items + (in_place ? 0 : static_cast<int>((c.head_dim - c.rotary) / 2 / v));
    a.magnitude = c.magnitude;
    a.direction = c.inverse ? -1.0f : 1.0f;
    if (a.items == 0) return SDT_OK;
    a.groups[0] = static_cast<int>((c.q_heads + kRopeHeads - 1) / kRopeHeads);
    a.groups[1] = static_cast<int>((c.k_heads + kRopeHeads - 1) / kRopeHeads);
    const uint32_t per_token = static_cast<uint32_t>(a.groups[0] + a.groups[1]) * static_cast<uint32_t>(a.items);
    a.total = static_cast<uint32_t>(c.tokens) * per_token;
    a.per_token = FastDiv::of(per_token);
    a.per_group = FastDiv::of(static_cast<uint32_t>(a.items));
    const dim3 grid((a.total + kRopeThreads - 1) / kRopeThreads);
    auto kern = c.dtype == SDT_DTYPE_F16 ? kernel_for<__half>(v, c.interleaved != 0) : kernel_for<__nv_bfloat16>(v, c.interleaved != 0);
    const cudaError_t e = launch_kernel(kern, grid, dim3(kRopeThreads), 0, reinterpret_cast<cudaStream_t>(stream), 1, a);
    if (e != cudaSuccess) return fail(SDT_ERR_LAUNCH, "rope_qk launch failed: %s", cudaGetErrorString(e));
    return SDT_OK;
}
