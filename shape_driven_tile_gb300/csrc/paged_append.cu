// paged_append.cu -- new keys and values into a paged cache: cache[slot[t]] = x[t], as they
// are or as q8 (int8 and one fp16 scale per 32 values, gemv_m1_q8's weight format).
//
// q8 of one group of 32 values: s = fp16(max|x| * fl32(1/127)) (at most 65504), q = x / s
// rounded to the nearest integer, ties to even, within +-127; s = 0 gives q = 0, and a NaN
// is stored as 0.  Divisions take more time than the memory traffic (8191 tokens of 8 heads of
// 128: 23.8 us with them, 15.0 without), and x times fl(1/s) is enough: x has at most 11
// bits, is at least s/2 where a tie can be, and s has 11, so x/s is a tie exactly or at least
// 2^-12 away from one, while the product is off by 2^-15 at most.  Adding and taking away
// 1536 = 1.5 * 2^10 rounds it to a multiple of 2^-13, which puts a tie back where it belongs;
// adding 1.5 * 2^23 then rounds to the integer, ties to even, in the last bits.
//
// What bounds it: HBM for prompts in 16 bits (each value read once and written once: 16384
// tokens of 8 heads of 128 take 21.6 us, 92 % of the measured copy rate), arithmetic in q8
// (27.4 us; issue slots 82 % busy), the launch for a decode step's few tokens (64 tokens of
// 32 heads: 1.7 us).  A thread moves 16-byte pieces of 8 values; four neighbouring
// threads hold one q8 group and find its maximum by two shuffles, so q8 needs no second
// pass and no shared memory.
#include <type_traits>

#include "launch.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace sdt {

constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 4;  // 16-byte loads in flight per thread

struct AppendArgs {
    const char *x[2];          // keys, values
    int64_t x_token[2], x_head[2];  // bytes
    KvRows rows[2];
    ScaleRows scales[2];
    const int64_t *slots;
    int64_t num_slots_cache;   // pages * page size
    int tokens;
    FastDiv per_token, per_head, page;  // 16-byte pieces of 8 values per token (all heads), per head
    int *status;
};

template <typename T>
__device__ __forceinline__ void to_f32(const uint4 &v, float (&f)[8]) {
    const T *p = reinterpret_cast<const T *>(&v);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = static_cast<float>(p[i]);
}

// A 16-bit value's bits (sign bit clear) as a number, and back (exact for values of T).
template <typename T>
__device__ __forceinline__ float value_of(uint32_t bits) {
    if constexpr (std::is_same_v<T, __half>) return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
    else return __uint_as_float(bits << 16);
}
template <typename T>
__device__ __forceinline__ uint32_t bits_of(float x) {
    if constexpr (std::is_same_v<T, __half>) return __half_as_ushort(__float2half_rn(x));
    else return __float_as_uint(x) >> 16;
}

template <typename T, bool Q8>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const AppendArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int kv = blockIdx.y;
    const int64_t total = static_cast<int64_t>(a.tokens) * a.per_token.d;
    const int64_t base = (static_cast<int64_t>(blockIdx.x) * kAppendThreads * kAppendUnroll) + threadIdx.x;
    uint4 val[kAppendUnroll];
    int64_t slot[kAppendUnroll];
    uint32_t head[kAppendUnroll], piece[kAppendUnroll];
#pragma unroll
    for (int u = 0; u < kAppendUnroll; ++u) {
        const int64_t i = base + u * kAppendThreads;
        slot[u] = -1;
        val[u] = make_uint4(0, 0, 0, 0);
        if (i >= total) continue;
        const uint32_t t = a.per_token.div(static_cast<uint32_t>(i));
        const uint32_t rest = static_cast<uint32_t>(i) - t * a.per_token.d;
        head[u] = a.per_head.div(rest);
        piece[u] = rest - head[u] * a.per_head.d;
        slot[u] = a.slots[t];
        val[u] = *reinterpret_cast<const uint4 *>(a.x[kv] + t * a.x_token[kv] + head[u] * a.x_head[kv] + piece[u] * 16);
    }
#pragma unroll
    for (int u = 0; u < kAppendUnroll; ++u) {
        if (slot[u] >= a.num_slots_cache) {
            paged_status(a.status, kSiteSlot);
            slot[u] = -1;
        }
        const bool write = slot[u] >= 0;
        const uint32_t s = write ? static_cast<uint32_t>(slot[u]) : 0;
        const uint32_t page = a.page.div(s), off = s - page * a.page.d;
        if constexpr (!Q8) {
            if (write)
                *reinterpret_cast<uint4 *>(a.rows[kv].at(page, off, head[u]) + piece[u] * 16) = val[u];
        } else {
            // the group's largest |x| by its bits: they order as the values do, NaNs above infinity
            const uint32_t *w = reinterpret_cast<const uint32_t *>(&val[u]);
            uint32_t most = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
            most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, 2));
            most = max(most & 0xffffu, most >> 16);
            float f[8];
            to_f32<T>(val[u], f);
            constexpr uint32_t inf = std::is_same_v<T, __half> ? 0x7c00u : 0x7f80u;
            if (__any_sync(0xffffffffu, most > inf)) {  // NaNs: they count as 0
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    f[i] = f[i] == f[i] ? f[i] : 0.f;
                    top = fmaxf(top, fabsf(f[i]));
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                most = bits_of<T>(top);
            }
            const __half hs = __float2half_rn(fminf(value_of<T>(most) * (1.0f / 127.0f), 65504.0f));
            const float sc = __half2float(hs), inv = sc > 0.f ? __frcp_rn(sc) : 0.f;
            uint32_t r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = fminf(fmaxf(f[i] * inv, -127.f), 127.f);
                r[i] = __float_as_uint(((y + 1536.f) - 1536.f) + 12582912.f);
            }
            const uint32_t q[2] = {__byte_perm(__byte_perm(r[0], r[1], 0x0040), __byte_perm(r[2], r[3], 0x0040), 0x5410),
                                   __byte_perm(__byte_perm(r[4], r[5], 0x0040), __byte_perm(r[6], r[7], 0x0040), 0x5410)};
            if (write) {
                *reinterpret_cast<uint2 *>(a.rows[kv].at(page, off, head[u]) + piece[u] * 8) =
                    make_uint2(q[0], q[1]);
                if ((piece[u] & 3) == 0)
                    *reinterpret_cast<__half *>(a.scales[kv].at(page, off, head[u]) + (piece[u] >> 2) * 2) = hs;
            }
        }
    }
}

static bool stride_ok(int64_t s, int64_t mult) { return s >= 0 && s % mult == 0; }

static int check_rows(const char *what, const void *p, int64_t sp, int64_t st, int64_t sh, int64_t bytes_el, int64_t align) {
    if (!p) return fail(SDT_ERR_NULL, "paged cache: %s is NULL", what);
    if (!aligned(p, align)) return fail(SDT_ERR_ALIGN, "paged cache: %s must be %lld-byte aligned", what, (long long)align);
    const int64_t mult = align / bytes_el, most = int64_t(UINT32_MAX) * 4 / bytes_el;  // strides fit 32 bits in units of 4 bytes
    for (int64_t s : {sp, st, sh})
        if (!stride_ok(s, mult) || s > most)
            return fail(SDT_ERR_ARG, "paged cache: strides of %s must be multiples of %lld elements, 0 to 16 GiB", what, (long long)mult);
    return SDT_OK;
}

int check_cache(const sdt_paged_cache *c) {
    if (!c) return fail(SDT_ERR_NULL, "paged cache: NULL descriptor");
    if (c->dtype != SDT_DTYPE_F16 && c->dtype != SDT_DTYPE_BF16 && c->dtype != SDT_DTYPE_Q8)
        return fail(SDT_ERR_ARG, "paged cache: unknown dtype %d", c->dtype);
    const bool q8 = c->dtype == SDT_DTYPE_Q8;
    const int step = q8 ? 64 : 8;
    if (c->head_dim < step || c->head_dim > kPagedMaxHeadDim || c->head_dim % step)
        return fail(SDT_ERR_SHAPE, "paged cache: head_dim must be a multiple of %d up to %d (got %lld)", step, kPagedMaxHeadDim,
                    (long long)c->head_dim);
    if (c->num_pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->kv_heads > 65535 || c->page_size > INT32_MAX ||
        c->num_pages > INT32_MAX / c->page_size)
        return fail(SDT_ERR_SHAPE, "paged cache: pages, page size and heads must be positive, heads at most 65535 and pages * page size < 2^31");
    int rc = check_rows("k", c->k, c->k_page, c->k_token, c->k_head, q8 ? 1 : 2, 16);
    if (!rc) rc = check_rows("v", c->v, c->v_page, c->v_token, c->v_head, q8 ? 1 : 2, 16);
    const int row = c->head_dim == 128 ? 8 : 4;  // scales are copied in pieces of this size
    if (!rc && q8) rc = check_rows("k_scales", c->k_scales, c->ks_page, c->ks_token, c->ks_head, 2, row);
    if (!rc && q8) rc = check_rows("v_scales", c->v_scales, c->vs_page, c->vs_token, c->vs_head, 2, row);
    return rc;
}

template <int UNIT>
static PagedRows<UNIT> rows_of(void *p, int64_t sp, int64_t st, int64_t sh, int el) {
    auto u = [&](int64_t s) { return static_cast<uint32_t>(s * el / UNIT); };
    return {static_cast<char *>(p), u(sp), u(st), u(sh)};
}
static int width(const sdt_paged_cache &c) { return c.dtype == SDT_DTYPE_Q8 ? 1 : 2; }
KvRows rows_k(const sdt_paged_cache &c) { return rows_of<16>(c.k, c.k_page, c.k_token, c.k_head, width(c)); }
KvRows rows_v(const sdt_paged_cache &c) { return rows_of<16>(c.v, c.v_page, c.v_token, c.v_head, width(c)); }
ScaleRows rows_ks(const sdt_paged_cache &c) { return rows_of<4>(c.k_scales, c.ks_page, c.ks_token, c.ks_head, 2); }
ScaleRows rows_vs(const sdt_paged_cache &c) { return rows_of<4>(c.v_scales, c.vs_page, c.vs_token, c.vs_head, 2); }

}  // namespace sdt

using namespace sdt;

extern "C" int paged_append(int64_t tokens, const void *k, int64_t k_token, int64_t k_head, const void *v, int64_t v_token,
                            int64_t v_head, int dtype, const int64_t *slots, const sdt_paged_cache *cache,
                            sdt_stream_t stream) {
    clear_error();
    int rc = check_cache(cache);
    if (rc) return rc;
    if (dtype != SDT_DTYPE_F16 && dtype != SDT_DTYPE_BF16) return fail(SDT_ERR_ARG, "paged_append: dtype must be fp16 or bf16 (got %d)", dtype);
    const bool q8 = cache->dtype == SDT_DTYPE_Q8;
    if (!q8 && cache->dtype != dtype) return fail(SDT_ERR_ARG, "paged_append: a 16-bit cache takes values of its own type");
    const int64_t per_head = cache->head_dim / 8, per_token = per_head * cache->kv_heads;
    if (tokens < 0 || tokens > (INT32_MAX - kAppendThreads * kAppendUnroll) / per_token)
        return fail(SDT_ERR_SHAPE, "paged_append: tokens * kv_heads * head_dim must be in 0 .. 2^34 (got %lld tokens)", (long long)tokens);
    if (tokens == 0) return SDT_OK;
    if (tokens == 1) k_token = v_token = 0;  // a dimension of one never steps: its stride may be anything
    if (cache->kv_heads == 1) k_head = v_head = 0;
    if (!k || !v || !slots) return fail(SDT_ERR_NULL, "paged_append: NULL pointer");
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))
        return fail(SDT_ERR_ALIGN, "paged_append: k and v must be 16-byte aligned, slots 8-byte");
    if (!stride_ok(k_token, 8) || !stride_ok(k_head, 8) || !stride_ok(v_token, 8) || !stride_ok(v_head, 8))
        return fail(SDT_ERR_ARG, "paged_append: strides of k and v must be non-negative multiples of 8 elements");
    int *status = nullptr;
    rc = status_word(&status);
    if (rc) return rc;
    AppendArgs a{{static_cast<const char *>(k), static_cast<const char *>(v)},
                 {k_token * 2, v_token * 2},
                 {k_head * 2, v_head * 2},
                 {rows_k(*cache), rows_v(*cache)},
                 {rows_ks(*cache), rows_vs(*cache)},
                 slots,
                 cache->num_pages * cache->page_size,
                 static_cast<int>(tokens),
                 FastDiv::of(static_cast<uint32_t>(per_token)),
                 FastDiv::of(static_cast<uint32_t>(per_head)),
                 FastDiv::of(static_cast<uint32_t>(cache->page_size)),
                 status};
    const int64_t per_cta = kAppendThreads * kAppendUnroll;
    const dim3 grid(static_cast<unsigned>((tokens * per_token + per_cta - 1) / per_cta), 2);
    auto kern = !q8 ? paged_append_kernel<__half, false>
                    : dtype == SDT_DTYPE_F16 ? paged_append_kernel<__half, true> : paged_append_kernel<__nv_bfloat16, true>;
    cudaError_t e = launch_kernel(kern, grid, dim3(kAppendThreads), 0, reinterpret_cast<cudaStream_t>(stream), 1, a);
    if (e != cudaSuccess) return fail(SDT_ERR_LAUNCH, "paged_append launch failed: %s", cudaGetErrorString(e));
    return SDT_OK;
}
