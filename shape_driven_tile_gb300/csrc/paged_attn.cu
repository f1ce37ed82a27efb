// paged_attn.cu -- paged_attn_m1: argument checks and dispatch of the paged attention kernel.
#include <algorithm>

#include "launch.cuh"
#include "paged_attn.cuh"
#include "paged_attn_plan.cuh"

namespace sdt {

// Joins the pieces of split items: a CTA takes 64 columns of one row, 16 groups of 16 threads every
// sixteenth piece, and meets at the end in the order of the groups.  The pieces lie in L2 and one CTA's
// loads in flight bound the join, so it is spread over rows and columns: 32 query heads on one key head,
// 32768 tokens, 15.2 us for both kernels (36.0 joined by one CTA an item).
constexpr int kJoinGroups = 16, kJoinWide = 16, kJoinThreads = kJoinGroups * kJoinWide;
constexpr int kJoinPieces = 1024;  // no grid of four-warp CTAs is larger

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) paged_attn_join_kernel(const PagedAttnArgs p, int width, int rows) {
    __shared__ float weight[kJoinPieces];
    __shared__ float red[2][kJoinThreads / 32];
    __shared__ float4 meet[kJoinThreads];
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, item = blockIdx.y;
    const int parts = width / 64, r = blockIdx.x / parts, part = blockIdx.x % parts;
    const int hb = item % p.head_blocks, h = item / p.head_blocks % p.kv_heads, b = item / p.head_blocks / p.kv_heads;
    const int2 split = p.split[item];
    const int n = min(split.y, kJoinPieces);
    if (n == 0 || hb * rows + r >= p.group) return;
    const int slot = rows * (width + 2);  // floats
    // piece 0 lies in its CTA's second slot, the others in their first
    auto at = [&](int i) { return p.partials + static_cast<size_t>(2 * (split.x + i) + (i == 0 ? 1 : 0)) * slot; };
    float M = -INFINITY, L = 0.f;
    for (int i = tid; i < n; i += kJoinThreads) {
        weight[i] = at(i)[rows * width + r];
        M = fmaxf(M, weight[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) red[0][warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) M = fmaxf(M, red[0][w]);
    for (int i = tid; i < n; i += kJoinThreads) {
        const float w = weight[i] == M ? 1.f : pow2(weight[i] - M);  // (both -inf: zeros either way)
        L += at(i)[rows * (width + 1) + r] * w;
        weight[i] = w;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) red[1][warp] = L;
    __syncthreads();
    L = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) L += red[1][w];
    const int group = tid / kJoinWide, col = part * 64 + (tid % kJoinWide) * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = group; i < n; i += kJoinGroups) {
        const float4 v = *reinterpret_cast<const float4 *>(at(i) + r * width + col);
        const float w = weight[i];
        acc = make_float4(acc.x + v.x * w, acc.y + v.y * w, acc.z + v.z * w, acc.w + v.w * w);
    }
    meet[tid] = acc;
    __syncthreads();
    if (group > 0) return;
    for (int g = 1; g < kJoinGroups; ++g) {
        const float4 v = meet[g * kJoinWide + tid];
        acc = make_float4(acc.x + v.x, acc.y + v.y, acc.z + v.z, acc.w + v.w);
    }
    const int head = h * p.group + hb * rows + r;
    const float inv = L > 0.f ? reciprocal(L) : L == 0.f ? 0.f : L;  // no key: zeros; a NaN sum stays NaN
    if (col < p.head_dim)
        *reinterpret_cast<uint2 *>(p.out + b * p.o_batch + head * p.o_head + col * 2) =
            make_uint2(pack2<T>(acc.x * inv, acc.y * inv), pack2<T>(acc.z * inv, acc.w * inv));
    if (p.lse && col == 0)
        p.lse[static_cast<int64_t>(b) * p.kv_heads * p.group + head] = L == 0.f ? -INFINITY : M * 0.6931471805599453f + logf(L);
}

cudaError_t launch_paged_attn_join(const PagedAttnArgs &a, bool f16, int width, int rows, int items, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(std::min(a.group, rows) * (width / 64)), static_cast<unsigned>(items));
    return launch_kernel(f16 ? paged_attn_join_kernel<__half> : paged_attn_join_kernel<__nv_bfloat16>, grid, dim3(kJoinThreads), 0,
                         stream, 1, a, width, rows);
}

}  // namespace sdt

using namespace sdt;

static constexpr size_t kSplitBytes = size_t(kAttnSplitItems) * sizeof(int2);
static constexpr size_t kCounterBytes = size_t(1) << 20;  // the counter region of the split-K workspaces
static constexpr int64_t kMaxTokens = INT32_MAX - 1024;   // a row's tokens; key indices run past them by a unit at most

// Workspace bytes of any call with `group` query heads per key head: of the variants that it may
// take, whatever the batch.
static size_t workspace_for(int64_t group, int64_t head_dim, int sm_count) {
    size_t most = 0;
    for (int64_t items : {int64_t(1), INT64_MAX}) {
        const PagedAttnVariant v = paged_attn_variant(group, items, head_dim, false, sm_count);
        const size_t slot = static_cast<size_t>(8 * v.nh * v.wh) * (paged_attn_width(head_dim) + 2) * sizeof(float);
        most = std::max(most, 2 * static_cast<size_t>(sm_count) * paged_attn_ctas(v.nw) * slot);  // two pieces a CTA
    }
    return kCounterBytes + kSplitBytes + most;
}

extern "C" {

size_t sdt_paged_attn_workspace_bytes(int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
    DeviceInfo dev;
    if (kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads || head_dim < 8 || head_dim > kPagedMaxHeadDim) {
        fail(SDT_ERR_SHAPE, "sdt_paged_attn_workspace_bytes: bad sizes");
        return 0;
    }
    return current_device(&dev) ? 0 : workspace_for(q_heads / kv_heads, head_dim, dev.sm_count);
}

int paged_attn_m1(const sdt_paged_attn *call, sdt_stream_t stream) {
    clear_error();
    if (!call) return fail(SDT_ERR_NULL, "paged_attn_m1: NULL arguments");
    const auto &[q, out, lse, table, lens, cache, workspace, batch, q_heads, q_batch, q_head, out_batch, out_head, table_stride,
                 max_pages, window, workspace_bytes, scale, dtype] = *call;
    int rc = check_cache(cache);
    if (rc) return rc;
    if (dtype != SDT_DTYPE_F16 && dtype != SDT_DTYPE_BF16) return fail(SDT_ERR_ARG, "paged_attn_m1: dtype must be fp16 or bf16 (got %d)", dtype);
    const bool q8 = cache->dtype == SDT_DTYPE_Q8;
    if (!q8 && cache->dtype != dtype) return fail(SDT_ERR_ARG, "paged_attn_m1: a 16-bit cache takes queries of its own type");
    const int64_t kvh = cache->kv_heads;
    if (batch < 0 || batch > (1 << 20) || q_heads < kvh || q_heads % kvh || q_heads > 65536)
        return fail(SDT_ERR_SHAPE, "paged_attn_m1: batch in 0 .. 2^20, q_heads a multiple of the cache's %lld heads up to 65536 (got %lld, %lld)",
                    (long long)kvh, (long long)batch, (long long)q_heads);
    if (max_pages < 0 || (max_pages && cache->page_size > kMaxTokens / max_pages))
        return fail(SDT_ERR_SHAPE, "paged_attn_m1: a table row must hold 0 .. %lld tokens", (long long)kMaxTokens);
    if (table_stride < max_pages) return fail(SDT_ERR_ARG, "paged_attn_m1: table rows of %lld entries, %lld apart", (long long)max_pages, (long long)table_stride);
    if (window < 0) return fail(SDT_ERR_ARG, "paged_attn_m1: window must be >= 0 (got %lld)", (long long)window);
    if (batch == 0) return SDT_OK;
    if (!q || !out || !lens || !workspace || (max_pages && !table)) return fail(SDT_ERR_NULL, "paged_attn_m1: NULL pointer");
    if (!aligned(q, 16) || !aligned(out, 8) || !aligned(lens, 4) || !aligned(table, 4) || !aligned(lse, 4) || !aligned(workspace, 256))
        return fail(SDT_ERR_ALIGN, "paged_attn_m1: q must be 16-byte, out 8-byte, lens, table and lse 4-byte, workspace 256-byte aligned");
    if (q_batch % 8 || q_head % 8 || out_batch % 4 || out_head % 4)
        return fail(SDT_ERR_ARG, "paged_attn_m1: strides of q must be multiples of 8, of out of 4 elements");
    DeviceInfo dev;
    rc = current_device(&dev);
    if (rc) return rc;
    const size_t need = workspace_for(q_heads / kvh, cache->head_dim, dev.sm_count);
    if (workspace_bytes < 0 || static_cast<size_t>(workspace_bytes) < need)
        return fail(SDT_ERR_ARG, "paged_attn_m1: workspace of %lld bytes, %zu needed", (long long)workspace_bytes, need);
    int *status = nullptr;
    rc = status_word(&status);
    if (rc) return rc;

    const int64_t cap = max_pages * cache->page_size;
    PagedAttnLaunch l{paged_attn_variant(q_heads / kvh, batch * kvh, cache->head_dim, q8, dev.sm_count), q8, dev.device, dev.sm_count,
                      window > 0 && window < cap ? window : cap, reinterpret_cast<cudaStream_t>(stream)};
    PagedAttnArgs a{};
    a.q = static_cast<const char *>(q);
    a.out = static_cast<char *>(out);
    a.lse = lse;
    a.q_batch = q_batch * 2;
    a.q_head = q_head * 2;
    a.o_batch = out_batch * 2;
    a.o_head = out_head * 2;
    a.k = rows_k(*cache);
    a.v = rows_v(*cache);
    a.ks = rows_ks(*cache);
    a.vs = rows_vs(*cache);
    a.table = table;
    a.table_stride = table_stride;
    a.lens = lens;
    a.batch = static_cast<int>(batch);
    a.kv_heads = static_cast<int>(kvh);
    a.group = static_cast<int>(q_heads / kvh);
    const int heads = 8 * l.variant.nh * l.variant.wh;  // query heads of a CTA
    a.head_blocks = (a.group + heads - 1) / heads;
    a.head_dim = static_cast<int>(cache->head_dim);
    a.max_pages = static_cast<int>(max_pages);
    a.num_pages = static_cast<int>(cache->num_pages);
    a.window = window < INT32_MAX ? static_cast<int>(window) : 0;  // longer than any row: no window
    a.whole_pages = cache->page_size % 16 == 0 && a.window == 0 && a.k.token < (1 << 22) && a.v.token < (1 << 22);
    a.page = FastDiv::of(static_cast<uint32_t>(cache->page_size));
    a.scale_log2 = scale * 1.4426950408889634f;
    a.counters = static_cast<unsigned *>(workspace);
    a.split = reinterpret_cast<int2 *>(static_cast<char *>(workspace) + kCounterBytes);
    a.partials = reinterpret_cast<float *>(static_cast<char *>(workspace) + kCounterBytes + kSplitBytes);
    a.status = status;
    const int dp = paged_attn_width(a.head_dim);
    cudaError_t e;
    if (dtype == SDT_DTYPE_F16)
        e = dp == 64 ? launch_paged_attn<__half, 64>(a, l) : dp == 128 ? launch_paged_attn<__half, 128>(a, l) : launch_paged_attn<__half, 256>(a, l);
    else
        e = dp == 64 ? launch_paged_attn<__nv_bfloat16, 64>(a, l)
                     : dp == 128 ? launch_paged_attn<__nv_bfloat16, 128>(a, l) : launch_paged_attn<__nv_bfloat16, 256>(a, l);
    if (e != cudaSuccess) return fail(SDT_ERR_LAUNCH, "paged_attn_m1 launch failed: %s", cudaGetErrorString(e));
    return SDT_OK;
}

}  // extern "C"
