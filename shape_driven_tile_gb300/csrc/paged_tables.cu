// paged_tables.cu -- block tables and slot maps of one serving step, from the requests'
// lengths alone.
//
// Request b holds lens[b] tokens in ceil(lens[b] / p) pages of p tokens and adds new[b].
// With held = ceil(lens / p), fresh = ceil((lens + new) / p) - held, and the exclusive
// prefix sums S of new and F of fresh over the requests,
//     table[b][held + i] = free[F_b + i]                      i < fresh_b
//     slots[S_b + i]     = table[b][pos / p] * p + pos % p    pos = lens_b + i, i < new_b.
//
// What bounds it: nothing is worth streaming (8 bytes a token), so a call costs its launch
// and one chain of dependent loads: 2.9 us for 256 requests, 6.2 us for 1021 requests with
// 68 thousand new tokens, back to back on GB300.  Every CTA therefore computes both prefix sums over all
// requests itself (one load per request and thread, a block scan) instead of waiting for
// another launch or CTA, keeps them in shared memory and finds the request of a token or of
// a fresh page by bisection.  A slot on a fresh page takes its page from `free`, not from
// the table entry that another CTA may be writing.
//
// With `taken` the place in the free list lives on the device and moves with each call, and the
// lengths may be updated in place, so that a captured step can be replayed by itself.  What
// every CTA still reads may then change only when all have read it: the last CTA to arrive
// (a counter beside the place, zero between calls) writes both: 3.9 us for 256 requests, 8.8
// for 1021 with 67 new tokens each (2.9 and 6.8 without).
#include <atomic>

#include "launch.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace sdt {

constexpr int kTablesThreads = 256;
constexpr int kTablesMaxBatch = 16384;  // two int32 prefix sums in shared memory: 128 KB
constexpr int kTablesPerThread = 4;     // tokens per thread that a CTA is launched for

struct TablesArgs {
    const int *lens, *fresh_tokens, *free_pages;
    int *table;
    int64_t table_stride;
    int *kv_lens, *starts, *used;
    int64_t *slots;
    int64_t num_slots;
    int batch, max_pages, num_free;
    FastDiv page;
    int *taken;  // null, or [2]: entries of free_pages used by earlier calls, CTAs that have arrived
};

// Index of the last of `n` non-decreasing prefix sums that is <= x (sums[0] = 0, x >= 0).
__device__ __forceinline__ int bisect(const int *sums, int n, int x) {
    int lo = 0, hi = n;  // sums[lo] <= x, everything from hi on is > x
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <bool TAKEN>
__global__ void __launch_bounds__(kTablesThreads) paged_tables_kernel(const TablesArgs a) {
    extern __shared__ int sums[];  // [batch] first token, [batch] first fresh page of each request
    int *tok = sums, *pg = sums + a.batch;
    __shared__ int warp_tok[kTablesThreads / 32], warp_pg[kTablesThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_launch_dependents();
    griddep_wait();

    const int base = TAKEN ? min(max(a.taken[0], 0), a.num_free) : 0;  // of the free list
    const int num_free = a.num_free - base;
    const int capacity = a.max_pages * static_cast<int>(a.page.d);  // tokens of a table row (< 2^31: checked on the host)
    auto length_of = [&](int b) { return min(max(a.lens[b], 0), capacity); };
    auto added = [&](int b, int len) { return min(max(a.fresh_tokens[b], 0), INT32_MAX - len); };
    auto held_of = [&](int len) {
        return min(static_cast<int>(a.page.div(static_cast<uint32_t>(len) + a.page.d - 1u)), a.max_pages);
    };
    // a thread's requests are consecutive, so that one scan over the threads' sums is enough
    const int per = (a.batch + kTablesThreads - 1) / kTablesThreads;
    const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    int my_tok = 0, my_pg = 0;
    for (int b = b0; b < b1; ++b) {
        const int len = length_of(b), add = added(b, len);
        tok[b] = my_tok;
        pg[b] = my_pg;
        my_tok += add;
        my_pg += held_of(len + add) - held_of(len);
        if (!TAKEN && blockIdx.x == 0) a.kv_lens[b] = len + add;
    }
    int inc_tok = my_tok, inc_pg = my_pg;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, inc_tok, o), p = __shfl_up_sync(0xffffffffu, inc_pg, o);
        if (lane >= o) {
            inc_tok += t;
            inc_pg += p;
        }
    }
    if (lane == 31) {
        warp_tok[warp] = inc_tok;
        warp_pg[warp] = inc_pg;
    }
    __syncthreads();
    int off_tok = inc_tok - my_tok, off_pg = inc_pg - my_pg, all_tok = 0, all_pg = 0;
#pragma unroll
    for (int w = 0; w < kTablesThreads / 32; ++w) {
        if (w < warp) {
            off_tok += warp_tok[w];
            off_pg += warp_pg[w];
        }
        all_tok += warp_tok[w];
        all_pg += warp_pg[w];
    }
    for (int b = b0; b < b1; ++b) {
        tok[b] += off_tok;
        pg[b] += off_pg;
        if (blockIdx.x == 0) a.starts[b] = tok[b];
    }
    if (blockIdx.x == 0 && tid == 0) {
        a.starts[a.batch] = all_tok;
        a.used[0] = all_pg;
    }
    __syncthreads();

    const int64_t step = static_cast<int64_t>(gridDim.x) * kTablesThreads;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kTablesThreads + tid;
    for (int64_t i = first; i < all_pg; i += step) {
        const int b = bisect(pg, a.batch, static_cast<int>(i));
        const int j = held_of(length_of(b)) + static_cast<int>(i) - pg[b];
        if (j >= 0 && j < a.max_pages)
            a.table[b * a.table_stride + j] = i < num_free ? a.free_pages[base + i] : -1;
    }
    for (int64_t i = first; i < a.num_slots; i += step) {
        int64_t slot = -1;
        if (i < all_tok) {
            const int b = bisect(tok, a.batch, static_cast<int>(i));
            const int len = length_of(b);
            const uint32_t pos = static_cast<uint32_t>(len) + static_cast<uint32_t>(i) - static_cast<uint32_t>(tok[b]);
            const int p = static_cast<int>(a.page.div(pos & 0x7fffffffu)), held = held_of(len);
            int id = -1;
            if (p < a.max_pages) {
                const int64_t f = static_cast<int64_t>(pg[b]) + p - held;
                if (p < held) id = a.table[b * a.table_stride + p];
                else if (f >= 0 && f < num_free) id = a.free_pages[base + f];
            }
            if (id >= 0) slot = static_cast<int64_t>(id) * a.page.d + (pos - static_cast<uint32_t>(p) * a.page.d);
        }
        a.slots[i] = slot;
    }
    if constexpr (TAKEN) {
        __shared__ int last;
        __syncthreads();  // this CTA has read everything
        if (tid == 0) {
            unsigned was;  // (wraps to 0 at the last CTA)
            asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(was) : "l"(a.taken + 1), "r"(gridDim.x - 1) : "memory");
            last = was == gridDim.x - 1;
        }
        __syncthreads();
        if (!last) return;
        for (int b = tid; b < a.batch; b += kTablesThreads) {
            const int len = length_of(b);
            a.kv_lens[b] = len + added(b, len);
        }
        if (tid == 0) a.taken[0] = base + min(all_pg, num_free);
    }
}

// A buffer of the call: `rows` stretches of `len` bytes, `step` bytes apart.
struct Buffer {
    const char *name, *p;
    int64_t rows, len, step;
};

// Whether a byte of x lies in y; x is one stretch.
static bool lies_in(const Buffer &x, const Buffer &y) {
    if (!x.len || !y.len || !y.rows) return false;
    if (x.p + x.len <= y.p || x.p >= y.p + (y.rows - 1) * y.step + y.len) return false;
    if (x.p < y.p) return true;
    const int64_t off = x.p - y.p, row = off / y.step;  // x begins in row `row` of y or behind it, before the next
    return off - row * y.step < y.len || off + x.len > (row + 1) * y.step;
}

}  // namespace sdt

using namespace sdt;

static int tables(const sdt_paged_step *step, int32_t *taken, sdt_stream_t stream) {
    clear_error();
    if (!step) return fail(SDT_ERR_NULL, "paged_tables: NULL arguments");
    const auto &[lens, new_tokens, free_pages, table, kv_lens, starts, used, slots, batch, page_size, max_pages, table_stride,
                 num_free, num_slots] = *step;
    if (batch < 1 || batch > kTablesMaxBatch)
        return fail(SDT_ERR_SHAPE, "paged_tables: batch must be in 1 .. %d (got %lld)", kTablesMaxBatch, (long long)batch);
    if (page_size < 1 || max_pages < 0 || num_free < 0 || num_slots < 0 || max_pages > INT32_MAX || num_free > INT32_MAX ||
        num_slots > INT32_MAX || page_size > INT32_MAX || page_size * max_pages > INT32_MAX)
        return fail(SDT_ERR_SHAPE, "paged_tables: page_size >= 1, sizes >= 0 and page_size * max_pages, num_free, num_slots < 2^31");
    if (table_stride < max_pages) return fail(SDT_ERR_ARG, "paged_tables: table rows of %lld entries, %lld apart", (long long)max_pages, (long long)table_stride);
    if (!lens || !new_tokens || !kv_lens || !starts || !used || (num_free && !free_pages) || (max_pages && !table) ||
        (num_slots && !slots))
        return fail(SDT_ERR_NULL, "paged_tables: NULL pointer");
    if (!aligned(lens, 4) || !aligned(new_tokens, 4) || !aligned(free_pages, 4) || !aligned(table, 4) || !aligned(kv_lens, 4) ||
        !aligned(starts, 4) || !aligned(used, 4) || !aligned(slots, 8) || !aligned(taken, 4))
        return fail(SDT_ERR_ALIGN, "paged_tables: pointers must be aligned to their elements");
    // Every CTA reads the inputs at its own time, and CTA 0 writes sums before the others have read: no output
    // may lie over an input or over another output.  Only with `taken` kv_lens waits for all CTAs.
    const int64_t vec = 4 * batch;
    const Buffer all[] = {{"lens", reinterpret_cast<const char *>(lens), 1, vec, vec},
                          {"new_tokens", reinterpret_cast<const char *>(new_tokens), 1, vec, vec},
                          {"free_pages", reinterpret_cast<const char *>(free_pages), 1, 4 * num_free, 4 * num_free},
                          {"kv_lens", reinterpret_cast<const char *>(kv_lens), 1, vec, vec},
                          {"starts", reinterpret_cast<const char *>(starts), 1, vec + 4, vec + 4},
                          {"used", reinterpret_cast<const char *>(used), 1, 4, 4},
                          {"slots", reinterpret_cast<const char *>(slots), 1, 8 * num_slots, 8 * num_slots},
                          {"taken", reinterpret_cast<const char *>(taken), 1, taken ? 8 : 0, 8},
                          {"table", reinterpret_cast<const char *>(table), batch, 4 * max_pages, 4 * table_stride}};
    constexpr int kLens = 0, kInputs = 3, kKvLens = 3, kBuffers = sizeof(all) / sizeof(all[0]);
    for (int i = kInputs; i < kBuffers; ++i)
        for (int j = 0; j < i; ++j)
            if (lies_in(all[j], all[i]) && !(taken && j == kLens && i == kKvLens && kv_lens == lens))
                return fail(SDT_ERR_ARG, "paged_tables: %s and %s overlap", all[j].name, all[i].name);
    DeviceInfo dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    TablesArgs a{lens, new_tokens, free_pages, table, table_stride, kv_lens, starts, used, slots, num_slots,
                 static_cast<int>(batch), static_cast<int>(max_pages), static_cast<int>(num_free),
                 FastDiv::of(static_cast<uint32_t>(page_size)), taken};
    const size_t smem = 2 * sizeof(int) * static_cast<size_t>(batch);
    auto kern = taken ? paged_tables_kernel<true> : paged_tables_kernel<false>;
    static std::atomic<bool> ready[kMaxDevices][2];  // the attribute call takes longer than the launch: once a device
    cudaError_t e = cudaSuccess;
    if (!ready[dev.device][taken != nullptr].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * static_cast<int>(sizeof(int)) * kTablesMaxBatch);
        if (e == cudaSuccess) ready[dev.device][taken != nullptr].store(true, std::memory_order_release);
    }
    if (e == cudaSuccess) {
        const int64_t want = (num_slots + kTablesThreads * kTablesPerThread - 1) / (kTablesThreads * kTablesPerThread);
        const int64_t grid = want < 1 ? 1 : want > dev.sm_count ? dev.sm_count : want;
        e = launch_kernel(kern, dim3(static_cast<unsigned>(grid)), dim3(kTablesThreads), smem,
                          reinterpret_cast<cudaStream_t>(stream), 1, a);
    }
    if (e != cudaSuccess) return fail(SDT_ERR_LAUNCH, "paged_tables launch failed: %s", cudaGetErrorString(e));
    return SDT_OK;
}

extern "C" int paged_tables(const sdt_paged_step *step, sdt_stream_t stream) { return tables(step, nullptr, stream); }

extern "C" int paged_tables_taken(const sdt_paged_step *step, int32_t *taken, sdt_stream_t stream) {
    if (!taken) {
        clear_error();
        return fail(SDT_ERR_NULL, "paged_tables_taken: NULL pointer");
    }
    return tables(step, taken, stream);
}
