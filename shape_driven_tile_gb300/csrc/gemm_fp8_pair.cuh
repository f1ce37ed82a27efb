// gemm_fp8_pair.cuh -- gemm_fp8 for many tokens: persistent two-CTA tiles of 256 tokens by 256
// (or 192) outputs.
//
// A pair of CTAs runs M = 256 MMAs (cta_group::2) as gemm_pair.cuh does: each CTA stages its own
// 128 token rows and half of the tile's weight rows per 128-deep block, 32 KB that feed 512
// cycles of MMAs.  Two accumulators of 256 columns fill tensor memory and hold one block's sums
// each: while the tensor cores fill one, eight epilogue warps per CTA (twelve for 192 outputs) read
// the other, scale it and add it to registers (128 columns a thread, or 64).  A thread's lane is a
// token row and its columns lie in one block of 128 outputs, so its scale is one register.  Scales arrive eight blocks at a time in three buffers of shared memory, by 4-byte
// asynchronous copies that pass over tile borders.
//
// What bounds it is the epilogue's 680 to 750 cycles a block, most of them the way round a pair of
// accumulators (MMAs, the commit, the reads, the arrivals of both CTAs' warps), where the tensor
// cores need 512: 8192^3 takes 369 to 378 us, GPU by GPU (2.9 to 3.0 PFLOP/s).  16 epilogue warps of
// 64 columns take 394 where eight take 378.  With one multiply-add a value it took 380, and 321 with a
// quarter of the columns read; tried then and not faster: four accumulators of 128 columns, half a
// tile each (382 us; 313 with a quarter read), the next block's first columns on their way while the
// last ones are added (407), all of a warp's results staged at once in place of the fifth ring slot
// (405), one-CTA tiles (522).
//
// The tiles of a last, partly empty round run as two half-width items each.  192-wide tiles are for
// shapes of few tiles, which 256-wide ones spread over fewer pairs (1021 x 2560 x 7168: 56 tiles on
// 76 pairs instead of 40, 21.8 us against 26.4); with eight epilogue warps of 96 columns they take 22.1.
//
// Roles: warp 0 feeds the ring (TMA), warp 1 of the leader issues the MMAs, warps 2 and 3 copy
// scales, the others are the epilogue, which takes over registers of the first four (setmaxnreg:
// 56 a thread there, 224 in eight epilogue warps, of 168 at launch; 152 in twelve, of 128).
#pragma once

#include "gemm_fp8.cuh"
#include "gemm_persistent.cuh"

namespace sdt {

template <int WIDTH>
struct Fp8PairCfg {
    static constexpr int BM = 256, BN = WIDTH, CTA_M = 128;
    static constexpr int A_BYTES = CTA_M * kFp8Block, B_BYTES = BN / 2 * kFp8Block;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = 5;
    static constexpr int PARTS = WIDTH == 256 ? 2 : 3;  // epilogue warps side by side, each with a part of the columns
    static constexpr int EPI_WARPS = 4 * PARTS, THREADS = 128 + 32 * EPI_WARPS;
    // registers of a thread: what the launch gives all, and after the roles have parted
    static constexpr int ROLE_REGS = 56, EPI_REGS = PARTS == 2 ? 224 : 152;
    static constexpr int SPLIT_REGS = 128 * ROLE_REGS + 32 * EPI_WARPS * EPI_REGS;
    static_assert(SPLIT_REGS <= THREADS * (65536 / THREADS / 8 * 8), "within what a launch can have");
    static constexpr int ACC_BUFS = 2, ACC_STEP = 256, TMEM_COLS = ACC_BUFS * ACC_STEP;  // step: columns from one to the other
    static constexpr int COLS = BN / PARTS;  // columns of an epilogue thread
    static constexpr int C_STAGE_BYTES = EPI_WARPS * 2 * kCStageBytes;
    static constexpr int AHEAD = 8;       // blocks whose scales are loaded together
    static constexpr int SCALE_BUFS = 3;
    static constexpr int SCALE_THREADS = 64;
    static constexpr int SCALE_BYTES = AHEAD * (CTA_M + 2) * 4;  // [block][token row], then [half][block] of the weights
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + C_STAGE_BYTES + SCALE_BUFS * SCALE_BYTES + 512;
};

// Arrive on the leader's barrier without publishing any writes: what it announces is that the
// warp's reads of tensor memory have completed (tcgen05.wait::ld), and a release at cluster scope
// would wait for every load and store of the thread in flight (4096^3: 158 us with one, 90 without).
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Item -> tile, and for the halves of the last round the column offset and width.
struct Fp8Item {
    int m_tile, n0, width;
};
template <int BN>
__device__ __forceinline__ Fp8Item fp8_item(int item, const Fp8Args &p) {
    Fp8Item r;
    int tile = item, off = 0, n_tile;
    r.width = BN;
    if (item >= p.tail_start) {
        const int h = item - p.tail_start;
        tile = p.tail_start + (h >> 1);
        off = (h & 1) * (BN / 2);
        r.width = BN / 2;
    }
    tile_coords(tile, p.num_m_tiles, p.num_n_tiles, p.raster_group, r.m_tile, n_tile);
    r.n0 = n_tile * BN + off;
    return r;
}

// 32 columns of a warp's 32 rows through the staging buffers: 16-bit values as one box of 32
// columns, fp32 as two of 16 (64-byte rows either way; see store_chunk_tma).
__device__ __forceinline__ void fp8_store_chunk(const CUtensorMap *tmC, uint32_t buf0, int &nst, const uint32_t (&r)[32],
                                                int c_dtype, int x, int y, int lane) {
    if (c_dtype != SDT_DTYPE_F32) {
        store_chunk_tma(tmC, buf0, nst++, r, c_dtype == SDT_DTYPE_BF16, x, y, lane);
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t buf = buf0 + static_cast<uint32_t>(nst++ & 1) * kCStageBytes;
        if (lane == 0) bulk_wait_group_read<1>();
        __syncwarp();
        const uint32_t row = buf + static_cast<uint32_t>(lane) * 64u;
        const uint32_t sw = static_cast<uint32_t>((lane >> 1) & 3);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((static_cast<uint32_t>(c) ^ sw) << 4)),
                         "r"(r[16 * h + 4 * c]), "r"(r[16 * h + 4 * c + 1]), "r"(r[16 * h + 4 * c + 2]), "r"(r[16 * h + 4 * c + 3])
                         : "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(tmC, buf, x + 16 * h, y);
            bulk_commit_group();
        }
    }
}

// acc[j] += scale * column j of COLS columns of tensor memory, 32 at a time, the next ones on their
// way while these are added; done() as soon as all have been read.
template <int COLS, int N, typename Done>
__device__ __forceinline__ void fp8_scale_add(uint32_t taddr, float scale, float (&acc)[N], Done done) {
    uint32_t v[2][32];
    tmem_ld_32x32b_x32(taddr, v[0]);
#pragma unroll
    for (int c = 0; c < COLS; c += 32) {
        tmem_ld_wait();
        if (c + 32 < COLS) tmem_ld_32x32b_x32(taddr + c + 32, v[(c / 32 + 1) & 1]);
        else done();
#pragma unroll
        for (int j = 0; j < 32; j += 2) fma2(acc + c + j, v[(c / 32) & 1] + j, make_float2(scale, scale));
    }
}

template <int REGS>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS)); }
template <int REGS>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS)); }

// One fp32 value global -> shared, asynchronously; zero (and nothing read) if `in` is false.
__device__ __forceinline__ void copy_f32_async(uint32_t dst, const float *src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
// Arrive on `bar` once this thread's asynchronous copies so far have landed.
__device__ __forceinline__ void mbar_arrive_copies(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <int WIDTH>
__global__ void __launch_bounds__(Fp8PairCfg<WIDTH>::THREADS, 1)
    gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmC, const Fp8Args p) {
    using Cfg = Fp8PairCfg<WIDTH>;
    constexpr int S = Cfg::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t smA = base, smB = base + S * Cfg::A_BYTES, smC = base + S * Cfg::STAGE_BYTES;
    const uint32_t smS = smC + Cfg::C_STAGE_BYTES, bars = smS + Cfg::SCALE_BUFS * Cfg::SCALE_BYTES;
    const uint32_t full = bars, empty = bars + 8 * S, acc_full = bars + 16 * S, acc_empty = acc_full + 8 * Cfg::ACC_BUFS;
    const uint32_t sc_full = acc_empty + 8 * Cfg::ACC_BUFS, sc_empty = sc_full + 8 * Cfg::SCALE_BUFS, mma_done = sc_empty + 8 * Cfg::SCALE_BUFS;
    volatile uint32_t *ctrl = reinterpret_cast<volatile uint32_t *>(smem_raw + (mma_done + 8 - smem_u32(smem_raw)));
    // ctrl[0]: TMEM base   ctrl[1]: a role gave up   ctrl[2]: blocks the producer asked for

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = static_cast<int>(blockIdx.x >> 1), num_pairs = static_cast<int>(gridDim.x >> 1);
    const int nkb = p.num_kb;
    const uint64_t lim = p.timeout_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < Cfg::ACC_BUFS; ++b) {
            mbar_init(acc_full + 8 * b, 1);
            mbar_init(acc_empty + 8 * b, 2 * Cfg::EPI_WARPS);
        }
        for (int b = 0; b < Cfg::SCALE_BUFS; ++b) {
            mbar_init(sc_full + 8 * b, Cfg::SCALE_THREADS);
            mbar_init(sc_empty + 8 * b, Cfg::EPI_WARPS);
        }
        mbar_init(mma_done, 1);
        ctrl[1] = 0;
        ctrl[2] = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(const_cast<uint32_t *>(&ctrl[0])), Cfg::TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = ctrl[0];
    griddep_wait();

    if (warp < 4) {
        regs_dec<Cfg::ROLE_REGS>();
        if (warp == 0) {
            if (elect_one()) {
                tma_prefetch_desc(&tmA);
                tma_prefetch_desc(&tmB);
            }
            const uint32_t full_leader = mapa_shared(full, 0);
            int s = 0, issued = 0;
            uint32_t phase = 0;
            bool stop = false, ready = true;  // the ring's slots are free at first
            for (int item = pair; item < p.num_items && !stop; item += num_pairs) {
                const Fp8Item it = fp8_item<WIDTH>(item, p);
                const int m0 = it.m_tile * Cfg::BM + static_cast<int>(rank) * Cfg::CTA_M;
                const int nb = it.n0 + static_cast<int>(rank) * (it.width / 2);
                const bool whole = it.width == Cfg::BN;
                if (item + num_pairs >= p.num_items) griddep_launch_dependents();
                const uint32_t bytes = 2u * static_cast<uint32_t>(whole ? Cfg::STAGE_BYTES : Cfg::A_BYTES + Cfg::B_BYTES / 2);
                for (int i = 0; i < nkb; ++i) {
                    if (!warp_wait_peeked(ready, empty + 8 * s, phase ^ 1u, lim)) {
                        if (lane == 0) record_status(p.status, kSiteProducer | static_cast<int>(rank << 4) | (issued << 8));
                        ctrl[1] = 1;
                        stop = true;
                        break;
                    }
                    if ((i & 7) == 0 && ctrl[1]) { stop = true; break; }
                    const int s_next = s + 1 == S ? 0 : s + 1;
                    const uint32_t phase_next = s + 1 == S ? phase ^ 1u : phase;
                    ready = mbar_peek(empty + 8 * s_next, phase_next ^ 1u);
                    if (elect_one()) {
                        if (leader) mbar_arrive_expect_tx(full + 8 * s, bytes);
                        const uint32_t fb = full_leader + 8 * s;
                        tma_load_2d_pair(smA + s * Cfg::A_BYTES, &tmA, fb, i * kFp8Block, m0);
                        tma_load_2d_pair(smB + s * Cfg::B_BYTES, &tmB, fb, i * kFp8Block, nb);
                        if (Cfg::BN == 256 && whole) tma_load_2d_pair(smB + s * Cfg::B_BYTES + Cfg::B_BYTES / 2, &tmB, fb, i * kFp8Block, nb + Cfg::BN / 4);
                    }
                    __syncwarp();
                    ++issued;
                    s = s_next;
                    phase = phase_next;
                }
            }
            ctrl[2] = issued;
        } else if (warp == 1 && leader) {
            const uint64_t a0 = smem_desc_sw128(smA, 16, 1024), b0 = smem_desc_sw128(smB, 16, 1024);
            int s = 0, j = 0;
            uint32_t phase = 0, n = 0;  // n: blocks so far, whose accumulators alternate
            bool stop = false, loaded = false, empty_acc = true;
            for (int item = pair; item < p.num_items && !stop; item += num_pairs, ++j) {
                const uint32_t idesc = idesc_for(p.idesc, Cfg::BM, item < p.tail_start ? Cfg::BN : Cfg::BN / 2);
                for (int i = 0; i < nkb; ++i, ++n) {
                    const uint32_t b = n & 1;
                    if (!warp_wait_peeked(loaded, full + 8 * s, phase, lim) ||
                        !warp_wait_peeked<true>(empty_acc, acc_empty + 8 * b, ((n >> 1) & 1) ^ 1u, lim)) {
                        if (lane == 0) record_status(p.status, kSiteMma | (((j << 12) | i) << 8));
                        ctrl[1] = 1;
                        stop = true;
                        break;
                    }
                    tc_fence_after();
                    const int s_next = s + 1 == S ? 0 : s + 1;
                    const uint32_t phase_next = s + 1 == S ? phase ^ 1u : phase;
                    loaded = mbar_peek(full + 8 * s_next, phase_next);
                    empty_acc = mbar_peek<true>(acc_empty + 8 * (b ^ 1), (((n + 1) >> 1) & 1) ^ 1u);
                    if (elect_one()) {
                        const uint64_t ad = a0 + static_cast<uint64_t>(s) * (Cfg::A_BYTES >> 4);
                        const uint64_t bd = b0 + static_cast<uint64_t>(s) * (Cfg::B_BYTES >> 4);
#pragma unroll
                        for (int kk = 0; kk < kFp8Block / 32; ++kk)
                            umma_fp8_pair(tmem_base + b * Cfg::ACC_STEP, ad + 2 * kk, bd + 2 * kk, idesc, kk > 0);
                        umma_commit_pair(acc_full + 8 * b, 0x3);  // (the epilogue hands the ring's slot back)
                    }
                    __syncwarp();
                    s = s_next;
                    phase = phase_next;
                }
            }
            if (elect_one()) umma_commit_pair(mma_done, 0x1);
            __syncwarp();
            if (!mbar_wait_for(mma_done, 0, lim) && lane == 0) record_status(p.status, kSiteDrain);
        } else if (warp >= 2) {
            // scales of AHEAD blocks at a time, in 16 steps of 64 values: 8 blocks of 8 rows a step, or,
            // where rows are neighbours in memory, one block of half of the rows.  Steps 2 v and
            // 2 v + 1 lie `near` apart, steps v and v + 2 `far`.
            const int t = static_cast<int>(threadIdx.x) - 64;
            const bool by_row = p.as_row == 1;
            const int row0 = by_row ? t : t >> 3, kb0 = by_row ? 0 : t & 7;
            const int near_rows = by_row ? 64 : 8, far_rows = by_row ? 0 : 16, far_kb = by_row ? 1 : 0;
            const int64_t near = near_rows * p.as_row, far = far_rows * p.as_row + far_kb * p.as_block;
            const uint32_t near_dst = near_rows * 4, far_dst = (far_rows + far_kb * Cfg::CTA_M) * 4;
            int buf = 0;
            uint32_t sc_phase = 0;
            bool stop = false;
            for (int item = pair; item < p.num_items && !stop; item += num_pairs) {
                const Fp8Item it = fp8_item<WIDTH>(item, p);
                const int m0 = it.m_tile * Cfg::BM + static_cast<int>(rank) * Cfg::CTA_M;
                for (int i0 = 0; i0 < nkb; i0 += Cfg::AHEAD) {
                    if (ctrl[1] || !mbar_wait_soon(sc_empty + 8 * buf, sc_phase ^ 1u, 4 * lim)) {
                        stop = true;  // (whoever gave up first has said so)
                        break;
                    }
                    const uint32_t dst = smS + buf * Cfg::SCALE_BYTES;
                    const float *src = p.a_scales + (m0 + row0) * p.as_row + (i0 + kb0) * p.as_block;
                    uint32_t to = dst + (kb0 * Cfg::CTA_M + row0) * 4;
                    int rows = p.M - m0 - row0, blocks = nkb - i0 - kb0;  // left from this thread's first value on
#pragma unroll 2
                    for (int v = 0; v < 8; ++v) {
                        const bool in = rows > 0 && blocks > 0, in_near = rows > near_rows && blocks > 0;
                        copy_f32_async(to, in ? src : p.a_scales, in);
                        copy_f32_async(to + near_dst, in_near ? src + near : p.a_scales, in_near);
                        src += far;
                        to += far_dst;
                        rows -= far_rows;
                        blocks -= far_kb;
                    }
                    if (t < 2 * Cfg::AHEAD) {
                        const int h = t / Cfg::AHEAD, kb = t % Cfg::AHEAD;
                        const int nb = (it.n0 + h * (it.width == kFp8Block ? 0 : kFp8Block)) / kFp8Block;  // the tile's two blocks
                        const bool in = nb * kFp8Block < p.N && i0 + kb < nkb;
                        copy_f32_async(dst + (Cfg::AHEAD * Cfg::CTA_M + t) * 4, in ? p.w_scales + nb * p.ws_row + (i0 + kb) * p.ws_block : p.w_scales, in);
                    }
                    mbar_arrive_copies(sc_full + 8 * buf);
                    if (++buf == Cfg::SCALE_BUFS) { buf = 0; sc_phase ^= 1u; }
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else {
        regs_inc<Cfg::EPI_REGS>();
        const int q = warp & 3, part = (warp - 4) >> 2;
        const uint32_t cbuf = smC + static_cast<uint32_t>(warp - 4) * 2u * kCStageBytes;
        const uint32_t acc_empty_leader = mapa_shared(acc_empty, 0);
        const uint32_t my_scales = smS + (q * 32 + lane) * 4, lanes = static_cast<uint32_t>(q * 32) << 16;
        int nst = 0, s = 0, buf = 0;
        uint32_t n = 0, sc_phase = 0;
        bool good = true, done = false;
        for (int item = pair; item < p.num_items && good; item += num_pairs) {
            const Fp8Item it = fp8_item<WIDTH>(item, p);
            const int cols = it.width / Cfg::PARTS;
            const uint32_t taddr = tmem_base + lanes + part * cols;
            // a part's outputs lie in one block of weight scales, the tile's first or second
            const int second = WIDTH == 256 ? part : it.n0 % kFp8Block + part * cols >= kFp8Block;
            const uint32_t w_scales = smS + (Cfg::AHEAD * Cfg::CTA_M + second * Cfg::AHEAD) * 4;
            float acc[Cfg::COLS];
#pragma unroll
            for (int j = 0; j < Cfg::COLS; ++j) acc[j] = 0.f;
            for (int i0 = 0; i0 < nkb && good; i0 += Cfg::AHEAD) {
                const int left = min(Cfg::AHEAD, nkb - i0);
                good = warp_wait_soon(sc_full + 8 * buf, sc_phase, 4 * lim);
                uint32_t sc = my_scales + buf * Cfg::SCALE_BYTES, sw = w_scales + buf * Cfg::SCALE_BYTES;
                float token = ld_shared_f32(sc), weight = ld_shared_f32(sw);
                for (int u = 0; u < left && good; ++u, ++n) {
                    const uint32_t b = n & 1;
                    const float scale = token * weight;
                    good = warp_wait_peeked(done, acc_full + 8 * b, (n >> 1) & 1, 4 * lim);
                    if (!good) break;
                    tc_fence_after();
                    if (warp == 4 && lane == 0) mbar_arrive(empty + 8 * s);  // the block's MMAs have read the ring
                    if (++s == S) s = 0;
                    if (u + 1 < left) {
                        token = ld_shared_f32(sc += Cfg::CTA_M * 4);
                        weight = ld_shared_f32(sw += 4);
                    }
                    const auto read = [&] {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty_leader + 8 * b);
                        done = mbar_peek(acc_full + 8 * (b ^ 1), ((n + 1) >> 1) & 1);
                    };
                    if (WIDTH != 256 || cols == Cfg::COLS) fp8_scale_add<Cfg::COLS>(taddr + b * Cfg::ACC_STEP, scale, acc, read);
                    else fp8_scale_add<Cfg::COLS / 2>(taddr + b * Cfg::ACC_STEP, scale, acc, read);
                }
                if (lane == 0) mbar_arrive(sc_empty + 8 * buf);
                if (++buf == Cfg::SCALE_BUFS) { buf = 0; sc_phase ^= 1u; }
            }
            if (!good) {
                if (lane == 0) {
                    record_status(p.status, kSiteEpilogue | static_cast<int>(rank << 4) | (item << 8));
                    ctrl[1] = 1;
                }
                break;
            }
            const int row0 = it.m_tile * Cfg::BM + static_cast<int>(rank) * Cfg::CTA_M + q * 32, x0 = it.n0 + part * cols;
#pragma unroll
            for (int c = 0; c < Cfg::COLS; c += 32)
                if (c < cols && x0 + c < p.N && row0 < p.M) {
                    uint32_t r[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(acc[c + j]);
                    fp8_store_chunk(&tmC, cbuf, nst, r, p.c_dtype, x0 + c, row0, lane);
                }
        }
        if (lane == 0) bulk_wait_group<0>();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && leader && ctrl[1]) {
        const int issued = static_cast<int>(ctrl[2]);
        for (int i = max(0, issued - S); i < issued; ++i)
            if (!mbar_wait_for(full + 8 * (i % S), static_cast<uint32_t>((i / S) & 1), lim)) {
                record_status(p.status, kSiteDrain);
                break;
            }
    }
    cluster_sync();  // both CTAs done with each other's shared memory, barriers and TMEM
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
    }
}

}  // namespace sdt
