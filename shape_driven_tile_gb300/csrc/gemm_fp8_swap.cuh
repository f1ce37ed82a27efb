// gemm_fp8_swap.cuh -- gemm_fp8 for few tokens: 128 weight rows by BT tokens per tile, the
// tile's k-blocks shared by a cluster of CTAs.
//
// Up to 64 tokens the product runs as W . A^T, so that the many weight rows fill the MMA's 128 rows
// and BT (16, 32 or 64) tokens its columns: a weight byte is read from memory once for up to BT
// tokens, and a single token costs what the weights' bytes cost.  The accumulator's lane is a
// weight row and its column a token: the weight scale is the tile's, the token scales come from
// shared memory as four at a time, and two CTAs share an SM.  With 128 tokens the tile is as wide
// as it is high, and tokens are the rows: a thread then holds one token, whose scale it multiplies
// by, and no longer reads a scale per value (333 x 5000 x 4208: 17.6 us against 19.5 with weights as
// rows).
//
// What bounds it at few tokens is the stream of weights, so the work is cut to fill the GPU:
// the CTAs of a cluster take consecutive ranges of the k-blocks of one tile and hold their sums
// in registers.  At the end each token belongs to one of them, and the others store their sums of
// it into a buffer of that CTA's shared memory that nothing else uses, so one meeting of the
// cluster is enough; they are added in rank order (results do not depend on timing), without a
// workspace.  (Sums left in place and read by the owner took a second meeting and eight dependent
// reads from other SMs: 2 us of a 5 us call.)
//
// No CTA holds tensor memory while it waits for another one (it asks for it after it has said that
// it started, and frees it before it waits for the sums), so kernels of several streams cannot
// block each other over it.
//
// Roles: warp 0 feeds the ring (TMA), warp 1 issues the MMAs, the rest scale and add.
#pragma once

#include "gemm_fp8.cuh"

namespace sdt {

template <int BT>
struct SwapCfg {
    static constexpr int ROWS = 128;  // weight rows per tile
    static constexpr bool SWAP = BT < 128;  // weight rows are the MMA's rows
    static constexpr int EPI_WARPS = BT == 16 ? 4 : 8;
    static constexpr int COLS = BT * 4 / EPI_WARPS;  // columns per epilogue warp
    static constexpr int THREADS = 64 + 32 * EPI_WARPS;
    static constexpr int W_BYTES = ROWS * kFp8Block;
    static constexpr int X_BYTES = BT * kFp8Block;
    static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
    static constexpr int ACC_BUFS = 4;
    static constexpr int TMEM_COLS = ACC_BUFS * BT;  // an SM's CTAs always fit
    // ring slots: beside a buffer for the sums of a cluster's CTAs, and with 128 tokens and no cluster, where the
    // sums go where the ring was (128 x 16384 x 4096: 16.6 us, 18.0 with four slots; with 64 tokens a fourth slot
    // in place of the buffer takes 48 us for 64 x 28672 x 8192 instead of 42)
    static constexpr int STAGES = BT == 16 ? 5 : BT == 64 ? 3 : 4;
    static constexpr int STAGES_ALONE = 6;
    static constexpr int PER_SM = BT == 128 ? 1 : 2;  // CTAs of an SM
    static constexpr int CHUNK = BT == 128 ? 8 : 512 / BT;  // k-blocks whose scales are in shared memory at a time
    static constexpr int SCALE_BYTES = CHUNK * BT * 4;
    static constexpr int PER_THREAD = CHUNK * BT / (32 * EPI_WARPS);  // scales each epilogue thread brings
    // rows of 128 sums that a CTA receives: S shares of at most ceil(BT / S) tokens, S <= 8
    static constexpr int SUM_ROWS = BT == 16 ? 21 : BT == 32 ? 36 : BT == 64 ? 70 : 133;
    static constexpr int SUM_PITCH = SWAP ? ROWS : ROWS + 4;  // floats (16-byte stores of 8 neighbouring lanes reach all banks)
    static constexpr int SUM_BYTES = SUM_ROWS * SUM_PITCH * 4;
    static constexpr int CTRL_BYTES = 512;
    static constexpr int OTHER_BYTES = 1024 + 2 * SCALE_BYTES + CTRL_BYTES;
    static constexpr int SMEM_BYTES = OTHER_BYTES + STAGES * STAGE_BYTES + SUM_BYTES;
    static constexpr int SMEM_ALONE = OTHER_BYTES + STAGES_ALONE * STAGE_BYTES;
    static constexpr int SMEM_MOST = BT == 128 && SMEM_ALONE > SMEM_BYTES ? SMEM_ALONE : SMEM_BYTES;
    static_assert(BT == 16 || BT == 32 || BT == 64 || BT == 128, "tokens per tile");
    static_assert(TMEM_COLS * PER_SM <= 512 && SMEM_MOST <= (PER_SM == 2 ? 115712 : 232448), "an SM holds PER_SM CTAs");
    static_assert(BT < 128 || BT * SUM_PITCH * 4 <= STAGES_ALONE * STAGE_BYTES, "the sums fit where the ring was");
};

__device__ __forceinline__ void st_cluster_f4(uint32_t addr, float x, float y, float z, float w) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}
// One value to the same place of another CTA's shared memory.
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

template <int BT>
__global__ void __launch_bounds__(SwapCfg<BT>::THREADS, SwapCfg<BT>::PER_SM)
    gemm_fp8_swap_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                         const Fp8Args p) {
    using Cfg = SwapCfg<BT>;
    constexpr int NB = Cfg::ACC_BUFS, E = Cfg::EPI_WARPS * 32;
    const bool alone = BT == 128 && p.splits == 1;
    const int S = alone ? Cfg::STAGES_ALONE : Cfg::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t smW = base, smX = base + S * Cfg::W_BYTES;
    const uint32_t smS = base + S * Cfg::STAGE_BYTES;  // two chunks of scales
    // sums from the cluster's CTAs: [CTA][token of this one's share][row]; a CTA alone takes the ring,
    // which nothing reads or fills once the last block's MMAs are done
    const uint32_t smR = alone ? base : smS + 2 * Cfg::SCALE_BYTES;
    const uint32_t bars = smS + 2 * Cfg::SCALE_BYTES + (alone ? 0 : Cfg::SUM_BYTES);
    const uint32_t full = bars, empty = bars + 8 * S, acc_full = bars + 16 * S, acc_empty = acc_full + 8 * NB;
    volatile uint32_t *ctrl = reinterpret_cast<volatile uint32_t *>(smem_raw + (acc_empty + 8 * NB - smem_u32(smem_raw)));
    // ctrl[0]: TMEM base   ctrl[1]: a role gave up   ctrl[2]: blocks the producer asked for

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = p.splits > 1 ? cluster_ctarank() : 0;
    const int tile = static_cast<int>(blockIdx.x) / p.splits;
    // tokens fastest: CTAs that run together share weights through L2
    const int n_tile = tile / p.num_m_tiles, m_tile = tile - n_tile * p.num_m_tiles;
    const int n0 = n_tile * Cfg::ROWS, m0 = m_tile * BT;
    const int kb0 = static_cast<int>(static_cast<int64_t>(rank) * p.num_kb / p.splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(rank + 1) * p.num_kb / p.splits);
    const int nkb = kb1 - kb0;
    const int tokens = min(BT, p.M - m0), share = (tokens + p.splits - 1) / p.splits;  // of this tile, of a CTA in the end
    const uint64_t lim = p.timeout_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < NB; ++b) {
            mbar_init(acc_full + 8 * b, 1);
            mbar_init(acc_empty + 8 * b, Cfg::EPI_WARPS);
        }
        ctrl[1] = 0;
        ctrl[2] = 0;
        fence_mbar_init();
    }
    if (p.splits > 1) {
        // "this CTA has started", before it asks for tensor memory: the others wait for this and must
        // not wait for that
        __syncwarp();
        cluster_arrive_relaxed();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(const_cast<uint32_t *>(&ctrl[0])), Cfg::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = ctrl[0];
    griddep_launch_dependents();
    // while the kernel before this one still runs, L2 may fetch this CTA's first weights (what L2
    // holds is never stale); nothing else is read yet
    if (warp == 0) {
        if (lane < min(S, nkb)) tma_prefetch_l2_2d(&tmW, (kb0 + lane) * kFp8Block, n0);
        if (lane == 31) tma_prefetch_desc(&tmX);
    }
    griddep_wait();

    float acc[Cfg::COLS];
#pragma unroll
    for (int j = 0; j < Cfg::COLS; ++j) acc[j] = 0.f;
    bool good = true;

    if (warp == 0) {
        int s = 0, issued = 0;
        uint32_t phase = 0;
        bool ready = true;  // the ring's slots are free at first
        for (int i = 0; i < nkb; ++i) {
            if (!warp_wait_peeked(ready, empty + 8 * s, phase ^ 1u, lim)) {
                if (lane == 0) record_status(p.status, kSiteProducer | (i << 8));
                ctrl[1] = 1;
                break;
            }
            if (i >= S && ctrl[1]) break;
            const int s_next = s + 1 == S ? 0 : s + 1;
            const uint32_t phase_next = s + 1 == S ? phase ^ 1u : phase;
            if (i + 1 >= S) ready = mbar_peek(empty + 8 * s_next, phase_next ^ 1u);
            if (elect_one()) {
                mbar_arrive_expect_tx(full + 8 * s, Cfg::STAGE_BYTES);
                tma_load_2d(smW + s * Cfg::W_BYTES, &tmW, full + 8 * s, (kb0 + i) * kFp8Block, n0);
                tma_load_2d(smX + s * Cfg::X_BYTES, &tmX, full + 8 * s, (kb0 + i) * kFp8Block, m0);
            }
            __syncwarp();
            ++issued;
            s = s_next;
            phase = phase_next;
        }
        ctrl[2] = issued;
    } else if (warp == 1) {
        const uint32_t idesc = idesc_for(p.idesc, Cfg::ROWS, BT);  // (128 x 128 is the same either way)
        const uint64_t w0 = smem_desc_sw128(smW, 16, 1024), x0 = smem_desc_sw128(smX, 16, 1024);
        int s = 0, b = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool loaded = false, empty_acc = true;
        for (int i = 0; i < nkb; ++i) {
            if (!warp_wait_peeked(empty_acc, acc_empty + 8 * b, acc_phase ^ 1u, lim) ||
                !warp_wait_peeked(loaded, full + 8 * s, phase, lim)) {
                if (lane == 0) record_status(p.status, kSiteMma | (i << 8));
                ctrl[1] = 1;
                break;
            }
            tc_fence_after();
            const int s_next = s + 1 == S ? 0 : s + 1, b_next = b + 1 == NB ? 0 : b + 1;
            const uint32_t phase_next = s + 1 == S ? phase ^ 1u : phase, acc_phase_next = b + 1 == NB ? acc_phase ^ 1u : acc_phase;
            loaded = mbar_peek(full + 8 * s_next, phase_next);
            if (i + 1 >= NB) empty_acc = mbar_peek(acc_empty + 8 * b_next, acc_phase_next ^ 1u);
            if (elect_one()) {
                const uint64_t wd = w0 + static_cast<uint64_t>(s) * (Cfg::W_BYTES >> 4);
                const uint64_t xd = x0 + static_cast<uint64_t>(s) * (Cfg::X_BYTES >> 4);
#pragma unroll
                for (int kk = 0; kk < kFp8Block / 32; ++kk)
                    umma_fp8(tmem_base + b * BT, (Cfg::SWAP ? wd : xd) + 2 * kk, (Cfg::SWAP ? xd : wd) + 2 * kk, idesc, kk > 0);
                umma_commit(empty + 8 * s);
                umma_commit(acc_full + 8 * b);
            }
            __syncwarp();
            s = s_next;
            b = b_next;
            phase = phase_next;
            acc_phase = acc_phase_next;
        }
    } else {
        const int q = warp & 3;                                   // TMEM lane quarter
        const int col0 = Cfg::EPI_WARPS == 8 ? ((warp - 2) >> 2) * Cfg::COLS : 0;
        const int t = static_cast<int>(threadIdx.x) - 64;
        // scales of chunk c, weight and token scale multiplied (on their way into shared memory, when
        // the loads have long arrived): [block][token]
        float token[Cfg::PER_THREAD], weight[Cfg::PER_THREAD];
        const bool by_token = p.as_row == 1;  // neighbouring threads take neighbouring values
        auto place = [&](int u, int &kb, int &j) {
            const int e = u * E + t;
            if (by_token) { kb = e / BT; j = e % BT; }
            else { kb = e % Cfg::CHUNK; j = e / Cfg::CHUNK; }
        };
        auto fetch = [&](int c) {
#pragma unroll
            for (int u = 0; u < Cfg::PER_THREAD; ++u) {
                int kb, j;
                place(u, kb, j);
                kb += kb0 + c * Cfg::CHUNK;
                const bool in = kb < kb1 && m0 + j < p.M;
                token[u] = in ? p.a_scales[(m0 + j) * p.as_row + kb * p.as_block] : 0.f;
                weight[u] = in ? p.w_scales[n_tile * p.ws_row + kb * p.ws_block] : 0.f;
            }
        };
        auto store = [&](int c) {
#pragma unroll
            for (int u = 0; u < Cfg::PER_THREAD; ++u) {
                int kb, j;
                place(u, kb, j);
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(smS + (c & 1) * Cfg::SCALE_BYTES + (kb * BT + j) * 4), "f"(token[u] * weight[u]) : "memory");
            }
        };
        fetch(0);
        store(0);
        named_barrier(1, E);
        int b = 0;
        uint32_t acc_phase = 0;
        bool done = false;
        const uint32_t taddr0 = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + col0;
        for (int i = 0; i < nkb; ++i) {
            const int c = i / Cfg::CHUNK, r = i % Cfg::CHUNK;
            const bool more = (c + 1) * Cfg::CHUNK < nkb;
            if (r == 0 && more) fetch(c + 1);
            if (good && !warp_wait_peeked(done, acc_full + 8 * b, acc_phase, 4 * lim)) {
                if (lane == 0) {
                    record_status(p.status, kSiteEpilogue | (i << 8));
                    ctrl[1] = 1;
                }
                good = false;  // (the warps still meet at their barriers)
            }
            if (good) {
                tc_fence_after();
                const auto have_read = [&] {  // every column is in registers
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acc_empty + 8 * b);
                    done = mbar_peek(acc_full + 8 * (b + 1 == NB ? 0 : b + 1), b + 1 == NB ? acc_phase ^ 1u : acc_phase);
                };
                if constexpr (Cfg::SWAP) {
                    const uint32_t sc = smS + (c & 1) * Cfg::SCALE_BYTES + (r * BT + col0) * 4;
                    // up to 32 columns on their way while the scales of the first 16 come from shared memory
                    constexpr int parts = Cfg::COLS / 16;
                    uint32_t v[parts][32];
#pragma unroll
                    for (int g = 0; g < parts; ++g) tmem_ld_32x32b_x16(taddr0 + b * BT + 16 * g, v[g]);
#pragma unroll
                    for (int g = 0; g < parts; ++g) {
                        float4 f[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) f[j] = ld_shared_f4(sc + (16 * g + 4 * j) * 4);
                        if (g == 0) {
                            tmem_ld_wait();
                            have_read();
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            fma2(acc + 16 * g + 4 * j, v[g] + 4 * j, make_float2(f[j].x, f[j].y));
                            fma2(acc + 16 * g + 4 * j + 2, v[g] + 4 * j + 2, make_float2(f[j].z, f[j].w));
                        }
                    }
                } else {
                    uint32_t v[2][32];
                    tmem_ld_32x32b_x32(taddr0 + b * BT, v[0]);
                    tmem_ld_32x32b_x32(taddr0 + b * BT + 32, v[1]);
                    const float scale = ld_shared_f32(smS + (c & 1) * Cfg::SCALE_BYTES + (r * BT + q * 32 + lane) * 4);
                    tmem_ld_wait();
                    have_read();
#pragma unroll
                    for (int j = 0; j < 64; j += 2) fma2(acc + j % Cfg::COLS, v[j / 32] + j % 32, make_float2(scale, scale));
                }
            }
            if (++b == NB) { b = 0; acc_phase ^= 1u; }
            if (r == Cfg::CHUNK - 1 && more) {
                // chunk c+1 goes where chunk c-1 was: every warp has left that one at the last barrier
                store(c + 1);
                named_barrier(1, E);
            }
        }
        // each token's sums to the CTA that adds them up
        if (p.splits > 1) cluster_wait();
        if constexpr (Cfg::SWAP) {
            const uint32_t to = smR + rank * static_cast<uint32_t>(share * Cfg::SUM_PITCH * 4) + (q * 32 + lane) * 4;
            int owner = col0 / share, at = col0 - owner * share;
#pragma unroll
            for (int j = 0; j < Cfg::COLS; ++j) {
                if (good && col0 + j < tokens) {
                    const uint32_t here = to + at * (Cfg::SUM_PITCH * 4);
                    st_cluster_f32(p.splits > 1 ? mapa_shared(here, static_cast<uint32_t>(owner)) : here, acc[j]);
                    if (++at == share) { at = 0; ++owner; }
                }
            }
        } else if (good && q * 32 + lane < tokens) {
            const int owner = (q * 32 + lane) / share, at = q * 32 + lane - owner * share;
            const uint32_t here = smR + ((rank * share + at) * Cfg::SUM_PITCH + col0) * 4;
            const uint32_t to = p.splits > 1 ? mapa_shared(here, static_cast<uint32_t>(owner)) : here;
#pragma unroll
            for (int j = 0; j < Cfg::COLS; j += 4) st_cluster_f4(to + j * 4, acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
        }
    }
    if (warp < 2 && p.splits > 1) cluster_wait();

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && ctrl[1]) {  // copies in flight end before the CTA does
        const int issued = static_cast<int>(ctrl[2]);
        for (int i = max(0, issued - S); i < issued; ++i)
            if (!mbar_wait_for(full + 8 * (i % S), static_cast<uint32_t>((i / S) & 1), lim)) {
                record_status(p.status, kSiteDrain);
                break;
            }
    }
    // every CTA's sums are where they are added; between the two halves of the meeting tensor memory is freed
    if (p.splits > 1) cluster_arrive();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
    }
    if (p.splits > 1) cluster_wait();

    // this CTA's share of the tokens, in rank order, 4 weight rows a thread
    const int first = static_cast<int>(rank) * share, count = min(share, tokens - first);
    for (int e = static_cast<int>(threadIdx.x); e < count * 32; e += Cfg::THREADS) {
        const int j = e >> 5, n = (e & 31) * 4;
        if (n0 + n >= p.N) continue;
        float4 f = ld_shared_f4(smR + (j * Cfg::SUM_PITCH + n) * 4);
        for (int r = 1; r < p.splits; ++r) {
            const float4 g = ld_shared_f4(smR + ((r * share + j) * Cfg::SUM_PITCH + n) * 4);
            f.x += g.x; f.y += g.y; f.z += g.z; f.w += g.w;
        }
        const int64_t to = static_cast<int64_t>(m0 + first + j) * p.ldc + n0 + n;  // N is a multiple of 8
        if (p.c_dtype == SDT_DTYPE_F32) {
            *reinterpret_cast<float4 *>(static_cast<float *>(p.C) + to) = f;
        } else {
            const uint4 h = pack8_f32(f, f, p.c_dtype == SDT_DTYPE_BF16);
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.C) + to) = make_uint2(h.x, h.y);
        }
    }
}

}  // namespace sdt
