// gemm_fp8.cu -- host side of gemm_fp8: checks, the choice of tile and splits, tensor maps.
#include "gemm_fp8.cuh"

#include <algorithm>
#include <cstring>

#include "gemm_fp8_launch.cuh"
#include "host_common.cuh"
#include "overlap.cuh"
#include "tensor_map.cuh"

namespace sdt {

constexpr int64_t kFp8MaxDim = int64_t(1) << 30;
constexpr int kFp8MaxSms = 65536;  // of a plan
constexpr int kFp8MaxSplits = 8;  // CTAs of a portable cluster

struct Fp8Plan {
    int tile, splits;
};

// The items of the two-CTA tiles (256 tokens by `width` outputs): whole tiles up to tail_start, then, if
// the last round would leave at least half of the pairs idle, 256-wide tiles as two halves each.
struct Fp8PairItems {
    int64_t tail_start, num_items, pairs;
};
static Fp8PairItems fp8_pair_items(int64_t M, int64_t N, int sm_count, int width) {
    const int64_t tiles = ((M + 255) / 256) * ((N + width - 1) / width), pairs = std::max(1, sm_count / 2), left = tiles % pairs;
    const int64_t whole = width == 256 && 2 * left <= pairs ? tiles - left : tiles;
    return {whole, whole + 2 * (tiles - whole), pairs};
}

// Tiles of up to 128 tokens run with as many CTAs per tile as still run at once, two to an SM (one
// with 128 tokens).  kResident is the share of those places that clusters of 1 .. 8 CTAs can take
// (GPCs hold whole clusters only; by occupancy queries and start times on 152 SMs).  A second round
// costs more than the split gains: 64 x 6144 x 4096 takes 8.4 us in 48 clusters of 4 and 13.2 us in 48 of 6, of which 46 fit;
// 1 x 28672 x 8192 takes 37 us unsplit and 42 split in 4.
static int fp8_splits(int tile, int64_t tiles, int64_t kb, int sm_count) {
    constexpr double kResident[2][kFp8MaxSplits] = {{1.0, 1.0, 0.908, 0.947, 0.921, 0.908, 0.737, 0.843},
                                                    {1.0, 1.0, 0.908, 0.947, 0.921, 0.908, 0.691, 0.789}};
    const bool alone = tile == 128;
    const int places = alone ? sm_count : 2 * sm_count;
    int splits = 1;
    for (int s = 2; s <= kFp8MaxSplits && 2 * s <= kb; ++s)  // (two blocks a CTA at least)
        if (double(tiles) * s <= kResident[alone][s - 1] * places) splits = s;
    return splits;
}

// The tile: up to 64 tokens the smallest that holds them (larger ones are mostly empty rows), above
// that the smallest of four estimates in microseconds, fitted to measured shapes: a block takes a
// CTA of 64 tokens 0.50 beside another one, a CTA of 128 alone 0.29, a two-CTA tile 0.40 (0.33 if it
// is 192 wide, 0.29 as half-width items).  Where rows of both operands start within 32-byte sectors, the
// first two, which load most per product, cost 22 % more: whether they do follows from the rows' pitch and
// the bases, not from K (333 x 5000 x 4208 with 64, 128, 192 and 256, rows 4208 apart: 22.7, 16.8, 15.5, 17.9; 4224
// apart 19.6, 13.7, 14.9, 17.7; A alone 4208 apart 19.6, 14.4, 15.2, 17.7; W alone 19.9, 14.2, 15.1, 17.7; 4224 apart
// from bases in the middle of a sector 24.8, 18.2, 16.7, 19.1; 512 x 4096 x 4096 with rows 4112 apart 22.0, 16.5, 14.9,
// 14.0, in whole sectors 18.6, 13.2, 13.9, 13.3).  Measured with 64, 128, 192 and 256: 96 x 4096 x 4096 8.5, 8.2, 13.4, 12.5;
// 256 x 4096 x 4096 12.4, 10.5, 13.7, 12.7; 96 x 4096 x 14336 18.0, 16.9, 38.3, 35.7; 512 x 4096 x 4096
// 19.0, 13.4, 14.3, 13.5; 700 x 4096 x 14336 87, 68, 39.6, 46.9; 1021 x 2560 x 7168 47, 38, 22.1, 26.1;
// 1021 x 12288 x 4096 96, 78, 48.6, 45.1.  Over 48 shapes of 96 to 1021 tokens the choice is 0.1 % slower
// than the best on average, 4 % at worst.
// broken: whether rows of both operands start within sectors.  `tile`: 0, or the tile that the caller asks for.
static Fp8Plan fp8_plan(int64_t M, int64_t N, int64_t K, int sm_count, bool broken, int tile = 0) {
    const int64_t kb = (K + kFp8Block - 1) / kFp8Block;
    const auto tiles = [&](int t) { return ((M + t - 1) / t) * ((N + 127) / 128); };
    if (tile == 0) tile = M <= 16 ? 16 : M <= 32 ? 32 : 64;
    else if (tile > 128) return {tile, 1};
    else return {tile, fp8_splits(tile, tiles(tile), kb, sm_count)};
    Fp8Plan best{tile, fp8_splits(tile, tiles(tile), kb, sm_count)};
    if (M <= 64) return best;
    const auto blocks = [&](int splits) { return double((kb + splits - 1) / splits); };
    const double sectors = broken ? 1.22 : 1.0;
    double least = 3.5 + 0.50 * sectors * blocks(best.splits) * std::max(1.0, double(tiles(64)) * best.splits / (2 * sm_count));
    const int splits = fp8_splits(128, tiles(128), kb, sm_count);
    const double alone = 3.5 + 0.29 * sectors * blocks(splits) * double((tiles(128) * splits + sm_count - 1) / sm_count);
    if (alone < least) {
        least = alone;
        best = {128, splits};
    }
    for (int width : {256, 192}) {
        const Fp8PairItems items = fp8_pair_items(M, N, sm_count, width);
        const double rounds = double((items.tail_start + items.pairs - 1) / items.pairs);
        const double paired = 4.0 + double(kb) * ((width == 256 ? 0.40 : 0.33) * rounds + (items.num_items > items.tail_start ? 0.29 : 0.0));
        if (paired < least) {
            least = paired;
            best = {width, 1};
        }
    }
    return best;
}

// The stride of rows of k 8-bit values that lie behind one another.
static int64_t fp8_packed_row(int64_t k) { return (k + 15) / 16 * 16; }

// The plan of a checked call of at least one row, column and k.
static Fp8Plan fp8_plan(const sdt_gemm_fp8 &c, int sm_count) {
    const auto broken = [](const void *p, int64_t rows, int64_t stride) {
        return reinterpret_cast<uintptr_t>(p) % 32 != 0 || (rows > 1 && stride % 32 != 0);
    };
    Fp8Plan plan = fp8_plan(c.M, c.N, c.K, sm_count, broken(c.a, c.M, c.lda) && broken(c.w, c.N, c.ldw), c.tile);
    if (c.splits && plan.tile <= 128) plan.splits = c.splits;
    plan.splits = int(std::min<int64_t>(plan.splits, (c.K + kFp8Block - 1) / kFp8Block));
    return plan;
}

static bool is_fp8(int t) { return t == SDT_DTYPE_E4M3 || t == SDT_DTYPE_E5M2; }
static bool at(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

static int check_fp8(const sdt_gemm_fp8 &c) {
    if (c.M < 0 || c.N < 0 || c.K < 0 || c.M > kFp8MaxDim || c.N > kFp8MaxDim || c.K > kFp8MaxDim)
        return fail(SDT_ERR_SHAPE, "gemm_fp8: M, N and K must be in 0 .. 2^30 (got %lld, %lld, %lld)", (long long)c.M,
                    (long long)c.N, (long long)c.K);
    if (c.N % 8) return fail(SDT_ERR_SHAPE, "gemm_fp8: N must be a multiple of 8 (got %lld)", (long long)c.N);
    if (!is_fp8(c.a_dtype) || !is_fp8(c.w_dtype)) return fail(SDT_ERR_ARG, "gemm_fp8: A and W must be e4m3 or e5m2");
    if (c.c_dtype != SDT_DTYPE_F16 && c.c_dtype != SDT_DTYPE_BF16 && c.c_dtype != SDT_DTYPE_F32)
        return fail(SDT_ERR_ARG, "gemm_fp8: C must be fp16, bf16 or fp32 (dtype %d)", c.c_dtype);
    if (c.tile != 0 && c.tile != 16 && c.tile != 32 && c.tile != 64 && c.tile != 128 && c.tile != 192 && c.tile != 256)
        return fail(SDT_ERR_TILE, "gemm_fp8: no tile %d", c.tile);
    if (c.splits < 0 || c.splits > kFp8MaxSplits) return fail(SDT_ERR_ARG, "gemm_fp8: splits must be in 0 .. %d", kFp8MaxSplits);
    if (c.M == 0 || c.N == 0) return SDT_OK;
    if (!c.c) return fail(SDT_ERR_NULL, "gemm_fp8: C is NULL");
    if (!at(c.c, 16)) return fail(SDT_ERR_ALIGN, "gemm_fp8: C must be 16-byte aligned");
    if (c.M > 1 && (c.ldc < c.N || c.ldc % 8)) return fail(SDT_ERR_ARG, "gemm_fp8: ldc must be a multiple of 8, at least N (got %lld)", (long long)c.ldc);
    if (c.K == 0) return SDT_OK;
    if (!c.a || !c.w || !c.a_scales || !c.w_scales) return fail(SDT_ERR_NULL, "gemm_fp8: NULL operand or scales");
    if (!at(c.a, 16) || !at(c.w, 16)) return fail(SDT_ERR_ALIGN, "gemm_fp8: A and W must be 16-byte aligned");
    if (!at(c.a_scales, 4) || !at(c.w_scales, 4)) return fail(SDT_ERR_ALIGN, "gemm_fp8: scales must be 4-byte aligned");
    if (c.M > 1 && (c.lda < c.K || c.lda % 16)) return fail(SDT_ERR_ARG, "gemm_fp8: lda must be a multiple of 16, at least K (got %lld)", (long long)c.lda);
    if (c.N > 1 && (c.ldw < c.K || c.ldw % 16)) return fail(SDT_ERR_ARG, "gemm_fp8: ldw must be a multiple of 16, at least K (got %lld)", (long long)c.ldw);
    // strides that TMA takes (below 2^40 bytes), and scale offsets within 64 bits
    constexpr int64_t most = int64_t(1) << 32;
    if ((c.M > 1 && (c.lda >= most || c.ldc >= most)) || (c.N > 1 && c.ldw >= most)) return fail(SDT_ERR_ARG, "gemm_fp8: strides must be below 2^32 elements");
    const bool rows = c.M > 1, blocks = c.K > kFp8Block, panels = c.N > kFp8Block;  // (a dimension of one never steps)
    for (int64_t s : {rows ? c.as_row : 0, blocks ? c.as_block : 0, panels ? c.ws_row : 0, blocks ? c.ws_block : 0})
        if (s < 0 || s >= most) return fail(SDT_ERR_ARG, "gemm_fp8: scale strides must be in 0 .. 2^32 (got %lld)", (long long)s);
    const int64_t size = c.c_dtype == SDT_DTYPE_F32 ? 4 : 2, kb = (c.K + kFp8Block - 1) / kFp8Block, nb = (c.N + kFp8Block - 1) / kFp8Block;
    const Stretches out = rows_of(c.c, c.M, step_bytes(c.M, c.ldc, size), c.N * size);
    if (overlap(out, rows_of(c.a, c.M, c.lda, c.K)) || overlap(out, rows_of(c.w, c.N, c.ldw, c.K)))
        return fail(SDT_ERR_ARG, "gemm_fp8: C and an operand overlap");
    if (overlap(out, {c.a_scales, c.M, step_bytes(c.M, c.as_row, 4), kb, step_bytes(kb, c.as_block, 4), 4}) ||
        overlap(out, {c.w_scales, nb, step_bytes(nb, c.ws_row, 4), kb, step_bytes(kb, c.ws_block, 4), 4}))
        return fail(SDT_ERR_ARG, "gemm_fp8: C and the scales overlap");
    return SDT_OK;
}

static int run_swap(const sdt_gemm_fp8 &c, const Fp8Plan &plan, Fp8Args &a, int64_t lda, int64_t ldw, cudaStream_t stream) {
    a.num_m_tiles = int((c.M + plan.tile - 1) / plan.tile);
    a.num_n_tiles = int((c.N + 127) / 128);
    a.splits = plan.splits;
    if (int64_t(a.num_m_tiles) * a.num_n_tiles * a.splits > INT32_MAX) return fail(SDT_ERR_SHAPE, "gemm_fp8: grid too large");
    // W is the MMA's first operand, but for tiles of 128 tokens
    const uint32_t a_type = c.a_dtype == SDT_DTYPE_E5M2 ? 1u : 0u, w_type = c.w_dtype == SDT_DTYPE_E5M2 ? 1u : 0u;
    a.idesc = (1u << 4) | ((plan.tile == 128 ? a_type : w_type) << 7) | ((plan.tile == 128 ? w_type : a_type) << 10);
    CUtensorMap tmW, tmX;
    int rc = tensor_map_2d(c.w, c.w_dtype, uint64_t(c.K), uint64_t(c.N), uint64_t(ldw), 128, &tmW, kFp8Block);
    if (!rc) rc = tensor_map_2d(c.a, c.a_dtype, uint64_t(c.K), uint64_t(c.M), uint64_t(lda), plan.tile, &tmX, kFp8Block);
    if (rc) return rc;
    int e = plan.tile == 16   ? launch_fp8_swap<16>(tmW, tmX, a, stream)
            : plan.tile == 32 ? launch_fp8_swap<32>(tmW, tmX, a, stream)
            : plan.tile == 64 ? launch_fp8_swap<64>(tmW, tmX, a, stream)
                              : launch_fp8_swap<128>(tmW, tmX, a, stream);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(SDT_ERR_LAUNCH, "gemm_fp8 launch failed: %s", cudaGetErrorString(cudaError_t(e)));
    }
    return SDT_OK;
}

static int run_pair(const sdt_gemm_fp8 &c, int width, Fp8Args &a, int64_t lda, int64_t ldw, const DeviceInfo &dev, cudaStream_t stream) {
    const Fp8PairItems items = fp8_pair_items(c.M, c.N, dev.sm_count, width);
    if (items.num_items > INT32_MAX / 2) return fail(SDT_ERR_SHAPE, "gemm_fp8: grid too large");
    a.num_m_tiles = int((c.M + 255) / 256);
    a.num_n_tiles = int((c.N + width - 1) / width);
    a.splits = 1;
    a.raster_group = 8;
    a.tail_start = int(items.tail_start);
    a.num_items = int(items.num_items);
    a.idesc = (1u << 4) | ((c.a_dtype == SDT_DTYPE_E5M2 ? 1u : 0u) << 7) | ((c.w_dtype == SDT_DTYPE_E5M2 ? 1u : 0u) << 10);
    CUtensorMap tmA, tmB, tmC;
    int rc = tensor_map_2d(c.a, c.a_dtype, uint64_t(c.K), uint64_t(c.M), uint64_t(lda), 128, &tmA, kFp8Block);
    if (!rc) rc = tensor_map_2d(c.w, c.w_dtype, uint64_t(c.K), uint64_t(c.N), uint64_t(ldw), width == 256 ? 64 : width / 2, &tmB, kFp8Block);
    // C leaves in boxes of 64-byte rows
    const uint64_t size = c.c_dtype == SDT_DTYPE_F32 ? 4 : 2;
    if (!rc) rc = tensor_map_2d(c.c, c.c_dtype, uint64_t(c.N), uint64_t(c.M), uint64_t(a.ldc) * size, 32, &tmC, int(64 / size), CU_TENSOR_MAP_SWIZZLE_64B);
    if (rc) return rc;
    const int pairs = int(std::min(items.pairs, items.num_items));
    const int e = width == 256 ? launch_fp8_pair<256>(tmA, tmB, tmC, a, pairs, stream) : launch_fp8_pair<192>(tmA, tmB, tmC, a, pairs, stream);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(SDT_ERR_LAUNCH, "gemm_fp8 launch failed: %s", cudaGetErrorString(cudaError_t(e)));
    }
    return SDT_OK;
}

}  // namespace sdt

using namespace sdt;

extern "C" {

int sdt_gemm_fp8_plan_for(int64_t M, int64_t N, int64_t K, int sm_count, int *tile, int *splits) {
    clear_error();
    if (!tile || !splits) return fail(SDT_ERR_NULL, "NULL output pointer");
    if (M < 1 || N < 1 || K < 1 || M > kFp8MaxDim || N > kFp8MaxDim || K > kFp8MaxDim || sm_count < 1 || sm_count > kFp8MaxSms)
        return fail(SDT_ERR_SHAPE, "M, N, K must be in 1 .. 2^30, sm_count in 1 .. 65536");
    const Fp8Plan p = fp8_plan(M, N, K, sm_count, fp8_packed_row(K) % 32 != 0);
    *tile = p.tile;
    *splits = p.splits;
    return SDT_OK;
}

int sdt_gemm_fp8_plan_call(const sdt_gemm_fp8 *call, int sm_count, int *tile, int *splits) {
    clear_error();
    if (!call || !tile || !splits) return fail(SDT_ERR_NULL, "gemm_fp8: NULL call or output pointer");
    sdt_gemm_fp8 c;
    memcpy(&c, call, sizeof c);
    const int rc = check_fp8(c);
    if (rc) return rc;
    if (c.M < 1 || c.N < 1 || c.K < 1 || sm_count < 1 || sm_count > kFp8MaxSms)
        return fail(SDT_ERR_SHAPE, "M, N, K must be at least 1, sm_count in 1 .. 65536");
    const Fp8Plan p = fp8_plan(c, sm_count);
    *tile = p.tile;
    *splits = p.splits;
    return SDT_OK;
}

int gemm_fp8(const sdt_gemm_fp8 *call, sdt_stream_t stream_h) {
    clear_error();
    if (!call) return fail(SDT_ERR_NULL, "gemm_fp8: NULL call");
    sdt_gemm_fp8 c;
    memcpy(&c, call, sizeof c);  // (a packed call may lie at any address)
    int rc = check_fp8(c);
    if (rc || c.M == 0 || c.N == 0) return rc;
    DeviceInfo dev;
    rc = current_device(&dev);
    if (rc) return rc;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_h);
    // a dimension of one never steps: its stride may be anything
    const int64_t lda = c.M > 1 ? c.lda : fp8_packed_row(c.K), ldw = c.N > 1 ? c.ldw : fp8_packed_row(c.K), ldc = c.M > 1 ? c.ldc : c.N;
    const size_t size = c.c_dtype == SDT_DTYPE_F32 ? 4 : 2;
    if (c.K == 0) {
        const cudaError_t e = cudaMemset2DAsync(c.c, size_t(ldc) * size, 0, size_t(c.N) * size, size_t(c.M), stream);
        if (e == cudaSuccess) return SDT_OK;
        cudaGetLastError();
        return fail(SDT_ERR_CUDA, "gemm_fp8: zeroing C failed: %s", cudaGetErrorString(e));
    }
    Fp8Args a;
    memset(&a, 0, sizeof a);
    a.a_scales = c.a_scales;
    a.w_scales = c.w_scales;
    a.C = c.c;
    a.as_row = c.M > 1 ? c.as_row : 0;
    a.as_block = c.K > kFp8Block ? c.as_block : 0;
    a.ws_row = c.N > kFp8Block ? c.ws_row : 0;
    a.ws_block = c.K > kFp8Block ? c.ws_block : 0;
    a.ldc = ldc;
    a.M = int(c.M);
    a.N = int(c.N);
    a.num_kb = int((c.K + kFp8Block - 1) / kFp8Block);
    a.c_dtype = c.c_dtype;
    a.timeout_ns = wait_timeout_ns();
    rc = status_word(&a.status);
    if (rc) return rc;
    const Fp8Plan plan = fp8_plan(c, dev.sm_count);
    if (plan.tile > 128) return run_pair(c, plan.tile, a, lda, ldw, dev, stream);
    return run_swap(c, plan, a, lda, ldw, stream);
}

}  // extern "C"
