// w4.hip -- products with 4-bit weights and group scales: contexts, packing
// and the entry points. The formula and the layout are in w4.h.
#include "w4_rows.h"
#include "w4_tile.h"

#include <algorithm>
#include <new>
#include <stdio.h>

namespace {

using namespace dq;

// bytes of x that the kernel for few rows takes to LDS
constexpr int64_t kXLds = 64 << 10;
// rows an expert from which the kernel for many rows is taken
constexpr int kTileMean = 64;
// bytes that a context keeps for prepared rows; more rows go in several launches
constexpr int64_t kCopyBytes = 64 << 20, kSumsBytes = 32 << 20;

struct PackArgs {
    const uint8_t* codes;   // [experts][rows][(K + 1) / 2]
    const uint8_t* scales;  // [experts][rows][G], 2 or 4 bytes each
    const uint8_t* zeros;   // [experts][rows][(G + 1) / 2]
    const float* bias;      // [experts][rows]
    uint8_t* codes_out;
    uint8_t* scales_out;
    uint8_t* zeros_out;
    float* bias_out;
    int N, K, group, G, gated, tiles, blocks, S, scale_bytes;
};

// The caller's row of a packed one, -1 where there is none.
__device__ __forceinline__ int packed_row(const PackArgs& A, int tile, int c) {
    if (!A.gated) {
        const int n = tile * 16 + c;
        return n < A.N ? n : -1;
    }
    const int n = tile / 2 * 16 + c;
    return n < A.N ? n + (tile & 1) * A.N : -1;
}

// One workgroup of 64 lanes a block of a tile; grid x: tiles, y: blocks, z: experts.
__global__ void __launch_bounds__(64) k_w4_pack(PackArgs A) {
    const int lane = threadIdx.x, tile = blockIdx.x, block = blockIdx.y, e = blockIdx.z;
    const int rows = A.N * (A.gated ? 2 : 1);
    const size_t out = ((size_t)e * A.tiles + tile) * A.blocks + block;
    const int n = packed_row(A, tile, lane & 15), half = (A.K + 1) / 2;
    u4 w = {0, 0, 0, 0};
    if (n >= 0) {
        const uint8_t* row = A.codes + ((size_t)e * rows + n) * half;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            // element i of the caller's order, in byte i / 2, goes to byte i % 4, half i / 4
            const int k = block * kW4Block + q * 32 + (lane >> 4) * 8;
            unsigned v = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const unsigned code = k + i < A.K ? (row[(k + i) >> 1] >> (4 * (i & 1))) & 15u : 0u;
                v |= code << (8 * (i & 3) + 4 * (i >> 2));
            }
            w[q] = v;
        }
    }
    reinterpret_cast<u4*>(A.codes_out)[out * 64 + lane] = w;
    // scales and zero points of 16 rows and S groups
    if (lane < 16 * A.S) {
        const int r = packed_row(A, tile, lane / A.S);
        const int g = (block * kW4Block + lane % A.S * (kW4Block / A.S)) / A.group;
        const bool some = r >= 0 && g < A.G;
        const size_t i = some ? ((size_t)e * rows + r) * A.G + g : 0, o = out * 16 * A.S + lane;
        for (int b = 0; b < A.scale_bytes; ++b)
            A.scales_out[o * A.scale_bytes + b] = some ? A.scales[i * A.scale_bytes + b] : 0;
        if (A.zeros_out) {
            const size_t at = some ? ((size_t)e * rows + r) * ((A.G + 1) / 2) + g / 2 : 0;
            A.zeros_out[o] = some ? (A.zeros[at] >> (4 * (g & 1))) & 15 : 0;
        }
    }
    if (A.bias_out && block == 0 && lane < 16) {
        const int r = packed_row(A, tile, lane);
        A.bias_out[((size_t)e * A.tiles + tile) * 16 + lane] = r >= 0 ? A.bias[(size_t)e * rows + r] : 0.0f;
    }
}

int elem_bytes(int type) { return type == DQ_F32 ? 4 : 2; }
bool is_float(dq_dtype t) { return t == DQ_F32 || t == DQ_BF16 || t == DQ_F16; }

int check_device(const dq_w4_ctx* c) {
    int dev = 0;
    (void)hipGetDevice(&dev);
    if (dev != c->device) DQ_FAIL(DQ_ERR_STATE, "the context belongs to another device");
    return DQ_OK;
}

// The tensors of a forward, after its sizes.
int check_forward(const dq_w4_ctx* c, const void* x, int64_t x_row_stride, const void* y) {
    if (!c->ready) DQ_FAIL(DQ_ERR_STATE, "no weights: dq_w4_set_w first");
    if (!x || !y) DQ_FAIL(DQ_ERR_ARG, "x and y must not be NULL");
    if (x_row_stride < 0) DQ_FAIL(DQ_ERR_ARG, "x_row_stride must be >= 0");
    if ((uintptr_t)x % elem_bytes(c->x_type) || (uintptr_t)y % elem_bytes(c->y_type))
        DQ_FAIL(DQ_ERR_ARG, "a tensor is not aligned to its elements");
    return check_device(c);
}

W4Args forward_args(const dq_w4_ctx* c, const void* x, int64_t x_row_stride, void* y) {
    W4Args A{};
    A.x = x;
    A.x_stride = x_row_stride;
    A.codes = c->codes;
    A.scales = c->scales;
    A.zeros = c->has_zeros ? c->zeros : nullptr;
    A.bias = c->has_bias ? c->bias : nullptr;
    A.y = y;
    A.N = c->N;
    A.K = c->K;
    A.experts = c->experts;
    A.tiles = c->tiles;
    A.blocks = c->blocks;
    A.scale_type = c->scale_type;
    A.y_type = c->y_type;
    A.gated = c->gated;
    // 8 elements at a time, 16 bytes each load: rows start at a multiple of those, and K ends at one
    const int per16 = 16 / elem_bytes(c->x_type);
    A.vec = (uintptr_t)x % 16 == 0 && x_row_stride % per16 == 0 && c->K % 8 == 0;
    return A;
}

W4Kernels kernels_of(const dq_w4_ctx* c) {
    return c->x_type == DQ_F32 ? w4_kernels_f32() : c->x_type == DQ_BF16 ? w4_kernels_bf16() : w4_kernels_f16();
}

int launch_rows(const dq_w4_ctx* c, W4Args A, hipStream_t s) {
    const bool gated = c->gated;
    const int used = (c->N + 15) / 16 * (gated ? 2 : 1), least = gated ? 2 : 1;
    const int mean = A.offsets ? (A.rows + c->experts - 1) / c->experts : A.rows;
    // rows that start 16 bytes apart, in reach of 31 bits
    const __int128 reach = (__int128)(A.row_index ? A.x_rows : 64) * A.x_stride + A.K;
    const bool fast = A.vec && reach * elem_bytes(c->x_type) < (__int128)kW4Far;
    int TM, col_tiles, waves;
    bool in_lds = false;
    const int64_t x_row = ((int64_t)c->blocks * kW4Block * 2 + 64) * (c->x_type == DQ_F32 ? 3 : 1);
    if (fast) {
        // experts' rows differ: twice the mean in one tile of rows
        const int rows = A.offsets ? 2 * mean : mean;
        auto fits = [&](int tm) { return (A.offsets ? tm : std::min(tm, A.rows)) * x_row <= kXLds; };
        TM = rows <= 4 && fits(4) ? 4 : rows >= 64 ? 64 : (rows + 15) / 16 * 16;
        in_lds = TM == 4;
    } else {
        TM = mean <= 16 ? 16 : 64;
    }
    const int row_tiles = (TM + 15) / 16;
    const int64_t tiles_m = A.offsets ? (int64_t)A.rows / TM + std::min(A.rows, c->experts) : (A.rows + TM - 1) / TM;
    if (fast) {
        // Wide workgroups read x less often (rows of 48: 4 column tiles take half
        // the time of 1), as long as there are waves for the whole chip: 16 a
        // compute unit, 8 of those that hold many sums
        const int narrow = in_lds ? least : 2;
        col_tiles = 4;
        auto most = [&](int ct) {
            return std::min(in_lds && ct <= 2 ? 16 : !in_lds && c->x_type == DQ_F32 && row_tiles >= 3 ? 4 : 8, c->blocks);
        };
        auto want = [&](int ct) { return (int64_t)c->cus * (in_lds && ct <= 2 ? 16 : 8); };
        while (col_tiles > narrow && tiles_m * (used / col_tiles) * most(col_tiles) < want(col_tiles)) col_tiles /= 2;
        waves = std::min(in_lds ? 1 : 4, most(col_tiles));
        while (waves * 2 <= most(col_tiles) && tiles_m * (used / col_tiles) * waves < want(col_tiles)) waves *= 2;
    } else {
        col_tiles = least;
        waves = 8;
        while (waves > 1 && waves / 2 >= c->blocks) waves /= 2;
    }
    A.col_groups = (used + col_tiles - 1) / col_tiles;
    const int64_t grid = tiles_m * A.col_groups;
    if (grid > INT32_MAX) DQ_FAIL(DQ_ERR_RANGE, "too many rows for one launch");
    const W4Kernels k = kernels_of(c);
    // LDS that the launch brings: rows of x or the waves' parts, 64 KiB at most; the
    // rings are the kernel's own
    size_t lds = 0;
    if (!fast) lds = (size_t)waves * col_tiles * row_tiles * 1024;
    else if (in_lds) lds = std::max((size_t)waves * col_tiles * 256, (size_t)((A.offsets ? TM : std::min(TM, A.rows)) * x_row));
    A.per_row = make_fastdiv((uint32_t)c->blocks * (kW4Block / 8));
    const W4RowsKernel f = fast ? k.rows(TM, col_tiles, c->S, c->scale_type) : k.any(TM, col_tiles, c->S);
    if (!f) DQ_FAIL(DQ_ERR_RANGE, "no kernel of %d rows by %d column tiles", TM, col_tiles);
    hipLaunchKernelGGL(f, dim3((unsigned)grid), dim3(waves * 64), lds, s, A);
    DQ_LAUNCH_CHECK("product with 4-bit weights");
    return DQ_OK;
}

// The tile kernel's offsets within x are 32 bits.
bool tile_reaches(const dq_w4_ctx* c, const W4Args& A) {
    const __int128 rows = A.row_index ? A.x_rows : kW4TileRows;
    return rows * A.x_stride * 2 + A.K * 2 < ((__int128)1 << 32);
}

int launch_tile(const dq_w4_ctx* c, const W4Args& A, hipStream_t s) {
    const W4Kernels k = kernels_of(c);
    // rows of whole blocks of 16 bits that lie 16 bytes apart are taken where they are
    const bool copy = c->x_type == DQ_F32 || !A.vec || c->K % kW4Block || !tile_reaches(c, A);
    const int64_t slab = copy ? c->copy_rows : c->sums_rows;
    // rows of x are prepared once where they all fit, else as rows of y
    const bool by_row = A.row_index ? A.x_rows > slab || A.x_rows > A.rows : true;
    const int P = c->x_type == DQ_F32 ? 3 : 1, Kp = c->blocks * kW4Block;
    for (int64_t lo = 0; lo < A.rows; lo += slab) {
        const int64_t hi = std::min<int64_t>(A.rows, lo + slab);
        if (by_row || lo == 0) {
            W4Prepare B{};
            B.x = A.x;
            B.x_stride = A.x_stride;
            B.rows = by_row ? (int)(hi - lo) : A.x_rows;
            B.x_rows = A.x_rows;
            if (by_row && A.row_index) B.row_index = A.row_index + lo;
            else if (by_row) {
                B.x = (const char*)A.x + lo * A.x_stride * elem_bytes(c->x_type);
                B.x_rows = B.rows;
            }
            B.K = c->K;
            B.blocks = c->blocks;
            B.S = c->S;
            B.vec = A.vec;
            B.copy = copy ? c->copy : nullptr;
            B.sums = c->sums;
            hipLaunchKernelGGL(k.prepare, dim3((unsigned)((B.rows + 3) / 4)), dim3(256), 0, s, B);
            DQ_LAUNCH_CHECK("preparation of rows");
        }
        W4TileArgs T{};
        T.a = A;
        T.sums = c->sums;
        T.by_row = by_row;
        T.x_by_row = by_row && copy;
        if (copy) {
            T.a.x = c->copy;
            T.a.x_stride = (long long)P * Kp;
        }
        T.row_lo = (int)lo;
        T.row_hi = (int)hi;
        const int used = (c->N + 15) / 16 * (c->gated ? 2 : 1);
        const int64_t rows = hi - lo;
        const int64_t tiles_m = A.offsets ? rows / kW4TileRows + std::min<int64_t>(rows, c->experts)
                                          : (rows + kW4TileRows - 1) / kW4TileRows;
        // 256 columns a workgroup where that leaves one for every compute unit, else 128
        // (us of 256 / 128: 4096 rows of 4096 x 4096 154 / 161, 1024 rows 67 / 53)
        const int wide = (rows + kW4TileRows - 1) / kW4TileRows * ((used + 15) / 16) >= c->cus ? 4 : 2;
        T.tiles_n = (used + 4 * wide - 1) / (4 * wide);
        T.tiles_m = (int)tiles_m;
        // units of 4 x 4 tiles (of 256 columns, else 4 x 8) to an XCD, smaller ones where there are few
        T.gm = 4;
        T.gn = 16 / wide;
        auto units = [&] { return (tiles_m + T.gm - 1) / T.gm * ((T.tiles_n + T.gn - 1) / T.gn); };
        while (T.gn > 1 && units() < 32) T.gn /= 2;
        while (T.gm > 1 && units() < 32) T.gm /= 2;
        const int64_t grid = (units() + 7) / 8 * 8 * T.gm * T.gn;
        if (grid > INT32_MAX) DQ_FAIL(DQ_ERR_RANGE, "too many rows for one launch");
        T.vec_store = (uintptr_t)A.y % 16 == 0 && c->N % 8 == 0;
        hipLaunchKernelGGL(k.tile(wide, c->S, c->scale_type, A.row_index && !T.x_by_row), dim3((unsigned)grid), dim3(128 * wide), 0, s, T);
        DQ_LAUNCH_CHECK("product with 4-bit weights");
    }
    return DQ_OK;
}

// Many rows, where an expert has more than a tile of the other kernel's (kTileMean) and there
// are tiles of 128 x 128 for three quarters of the chip: a tile takes its time
// whatever the others do, and few of them leave the rest idle. 4096 x 4096, us
// (this one / the other): 512 rows (128 tiles) 51.8 / 44.0, 1024 rows 53.9 / 84.1;
// 16384 x 4096: 128 rows (128 tiles) 72.2 / 44.7, 256 rows 72.1 / 86.0. Rows that
// do not lie 16 bytes apart go there from the same rows on: it copies them first.
int launch(const dq_w4_ctx* c, const W4Args& A, hipStream_t s) {
    const int mean = A.offsets ? (A.rows + c->experts - 1) / c->experts : A.rows;
    const int used = (c->N + 15) / 16 * (c->gated ? 2 : 1);
    const int64_t tiles = (int64_t)((A.rows + kW4TileRows - 1) / kW4TileRows) * ((used + 7) / 8);
    if (mean > kTileMean && (tiles * 4 > c->cus * 3 || !A.vec) && c->copy_rows) return launch_tile(c, A, s);
    return launch_rows(c, A, s);
}

}  // namespace

extern "C" int dq_w4_init(dq_w4_ctx** ctx, int64_t experts, int64_t N, int64_t K, int64_t group, dq_dtype x_type,
                          dq_dtype scale_type, dq_dtype y_type, int gated, int64_t max_rows) {
    if (!ctx) DQ_FAIL(DQ_ERR_ARG, "ctx is NULL");
    *ctx = nullptr;
    if (experts < 1 || N < 1 || K < 1 || max_rows < 1) DQ_FAIL(DQ_ERR_ARG, "sizes must be >= 1");
    if (group != 32 && group != 64 && (group < 128 || group % 128))
        DQ_FAIL(DQ_ERR_ARG, "group must be 32, 64 or a multiple of 128");
    if (!is_float(x_type) || !is_float(scale_type) || !is_float(y_type))
        DQ_FAIL(DQ_ERR_TYPE, "x, scales and y must be fp32, bf16 or fp16");
    if (experts > DQ_W4_EXPERTS_MAX || N > DQ_W4_N_MAX || K > DQ_W4_K_MAX || max_rows > DQ_W4_ROWS_MAX)
        DQ_FAIL(DQ_ERR_RANGE, "experts, N, K or max_rows exceed %d, %d, %d, %d", DQ_W4_EXPERTS_MAX, DQ_W4_N_MAX,
                DQ_W4_K_MAX, DQ_W4_ROWS_MAX);
    dq_w4_ctx* c = new (std::nothrow) dq_w4_ctx();
    if (!c) DQ_FAIL(DQ_ERR_ALLOC, "host allocation for the 4-bit weights' context failed");
    (void)hipGetDevice(&c->device);
    if (hipDeviceGetAttribute(&c->cus, hipDeviceAttributeMultiprocessorCount, c->device) != hipSuccess || c->cus < 1)
        c->cus = 256;
    c->experts = (int)experts;
    c->N = (int)N;
    c->K = (int)K;
    c->group = (int)std::min<int64_t>(group, 1 << 30);
    c->x_type = x_type;
    c->scale_type = scale_type;
    c->y_type = y_type;
    c->gated = gated != 0;
    c->max_rows = max_rows;
    c->tiles = (int)(((N + 15) / 16 * (gated ? 2 : 1) + kW4TilePad - 1) / kW4TilePad * kW4TilePad);
    c->blocks = (int)((K + kW4Block - 1) / kW4Block);
    c->S = group >= 128 ? 1 : (int)(128 / group);
    const size_t units = (size_t)experts * c->tiles * c->blocks;
    if (max_rows > kTileMean) {
        const int64_t row = (int64_t)c->blocks * kW4Block * 2 * (x_type == DQ_F32 ? 3 : 1), sum = (int64_t)c->blocks * c->S * 4;
        auto fit = [&](int64_t bytes, int64_t one) {
            return std::min(max_rows, std::max<int64_t>(kW4TileRows, bytes / one / kW4TileRows * kW4TileRows));
        };
        c->copy_rows = fit(kCopyBytes, row);
        c->sums_rows = std::max(c->copy_rows, fit(kSumsBytes, sum));
        if (hipMalloc(&c->copy, c->copy_rows * row) != hipSuccess || hipMalloc(&c->sums, c->sums_rows * sum) != hipSuccess) {
            dq_w4_release(c);
            DQ_FAIL(DQ_ERR_ALLOC, "device allocation for the 4-bit weights' context failed");
        }
    }
    const bool ok = hipMalloc(&c->codes, units * 1024) == hipSuccess &&
                    hipMalloc(&c->scales, units * 16 * c->S * elem_bytes(scale_type)) == hipSuccess &&
                    hipMalloc(&c->zeros, units * 16 * c->S) == hipSuccess &&
                    hipMalloc(&c->bias, (size_t)experts * c->tiles * 64) == hipSuccess;
    if (!ok) {
        dq_w4_release(c);
        DQ_FAIL(DQ_ERR_ALLOC, "device allocation for the 4-bit weights' context failed");
    }
    const char* names[] = {"fp32", "bf16", "int8", "uint8", "fp16"};
    snprintf(c->info, sizeof c->info, "gfx950 4-bit weights: %d experts, N %d, K %d, groups of %lld, %s x, %s scales, "
             "%s y%s", c->experts, c->N, c->K, (long long)group, names[x_type], names[scale_type], names[y_type],
             gated ? ", gated" : "");
    *ctx = c;
    return DQ_OK;
}

extern "C" int dq_w4_set_w(dq_w4_ctx* ctx, const void* codes, const void* scales, const void* zeros, const float* bias,
                           void* stream) {
    if (!ctx) DQ_FAIL(DQ_ERR_STATE, "no context");
    if (!codes || !scales) DQ_FAIL(DQ_ERR_ARG, "codes and scales must not be NULL");
    if ((uintptr_t)scales % elem_bytes(ctx->scale_type) || (uintptr_t)bias % 4)
        DQ_FAIL(DQ_ERR_ARG, "a tensor is not aligned to its elements");
    if (int rc = check_device(ctx)) return rc;
    PackArgs A{};
    A.codes = (const uint8_t*)codes;
    A.scales = (const uint8_t*)scales;
    A.zeros = (const uint8_t*)zeros;
    A.bias = bias;
    A.codes_out = ctx->codes;
    A.scales_out = (uint8_t*)ctx->scales;
    A.zeros_out = zeros ? ctx->zeros : nullptr;
    A.bias_out = bias ? ctx->bias : nullptr;
    A.N = ctx->N;
    A.K = ctx->K;
    A.group = ctx->group;
    A.G = (ctx->K - 1) / ctx->group + 1;
    A.gated = ctx->gated;
    A.tiles = ctx->tiles;
    A.blocks = ctx->blocks;
    A.S = ctx->S;
    A.scale_bytes = elem_bytes(ctx->scale_type);
    const hipStream_t s = (hipStream_t)stream;
    ctx->ready = false;
    hipLaunchKernelGGL(k_w4_pack, dim3(ctx->tiles, ctx->blocks, ctx->experts), dim3(64), 0, s, A);
    DQ_LAUNCH_CHECK("packing of 4-bit weights");
    DQ_HIP_CHECK(hipStreamSynchronize(s));
    ctx->has_zeros = zeros != nullptr;
    ctx->has_bias = bias != nullptr;
    ctx->ready = true;
    return DQ_OK;
}

extern "C" int dq_w4_forward(dq_w4_ctx* ctx, int64_t rows, const void* x, int64_t x_row_stride, void* y,
                             void* stream) {
    if (!ctx) DQ_FAIL(DQ_ERR_STATE, "no context");
    if (ctx->experts != 1) DQ_FAIL(DQ_ERR_ARG, "a context of several experts takes dq_w4_forward_grouped");
    if (rows < 0 || rows > ctx->max_rows) DQ_FAIL(DQ_ERR_ARG, "rows must lie in [0, %lld]", (long long)ctx->max_rows);
    if (rows == 0) return DQ_OK;
    if (int rc = check_forward(ctx, x, x_row_stride, y)) return rc;
    W4Args A = forward_args(ctx, x, x_row_stride, y);
    A.rows = A.x_rows = (int)rows;
    return launch(ctx, A, (hipStream_t)stream);
}

extern "C" int dq_w4_forward_grouped(dq_w4_ctx* ctx, int64_t rows, const int32_t* offsets, int64_t x_rows,
                                     const void* x, int64_t x_row_stride, const int32_t* row_index, void* y,
                                     void* stream) {
    if (!ctx) DQ_FAIL(DQ_ERR_STATE, "no context");
    if (rows < 0 || rows > ctx->max_rows) DQ_FAIL(DQ_ERR_ARG, "rows must lie in [0, %lld]", (long long)ctx->max_rows);
    if (rows == 0) return DQ_OK;
    if (!offsets) DQ_FAIL(DQ_ERR_ARG, "offsets must not be NULL");
    if (x_rows < 1 || x_rows > INT32_MAX || (!row_index && x_rows < rows))
        DQ_FAIL(DQ_ERR_ARG, "x_rows must be >= 1, and cover the rows where there is no row_index");
    if ((uintptr_t)offsets % 4 || (uintptr_t)row_index % 4)
        DQ_FAIL(DQ_ERR_ARG, "a tensor is not aligned to its elements");
    if (int rc = check_forward(ctx, x, x_row_stride, y)) return rc;
    W4Args A = forward_args(ctx, x, x_row_stride, y);
    A.rows = (int)rows;
    A.x_rows = (int)x_rows;
    A.offsets = offsets;
    A.row_index = row_index;
    return launch(ctx, A, (hipStream_t)stream);
}

extern "C" const char* dq_w4_info(const dq_w4_ctx* ctx) { return ctx ? ctx->info : nullptr; }

extern "C" void dq_w4_release(dq_w4_ctx* ctx) {
    if (!ctx) return;
    (void)hipFree(ctx->codes);
    (void)hipFree(ctx->scales);
    (void)hipFree(ctx->zeros);
    (void)hipFree(ctx->bias);
    (void)hipFree(ctx->sums);
    (void)hipFree(ctx->copy);
    delete ctx;
}
