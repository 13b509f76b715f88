// w4_any.h -- the kernel of products with 4-bit weights for few rows that
// w4_rows.h cannot take: rows that do not start 16 bytes apart, a K that
// does not end there, offsets beyond 31 bits. The same arithmetic, with x read
// from 64-bit addresses of any alignment, and the end of a row element by
// element. 16 rows of 4100 by 4096 columns in bf16: 11.5 us, of 4104 by the other
// kernel 7.4.
#pragma once

#include "w4_device.h"

namespace dq {

constexpr int kW4AnyWaves = 8;

template <int T, int RT, int CT, int S>
__global__ void __launch_bounds__(kW4AnyWaves * 64) k_w4_any(W4Args A) {
    using O = W4Op<T>;
    constexpr int P = O::P, TM = RT * 16;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int c = lane & 15, quad = lane >> 4;
    const int group = blockIdx.x % A.col_groups;
    const W4Tile tile = w4_tile(A, blockIdx.x / A.col_groups, TM, 0, A.rows);
    if (tile.first >= tile.end) return;
    const int t0 = group * CT;

    // this lane's rows of x; those past the tile's end repeat the last one
    // (their results are not stored)
    const char* row[RT];
    bool bad[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        int i = min(tile.first + r * 16 + c, tile.end - 1);
        if (A.row_index) i = A.row_index[i];
        bad[r] = i < 0 || i >= A.x_rows;
        row[r] = static_cast<const char*>(A.x) + (bad[r] ? 0 : i * A.x_stride * O::elem);
    }
    const size_t base = (size_t)tile.expert * A.tiles + t0;
    f4 acc[CT][RT] = {};
    const u4 ones = {O::kOnes, O::kOnes, O::kOnes, O::kOnes};
    for (int b = wave; b < A.blocks; b += waves) {
        u4 code[CT];
#pragma unroll
        for (int j = 0; j < CT; ++j)
            code[j] = reinterpret_cast<const u4*>(A.codes)[((base + j) * A.blocks + b) * 64 + lane];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            f4 sum[CT][RT] = {}, xs[RT] = {};
#pragma unroll
            for (int q = s * (4 / S); q < (s + 1) * (4 / S); ++q) {
                u4 w[CT];
#pragma unroll
                for (int j = 0; j < CT; ++j) w[j] = O::codes(code[j][q]);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    u4 x[P];
                    w4_load8<T>(row[r], b * kW4Block + q * 32 + quad * 8, A.K, A.vec, x);
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        xs[r] = O::mfma(x[p], ones, xs[r]);
#pragma unroll
                        for (int j = 0; j < CT; ++j) sum[j][r] = O::mfma(x[p], w[j], sum[j][r]);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const size_t i = (((base + j) * A.blocks + b) * 16 + c) * S + s;
                const float sc = w4_scale(A.scales, i, A.scale_type);
                const float z = A.zeros ? (float)A.zeros[i] : 8.0f;
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        acc[j][r][v] = __builtin_fmaf(sc, __builtin_fmaf(-z, xs[r][v], sum[j][r][v]), acc[j][r][v]);
            }
        }
    }
    f4* part = reinterpret_cast<f4*>(lds);
    __shared__ int s_bad[TM];
#pragma unroll
    for (int j = 0; j < CT; ++j)
#pragma unroll
        for (int r = 0; r < RT; ++r) part[(wave * (CT * RT) + j * RT + r) * 64 + lane] = acc[j][r];
    if (wave == 0 && quad == 0)
#pragma unroll
        for (int r = 0; r < RT; ++r) s_bad[r * 16 + c] = bad[r];
    __syncthreads();

    // the waves' sums in their order, then bias, gate and the store: a thread
    // takes 4 rows of a column
    const int outs = A.gated ? CT / 2 : CT;
    auto total = [&](int j, int r, int l) {
        f4 v = part[(j * RT + r) * 64 + l];
        for (int w = 1; w < waves; ++w) {
            const f4 u = part[(w * (CT * RT) + j * RT + r) * 64 + l];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += u[i];
        }
        if (A.bias) {
            const float bias = A.bias[(base + j) * 16 + (l & 15)];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += bias;
        }
        return v;
    };
    for (int o = threadIdx.x; o < outs * RT * 64; o += blockDim.x) {
        const int l = o & 63, r = (o >> 6) % RT, j = (o >> 6) / RT;
        f4 v;
        if (A.gated) {
            v = total(2 * j, r, l);
            const f4 u = total(2 * j + 1, r, l);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = w4_silu(v[i]) * u[i];
        } else {
            v = total(j, r, l);
        }
        const int n = ((A.gated ? t0 / 2 : t0) + j) * 16 + (l & 15);
        if (n >= A.N) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = r * 16 + (l >> 4) * 4 + i;
            if (tile.first + m < tile.end)
                w4_store(A.y, (size_t)(tile.first + m) * A.N + n, s_bad[m] ? __builtin_nanf("") : v[i], A.y_type);
        }
    }
}

// the instances for one type of x: 16 rows a workgroup, or 64
template <int T, int RT, int CT>
W4RowsKernel w4_any_pick(int S) {
    return S == 4 ? k_w4_any<T, RT, CT, 4> : S == 2 ? k_w4_any<T, RT, CT, 2> : k_w4_any<T, RT, CT, 1>;
}
template <int T>
W4RowsKernel w4_any_pick(int rows, int col_tiles, int S) {
    if (col_tiles == 2) return rows == 64 ? w4_any_pick<T, 4, 2>(S) : w4_any_pick<T, 1, 2>(S);
    return rows == 64 ? w4_any_pick<T, 4, 1>(S) : w4_any_pick<T, 1, 1>(S);
}

}  // namespace dq
