// w4_rows.h -- the kernel of products with 4-bit weights for few rows.
//
// Bound by the bytes of the codes, each read once for a row tile. A workgroup
// takes CT tiles of 16 columns and RT tiles of 16 rows; its W waves take every
// W-th block of 128 of K, so together they read one stream, and their partial
// sums meet in LDS in a fixed order.
//
// The operands: A = 16 rows of x, B = 16 columns' codes. A row past the tile's
// end and a k past K are offsets out of the buffer's range: such a load returns
// zeros and moves nothing, without a branch, so the waits are exact. Loads
// return in the order of their issue, codes from the memory, x from the caches:
// a wait for x is one for every code that was asked for before it. So up to 4
// rows of x go to LDS first, and codes are on their way two or three blocks
// ahead (16 rows of 1400 in LDS: no faster, they fill it); of more rows, x comes from the caches a block ahead, a
// pair of steps of 32 at a time (the two halves of a cache line), and codes
// with it. The sum of a group's x, which its zero point multiplies, is one
// more product, with ones: in the accumulators' layout without any exchange,
// on matrix cores that are idle most of the time here.
#pragma once

#include "w4_device.h"

namespace dq {

constexpr uint32_t kW4Far = 0x80000000u;  // the buffer's size: an offset from here on reads as zeros

// Eight elements of x for one lane, as they lie in memory.
template <int T>
struct W4X {
    u4 v[W4Op<T>::elem / 2];
};

// V: rows of y that a lane holds of a tile. The four lanes with the same column hold
// 4 V rows: 16, or 4 where there are no more (row m of x then lies in the operand's
// row 4 m, so that a lane's first value is all that it scales and adds).
// ST: the scales' type.
template <int T, int RT, int CT, int S, int ST, int V>
__global__ void __launch_bounds__(RT * CT >= 3 ? 512 : 1024) k_w4_rows(W4Args A) {
    using O = W4Op<T>;
    constexpr int P = O::P, TM = RT * 4 * V, SB = ST == DQ_F32 ? 4 : 2;
    constexpr bool XL = V == 1;  // x through LDS
    static_assert(!XL || RT == 1, "one tile of rows in LDS");
    typedef float fv __attribute__((ext_vector_type(V)));
    extern __shared__ __attribute__((aligned(16))) char lds[];
    __shared__ int s_bad[TM];
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, quad = lane >> 4;
    const int group = blockIdx.x % A.col_groups;
    const W4Tile tile = w4_tile(A, blockIdx.x / A.col_groups, TM, 0, A.rows);
    if (tile.first >= tile.end) return;
    const int t0 = group * CT;

    // this lane's rows of x, as offsets in bytes from the first one's (with an index
    // from x's)
    const long long row0 = A.row_index ? 0 : tile.first;
    __amdgpu_buffer_rsrc_t xbuf = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(static_cast<const char*>(A.x) + row0 * A.x_stride * O::elem), 0, (int)kW4Far, 0x00027000);
    uint32_t row[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int m = V == 4 ? r * 16 + c : c >> 2, i = tile.first + m;
        const bool one = V == 4 || (c & 3) == 0;  // a lane that holds a row
        int src = min(i, tile.end - 1);
        if (A.row_index) src = A.row_index[src];
        const bool bad = A.row_index && (src < 0 || src >= A.x_rows);
        row[r] = i >= tile.end || bad || !one ? kW4Far : (uint32_t)((src - (int)row0) * A.x_stride * O::elem);
        if (wave == 0 && quad == 0 && one) s_bad[m] = bad;
    }

    const size_t base = (size_t)tile.expert * A.tiles + t0;
    const u4* codes = reinterpret_cast<const u4*>(A.codes) + base * A.blocks * 64 + lane;
    const char* scales = static_cast<const char*>(A.scales) + (base * A.blocks * 16 + c) * (S * SB);
    const uint8_t* zeros = A.zeros + (base * A.blocks * 16 + c) * S;

    struct Block {
        u4 code[CT];
        uint32_t scale[CT][(S * SB + 3) / 4];
        uint32_t zero[CT];
    };
    auto fetch = [&](Block& k, int b) {
#pragma unroll
        for (int j = 0; j < CT; ++j) k.code[j] = codes[((size_t)j * A.blocks + b) * 64];
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const size_t at = ((size_t)j * A.blocks + b) * 16;
            w4_words<S * SB>(scales + at * (S * SB), k.scale[j]);
            if (A.zeros) {
                const uint8_t* z = zeros + at * S;
                if constexpr (S == 4) k.zero[j] = *reinterpret_cast<const uint32_t*>(z);
                else if constexpr (S == 2) k.zero[j] = *reinterpret_cast<const uint16_t*>(z);
                else k.zero[j] = *z;
            } else {
                k.zero[j] = 0x08080808u;
            }
        }
    };
    // x in LDS: [P][rows][K padded, and 64 bytes], so that the rows of an operand begin in
    // different banks; a lane without a row reads another's (not stored)
    const int x_stride = A.blocks * (kW4Block * 2) + 64, x_rows = min(tile.end - tile.first, TM);
    const int x_at = min(V == 4 ? c : c >> 2, x_rows - 1) * x_stride + quad * 16;
    auto read_x = [&](u4* x, int b, int q) {
#pragma unroll
        for (int i = 0; i < P; ++i)
            x[i] = *reinterpret_cast<const u4*>(lds + i * x_rows * x_stride + x_at + (b * kW4Block + q * 32) * 2);
    };
    auto fetch_x = [&](W4X<T>* x, int b, int q) {
        const int k = b * kW4Block + q * 32 + quad * 8;
        const uint32_t at = k < A.K ? (uint32_t)k * O::elem : kW4Far;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int h = 0; h < O::elem / 2; ++h)
                x[r].v[h] = __builtin_bit_cast(
                    u4, __builtin_amdgcn_raw_buffer_load_b128(xbuf, (int)(row[r] + at), h * 16, 0));
    };

    auto pieces = [](const W4X<T>& x, u4* p) {
        if constexpr (T == DQ_F32) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(x.v[i / 4][i % 4]);
            split3(v, &p[0], &p[1], &p[2]);
        } else {
            p[0] = x.v[0];
        }
    };
    fv acc[CT][RT] = {};
    const u4 ones = {O::kOnes, O::kOnes, O::kOnes, O::kOnes};
    // Blocks ahead of the codes; steps ahead of x (in LDS it is one step away). Past the
    // end the last block again: in bounds, not used.
    constexpr int D = !XL ? 1 : CT == 4 ? 2 : 3;
    constexpr int XR = XL ? 2 : RT * CT * O::elem <= 24 ? 4 : 2;
    const int last = A.blocks - 1;
    Block ahead[D];
    W4X<T> x_ring[XL ? 1 : XR][RT];
    u4 x_lds[2][P];
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(ahead[d], min(wave + d * waves, last));
    if constexpr (XL) {
        const uint32_t items = (uint32_t)x_rows * A.per_row.d;  // of 8 elements
        for (uint32_t i = threadIdx.x; i < items; i += blockDim.x) {
            const uint32_t m = fdiv(i, A.per_row), k = (i - m * A.per_row.d) * 8;
            int src = tile.first + (int)m;
            if (A.row_index) src = A.row_index[src];
            const bool bad = A.row_index && (src < 0 || src >= A.x_rows);
            const uint32_t at = bad || (int)k >= A.K ? kW4Far : (uint32_t)((src - (int)row0) * A.x_stride + k) * O::elem;
            W4X<T> x;
#pragma unroll
            for (int h = 0; h < O::elem / 2; ++h)
                x.v[h] = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(xbuf, (int)at, h * 16, 0));
            u4 p[P];
            pieces(x, p);
#pragma unroll
            for (int j = 0; j < P; ++j) *reinterpret_cast<u4*>(lds + (j * x_rows + (int)m) * x_stride + k * 2) = p[j];
        }
        __syncthreads();
        read_x(x_lds[0], min(wave, last), 0);
    } else {
#pragma unroll
        for (int q = 0; q < XR; ++q) fetch_x(x_ring[q], min(wave, last), q);
    }
    for (int b = wave; b < A.blocks; b += waves) {
        const Block now = ahead[0];
        const int nb = min(b + waves, last);
#pragma unroll
        for (int d = 0; d + 1 < D; ++d) ahead[d] = ahead[d + 1];
        fetch(ahead[D - 1], min(b + D * waves, last));
        f4 sum[CT][RT], xs[RT];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            __builtin_amdgcn_sched_barrier(0);  // one step's operands in registers at a time
            if (q % (4 / S) == 0) {
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    xs[r] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < CT; ++j) sum[j][r] = f4{0.0f, 0.0f, 0.0f, 0.0f};
                }
            }
            u4 w[CT];
#pragma unroll
            for (int j = 0; j < CT; ++j) w[j] = O::codes(now.code[j][q]);
            if constexpr (XL) read_x(x_lds[(q + 1) & 1], q < 3 ? b : nb, (q + 1) & 3);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                u4 p[P];
                if constexpr (XL) {
#pragma unroll
                    for (int i = 0; i < P; ++i) p[i] = x_lds[q & 1][i];
                } else {
                    pieces(x_ring[q % XR][r], p);
                }
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    xs[r] = O::mfma(p[i], ones, xs[r]);
#pragma unroll
                    for (int j = 0; j < CT; ++j) sum[j][r] = O::mfma(p[i], w[j], sum[j][r]);
                }
            }
            if constexpr (!XL)
                if (q & 1) {
                    fetch_x(x_ring[(q - 1) % XR], q - 1 + XR < 4 ? b : nb, (q - 1 + XR) & 3);
                    fetch_x(x_ring[q % XR], q + XR < 4 ? b : nb, (q + XR) & 3);
                }
            if ((q + 1) % (4 / S) == 0) {
                constexpr int per = 4 / S;
                const int g = q / per;
#pragma unroll
                for (int j = 0; j < CT; ++j) {
                    const float sc = w4_scale_word<ST>(now.scale[j], g);
                    const float z = (float)(now.zero[j] >> (8 * g) & 255u);
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            acc[j][r][v] = __builtin_fmaf(sc, __builtin_fmaf(-z, xs[r][v], sum[j][r][v]), acc[j][r][v]);
                }
            }
        }
    }

    if constexpr (XL) __syncthreads();  // nobody reads x any more
    fv* part = reinterpret_cast<fv*>(lds);
    auto put = [&](int w) {
#pragma unroll
        for (int j = 0; j < CT; ++j)
#pragma unroll
            for (int r = 0; r < RT; ++r) part[(w * (CT * RT) + j * RT + r) * 64 + lane] = acc[j][r];
    };
    // more than 64 KiB of parts: the upper half of the waves first hand theirs
    // to the lower half
    int parts = waves;
    if (waves * CT * RT > 64) {
        parts = waves / 2;
        if (wave >= parts) put(wave - parts);
        __syncthreads();
        if (wave < parts)
#pragma unroll
            for (int j = 0; j < CT; ++j)
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const fv u = part[(wave * (CT * RT) + j * RT + r) * 64 + lane];
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[j][r][v] += u[v];
                }
    }
    if (wave < parts) put(wave);
    __syncthreads();

    // the waves' sums in their order, then bias, gate and the store: a thread
    // takes V rows of a column
    const int outs = A.gated ? CT / 2 : CT;
    auto total = [&](int j, int r, int l) {
        fv v = part[(j * RT + r) * 64 + l];
        for (int w = 1; w < parts; ++w) {
            const fv u = part[(w * (CT * RT) + j * RT + r) * 64 + l];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] += u[i];
        }
        if (A.bias) {
            const float bias = A.bias[(base + j) * 16 + (l & 15)];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] += bias;
        }
        return v;
    };
    for (int o = threadIdx.x; o < outs * RT * 64; o += blockDim.x) {
        const int l = o & 63, r = (o >> 6) % RT, j = (o >> 6) / RT;
        const int n = ((A.gated ? t0 / 2 : t0) + j) * 16 + (l & 15), m0 = r * 4 * V + (l >> 4) * V;
        if (n >= A.N || tile.first + m0 >= tile.end) continue;
        fv v;
        if (A.gated) {
            v = total(2 * j, r, l);
            const fv u = total(2 * j + 1, r, l);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = w4_silu(v[i]) * u[i];
        } else {
            v = total(j, r, l);
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (tile.first + m0 + i < tile.end)
                w4_store(A.y, (size_t)(tile.first + m0 + i) * A.N + n, s_bad[m0 + i] ? __builtin_nanf("") : v[i], A.y_type);
    }
}

// the instances for one type of x; NULL where there is none
template <int T, int RT, int CT, int V, int S>
W4RowsKernel w4_rows_pick(int scales) {
    return scales == DQ_F32    ? k_w4_rows<T, RT, CT, S, DQ_F32, V>
           : scales == DQ_BF16 ? k_w4_rows<T, RT, CT, S, DQ_BF16, V>
                               : k_w4_rows<T, RT, CT, S, DQ_F16, V>;
}
template <int T, int RT, int CT, int V>
W4RowsKernel w4_rows_pick(int S, int scales) {
    return S == 4   ? w4_rows_pick<T, RT, CT, V, 4>(scales)
           : S == 2 ? w4_rows_pick<T, RT, CT, V, 2>(scales)
                    : w4_rows_pick<T, RT, CT, V, 1>(scales);
}
template <int T, int RT, int V>
W4RowsKernel w4_rows_pick(int col_tiles, int S, int scales) {
    if constexpr (V == 1)
        if (col_tiles == 1) return w4_rows_pick<T, RT, 1, V>(S, scales);
    return col_tiles == 4   ? w4_rows_pick<T, RT, 4, V>(S, scales)
           : col_tiles == 2 ? w4_rows_pick<T, RT, 2, V>(S, scales)
                            : nullptr;
}
template <int T>
W4RowsKernel w4_rows_pick(int rows, int col_tiles, int S, int scales) {
    return rows == 4    ? w4_rows_pick<T, 1, 1>(col_tiles, S, scales)
           : rows == 16 ? w4_rows_pick<T, 1, 4>(col_tiles, S, scales)
           : rows == 32 ? w4_rows_pick<T, 2, 4>(col_tiles, S, scales)
           : rows == 48 ? w4_rows_pick<T, 3, 4>(col_tiles, S, scales)
           : rows == 64 ? w4_rows_pick<T, 4, 4>(col_tiles, S, scales)
                        : nullptr;
}

}  // namespace dq
