// w4_tile.h -- the kernel of products with 4-bit weights for many rows.
//
// Bound by the matrix cores and the vector operations beside them. A workgroup
// of 2 x WN waves computes 128 rows by 64 WN columns of the packed order, a wave
// 64 x 64 of them (4 x 4 blocks of 16 x 16). K advances by a block of 128: the
// rows of x come straight to LDS (two stages, 32 KiB each, the next one on its
// way while this one is multiplied), swizzled so that the 16 rows of an operand
// lie in different banks; the codes come straight to registers, one 1 KiB load
// for 16 columns, and are unpacked there. A stage is 64 products of a wave
// (1024 cycles of its matrix core), 112 vector operations that unpack and 64
// that scale (about 700), so neither waits for the other as long as they are issued
// in turn and nothing is spilled: with 17 registers in scratch memory, whose loads wait
// for every copy before them, 16384 rows of experts took 1168 us, with none 572.
//
// The scale of a group multiplies its sum: sums start anew with every group
// and are added to the result with one fused multiply-add each. (Scaled weights
// rounded to bf16 would need no second set of sums, but their error is as large
// as the output's own rounding.) A group's sum starts at -8 times the group's sum
// of x, which takes the middle of the codes out at no cost (the operand is there
// anyway); the rest of a zero point, z - 8, is one small product over the
// groups at the end, in three bf16 pieces of each side (24 bits). The sums of x
// come from k_w4_prepare, which also makes aligned rows of what is not: K padded
// to whole blocks, fp32 as three bf16 pieces one behind the other.
//
// Copies of x are a fifth of the time (without them 128 x 128 tiles took 135 us
// where it was 163 with them): WN is 4 where there are that many tiles, and 2 below.
// 4096 rows of 4096 x 4096 in bf16: 151 to 163 us by the card, 910 TFLOP/s at best; 16384 rows of 16 gated
// experts of 4096 x 4096: 560 to 608 us, 980; a large product of bf16 matrices by the
// library reaches 1116 (4096^3) to 1255 (8192^3). Wave tiles of 48 x 64, which
// leave 40 registers over, 198 and 645 us.
#pragma once

#include "w4_device.h"

#include <type_traits>

namespace dq {

constexpr int kW4TileM = 4;  // row tiles of 16 of a wave
constexpr int kW4TileRows = 2 * 16 * kW4TileM;

// Rows of x as the tile kernel takes them, and the sums of their groups.
struct W4Prepare {
    const void* x;
    long long x_stride;
    const int32_t* row_index;  // row r is x's row_index[r] (NULL: r)
    int rows, x_rows, K, blocks, S, vec;
    uint16_t* copy;  // [rows][P][blocks * 128] (NULL: sums only)
    float* sums;     // [rows][blocks * S]: -8 times a group's sum
};

// A wave a row; each lane takes 8 elements of a block's 128, four blocks at a time.
template <int T>
__global__ void __launch_bounds__(256) k_w4_prepare(W4Prepare A) {
    using O = W4Op<T>;
    constexpr int P = O::P;
    const int lane = threadIdx.x & 63;
    const int r = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (r >= A.rows) return;
    long long src = A.row_index ? A.row_index[r] : r;
    if (src < 0 || src >= A.x_rows) src = 0;  // its results are NaN in any case
    const char* row = static_cast<const char*>(A.x) + src * A.x_stride * O::elem;
    const int Kp = A.blocks * kW4Block;
    for (int b = lane >> 4; b < A.blocks; b += 4) {
        const int k = b * kW4Block + (lane & 15) * 8;
        u4 x[P];
        w4_load8<T>(row, k, A.K, A.vec, x);
        if (A.copy)
#pragma unroll
            for (int p = 0; p < P; ++p)
                *reinterpret_cast<u4*>(A.copy + ((size_t)r * P + p) * Kp + k) = x[p];
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v = 0.0f;
#pragma unroll
                for (int p = P - 1; p >= 0; --p) v += O::value((x[p][i] >> (16 * h)) & 0xffffu);
                s += v;
            }
        // the 16 lanes of a block hold 16, 8 or 4 lanes of a group
        s += __shfl_xor(s, 1);
        s += __shfl_xor(s, 2);
        if (A.S <= 2) s += __shfl_xor(s, 4);
        if (A.S == 1) s += __shfl_xor(s, 8);
        const int per = 16 / A.S;
        if ((lane & (per - 1)) == 0) A.sums[(size_t)r * A.blocks * A.S + b * A.S + (lane & 15) / per] = -8.0f * s;
    }
}

struct W4TileArgs {
    W4Args a;           // x: rows of P * blocks * 128 elements
    const float* sums;  // by the row of x, or of y from row_lo on where by_row
    int by_row;
    int x_by_row;       // and so are the rows of a.x
    int row_lo, row_hi; // the rows of y that this launch takes
    int tiles_m, tiles_n, gm, gn;  // the most tiles; gm x gn neighbours go to one XCD
    int vec_store;
};

// G: the rows of x are looked up in row_index. ST: the scales' type.
template <int T, int WN, int S, int ST, bool G>
__global__ void __launch_bounds__(2 * WN * 64, 2) k_w4_tile(W4TileArgs A) {
    using O = W4Op<T>;
    constexpr int P = O::P, NW = 2 * WN, CPW = kW4TileRows / 4 / NW;  // waves, copies a wave and stage
    constexpr int SB = ST == DQ_F32 ? 4 : 2, SW = (S * SB + 3) / 4;  // words of a column's scales
    __shared__ __attribute__((aligned(16))) char st0[kW4TileRows * 256];
    __shared__ __attribute__((aligned(16))) char st1[kW4TileRows * 256];
    // with the stages 16 KiB for each wave's results at the end
    constexpr int kMore = NW * 16 * kW4TileM * 256 - 2 * kW4TileRows * 256;
    __shared__ __attribute__((aligned(16))) char st2[kMore > 0 ? kMore : 16];
    __shared__ __attribute__((aligned(16))) float s_sum[2][S][kW4TileRows];
    __shared__ int s_bad[kW4TileRows];
    const W4Args& a = A.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, quad = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;

    // Neighbouring workgroups land on different XCDs (round robin): each XCD
    // takes whole units of gm x gn tiles, which share x and codes in its L2.
    const int per = A.gm * A.gn, xcd = blockIdx.x & 7, j = blockIdx.x >> 3;
    const int unit = (j / per) * 8 + xcd, in = j % per;
    const int units_n = (A.tiles_n + A.gn - 1) / A.gn;
    const int tm = unit / units_n * A.gm + in % A.gm, tn = unit % units_n * A.gn + in / A.gm;
    if (tm >= A.tiles_m || tn >= A.tiles_n) return;
    const W4Tile tile = w4_tile(a, tm, kW4TileRows, A.row_lo, A.row_hi);
    if (tile.first >= tile.end) return;

    // Copies of x: each takes 4 rows of 256 bytes, lane l the 16-byte piece (l %
    // 16) ^ (row % 16) of row l / 16, to LDS in the order of the lanes. Rows past the
    // tile's end repeat its last one (their results are not stored), one that does not
    // exist the first of x (its result is NaN): every copy lies inside x.
    const int last = tile.end - 1;
    uint32_t voff[CPW];
    const int row0 = G ? 0 : tile.first - (A.x_by_row ? A.row_lo : 0);
    const uint32_t x_bytes = (uint32_t)(a.x_stride * 2);
    const int rows_here = tile.end - tile.first;
    __amdgpu_buffer_rsrc_t xbuf = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(static_cast<const char*>(a.x) + (long long)row0 * a.x_stride * 2), 0, -1, 0x00027000);
#pragma unroll
    for (int i = 0; i < CPW; ++i) {
        const int r = (wave * CPW + i) * 4 + quad;
        int src = min(r, rows_here - 1);
        bool bad = false;
        if (a.row_index) {
            const int at = a.row_index[tile.first + src];
            bad = at < 0 || at >= a.x_rows;
            if (G) src = bad ? 0 : at;
        }
        if (c == 0) s_bad[r] = bad;
        voff[i] = (uint32_t)src * x_bytes + (uint32_t)((c ^ (r & 15)) * 16);
    }
    auto copy = [&](int stage_k, char* dst) {
        // stage_k: the element of a row at which the stage's 128 begin
#pragma unroll
        for (int i = 0; i < CPW; ++i)
            buffer16_to_lds(xbuf, dst + (wave * CPW + i) * 1024, voff[i], (uint32_t)stage_k * 2);
    };
    // the sums of x of thread t's row, as an offset (they take less than 2^32 bytes)
    uint32_t sum_at;
    {
        const int r = min(tile.first + (int)threadIdx.x, last);
        int src = r;
        if (A.by_row) src = r - A.row_lo;
        else if (a.row_index) {
            src = a.row_index[r];
            if (src < 0 || src >= a.x_rows) src = 0;
        }
        sum_at = (uint32_t)src * (uint32_t)(a.blocks * S) * 4u;
    }
    const int nt0 = tn * (WN * 4) + wn * 4;  // this wave's column tiles
    const size_t base = (size_t)tile.expert * a.tiles + nt0;
    // uniform addresses, and each lane's part of them
    const char* codes = reinterpret_cast<const char*>(a.codes) + base * a.blocks * 1024;
    const char* scales = static_cast<const char*>(a.scales) + base * a.blocks * (16 * S * SB);
    const uint32_t code_at = lane * 16, scale_at = c * (S * SB);

    f4 acc[kW4TileM][4];
#pragma unroll
    for (int m = 0; m < kW4TileM; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) acc[m][n] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    u4 code[2][4];
    uint32_t sc[2][4][SW];  // a column's scales as they lie in memory
    float sum[S];
    const int nstages = a.blocks * P, Kp = a.blocks * kW4Block;

    auto fetch = [&](int b, u4* w, uint32_t (*s)[SW]) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
            w[n] = *reinterpret_cast<const u4*>(codes + ((size_t)n * a.blocks + b) * 1024 + code_at);
#pragma unroll
        for (int n = 0; n < 4; ++n) w4_words<S * SB>(scales + ((size_t)n * a.blocks + b) * (16 * S * SB) + scale_at, s[n]);
    };
    auto fetch_sums = [&](int b) {
        const char* p = reinterpret_cast<const char*>(A.sums) + b * (S * 4) + sum_at;
#pragma unroll
        for (int g = 0; g < S; ++g) sum[g] = reinterpret_cast<const float*>(p)[g];
    };

    copy(0, st0);
    fetch(0, code[0], sc[0]);
    fetch_sums(0);

    // One stage: 4 steps of 32 k, each 16 products of a wave, column by column: a
    // column's operand is free after its 4, and the next step's is unpacked into it
    // while the next column's run; behind a group's last step its sums are scaled and
    // added likewise. (Named scheduling groups, a raised wave priority and codes
    // fetched half a stage earlier or later made no difference.)
    u4 w[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) w[n] = O::codes(code[0][n][0]);
    auto stage = [&](auto CUR, int i) {
        constexpr int cur = decltype(CUR)::value;
        const char* L = cur ? st1 : st0;
        if ((int)threadIdx.x < kW4TileRows)
#pragma unroll
            for (int g = 0; g < S; ++g) s_sum[cur][g][threadIdx.x] = sum[g];
        wait_vmcnt_lgkm0<0>();
        lds_barrier();
        // past the end the last stage again: in bounds, not used
        const int nx = min(i + 1, nstages - 1), nb = P == 1 ? nx : nx / P;
        copy(nb * kW4Block + (nx - nb * P) * Kp, cur ? st0 : st1);
        const bool first = P == 1 || i % P == 0;
        u4 x[2][kW4TileM];
        auto read_x = [&](u4* to, int q) {
#pragma unroll
            for (int m = 0; m < kW4TileM; ++m) {
                const int r = wm * (16 * kW4TileM) + m * 16 + c;
                to[m] = *reinterpret_cast<const u4*>(L + r * 256 + (((q * 4 + quad) ^ c) * 16));
            }
        };
        read_x(x[0], 0);
        f4 t[kW4TileM][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            constexpr int per = 4 / S;
            const int g = q / per;
            const bool begins = q % per == 0, ends = (q + 1) % per == 0;
            __builtin_amdgcn_sched_barrier(0);
            if (begins)
#pragma unroll
                for (int m = 0; m < kW4TileM; ++m) {
                    f4 t0 = *reinterpret_cast<const f4*>(&s_sum[cur][g][wm * (16 * kW4TileM) + m * 16 + quad * 4]);
                    if (!first) t0 = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int n = 0; n < 4; ++n) t[m][n] = t0;
                }
            if (q < 3) read_x(x[(q + 1) & 1], q + 1);
            if (q == 1) {  // half a stage ahead: registers are scarce before
                fetch(nb, code[cur ^ 1], sc[cur ^ 1]);
                fetch_sums(nb);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
#pragma unroll
                for (int m = 0; m < kW4TileM; ++m) t[m][n] = O::mfma(x[q & 1][m], w[n], t[m][n]);
                // behind the last step the next stage's first
                w[n] = O::codes(q < 3 ? code[cur][n][q + 1] : code[cur ^ 1][n][0]);
                if (ends) {
                    const float s = w4_scale_word<ST>(sc[cur][n], g);
#pragma unroll
                    for (int m = 0; m < kW4TileM; ++m)
#pragma unroll
                        for (int v = 0; v < 4; ++v) acc[m][n][v] = __builtin_fmaf(s, t[m][n][v], acc[m][n][v]);
                }
            }
            // results are due here: left to itself the compiler moves the additions into the
            // next stage, and keeps every group's sums until then
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                asm volatile("" : "+v"(w[n]));
                if (ends)
#pragma unroll
                    for (int m = 0; m < kW4TileM; ++m) asm volatile("" : "+v"(acc[m][n]));
            }
        }
    };
    int i = 0;
    for (; i + 2 <= nstages; i += 2) {
        stage(std::integral_constant<int, 0>{}, i);
        stage(std::integral_constant<int, 1>{}, i + 1);
    }
    if (i < nstages) stage(std::integral_constant<int, 0>{}, i);
    wait_vmcnt_lgkm0<0>();
    lds_barrier();  // nobody reads a stage any more, nothing is on its way to one

    // what is left of the zero points: (z - 8) s of 32 groups at a time against
    // the sums of x, which are there times -8. All is asked for before the first is
    // used
    if (a.zeros) {
        const int groups = a.blocks * S;
        const uint8_t* zeros = a.zeros + base * a.blocks * (16 * S);
        uint32_t x_at[kW4TileM];
#pragma unroll
        for (int m = 0; m < kW4TileM; ++m) {
            const int r = min(tile.first + wm * (16 * kW4TileM) + m * 16 + c, last);
            int src = A.by_row ? r - A.row_lo : r;
            if (!A.by_row && a.row_index) {
                src = a.row_index[r];
                if (src < 0 || src >= a.x_rows) src = 0;
            }
            x_at[m] = (uint32_t)src * (uint32_t)groups;
        }
        for (int g0 = 0; g0 < groups; g0 += 32) {
            uint32_t s_raw[4][8], z_raw[4][8];
            float x_sum[kW4TileM][8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int g = min(g0 + quad * 8 + k, groups - 1);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const uint32_t at = (uint32_t)(((n * a.blocks + g / S) * 16 + c) * S + g % S);
                    if constexpr (SB == 4) s_raw[n][k] = reinterpret_cast<const uint32_t*>(scales)[at];
                    else s_raw[n][k] = reinterpret_cast<const uint16_t*>(scales)[at];
                    z_raw[n][k] = zeros[at];
                }
            }
            // a lane's 8 sums at once: one by one each of a load's lanes is an access of its own
#pragma unroll
            for (int m = 0; m < kW4TileM; ++m) {
                const int g = g0 + quad * 8;
                const float* p = A.sums + x_at[m];
                if (g + 8 <= groups) {
                    __builtin_memcpy(x_sum[m], p + g, 32);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) x_sum[m][k] = p[min(g + k, groups - 1)];
                }
            }
            issue_fence();
            u4 zs[4][3];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = g0 + quad * 8 + k < groups
                               ? w4_scale_word<ST>(&s_raw[n][k], 0) * (((float)z_raw[n][k] - 8.0f) * 0.125f)
                               : 0.0f;
                split3(v, &zs[n][0], &zs[n][1], &zs[n][2]);
            }
#pragma unroll
            for (int m = 0; m < kW4TileM; ++m) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (g0 + quad * 8 + k >= groups) x_sum[m][k] = 0.0f;
                u4 xs[3];
                split3(x_sum[m], &xs[0], &xs[1], &xs[2]);
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int u = 0; u < 3; ++u)
#pragma unroll
                        for (int w = 0; u + w < 3; ++w)
                            acc[m][n] = W4Op<DQ_BF16>::mfma(xs[u], zs[n][w], acc[m][n]);
            }
        }
    }

    // bias and gate, through this wave's part of the stages 
    // so that whole rows go out, 16 bytes a lane
    constexpr int kRows = 16 * kW4TileM, kPart = kRows * 256, kIn = kW4TileRows * 256 / kPart;
    char* part_base = wave < kIn ? st0 + wave * kPart : wave < 2 * kIn ? st1 + (wave - kIn) * kPart : st2 + (wave - 2 * kIn) * kPart;
    float* part = reinterpret_cast<float*>(part_base);
    const int cols = a.gated ? 32 : 64;
    const int n0 = (a.gated ? nt0 / 2 : nt0) * 16;
    if (a.bias)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float bias = a.bias[(base + n) * 16 + c];
#pragma unroll
            for (int m = 0; m < kW4TileM; ++m)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[m][n][v] += bias;
        }
    {
#pragma unroll
        for (int m = 0; m < kW4TileM; ++m)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                f4 v = acc[m][n];
                int col = n * 16;
                if (a.gated) {
                    if (n & 1) continue;
                    const f4 u = acc[m][n | 1];
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = w4_silu(v[k]) * u[k];
                    col = n * 8;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) part[(m * 16 + quad * 4 + k) * 64 + ((col + c) ^ (quad * 16))] = v[k];
            }
        wave_lds_fence();
        const int lanes = cols / 8, rows_at = 64 / lanes;
        for (int r0 = 0; r0 < kRows; r0 += rows_at) {
            const int r = r0 + lane / lanes, col = lane % lanes * 8;
            const int in_tile = wm * kRows + r;
            const float* from = part + r * 64 + (col ^ ((r >> 2 & 3) * 16));
            const f4 lo = *reinterpret_cast<const f4*>(from), hi = *reinterpret_cast<const f4*>(from + 4);
            if (tile.first + in_tile > last) continue;
            float v[8];
            const bool bad = s_bad[in_tile];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = bad ? __builtin_nanf("") : lo[k];
                v[4 + k] = bad ? __builtin_nanf("") : hi[k];
            }
            w4_store8(a.y, (size_t)(tile.first + in_tile) * a.N, n0 + col, a.N, v, a.y_type, A.vec_store);
        }
        wave_lds_fence();
    }
}

// the instances for one type of x
typedef void (*W4TileKernel)(W4TileArgs);
typedef void (*W4PrepareKernel)(W4Prepare);
template <int T, int WN, int S, int ST>
W4TileKernel w4_tile_pick(bool gather) {
    return gather ? k_w4_tile<T, WN, S, ST, true> : k_w4_tile<T, WN, S, ST, false>;
}
template <int T, int WN, int S>
W4TileKernel w4_tile_pick(int scales, bool g) {
    return scales == DQ_F32    ? w4_tile_pick<T, WN, S, DQ_F32>(g)
           : scales == DQ_BF16 ? w4_tile_pick<T, WN, S, DQ_BF16>(g)
                               : w4_tile_pick<T, WN, S, DQ_F16>(g);
}
template <int T, int WN>
W4TileKernel w4_tile_pick(int S, int scales, bool g) {
    return S == 4   ? w4_tile_pick<T, WN, 4>(scales, g)
           : S == 2 ? w4_tile_pick<T, WN, 2>(scales, g)
                    : w4_tile_pick<T, WN, 1>(scales, g);
}
template <int T>
W4TileKernel w4_tile_pick(int WN, int S, int scales, bool gather) {
    return WN == 4 ? w4_tile_pick<T, 4>(S, scales, gather) : w4_tile_pick<T, 2>(S, scales, gather);
}

}  // namespace dq
