// w4_rows.h -- the kernel of products with 4-bit weights for few rows.
//
// Bound by the bytes of the codes, each read once for a row tile. A workgroup
// takes CT tiles of 16 columns and RT tiles of 16 rows; its W waves take every
// W-th block of 128 of K, so together they read one stream, and their partial
// sums meet in LDS in a fixed order.
//
// The operands: A = 16 rows of x, B = 16 columns' codes. x comes through LDS:
// straight from the caches the operand takes 16 bytes of 16 rows from
// neighbouring lanes, and each is an access of its own (64 cycles a load, 48
// rows of 16384 x 4096: 13.5 us per 4096 of K, 5.6 of them the codes'). Up to 4
// rows are put there whole before the loop. Of more, each wave keeps a ring of
// two half blocks of 64 k for itself, filled by loads of whole lines straight to
// LDS. A row past the tile's end and a k past K are offsets out of the buffer's
// range: such a load gives zeros and moves nothing, without a branch, so the
// waits are exact. Loads return in the order of their issue: codes are asked
// for a block (or more) ahead, behind the x that is needed before them.
// The sum of a group's x, which its zero point multiplies, is one more
// product, with ones: in the accumulators' layout without any exchange, on
// matrix cores that are idle most of the time here.
//
// One row of 16384 x 8192 in groups of 32 with zero points, fp16 (77.6 MB):
// 17.5 to 18.6 us, 4.2 to 4.4 TB/s. A launch that does nothing but find its tile, ask for the
// first blocks and store takes 3.4 to 5.5 us; the rest runs at 5.5 TB/s and
// more. 48 gated rows of 16384 x 4096 (35.8 MB): 14.7 to 15.5 us, of which the
// products of a wave of 48 x 64 are 3.2 and the vector operations about as much.
#pragma once

#include "w4_device.h"

namespace dq {

constexpr uint32_t kW4Far = 0x80000000u;  // the buffer's size: an offset from here on reads as zeros

// The most waves of a workgroup: by their registers, and by their rings.
template <int T, int RT, int CT, int V>
constexpr int w4_rows_waves() {
    return V == 1 && CT <= 2 ? 16 : V == 4 && T == DQ_F32 && RT >= 3 ? 4 : 8;
}

// V: rows of y that a lane holds of a tile. The four lanes with the same column hold
// 4 V rows: 16, or 4 where there are no more (row m of x then lies in the operand's
// row 4 m, so that a lane's first value is all that it scales and adds).
// ST: the scales' type.
template <int T, int RT, int CT, int S, int ST, int V>
__global__ void __launch_bounds__((w4_rows_waves<T, RT, CT, V>() * 64)) k_w4_rows(W4Args A) {
    using O = W4Op<T>;
    constexpr int P = O::P, TM = RT * 4 * V, SB = ST == DQ_F32 ? 4 : 2;
    constexpr bool WHOLE = V == 1;  // the rows of x lie in LDS whole
    static_assert(!WHOLE || RT == 1, "one tile of rows");
    typedef float fv __attribute__((ext_vector_type(V)));
    // a ring's half blocks in arrays of their own: a read of one is then known not to
    // depend on a load to the other
    constexpr int kHalfRow = 64 * O::elem, kHalf = TM * kHalfRow;
    constexpr int kRing = WHOLE ? 16 : w4_rows_waves<T, RT, CT, V>() * kHalf;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    __shared__ __attribute__((aligned(16))) char ring0[kRing];
    __shared__ __attribute__((aligned(16))) char ring1[kRing];
    __shared__ int s_bad[TM];
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, quad = lane >> 4;
    const int group = blockIdx.x % A.col_groups;
    const W4Tile tile = w4_tile(A, blockIdx.x / A.col_groups, TM, 0, A.rows);
    if (tile.first >= tile.end) return;
    const int t0 = group * CT;

    const size_t base = (size_t)tile.expert * A.tiles + t0;
    const char* codes = reinterpret_cast<const char*>(A.codes) + base * A.blocks * 1024;
    const char* scales = static_cast<const char*>(A.scales) + base * A.blocks * (16 * S * SB);
    // without zero points a buffer of no size, whose zeros become 8
    __amdgpu_buffer_rsrc_t zbuf = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(A.zeros) + (A.zeros ? base * A.blocks * (16 * S) : 0), 0, A.zeros ? (int)kW4Far : 0, 0x00027000);
    const uint32_t z_default = A.zeros ? 0u : 0x08080808u;
    const uint32_t code_at = lane * 16, scale_at = c * (S * SB);

    struct Block {
        u4 code[CT];
        uint32_t scale[CT][(S * SB + 3) / 4];
        uint32_t zero[CT];
    };
    const int last = A.blocks - 1;
    // past the end the last block again: in bounds, not used
    auto fetch = [&](Block& k, int at) {
        const int b = min(at, last);
#pragma unroll
        for (int j = 0; j < CT; ++j)
            k.code[j] = *reinterpret_cast<const u4*>(codes + ((size_t)j * A.blocks + b) * 1024 + code_at);
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            w4_words<S * SB>(scales + ((size_t)j * A.blocks + b) * (16 * S * SB) + scale_at, k.scale[j]);
            // all of the offset in the lane's part, which is what the buffer's size is held against
            const int z = (j * A.blocks + b) * (16 * S) + c * S;
            if constexpr (S == 4) k.zero[j] = __builtin_amdgcn_raw_buffer_load_b32(zbuf, z, 0, 0);
            else if constexpr (S == 2) k.zero[j] = __builtin_amdgcn_raw_buffer_load_b16(zbuf, z, 0, 0);
            else k.zero[j] = __builtin_amdgcn_raw_buffer_load_b8(zbuf, z, 0, 0);
        }
    };
    // The blocks in registers: one is multiplied, the others are on their way.
    constexpr int NB = !WHOLE ? 2 : CT == 4 ? 3 : 4;
    Block block[NB];
    fetch(block[0], wave);

    // x, as offsets in bytes from the tile's first row (with an index from x's)
    const long long row0 = A.row_index ? 0 : tile.first;
    __amdgpu_buffer_rsrc_t xbuf = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(static_cast<const char*>(A.x) + row0 * A.x_stride * O::elem), 0, (int)kW4Far, 0x00027000);
    const int x_rows = min(tile.end - tile.first, TM);
    auto row_at = [&](int m) -> uint32_t {
        int src = tile.first + min(m, x_rows - 1);
        if (A.row_index) src = A.row_index[src];
        const bool bad = A.row_index && (src < 0 || src >= A.x_rows);
        return m >= x_rows || bad ? kW4Far : (uint32_t)((src - (int)row0) * A.x_stride * O::elem);
    };
    for (int m = threadIdx.x; m < x_rows; m += blockDim.x) s_bad[m] = row_at(m) == kW4Far;
    auto pieces = [](const u4* x, u4* p) {
        if constexpr (T == DQ_F32) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(x[i / 4][i % 4]);
            split3(v, &p[0], &p[1], &p[2]);
        } else {
            p[0] = x[0];
        }
    };
    // whole rows: [P][rows][K padded, and 64 bytes], so that the rows of an operand begin in
    // different banks; a lane without a row reads another's (not stored)
    const int x_stride = A.blocks * (kW4Block * 2) + 64;
    const int x_at = min(c >> 2, x_rows - 1) * x_stride + quad * 16;
    // rings: a load takes 1024 bytes of half rows, lane by lane; piece i of 16 bytes of
    // row m lies at i ^ (m / 2 % 8) (rows of 256 bytes: i ^ (m % 16)), so that 16 rows'
    // pieces lie in different banks
    constexpr int kLanes = kHalfRow / 16, kLoads = WHOLE ? 1 : kHalf / 1024;
    constexpr int kSwizzle = O::elem == 2 ? 1 : 0;
    uint32_t x_row[kLoads];
    int x_k[kLoads];  // of the half block's 64, this lane's first
    if constexpr (!WHOLE)
#pragma unroll
        for (int d = 0; d < kLoads; ++d) {
            const int m = d * (64 / kLanes) + lane / kLanes;
            const int piece = lane % kLanes ^ (m >> kSwizzle) % kLanes;
            x_row[d] = row_at(m) + piece * 16;
            x_k[d] = piece * (16 / O::elem);
        }
    issue_fence();
    char* const half0 = ring0 + wave * kHalf;
    char* const half1 = ring1 + wave * kHalf;
    auto fetch_x = [&](int at, int h) {
        const int k0 = min(at, last) * kW4Block + h * 64;
#pragma unroll
        for (int d = 0; d < kLoads; ++d)
            buffer16_to_lds(xbuf, (h ? half1 : half0) + d * 1024, x_k[d] < A.K - k0 ? x_row[d] : kW4Far, k0 * O::elem);
    };
    if constexpr (WHOLE) {
        const uint32_t items = (uint32_t)x_rows * A.per_row.d;  // of 8 elements
        for (uint32_t i = threadIdx.x; i < items; i += blockDim.x) {
            const uint32_t m = fdiv(i, A.per_row), k = (i - m * A.per_row.d) * 8;
            const uint32_t at = (int)k >= A.K ? kW4Far : row_at((int)m) + k * O::elem;
            u4 x[O::elem / 2], p[P];
#pragma unroll
            for (int h = 0; h < O::elem / 2; ++h)
                x[h] = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(xbuf, (int)at, h * 16, 0));
            pieces(x, p);
#pragma unroll
            for (int j = 0; j < P; ++j) *reinterpret_cast<u4*>(lds + (j * x_rows + (int)m) * x_stride + k * 2) = p[j];
        }
    } else {
        fetch_x(wave, 0);
        fetch_x(wave, 1);
    }
    issue_fence();
#pragma unroll
    for (int d = 1; d < NB; ++d) fetch(block[d], wave + d * waves);
    issue_fence();
    if constexpr (WHOLE) __syncthreads();

    fv acc[CT][RT] = {};
    const u4 ones = {O::kOnes, O::kOnes, O::kOnes, O::kOnes};
    auto multiply = [&](Block& now, int b) {
        f4 sum[CT][RT], xs[RT];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            // this half of x has come when no more are on their way than the loads behind
            // it: the other half's, and the next block's codes and scales
            if constexpr (!WHOLE)
                if (q % 2 == 0) {
                    wait_vmcnt<kLoads + 2 * CT>();
                    issue_fence();
                }
            __builtin_amdgcn_sched_barrier(0);  // one step's operands in registers at a time
            if (q % (4 / S) == 0)
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    xs[r] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < CT; ++j) sum[j][r] = f4{0.0f, 0.0f, 0.0f, 0.0f};
                }
            u4 w[CT];
#pragma unroll
            for (int j = 0; j < CT; ++j) w[j] = O::codes(now.code[j][q]);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                u4 p[P];
                if constexpr (WHOLE) {
#pragma unroll
                    for (int i = 0; i < P; ++i)
                        p[i] = *reinterpret_cast<const u4*>(lds + i * x_rows * x_stride + x_at + (b * kW4Block + q * 32) * 2);
                } else {
                    u4 x[O::elem / 2];
                    const int first = (q % 2) * (kLanes / 2) + quad * (O::elem / 2);
#pragma unroll
                    for (int h = 0; h < O::elem / 2; ++h)
                        x[h] = *reinterpret_cast<const u4*>((q < 2 ? half0 : half1) + (r * 16 + c) * kHalfRow +
                                                            (((first + h) ^ (c >> kSwizzle) % kLanes) * 16));
                    pieces(x, p);
                }
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    xs[r] = O::mfma(p[i], ones, xs[r]);
#pragma unroll
                    for (int j = 0; j < CT; ++j) sum[j][r] = O::mfma(p[i], w[j], sum[j][r]);
                }
            }
            if ((q + 1) % (4 / S) == 0) {
                constexpr int per = 4 / S;
                const int g = q / per;
#pragma unroll
                for (int j = 0; j < CT; ++j) {
                    const float sc = w4_scale_word<ST>(now.scale[j], g);
                    const float z = (float)((now.zero[j] | z_default) >> (8 * g) & 255u);
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            float u = __builtin_fmaf(sc, __builtin_fmaf(-z, xs[r][v], sum[j][r][v]), acc[j][r][v]);
                            // due here: the compiler would add in the next step, and keep the sums until then
                            asm volatile("" : "+v"(u));
                            acc[j][r][v] = u;
                        }
                }
            }
            // the half that has been read is filled with the wave's next block's
            if constexpr (!WHOLE)
                if (q % 2 == 1) {
                    wave_lds_fence();
                    fetch_x(b + waves, q / 2);
                    issue_fence();
                }
        }
        fetch(now, b + NB * waves);
        issue_fence();
    };
    // left at once behind the last block: a way round the others back to the loop's
    // head would cost every turn the waits of the shortest one
    if (wave < A.blocks)
        for (int b = wave;;) {
#pragma unroll
            for (int d = 0; d < NB; ++d) {
                multiply(block[d], b);
                b += waves;
                if (b >= A.blocks) goto multiplied;
            }
        }
multiplied:
    if constexpr (!WHOLE) wait_vmcnt<0>();  // nothing is on its way to LDS any more
    __syncthreads();                        // and nobody reads x
    char* const parts_at = WHOLE ? lds : ring0;
    constexpr int kParts = WHOLE ? 64 << 10 : kRing;  // bytes there
    fv* part = reinterpret_cast<fv*>(parts_at);
    auto put = [&](int w) {
#pragma unroll
        for (int j = 0; j < CT; ++j)
#pragma unroll
            for (int r = 0; r < RT; ++r) part[(w * (CT * RT) + j * RT + r) * 64 + lane] = acc[j][r];
    };
    // more parts than fit: the upper half of the waves first hand theirs to the lower half
    static_assert(WHOLE || w4_rows_waves<T, RT, CT, V>() / 2 * CT * RT * 256 * V <= kRing, "half of the parts fit");
    int parts = waves;
    if (waves * CT * RT * (256 * V) > kParts) {
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
