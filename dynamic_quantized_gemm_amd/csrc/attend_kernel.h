// attend_kernel.h -- the attention kernel over the paged cache, a template on
// the cache's type; paged_attend_*.hip hold its instances.
//
//   s_t = sm_scale q . k_t     for the tokens t in [max(0, len - window), len)
//   p   = softmax(s),  out = sum_t p_t v_t,  lse = log sum_t exp(s_t)
//
// Bound by the bytes of keys and values, each read once. The units of 128
// tokens of all sequences and head tiles (16 query heads of one key-value
// head) are shared out evenly over as many workgroups as the chip holds at
// once (kv_plan.h), whatever the lengths, which only the device knows. A
// workgroup walks its units; where it holds all of a sequence's units for a
// head tile it writes the output, else a partial result (maximum, sum,
// weighted values) that k_attend_finish combines. Where that is faster, a
// workgroup takes whole heads and gathers their weights itself (`whole`).
// 131071 tokens of 4 heads of 128 in bf16: 44.5 us, 6.0 TB/s; 32 sequences of
// up to 4096, 8 heads of 128: 54 us, 6.0 TB/s, of what a copy reaches 6.2.
//
// A wave takes 32 of a unit's 128 tokens, on its own until its units end:
//   S^T = K Q^T     tokens x heads, A = 16 rows of K as they lie in memory;
//   O^T = V^T P^T   d x heads. The MFMA's layout puts a head's scores of 8
//                   tokens into one lane, which are the 8 that the same lane
//                   has to supply as the operand P^T: the weights never leave
//                   their registers.
// A lane loads E = DP / 16 values of V for its 8 tokens (neighbours; of 192
// eight and four, of 96 four and two), and the A operand for d = E n + i (i < E) is the i-th of
// each: the transposition is within a lane, one byte permutation for two values. Nothing goes through
// LDS but 32 row numbers and scales for each 32 tokens.
//
// Precision. Products are of 16-bit operands, summed in fp32. int8 codes are
// exact in bf16. An fp32 query is the sum of three bf16 or fp16 pieces (all 24
// bits), an fp16 query on a bf16 or int8 cache of two; against an fp16 cache
// other queries are first scaled by a power of two of the row's largest. The
// weights are split in two pieces (2^-18 of a weight, below half a step of
// the output), three for fp32 outputs on bf16 (fp16 weights are scaled by
// 2^15 so that their second piece keeps them to 2^-22). Scores are in units of
// log2 in fp32, where exp is v_exp_f32.
#pragma once

#include "paged_kv.h"

namespace dq {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kHeadTile = 16;  // query heads of a workgroup's item: the MFMA's columns

struct AttendArgs {
    DqAttendArgs a;
    int q_type, Hq, Hk, D, cap, G, tiles;  // tiles: head tiles of a key-value head
    int workers;
    int q_vec;  // queries can be loaded 16 bytes at a time
    int whole;  // a workgroup takes whole items, and there is nothing to finish
    float* s;         // NULL: scores are not kept; else for each key-value head
    size_t s_stride;  // (s_stride apart), runs of 32 tokens: [G][32]
    float* l2;    // [batch * Hq] log2 of the sum of exp
    float* part;  // [workers][2][16][D + 4]: maximum, sum, -, -, weighted values
    int2* parts;  // [batch * Hk * tiles]: the first of the workers that share an
                  // item's units and their number, 0 where the item needs no join
    int32_t* bad;
    KvGeom geom;
};

// A sequence's length, 0 where it is out of range (`bad` then).
__device__ __forceinline__ int attend_len(const AttendArgs& A, int b, bool* bad) {
    const int n = A.a.lens[b];
    *bad = n < 0 || n > A.cap;
    return *bad ? 0 : n;
}

struct AttendScan {
    int64_t sum[4];  // of each wave
    int64_t base;
    int b, len;
};

// All units of the batch, by a workgroup of 256 threads that take runs of
// sequences. The thread whose run has the first unit of worker w leaves that
// unit's sequence, its length and the number of units before it in *sh (the
// caller's barrier makes them seen).
__device__ __forceinline__ KvShare attend_scan(const AttendArgs& A, AttendScan* sh, int w) {
    const int tid = threadIdx.x, lane = tid & 63, run = (A.a.batch + 255) / 256;
    const int items = A.Hk * A.tiles;
    int64_t x = 0;
    int len = 0;
    for (int i = 0; i < run; ++i) {
        const int b = tid * run + i;
        bool bad;
        len = b < A.a.batch ? attend_len(A, b, &bad) : 0;
        x += (int64_t)kv_units(len, A.a.window) * items;
    }
    int64_t y = x;
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t z = __shfl_up(y, o);
        if (lane >= o) y += z;
    }
    if (lane == 63) sh->sum[tid >> 6] = y;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < 4; ++w) {
        if (w < (tid >> 6)) y += sh->sum[w];
        total += sh->sum[w];
    }
    const KvShare share = kv_share(total, A.workers);
    const int64_t u = w < share.workers ? kv_first(w, share) : -1;
    int64_t base = y - x;
    if (u >= base && u < y) {
        int b = tid * run;
        if (run > 1)
            for (;; ++b) {
                bool bad;
                len = attend_len(A, b, &bad);
                const int64_t n = (int64_t)kv_units(len, A.a.window) * items;
                if (u < base + n) break;
                base += n;
            }
        sh->b = b;
        sh->len = len;
        sh->base = base;
    }
    return share;
}

// The scores of a run of 32 tokens (from the window's first on) of a
// key-value head: one piece of memory for all its query heads.
__device__ __forceinline__ size_t attend_score_at(const AttendArgs& A, int item, int run) {
    return (size_t)item * A.s_stride + (size_t)run * (32 * A.G);
}

// A value that is the same in all lanes, kept in scalar registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
    return (int64_t)((uint64_t)(uint32_t)uniform((int)(x >> 32)) << 32 | (uint32_t)uniform((int)x));
}

// max and sum over the four lanes that hold one head (lane & 15)
__device__ __forceinline__ float head_max(float x) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __builtin_fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __builtin_fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float head_sum(float x) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// a byte of a word as a signed value
template <int I>
__device__ __forceinline__ float code_f32(uint32_t w) {
    return (float)((int32_t)(w << (24 - 8 * I)) >> 24);
}
// two fp32 values that are exact in bf16, as two bf16
__device__ __forceinline__ uint32_t exact_bf16x2(float lo, float hi) {
    return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
// four int8 codes as four bf16
__device__ __forceinline__ u2 codes_bf16x4(uint32_t w) {
    const u2 r = {exact_bf16x2(code_f32<0>(w), code_f32<1>(w)), exact_bf16x2(code_f32<2>(w), code_f32<3>(w))};
    return r;
}

// N words that will not be needed again, as many as possible at a time
template <int N>
__device__ __forceinline__ void load_words(const char* p, uint32_t* w) {
    constexpr int M = N >= 4 ? 4 : N >= 2 ? 2 : 1;
    typedef uint32_t V __attribute__((ext_vector_type(M), aligned(4)));
    if constexpr (M == 1) {
        w[0] = __builtin_nontemporal_load((const uint32_t*)p);
    } else {
        const V x = __builtin_nontemporal_load((const V*)p);
#pragma unroll
        for (int i = 0; i < M; ++i) w[i] = x[i];
    }
    if constexpr (N > M) load_words<N - M>(p + 4 * M, w + M);
}

template <int CT> struct AttendOps {  // bf16 products: bf16 and int8 caches
    static constexpr float kOffset = 0.0f;
    typedef __bf16 T;
    static __device__ __forceinline__ f4 mfma(u4 a, u4 b, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
    }
};
template <> struct AttendOps<DQ_F16> {
    static constexpr float kOffset = 15.0f;  // weights are kept times 2^15
    typedef _Float16 T;
    static __device__ __forceinline__ f4 mfma(u4 a, u4 b, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
    }
};

// eight fp32 values as NP pieces of T that add up to them
template <typename T, int NP>
__device__ __forceinline__ void pieces(const float (&x)[8], u4 (&out)[NP]) {
    typedef T V __attribute__((ext_vector_type(8)));
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = x[j];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        V v;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = (T)r[j];
            r[j] -= (float)v[j];
        }
        out[p] = __builtin_bit_cast(u4, v);
    }
}

// Of each value its first piece that is not 0, which has its sign (the others can
// be 0 or of the other sign). magnitude: 0x7fff.
template <int NP>
__device__ __forceinline__ u4 lead_piece(const u4 (&p)[NP], uint32_t magnitude) {
    u4 r = p[0];
#pragma unroll
    for (int i = 1; i < NP; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t keep = (r[w] & magnitude ? 0xffffu : 0u) | (r[w] & magnitude << 16 ? 0xffff0000u : 0u);
            r[w] = (r[w] & keep) | (p[i][w] & ~keep);
        }
    return r;
}

// CT: the cache's type; NQ, NP: pieces of queries and weights; DP: the head
// size rounded up to 64, 128, 192 or 256, or 96 itself (16-bit caches); FULL:
// it is that size.
// Two workgroups are on a compute unit where their registers fit.
constexpr int attend_per_cu(int CT, int NQ, int DP) {
    return DP == 256 ? (CT == DQ_I8 && NQ == 1 ? 2 : 1) : DP == 192 ? (NQ == 3 ? 1 : 2) : 2;
}
template <int CT, int NQ, int NP, int DP, bool FULL>
__global__ void __launch_bounds__(256, attend_per_cu(CT, NQ, DP)) k_attend(const AttendArgs A) {
    typedef AttendOps<CT> Ops;
    typedef typename Ops::T T;
    constexpr int EB = CT == DQ_I8 ? 1 : 2;       // bytes of a value
    constexpr int E = DP / 16;                    // values of V a lane loads for a token
    constexpr int VW = E * EB / 4;                // their words
    // of them neighbours; of 96 and 192 the others lie past d = 64 and 128
    constexpr int EA = DP == 192 ? 8 : DP == 96 ? 4 : E, EX = E - EA;
    constexpr int C = DP / 32;                    // steps of 32 of q . k
    constexpr int KL = DP * EB / 64;              // 16-byte loads of K for 16 tokens
    constexpr int kAcc = DP + 4;
    // V's loads take whole rows and pass the caches by. K's take 64 bytes of 16
    // rows: the rest of a line is the next load's, and is mostly better kept
    // (80 values of 16 bits 42 -> 33 us, 256 of 16 bits 1091 -> 1008, int8 with
    // weights 316 -> 301), but not for rows of 256 bytes (53 -> 51, 64 -> 61).
    constexpr bool KSTREAM = FULL && DP == 128 && EB == 2;
    __shared__ AttendScan scan;
    __shared__ int32_t s_row[4][32];
    __shared__ float s_scale[4][64];
    __shared__ float j_max[4][16], j_sum[4][16], j_l2[16];
    __shared__ float j_acc[4][16 * kAcc];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int n16 = lane & 15, g = lane >> 4;
    const int D = A.D, row_bytes = D * EB;
    const int items = A.Hk * A.tiles;

    // ---- this workgroup's units
    // [u, u_end) are units, or items where a workgroup takes whole items
    KvShare share{};
    int b = 0, len = 0;
    int64_t base = 0, u = blockIdx.x, u_end = (int64_t)A.a.batch * items;
    if (!A.whole) {
        share = attend_scan(A, &scan, blockIdx.x);
        share.units = uniform(share.units);
        share.workers = uniform(share.workers);
        share.each = uniform(share.each);
        __syncthreads();
        b = uniform(scan.b);
        len = uniform(scan.len);
        base = uniform(scan.base);
        const bool works = (int)blockIdx.x < share.workers;
        u = works ? kv_first(blockIdx.x, share) : 0;
        u_end = works ? kv_first(blockIdx.x + 1, share) : 0;
    }

    while (u < u_end) {
        if (A.whole) {
            bool bad;
            b = (int)((uint32_t)u / (uint32_t)items);
            len = uniform(attend_len(A, b, &bad));
        }
        const int first = kv_first_token(len, A.a.window), nb = kv_units(len, A.a.window);
        if (A.whole ? nb == 0 : u >= base + (int64_t)nb * items) {
            if (A.whole) {
                u += A.workers;
                continue;
            }
            base += (int64_t)nb * items;
            bool bad;
            len = attend_len(A, ++b, &bad);
            continue;
        }
        int item, unit0 = 0, count = nb;
        int64_t item_u = 0;
        if (A.whole) {
            item = (int)((uint32_t)u - (uint32_t)b * (uint32_t)items);
        } else {
            const int64_t rel = u - base;
            item = rel >> 32 ? (int)(rel / nb) : (int)((uint32_t)rel / (uint32_t)nb);
            item_u = base + (int64_t)item * nb;
            unit0 = (int)(u - item_u);
            count = (int)(min(u_end, item_u + nb) - u);
        }
        const int hk = item / A.tiles, h0 = hk * A.G + (item - hk * A.tiles) * kHeadTile;
        const int heads = min(kHeadTile, (hk + 1) * A.G - h0);
        const int32_t* line = A.a.table + (size_t)b * A.geom.per_seq;
        const int t_end = min(len, first + (unit0 + count) * kKvUnit);
        int t0 = first + unit0 * kKvUnit + wave * 32;

        // ---- queries: head n16, the values of d that this lane's rows of K
        // have; on their way while the first rows are looked up
        constexpr int QW = NQ == 3 ? 8 : 4;  // words of eight values: fp32 or 16 bits
        uint32_t raw[C][QW];
        {
            constexpr int QE = QW / 2;  // bytes of a value
            const char* p = (const char*)A.a.q + ((long long)b * A.a.q_ts + (long long)(h0 + min(n16, heads - 1)) * A.a.q_hs) * QE;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int d0 = CT == DQ_I8 ? (c >> 1) * 64 + g * 16 + (c & 1) * 8 : c * 32 + g * 8;
                const char* x = p + (FULL || d0 < D ? d0 : 0) * QE;
                if (A.q_vec) {
#pragma unroll
                    for (int w = 0; w < QW; w += 4) {
                        const u4 y = *(const u4*)(x + 4 * w);
#pragma unroll
                        for (int i = 0; i < 4; ++i) raw[c][w + i] = y[i];
                    }
                } else {
#pragma unroll
                    for (int w = 0; w < QW; ++w)
                        raw[c][w] = QE == 4 ? ((const uint32_t*)x)[w]
                                            : ((const uint16_t*)x)[2 * w] | (uint32_t)((const uint16_t*)x)[2 * w + 1] << 16;
                }
            }
        }
        issue_fence();

        f4 acc[E];
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = f4{0, 0, 0, 0};
        float m = -__builtin_inff(), l = 0.0f;
        bool lost = false;

        // the block table's entry for token t + (lane & 31), and that token's row;
        // a token past the end stands for the last one and is masked below
        // (t_end is at most a sequence's slots, so the entry is in the table)
        auto entry_of = [&](int t) { return line[kv_div((uint32_t)min(t + (lane & 31), t_end - 1), A.geom.page)]; };
        auto row_of = [&](int t, int32_t page) {
            const int32_t r = kv_row_of(page, (uint32_t)min(t + (lane & 31), t_end - 1), hk, A.geom);
            lost = lost || r < 0;
            return max(r, 0);
        };
        u4 kf[2][KL];
        auto load_k = [&](int32_t r0, int32_t r1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const char* p = (const char*)A.a.k + (size_t)(uint32_t)(h ? r1 : r0) * row_bytes;
#pragma unroll
                for (int c = 0; c < KL; ++c) {
                    const int o = c * 64 + g * 16;
                    const u4* x = (const u4*)(p + (FULL || o < row_bytes ? o : 0));
                    kf[h][c] = KSTREAM ? __builtin_nontemporal_load(x) : *x;
                }
            }
        };
        // for an int8 cache, the scale of a token's key (lanes below 32) or value
        const float* scales = CT == DQ_I8 ? (lane < 32 ? A.a.ks : A.a.vs) : nullptr;
        float sc = 0.0f;
        int32_t page1 = 0;
        if (t0 < t_end) {
            const int32_t page0 = entry_of(t0);
            page1 = entry_of(t0 + 4 * 32);
            const int32_t r = row_of(t0, page0);
            if (CT == DQ_I8) sc = scales[r];
            s_row[wave][lane & 31] = r;
            wave_lds_fence();
            load_k(s_row[wave][n16], s_row[wave][16 + n16]);
        }
        // kept scores go out as buffer stores, which drop the lanes without a
        // head (and all, where none are kept): no branch around them
        const auto s_out = __builtin_amdgcn_make_buffer_rsrc(
            A.s + attend_score_at(A, b * A.Hk + hk, 0), 0, A.s ? (int)(A.s_stride * 4) : 0, 0x00027000);

        // ---- queries as MFMA operands
        u4 q[C][NQ];
        float scale = A.a.sm_scale * kLog2e;
        if (NQ == 1 && (CT != DQ_F16 || A.q_type == DQ_F16)) {
            // as they are
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int d0 = CT == DQ_I8 ? (c >> 1) * 64 + g * 16 + (c & 1) * 8 : c * 32 + g * 8;
                const bool in = n16 < heads && (FULL || d0 < D);
#pragma unroll
                for (int w = 0; w < 4; ++w) q[c][0][w] = in ? raw[c][w] : 0;
            }
        } else {
            float x[C][8];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int d0 = CT == DQ_I8 ? (c >> 1) * 64 + g * 16 + (c & 1) * 8 : c * 32 + g * 8;
                const bool in = n16 < heads && (FULL || d0 < D);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float y;
                    if (NQ == 3) {
                        y = __uint_as_float(raw[c][j % QW]);
                    } else {
                        // fp16 on a bf16 or int8 cache, bf16 on an fp16 one
                        const uint16_t h = (uint16_t)(raw[c][j / 2] >> (16 * (j & 1)));
                        y = CT == DQ_F16 ? bf16_bits_to_f32(h) : (float)__builtin_bit_cast(_Float16, h);
                    }
                    x[c][j] = in ? y : 0.0f;
                }
            }
            if (CT == DQ_F16) {
                // to [2^14, 2^15): the power of two of the row's largest
                float top = 0.0f;
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int j = 0; j < 8; ++j) top = __builtin_fmaxf(top, __builtin_fabsf(x[c][j]));
                top = head_max(top);
                const int e = top > 0.0f && top < __builtin_inff() ? 15 - __builtin_amdgcn_frexp_expf(top) : 0;
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[c][j] = __builtin_ldexpf(x[c][j], e);
                scale = __builtin_ldexpf(scale, -e);
            }
#pragma unroll
            for (int c = 0; c < C; ++c) pieces<T, NQ>(x[c], q[c]);
        }

        // Loads return in order and a wait names how many may be outstanding, so
        // no load or store of the loop is behind a branch: an iteration's
        // values are waited for while the next one's keys are on their way.
        for (; t0 < t_end; t0 += 4 * 32) {
            const int32_t page2 = entry_of(t0 + 2 * 4 * 32);
            // rows of V, tokens 4 g + j and 16 + 4 g + j
            const v4i ra = *(const v4i*)&s_row[wave][4 * g], rb = *(const v4i*)&s_row[wave][16 + 4 * g];
            f4 ks[2], vs[2];
            if (CT == DQ_I8) {
                s_scale[wave][lane] = sc;
                wave_lds_fence();
                ks[0] = *(const f4*)&s_scale[wave][4 * g];
                ks[1] = *(const f4*)&s_scale[wave][16 + 4 * g];
                vs[0] = *(const f4*)&s_scale[wave][32 + 4 * g];
                vs[1] = *(const f4*)&s_scale[wave][48 + 4 * g];
            }
            uint32_t vf[8][VW];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int32_t r = j < 4 ? ra[j] : rb[j - 4];
                const char* p = (const char*)A.a.v + (size_t)(uint32_t)r * row_bytes;
                const int o = n16 * EA * EB;
                load_words<EA * EB / 4>(p + (FULL || o < row_bytes ? o : 0), vf[j]);
                if constexpr (EX > 0) {
                    const int o2 = (EA * 16 + n16 * EX) * EB;
                    load_words<EX * EB / 4>(p + (FULL || o2 < row_bytes ? o2 : 0), vf[j] + EA * EB / 4);
                }
            }
            issue_fence();
            // ---- scores
            f4 s[2] = {f4{0, 0, 0, 0}, f4{0, 0, 0, 0}};
            // h's 16 tokens and 32 values of d (int8: 64) of K
            auto keys = [&](int h, int c) {
                u4 x = kf[h][c];
                if (!FULL && c * 64 + g * 16 >= row_bytes) x = u4{0, 0, 0, 0};
                return x;
            };
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int c = 0; c < KL; ++c) {
                    const u4 x = keys(h, c);
                    if constexpr (CT == DQ_I8) {
                        const u2 a = codes_bf16x4(x[0]), e = codes_bf16x4(x[1]), i = codes_bf16x4(x[2]),
                                 o = codes_bf16x4(x[3]);
#pragma unroll
                        for (int p = 0; p < NQ; ++p) {
                            s[h] = Ops::mfma(u4{a[0], a[1], e[0], e[1]}, q[2 * c][p], s[h]);
                            s[h] = Ops::mfma(u4{i[0], i[1], o[0], o[1]}, q[2 * c + 1][p], s[h]);
                        }
                    } else {
#pragma unroll
                        for (int p = 0; p < NQ; ++p) s[h] = Ops::mfma(x, q[c][p], s[h]);
                    }
                }
            if constexpr (NQ > 1 && CT != DQ_I8) {
                // Times an infinite key the pieces of one value can be of both
                // signs or 0, and their sum a NaN where the product is infinite:
                // a score that is not finite is taken from one piece a value (one
                // such leaves no finite sum of the eight). The check costs 4 x
                // 400 tokens of 8 heads of 64, fp32 on bf16, 8.1 to 8.4 us, with
                // 128 values or 32 x 3000 tokens nothing.
                auto finite = [](float y) { return __builtin_fabsf(y) < __builtin_inff(); };
                const f4 sum = s[0] + s[1];
                if (__builtin_expect(__ballot(!finite((sum[0] + sum[1]) + (sum[2] + sum[3]))) != 0, 0)) {
                    // (found here when they are needed: kept through the loop
                    // they would take 4 C registers)
                    uint32_t magnitude = 0x7fffu;
                    asm volatile("" : "+s"(magnitude));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        f4 y = {0, 0, 0, 0};
#pragma unroll
                        for (int c = 0; c < KL; ++c) y = Ops::mfma(keys(h, c), lead_piece<NQ>(q[c], magnitude), y);
#pragma unroll
                        for (int r = 0; r < 4; ++r) s[h][r] = finite(s[h][r]) ? s[h][r] : y[r];
                    }
                }
            }
            // ---- weights
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float y = s[j >> 2][j & 3];
                if (CT == DQ_I8) y *= ks[j >> 2][j & 3];
                y *= scale;
                x[j] = t0 + 16 * (j >> 2) + 4 * g + (j & 3) < t_end ? y : -__builtin_inff();
            }
            {
                const int o = (((t0 - first) >> 5) * A.G + (h0 - hk * A.G + n16)) * 32 + 4 * g;
                const int at = n16 < heads ? o * 4 : -256;
                const f4 y0 = {x[0], x[1], x[2], x[3]}, y1 = {x[4], x[5], x[6], x[7]};
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, y0), s_out, at, 0, 0);
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, y1), s_out, at + 64, 0, 0);
            }
            // ---- next keys; past the end, the last row once more
            {
                const int32_t r = row_of(t0 + 4 * 32, page1);
                page1 = page2;
                if (CT == DQ_I8) sc = scales[r];
                s_row[wave][lane & 31] = r;
                wave_lds_fence();
                load_k(s_row[wave][n16], s_row[wave][16 + n16]);
            }
            issue_fence();
            // ---- the running maximum
            float top = x[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) top = __builtin_fmaxf(top, x[j]);
            top = __builtin_fmaxf(head_max(top) - Ops::kOffset, m);
            const float ref = top == -__builtin_inff() ? 0.0f : top;
            if (__ballot(top != m)) {
                const float f = __builtin_amdgcn_exp2f(m - ref);
                l *= f;
#pragma unroll
                for (int i = 0; i < E; ++i) acc[i] *= f;
                m = top;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = __builtin_amdgcn_exp2f(x[j] - ref);
                l += x[j];
                if (CT == DQ_I8) x[j] *= vs[j >> 2][j & 3];
            }
            if (t0 + 32 > t_end) {
                // the tokens that stand in past the end: their weight is 0, but
                // 0 times what is not finite would not be
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (t0 + 16 * (j >> 2) + 4 * g + (j & 3) >= t_end) {
                        x[j] = 0.0f;
#pragma unroll
                        for (int w = 0; w < VW; ++w) vf[j][w] = 0;
                    }
            }
            u4 p[NP];
            pieces<T, NP>(x, p);
            // ---- values: operand i has value i of each of the lane's tokens
#pragma unroll
            for (int i = 0; i < E; ++i) {
                u4 a;
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    if constexpr (CT == DQ_I8) {
                        const uint32_t x0 = vf[2 * jj][i >> 2] << (24 - 8 * (i & 3));
                        const uint32_t x1 = vf[2 * jj + 1][i >> 2] << (24 - 8 * (i & 3));
                        a[jj] = exact_bf16x2((float)((int32_t)x0 >> 24), (float)((int32_t)x1 >> 24));
                    } else {
                        a[jj] = __builtin_amdgcn_perm(vf[2 * jj + 1][i >> 1], vf[2 * jj][i >> 1],
                                                      i & 1 ? 0x07060302u : 0x05040100u);
                    }
                }
#pragma unroll
                for (int w = 0; w < NP; ++w) acc[i] = Ops::mfma(a, p[w], acc[i]);
            }
        }

        // ---- the four waves' results
        l = head_sum(l);
        if (__ballot(lost)) {
            l = __builtin_nanf("");
            if (lane == 0) atomicAdd(A.bad, 1);
        }
        if (g == 0) {
            j_max[wave][n16] = m;
            j_sum[wave][n16] = l;
        }
        if (n16 < heads) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int i = 0; i < E; i += 2)
                    *(f2*)&j_acc[wave][n16 * kAcc + (i < EA ? EA * (4 * g + r) + i : EA * 16 + EX * (4 * g + r) + i - EA)] =
                        f2{acc[i][r], acc[i + 1][r]};
        }
        __syncthreads();
        const bool whole = unit0 == 0 && count == nb;
        if (unit0 == 0 && tid == 0 && !A.whole)
            A.parts[(size_t)b * items + item] =
                int2{(int)blockIdx.x, whole ? 0 : kv_worker(item_u + nb - 1, share) - (int)blockIdx.x + 1};
        float* part = A.part + (size_t)(2 * blockIdx.x + (unit0 == 0 ? 1 : 0)) * kHeadTile * (D + 4);
        for (int e = tid; e < heads * (D / 4); e += 256) {
            const int n = e / (D / 4), d = (e - n * (D / 4)) * 4;
            float top = j_max[0][n];
#pragma unroll
            for (int w = 1; w < 4; ++w) top = __builtin_fmaxf(top, j_max[w][n]);
            const float ref = top == -__builtin_inff() ? 0.0f : top;
            float sum = 0.0f;
            f4 o = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float f = __builtin_amdgcn_exp2f(j_max[w][n] - ref);
                sum += j_sum[w][n] * f;
                o += *(const f4*)&j_acc[w][n * kAcc + d] * f;
            }
            if (whole) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                const size_t i = (size_t)b * A.Hq + h0 + n;
                if (sum == 0.0f) o = f4{0, 0, 0, 0};
                store4_any(A.a.out, A.q_type, i * D + d, o * inv);
                if (d == 0) {
                    const float l2 = sum == 0.0f ? -__builtin_inff() : ref + __builtin_amdgcn_logf(sum);
                    A.l2[i] = l2;
                    // for the gathered weights: 2^(s - inf) = 0 where there is none
                    j_l2[n] = sum == 0.0f ? __builtin_inff() : l2;
                    if (A.a.lse) A.a.lse[i] = l2 * kLn2;
                }
            } else {
                *(f4*)&part[n * (D + 4) + 4 + d] = o;
                if (d == 0) {
                    part[n * (D + 4)] = top;
                    part[n * (D + 4) + 1] = sum;
                }
            }
        }
        if (A.whole && A.s) {
            // ---- gathered weights; the scores that the waves kept are read
            // back by others, once all of them have reached the L2 cache
            wait_vmcnt<0>();
            __syncthreads();
            // (at most kWholeBefore slots before the window)
            const size_t row = (size_t)(b * A.Hk + hk) * A.cap;
            for (int t = tid; t < first; t += 256) A.a.scores_out[row + t] = A.a.scores[row + t] * A.a.decay;
            const float* kept = A.s + attend_score_at(A, b * A.Hk + hk, 0);
            for (int r = tid; r < len - first; r += 256) {
                const float* y = kept + (size_t)(r >> 5) * (32 * A.G) + (r & 31);
                float p = 0.0f;
                for (int x = 0; x < heads; ++x) p += __builtin_amdgcn_exp2f(y[x * 32] - j_l2[x]);
                A.a.scores_out[row + first + r] = A.a.scores[row + first + r] * A.a.decay + p;
            }
        }
        __syncthreads();
        u += A.whole ? A.workers : count;
    }

    // ---- sequences without a token
    for (int b = blockIdx.x; b < A.a.batch; b += A.workers) {
        bool bad;
        if (attend_len(A, b, &bad) > 0) continue;
        if (bad && tid == 0) atomicAdd(A.bad, 1);
        const float o = bad ? __builtin_nanf("") : 0.0f, l2 = bad ? __builtin_nanf("") : -__builtin_inff();
        for (int i = tid; i < A.Hq * D; i += 256) store_any(A.a.out, A.q_type, (long long)b * A.Hq * D + i, o);
        for (int i = tid; i < A.Hq; i += 256) {
            A.l2[(size_t)b * A.Hq + i] = l2;
            if (A.a.lse) A.a.lse[(size_t)b * A.Hq + i] = l2;
        }
        for (int i = tid; i < items && !A.whole; i += 256) A.parts[(size_t)b * items + i] = int2{0, 0};
    }
}

// instances of one cache type (paged_attend_*.hip)
typedef void (*AttendKernel)(const AttendArgs);
AttendKernel attend_bf16(dq_dtype q, int D);
AttendKernel attend_f16(dq_dtype q, int D);
AttendKernel attend_i8(dq_dtype q, int D);

template <int CT, int NQ, int NP>
AttendKernel attend_pick(int D) {
    if (D <= 64) return D == 64 ? k_attend<CT, NQ, NP, 64, true> : k_attend<CT, NQ, NP, 64, false>;
    // (80 on tiles of 96 was slower than on tiles of 128)
    if constexpr (CT != DQ_I8)
        if (D == 96) return k_attend<CT, NQ, NP, 96, true>;
    if (D <= 128) return D == 128 ? k_attend<CT, NQ, NP, 128, true> : k_attend<CT, NQ, NP, 128, false>;
    if (D <= 192) return D == 192 ? k_attend<CT, NQ, NP, 192, true> : k_attend<CT, NQ, NP, 192, false>;
    return D == 256 ? k_attend<CT, NQ, NP, 256, true> : k_attend<CT, NQ, NP, 256, false>;
}

}  // namespace dq
