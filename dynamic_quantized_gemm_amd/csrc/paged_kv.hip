// paged_kv.hip -- the paged key-value cache: its context, the append of new
// keys and values (rotated, and quantized per row for an int8 cache), the read
// of stored rows, and the eviction of the tokens with the least gathered
// attention. The attention itself is in paged_attend.hip.
//
// The cache is [pages, Hk, page_size, D]: one head's slots of a page are one
// run of memory, so a head's tokens stream in runs of page_size rows. An int8
// row's scale is one fp32 of [pages, Hk, page_size].
#include <math.h>
#include <stdio.h>

#include <algorithm>
#include <new>
#include <type_traits>

#include "paged_kv.h"

using namespace dq;

namespace {

// ------------------------------------------------------------------ append
//
// A row is one head's D values of one token: the query heads (rotated into
// q_out), the key heads (rotated, then stored) and the value heads (stored).
// Sixteen lanes hold a row, in virtual pairs (kv_pair), and walk `chunk` rows
// of one token with the same cosines and sines, which the workgroup computes
// once for its tokens. For an int8 cache the row's
// largest magnitude is reduced over those sixteen lanes in registers, so each
// row is read once and its codes and scale written once.
// Bound by that traffic: 6001 tokens of 32 + 16 heads of 128 in bf16 25.9 to
// 27.1 us, 5.4 to 5.7 TB/s; a plain copy of as much takes 26.0 to 26.5 us.

struct AppendArgs {
    const void *q, *k, *v;
    void* q_out;
    long long qt, qh, kt, kh, vt, vh;  // strides in elements
    const int32_t* index;
    const int32_t* seq_ids;  // NULL: token t belongs to sequence t
    const int32_t* table;
    void *kc, *vc;
    float *ks, *vs;
    int32_t* bad;
    const int32_t* pos;  // NULL: no rotation
    const double2* freq;
    const int32_t* axis;
    uint32_t groups;  // tokens * chunks
    int tokens, batch, Hq, Hk, D, R, chunk;
    KvDiv chunks;
    KvGeom geom;
};

__device__ __forceinline__ uint32_t max16(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kDppXor1, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kDppXor2, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kDppRowHalfMirror, 0xF, 0xF, false));
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kDppRowMirror, 0xF, 0xF, false));
}

constexpr int kKvDimMax = 256;  // 128 pairs: eight a lane

template <int TI, int TC, int VP, bool IL>
__global__ void __launch_bounds__(256) k_kv_append(const AppendArgs A) {
    typedef typename Elem<TI>::S SI;
    typedef typename Elem<TC>::S SC;
    constexpr int NIT = kKvDimMax / 2 / 16 / VP;
    extern __shared__ float2 tab[];
    const int l = threadIdx.x & 15;
    const uint32_t g0 = blockIdx.x * 16u, last = min(g0 + 15u, A.groups - 1);
    const uint32_t g = min(g0 + (threadIdx.x >> 4), last);
    const uint32_t t = kv_div(g, A.chunks);
    const int rows = A.Hq + 2 * A.Hk;
    const int r0 = (int)(g - t * A.chunks.d) * A.chunk, r1 = min(rows, r0 + A.chunk);
    const int pairs = A.D / 2;
    const int turned = A.pos ? A.R / 2 : 0;

    // the workgroup's tokens share their angles
    const int t0 = (int)kv_div(g0, A.chunks);
    if (A.pos)
        rope_table(tab, t0, (int)kv_div(last, A.chunks) - t0 + 1, A.R / 2, A.pos, A.tokens, A.freq, A.axis, false);
    if (g0 + (threadIdx.x >> 4) > last) return;
    float c[NIT][VP], s[NIT][VP];
    int lo[NIT], hi[NIT];
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
        const int i0 = (it * 16 + l) * VP;
        kv_pair(i0, A.D, turned ? A.R : A.D, IL, &lo[it], &hi[it]);
        if (i0 < turned) {
#pragma unroll
            for (int i = 0; i < VP; ++i) {
                const float2 cs = tab[((int)t - t0) * (A.R / 2) + i0 + i];
                c[it][i] = cs.x;
                s[it][i] = cs.y;
            }
        }
    }
    // where this token goes
    const int at = r1 > A.Hq ? A.index[t] : -1;
    const int seq = at < 0 ? 0 : A.seq_ids ? A.seq_ids[t] : (int)t;
    const bool seq_ok = (uint32_t)seq < (uint32_t)A.batch;
    const int32_t* line = A.table + (size_t)(seq_ok ? seq : 0) * A.geom.per_seq;

    for (int r = r0; r < r1; ++r) {
        const bool is_q = r < A.Hq, is_v = r >= A.Hq + A.Hk;
        const int h = is_q ? r : is_v ? r - A.Hq - A.Hk : r - A.Hq;
        int32_t row = -1;
        if (!is_q) {
            if (at < 0) continue;
            row = seq_ok ? kv_row(line, (uint32_t)at, h, A.geom) : -1;
            if (row < 0) {
                if (l == 0) atomicAdd(A.bad, 1);
                continue;
            }
        }
        const SI* x = is_q ? (const SI*)A.q + t * A.qt + h * A.qh
                           : is_v ? (const SI*)A.v + t * A.vt + h * A.vh : (const SI*)A.k + t * A.kt + h * A.kh;
        float a[NIT][VP], b[NIT][VP];
        uint32_t top = 0;
#pragma unroll
        for (int it = 0; it < NIT; ++it) {
            const int i0 = (it * 16 + l) * VP;
            if (i0 >= pairs) continue;
            load_pairs<SI, VP, IL>(x, lo[it], hi[it], a[it], b[it]);
            if (!is_v && i0 < turned) {
#pragma unroll
                for (int i = 0; i < VP; ++i) {
                    const float u = a[it][i] * c[it][i] - b[it][i] * s[it][i];
                    b[it][i] = b[it][i] * c[it][i] + a[it][i] * s[it][i];
                    a[it][i] = u;
                }
            }
#pragma unroll
            for (int i = 0; i < VP; ++i)
                top = max(top, max(__float_as_uint(a[it][i]) & 0x7fffffffu, __float_as_uint(b[it][i]) & 0x7fffffffu));
        }
        if (is_q) {
            SI* y = (SI*)A.q_out + ((size_t)t * A.Hq + h) * A.D;
#pragma unroll
            for (int it = 0; it < NIT; ++it)
                if ((it * 16 + l) * VP < pairs) store_pairs<SI, VP, IL>(y, lo[it], hi[it], a[it], b[it]);
            continue;
        }
        SC* y = (SC*)(is_v ? A.vc : A.kc) + (size_t)row * A.D;
        if constexpr (TC == DQ_I8) {
            // magnitudes as integers keep a NaN above infinity: a row that is
            // not finite is stored as zeros with a NaN for its scale, so that
            // it reads back as NaN
            top = max16(top);
            const bool finite = top < 0x7f800000u;
            float scale = __uint_as_float(top) / 127.0f;
            if (!(scale > 0.0f)) scale = 1.0f;
            const QDiv d = make_qdiv(scale);
#pragma unroll
            for (int it = 0; it < NIT; ++it) {
                if ((it * 16 + l) * VP >= pairs) continue;
#pragma unroll
                for (int i = 0; i < VP; ++i) {
                    a[it][i] = finite ? fminf(fmaxf(rne(qdiv(a[it][i], d)), -127.0f), 127.0f) : 0.0f;
                    b[it][i] = finite ? fminf(fmaxf(rne(qdiv(b[it][i], d)), -127.0f), 127.0f) : 0.0f;
                }
                store_pairs<SC, VP, IL>(y, lo[it], hi[it], a[it], b[it]);
            }
            if (l == 0) (is_v ? A.vs : A.ks)[row] = finite ? scale : __uint_as_float(0x7fc00000u);
        } else {
#pragma unroll
            for (int it = 0; it < NIT; ++it)
                if ((it * 16 + l) * VP < pairs) store_pairs<SC, VP, IL>(y, lo[it], hi[it], a[it], b[it]);
        }
    }
}

// -------------------------------------------------------------------- read

struct ReadArgs {
    const int32_t* index;
    const int32_t* seq_ids;
    const int32_t* table;
    const void *kc, *vc;
    const float *ks, *vs;
    void *k_out, *v_out;
    int32_t* bad;
    uint32_t threads;  // tokens * heads * D / 8
    int Hk, D, batch;
    KvDiv pieces, heads;
    KvGeom geom;
};

// eight values of one row a thread; a slot that holds nothing (index < 0)
// reads as zeros, one that cannot exist as NaN
template <int TO, int TC>
__global__ void __launch_bounds__(256) k_kv_read(const ReadArgs A) {
    typedef typename Elem<TO>::S SO;
    typedef typename Elem<TC>::S SC;
    const uint32_t id = blockIdx.x * 256u + threadIdx.x;
    if (id >= A.threads) return;
    const uint32_t rest = kv_div(id, A.pieces);
    const int e = (int)(id - rest * A.pieces.d) * 8;
    const uint32_t t = kv_div(rest, A.heads);
    const int h = (int)(rest - t * A.heads.d);
    const int at = A.index[t], seq = A.seq_ids ? A.seq_ids[t] : (int)t;
    int32_t row = -1;
    if (at >= 0) {
        if ((uint32_t)seq < (uint32_t)A.batch)
            row = kv_row(A.table + (size_t)seq * A.geom.per_seq, (uint32_t)at, h, A.geom);
        if (row < 0 && e == 0) atomicAdd(A.bad, 1);
    }
    const size_t o = ((size_t)t * A.Hk + h) * A.D + e;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        SO* out = (SO*)(w ? A.v_out : A.k_out);
        if (!out) continue;
        float f[8];
        if (row < 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = at < 0 ? 0.0f : __uint_as_float(0x7fc00000u);
        } else {
            load_vec((const SC*)(w ? A.vc : A.kc) + (size_t)row * A.D + e, f);
            if constexpr (TC == DQ_I8) {
                const float scale = (w ? A.vs : A.ks)[row];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] *= scale;
            }
        }
        if constexpr (TO == DQ_F32) {
            const float f0[4] = {f[0], f[1], f[2], f[3]}, f1[4] = {f[4], f[5], f[6], f[7]};
            store_vec(out + o, f0);
            store_vec(out + o + 4, f1);
        } else {
            store_vec(out + o, f);
        }
    }
}

// ---------------------------------------------------------------- eviction
//
// Of a head's n > budget tokens those with the `budget` largest keys stay,
// where a key is the gathered weight as an ordered integer, one above all weights
// for the first `sinks` and last `recent` tokens, ties going to the lowest
// slot. One workgroup of 16 waves selects for one head, each wave a run of
// slots, so that ballots count in slot order:
//   the keys, read once and kept in registers up to 64 a lane (beyond 65536
//   tokens they are read again for every pass);
//   the budget-th largest key, 8 bits at a time, from histograms in LDS, of
//   which there are eight, by lane: weights of one magnitude would otherwise
//   meet in one counter. The keys with the first 8 bits are left in LDS on the
//   way, and the third and fourth pass look at those alone (32768 tokens: 28.5 to
//   26.7 us), unless they are more than 4096;
//   the slots below the budget that came free and the slots beyond it that
//   stay, in order, as two lists.
// One token over the budget takes one pass instead (32769 tokens of 128 heads:
// 95 to 18.6 us). Bound by its chain of passes on one compute unit a head: 64
// heads of up to 32768 tokens 28 us, the moves 25 us, 4.6 TB/s of 256-byte rows.
// A second launch moves the rows, which are most of the traffic, with the whole
// chip; where at most 64 rows of a head can move (a token at a time over the
// budget) the first moves them itself.

struct EvictArgs {
    const int32_t *lens, *newest;
    const float* scores;
    const int32_t* order;
    const int32_t* table;
    void *kc, *vc;
    float *ks, *vs;
    float* scores_out;
    int32_t* order_out;
    int32_t* lens_out;
    int32_t* moves;
    size_t moves_stride;
    int32_t* bad;
    int batch, Hk, cap, budget, sinks, recent, row_bytes;
    int moves_too;  // the selection moves the rows itself
    KvGeom geom;
};

constexpr int kSelThreads = 1024, kSelWaves = kSelThreads / 64;

__device__ __forceinline__ uint32_t evict_key(float score, int order, int sinks, long long recent_from) {
    const uint32_t k = score != score ? 0xfffffffeu : f2ord(score);  // a NaN is the largest weight
    // (both compared, no branch: with one, 100000 tokens of 8 heads take 176 us, not 167)
    return (order < sinks) | (order > recent_from) ? 0xffffffffu : k;  // stays before any weight
}

// Up to R rows of keys, values, scales, weights and numbers by sixteen lanes:
// lane j < R finds row j's place, then all rows are on their way before the
// first is written. A key row and its value row are one run of pieces.
constexpr int kMoveRows = 4;

__device__ __forceinline__ void move_rows(const EvictArgs& A, int item, int b, int h, const int32_t* dst,
                                          const int32_t* src, int count, int l) {
    const int32_t* line = A.table + (size_t)b * A.geom.per_seq;
    const size_t base = (size_t)item * A.cap;
    int32_t to = -1, from = -1;
    if (l < min(count, kMoveRows)) {
        const int d = dst[l], s = src[l];
        to = kv_row(line, (uint32_t)d, h, A.geom);
        from = kv_row(line, (uint32_t)s, h, A.geom);
        A.scores_out[base + d] = A.scores[base + s];
        A.order_out[base + d] = A.order[base + s];
        if (to < 0 || from < 0) {
            atomicAdd(A.bad, 1);
            to = from = -1;
        } else if (A.ks) {
            A.ks[to] = A.ks[from];
            A.vs[to] = A.vs[from];
        }
    }
    // (all sixteen lanes take part in the exchange; in the loop some may not)
    int32_t t[kMoveRows], f[kMoveRows];
#pragma unroll
    for (int j = 0; j < kMoveRows; ++j) {
        t[j] = __shfl(to, j, 16);
        f[j] = __shfl(from, j, 16);
    }
    const int pieces = A.row_bytes / 16;
    for (int o = l; o < 2 * pieces; o += 16) {
        char* c = (char*)(o < pieces ? A.kc : A.vc) + (o < pieces ? o : o - pieces) * 16;
        v4i x[kMoveRows];
#pragma unroll
        for (int j = 0; j < kMoveRows; ++j)
            if (f[j] >= 0) x[j] = __builtin_nontemporal_load((const v4i*)(c + (size_t)f[j] * A.row_bytes));
#pragma unroll
        for (int j = 0; j < kMoveRows; ++j)
            if (t[j] >= 0) *(v4i*)(c + (size_t)t[j] * A.row_bytes) = x[j];
    }
}

constexpr int kHistCopies = 8;
constexpr int kNear = 4096;  // keys that share the first 8 bits, kept in LDS

struct SelectShared {
    uint32_t hist[256 * kHistCopies];
    uint32_t a[kSelWaves], b[kSelWaves];
    uint32_t digit, left, ties, count, found;
    uint32_t near[kNear];
    unsigned long long least[kSelWaves];
};

// One token over the budget, the steady state of decoding: the least key
// leaves, of equal ones that in the highest slot, and the token in the slot
// beyond the budget takes its place. One pass over the keys, whatever their
// number.
__device__ __forceinline__ void evict_one(const EvictArgs& A, SelectShared& sh, int item, int b, int n) {
    const int tid = threadIdx.x;
    const size_t base = (size_t)item * A.cap;
    const float* sc = A.scores + base;
    const int32_t* od = A.order + base;
    float* sco = A.scores_out + base;
    int32_t* odo = A.order_out + base;
    const bool copies = sco != sc || odo != od;
    const long long recent_from = (long long)A.newest[b] - A.recent;
    unsigned long long least = ~0ull;
    constexpr int KG = 8;
    for (int k0 = 0; k0 < n; k0 += KG * kSelThreads) {
        float f[KG];
        int32_t o[KG];
#pragma unroll
        for (int k = 0; k < KG; ++k) {
            const int i = min(k0 + k * kSelThreads + tid, n - 1);
            f[k] = sc[i];
            o[k] = od[i];
        }
        issue_fence();
#pragma unroll
        for (int k = 0; k < KG; ++k) {
            const int i = min(k0 + k * kSelThreads + tid, n - 1);
            const uint32_t x = evict_key(f[k], o[k], A.sinks, recent_from);
            least = min(least, (unsigned long long)x << 32 | (0xffffffffu - (uint32_t)i));
            if (copies && i < A.budget) {
                sco[i] = f[k];
                odo[i] = o[k];
            }
        }
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) least = min(least, (unsigned long long)__shfl_xor(least, o));
    if ((tid & 63) == 0) sh.least[tid >> 6] = least;
    wait_vmcnt<0>();  // what is copied has arrived before a moved value goes to the same place
    __syncthreads();
    if (tid == 0) {
        for (int w = 0; w < kSelWaves; ++w) least = min(least, sh.least[w]);
        const int slot = (int)(0xffffffffu - (uint32_t)least);
        int32_t* dst = A.moves + (size_t)A.batch * A.Hk + (size_t)item * 2 * A.moves_stride;
        dst[0] = slot;
        dst[A.moves_stride] = A.budget;
        sh.count = slot < A.budget ? 1 : 0;
    }
}

// KPT (a multiple of 4, up to 64): keys a lane holds at a time, runs of four
// neighbouring slots. MEM: there are more than that, and every pass reads them
// again, KPT at a time.
template <int KPT, bool MEM>
__device__ __forceinline__ void evict_select(const EvictArgs& A, SelectShared& sh, int item, int b, int n) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const size_t base = (size_t)item * A.cap;
    const float* sc = A.scores + base;
    const int32_t* od = A.order + base;
    const long long recent_from = (long long)A.newest[b] - A.recent;
    // run k of a lane: slots i0 + 256 k + (0 .. 3); a wave's slots are one run
    constexpr int KV = KPT / 4;
    typedef typename std::conditional<KPT <= 32, uint32_t, uint64_t>::type Bits;
    const int iters = (n + 4 * kSelThreads - 1) / (4 * kSelThreads);
    const int i0 = wave * iters * 256 + lane * 4;
    // f(k, weights, numbers, how many there are) for the lane's runs k0 + k, up
    // to four of each on their way at a time
    typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));
    typedef int i4u __attribute__((ext_vector_type(4), aligned(4)));
    constexpr int KG = KV < 4 ? KV : 4;
    auto runs = [&](int k0, auto fn) {
#pragma unroll
        for (int g = 0; g < KV; g += KG) {
            f4u f[KG];
            i4u o[KG];
#pragma unroll
            for (int k = 0; k < KG; ++k) {
                const int i = i0 + (k0 + g + k) * 256;
                f[k] = f4u{0, 0, 0, 0};
                o[k] = i4u{0, 0, 0, 0};
                if (k0 + g + k < iters && i + 4 <= n) {
                    f[k] = *(const f4u*)(sc + i);
                    o[k] = *(const i4u*)(od + i);
                } else if (k0 + g + k < iters) {
#pragma unroll
                    for (int j = 0; j < 3; ++j)
                        if (i + j < n) {
                            f[k][j] = sc[i + j];
                            o[k][j] = od[i + j];
                        }
                }
            }
            issue_fence();
#pragma unroll
            for (int k = 0; k < KG; ++k)
                fn(g + k, f[k], o[k], k0 + g + k < iters ? max(0, min(4, n - (i0 + (k0 + g + k) * 256))) : 0);
        }
    };
    uint32_t x[KPT];
    // 0 is below every key: what stands in past a wave's or the head's end is
    // never reached, since n > budget keys are above it
    auto load = [&](int k0) {
        runs(k0, [&](int k, f4u f, i4u o, int have) {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[4 * k + j] = j < have ? evict_key(f[j], o[j], A.sinks, recent_from) : 0;
        });
    };
    // f(k0): the keys x of the lane's runs k0 ..
    auto blocks = [&](auto f) {
        for (int k0 = 0; k0 < (MEM ? iters : 1); k0 += KV) {
            if (MEM) load(k0);
            f(k0);
        }
    };
    if (!MEM) load(0);
    uint32_t prefix = 0, left = (uint32_t)A.budget;  // of the keys that tie with the prefix, so many stay
    uint32_t* mine = sh.hist + (lane & (kHistCopies - 1));
    bool listed = false;  // the keys with the prefix's first 8 bits are in LDS
    uint32_t found = 0;   // so many
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256 * kHistCopies; i += kSelThreads) sh.hist[i] = 0;
        if (tid == 0) sh.found = 0;
        __syncthreads();
        if (shift < 16 && listed) {
            for (uint32_t i = tid; i < found; i += kSelThreads) {
                const uint32_t y = sh.near[i];
                if (((y ^ prefix) >> (shift + 8)) == 0) atomicAdd(mine + ((y >> shift) & 255u) * kHistCopies, 1u);
            }
        } else {
            blocks([&](int) {
#pragma unroll
                for (int k = 0; k < KPT; ++k)
                    if (shift == 24 || ((x[k] ^ prefix) >> (shift + 8)) == 0) {
                        atomicAdd(mine + ((x[k] >> shift) & 255u) * kHistCopies, 1u);
                        if (shift == 16 && listed) sh.near[atomicAdd(&sh.found, 1u)] = x[k];
                    }
            });
        }
        __syncthreads();
        if (tid < 64) {
            // four digits a lane, from 255 down; the digit at which the count
            // of larger ones would pass `left`
            uint32_t c[4], sum = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const u4* h = (const u4*)&sh.hist[(255 - (4 * lane + j)) * kHistCopies];
                const u4 p = h[0], q = h[1];
                c[j] = p[0] + p[1] + p[2] + p[3] + q[0] + q[1] + q[2] + q[3];
                sum += c[j];
            }
            uint32_t before = sum;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const uint32_t z = __shfl_up(before, o);
                if (lane >= o) before += z;
            }
            before -= sum;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (before < left && before + c[j] >= left) {
                    sh.digit = 255 - (4 * lane + j);
                    sh.left = left - before;
                    sh.ties = c[j];
                }
                before += c[j];
            }
        }
        __syncthreads();
        prefix |= sh.digit << shift;
        left = sh.left;
        if (sh.ties == left) break;  // all of the prefix stay, whatever follows it
        if (shift == 24) {
            found = sh.ties;
            listed = found <= kNear;
        }
    }
    // Which stay: key > prefix, or key == prefix among the first `left` such
    // slots. Mostly all of those stay, and no order has to be found.
    const bool all_ties = sh.ties == left;
    const unsigned long long below = (1ull << lane) - 1;
    uint32_t tie = 0;
    if (!all_ties) {
        blocks([&](int) {
#pragma unroll
            for (int k = 0; k < KPT; ++k) tie += __popcll(__ballot(x[k] == prefix));
        });
        if (lane == 0) sh.a[wave] = tie;
        __syncthreads();
        tie = 0;
        for (int w = 0; w < wave; ++w) tie += sh.a[w];
        __syncthreads();
    }
    // f(k0, kept, under): bits of the block's slots that stay, and of those
    // below the budget
    auto sort_out = [&](auto f) {
        uint32_t t = tie;
        blocks([&](int k0) {
            Bits kept = 0, under = 0;
#pragma unroll
            for (int k = 0; k < KV; ++k) {
                const int low = k0 + k < iters ? max(0, min(4, A.budget - (i0 + (k0 + k) * 256))) : 0;
                under |= (Bits)((1u << low) - 1) << (4 * k);
                uint32_t before = 0;
                if (!all_ties) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) before += __popcll(__ballot(x[4 * k + j] == prefix) & below);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t y = x[4 * k + j];
                    const bool stays = all_ties ? y >= prefix : y > prefix || (y == prefix && t + before < left);
                    kept |= (Bits)(stays ? 1u : 0u) << (4 * k + j);
                    before += y == prefix;
                }
                if (!all_ties) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) t += __popcll(__ballot(x[4 * k + j] == prefix));
                }
            }
            f(k0, kept, under);
        });
    };
    uint32_t holes = 0, movers = 0;
    Bits kept0 = 0, under0 = 0;
    sort_out([&](int, Bits kept, Bits under) {
        if constexpr (KPT <= 32) {
            holes += __popc(under & ~kept);
            movers += __popc(kept & ~under);
        } else {
            holes += __popcll(under & ~kept);
            movers += __popcll(kept & ~under);
        }
        kept0 = kept;
        under0 = under;
    });
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        holes += __shfl_xor(holes, o);
        movers += __shfl_xor(movers, o);
    }
    if (lane == 0) {
        sh.a[wave] = holes;
        sh.b[wave] = movers;
    }
    __syncthreads();
    uint32_t hole0 = 0, mover0 = 0, total = 0;
    for (int w = 0; w < kSelWaves; ++w) {
        if (w < wave) {
            hole0 += sh.a[w];
            mover0 += sh.b[w];
        }
        total += sh.a[w];
    }
    if (tid == 0) sh.count = total;
    int32_t* dst = A.moves + (size_t)A.batch * A.Hk + (size_t)item * 2 * A.moves_stride;
    int32_t* src = dst + A.moves_stride;
    float* sco = A.scores_out + base;
    int32_t* odo = A.order_out + base;
    const bool copies = sco != sc || odo != od;
    // the slots i + j of bits j, behind those of lower lanes and earlier runs
    auto list = [&](int32_t* to, uint32_t& at, uint32_t bits, int i) {
        if (!__ballot(bits)) return;
        uint32_t before = at;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const unsigned long long m = __ballot(bits >> j & 1);
            before += __popcll(m & below);
            at += __popcll(m);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (bits >> j & 1) to[before++] = i + j;
    };
    auto put = [&](int k0, Bits kept, Bits under) {
        // weights and numbers of the slots that stay where they are
        if (copies && __ballot(kept & under))
            runs(k0, [&](int k, f4u f, i4u o, int) {
                const int i = i0 + (k0 + k) * 256;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if ((kept & under) >> (4 * k + j) & 1) {
                        sco[i + j] = f[j];
                        odo[i + j] = o[j];
                    }
            });
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            const int i = i0 + (k0 + k) * 256;
            list(dst, hole0, (uint32_t)((under & ~kept) >> (4 * k)) & 15u, i);
            list(src, mover0, (uint32_t)((kept & ~under) >> (4 * k)) & 15u, i);
        }
    };
    if (MEM) sort_out(put);
    else put(0, kept0, under0);
}

template <int KPT>
__global__ void __launch_bounds__(kSelThreads) k_kv_evict_select(const EvictArgs A) {
    __shared__ SelectShared sh;
    const int item = blockIdx.x, b = item / A.Hk, h = item - b * A.Hk, tid = threadIdx.x;
    int n = A.lens[b];
    if (n < 0 || n > A.cap) {
        if (tid == 0 && h == 0) atomicAdd(A.bad, 1);
        n = n < 0 ? 0 : A.cap;
    }
    if (A.moves_too && h == 0 && tid == 0) A.lens_out[b] = min(n, A.budget);
    if (n <= A.budget) {
        const size_t base = (size_t)item * A.cap;
        const bool copies = A.scores_out != A.scores || A.order_out != A.order;
        for (int i = tid; copies && i < n; i += kSelThreads) {
            A.scores_out[base + i] = A.scores[base + i];
            A.order_out[base + i] = A.order[base + i];
        }
        if (tid == 0) A.moves[item] = 0;
        return;
    }
    if (n == A.budget + 1) evict_one(A, sh, item, b, n);
    else if (n <= (KPT < 32 ? KPT : 32) * kSelThreads) evict_select<(KPT < 32 ? KPT : 32), false>(A, sh, item, b, n);
    else if constexpr (KPT == 64) {
        if (n <= KPT * kSelThreads) evict_select<KPT, false>(A, sh, item, b, n);
        else evict_select<32, true>(A, sh, item, b, n);
    }
    __syncthreads();
    if (!A.moves_too) {
        if (tid == 0) A.moves[item] = (int32_t)sh.count;
        return;
    }
    const int32_t* dst = A.moves + (size_t)A.batch * A.Hk + (size_t)item * 2 * A.moves_stride;
    const int32_t* src = dst + A.moves_stride;
    for (int m = (tid >> 4) * kMoveRows; m < (int)sh.count; m += kSelThreads / 16 * kMoveRows)
        move_rows(A, item, b, h, dst + m, src + m, (int)sh.count - m, tid & 15);
}

// 64 rows of both keys and values a workgroup. Bound by their traffic.
__global__ void __launch_bounds__(256) k_kv_evict_move(const EvictArgs A) {
    const int item = blockIdx.y, b = item / A.Hk, h = item - b * A.Hk;
    const int count = A.moves[item];
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) {
        const int n = A.lens[b];
        A.lens_out[b] = n < 0 ? 0 : min(min(n, A.cap), A.budget);
    }
    const int32_t* dst = A.moves + (size_t)A.batch * A.Hk + (size_t)item * 2 * A.moves_stride;
    const int32_t* src = dst + A.moves_stride;
    for (int m = (blockIdx.x * 16 + (threadIdx.x >> 4)) * kMoveRows; m < count; m += gridDim.x * 16 * kMoveRows)
        move_rows(A, item, b, h, dst + m, src + m, count - m, threadIdx.x & 15);
}

__global__ void k_kv_take_bad(int32_t* bad, int32_t* out) { *out = atomicExch(bad, 0); }

int check_cache(const dq_kv_ctx* c, const int32_t* table, const void* k, const void* v, const float* ks,
                const float* vs) {
    if (!table || !k || !v) DQ_FAIL(DQ_ERR_ARG, "block_table, k_cache and v_cache must not be NULL");
    if ((c->cache_type == DQ_I8) != (ks != nullptr) || (c->cache_type == DQ_I8) != (vs != nullptr))
        DQ_FAIL(DQ_ERR_ARG, "an int8 cache has k_scale and v_scale, another has neither");
    if ((uintptr_t)k % 16 || (uintptr_t)v % 16) DQ_FAIL(DQ_ERR_ARG, "k_cache and v_cache must be 16-byte aligned");
    if ((uintptr_t)table % 4 || (uintptr_t)ks % 4 || (uintptr_t)vs % 4)
        DQ_FAIL(DQ_ERR_ARG, "a tensor is not aligned to its elements");
    return dq_kv_check_device(c);
}

// pairs a lane takes at a time: 4 where the vectors of four pairs are aligned
// and none straddles the end of the rotated part, else 1
template <int TI, int TC>
void launch_append(const AppendArgs& A, int vp, bool il, hipStream_t s) {
    const dim3 grid((A.groups + 15) / 16), block(256);
    // the angles of the tokens that sixteen groups can touch
    const size_t lds = A.pos ? (size_t)(14 / A.chunks.d + 2) * (A.R / 2) * sizeof(float2) : 0;
#define DQ_APPEND(VP_, IL_) hipLaunchKernelGGL((k_kv_append<TI, TC, VP_, IL_>), grid, block, lds, s, A)
    if (vp == 4) {
        if constexpr (sizeof(typename Elem<TI>::S) == 2) {
            if (il) {
                DQ_APPEND(4, true);
                return;
            }
        }
        DQ_APPEND(4, false);
    } else if (il) {
        DQ_APPEND(1, true);
    } else {
        DQ_APPEND(1, false);
    }
#undef DQ_APPEND
}

template <int TI>
void launch_append_cache(dq_dtype tc, const AppendArgs& A, int vp, bool il, hipStream_t s) {
    if (tc == DQ_I8) launch_append<TI, DQ_I8>(A, vp, il, s);
    else if (tc == DQ_BF16) launch_append<TI, DQ_BF16>(A, vp, il, s);
    else launch_append<TI, DQ_F16>(A, vp, il, s);
}

template <int TO>
void launch_read(dq_dtype tc, const ReadArgs& A, hipStream_t s) {
    const dim3 grid((A.threads + 255) / 256), block(256);
    if (tc == DQ_I8) hipLaunchKernelGGL((k_kv_read<TO, DQ_I8>), grid, block, 0, s, A);
    else if (tc == DQ_BF16) hipLaunchKernelGGL((k_kv_read<TO, DQ_BF16>), grid, block, 0, s, A);
    else hipLaunchKernelGGL((k_kv_read<TO, DQ_F16>), grid, block, 0, s, A);
}

}  // namespace

int dq_kv_check_device(const dq_kv_ctx* c) {
    int dev = 0;
    (void)hipGetDevice(&dev);
    if (dev != c->device) DQ_FAIL(DQ_ERR_STATE, "the context belongs to another device");
    return DQ_OK;
}

extern "C" int dq_kv_init(dq_kv_ctx** ctx, int batch, int q_heads, int kv_heads, int head_dim, int pages,
                          int page_size, int pages_per_seq, dq_dtype q_type, dq_dtype cache_type, int gather_scores) {
    if (!ctx) DQ_FAIL(DQ_ERR_ARG, "ctx is NULL");
    *ctx = nullptr;
    if (batch < 1 || q_heads < 1 || kv_heads < 1 || pages < 1 || page_size < 1 || pages_per_seq < 1)
        DQ_FAIL(DQ_ERR_ARG, "sizes must be >= 1");
    if (q_heads % kv_heads) DQ_FAIL(DQ_ERR_ARG, "q_heads must be a multiple of kv_heads");
    if (head_dim < 16 || head_dim % 16) DQ_FAIL(DQ_ERR_ARG, "head_dim must be a positive multiple of 16");
    if (q_type != DQ_F32 && q_type != DQ_BF16 && q_type != DQ_F16)
        DQ_FAIL(DQ_ERR_TYPE, "queries must be fp32, bf16 or fp16");
    if (cache_type != DQ_BF16 && cache_type != DQ_F16 && cache_type != DQ_I8)
        DQ_FAIL(DQ_ERR_TYPE, "the cache must be bf16, fp16 or int8");
    if (head_dim > DQ_KV_DIM_MAX) DQ_FAIL(DQ_ERR_RANGE, "head_dim exceeds %d", DQ_KV_DIM_MAX);
    if (batch > DQ_KV_BATCH_MAX) DQ_FAIL(DQ_ERR_RANGE, "batch exceeds %d", DQ_KV_BATCH_MAX);
    if ((int64_t)batch * kv_heads > 65535 || (int64_t)batch * q_heads > (1 << 24))
        DQ_FAIL(DQ_ERR_RANGE, "batch * kv_heads exceeds 65535 or batch * q_heads 2^24");
    if ((int64_t)pages_per_seq * page_size > (1 << 30))
        DQ_FAIL(DQ_ERR_RANGE, "pages_per_seq * page_size exceeds 2^30 tokens");
    if ((__int128)pages * kv_heads * page_size > INT32_MAX)
        DQ_FAIL(DQ_ERR_RANGE, "pages * kv_heads * page_size exceeds 2^31 - 1 rows");
    if (gather_scores && ((int64_t)pages_per_seq * page_size + 127) / 128 * 128 * (q_heads / kv_heads) > INT32_MAX / 4 - 64)
        DQ_FAIL(DQ_ERR_RANGE, "pages_per_seq * page_size * (q_heads / kv_heads) scores exceed 2^31 bytes");
    dq_kv_ctx* c = new (std::nothrow) dq_kv_ctx();
    if (!c) DQ_FAIL(DQ_ERR_ALLOC, "host allocation for the cache context failed");
    (void)hipGetDevice(&c->device);
    c->batch = batch;
    c->Hq = q_heads;
    c->Hk = kv_heads;
    c->D = head_dim;
    c->pages = pages;
    c->page_size = page_size;
    c->per_seq = pages_per_seq;
    c->cap = pages_per_seq * page_size;
    c->q_type = q_type;
    c->cache_type = cache_type;
    c->scores = gather_scores != 0;
    c->geom.page = make_kvdiv((uint32_t)page_size);
    c->geom.pages = pages;
    c->geom.per_seq = pages_per_seq;
    c->geom.heads = kv_heads;
    if (hipDeviceGetAttribute(&c->cus, hipDeviceAttributeMultiprocessorCount, c->device) != hipSuccess || c->cus < 1)
        c->cus = 256;
    // a head's moves: at most half its slots come free and as many fill them
    c->moves_stride = (size_t)c->cap / 2 + 1;
    const size_t moves = (size_t)batch * kv_heads * (1 + 2 * c->moves_stride);
    if (int rc = dq_attend_plan(c)) {
        dq_kv_release(c);
        return rc;
    }
    if (c->scores) c->s_stride = ((size_t)c->cap + 127) / 128 * 128 * (q_heads / kv_heads);
    bool ok = hipMalloc(&c->bad, 8) == hipSuccess && hipMalloc(&c->moves, moves * 4) == hipSuccess &&
              hipMalloc(&c->part, c->part_floats * 4) == hipSuccess &&
              (!c->scores || hipMalloc(&c->s, (size_t)batch * kv_heads * c->s_stride * 4) == hipSuccess);
    if (!ok) {
        dq_kv_release(c);
        DQ_FAIL(DQ_ERR_ALLOC, "device allocation for the cache context failed");
    }
    if (hipMemset(c->bad, 0, 8) != hipSuccess) {
        dq_kv_release(c);
        DQ_FAIL(DQ_ERR_HIP, "clearing the cache context failed");
    }
    const char* names[] = {"fp32", "bf16", "int8", "uint8", "fp16"};
    snprintf(c->info, sizeof c->info, "gfx950 paged cache: %d sequences, %d query and %d key-value heads of %d, %d pages "
             "of %d, %s queries, %s cache", batch, q_heads, kv_heads, head_dim, pages, page_size, names[q_type],
             names[cache_type]);
    *ctx = c;
    return DQ_OK;
}

extern "C" int dq_kv_append(dq_kv_ctx* ctx, int64_t tokens, const void* k, int64_t k_token_stride,
                            int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride,
                            const int32_t* index, const int32_t* seq_ids, const int32_t* block_table, void* k_cache,
                            void* v_cache, float* k_scale, float* v_scale, const void* q, int64_t q_token_stride,
                            int64_t q_head_stride, void* q_out, const dq_rope_ctx* rope, const int32_t* positions,
                            void* stream) {
    if (!ctx) DQ_FAIL(DQ_ERR_STATE, "no context");
    if (tokens < 0) DQ_FAIL(DQ_ERR_ARG, "tokens must be >= 0");
    if (tokens == 0) return DQ_OK;
    if (!k || !v || !index) DQ_FAIL(DQ_ERR_ARG, "k, v and index must not be NULL");
    if ((q != nullptr) != (q_out != nullptr)) DQ_FAIL(DQ_ERR_ARG, "q and q_out go together");
    if ((rope != nullptr) != (positions != nullptr)) DQ_FAIL(DQ_ERR_ARG, "rope and positions go together");
    if (!seq_ids && tokens > ctx->batch) DQ_FAIL(DQ_ERR_ARG, "more tokens than sequences need seq_ids");
    if (rope && rope->D != ctx->D) DQ_FAIL(DQ_ERR_ARG, "the rotary context's head_dim is not the cache's");
    const size_t es = kv_elem_bytes(ctx->q_type);
    if ((uintptr_t)k % es || (uintptr_t)v % es || (uintptr_t)q % es || (uintptr_t)q_out % es ||
        (uintptr_t)index % 4 || (uintptr_t)seq_ids % 4 || (uintptr_t)positions % 4)
        DQ_FAIL(DQ_ERR_ARG, "a tensor is not aligned to its elements");
    if (q && q == q_out && (q_head_stride != ctx->D || q_token_stride != (int64_t)ctx->Hq * ctx->D))
        DQ_FAIL(DQ_ERR_ARG, "q_out is dense: in place q has to be dense too");
    if (int rc = check_cache(ctx, block_table, k_cache, v_cache, k_scale, v_scale)) return rc;
    if (rope)
        if (int rc = dq_rope_check_device(rope)) return rc;
    if (tokens > INT32_MAX / 16) DQ_FAIL(DQ_ERR_RANGE, "too many tokens for one launch");
    AppendArgs A{};
    A.q = q;
    A.k = k;
    A.v = v;
    A.q_out = q_out;
    A.qt = q_token_stride;
    A.qh = q_head_stride;
    A.kt = k_token_stride;
    A.kh = k_head_stride;
    A.vt = v_token_stride;
    A.vh = v_head_stride;
    A.index = index;
    A.seq_ids = seq_ids;
    A.table = block_table;
    A.kc = k_cache;
    A.vc = v_cache;
    A.ks = k_scale;
    A.vs = v_scale;
    A.bad = ctx->bad;
    A.pos = positions;
    A.freq = rope ? rope->freq : nullptr;
    A.axis = rope ? rope->axis : nullptr;
    A.tokens = (int)tokens;
    A.batch = ctx->batch;
    A.Hq = q ? ctx->Hq : 0;
    A.Hk = ctx->Hk;
    A.D = ctx->D;
    A.R = rope ? rope->R : ctx->D;
    A.geom = ctx->geom;
    // rows per group: as many as leave the chip filled (2^14 groups), at most 4
    // (6001 tokens of 32 + 16 heads of 128 in bf16: 27.3 us when chosen, with 8 30.8)
    const int64_t rows = A.Hq + 2 * (int64_t)A.Hk;
    int chunk = 1;
    while (chunk < 4 && tokens * (rows / (2 * chunk)) >= (1 << 14)) chunk *= 2;
    A.chunk = chunk;
    const int64_t chunks = (rows + chunk - 1) / chunk;
    A.chunks = make_kvdiv((uint32_t)chunks);
    A.groups = (uint32_t)(tokens * chunks);
    if (tokens * chunks > INT32_MAX) DQ_FAIL(DQ_ERR_RANGE, "too many tokens for one launch");
    const bool il = rope && rope->interleaved;
    const size_t bytes = (il ? 8 : 4) * es;
    bool wide = A.R / 2 % 4 == 0 && bytes <= 16 && (uintptr_t)k % bytes == 0 && (uintptr_t)v % bytes == 0 &&
                (uintptr_t)q % bytes == 0 && (uintptr_t)q_out % bytes == 0;
    const long long st[6] = {A.qt, A.qh, A.kt, A.kh, A.vt, A.vh};
    for (int i = q ? 0 : 2; i < 6; ++i) wide = wide && st[i] % (il ? 8 : 4) == 0;
    const hipStream_t s = (hipStream_t)stream;
    const int vp = wide ? 4 : 1;
    if (ctx->q_type == DQ_F32) launch_append_cache<DQ_F32>(ctx->cache_type, A, vp, il, s);
    else if (ctx->q_type == DQ_BF16) launch_append_cache<DQ_BF16>(ctx->cache_type, A, vp, il, s);
    else launch_append_cache<DQ_F16>(ctx->cache_type, A, vp, il, s);
    DQ_LAUNCH_CHECK("cache append");
    return DQ_OK;
}

extern "C" int dq_kv_read(dq_kv_ctx* ctx, int64_t tokens, const int32_t* index, const int32_t* seq_ids,
                          const int32_t* block_table, const void* k_cache, const void* v_cache, const float* k_scale,
                          const float* v_scale, void* k_out, void* v_out, void* stream) {
    if (!ctx) DQ_FAIL(DQ_ERR_STATE, "no context");
    if (tokens < 0) DQ_FAIL(DQ_ERR_ARG, "tokens must be >= 0");
    if (tokens == 0) return DQ_OK;
    if (!index || (!k_out && !v_out)) DQ_FAIL(DQ_ERR_ARG, "index and one of k_out and v_out must not be NULL");
    if (!seq_ids && tokens > ctx->batch) DQ_FAIL(DQ_ERR_ARG, "more tokens than sequences need seq_ids");
    if ((uintptr_t)k_out % 16 || (uintptr_t)v_out % 16) DQ_FAIL(DQ_ERR_ARG, "k_out and v_out must be 16-byte aligned");
    if ((uintptr_t)index % 4 || (uintptr_t)seq_ids % 4)
        DQ_FAIL(DQ_ERR_ARG, "a tensor is not aligned to its elements");
    if (int rc = check_cache(ctx, block_table, k_cache, v_cache, k_scale, v_scale)) return rc;
    const int64_t pieces = ctx->D / 8;
    if (tokens > INT32_MAX || tokens * ctx->Hk > INT32_MAX || tokens * ctx->Hk * pieces > (int64_t)UINT32_MAX - 256)
        DQ_FAIL(DQ_ERR_RANGE, "too many tokens for one launch");
    ReadArgs A{};
    A.index = index;
    A.seq_ids = seq_ids;
    A.table = block_table;
    A.kc = k_cache;
    A.vc = v_cache;
    A.ks = k_scale;
    A.vs = v_scale;
    A.k_out = k_out;
    A.v_out = v_out;
    A.bad = ctx->bad;
    A.threads = (uint32_t)(tokens * ctx->Hk * pieces);
    A.Hk = ctx->Hk;
    A.D = ctx->D;
    A.batch = ctx->batch;
    A.pieces = make_kvdiv((uint32_t)pieces);
    A.heads = make_kvdiv((uint32_t)ctx->Hk);
    A.geom = ctx->geom;
    const hipStream_t s = (hipStream_t)stream;
    if (ctx->q_type == DQ_F32) launch_read<DQ_F32>(ctx->cache_type, A, s);
    else if (ctx->q_type == DQ_BF16) launch_read<DQ_BF16>(ctx->cache_type, A, s);
    else launch_read<DQ_F16>(ctx->cache_type, A, s);
    DQ_LAUNCH_CHECK("cache read");
    return DQ_OK;
}

extern "C" int dq_kv_attend(dq_kv_ctx* ctx, int batch, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                            const int32_t* lens, const int32_t* block_table, const void* k_cache, const void* v_cache,
                            const float* k_scale, const float* v_scale, void* out, float sm_scale, float* lse,
                            int window, const float* scores, float* scores_out, float decay, void* stream) {
    if (!ctx) DQ_FAIL(DQ_ERR_STATE, "no context");
    if (batch < 0 || batch > ctx->batch) DQ_FAIL(DQ_ERR_ARG, "batch must lie in [0, %d]", ctx->batch);
    if (batch == 0) return DQ_OK;
    if (!q || !lens || !out) DQ_FAIL(DQ_ERR_ARG, "q, lens and out must not be NULL");
    if (window < 0) DQ_FAIL(DQ_ERR_ARG, "window must be >= 0 (0: none)");
    if (!isfinite(sm_scale)) DQ_FAIL(DQ_ERR_ARG, "sm_scale must be finite");
    if ((scores != nullptr) != (scores_out != nullptr)) DQ_FAIL(DQ_ERR_ARG, "scores and scores_out go together");
    if (scores && !ctx->scores) DQ_FAIL(DQ_ERR_STATE, "the context was made without gather_scores");
    const size_t es = kv_elem_bytes(ctx->q_type);
    if ((uintptr_t)q % es || (uintptr_t)lens % 4 || (uintptr_t)lse % 4 || (uintptr_t)scores % 4 ||
        (uintptr_t)scores_out % 4)
        DQ_FAIL(DQ_ERR_ARG, "a tensor is not aligned to its elements");
    if ((uintptr_t)out % 16) DQ_FAIL(DQ_ERR_ARG, "out must be 16-byte aligned");
    if (int rc = check_cache(ctx, block_table, k_cache, v_cache, k_scale, v_scale)) return rc;
    const DqAttendArgs A{q,   q_token_stride, q_head_stride, lens,   block_table, k_cache,    v_cache, k_scale, v_scale,
                         out, lse,            batch,         sm_scale, window,    scores, scores_out, decay};
    return dq_launch_attend(ctx, A, (hipStream_t)stream);
}

extern "C" int dq_kv_evict(dq_kv_ctx* ctx, int batch, int budget, int recent, int sinks, const int32_t* lens,
                           const int32_t* newest, const float* scores, const int32_t* order,
                           const int32_t* block_table, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                           float* scores_out, int32_t* order_out, int32_t* lens_out, void* stream) {
    if (!ctx) DQ_FAIL(DQ_ERR_STATE, "no context");
    if (batch < 0 || batch > ctx->batch) DQ_FAIL(DQ_ERR_ARG, "batch must lie in [0, %d]", ctx->batch);
    if (budget < 1 || recent < 0 || sinks < 0) DQ_FAIL(DQ_ERR_ARG, "budget must be >= 1, recent and sinks >= 0");
    if (batch == 0) return DQ_OK;
    if (!lens || !newest || !scores || !order || !scores_out || !order_out || !lens_out)
        DQ_FAIL(DQ_ERR_ARG, "lens, newest, scores, order and their outputs must not be NULL");
    if ((uintptr_t)lens % 4 || (uintptr_t)newest % 4 || (uintptr_t)scores % 4 || (uintptr_t)order % 4 ||
        (uintptr_t)scores_out % 4 || (uintptr_t)order_out % 4 || (uintptr_t)lens_out % 4)
        DQ_FAIL(DQ_ERR_ARG, "a tensor is not aligned to its elements");
    if (int rc = check_cache(ctx, block_table, k_cache, v_cache, k_scale, v_scale)) return rc;
    EvictArgs A{};
    A.lens = lens;
    A.newest = newest;
    A.scores = scores;
    A.order = order;
    A.table = block_table;
    A.kc = k_cache;
    A.vc = v_cache;
    A.ks = k_scale;
    A.vs = v_scale;
    A.scores_out = scores_out;
    A.order_out = order_out;
    A.lens_out = lens_out;
    A.moves = ctx->moves;
    A.moves_stride = ctx->moves_stride;
    A.bad = ctx->bad;
    A.batch = batch;
    A.Hk = ctx->Hk;
    A.cap = ctx->cap;
    A.budget = budget;
    A.sinks = sinks;
    A.recent = recent;
    A.row_bytes = ctx->D * (int)kv_elem_bytes(ctx->cache_type);
    A.geom = ctx->geom;
    const hipStream_t s = (hipStream_t)stream;
    const int items = batch * ctx->Hk;
    // the most rows of a head that can move. A workgroup moves 64 by itself in
    // less than a second launch takes (one over 1024, 128 heads, replayed from
    // a graph: 6.3 us, with the launch 8.7); lens_out is then written while other
    // heads still read lens, so not where they are one tensor
    const int most = std::max(0, std::min(budget, ctx->cap - budget));
    A.moves_too = most <= 64 && lens_out != lens;
    const dim3 grid((unsigned)items), block(kSelThreads);
    if (ctx->cap <= 4 * kSelThreads) hipLaunchKernelGGL((k_kv_evict_select<4>), grid, block, 0, s, A);
    else if (ctx->cap <= 8 * kSelThreads) hipLaunchKernelGGL((k_kv_evict_select<8>), grid, block, 0, s, A);
    else if (ctx->cap <= 32 * kSelThreads) hipLaunchKernelGGL((k_kv_evict_select<32>), grid, block, 0, s, A);
    else hipLaunchKernelGGL((k_kv_evict_select<64>), grid, block, 0, s, A);
    DQ_LAUNCH_CHECK("eviction's selection");
    if (!A.moves_too) {
        // workgroups for the most rows that can move, at most 2^14 in all
        const int gx = std::max(1, std::min((most + 63) / 64, (1 << 14) / items));
        hipLaunchKernelGGL(k_kv_evict_move, dim3((unsigned)gx, (unsigned)items), dim3(256), 0, s, A);
        DQ_LAUNCH_CHECK("eviction's moves");
    }
    return DQ_OK;
}

extern "C" int dq_kv_take_errors(dq_kv_ctx* ctx, int* count, void* stream) {
    if (!ctx) DQ_FAIL(DQ_ERR_STATE, "no context");
    if (!count) DQ_FAIL(DQ_ERR_ARG, "count must not be NULL");
    if (int rc = dq_kv_check_device(ctx)) return rc;
    const hipStream_t s = (hipStream_t)stream;
    hipLaunchKernelGGL(k_kv_take_bad, dim3(1), dim3(1), 0, s, ctx->bad, ctx->bad + 1);
    DQ_LAUNCH_CHECK("cache error count");
    DQ_HIP_CHECK(hipMemcpyAsync(count, ctx->bad + 1, 4, hipMemcpyDeviceToHost, s));
    DQ_HIP_CHECK(hipStreamSynchronize(s));
    return DQ_OK;
}

extern "C" const char* dq_kv_info(const dq_kv_ctx* ctx) { return ctx ? ctx->info : nullptr; }

extern "C" void dq_kv_release(dq_kv_ctx* ctx) {
    if (!ctx) return;
    (void)hipFree(ctx->bad);
    (void)hipFree(ctx->moves);
    (void)hipFree(ctx->part);
    (void)hipFree(ctx->s);
    delete ctx;
}
