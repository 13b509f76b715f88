// moe.hip -- the router that sends tokens to experts, and the sum of the
// experts' results.
//
//   ids[t, j]   the j-th largest of a token's logits (ties: the lowest expert)
//   weights     softmax over all of the token's logits or sigmoid, of the chosen
//   rows        the pairs (t, j) in the order of the expert, then of the token
//   out[t] = add[t] + sum_j weights[t, j] y[row_of[t, j]]
#include "dq_device.h"

#include <algorithm>
#include <new>
#include <stdio.h>

struct dq_moe_ctx {
    int device = 0;
    int64_t max_tokens = 0;
    int experts = 0, top_k = 0, scoring = 0, normalize = 0;
    dq_dtype logits_type = DQ_F32;
    float scale = 1.0f;
    uint8_t* counts = nullptr;    // the router's workspace (RouteArgs)
    int32_t* before = nullptr;
    int32_t* totals = nullptr;
    char info[192] = "";
};

namespace {

using namespace dq;

constexpr int kChunk = 64;         // tokens that one workgroup chooses for: a bit each of a 64-bit mask
constexpr int kPlace = 4;          // chunks whose rows one workgroup places
constexpr int kScanChunks = 256;   // more chunks are summed by a launch of their own

struct RouteArgs {
    const void* logits;
    long long stride;
    int32_t* ids;
    float* weights;
    int32_t* offsets;
    int32_t* row_token;
    int32_t* row_of;
    uint8_t* counts;   // [chunks][words * 4]: rows of each expert in a chunk
    int32_t* before;   // [chunks][words * 4]: its rows in earlier chunks
    int32_t* totals;   // [words * 4]
    int tokens, experts, top_k, chunks, words, type, sigmoid, normalize;
    int vec;  // a lane's neighbouring logits can be loaded at once
    float scale;
};

__device__ __forceinline__ float load1(const void* p, size_t i, int type) {
    if (type == DQ_F32) return static_cast<const float*>(p)[i];
    const uint16_t b = static_cast<const uint16_t*>(p)[i];
    return type == DQ_BF16 ? bf16_bits_to_f32(b) : (float)__builtin_bit_cast(_Float16, b);
}

// A logit and its expert as one number that compares as the order of choice
// does: a double in [1, 2) whose mantissa is the logit's ordered bits, then
// 1023 - expert. One v_max_f64 and one v_min_f64 compare and exchange two of them.
// 1.0 itself is none: a logit of -infinity or NaN.
typedef unsigned long long u64;
constexpr u64 kNoKey = 0x3ff0000000000000ull;
__device__ __forceinline__ u64 route_key(float l, int e) {
    if (!(l > -__builtin_inff())) return kNoKey;
    return kNoKey | (u64)f2ord(l) << 20 | (u64)(1023 - e) << 10;
}
__device__ __forceinline__ float key_logit(u64 k) { return ord2f((uint32_t)(k >> 20)); }
__device__ __forceinline__ int key_expert(u64 k) { return 1023 - ((int)(k >> 10) & 1023); }
__device__ __forceinline__ u64 key_max(u64 a, u64 b) {
    u64 r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ u64 key_min(u64 a, u64 b) {
    u64 r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
template <int CTRL>
__device__ __forceinline__ u64 key_dpp(u64 k) {
    const int lo = __builtin_amdgcn_update_dpp(0, (int)k, CTRL, 0xF, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(k >> 32), CTRL, 0xF, 0xF, false);
    return (u64)(uint32_t)hi << 32 | (uint32_t)lo;
}

// Over the L lanes of a token (16, 32 or 64), in all of them.
template <int L>
__device__ __forceinline__ u64 token_max(u64 k) {
    k = key_max(k, key_dpp<kDppXor1>(k));
    k = key_max(k, key_dpp<kDppXor2>(k));
    k = key_max(k, key_dpp<kDppRowHalfMirror>(k));
    k = key_max(k, key_dpp<kDppRowMirror>(k));
    for (int o = 16; o < L; o *= 2) k = key_max(k, __shfl_xor(k, o));
    return k;
}
template <int L>
__device__ __forceinline__ float token_sum(float v) {
    v += dpp_f<kDppXor1>(v);
    v += dpp_f<kDppXor2>(v);
    v += dpp_f<kDppRowHalfMirror>(v);
    v += dpp_f<kDppRowMirror>(v);
    for (int o = 16; o < L; o *= 2) v += __shfl_xor(v, o);
    return v;
}

// The experts' first rows: an exclusive prefix sum over totals s_total[0, E), by
// 1024 threads, left in s_first[0, E].
__device__ __forceinline__ void first_rows(const int* s_total, int* s_first, int* s_wave, int E) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = (int)threadIdx.x < E ? s_total[threadIdx.x] : 0;
    int upto = n;
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 63) s_wave[wave] = upto;
    __syncthreads();
    for (int w = 0; w < wave; ++w) upto += s_wave[w];
    if ((int)threadIdx.x < E) s_first[threadIdx.x + 1] = upto;
    if (threadIdx.x == 0) s_first[0] = 0;
    __syncthreads();
}

// The choice for a chunk of tokens. L lanes take a token, each V of its logits
// as sorted keys; every round takes the largest first key among the lanes and
// out of its lane. Bound by these rounds' dependent steps (four moves across lanes
// and maxima, then the shift): 16001 tokens of 256 experts in bf16, top 8, 8.3 us,
// of which the 8 MB of logits would take 1.3. With a wave a token, a maximum and
// its index as two values each, it was most of 257 us together with one
// workgroup's sums. A chunk's ranks come from a 64-bit mask of tokens for each
// expert, so they do not depend on the order of the atomics. One chunk alone is
// finished here: 8 tokens of 64 experts take one launch of 4.9 us, not two.
// V: logits of a lane; KEEP: how many of them, sorted, the rounds can need.
template <int V, int KEEP, int L>
__global__ void __launch_bounds__(1024) k_moe_choose(RouteArgs A) {
    __shared__ u64 s_mask[DQ_MOE_EXPERTS_MAX];
    __shared__ int s_total[DQ_MOE_EXPERTS_MAX], s_first[DQ_MOE_EXPERTS_MAX + 1], s_wave[16];
    constexpr int kAtOnce = 1024 / L;          // tokens of the workgroup
    constexpr int kSlots = L == 16 ? 2 : 1;    // choices that a lane keeps
    constexpr int kTurns = kChunk / kAtOnce > 0 ? kChunk / kAtOnce : 1;
    const int l = threadIdx.x % L;
    for (int e = threadIdx.x; e < A.words * 4; e += 1024) s_mask[e] = 0;
    __syncthreads();
    int id[kTurns][kSlots];
#pragma unroll
    for (int turn = 0; turn < kTurns; ++turn) {
        const int in = turn * kAtOnce + threadIdx.x / L;
        const long long t = (long long)blockIdx.x * kChunk + in;
        const bool some = t < A.tokens;
        const long long at = (some ? t : A.tokens - 1) * A.stride;
        u64 key[V];
        bool nan = false;
        auto take = [&](int i, int e, float v) {
            key[i] = e < A.experts ? route_key(v, e) : kNoKey;
            nan |= e < A.experts && v != v;
        };
        // which lane has which logit does not matter: a key carries its expert
        if (A.vec && A.type == DQ_F32) {
            constexpr int W = V < 4 ? V : 4;
            typedef float fw __attribute__((ext_vector_type(W)));
#pragma unroll
            for (int i = 0; i < V; i += W) {
                const int e = i * L + l * W;
                const fw v = *reinterpret_cast<const fw*>(static_cast<const float*>(A.logits) + at + min(e, A.experts - W));
#pragma unroll
                for (int k = 0; k < W; ++k) take(i + k, e + k, v[k]);
            }
        } else if (A.vec) {
            constexpr int W = V < 8 ? V : 8;
            typedef uint16_t hw __attribute__((ext_vector_type(W)));
#pragma unroll
            for (int i = 0; i < V; i += W) {
                const int e = i * L + l * W;
                const hw v = *reinterpret_cast<const hw*>(static_cast<const uint16_t*>(A.logits) + at + min(e, A.experts - W));
#pragma unroll
                for (int k = 0; k < W; ++k)
                    take(i + k, e + k, A.type == DQ_BF16 ? bf16_bits_to_f32(v[k]) : (float)__builtin_bit_cast(_Float16, (uint16_t)v[k]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = i * L + l;
                take(i, e, load1(A.logits, at + min(e, A.experts - 1), A.type));
            }
        }
        // Batcher's odd-even merge sort, falling
#pragma unroll
        for (int p = 1; p < V; p *= 2)
#pragma unroll
            for (int k = p; k >= 1; k /= 2)
#pragma unroll
                for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
                    for (int i = 0; i < k; ++i)
                        if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                            const u64 a = key[i + j], b = key[i + j + k];
                            key[i + j] = key_max(a, b);
                            key[i + j + k] = key_min(a, b);
                        }
        u64 won[kSlots];
#pragma unroll
        for (int s = 0; s < kSlots; ++s) won[s] = kNoKey;
        float high = 0.0f;
        for (int j = 0; j < A.top_k; ++j) {
            const u64 best = token_max<L>(key[0]);
            if (j == 0 && best != kNoKey) high = key_logit(best);
#pragma unroll
            for (int s = 0; s < kSlots; ++s)
                if (l + s * L == j) won[s] = best;
            if (key[0] == best) {
#pragma unroll
                for (int i = 0; i + 1 < KEEP; ++i) key[i] = key[i + 1];
                key[KEEP - 1] = kNoKey;
            }
        }
        float part[kSlots], sum = 0.0f;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            id[turn][s] = won[s] == kNoKey ? -1 : key_expert(won[s]);
            const float v = key_logit(won[s]);
            part[s] = won[s] == kNoKey ? 0.0f : A.sigmoid ? 1.0f / (1.0f + expf(-v)) : expf(v - high);
            sum += part[s];
        }
        float total = 1.0f;
        if (A.normalize) {
            total = token_sum<L>(sum);
        } else if (!A.sigmoid) {
            total = 0.0f;
            for (int e = l; e < A.experts; e += L) total += expf(load1(A.logits, at + e, A.type) - high);
            total = token_sum<L>(total);
        }
        if (!A.sigmoid && A.normalize && token_sum<L>(nan ? 1.0f : 0.0f) > 0.0f) total = __builtin_nanf("");
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            const int j = l + s * L;
            if (!some || j >= A.top_k) id[turn][s] = -1;
            if (some && j < A.top_k) {
                A.ids[t * A.top_k + j] = id[turn][s];
                A.weights[t * A.top_k + j] = id[turn][s] < 0 ? 0.0f : part[s] / total * A.scale;
                if (id[turn][s] >= 0) atomicOr(&s_mask[id[turn][s]], 1ull << in);
                else A.row_of[t * A.top_k + j] = -1;
            }
        }
    }
    __syncthreads();
    const bool whole = A.chunks == 1;
    if (whole) {
        if ((int)threadIdx.x < A.experts) s_total[threadIdx.x] = __popcll(s_mask[threadIdx.x]);
        __syncthreads();
        first_rows(s_total, s_first, s_wave, A.experts);
        for (int e = threadIdx.x; e <= A.experts; e += 1024) A.offsets[e] = s_first[e];
    } else {
        for (int e = threadIdx.x; e < A.words * 4; e += 1024)
            A.counts[(size_t)blockIdx.x * A.words * 4 + e] = (uint8_t)__popcll(s_mask[e]);
    }
#pragma unroll
    for (int turn = 0; turn < kTurns; ++turn)
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            if (id[turn][s] < 0) continue;
            const int in = turn * kAtOnce + threadIdx.x / L;
            const long long t = (long long)blockIdx.x * kChunk + in;
            const int rank = __popcll(s_mask[id[turn][s]] & ((1ull << in) - 1));
            const int row = whole ? s_first[id[turn][s]] + rank : rank;
            A.row_of[t * A.top_k + l + s * L] = row;
            if (whole) A.row_token[row] = (int)t;
        }
}

// Each expert's rows in the chunks before each one, and its total; 64 experts a
// workgroup, 16 runs of chunks.
__global__ void __launch_bounds__(1024) k_moe_scan(RouteArgs A) {
    __shared__ int s_run[16][64];
    const int e = blockIdx.x * 64 + (threadIdx.x & 63), run = threadIdx.x >> 6, width = A.words * 4;
    const int per = (A.chunks + 15) / 16, c0 = min(run * per, A.chunks), c1 = min(c0 + per, A.chunks);
    int n = 0;
    if (e < A.experts)
        for (int c = c0; c < c1; ++c) n += A.counts[(size_t)c * width + e];
    s_run[run][threadIdx.x & 63] = n;
    __syncthreads();
    if (e >= A.experts) return;
    int at = 0;
    for (int r = 0; r < run; ++r) at += s_run[r][threadIdx.x & 63];
    for (int c = c0; c < c1; ++c) {
        A.before[(size_t)c * width + e] = at;
        at += A.counts[(size_t)c * width + e];
    }
    if (run == 15) A.totals[e] = at;
}

// The rows of kPlace chunks: what their tokens' ranks begin at. Up to
// kScanChunks chunks, every workgroup sums all of their counts by itself (251
// chunks of 256 experts: 64 KB from the L2, 7.7 us in all, where a scan of one
// workgroup between two launches took some 200).
__global__ void __launch_bounds__(1024) k_moe_place(RouteArgs A) {
    __shared__ int s_total[DQ_MOE_EXPERTS_MAX], s_before[kPlace][DQ_MOE_EXPERTS_MAX];
    __shared__ int s_first[DQ_MOE_EXPERTS_MAX + 1], s_wave[16];
    const int c0 = blockIdx.x * kPlace, width = A.words * 4;
    for (int e = threadIdx.x; e < width; e += 1024) {
        s_total[e] = 0;
        s_before[0][e] = 0;
    }
    __syncthreads();
    if (A.chunks <= kScanChunks) {
        const int runs = 1024 / A.words, w = threadIdx.x % A.words, run = threadIdx.x / A.words;
        if (run < runs) {
            int before[4] = {}, total[4] = {};
            constexpr int J = 16;  // counts on their way at a time
            for (int c = run; c < A.chunks; c += J * runs) {
                uint32_t n[J];
#pragma unroll
                for (int j = 0; j < J; ++j)
                    n[j] = reinterpret_cast<const uint32_t*>(A.counts)[(size_t)min(c + j * runs, A.chunks - 1) * A.words + w];
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int cj = c + j * runs;
                    if (cj >= A.chunks) n[j] = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        total[i] += n[j] >> (8 * i) & 255;
                        before[i] += cj < c0 ? n[j] >> (8 * i) & 255 : 0;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                atomicAdd(&s_total[w * 4 + i], total[i]);
                atomicAdd(&s_before[0][w * 4 + i], before[i]);
            }
        }
    } else {
        for (int e = threadIdx.x; e < A.experts; e += 1024) {
            s_total[e] = A.totals[e];
            s_before[0][e] = A.before[(size_t)c0 * width + e];
        }
    }
    __syncthreads();
    first_rows(s_total, s_first, s_wave, A.experts);
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= A.experts; e += 1024) A.offsets[e] = s_first[e];
    for (int e = threadIdx.x; e < A.experts; e += 1024) {
        int at = s_first[e] + s_before[0][e];
#pragma unroll
        for (int i = 0; i < kPlace; ++i) {
            s_before[i][e] = at;
            if (c0 + i < A.chunks) at += A.counts[(size_t)(c0 + i) * width + e];
        }
    }
    __syncthreads();
    const long long p0 = (long long)c0 * kChunk * A.top_k, p1 = min((long long)A.tokens, (long long)(c0 + kPlace) * kChunk) * A.top_k;
    for (long long p = p0 + threadIdx.x; p < p1; p += 1024) {
        const int e = A.ids[p];
        if (e < 0) continue;
        const int t = (int)(p / A.top_k), row = s_before[t / kChunk - c0][e] + A.row_of[p];
        A.row_of[p] = row;
        A.row_token[row] = t;
    }
}

__global__ void k_moe_none(int32_t* offsets, int experts) {
    for (int e = threadIdx.x; e <= experts; e += 256) offsets[e] = 0;
}

struct CombineArgs {
    const void* y;
    const float* weights;
    const int32_t* row_of;
    const void* add;
    void* out;
    int top_k, rows;
    uint32_t pieces;  // E elements each of a token's N
    FastDiv piece;
    long long items, N;
};

// E neighbouring elements of a tensor as fp32: one load of 16 bytes for 8 elements
// of 16 bits, two for fp32.
template <int T, int E>
__device__ __forceinline__ void load_piece(const void* p, size_t i, float* v) {
    if constexpr (E == 1) {
        v[0] = load1(p, i, T);
    } else if constexpr (T == DQ_F32) {
        const f4* q = reinterpret_cast<const f4*>(static_cast<const float*>(p) + i);
        const f4 lo = __builtin_nontemporal_load(q), hi = __builtin_nontemporal_load(q + 1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = lo[k];
            v[4 + k] = hi[k];
        }
    } else {
        const u4 w = __builtin_nontemporal_load(reinterpret_cast<const u4*>(static_cast<const uint16_t*>(p) + i));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t b = w[k / 2] >> (16 * (k & 1)) & 0xffffu;
            v[k] = T == DQ_BF16 ? bf16_bits_to_f32(b) : (float)__builtin_bit_cast(_Float16, (uint16_t)b);
        }
    }
}

// Bound by memory: each row of y is read once. A thread takes E elements of a
// token, J of its rows on their way at a time: 8101 tokens of 4 rows of 4096 in
// fp32 with a bf16 sum, 664 MB, 116.8 us, 5.7 TB/s of what a copy reaches 6.2
// (an element a thread: 310 us).
template <int TY, int TO, int E>
__global__ void __launch_bounds__(256) k_moe_combine(CombineArgs A) {
    const uint32_t item = blockIdx.x * 256u + threadIdx.x;
    if (item >= A.items) return;
    const uint32_t t = fdiv(item, A.piece);
    const size_t n = (size_t)(item - t * A.pieces) * E, at = (size_t)t * A.N + n;
    constexpr int J = 4;
    float v[E];
#pragma unroll
    for (int k = 0; k < E; ++k) v[k] = 0.0f;
    if (A.add) load_piece<TO, E>(A.add, at, v);
    for (int j0 = 0; j0 < A.top_k; j0 += J) {
        int r[J];
        float w[J], y[J][E];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const size_t p = (size_t)t * A.top_k + min(j0 + j, A.top_k - 1);
            r[j] = j0 + j < A.top_k ? A.row_of[p] : -1;
            w[j] = r[j] < A.rows ? A.weights[p] : __builtin_nanf("");
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (r[j] >= 0 && r[j] < A.rows) load_piece<TY, E>(A.y, (size_t)r[j] * A.N + n, y[j]);
            else
#pragma unroll
                for (int k = 0; k < E; ++k) y[j][k] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (r[j] >= 0)
#pragma unroll
                for (int k = 0; k < E; ++k) v[k] += w[j] * y[j][k];
    }
    if constexpr (E == 1) {
        if (TO == DQ_F32) static_cast<float*>(A.out)[at] = v[0];
        else if (TO == DQ_BF16) static_cast<uint16_t*>(A.out)[at] = (uint16_t)f32_to_bf16_bits(v[0]);
        else static_cast<_Float16*>(A.out)[at] = (_Float16)v[0];
    } else {
        const f4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
        if constexpr (TO == DQ_F32) {
            f4* q = reinterpret_cast<f4*>(static_cast<float*>(A.out) + at);
            __builtin_nontemporal_store(lo, q);
            __builtin_nontemporal_store(hi, q + 1);
        } else {
            u4 w;
            if constexpr (TO == DQ_BF16) {
                const u2 a = f32x4_to_bf16x4(lo), b = f32x4_to_bf16x4(hi);
                w = u4{a[0], a[1], b[0], b[1]};
            } else {
                typedef _Float16 h2 __attribute__((ext_vector_type(2)));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const h2 h = {(_Float16)v[2 * k], (_Float16)v[2 * k + 1]};
                    w[k] = __builtin_bit_cast(unsigned, h);
                }
            }
            __builtin_nontemporal_store(w, reinterpret_cast<u4*>(static_cast<uint16_t*>(A.out) + at));
        }
    }
}

template <int TY, int TO>
void launch_combine(const CombineArgs& A, bool vec, hipStream_t s) {
    const dim3 grid((unsigned)((A.items + 255) / 256)), block(256);
    if (vec) hipLaunchKernelGGL((k_moe_combine<TY, TO, 8>), grid, block, 0, s, A);
    else hipLaunchKernelGGL((k_moe_combine<TY, TO, 1>), grid, block, 0, s, A);
}
template <int TY>
void launch_combine(dq_dtype to, const CombineArgs& A, bool vec, hipStream_t s) {
    if (to == DQ_F32) launch_combine<TY, DQ_F32>(A, vec, s);
    else if (to == DQ_BF16) launch_combine<TY, DQ_BF16>(A, vec, s);
    else launch_combine<TY, DQ_F16>(A, vec, s);
}

void launch_choose(const RouteArgs& A, hipStream_t s) {
    const dim3 grid((unsigned)A.chunks), block(1024);
    // 16 lanes a token, up to 16 logits each; more lanes beyond that. Of a lane's sorted
    // logits up to 8 choices can need the first 8
    const bool few = A.top_k <= 8;
    if (A.experts <= 32) hipLaunchKernelGGL((k_moe_choose<2, 2, 16>), grid, block, 0, s, A);
    else if (A.experts <= 64) hipLaunchKernelGGL((k_moe_choose<4, 4, 16>), grid, block, 0, s, A);
    else if (A.experts <= 128) hipLaunchKernelGGL((k_moe_choose<8, 8, 16>), grid, block, 0, s, A);
    else if (A.experts <= 256 && few) hipLaunchKernelGGL((k_moe_choose<16, 8, 16>), grid, block, 0, s, A);
    else if (A.experts <= 256) hipLaunchKernelGGL((k_moe_choose<16, 16, 16>), grid, block, 0, s, A);
    else if (A.experts <= 512) hipLaunchKernelGGL((k_moe_choose<16, 16, 32>), grid, block, 0, s, A);
    else hipLaunchKernelGGL((k_moe_choose<16, 16, 64>), grid, block, 0, s, A);
}

size_t float_bytes(int type) { return type == DQ_F32 ? 4 : 2; }
bool is_float(dq_dtype t) { return t == DQ_F32 || t == DQ_BF16 || t == DQ_F16; }

int check_device(const dq_moe_ctx* c) {
    int dev = 0;
    (void)hipGetDevice(&dev);
    if (dev != c->device) DQ_FAIL(DQ_ERR_STATE, "the context belongs to another device");
    return DQ_OK;
}

}  // namespace

extern "C" int dq_moe_init(dq_moe_ctx** ctx, int64_t max_tokens, int experts, int top_k, dq_dtype logits_type,
                           int scoring, int normalize, float scale) {
    if (!ctx) DQ_FAIL(DQ_ERR_ARG, "ctx is NULL");
    *ctx = nullptr;
    if (max_tokens < 1 || experts < 1 || top_k < 1) DQ_FAIL(DQ_ERR_ARG, "sizes must be >= 1");
    if (top_k > experts) DQ_FAIL(DQ_ERR_ARG, "top_k exceeds the experts");
    if (!is_float(logits_type)) DQ_FAIL(DQ_ERR_TYPE, "logits must be fp32, bf16 or fp16");
    if (scoring != DQ_MOE_SOFTMAX && scoring != DQ_MOE_SIGMOID) DQ_FAIL(DQ_ERR_ARG, "no such scoring");
    if (!(scale - scale == 0.0f)) DQ_FAIL(DQ_ERR_ARG, "scale must be finite");
    if (experts > DQ_MOE_EXPERTS_MAX || top_k > DQ_MOE_TOP_K_MAX || max_tokens > DQ_MOE_TOKENS_MAX)
        DQ_FAIL(DQ_ERR_RANGE, "experts, top_k or max_tokens exceed %d, %d, %d", DQ_MOE_EXPERTS_MAX, DQ_MOE_TOP_K_MAX,
                DQ_MOE_TOKENS_MAX);
    dq_moe_ctx* c = new (std::nothrow) dq_moe_ctx();
    if (!c) DQ_FAIL(DQ_ERR_ALLOC, "host allocation for the experts' context failed");
    (void)hipGetDevice(&c->device);
    c->max_tokens = max_tokens;
    c->experts = experts;
    c->top_k = top_k;
    c->logits_type = logits_type;
    c->scoring = scoring;
    c->normalize = normalize != 0;
    c->scale = scale;
    const size_t chunks = (size_t)(max_tokens + kChunk - 1) / kChunk;
    const size_t width = (size_t)(experts + 3) / 4 * 4;
    const bool scan = chunks > kScanChunks;
    if (hipMalloc(&c->counts, chunks * width) != hipSuccess ||
        (scan && (hipMalloc(&c->before, chunks * width * 4) != hipSuccess ||
                  hipMalloc(&c->totals, width * 4) != hipSuccess))) {
        dq_moe_release(c);
        DQ_FAIL(DQ_ERR_ALLOC, "device allocation for the experts' context failed");
    }
    snprintf(c->info, sizeof c->info, "gfx950 experts: the %d largest of %d by %s%s, up to %lld tokens", top_k, experts,
             scoring == DQ_MOE_SIGMOID ? "sigmoid" : "softmax", normalize ? ", normalised" : "", (long long)max_tokens);
    *ctx = c;
    return DQ_OK;
}

extern "C" int dq_moe_route(dq_moe_ctx* ctx, int64_t tokens, const void* logits, int64_t logits_stride, int32_t* ids,
                            float* weights, int32_t* offsets, int32_t* row_token, int32_t* row_of, void* stream) {
    if (!ctx) DQ_FAIL(DQ_ERR_STATE, "no context");
    if (tokens < 0 || tokens > ctx->max_tokens)
        DQ_FAIL(DQ_ERR_ARG, "tokens must lie in [0, %lld]", (long long)ctx->max_tokens);
    if (!offsets) DQ_FAIL(DQ_ERR_ARG, "offsets must not be NULL");
    if (tokens && (!logits || !ids || !weights || !row_token || !row_of))
        DQ_FAIL(DQ_ERR_ARG, "logits, ids, weights, row_token and row_of must not be NULL");
    if (logits_stride < 0) DQ_FAIL(DQ_ERR_ARG, "logits_stride must be >= 0");
    if ((uintptr_t)logits % float_bytes(ctx->logits_type) || (uintptr_t)ids % 4 || (uintptr_t)weights % 4 ||
        (uintptr_t)offsets % 4 || (uintptr_t)row_token % 4 || (uintptr_t)row_of % 4)
        DQ_FAIL(DQ_ERR_ARG, "a tensor is not aligned to its elements");
    if (int rc = check_device(ctx)) return rc;
    RouteArgs A{};
    A.logits = logits;
    A.stride = logits_stride;
    A.ids = ids;
    A.weights = weights;
    A.offsets = offsets;
    A.row_token = row_token;
    A.row_of = row_of;
    A.counts = ctx->counts;
    A.before = ctx->before;
    A.totals = ctx->totals;
    A.tokens = (int)tokens;
    A.experts = ctx->experts;
    A.top_k = ctx->top_k;
    A.chunks = (int)((tokens + kChunk - 1) / kChunk);
    A.words = (ctx->experts + 3) / 4;
    A.type = ctx->logits_type;
    A.sigmoid = ctx->scoring == DQ_MOE_SIGMOID;
    A.normalize = ctx->normalize;
    A.scale = ctx->scale;
    // as many logits as a lane takes at a time divide the experts, and rows begin at 16 bytes
    const int wide = ctx->experts <= 32 ? 2 : ctx->experts <= 64 ? 4 : 8;
    A.vec = (uintptr_t)logits % 16 == 0 && logits_stride * float_bytes(ctx->logits_type) % 16 == 0 && ctx->experts % wide == 0;
    const hipStream_t s = (hipStream_t)stream;
    if (tokens == 0) {
        hipLaunchKernelGGL(k_moe_none, dim3(1), dim3(256), 0, s, offsets, ctx->experts);
        DQ_LAUNCH_CHECK("experts' offsets");
        return DQ_OK;
    }
    launch_choose(A, s);
    DQ_LAUNCH_CHECK("choice of experts");
    if (A.chunks == 1) return DQ_OK;
    if (A.chunks > kScanChunks) {
        hipLaunchKernelGGL(k_moe_scan, dim3((ctx->experts + 63) / 64), dim3(1024), 0, s, A);
        DQ_LAUNCH_CHECK("experts' offsets");
    }
    hipLaunchKernelGGL(k_moe_place, dim3((A.chunks + kPlace - 1) / kPlace), dim3(1024), 0, s, A);
    DQ_LAUNCH_CHECK("experts' rows");
    return DQ_OK;
}

extern "C" int dq_moe_combine(dq_moe_ctx* ctx, int64_t tokens, int64_t N, const void* y, int64_t rows, dq_dtype y_type,
                              const float* weights, const int32_t* row_of, const void* add, dq_dtype out_type, void* out,
                              void* stream) {
    if (!ctx) DQ_FAIL(DQ_ERR_STATE, "no context");
    if (tokens < 0 || tokens > ctx->max_tokens)
        DQ_FAIL(DQ_ERR_ARG, "tokens must lie in [0, %lld]", (long long)ctx->max_tokens);
    if (N < 1 || rows < 0 || rows > INT32_MAX) DQ_FAIL(DQ_ERR_ARG, "N must be >= 1 and rows lie in [0, 2^31)");
    if (!is_float(y_type) || !is_float(out_type)) DQ_FAIL(DQ_ERR_TYPE, "y and out must be fp32, bf16 or fp16");
    if (tokens == 0) return DQ_OK;
    if ((!y && rows) || !weights || !row_of || !out) DQ_FAIL(DQ_ERR_ARG, "y, weights, row_of and out must not be NULL");
    if ((uintptr_t)y % float_bytes(y_type) || (uintptr_t)weights % 4 || (uintptr_t)row_of % 4 ||
        (uintptr_t)add % float_bytes(out_type) || (uintptr_t)out % float_bytes(out_type))
        DQ_FAIL(DQ_ERR_ARG, "a tensor is not aligned to its elements");
    if (int rc = check_device(ctx)) return rc;
    // 16 bytes at a time: every row starts at one
    const bool vec = N % 8 == 0 && (uintptr_t)y % 16 == 0 && (uintptr_t)out % 16 == 0 && (uintptr_t)add % 16 == 0;
    CombineArgs A{};
    A.y = y;
    A.weights = weights;
    A.row_of = row_of;
    A.add = add;
    A.out = out;
    A.top_k = ctx->top_k;
    A.rows = (int)rows;
    A.N = N;
    const int64_t pieces = vec ? N / 8 : N;
    if (N > INT32_MAX || (__int128)tokens * pieces > INT32_MAX) DQ_FAIL(DQ_ERR_RANGE, "too many elements for one launch");
    A.pieces = (uint32_t)pieces;
    A.piece = make_fastdiv(A.pieces);
    A.items = tokens * pieces;
    const hipStream_t s = (hipStream_t)stream;
    if (y_type == DQ_F32) launch_combine<DQ_F32>(out_type, A, vec, s);
    else if (y_type == DQ_BF16) launch_combine<DQ_BF16>(out_type, A, vec, s);
    else launch_combine<DQ_F16>(out_type, A, vec, s);
    DQ_LAUNCH_CHECK("sum of the experts' results");
    return DQ_OK;
}

extern "C" const char* dq_moe_info(const dq_moe_ctx* ctx) { return ctx ? ctx->info : nullptr; }

extern "C" void dq_moe_release(dq_moe_ctx* ctx) {
    if (!ctx) return;
    (void)hipFree(ctx->counts);
    (void)hipFree(ctx->before);
    (void)hipFree(ctx->totals);
    delete ctx;
}
