// paged_kv.h -- what the translation units of the paged key-value cache share:
// the contexts, element types and the angle of a rotary position.
#pragma once

#include "dq_device.h"
#include "kv_plan.h"

// Rotary positions: for every pair of the rotated part its position axis and
// its frequency in turns, inv_freq / 2 pi, as a double and its remainder.
struct dq_rope_ctx {
    int device = 0;
    int D = 0, R = 0, axes = 1, interleaved = 0;
    double2* freq = nullptr;  // [R / 2] (hi, lo)
    int32_t* axis = nullptr;  // [R / 2]
    char info[192] = "";
};

struct dq_kv_ctx {
    int device = 0;
    int batch = 0, Hq = 0, Hk = 0, D = 0, pages = 0, page_size = 0, per_seq = 0, cap = 0;
    dq_dtype q_type = DQ_BF16, cache_type = DQ_BF16;
    bool scores = false;
    dq::KvGeom geom{};
    int cus = 0;
    int32_t* bad = nullptr;    // [1] entries that named no page, sequence or length
    int32_t* moves = nullptr;  // eviction: [batch * Hk] counts, then per head the slots
                               // freed and those moved into them
    size_t moves_stride = 0;
    float* s = nullptr;        // [batch * Hk, s_stride] scores of the attention (log2)
    size_t s_stride = 0;
    float* part = nullptr;     // partial results of the attention
    size_t part_floats = 0;
    int attend_workers = 0;    // workgroups of the attention on the chip at once
    char info[192] = "";
};

int dq_kv_check_device(const dq_kv_ctx* c);
int dq_rope_check_device(const dq_rope_ctx* c);

// Attention (paged_attend.hip); the arguments have been checked.
struct DqAttendArgs {
    const void* q;
    long long q_ts, q_hs;  // strides in elements
    const int32_t* lens;
    const int32_t* table;
    const void* k;
    const void* v;
    const float* ks;
    const float* vs;
    void* out;
    float* lse;  // may be NULL
    int batch;
    float sm_scale;
    int window;
    const float* scores;  // NULL: not gathered
    float* scores_out;
    float decay;
};
// the attention's workers and the size of their partial results
int dq_attend_plan(dq_kv_ctx* c);
int dq_launch_attend(const dq_kv_ctx* c, const DqAttendArgs& a, hipStream_t s);

namespace dq {

inline size_t kv_elem_bytes(dq_dtype t) { return t == DQ_F32 ? 4 : t == DQ_I8 ? 1 : 2; }

// Storage of an element type and its conversions (round to nearest even).
template <int TYPE> struct Elem;
template <> struct Elem<DQ_F32> { typedef float S; };
template <> struct Elem<DQ_BF16> { typedef __bf16 S; };
template <> struct Elem<DQ_F16> { typedef _Float16 S; };
template <> struct Elem<DQ_I8> { typedef int8_t S; };

// N elements of type S moved as one access, N * sizeof(S) a power of two up to 16
// bytes. ALIGN: what p is aligned to, the access's own size unless given.
template <typename S, int N, int ALIGN = N * (int)sizeof(S)>
__device__ __forceinline__ void load_vec(const S* p, float (&f)[N]) {
    typedef S V __attribute__((ext_vector_type(N), aligned(ALIGN)));
    const V v = *(const V*)p;
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = (float)v[i];
}
template <typename S>
__device__ __forceinline__ void load_vec(const S* p, float (&f)[1]) { f[0] = (float)*p; }

// Stores past the caches: the rotation of 168 MB took 37.5 us with them and 43
// without, a prompt's append 34 and 46, small ones the same.
template <typename S, int N, int ALIGN = N * (int)sizeof(S)>
__device__ __forceinline__ void store_vec(S* p, const float (&f)[N]) {
    typedef S V __attribute__((ext_vector_type(N), aligned(ALIGN)));
    V v;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (S)f[i];
    __builtin_nontemporal_store(v, (V*)p);
}
template <typename S>
__device__ __forceinline__ void store_vec(S* p, const float (&f)[1]) { *p = (S)f[0]; }

// VP pairs of a row: VP elements from lo and from hi, or 2 VP neighbours from lo;
// aligned to VP elements or 2 VP neighbours, a single pair to its elements alone.
template <typename S, int VP, bool IL>
__device__ __forceinline__ void load_pairs(const S* row, int lo, int hi, float (&a)[VP], float (&b)[VP]) {
    if constexpr (IL) {
        float e[2 * VP];
        load_vec<S, 2 * VP, (VP > 1 ? 2 * VP : 1) * (int)sizeof(S)>(row + lo, e);
#pragma unroll
        for (int i = 0; i < VP; ++i) {
            a[i] = e[2 * i];
            b[i] = e[2 * i + 1];
        }
    } else {
        load_vec(row + lo, a);
        load_vec(row + hi, b);
    }
}

template <typename S, int VP, bool IL>
__device__ __forceinline__ void store_pairs(S* row, int lo, int hi, const float (&a)[VP], const float (&b)[VP]) {
    if constexpr (IL) {
        float e[2 * VP];
#pragma unroll
        for (int i = 0; i < VP; ++i) {
            e[2 * i] = a[i];
            e[2 * i + 1] = b[i];
        }
        store_vec<S, 2 * VP, (VP > 1 ? 2 * VP : 1) * (int)sizeof(S)>(row + lo, e);
    } else {
        store_vec(row + lo, a);
        store_vec(row + hi, b);
    }
}

// Element i of a tensor whose type is known at run time.
__device__ __forceinline__ void store_any(void* p, int type, long long i, float f) {
    if (type == DQ_F32) ((float*)p)[i] = f;
    else if (type == DQ_BF16) ((__bf16*)p)[i] = (__bf16)f;
    else ((_Float16*)p)[i] = (_Float16)f;
}

// Four neighbouring elements, aligned to their size.
__device__ __forceinline__ void store4_any(void* p, int type, size_t i, f4 f) {
    typedef __bf16 b4 __attribute__((ext_vector_type(4)));
    typedef _Float16 h4 __attribute__((ext_vector_type(4)));
    if (type == DQ_F32) *(f4*)((float*)p + i) = f;
    else if (type == DQ_BF16) *(b4*)((__bf16*)p + i) = __builtin_convertvector(f, b4);
    else *(h4*)((_Float16*)p + i) = __builtin_convertvector(f, h4);
}

// cos and sin of pos * freq (freq in turns, hi + lo, from kv_turns). The product
// is reduced to a fraction of a turn in fp64 with its remainder kept: a position
// of 31 bits is off by 1e-16 of a turn with frequencies up to 1 and by 3e-14 with
// the largest, 1e9 (n is the rounded product's then, so r can be some 70 turns).
// The Taylor series on [-pi/4, pi/4] (first term left
// out: x^17 / 17! < 5e-17) are summed in fp64, whose rate on this chip is
// fp32's: the results are fp32 values rounded once.
__device__ __forceinline__ void rope_cos_sin(int pos, double2 freq, float* c, float* s) {
    const double t = (double)pos;
    const double n = __builtin_rint(t * freq.x);
    const double r = __builtin_fma(t, freq.y, __builtin_fma(t, freq.x, -n));
    const double k = __builtin_rint(4.0 * r);
    const double x = (r - 0.25 * k) * 6.283185307179586476925;
    const double x2 = x * x;
    double a = -1.0 / 1307674368000.0;  // -1/15!
    a = __builtin_fma(a, x2, 1.0 / 6227020800.0);
    a = __builtin_fma(a, x2, -1.0 / 39916800.0);
    a = __builtin_fma(a, x2, 1.0 / 362880.0);
    a = __builtin_fma(a, x2, -1.0 / 5040.0);
    a = __builtin_fma(a, x2, 1.0 / 120.0);
    a = __builtin_fma(a, x2, -1.0 / 6.0);
    a = __builtin_fma(a * x2, x, x);
    double b = 1.0 / 20922789888000.0;  // 1/16!
    b = __builtin_fma(b, x2, -1.0 / 87178291200.0);
    b = __builtin_fma(b, x2, 1.0 / 479001600.0);
    b = __builtin_fma(b, x2, -1.0 / 3628800.0);
    b = __builtin_fma(b, x2, 1.0 / 40320.0);
    b = __builtin_fma(b, x2, -1.0 / 720.0);
    b = __builtin_fma(b, x2, 1.0 / 24.0);
    b = __builtin_fma(b, x2, -0.5);
    b = __builtin_fma(b, x2, 1.0);
    const int q = (int)k & 3;
    const double cc = (q & 1) ? a : b, ss = (q & 1) ? b : a;
    *c = (float)((q == 1 || q == 2) ? -cc : cc);
    *s = (float)((q & 2) ? -ss : ss);
}

// The cosines and sines of `pairs` pairs of tokens t0 .. t0 + n - 1 into tab
// [n][pairs], by the 256 threads of a workgroup: its threads share a token's
// angles (about 40 operations each) among many heads.
__device__ __forceinline__ void rope_table(float2* tab, int t0, int n, int pairs, const int32_t* pos, int tokens,
                                           const double2* freq, const int32_t* axis, bool inverse) {
    for (int e = threadIdx.x; e < n * pairs; e += 256) {
        const int t = e / pairs, i = e - t * pairs;
        float c, s;
        rope_cos_sin(pos[(size_t)axis[i] * tokens + t0 + t], freq[i], &c, &s);
        tab[e] = float2{c, inverse ? -s : s};
    }
    __syncthreads();
}

}  // namespace dq
