// kv_plan.h -- index arithmetic of the paged key-value cache: where a token's
// row lies, which elements a rotated pair joins, and how the attention's work
// is shared out. Plain C++ that both the kernels and a host-compiled check
// use (no HIP header is needed).
#pragma once

#include <math.h>
#include <stdint.h>

#if defined(__HIPCC__)
#define DQ_HD __host__ __device__ __forceinline__
#else
#define DQ_HD inline
#endif

namespace dq {

// n / d of 32-bit unsigned numbers for a constant d >= 1 by one multiplication
// (the round-up form of Granlund & Montgomery, PLDI 1994).
struct KvDiv {
    uint32_t d, m, s;
};

inline KvDiv make_kvdiv(uint32_t d) {
    KvDiv f;
    f.d = d;
    f.s = 0;
    while ((1ull << f.s) < d) ++f.s;
    f.m = (uint32_t)(((1ull << 32) * ((1ull << f.s) - d)) / d + 1);
    return f;
}

DQ_HD uint32_t kv_div(uint32_t n, const KvDiv& f) {
    const uint64_t hi = ((uint64_t)n * f.m) >> 32;
    return (uint32_t)((hi + n) >> f.s);
}

// The part of a cache that an index needs: `pages` pages of `page.d` slots for
// each of `heads` key-value heads, `per_seq` block table entries a sequence.
struct KvGeom {
    KvDiv page;
    int pages, per_seq, heads;
};

// Row (of D values) of token t of a sequence for key-value head h, where table
// is the sequence's line of the block table; -1 where t lies beyond the table
// or its entry names no page (kv_row_of: given the entry). The largest row fits 31 bits (checked when a
// context is made); byte offsets are taken from it in 64 bits.
DQ_HD int32_t kv_row_of(int32_t entry, uint32_t t, int h, const KvGeom& g) {
    const uint32_t p = (uint32_t)entry;
    if (p >= (uint32_t)g.pages) return -1;
    return (int32_t)((p * (uint32_t)g.heads + (uint32_t)h) * g.page.d + (t - kv_div(t, g.page) * g.page.d));
}
DQ_HD int32_t kv_row(const int32_t* table, uint32_t t, int h, const KvGeom& g) {
    const uint32_t e = kv_div(t, g.page);
    return e < (uint32_t)g.per_seq ? kv_row_of(table[e], t, h, g) : -1;
}

// The two elements of virtual pair i of a row of D elements, the first R of
// which are rotated: pairs below R/2 are the rotated ones (halves apart, or
// neighbours), the others join what passes through unchanged.
DQ_HD void kv_pair(int i, int D, int R, bool interleaved, int* a, int* b) {
    if (interleaved) {
        *a = 2 * i;
        *b = 2 * i + 1;
    } else if (i < R / 2) {
        *a = i;
        *b = i + R / 2;
    } else {
        *a = R + (i - R / 2);
        *b = *a + (D - R) / 2;
    }
}

// A rotary pair's frequency in turns, f / 2 pi = hi + lo to 2^-103 of it (1 / 2 pi
// is its double and the rest's; the product's own rest by fma). Times a position
// of 31 bits that is 3e-14 of a turn for the largest frequency, 1e9, and 4e-23 for
// those up to 1.
inline void kv_turns(double f, double* hi, double* lo) {
    const double c0 = 0x1.45f306dc9c883p-3, c1 = -0x1.6b01ec5417056p-57;
    *hi = f * c0;
    *lo = fma(f, c0, -*hi) + f * c1;
}

// ------------------------------------------------------- sharing out tokens
//
// The attention's tokens are cut into units of kKvUnit tokens of one sequence
// and one head tile. Units are numbered sequence by sequence, head tile by
// head tile, and each worker takes a run of them, so all have the same number
// to within one, whatever the lengths. Up to kKvRound units a worker, all runs
// are of the same whole number (fewer workers then, none with more to do):
// runs that begin in the middle of a sequence and end in the next one's cost
// more than an idle worker (108 heads with a window of 1000 tokens 19.7 to 20.1
// us, shared to within one 23.4).
constexpr int kKvUnit = 128;
constexpr int kKvRound = 8;

DQ_HD int kv_first_token(int len, int window) { return window > 0 && len > window ? len - window : 0; }
DQ_HD int kv_units(int len, int window) {
    return (len - kv_first_token(len, window) + kKvUnit - 1) / kKvUnit;
}

struct KvShare {
    int64_t units;
    int workers;  // that have a unit
    int each;     // units of a worker; 0: shares to within one
};
DQ_HD KvShare kv_share(int64_t units, int most) {
    const int64_t each = (units + most - 1) / most;
    KvShare s;
    s.units = units;
    s.each = each <= kKvRound ? (int)each : 0;
    s.workers = each == 0 ? 0 : s.each ? (int)((units + each - 1) / each) : most;
    return s;
}
// the first unit of worker w
DQ_HD int64_t kv_first(int w, const KvShare& s) {
    if (!s.each) return s.units * w / s.workers;
    const int64_t u = (int64_t)w * s.each;
    return u < s.units ? u : s.units;
}
// the worker that takes unit u: the largest w with kv_first(w) <= u
DQ_HD int kv_worker(int64_t u, const KvShare& s) {
    return s.each ? (int)(u / s.each) : (int)(((u + 1) * s.workers - 1) / s.units);
}

}  // namespace dq
