// w4_device.h -- device helpers of the products with 4-bit weights: operand
// types, unpacking, the rows of x, finding a workgroup's rows.
#pragma once

#include "w4.h"

namespace dq {

typedef void (*W4RowsKernel)(W4Args);
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));

// An fp32 value as three bf16 values that sum to it exactly (24 bits; below
// 2^-110 the last ones may be lost).
__device__ __forceinline__ void split3(const float* v, u4* hi, u4* mid, u4* lo) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f2 a = {v[2 * i], v[2 * i + 1]};
        const bf16x2 h = __builtin_convertvector(a, bf16x2);
        const f2 r = {a[0] - (float)h[0], a[1] - (float)h[1]};
        const bf16x2 m = __builtin_convertvector(r, bf16x2);
        const f2 t = {r[0] - (float)m[0], r[1] - (float)m[1]};
        (*hi)[i] = __builtin_bit_cast(unsigned, h);
        (*mid)[i] = __builtin_bit_cast(unsigned, m);
        (*lo)[i] = __builtin_bit_cast(unsigned, __builtin_convertvector(t, bf16x2));
    }
}

// 16 bytes a lane from a bounded buffer straight into LDS, the wave's lanes one behind
// the other from `block` (uniform) on; zeros for an offset beyond the buffer. A plain
// device function: in a lambda it would be compiled for the host too.
__device__ __forceinline__ void buffer16_to_lds(__amdgpu_buffer_rsrc_t buf, char* block, uint32_t lane_at, uint32_t at) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (__attribute__((address_space(3))) void*)block, 16, (int)lane_at, (int)at, 0, 0);
}

// The matrix operands that a type of x is multiplied in, P pieces of it.
template <int T>
struct W4Op;
template <>
struct W4Op<DQ_BF16> {
    static constexpr int P = 1, elem = 2;
    static constexpr unsigned kOnes = 0x3f803f80u;
    // Eight codes as eight bf16. A byte with a value below 16 is, read as an
    // fp8 number (e4m3), that value times 2^-9: 0 to 7 are its subnormals, 8 to
    // 15 its first binade. So the conversion of fp8 pairs with a scale of 2^9
    // makes exact integers of them, 4 instructions for 8 codes and 3 for the
    // bytes.
    static __device__ __forceinline__ u4 codes(unsigned w) {
        const unsigned lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
        const u4 r = {__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false)),
                      __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true)),
                      __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false)),
                      __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true))};
        return r;
    }
    static __device__ __forceinline__ float value(unsigned b) { return bf16_bits_to_f32(b); }
    static __device__ __forceinline__ f4 mfma(u4 a, u4 b, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
    }
};
template <>
struct W4Op<DQ_F32> : W4Op<DQ_BF16> {
    static constexpr int P = 3, elem = 4;
};
template <>
struct W4Op<DQ_F16> {
    static constexpr int P = 1, elem = 2;
    static constexpr unsigned kOnes = 0x3c003c00u;
    static __device__ __forceinline__ u4 codes(unsigned w) {
        const unsigned lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
        const u4 r = {__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, false)),
                      __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, true)),
                      __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, false)),
                      __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, true))};
        return r;
    }
    static __device__ __forceinline__ float value(unsigned b) {
        return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
    }
    static __device__ __forceinline__ f4 mfma(u4 a, u4 b, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
    }
};

// Eight elements of a row of x from k on, as the P pieces of the operand;
// elements from K on are zeros and not read.
template <int T>
__device__ __forceinline__ void w4_load8(const char* row, int k, int K, bool vec, u4* out) {
    using O = W4Op<T>;
    const char* p = row + (size_t)k * O::elem;
    if constexpr (T == DQ_F32) {
        float v[8];
        if (vec) {
            // K is a multiple of 8 here
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f4 t = {0.0f, 0.0f, 0.0f, 0.0f};
                if (k < K) t = *reinterpret_cast<const f4*>(p + 16 * h);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[4 * h + i] = t[i];
            }
        } else if (k + 8 <= K) {  // loads of 16 bytes from any address
            __builtin_memcpy(v, p, 32);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = k + i < K ? reinterpret_cast<const float*>(p)[i] : 0.0f;
        }
        split3(v, out, out + 1, out + 2);
    } else if (vec) {
        u4 t = {0, 0, 0, 0};
        if (k < K) t = *reinterpret_cast<const u4*>(p);
        out[0] = t;
    } else if (k + 8 <= K) {
        __builtin_memcpy(out, p, 16);
    } else {
        unsigned v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = k + i < K ? reinterpret_cast<const uint16_t*>(p)[i] : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) out[0][i] = v[2 * i] | v[2 * i + 1] << 16;
    }
}

// A group's scale and zero point as fp32.
__device__ __forceinline__ float w4_scale(const void* scales, size_t i, int type) {
    if (type == DQ_F32) return static_cast<const float*>(scales)[i];
    const uint16_t b = static_cast<const uint16_t*>(scales)[i];
    return type == DQ_BF16 ? bf16_bits_to_f32(b) : (float)__builtin_bit_cast(_Float16, b);
}

// A column's scales of a block: N bytes as words, and the g-th of them.
template <int N>
__device__ __forceinline__ void w4_words(const char* p, uint32_t* w) {
    if constexpr (N == 2) {
        w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else if constexpr (N == 4) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (N == 8) {
        const u2 t = *reinterpret_cast<const u2*>(p);
        w[0] = t[0];
        w[1] = t[1];
    } else {
        const u4 t = *reinterpret_cast<const u4*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = t[i];
    }
}
template <int ST>
__device__ __forceinline__ float w4_scale_word(const uint32_t* w, int g) {
    if constexpr (ST == DQ_F32) return __uint_as_float(w[g]);
    const uint32_t h = w[g / 2] >> (16 * (g & 1)) & 0xffffu;
    return ST == DQ_BF16 ? bf16_bits_to_f32(h) : (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}

__device__ __forceinline__ void w4_store(void* y, size_t i, float v, int type) {
    if (type == DQ_F32) static_cast<float*>(y)[i] = v;
    else if (type == DQ_BF16) static_cast<uint16_t*>(y)[i] = (uint16_t)f32_to_bf16_bits(v);
    else static_cast<_Float16*>(y)[i] = (_Float16)v;
}

// Eight neighbouring elements of a row of y, from column n on; those from N on
// are not stored. vec: every row and n is 16-byte aligned.
__device__ __forceinline__ void w4_store8(void* y, size_t row, int n, int N, const float* v, int type, bool vec) {
    if (vec && n + 8 <= N) {
        const f4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
        if (type == DQ_F32) {
            f4* p = reinterpret_cast<f4*>(static_cast<float*>(y) + row + n);
            p[0] = lo;
            p[1] = hi;
            return;
        }
        u4 w;
        if (type == DQ_BF16) {
            const u2 l = f32x4_to_bf16x4(lo), h = f32x4_to_bf16x4(hi);
            w = u4{l[0], l[1], h[0], h[1]};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const h2 p = {(_Float16)v[2 * i], (_Float16)v[2 * i + 1]};
                w[i] = __builtin_bit_cast(unsigned, p);
            }
        }
        *reinterpret_cast<u4*>(static_cast<uint16_t*>(y) + row + n) = w;
        return;
    }
    for (int i = 0; i < 8; ++i)
        if (n + i < N) w4_store(y, row + n + i, v[i], type);
}

__device__ __forceinline__ float w4_silu(float v) { return v / (1.0f + expf(-v)); }

// The rows of the t-th row tile of TM rows: expert, first row, end. Without
// offsets there is one expert. Offsets that do not increase or leave
// [lo, hi] are taken as the nearest that do. Every wave finds its tile by
// itself: 64 experts at a time, a prefix sum of their tiles.
struct W4Tile {
    int expert, first, end;  // first == end: no such tile
};
__device__ __forceinline__ W4Tile w4_tile(const W4Args& A, int t, int TM, int lo, int hi) {
    if (!A.offsets) return {0, min(lo + t * TM, hi), min(hi, lo + t * TM + TM)};
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int e0 = 0; e0 < A.experts; e0 += 64) {
        const int e = e0 + lane;
        int a = 0, b = 0;
        if (e < A.experts) {
            a = min(max(A.offsets[e], lo), hi);
            b = min(max(A.offsets[e + 1], a), hi);
        }
        const int n = (b - a + TM - 1) / TM;
        int upto = n;
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(upto, o);
            if (lane >= o) upto += v;
        }
        const int total = __builtin_amdgcn_readlane(upto, 63);  // uniform, and seen as such
        if (t < before + total) {
            const int l = __ffsll((unsigned long long)__ballot(before + upto > t)) - 1;
            const int first = __builtin_amdgcn_readlane(a, l) + (t - before - __builtin_amdgcn_readlane(upto - n, l)) * TM;
            return {e0 + l, first, min(first + TM, __builtin_amdgcn_readlane(b, l))};
        }
        before += total;
    }
    return {0, 0, 0};
}

}  // namespace dq
