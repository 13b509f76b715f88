// paged_attend.hip -- attention of one new token of every sequence over the
// paged key-value cache.
//
//   s_t = sm_scale q . k_t     for the tokens t in [max(0, len - window), len)
//   p   = softmax(s),  out = sum_t p_t v_t,  lse = log sum_t exp(s_t)
// and, where weights are gathered, scores' = decay scores + sum of p_t over
// the query heads of a key-value head.
//
// One workgroup for a sequence and a query head: each wave takes every fourth
// token, with a running maximum and sum, and the waves are joined in LDS.
// Scores are kept in units of log2 (s log2 e), so that exp is v_exp_f32.
#include "paged_kv.h"

using namespace dq;

namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct SimpleArgs {
    DqAttendArgs a;
    int q_type, cache_type, Hq, Hk, D, cap;
    float* s;
    size_t s_stride;
    float* l2;  // [batch * Hq] log2 of the sum
    int32_t* bad;
    KvGeom geom;
};

__device__ __forceinline__ float wave_sum(float v) {
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

__device__ __forceinline__ int seq_len(const int32_t* lens, int b, int cap, bool* bad) {
    const int n = lens[b];
    *bad = n < 0 || n > cap;
    return n < 0 ? 0 : min(n, cap);
}

__global__ void __launch_bounds__(256) k_attend(const SimpleArgs A) {
    __shared__ float sm[4], sl[4], sacc[4][256];
    const int hq = blockIdx.x, b = blockIdx.y, hk = hq / (A.Hq / A.Hk);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    bool bad;
    const int n = seq_len(A.a.lens, b, A.cap, &bad);
    if (bad && threadIdx.x == 0) atomicAdd(A.bad, 1);
    const int first = kv_first_token(n, A.a.window);
    const int32_t* line = A.a.table + (size_t)b * A.geom.per_seq;
    float q[4], acc[4] = {0, 0, 0, 0}, m = -__builtin_inff(), l = 0.0f;
    for (int j = 0; j < 4; ++j) {
        const int d = lane + 64 * j;
        q[j] = d < A.D ? load_any(A.a.q, A.q_type, b * A.a.q_ts + hq * A.a.q_hs + d) : 0.0f;
    }
    for (int t = first + wave; t < n; t += 4) {
        int32_t row = kv_row(line, (uint32_t)t, hk, A.geom);
        const bool lost = row < 0;
        if (lost) {
            if (lane == 0) atomicAdd(A.bad, 1);
            row = 0;
        }
        float x = 0.0f;
        for (int j = 0; j < 4; ++j) {
            const int d = lane + 64 * j;
            if (d < A.D) x += q[j] * load_any(A.a.k, A.cache_type, (long long)row * A.D + d);
        }
        x = wave_sum(x);
        if (A.a.ks) x *= A.a.ks[row];
        x *= A.a.sm_scale * kLog2e;
        if (lost) x = __builtin_nanf("");
        if (A.a.scores && lane == 0) A.s[(size_t)(b * A.Hq + hq) * A.s_stride + (t - first)] = x;
        const float m1 = __builtin_fmaxf(m, x);
        const float ref = m1 == -__builtin_inff() ? 0.0f : m1;
        const float f = __builtin_amdgcn_exp2f(m - ref), p = __builtin_amdgcn_exp2f(x - ref);
        const float w = A.a.vs ? p * A.a.vs[row] : p;
        l = l * f + p;
        for (int j = 0; j < 4; ++j) {
            const int d = lane + 64 * j;
            if (d < A.D) acc[j] = acc[j] * f + w * load_any(A.a.v, A.cache_type, (long long)row * A.D + d);
        }
        m = m1;
    }
    if (lane == 0) {
        sm[wave] = m;
        sl[wave] = l;
    }
    for (int j = 0; j < 4; ++j) sacc[wave][lane + 64 * j] = acc[j];
    __syncthreads();
    float top = __builtin_fmaxf(__builtin_fmaxf(sm[0], sm[1]), __builtin_fmaxf(sm[2], sm[3]));
    const float ref = top == -__builtin_inff() ? 0.0f : top;
    float sum = 0.0f, o = 0.0f;
    const int d = threadIdx.x;
    for (int w = 0; w < 4; ++w) {
        const float f = __builtin_amdgcn_exp2f(sm[w] - ref);
        sum += sl[w] * f;
        o += sacc[w][d] * f;
    }
    o = sum == 0.0f ? 0.0f : o / sum;
    float l2 = sum == 0.0f ? -__builtin_inff() : ref + __builtin_amdgcn_logf(sum);
    if (bad) o = l2 = __builtin_nanf("");
    const size_t i = (size_t)b * A.Hq + hq;
    if (d < A.D) store_any(A.a.out, A.q_type, (long long)(i * A.D + d), o);
    if (d == 0) {
        A.l2[i] = l2;
        if (A.a.lse) A.a.lse[i] = l2 * kLn2;
    }
}

__global__ void __launch_bounds__(256) k_gather_scores(const SimpleArgs A) {
    const int item = blockIdx.y, b = item / A.Hk, hk = item - b * A.Hk, G = A.Hq / A.Hk;
    bool bad;
    const int n = seq_len(A.a.lens, b, A.cap, &bad), first = kv_first_token(n, A.a.window);
    for (int t = blockIdx.x * 256 + threadIdx.x; t < n; t += gridDim.x * 256) {
        float sum = A.a.scores[(size_t)item * A.cap + t] * A.a.decay;
        float p = 0.0f;
        if (t >= first)
            for (int g = 0; g < G; ++g) {
                const size_t i = (size_t)b * A.Hq + hk * G + g;
                const float l2 = A.l2[i];
                if (l2 != -__builtin_inff()) p += __builtin_amdgcn_exp2f(A.s[i * A.s_stride + (t - first)] - l2);
            }
        A.a.scores_out[(size_t)item * A.cap + t] = sum + p;
    }
}

}  // namespace

size_t dq_attend_part_floats(const dq_kv_ctx* c) { return (size_t)c->batch * c->Hq; }

int dq_launch_attend(const dq_kv_ctx* c, const DqAttendArgs& a, hipStream_t s) {
    const SimpleArgs A{a, c->q_type, c->cache_type, c->Hq, c->Hk, c->D, c->cap, c->s, c->s_stride, c->part, c->bad,
                       c->geom};
    hipLaunchKernelGGL(k_attend, dim3((unsigned)c->Hq, (unsigned)a.batch), dim3(256), 0, s, A);
    DQ_LAUNCH_CHECK("attention");
    if (a.scores) {
        hipLaunchKernelGGL(k_gather_scores, dim3((unsigned)((c->cap + 1023) / 1024), (unsigned)(a.batch * c->Hk)),
                           dim3(256), 0, s, A);
        DQ_LAUNCH_CHECK("gathered weights");
    }
    return DQ_OK;
}
