// paged_attend.hip -- attention of one new token of every sequence over the
// paged key-value cache: the join of partial results, the gathered weights,
// and the launches. The attention itself is in attend_kernel.h.
#include <algorithm>

#include "attend_kernel.h"

using namespace dq;

namespace {

// Joins the partial results of a query head whose units several workgroups
// took: o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i. One workgroup a head;
// groups of D / 4 lanes take the parts in turn and are added in order in LDS,
// so a result never depends on timing.
__global__ void __launch_bounds__(256) k_attend_join(const AttendArgs A) {
    __shared__ AttendScan scan;
    __shared__ float s_top[4], s_sum[16];
    __shared__ f4 s_acc[256];
    const int tid = threadIdx.x, h = blockIdx.x, b = blockIdx.y;
    int64_t mine;
    int run;
    const int64_t units = attend_scan(A, &scan, &mine, &run);
    if (tid == b / run) {
        for (int i = tid * run; i < b; ++i) mine += attend_units(A, i);
        scan.base = mine;
    }
    __syncthreads();
    bool bad;
    const int len = attend_len(A, b, &bad), nb = kv_units(len, A.a.window);
    if (nb == 0) return;
    const int hk = h / A.G, x = h - hk * A.G;
    const int64_t first_u = scan.base + (int64_t)(hk * A.tiles + x / kHeadTile) * nb;
    const int workers = attend_workers(A, units);
    const int w0 = kv_worker(first_u, workers, units), w1 = kv_worker(first_u + nb - 1, workers, units);
    if (w0 == w1) return;
    const int stride = kHeadTile * (A.D + 4), parts = w1 - w0 + 1;
    // the first worker's part began with the head's first unit: its second
    // slot; the others' is their first
    const float* base = A.part + (size_t)2 * w0 * stride + (size_t)(x % kHeadTile) * (A.D + 4);
    auto part = [&](int i) { return base + (size_t)(2 * i + (i == 0)) * stride; };
    float top = -__builtin_inff();
    for (int i = tid; i < parts; i += 256) top = __builtin_fmaxf(top, part(i)[0]);
    top = wave_max_uniform(top);
    if ((tid & 63) == 0) s_top[tid >> 6] = top;
    __syncthreads();
    top = __builtin_fmaxf(__builtin_fmaxf(s_top[0], s_top[1]), __builtin_fmaxf(s_top[2], s_top[3]));
    const float ref = top == -__builtin_inff() ? 0.0f : top;
    const int lanes = A.D / 4, groups = min(16, 256 / lanes), grp = tid / lanes, d = tid - grp * lanes;
    float sum = 0.0f;
    f4 o = {0, 0, 0, 0};
    if (grp < groups) {
        for (int i = grp; i < parts; i += groups) {
            const float* p = part(i);
            const float f = __builtin_amdgcn_exp2f(p[0] - ref);
            sum += p[1] * f;
            o += *(const f4*)(p + 4 + 4 * d) * f;
        }
        s_acc[tid] = o;
        if (d == 0) s_sum[grp] = sum;
    }
    __syncthreads();
    if (grp > 0) return;
    sum = 0.0f;
    o = f4{0, 0, 0, 0};
    for (int i = 0; i < groups; ++i) {
        sum += s_sum[i];
        o += s_acc[i * lanes + d];
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const size_t i = (size_t)b * A.Hq + h;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        store_any(A.a.out, A.q_type, (long long)(i * A.D + 4 * d + k), sum == 0.0f ? 0.0f : o[k] * inv);
    if (d == 0) {
        const float l2 = sum == 0.0f ? -__builtin_inff() : ref + __builtin_amdgcn_logf(sum);
        A.l2[i] = l2;
        if (A.a.lse) A.a.lse[i] = l2 * kLn2;
    }
}

// scores' = decay scores + the sum of 2^(s - l2) over a key-value head's heads
__global__ void __launch_bounds__(256) k_gather_scores(const AttendArgs A) {
    const int item = blockIdx.y, b = item / A.Hk, hk = item - b * A.Hk;
    bool bad;
    const int n = attend_len(A, b, &bad), first = kv_first_token(n, A.a.window);
    for (int t = blockIdx.x * 256 + threadIdx.x; t < n; t += gridDim.x * 256) {
        float p = 0.0f;
        if (t >= first)
            for (int g = 0; g < A.G; ++g) {
                const size_t i = (size_t)b * A.Hq + hk * A.G + g;
                const float l2 = A.l2[i];
                if (l2 != -__builtin_inff()) p += __builtin_amdgcn_exp2f(A.s[i * A.s_stride + (t - first)] - l2);
            }
        const size_t at = (size_t)item * A.cap + t;
        A.a.scores_out[at] = A.a.scores[at] * A.a.decay + p;
    }
}

constexpr int kPerCu = 2;  // workgroups of k_attend on a compute unit

int max_workers(const dq_kv_ctx* c) { return c->cus * kPerCu; }

}  // namespace

size_t dq_attend_part_floats(const dq_kv_ctx* c) {
    return (size_t)c->batch * c->Hq + 3 + (size_t)max_workers(c) * 2 * kHeadTile * (c->D + 4);
}

int dq_launch_attend(const dq_kv_ctx* c, const DqAttendArgs& a, hipStream_t s) {
    AttendArgs A{};
    A.a = a;
    A.q_type = c->q_type;
    A.Hq = c->Hq;
    A.Hk = c->Hk;
    A.D = c->D;
    A.cap = c->cap;
    A.G = c->Hq / c->Hk;
    A.tiles = (A.G + kHeadTile - 1) / kHeadTile;
    A.s = a.scores ? c->s : nullptr;
    A.s_stride = c->s_stride;
    A.part = c->part;
    A.l2 = c->part + (size_t)max_workers(c) * 2 * kHeadTile * (c->D + 4);
    A.bad = c->bad;
    A.geom = c->geom;
    // as many workers as the most units that the call can have, up to the chip's
    const int64_t per_item = kv_units(c->cap, a.window);
    const int64_t most = per_item * a.batch * A.Hk * A.tiles;
    A.workers = (int)std::min<int64_t>(most, max_workers(c));
    const AttendKernel k = c->cache_type == DQ_I8 ? attend_i8(c->q_type, c->D)
                           : c->cache_type == DQ_F16 ? attend_f16(c->q_type, c->D) : attend_bf16(c->q_type, c->D);
    hipLaunchKernelGGL(k, dim3((unsigned)A.workers), dim3(256), 0, s, A);
    DQ_LAUNCH_CHECK("attention");
    if (per_item > 1) {
        hipLaunchKernelGGL(k_attend_join, dim3((unsigned)c->Hq, (unsigned)a.batch), dim3(256), 0, s, A);
        DQ_LAUNCH_CHECK("join of the attention's parts");
    }
    if (a.scores) {
        hipLaunchKernelGGL(k_gather_scores, dim3((unsigned)((c->cap + 1023) / 1024), (unsigned)(a.batch * c->Hk)),
                           dim3(256), 0, s, A);
        DQ_LAUNCH_CHECK("gathered weights");
    }
    return DQ_OK;
}
