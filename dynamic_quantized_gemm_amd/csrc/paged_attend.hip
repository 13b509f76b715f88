// paged_attend.hip -- attention of one new token of every sequence over the
// paged key-value cache: the join of partial results with the
// gathered weights, and the launches. The attention itself is in attend_kernel.h.
#include <algorithm>

#include "attend_kernel.h"

using namespace dq;

namespace {

// Finishes a key-value head: the outputs of those query heads whose units
// several workgroups took,
//   o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,
// and the gathered weights, scores' = decay scores + the sum of 2^(s - l2) over
// the query heads. The workgroups of a key-value head share both out: query
// heads in turn, runs of 1024 tokens in turn; each finds the sums it needs
// from the parts itself, so that nothing waits for another workgroup. Parts
// are added in order, so a result never depends on timing. Bound by latency and
// its launch where no weights are gathered (4.5 to 5.6 us), else by the kept
// scores that it reads (48 sequences of up to 20479, 32 heads: 28 us).
constexpr int kFinishHeads = 64;  // query heads whose sums are kept at a time
constexpr int kMaxWorkers = 512;  // of k_attend, so the parts of a head

struct FinishParts {
    const float* base;
    int stride, count;  // count 0: the attention wrote the output itself
    __device__ __forceinline__ const float* at(int i) const {
        // the first worker's part began with the head's first unit: its
        // second slot; the others' is their first
        return base + (size_t)(2 * i + (i == 0)) * stride;
    }
};

__global__ void __launch_bounds__(256) k_attend_finish(const AttendArgs A) {
    __shared__ float s_top[4], s_sum[4], s_l2[kFinishHeads], s_f[kMaxWorkers];
    __shared__ f4 s_acc[256];
    const int tid = threadIdx.x, lane = tid & 63;
    const int item = blockIdx.y, b = item / A.Hk, hk = item - b * A.Hk;
    auto parts_of = [&](int x) {
        const int2 w = A.parts[(size_t)item * A.tiles + x / kHeadTile];
        FinishParts p;
        p.stride = kHeadTile * (A.D + 4);
        p.base = A.part + (size_t)2 * w.x * p.stride + (size_t)(x % kHeadTile) * (A.D + 4);
        p.count = w.y;
        return p;
    };
    // ---- outputs: the parts' factors once, in LDS, then groups of D / 4 lanes
    // take the parts in turn, four on their way at a time
    for (int x = blockIdx.x; x < A.G; x += gridDim.x) {
        const FinishParts p = parts_of(x);
        if (p.count == 0) continue;
        float m[2], l[2], top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = tid + 256 * k;
            m[k] = i < p.count ? p.at(i)[0] : -__builtin_inff();
            l[k] = i < p.count ? p.at(i)[1] : 0.0f;
            top = __builtin_fmaxf(top, m[k]);
        }
        top = wave_max_uniform(top);
        if (lane == 0) s_top[tid >> 6] = top;
        __syncthreads();
        top = __builtin_fmaxf(__builtin_fmaxf(s_top[0], s_top[1]), __builtin_fmaxf(s_top[2], s_top[3]));
        const float ref = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float f = __builtin_amdgcn_exp2f(m[k] - ref);
            s_f[tid + 256 * k] = f;
            sum += l[k] * f;
        }
        for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
        if (lane == 0) s_sum[tid >> 6] = sum;
        __syncthreads();
        sum = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
        const int lanes = A.D / 4, groups = min(16, 256 / lanes), grp = tid / lanes, d = tid - grp * lanes;
        f4 o = {0, 0, 0, 0};
        if (grp < groups) {
#pragma unroll 4
            for (int i = grp; i < p.count; i += groups) o += *(const f4*)(p.at(i) + 4 + 4 * d) * s_f[i];
            s_acc[tid] = o;
        }
        __syncthreads();
        if (grp == 0) {
            o = f4{0, 0, 0, 0};
            for (int i = 0; i < groups; ++i) o += s_acc[i * lanes + d];
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            const size_t at = (size_t)b * A.Hq + hk * A.G + x;
            if (sum == 0.0f) o = f4{0, 0, 0, 0};
            store4_any(A.a.out, A.q_type, at * A.D + 4 * d, o * inv);
            if (d == 0 && A.a.lse) A.a.lse[at] = (sum == 0.0f ? -__builtin_inff() : ref + __builtin_amdgcn_logf(sum)) * kLn2;
        }
        __syncthreads();
    }
    if (!A.s) return;
    // ---- gathered weights
    bool bad;
    const int len = attend_len(A, b, &bad), first = kv_first_token(len, A.a.window);
    const float* in = A.a.scores + (size_t)item * A.cap;
    float* out = A.a.scores_out + (size_t)item * A.cap;
    // the tokens before the window: vectors of four where the rows are aligned
    const int vec = (((uintptr_t)in | (uintptr_t)out) & 15) == 0 ? first & ~3 : 0;
    for (int t = (blockIdx.x * 256 + tid) * 4; t < vec; t += gridDim.x * 1024)
        *(f4*)(out + t) = *(const f4*)(in + t) * A.a.decay;
    for (int t = vec + blockIdx.x * 256 + tid; t < first; t += gridDim.x * 256) out[t] = in[t] * A.a.decay;
    if ((int)blockIdx.x * 1024 >= len - first) return;
    // whole vectors of four tokens where the caller's rows are aligned to them
    const bool wide = (((uintptr_t)(in + first) | (uintptr_t)(out + first)) & 15) == 0;
    for (int x0 = 0; x0 < A.G; x0 += kFinishHeads) {
        const int heads = min(kFinishHeads, A.G - x0);
        // a wave finds one head's sum at a time
        __syncthreads();
        for (int x = tid >> 6; x < heads; x += 4) {
            const FinishParts p = parts_of(x0 + x);
            float l2;
            if (p.count == 0) {
                l2 = A.l2[(size_t)b * A.Hq + hk * A.G + x0 + x];
            } else {
                float m[kMaxWorkers / 64], l[kMaxWorkers / 64], top = -__builtin_inff();
#pragma unroll
                for (int k = 0; k < kMaxWorkers / 64; ++k) {
                    const int i = lane + 64 * k;
                    m[k] = i < p.count ? p.at(i)[0] : -__builtin_inff();
                    l[k] = i < p.count ? p.at(i)[1] : 0.0f;
                    top = __builtin_fmaxf(top, m[k]);
                }
                top = wave_max_uniform(top);
                const float ref = top == -__builtin_inff() ? 0.0f : top;
                float sum = 0.0f;
#pragma unroll
                for (int k = 0; k < kMaxWorkers / 64; ++k) sum += l[k] * __builtin_amdgcn_exp2f(m[k] - ref);
                for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
                l2 = sum == 0.0f ? -__builtin_inff() : ref + __builtin_amdgcn_logf(sum);
            }
            // no weight at all: 2^(s - inf) = 0
            if (lane == 0) s_l2[x] = l2 == -__builtin_inff() ? __builtin_inff() : l2;
        }
        __syncthreads();
        // the first heads' pass takes the old weights, the others add to it
        const float* old = x0 == 0 ? in : out;
        const float decay = x0 == 0 ? A.a.decay : 1.0f;
        for (int r0 = blockIdx.x * 1024; r0 < len - first; r0 += gridDim.x * 1024) {
            const int r = r0 + 4 * tid, t = first + r;
            if (t >= len) break;
            const bool whole = wide && t + 4 <= len;
            f4 p;
            if (whole) {
                p = *(const f4*)(old + t);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) p[k] = t + k < len ? old[t + k] : 0.0f;
            }
            p *= decay;
            const float* s = A.s + attend_score_at(A, item, r >> 5) + x0 * 32 + (r & 31);
            f4 q = {0, 0, 0, 0};
#pragma unroll 4
            for (int x = 0; x < heads; ++x) {
                const f4 y = *(const f4*)(s + x * 32);
#pragma unroll
                for (int k = 0; k < 4; ++k) q[k] += __builtin_amdgcn_exp2f(y[k] - s_l2[x]);
            }
            p += q;
            if (whole) {
                *(f4*)(out + t) = p;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (t + k < len) out[t + k] = p[k];
            }
        }
    }
}

// Up to this many units of 128 tokens a workgroup takes a head alone rather than
// share it: always up to kWholeUnits, and up to kWholeUnitsMany where the heads
// alone fill half the chip and two workgroups fit on a compute unit. By what a
// sequence's slots, or the window, allow: the host does not know the lengths, so
// 32 of 1000 in a context of 4096 slots are shared. Microseconds
// whole and shared, 8 key-value heads of 128: 8 sequences of 250 tokens 8.4 and
// 11.7, of 500 11.8 and 12.2, of 1000 19.2 and 15.6; 32 of 1000 25.0 and 30.8, on
// int8 16.3 and 22.4; 160 of up to 1000 on int8 43.8 and 62.1; 80 of 2000 121 and
// 114. With one workgroup a unit (fp32 on 256 values) 40 of 1000 83 and 73.
constexpr int kWholeUnits = 4, kWholeUnitsMany = 8;
// With weights gathered, tokens that a sequence can hold before the window: a
// whole head decays their weights with its one workgroup, the finish with the
// chip. Whole and shared, int8, 8 heads of 128, window 512: 8 sequences of 4500
// slots 13.1 and 13.9, of 8500 15.5 and 14.3; window 1000: 32 of 4500 25.4 and
// 25.7, 64 of 4500 38.1 and 36.6; one of 131072, window 512: 73.5 and 14.5.
constexpr int kWholeBefore = 4096;

AttendKernel pick_kernel(const dq_kv_ctx* c) {
    return c->cache_type == DQ_I8 ? attend_i8(c->q_type, c->D)
           : c->cache_type == DQ_F16 ? attend_f16(c->q_type, c->D) : attend_bf16(c->q_type, c->D);
}

}  // namespace

int dq_attend_plan(dq_kv_ctx* c) {
    // two workgroups (eight waves) of a compute unit reach the memory's rate,
    // three no more, and leave more parts to join: 131071 tokens of 4 heads of
    // 128 in bf16 54 us with two, 58 with three
    int per_cu = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, (const void*)pick_kernel(c), 256, 0) != hipSuccess ||
        per_cu < 1)
        DQ_FAIL(DQ_ERR_HIP, "the attention kernel does not fit the device");
    c->attend_workers = std::min(kMaxWorkers, c->cus * std::min(per_cu, 2));
    const size_t items = (size_t)c->batch * c->Hk * ((c->Hq / c->Hk + kHeadTile - 1) / kHeadTile);
    c->part_floats = (size_t)c->attend_workers * 2 * kHeadTile * (c->D + 4) + 2 * items + (size_t)c->batch * c->Hq;
    return DQ_OK;
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
    A.parts = (int2*)(c->part + (size_t)c->attend_workers * 2 * kHeadTile * (c->D + 4));
    A.l2 = (float*)(A.parts + (size_t)a.batch * A.Hk * A.tiles);
    A.bad = c->bad;
    A.geom = c->geom;
    const size_t es = kv_elem_bytes(c->q_type);
    A.q_vec = (uintptr_t)a.q % 16 == 0 && a.q_ts * es % 16 == 0 && a.q_hs * es % 16 == 0;
    // as many workers as the most units that the call can have, up to the chip's
    const int64_t per_item = kv_units(c->cap, a.window);
    const int64_t items = (int64_t)a.batch * A.Hk * A.tiles;
    // Short sequences are not split: a workgroup takes whole items, finishes
    // them itself and looks up no other sequence's length.
    const bool many = items >= c->cus / 2 && c->attend_workers > c->cus;
    const int before = a.window > 0 ? std::max(0, c->cap - a.window) : 0;
    A.whole = per_item <= (many ? kWholeUnitsMany : kWholeUnits) &&
              (!a.scores || (A.tiles == 1 && before <= kWholeBefore));
    A.workers = (int)std::min<int64_t>(A.whole ? items : per_item * items, c->attend_workers);
    hipLaunchKernelGGL(pick_kernel(c), dim3((unsigned)A.workers), dim3(256), 0, s, A);
    DQ_LAUNCH_CHECK("attention");
    if (!A.whole) {
        const int chunks = a.scores ? (c->cap + 1023) / 1024 : 0;
        const int gx = std::max(std::min(A.G, 16), std::min(chunks, std::max(1, 8192 / (a.batch * c->Hk))));
        hipLaunchKernelGGL(k_attend_finish, dim3((unsigned)gx, (unsigned)(a.batch * c->Hk)), dim3(256), 0, s, A);
        DQ_LAUNCH_CHECK("finish of the attention");
    }
    return DQ_OK;
}
