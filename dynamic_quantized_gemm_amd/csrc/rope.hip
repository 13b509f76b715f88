// rope.hip -- rotary positions with several axes.
//
// Pair i of a token's head turns by the angle pos[axis(i)] * inv_freq[i]:
//   (a, b) -> (a cos - b sin, b cos + a sin),
// and by the opposite angle for the inverse, which is also the gradient's
// pass (the rotation is orthogonal). Elements past the rotated part pass
// through unchanged.
//
// Bound by the traffic of x and y. A thread keeps the cosines and sines of VP
// pairs in registers and walks heads with them, so x is read and y written
// once, VP elements (up to 16 bytes) at a time. Where several threads share a
// token and pairs, the workgroup computes the angles once, in LDS. 8205 tokens
// of 40 heads of 128 in bf16: 28.1 us, 6.0 TB/s; a plain copy of as much takes
// 29 to 30 us.
#include <math.h>
#include <stdio.h>

#include <algorithm>
#include <new>

#include "paged_kv.h"

using namespace dq;

namespace {

struct RopeArgs {
    const void* x;
    void* y;
    const int32_t* pos;
    const double2* freq;
    const int32_t* axis;
    long long xt, xh, yt, yh;
    uint32_t threads;  // tokens * chunks * lanes
    int tokens, heads, D, R, inverse;
    int shared;        // angles are computed once a workgroup
    KvDiv lanes, chunks;
};

constexpr int kRopeHeads = 4;  // heads of a thread, all on their way at a time

template <int TYPE, int VP, bool IL>
__global__ void __launch_bounds__(256) k_rope(const RopeArgs A) {
    typedef typename Elem<TYPE>::S S;
    extern __shared__ float2 tab[];
    const uint32_t id0 = blockIdx.x * 256u, last = min(id0 + 255u, A.threads - 1);
    const uint32_t id = min(id0 + threadIdx.x, last);
    const uint32_t rest = kv_div(id, A.lanes);
    const int i0 = (int)(id - rest * A.lanes.d) * VP;
    const uint32_t t = kv_div(rest, A.chunks);
    // heads h0, h0 + step, ..: neighbouring threads take neighbouring heads
    const int h0 = (int)(rest - t * A.chunks.d), step = (int)A.chunks.d;
    const bool turn = i0 < A.R / 2;
    int lo, hi;
    kv_pair(i0, A.D, A.R, IL, &lo, &hi);
    const S* x = (const S*)A.x + t * A.xt;
    S* y = (S*)A.y + t * A.yt;
    // the heads are on their way while the angles are computed
    float a[kRopeHeads][VP], b[kRopeHeads][VP];
#pragma unroll
    for (int k = 0; k < kRopeHeads; ++k)
        load_pairs<S, VP, IL>(x + (h0 + k * step < A.heads ? h0 + k * step : h0) * A.xh, lo, hi, a[k], b[k]);
    issue_fence();
    float c[VP], s[VP];
    if (A.shared) {
        const int t0 = (int)kv_div(kv_div(id0, A.lanes), A.chunks), t1 = (int)kv_div(kv_div(last, A.lanes), A.chunks);
        rope_table(tab, t0, t1 - t0 + 1, A.R / 2, A.pos, A.tokens, A.freq, A.axis, A.inverse);
        if (turn) {
#pragma unroll
            for (int i = 0; i < VP; ++i) {
                const float2 cs = tab[((int)t - t0) * (A.R / 2) + i0 + i];
                c[i] = cs.x;
                s[i] = cs.y;
            }
        }
    } else if (turn) {
#pragma unroll
        for (int i = 0; i < VP; ++i) {
            rope_cos_sin(A.pos[(size_t)A.axis[i0 + i] * A.tokens + t], A.freq[i0 + i], &c[i], &s[i]);
            if (A.inverse) s[i] = -s[i];
        }
    }
    if (id0 + threadIdx.x > last) return;
#pragma unroll
    for (int k = 0; k < kRopeHeads; ++k) {
        if (turn) {
#pragma unroll
            for (int i = 0; i < VP; ++i) {
                const float u = a[k][i] * c[i] - b[k][i] * s[i];
                b[k][i] = b[k][i] * c[i] + a[k][i] * s[i];
                a[k][i] = u;
            }
        }
        if (h0 + k * step < A.heads) store_pairs<S, VP, IL>(y + (h0 + k * step) * A.yh, lo, hi, a[k], b[k]);
    }
}

// the largest number of pairs a thread can take: the vectors of VP (or, for
// neighbouring pairs, 2 VP) elements have to be aligned in x and y and must
// not straddle the end of the rotated part
int pick_vp(const dq_rope_ctx* c, size_t es, const void* x, const void* y, const long long* strides) {
    for (int vp = 16 / (int)es; vp > 1; vp /= 2) {
        const int elems = c->interleaved ? 2 * vp : vp;
        const size_t bytes = elems * es;
        if (bytes > 16) continue;
        bool ok = (c->R / 2) % vp == 0 && (c->D - c->R) / 2 % vp == 0;
        if (c->interleaved) ok = ok && c->R % (2 * vp) == 0 && c->D % (2 * vp) == 0;
        ok = ok && (uintptr_t)x % bytes == 0 && (uintptr_t)y % bytes == 0;
        for (int i = 0; i < 4; ++i) ok = ok && strides[i] % elems == 0;
        if (ok) return vp;
    }
    return 1;
}

template <int TYPE, int VP>
void launch(const RopeArgs& A, size_t lds, bool il, hipStream_t s) {
    const dim3 grid((A.threads + 255) / 256), block(256);
    if constexpr (2 * VP * sizeof(typename Elem<TYPE>::S) <= 16) {
        if (il) {
            hipLaunchKernelGGL((k_rope<TYPE, VP, true>), grid, block, lds, s, A);
            return;
        }
    }
    hipLaunchKernelGGL((k_rope<TYPE, VP, false>), grid, block, lds, s, A);
}

template <int TYPE>
void launch_type(const RopeArgs& A, size_t lds, int vp, bool il, hipStream_t s) {
    switch (vp) {
        case 8:
            if constexpr (TYPE != DQ_F32) launch<TYPE, 8>(A, lds, il, s);
            break;
        case 4: launch<TYPE, 4>(A, lds, il, s); break;
        case 2: launch<TYPE, 2>(A, lds, il, s); break;
        default: launch<TYPE, 1>(A, lds, il, s); break;
    }
}

}  // namespace

int dq_rope_check_device(const dq_rope_ctx* c) {
    int dev = 0;
    (void)hipGetDevice(&dev);
    if (dev != c->device) DQ_FAIL(DQ_ERR_STATE, "the context belongs to another device");
    return DQ_OK;
}

extern "C" int dq_rope_init(dq_rope_ctx** ctx, int head_dim, int rotary_dim, const int32_t* axis_of_pair,
                            const double* inv_freq, int interleaved) {
    if (!ctx) DQ_FAIL(DQ_ERR_ARG, "ctx is NULL");
    *ctx = nullptr;
    if (head_dim < 2 || head_dim % 2 || rotary_dim < 2 || rotary_dim % 2 || rotary_dim > head_dim)
        DQ_FAIL(DQ_ERR_ARG, "head_dim and rotary_dim must be even, 2 <= rotary_dim <= head_dim");
    if (head_dim > DQ_ROPE_DIM_MAX) DQ_FAIL(DQ_ERR_RANGE, "head_dim exceeds %d", DQ_ROPE_DIM_MAX);
    if (!axis_of_pair || !inv_freq) DQ_FAIL(DQ_ERR_ARG, "axis_of_pair and inv_freq must not be NULL");
    const int P = rotary_dim / 2;
    int axes = 1;
    for (int i = 0; i < P; ++i) {
        if (axis_of_pair[i] < 0 || axis_of_pair[i] >= DQ_ROPE_AXES_MAX)
            DQ_FAIL(DQ_ERR_RANGE, "axis %d of pair %d is outside [0, %d)", axis_of_pair[i], i, DQ_ROPE_AXES_MAX);
        if (!isfinite(inv_freq[i]) || fabs(inv_freq[i]) > 1e9)
            DQ_FAIL(DQ_ERR_ARG, "inv_freq of pair %d is not finite or beyond 1e9", i);
        axes = std::max(axes, axis_of_pair[i] + 1);
    }
    double2 freq[DQ_ROPE_DIM_MAX / 2];
    for (int i = 0; i < P; ++i) kv_turns(inv_freq[i], &freq[i].x, &freq[i].y);
    dq_rope_ctx* c = new (std::nothrow) dq_rope_ctx();
    if (!c) DQ_FAIL(DQ_ERR_ALLOC, "host allocation for the rotary context failed");
    (void)hipGetDevice(&c->device);
    c->D = head_dim;
    c->R = rotary_dim;
    c->axes = axes;
    c->interleaved = interleaved ? 1 : 0;
    if (hipMalloc(&c->freq, P * sizeof(double2)) != hipSuccess || hipMalloc(&c->axis, P * 4) != hipSuccess) {
        dq_rope_release(c);
        DQ_FAIL(DQ_ERR_ALLOC, "device allocation for the rotary context failed");
    }
    if (hipMemcpy(c->freq, freq, P * sizeof(double2), hipMemcpyHostToDevice) != hipSuccess ||
        hipMemcpy(c->axis, axis_of_pair, P * 4, hipMemcpyHostToDevice) != hipSuccess) {
        dq_rope_release(c);
        DQ_FAIL(DQ_ERR_HIP, "copy of the rotary frequencies failed");
    }
    snprintf(c->info, sizeof c->info, "gfx950 rotary positions: %d of %d elements, %d axes, pairs of %s", rotary_dim, head_dim,
             axes, interleaved ? "neighbours" : "halves");
    *ctx = c;
    return DQ_OK;
}

extern "C" int dq_rope_forward(const dq_rope_ctx* ctx, const void* x, dq_dtype type, int64_t tokens, int heads,
                               int64_t x_token_stride, int64_t x_head_stride, const int32_t* positions, void* y,
                               int64_t y_token_stride, int64_t y_head_stride, int inverse, void* stream) {
    if (!ctx) DQ_FAIL(DQ_ERR_STATE, "no context");
    if (type != DQ_F32 && type != DQ_BF16 && type != DQ_F16) DQ_FAIL(DQ_ERR_TYPE, "x must be fp32, bf16 or fp16");
    if (tokens < 0 || heads < 0) DQ_FAIL(DQ_ERR_ARG, "negative sizes");
    if (tokens == 0 || heads == 0) return DQ_OK;
    if (!x || !y || !positions) DQ_FAIL(DQ_ERR_ARG, "x, y and positions must not be NULL");
    const size_t es = kv_elem_bytes(type);
    if ((uintptr_t)x % es || (uintptr_t)y % es || (uintptr_t)positions % 4)
        DQ_FAIL(DQ_ERR_ARG, "a tensor is not aligned to its elements");
    if (x == y && (x_token_stride != y_token_stride || x_head_stride != y_head_stride))
        DQ_FAIL(DQ_ERR_ARG, "in place the strides of x and y must be the same");
    if (tokens > INT32_MAX) DQ_FAIL(DQ_ERR_RANGE, "too many tokens for one launch");
    if (int rc = dq_rope_check_device(ctx)) return rc;
    RopeArgs A{};
    A.x = x;
    A.y = y;
    A.pos = positions;
    A.freq = ctx->freq;
    A.axis = ctx->axis;
    A.xt = x_token_stride;
    A.xh = x_head_stride;
    A.yt = y_token_stride;
    A.yh = y_head_stride;
    A.heads = heads;
    A.D = ctx->D;
    A.R = ctx->R;
    A.inverse = inverse ? 1 : 0;
    const long long st[4] = {A.xt, A.xh, A.yt, A.yh};
    const int vp = pick_vp(ctx, es, x, y, st);
    const int64_t lanes = ctx->D / 2 / vp;
    // heads per thread: as many as leave the chip filled (2^18 threads), at most
    // 4 (8205 x 40 heads of 128 in bf16: 29.5 us when chosen, with 8 32.5, with 32 34.8)
    int chunk = 1;
    while (chunk < kRopeHeads && chunk < heads && tokens * ((heads - 1) / (2 * chunk) + 1) * lanes >= (1 << 18))
        chunk *= 2;
    const int64_t chunks = (heads - 1) / chunk + 1;
    if (tokens * chunks > INT32_MAX || tokens * chunks * lanes > (int64_t)UINT32_MAX - 256)
        DQ_FAIL(DQ_ERR_RANGE, "too many tokens for one launch");
    A.tokens = (int)tokens;
    A.lanes = make_kvdiv((uint32_t)lanes);
    A.chunks = make_kvdiv((uint32_t)chunks);
    A.threads = (uint32_t)(tokens * chunks * lanes);
    // tokens that 256 threads can touch; from two threads a token and pairs on
    // the table pays (at 8 heads a thread 32.5 us with it, 34.4 without)
    A.shared = chunks > 1;
    const size_t lds = A.shared ? (size_t)(254 / (lanes * chunks) + 2) * (ctx->R / 2) * sizeof(float2) : 0;
    const hipStream_t s = (hipStream_t)stream;
    const bool il = ctx->interleaved;
    if (type == DQ_F32) launch_type<DQ_F32>(A, lds, vp, il, s);
    else if (type == DQ_BF16) launch_type<DQ_BF16>(A, lds, vp, il, s);
    else launch_type<DQ_F16>(A, lds, vp, il, s);
    DQ_LAUNCH_CHECK("rotary positions");
    return DQ_OK;
}

extern "C" const char* dq_rope_info(const dq_rope_ctx* ctx) { return ctx ? ctx->info : nullptr; }

extern "C" void dq_rope_release(dq_rope_ctx* ctx) {
    if (!ctx) return;
    (void)hipFree(ctx->freq);
    (void)hipFree(ctx->axis);
    delete ctx;
}
