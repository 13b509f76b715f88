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
    int32_t* counts = nullptr;  // [chunks][experts]: rows, then the first row, of each chunk's tokens
    char info[192] = "";
};

namespace {

using namespace dq;

constexpr int kChunk = 64;                           // tokens whose rows one workgroup places
constexpr int kPerLane = DQ_MOE_EXPERTS_MAX / 64;    // logits of a token that a lane holds

struct RouteArgs {
    const void* logits;
    long long stride;
    int32_t* ids;
    float* weights;
    int32_t* offsets;
    int32_t* row_token;
    int32_t* row_of;
    int32_t* counts;
    int tokens, experts, top_k, chunks, type, sigmoid, normalize;
    float scale;
};

__device__ __forceinline__ float logit(const RouteArgs& A, long long t, int e) {
    const long long i = t * A.stride + e;
    if (A.type == DQ_F32) return static_cast<const float*>(A.logits)[i];
    const uint16_t b = static_cast<const uint16_t*>(A.logits)[i];
    return A.type == DQ_BF16 ? bf16_bits_to_f32(b) : (float)__builtin_bit_cast(_Float16, b);
}

// A wave a token; four tokens at a time, kChunk a workgroup.
__global__ void __launch_bounds__(256) k_moe_choose(RouteArgs A) {
    __shared__ int s_count[DQ_MOE_EXPERTS_MAX];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int e = threadIdx.x; e < A.experts; e += 256) s_count[e] = 0;
    __syncthreads();
    const int end = min(A.tokens, (int)(blockIdx.x + 1) * kChunk);
    for (int t = blockIdx.x * kChunk + wave; t < end; t += 4) {
        float v[kPerLane];
        float high = -__builtin_inff(), all = 0.0f;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            const int e = lane + i * 64;
            v[i] = e < A.experts ? logit(A, t, e) : -__builtin_inff();
            high = __builtin_fmaxf(high, v[i]);
        }
        for (int o = 32; o; o >>= 1) high = __builtin_fmaxf(high, __shfl_xor(high, o));
        if (!(high > -__builtin_inff())) high = 0.0f;
        if (!A.sigmoid) {
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) all += expf(v[i] - high);  // a NaN stays one
            for (int o = 32; o; o >>= 1) all += __shfl_xor(all, o);
        }
        int id = -1;
        float part = 0.0f, sum = 0.0f;
        for (int j = 0; j < A.top_k; ++j) {
            float best = -__builtin_inff();
            int at = INT32_MAX;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i)
                if (v[i] > best) {
                    best = v[i];
                    at = lane + i * 64;
                }
            for (int o = 32; o; o >>= 1) {
                const float b = __shfl_xor(best, o);
                const int a = __shfl_xor(at, o);
                if (b > best || (b == best && a < at)) {
                    best = b;
                    at = a;
                }
            }
            if (at == INT32_MAX) break;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i)
                if (at == lane + i * 64) v[i] = -__builtin_inff();
            const float p = A.sigmoid ? 1.0f / (1.0f + expf(-best)) : expf(best - high);
            sum += p;
            if (lane == j) {
                id = at;
                part = p;
            }
        }
        if (lane < A.top_k) {
            const float total = A.normalize ? sum + (A.sigmoid ? 0.0f : all * 0.0f) : A.sigmoid ? 1.0f : all;
            A.ids[(size_t)t * A.top_k + lane] = id;
            A.weights[(size_t)t * A.top_k + lane] = id < 0 ? 0.0f : part / total * A.scale;
            if (id >= 0) atomicAdd(&s_count[id], 1);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < A.experts; e += 256) A.counts[(size_t)blockIdx.x * A.experts + e] = s_count[e];
}

// Counts to first rows, one workgroup: every expert's total, their prefix sum,
// then each expert's chunks in their order.
__global__ void __launch_bounds__(1024) k_moe_scan(RouteArgs A) {
    __shared__ int s_total[1024];
    const int e = threadIdx.x;
    int total = 0;
    if (e < A.experts)
        for (int c = 0; c < A.chunks; ++c) total += A.counts[(size_t)c * A.experts + e];
    s_total[e] = total;
    __syncthreads();
    for (int o = 1; o < 1024; o <<= 1) {
        const int v = e >= o ? s_total[e - o] : 0;
        __syncthreads();
        s_total[e] += v;
        __syncthreads();
    }
    if (e >= A.experts) return;
    int at = s_total[e] - total;
    A.offsets[e] = at;
    if (e == A.experts - 1) A.offsets[e + 1] = s_total[e];
    for (int c = 0; c < A.chunks; ++c) {
        const size_t i = (size_t)c * A.experts + e;
        const int n = A.counts[i];
        A.counts[i] = at;
        at += n;
    }
}

// The rows of a chunk's tokens: a thread an expert walks the chunk's pairs.
__global__ void __launch_bounds__(256) k_moe_place(RouteArgs A) {
    extern __shared__ int s_ids[];
    const int first = blockIdx.x * kChunk, n = (min(A.tokens, first + kChunk) - first) * A.top_k;
    const size_t base = (size_t)first * A.top_k;
    for (int i = threadIdx.x; i < n; i += 256) {
        s_ids[i] = A.ids[base + i];
        if (s_ids[i] < 0) A.row_of[base + i] = -1;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < A.experts; e += 256) {
        int row = A.counts[(size_t)blockIdx.x * A.experts + e];
        for (int i = 0; i < n; ++i)
            if (s_ids[i] == e) {
                A.row_token[row] = first + i / A.top_k;
                A.row_of[base + i] = row++;
            }
    }
}

struct CombineArgs {
    const void* y;
    const float* weights;
    const int32_t* row_of;
    const void* add;
    void* out;
    int tokens, top_k, rows, y_type, out_type;
    long long N;
};

__device__ __forceinline__ float load1(const void* p, size_t i, int type) {
    if (type == DQ_F32) return static_cast<const float*>(p)[i];
    const uint16_t b = static_cast<const uint16_t*>(p)[i];
    return type == DQ_BF16 ? bf16_bits_to_f32(b) : (float)__builtin_bit_cast(_Float16, b);
}

__global__ void __launch_bounds__(256) k_moe_combine(CombineArgs A) {
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (size_t)A.tokens * A.N) return;
    const size_t t = i / A.N, n = i % A.N;
    float v = A.add ? load1(A.add, i, A.out_type) : 0.0f;
    for (int j = 0; j < A.top_k; ++j) {
        const int r = A.row_of[t * A.top_k + j];
        if (r < 0) continue;
        v += r < A.rows ? A.weights[t * A.top_k + j] * load1(A.y, (size_t)r * A.N + n, A.y_type) : __builtin_nanf("");
    }
    if (A.out_type == DQ_F32) static_cast<float*>(A.out)[i] = v;
    else if (A.out_type == DQ_BF16) static_cast<uint16_t*>(A.out)[i] = (uint16_t)f32_to_bf16_bits(v);
    else static_cast<_Float16*>(A.out)[i] = (_Float16)v;
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
    if (hipMalloc(&c->counts, chunks * experts * 4) != hipSuccess) {
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
    A.tokens = (int)tokens;
    A.experts = ctx->experts;
    A.top_k = ctx->top_k;
    A.chunks = (int)((tokens + kChunk - 1) / kChunk);
    A.type = ctx->logits_type;
    A.sigmoid = ctx->scoring == DQ_MOE_SIGMOID;
    A.normalize = ctx->normalize;
    A.scale = ctx->scale;
    const hipStream_t s = (hipStream_t)stream;
    if (tokens) {
        hipLaunchKernelGGL(k_moe_choose, dim3(A.chunks), dim3(256), 0, s, A);
        DQ_LAUNCH_CHECK("choice of experts");
    }
    hipLaunchKernelGGL(k_moe_scan, dim3(1), dim3(1024), 0, s, A);
    DQ_LAUNCH_CHECK("experts' offsets");
    if (tokens) {
        hipLaunchKernelGGL(k_moe_place, dim3(A.chunks), dim3(256), kChunk * ctx->top_k * 4, s, A);
        DQ_LAUNCH_CHECK("experts' rows");
    }
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
    if (N > DQ_W4_N_MAX || (tokens * N + 255) / 256 > INT32_MAX) DQ_FAIL(DQ_ERR_RANGE, "too many elements for one launch");
    CombineArgs A{y, weights, row_of, add, out, (int)tokens, ctx->top_k, (int)rows, y_type, out_type, N};
    hipLaunchKernelGGL(k_moe_combine, dim3((unsigned)((tokens * N + 255) / 256)), dim3(256), 0, (hipStream_t)stream, A);
    DQ_LAUNCH_CHECK("sum of the experts' results");
    return DQ_OK;
}

extern "C" const char* dq_moe_info(const dq_moe_ctx* ctx) { return ctx ? ctx->info : nullptr; }

extern "C" void dq_moe_release(dq_moe_ctx* ctx) {
    if (!ctx) return;
    (void)hipFree(ctx->counts);
    delete ctx;
}
