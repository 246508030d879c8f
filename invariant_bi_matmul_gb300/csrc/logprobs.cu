// logprobs.cu -- log-probabilities of given tokens with entropy and top alternatives, and
// their gradient (include/bi_rowwise.h).
//
// Simple form: one CTA of 1024 threads per row that streams the row once per pass.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "bi.h"
#include "bi_rowwise.h"
#include "common.cuh"
#include "launch.h"

#define BI_EXPORT extern "C" __attribute__((visibility("default")))

namespace bi {

void set_last_error_message(const char* msg);

namespace {

constexpr int T = 1024;

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    if (DT == BI_F32) return static_cast<const float*>(p)[i];
    const uint16_t h = static_cast<const uint16_t*>(p)[i];
    return widen16(h, DT == BI_F16);
}

// Whole-number order of a value and its index: larger values first, then lower indices; NaN
// below every number.  +0 and -0 are one value.
__device__ __forceinline__ unsigned long long order_key(float x, int i) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    const uint32_t o = isnan(x) ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
    return (uint64_t(o) << 32) | uint32_t(0x7fffffff - i);
}

template <class F, class V>
__device__ __forceinline__ V block_fold(V v, V* scratch, F f) {
    for (int off = 16; off > 0; off >>= 1) v = f(v, __shfl_xor_sync(~0u, v, off));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = scratch[threadIdx.x & 31];
    for (int off = 16; off > 0; off >>= 1) v = f(v, __shfl_xor_sync(~0u, v, off));
    return v;
}

template <int DT>
__global__ void __launch_bounds__(T)
token_logprobs_kernel(const void* __restrict__ x, int64_t ldx, const int32_t* __restrict__ tokens,
                      int n, float* logp, float* entropy, float* lse_out, int top, float* top_logp,
                      int32_t* top_ids, unsigned int* err) {
    __shared__ float red[32];
    __shared__ unsigned long long redk[32];
    pdl_wait();
    pdl_trigger();
    const int64_t r = blockIdx.x;
    const void* xr = static_cast<const char*>(x) + size_t(r) * size_t(ldx) * (DT == BI_F32 ? 4 : 2);
    auto fmx = [](float a, float b) { return fmaxf(a, b); };
    auto add = [](float a, float b) { return a + b; };
    float m = -INFINITY;
    bool nan = false;
    for (int i = threadIdx.x; i < n; i += T) {
        const float v = load1<DT>(xr, i);
        nan |= isnan(v);
        m = fmaxf(m, v);
    }
    m = block_fold(m, red, fmx);
    nan = __syncthreads_or(nan);
    float s = 0.f, w = 0.f;
    for (int i = threadIdx.x; i < n; i += T) {
        const float d = load1<DT>(xr, i) - m;
        const float e = expf(d);
        s += e;
        if (e > 0.f) w += e * d;
    }
    s = block_fold(s, red, add);
    w = block_fold(w, red, add);
    const bool bad = nan || !isfinite(m);
    const float ls = bad ? __int_as_float(0x7fc00000) : logf(s);
    if (threadIdx.x == 0) {
        const int t = tokens[r];
        if (t >= 0 && t < n) {
            logp[r] = (load1<DT>(xr, t) - m) - ls;
        } else if (t == -1) {
            logp[r] = 0.f;
        } else {
            latch_error(err, kErrDeviceArg);
            logp[r] = __int_as_float(0x7fc00000);
        }
        if (entropy) entropy[r] = ls - w / s;
        if (lse_out) lse_out[r] = m + ls;
    }
    unsigned long long last = ~0ull;
    auto mx = [](unsigned long long a, unsigned long long b) { return a > b ? a : b; };
    for (int k = 0; k < top; ++k) {
        unsigned long long best = 0;
        for (int i = threadIdx.x; i < n; i += T) {
            const unsigned long long key = order_key(load1<DT>(xr, i), i);
            if (key < last && key > best) best = key;
        }
        last = block_fold(best, redk, mx);
        if (threadIdx.x == 0) {
            const int i = 0x7fffffff - int(uint32_t(last));
            top_ids[r * top + k] = i;
            top_logp[r * top + k] = (load1<DT>(xr, i) - m) - ls;
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(256)
token_logprobs_backward_kernel(const void* x, int64_t ldx, const int32_t* __restrict__ tokens,
                               int64_t rows, int n, const float* __restrict__ lse,
                               const float* __restrict__ entropy, const float* __restrict__ g_logp,
                               const float* __restrict__ g_entropy, void* dx, int64_t lddx,
                               unsigned int* err) {
    pdl_wait();
    pdl_trigger();
    const size_t es = DT == BI_F32 ? 4 : 2;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const void* xr = static_cast<const char*>(x) + size_t(r) * size_t(ldx) * es;
        char* dr = static_cast<char*>(dx) + size_t(r) * size_t(lddx) * es;
        const int t = tokens[r];
        if (blockIdx.x == 0 && threadIdx.x == 0 && (t < -1 || t >= n)) latch_error(err, kErrDeviceArg);
        const float gl = g_logp && t >= 0 && t < n ? g_logp[r] : 0.f;
        const float ge = g_entropy ? g_entropy[r] : 0.f;
        const float ls = lse[r], H = entropy ? entropy[r] : 0.f;
        for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
            const float lp = load1<DT>(xr, i) - ls;
            const float p = expf(lp);
            float d = p == 0.f ? 0.f : -p * (gl + ge * (lp + H));
            if (i == t) d += gl;
            if (DT == BI_F32)
                reinterpret_cast<float*>(dr)[i] = d;
            else
                reinterpret_cast<uint16_t*>(dr)[i] = round16(d, DT == BI_F16);
        }
    }
}

bi_status fail(bi_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_last_error_message(buf);
    return s;
}

bi_status launched(cudaError_t e, const char* fn) {
    if (e == cudaSuccess) return BI_OK;
    return fail(BI_ERR_CUDA, "%s: launch: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
}

constexpr int64_t kI32Max = 0x7fffffffLL;

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// What both entry points check of the logits.
bi_status check_rows(const char* fn, int dtype, int64_t rows, int64_t n, int64_t ldx) {
    if (dtype != BI_BF16 && dtype != BI_F16 && dtype != BI_F32)
        return fail(BI_ERR_INVALID_ARG, "%s: x_dtype must be BI_BF16, BI_F16 or BI_F32", fn);
    if (rows < 0 || n < 1 || n > kI32Max - 4)
        return fail(BI_ERR_INVALID_ARG, "%s: need rows >= 0 and 1 <= n < 2^31", fn);
    if (ldx < n) return fail(BI_ERR_INVALID_ARG, "%s: ldx < n", fn);
    if (rows > kI32Max) return fail(BI_ERR_UNSUPPORTED, "%s: too many rows", fn);
    return BI_OK;
}

}  // namespace
}  // namespace bi

using namespace bi;

BI_EXPORT bi_status bi_token_logprobs(const void* x, int64_t ldx, int x_dtype,
                                      const int32_t* tokens, int64_t rows, int64_t n, float* logp,
                                      float* entropy, float* lse, int64_t top, float* top_logp,
                                      int32_t* top_ids, bi_stream_t stream) {
    const char* fn = "bi_token_logprobs";
    bi_status st = check_rows(fn, x_dtype, rows, n, ldx);
    if (st != BI_OK) return st;
    if (top < 0 || top > BI_LOGPROBS_MAX_TOP || top > n)
        return fail(BI_ERR_INVALID_ARG, "%s: top must be in [0, min(n, %d)]", fn,
                    BI_LOGPROBS_MAX_TOP);
    if (rows == 0) return BI_OK;
    if (!x || !tokens || !logp || (top > 0 && (!top_logp || !top_ids)))
        return fail(BI_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(x, x_dtype == BI_F32 ? 4 : 2) || !aligned(tokens, 4) || !aligned(logp, 4) ||
        !aligned(entropy, 4) || !aligned(lse, 4) || !aligned(top_logp, 4) || !aligned(top_ids, 4))
        return fail(BI_ERR_INVALID_ARG, "%s: pointers not element-aligned", fn);
    cudaError_t why = cudaSuccess;
    const DeviceInfo* dev = current_device_info(&why);
    if (!dev) return launched(why, fn);
    auto kern = x_dtype == BI_F32   ? token_logprobs_kernel<BI_F32>
                : x_dtype == BI_F16 ? token_logprobs_kernel<BI_F16>
                                    : token_logprobs_kernel<BI_BF16>;
    return launched(launch_pdl(kern, dim3(unsigned(rows)), dim3(T), 0,
                               reinterpret_cast<cudaStream_t>(stream), x, ldx, tokens, int(n), logp,
                               entropy, lse, int(top), top_logp, top_ids, dev->err_word),
                    fn);
}

BI_EXPORT bi_status bi_token_logprobs_backward(const void* x, int64_t ldx, int x_dtype,
                                               const int32_t* tokens, int64_t rows, int64_t n,
                                               const float* lse, const float* entropy,
                                               const float* g_logp, const float* g_entropy,
                                               void* dx, int64_t lddx, bi_stream_t stream) {
    const char* fn = "bi_token_logprobs_backward";
    bi_status st = check_rows(fn, x_dtype, rows, n, ldx);
    if (st != BI_OK) return st;
    if (lddx < n) return fail(BI_ERR_INVALID_ARG, "%s: lddx < n", fn);
    if (rows == 0) return BI_OK;
    if (!x || !tokens || !lse || !dx) return fail(BI_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!g_logp && !g_entropy)
        return fail(BI_ERR_INVALID_ARG, "%s: g_logp and g_entropy are both null", fn);
    if (g_entropy && !entropy)
        return fail(BI_ERR_INVALID_ARG, "%s: g_entropy needs the forward's entropy", fn);
    if (dx == x && lddx != ldx)
        return fail(BI_ERR_INVALID_ARG, "%s: in place, lddx must be ldx", fn);
    const size_t es = x_dtype == BI_F32 ? 4 : 2;
    if (!aligned(x, es) || !aligned(dx, es) || !aligned(tokens, 4) || !aligned(lse, 4) ||
        !aligned(entropy, 4) || !aligned(g_logp, 4) || !aligned(g_entropy, 4))
        return fail(BI_ERR_INVALID_ARG, "%s: pointers not element-aligned", fn);
    cudaError_t why = cudaSuccess;
    const DeviceInfo* dev = current_device_info(&why);
    if (!dev) return launched(why, fn);
    auto kern = x_dtype == BI_F32   ? token_logprobs_backward_kernel<BI_F32>
                : x_dtype == BI_F16 ? token_logprobs_backward_kernel<BI_F16>
                                    : token_logprobs_backward_kernel<BI_BF16>;
    const int64_t per_row = (n + 4095) / 4096;
    return launched(launch_pdl(kern, dim3(unsigned(per_row), unsigned(rows < 65535 ? rows : 65535)),
                               dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), x, ldx, tokens,
                               rows, int(n), lse, entropy, g_logp, g_entropy, dx, lddx,
                               dev->err_word),
                    fn);
}
