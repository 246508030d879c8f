// logprobs.cu -- log-probabilities of given tokens with entropy and top alternatives, and
// their gradient (include/bi_rowwise.h).
//
// Forward.  With m a maximum and d_i = x_i - m:  s = sum exp(d_i),  w = sum exp(d_i) d_i,
// logp = (x_t - m) - log s,  entropy = log s - w / s.  A row is cut into P parts (P <= 8, of
// 16,384 elements where that is enough), one CTA each, the CTAs of a row in one cluster:
//   * the part is copied into shared memory by bulk copies, in four pieces with a barrier each;
//     thread t takes the 4-element groups t, t + T, ... and finds its maximum as they land;
//   * s and w against the part's maximum, from shared memory, ascending in the thread, then a
//     butterfly in each warp and the warps in ascending order;
//   * the parts' (m, s, w) are combined in ascending order by rank 0, w moved to the common
//     maximum by w + s (m_p - M).
// The tree is a function of n alone.  One read of the row; several CTAs share an SM, so one's
// copy runs under another's arithmetic.  Rows whose parts do not fit in shared memory are read
// from global memory once per step, with the same arithmetic.
//
// Top alternatives.  The k-th largest of the T thread maxima bounds the part's k-th largest
// element from below, so few elements (k, and a handful more) lie at or above it; they are
// gathered with their indices, ranked by counting, and the parts' first k ranked again by rank
// 0.  Where ties make them too many, k rounds of a maximum below the last one found.
//
// Backward.  Elementwise from the saved lse and entropy: one read, one write.
//
// Both are bound by memory: rows * n * size bytes, twice that for the gradient.
#include <algorithm>
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

constexpr int kMaxParts = 8;
constexpr int64_t kPart = 16384;       // elements of a part, while eight parts are enough
constexpr int kPieces = 4;             // bulk copies (and barriers) of a part
constexpr int kList = 512;             // candidates gathered for the top entries
constexpr size_t kMaxStage = 200 * 1024;  // bytes of a part that is staged in shared memory
constexpr float kNaN = __builtin_nanf("");

template <int DT>
constexpr int kSize = DT == BI_F32 ? 4 : 2;

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    if (DT == BI_F32) return static_cast<const float*>(p)[i];
    return widen16(static_cast<const uint16_t*>(p)[i], DT == BI_F16);
}

// Elements 4g .. 4g+3 of a row (those past n are -inf); vec: aligned to four elements.
template <int DT>
__device__ __forceinline__ void load4(const void* p, int g, int n, bool vec, float (&v)[4]) {
    if (vec && 4 * g + 4 <= n) {
        if (DT == BI_F32) {
            const float4 x = static_cast<const float4*>(p)[g];
            v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        } else {
            const uint2 x = static_cast<const uint2*>(p)[g];
            v[0] = widen16(uint16_t(x.x), DT == BI_F16);
            v[1] = widen16(uint16_t(x.x >> 16), DT == BI_F16);
            v[2] = widen16(uint16_t(x.y), DT == BI_F16);
            v[3] = widen16(uint16_t(x.y >> 16), DT == BI_F16);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = 4 * g + k < n ? load1<DT>(p, 4 * g + k) : -INFINITY;
    }
}

// Order of a value as a whole number: NaN below every number, +0 and -0 one value.
__device__ __forceinline__ uint32_t order(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return isnan(x) ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float ordered_value(uint32_t o) {
    return o == 0u ? kNaN : __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}
// ... and of an entry: larger values first, then lower indices.  Never 0.
__device__ __forceinline__ unsigned long long order_key(float x, int i) {
    return (uint64_t(order(x)) << 32) | uint32_t(0x7fffffff - i);
}

template <int T, class V, class F>
__device__ __forceinline__ V block_fold(V v, V* scratch, F f) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = f(v, __shfl_xor_sync(~0u, v, off));
    __syncthreads();  // scratch may still be read from the last fold
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = scratch[0];
#pragma unroll
    for (int w = 1; w < T / 32; ++w) v = f(v, scratch[w]);
    return v;
}

// e^d, d <= 0: at most 2 ulp from 2^(d log2 e), whose argument is rounded once.
__device__ __forceinline__ float exp_of(float d) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d * 1.4426950408889634f));
    return y;
}

__device__ __forceinline__ void st_cluster_b64(uint32_t addr, unsigned long long v) {
    asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

struct Stats {
    float m, s, w, bad;  // bad: a NaN among the entries
};

template <int DT, int T>
__global__ void __launch_bounds__(T)
token_logprobs_kernel(const void* __restrict__ x, int64_t ldx, const int32_t* __restrict__ tokens,
                      int n, int part, int parts, bool staged, float* logp, float* entropy,
                      float* lse_out, int top, float* top_logp, int32_t* top_ids,
                      unsigned int* err) {
    constexpr int ES = kSize<DT>;
    extern __shared__ __align__(16) uint8_t stage[];
    __shared__ uint64_t bar[kPieces];
    __shared__ float red[T / 32];
    __shared__ Stats stats[kMaxParts];
    __shared__ unsigned long long list[kList];
    __shared__ unsigned long long best[kMaxParts * BI_LOGPROBS_MAX_TOP];
    __shared__ unsigned long long redk[T / 32];
    __shared__ uint32_t tmax[T];
    __shared__ uint32_t floor_order;
    __shared__ int found;
    const int tid = threadIdx.x;
    const int row = blockIdx.x / parts, rank = blockIdx.x - row * parts;
    const int e0 = rank * part;                 // (a multiple of 8)
    const int cnt = max(0, min(part, n - e0));  // elements of this part
    const char* src = static_cast<const char*>(x) + (int64_t(row) * ldx + e0) * ES;
    const uint32_t skew = uint32_t(reinterpret_cast<uintptr_t>(src) & 15u);
    // the part as the threads read it: a copy with the row's own alignment, or the row
    const void* data = staged ? static_cast<const void*>(stage + skew) : src;
    const bool vec = (skew & (4 * ES - 1)) == 0;
    const int groups = (cnt + 3) / 4;
    // 16-byte units of the part lie at [lo, hi) of the skewed bytes; its first and last bytes
    // outside them are copied by threads
    const uint32_t bytes = uint32_t(cnt) * ES;
    const uint32_t lo = skew ? 16u : 0u, hi = (skew + bytes) & ~15u;
    const uint32_t units = hi > lo ? (hi - lo) / 16 : 0;
    const uint32_t per = (units + kPieces - 1) / kPieces;
    if (tid == 0) {
        for (int i = 0; i < kPieces; ++i) mbar_init(&bar[i], 1);
        fence_barrier_init();
        found = 0;
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    if (staged) {
        if (tid == 0) {
            for (int i = 0; i < kPieces; ++i) {
                const uint32_t u0 = min(units, i * per), u1 = min(units, (i + 1) * per);
                const uint32_t b = (u1 - u0) * 16;
                if (b) {
                    mbar_arrive_expect_tx(&bar[i], b);
                    asm volatile(
                        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
                        "[%0], [%1], %2, [%3];" ::"r"(smem_addr(stage + lo + u0 * 16)),
                        "l"(src - skew + lo + u0 * 16), "r"(b), "r"(smem_addr(&bar[i]))
                        : "memory");
                } else {
                    mbar_arrive(&bar[i]);
                }
            }
        }
        // the edges: elements with a byte outside the units
        const int head = min(cnt, lo ? int(lo - skew) / ES : 0);
        const int tail0 = units ? int(hi - skew) / ES : head;
        for (int i = tid; i < head; i += T) {
            if (ES == 4)
                reinterpret_cast<float*>(stage + skew)[i] = reinterpret_cast<const float*>(src)[i];
            else
                reinterpret_cast<uint16_t*>(stage + skew)[i] =
                    reinterpret_cast<const uint16_t*>(src)[i];
        }
        for (int i = tail0 + tid; i < cnt; i += T) {
            if (ES == 4)
                reinterpret_cast<float*>(stage + skew)[i] = reinterpret_cast<const float*>(src)[i];
            else
                reinterpret_cast<uint16_t*>(stage + skew)[i] =
                    reinterpret_cast<const uint16_t*>(src)[i];
        }
        __syncthreads();
    }
    // the thread's maximum, piece by piece
    float m = -INFINITY;
    bool nan = false;
    int ready = staged ? 0 : cnt;  // elements that have landed
    bool ok = true;
    int piece = 0;
    for (int g = tid; g < groups; g += T) {
        while (min(4 * g + 4, cnt) > ready) {
            if (!mbar_wait(&bar[piece], 0, nullptr, wait_budget_ns(err))) ok = false;
            ++piece;
            ready = piece == kPieces
                        ? cnt
                        : min(cnt, int(lo + min(units, piece * per) * 16 - min(skew, lo)) / ES);
        }
        float v[4];
        load4<DT>(data, g, cnt, vec, v);
#pragma unroll
        for (int k = 0; k < 4; ++k) nan |= isnan(v[k]);
        m = fmaxf(fmaxf(m, fmaxf(v[0], v[1])), fmaxf(v[2], v[3]));
    }
    if (staged)  // every thread has seen every piece land: all read all of it below
        for (; piece < kPieces; ++piece)
            if (!mbar_wait(&bar[piece], 0, nullptr, wait_budget_ns(err))) ok = false;
    if (!ok) latch_error(err, kErrTimeout);
    if (top > 0) tmax[tid] = tid < groups ? order(m) : 0u;
    const float pm =
        block_fold<T>(m, red, [](float a, float b) { return fmaxf(a, b); });
    const bool any_nan = __syncthreads_or(nan);
    // s and w of the part; a part of nothing but -inf has s = 0
    const float ref = pm == -INFINITY ? 0.f : pm;
    float s = 0.f, w = 0.f;
    for (int g = tid; g < groups; g += T) {
        float v[4];
        load4<DT>(data, g, cnt, vec, v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float d = v[k] - ref;
            const float e = exp_of(d);
            s = s + e;
            w = fmaf(e, fmaxf(d, -1e4f), w);  // (exp is 0 long before -1e4; 0 * -inf is not)
        }
    }
    auto add = [](float a, float b) { return a + b; };
    s = block_fold<T>(s, red, add);
    w = block_fold<T>(w, red, add);

    if (top > 0) {
        // the part's first `top` entries in order, as keys (0 where it has fewer)
        const int want = min(top, cnt);
        const uint32_t own = tmax[tid];
        int above = 0;
        for (int i = 0; i < T; ++i) above += tmax[i] > own || (tmax[i] == own && i < tid) ? 1 : 0;
        if (above == min(want, T) - 1) floor_order = own;
        for (int i = tid; i < BI_LOGPROBS_MAX_TOP; i += T) best[i] = 0ull;
        __syncthreads();
        const uint32_t fl = floor_order;
        if (own >= fl) {
            for (int g = tid; g < groups; g += T) {
                float v[4];
                load4<DT>(data, g, cnt, vec, v);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (4 * g + k < cnt && order(v[k]) >= fl) {
                        const int at = atomicAdd(&found, 1);
                        if (at < kList) list[at] = order_key(v[k], e0 + 4 * g + k);
                    }
                }
            }
        }
        __syncthreads();
        const int f = found;
        if (f >= want && f <= kList) {
            for (int i = tid; i < f; i += T) {
                const unsigned long long key = list[i];
                int r = 0;
                for (int j = 0; j < f; ++j) r += list[j] > key ? 1 : 0;
                if (r < want) best[r] = key;
            }
        } else {  // too many ties (or a row of NaN): one maximum after the other
            unsigned long long last = ~0ull;
            for (int k = 0; k < want; ++k) {
                unsigned long long b = 0;
                for (int g = tid; g < groups; g += T) {
                    float v[4];
                    load4<DT>(data, g, cnt, vec, v);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const unsigned long long key = order_key(v[q], e0 + 4 * g + q);
                        if (4 * g + q < cnt && key < last && key > b) b = key;
                    }
                }
                last = block_fold<T>(b, redk, [](unsigned long long p, unsigned long long q) {
                    return p > q ? p : q;
                });
                if (tid == 0) best[k] = last;
            }
        }
        __syncthreads();
    }

    // the parts meet in rank 0
    if (parts > 1) {
        cluster_sync_all();  // (rank 0 has started, and its list is built)
        if (rank != 0) {
            if (tid == 0) {
                const uint32_t a = cluster_map(smem_addr(&stats[rank]), 0);
                st_cluster_f32(a, pm);
                st_cluster_f32(a + 4, s);
                st_cluster_f32(a + 8, w);
                st_cluster_f32(a + 12, any_nan ? 1.f : 0.f);
            }
            if (tid < top)
                st_cluster_b64(cluster_map(smem_addr(&best[rank * top]), 0) + tid * 8, best[tid]);
        }
        cluster_sync_all();
        if (rank != 0) return;
    }
    if (tid == 0) stats[0] = Stats{pm, s, w, any_nan ? 1.f : 0.f};
    __syncthreads();
    float M = stats[0].m;
    bool bad = stats[0].bad != 0.f;
    for (int p = 1; p < parts; ++p) {
        M = fmaxf(M, stats[p].m);
        bad |= stats[p].bad != 0.f;
    }
    float S = 0.f, W = 0.f;
    for (int p = 0; p < parts; ++p) {
        const Stats a = stats[p];
        if (a.m == -INFINITY) continue;  // (a part of nothing but -inf adds nothing)
        const float d = a.m - M, f = exp_of(d);
        S = fmaf(a.s, f, S);
        W = fmaf(f, fmaf(a.s, d, a.w), W);
    }
    bad |= !isfinite(M);
    const float ls = bad ? kNaN : logf(S);
    if (tid == 0) {
        const int t = tokens[row];
        if (t >= 0 && t < n) {
            const float xt = load1<DT>(static_cast<const char*>(x) + int64_t(row) * ldx * ES, t);
            logp[row] = (xt - M) - ls;
        } else if (t == -1) {
            logp[row] = 0.f;
        } else {
            latch_error(err, kErrDeviceArg);
            logp[row] = kNaN;
        }
        if (entropy) entropy[row] = ls - W / S;
        if (lse_out) lse_out[row] = M + ls;
    }
    if (top > 0) {
        const int total = parts * top;  // part p's keys at best[p * top]
        for (int i = tid; i < total; i += T) {
            const unsigned long long key = best[i];
            int r = key ? 0 : top;
            for (int j = 0; j < total && r < top; ++j) r += best[j] > key ? 1 : 0;
            if (r < top) {
                top_ids[int64_t(row) * top + r] = 0x7fffffff - int(uint32_t(key));
                top_logp[int64_t(row) * top + r] =
                    (ordered_value(uint32_t(key >> 32)) - M) - ls;
            }
        }
    }
}

// How a row is cut, from n alone.
struct RowCut {
    int parts, part;
};
RowCut row_cut(int64_t n) {
    RowCut c;
    c.parts = int(std::min<int64_t>(kMaxParts, (n + kPart - 1) / kPart));
    c.part = int(((n + c.parts - 1) / c.parts + 7) / 8 * 8);
    return c;
}

template <int DT, int T>
cudaError_t launch_forward(const DeviceInfo& dev, const void* x, int64_t ldx,
                           const int32_t* tokens, int64_t rows, int64_t n, float* logp,
                           float* entropy, float* lse, int top, float* top_logp,
                           int32_t* top_ids, cudaStream_t stream) {
    const RowCut c = row_cut(n);
    const size_t bytes = size_t(c.part) * kSize<DT> + 32;
    const bool staged = bytes <= kMaxStage;
    auto kern = token_logprobs_kernel<DT, T>;
    static bool attr_done[64] = {};
    if (dev.device >= 0 && dev.device < 64 && !attr_done[dev.device]) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             int(kMaxStage));
        if (e != cudaSuccess) return e;
        attr_done[dev.device] = true;
    }
    return launch_pdl_cluster(kern, dim3(unsigned(rows * c.parts)), dim3(T), staged ? bytes : 0,
                              stream, unsigned(c.parts), x, ldx, tokens, int(n), c.part, c.parts,
                              staged, logp, entropy, lse, top, top_logp, top_ids, dev.err_word);
}

// ------------------------------------------------------------------------- backward

constexpr int GT = 256;  // threads of a gradient CTA
constexpr int GV = 4;    // 16-byte vectors per thread

template <int DT>
__device__ __forceinline__ float gradient_of(float x, int i, int t, float gl, float ge, float ls,
                                             float H) {
    const float lp = x - ls;
    const float p = exp_of(lp);
    const float d = p == 0.f ? 0.f : -p * fmaf(ge, lp + H, gl);
    return i == t ? d + gl : d;
}

// One CTA per GT * GV vectors of a row.  The row's elements before its first 16-byte boundary
// are taken by the row's first CTA, those behind the last by the CTA that reaches them; where
// x and dx are not aligned alike, all are taken one by one.
template <int DT>
__global__ void __launch_bounds__(GT)
token_logprobs_backward_kernel(const void* x, int64_t ldx, const int32_t* __restrict__ tokens,
                               int n, int per_row, const float* __restrict__ lse,
                               const float* __restrict__ entropy, const float* __restrict__ g_logp,
                               const float* __restrict__ g_entropy, void* dx, int64_t lddx,
                               unsigned int* err) {
    constexpr int ES = kSize<DT>, VE = 16 / ES;  // elements of a vector
    pdl_wait();
    pdl_trigger();
    const int64_t r = blockIdx.x / unsigned(per_row);
    const int c = int(blockIdx.x - unsigned(r) * unsigned(per_row));
    const char* xr = static_cast<const char*>(x) + r * ldx * ES;
    char* dr = static_cast<char*>(dx) + r * lddx * ES;
    const int t = tokens[r];
    if (c == 0 && threadIdx.x == 0 && (t < -1 || t >= n)) latch_error(err, kErrDeviceArg);
    const float gl = g_logp && t >= 0 && t < n ? g_logp[r] : 0.f;
    const float ge = g_entropy ? g_entropy[r] : 0.f;
    const float ls = lse[r], H = entropy ? entropy[r] : 0.f;
    auto one = [&](int i) {
        const float d = gradient_of<DT>(load1<DT>(xr, i), i, t, gl, ge, ls, H);
        if (DT == BI_F32)
            reinterpret_cast<float*>(dr)[i] = d;
        else
            reinterpret_cast<uint16_t*>(dr)[i] = round16(d, DT == BI_F16);
    };
    const uint32_t ax = uint32_t(reinterpret_cast<uintptr_t>(xr) & 15u);
    const uint32_t ad = uint32_t(reinterpret_cast<uintptr_t>(dr) & 15u);
    if (ax != ad) {
        const int i0 = c * (GT * GV * VE), i1 = min(n, i0 + GT * GV * VE);
#pragma unroll 4
        for (int i = i0 + int(threadIdx.x); i < i1; i += GT) one(i);
        return;
    }
    const int head = min(n, ax ? int(16 - ax) / ES : 0);
    const int vecs = (n - head) / VE;
    const uint4* xv = reinterpret_cast<const uint4*>(xr + head * ES);
    uint4* dv = reinterpret_cast<uint4*>(dr + head * ES);
    const int v0 = c * (GT * GV) + int(threadIdx.x);
    uint4 a[GV];
#pragma unroll
    for (int k = 0; k < GV; ++k)
        if (v0 + k * GT < vecs) a[k] = xv[v0 + k * GT];
#pragma unroll
    for (int k = 0; k < GV; ++k) {
        if (v0 + k * GT >= vecs) continue;
        const int i = head + (v0 + k * GT) * VE;
        const uint32_t w[4] = {a[k].x, a[k].y, a[k].z, a[k].w};
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (DT == BI_F32) {
                o[q] = __float_as_uint(
                    gradient_of<DT>(__uint_as_float(w[q]), i + q, t, gl, ge, ls, H));
            } else {
                constexpr bool F16 = DT == BI_F16;
                o[q] = pack16x2(
                    gradient_of<DT>(widen16(uint16_t(w[q]), F16), i + 2 * q, t, gl, ge, ls, H),
                    gradient_of<DT>(widen16(uint16_t(w[q] >> 16), F16), i + 2 * q + 1, t, gl, ge,
                                    ls, H),
                    F16);
            }
        }
        dv[v0 + k * GT] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (c == 0 && int(threadIdx.x) < head) one(int(threadIdx.x));
    const int tail = head + vecs * VE + int(threadIdx.x);
    if (c == per_row - 1 && threadIdx.x < VE && tail < n) one(tail);
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
    if (rows * row_cut(n).parts > kI32Max)
        return fail(BI_ERR_UNSUPPORTED, "%s: too many rows", fn);
    // short rows: CTAs of 128 threads
    auto run = [&](auto f) {
        return launched(f(*dev, x, ldx, tokens, rows, n, logp, entropy, lse, int(top), top_logp,
                          top_ids, reinterpret_cast<cudaStream_t>(stream)),
                        fn);
    };
    const bool small = n <= 8192;
    if (x_dtype == BI_F32) return run(small ? launch_forward<BI_F32, 128> : launch_forward<BI_F32, 256>);
    if (x_dtype == BI_F16) return run(small ? launch_forward<BI_F16, 128> : launch_forward<BI_F16, 256>);
    return run(small ? launch_forward<BI_BF16, 128> : launch_forward<BI_BF16, 256>);
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
    // (one more vector than n holds: a row's first and last elements may lie outside them)
    const int64_t vecs = n / int64_t(16 / es) + 1;
    const int64_t per_row = (vecs + GT * GV - 1) / (GT * GV);
    if (rows * per_row > kI32Max) return fail(BI_ERR_UNSUPPORTED, "%s: too many elements", fn);
    return launched(launch_pdl(kern, dim3(unsigned(rows * per_row)), dim3(GT), 0,
                               reinterpret_cast<cudaStream_t>(stream), x, ldx, tokens, int(n),
                               int(per_row), lse, entropy, g_logp, g_entropy, dx, lddx,
                               dev->err_word),
                    fn);
}
