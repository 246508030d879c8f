// logprobs.cu -- log-probabilities of given tokens with entropy and top alternatives, and
// their gradient (include/bi_rowwise.h).
//
// Forward.  With m a maximum and d_i = x_i - m:  s = sum exp(d_i),  w = sum exp(d_i) d_i,
// logp = (x_t - m) - log s,  entropy = log s - w / s.  A row is cut into P parts (P <= 8, of
// 16,384 elements where that is enough):
//   * thread t of T (256; 128 for 16-bit types, whose vectors hold twice as much, and for rows
//     of up to 8,192) takes the part's 16-byte vectors t, t + T, ..., eight at a time, all eight
//     requested before any is used; against a running maximum it keeps (m, s, w) in one pass,
//     rescaling when a batch raises the maximum;
//   * in rows of more than 524,288 elements it starts anew after every eight batches and adds
//     the groups pairwise, so that no sum has more than 264 terms in a row, whatever n is (with
//     running sums all along, log s of equal entries was off by 8e-4 at n = 2^27);
//   * one warp folds the threads' (m, s, w) of a part: each lane its T / 32 in ascending order,
//     then a butterfly; the parts are folded in ascending order.
// The tree depends on n and the type alone.  Who runs it does not matter to it: with few rows a
// cluster has a CTA for each part (the parts meet in rank 0's shared memory), with many a CTA
// takes a whole row and meets a barrier once per row.  1024 x 128256 fp32 takes 83 us (6.3 TB/s),
// 2048 x 128256 bf16 90 us (5.8 TB/s; there the instructions of an element, about ten, bind as
// much as its two bytes).  Staging the parts in shared memory by bulk copies, with a CTA and its
// barriers per part, took 170 and 247 us.
//
// Top alternatives.  The k-th largest of the thread maxima bounds the k-th largest element from
// below, so few elements (k, and a handful more) lie at or above it; all threads look again at
// the vectors of the few that hold one (each at its own, 1024 x 128256 fp32 with 20 took 133 us),
// the elements are ranked by counting, and rank 0 ranks the CTAs' first k.  Where ties make them
// too many, k rounds of a maximum below the last one found.
//
// Backward.  Elementwise from the saved lse and entropy: one read, one write.
//
// Both are bound by memory: rows * n * size bytes, twice that for the gradient.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <type_traits>

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
constexpr int kBatch = 8;              // vectors that a thread requests at a time
constexpr int kFold = 8;               // batches that a thread sums before it starts anew
constexpr int kLevels = 13;            // of pairwise sums: 2^12 groups at the longest row
constexpr int kList = 512;             // candidates gathered for the top entries
constexpr float kNaN = __builtin_nanf("");

template <int DT>
constexpr int kSize = DT == BI_F32 ? 4 : 2;
template <int DT>  // -inf, in both halves for 16 bits
constexpr uint32_t kMinusInf = DT == BI_F32   ? 0xff800000u
                               : DT == BI_F16 ? 0xfc00fc00u
                                              : 0xff80ff80u;

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    if (DT == BI_F32) return static_cast<const float*>(p)[i];
    return widen16(static_cast<const uint16_t*>(p)[i], DT == BI_F16);
}

// Vector g of a row of n elements, as its 16 bytes: elements VE g .. VE g + VE - 1 (those from n
// on are -inf and not read).  vec: the row starts on a 16-byte boundary.
template <int DT>
__device__ __forceinline__ uint4 load_vec(const char* row, bool vec, int g, int n) {
    constexpr int ES = kSize<DT>, VE = 16 / ES;
    if (vec && VE * g + VE <= n) return __ldg(reinterpret_cast<const uint4*>(row) + g);
    uint32_t o[4] = {kMinusInf<DT>, kMinusInf<DT>, kMinusInf<DT>, kMinusInf<DT>};
#pragma unroll
    for (int k = 0; k < VE; ++k) {
        const int i = VE * g + k;
        if (i < n) {
            if (ES == 4) {
                o[k] = reinterpret_cast<const uint32_t*>(row)[i];
            } else {
                const uint32_t h = reinterpret_cast<const uint16_t*>(row)[i];
                o[k >> 1] = k & 1 ? (o[k >> 1] & 0xffffu) | (h << 16)
                                  : (o[k >> 1] & 0xffff0000u) | h;
            }
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// kBatch vectors g, g + T, ... below v1 (this thread's g = base + tid), -inf from there on; none
// of them is used before all are requested.  A row off its 16-byte boundary by `skew` bytes is
// read as aligned vectors: the one that starts in front of the wanted 16 bytes, and its
// neighbour, which the next lane has read (lane 31 reads it itself).  Vectors at the row's ends,
// whose aligned ones reach outside it, are read element by element.  All threads of the CTA call
// it together, with one base and v1.
template <int DT, int T, bool ALIGNED>
__device__ __forceinline__ void load_batch(uint4 (&a)[kBatch], const char* row, uint32_t skew,
                                           int base, int v1, int n) {
    constexpr int ES = kSize<DT>;
    const uint4 none = make_uint4(kMinusInf<DT>, kMinusInf<DT>, kMinusInf<DT>, kMinusInf<DT>);
    if (ALIGNED) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int g = base + k * T + int(threadIdx.x);
            a[k] = none;
            if (g < v1) a[k] = load_vec<DT>(row, true, g, n);
        }
        return;
    }
    const uint4* p = reinterpret_cast<const uint4*>(row - skew);
    const int lane = threadIdx.x & 31;
    // aligned vectors lo .. hi - 1 lie within the row
    const int lo = skew ? 1 : 0, hi = int((int64_t(n) * ES + skew) / 16);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const int g = base + k * T + int(threadIdx.x);
        a[k] = none;
        if (g < v1 && g >= lo && g < hi) a[k] = __ldg(p + g);
    }
    if (skew == 0) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int g = base + k * T + int(threadIdx.x);
            if (g < v1 && g >= hi) a[k] = load_vec<DT>(row, false, g, n);
        }
        return;
    }
    const bool one = (skew & 4u) != 0, two = (skew & 8u) != 0;
    const uint32_t bits = (skew & 3u) * 8u;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        if (base + k * T >= v1) break;
        const int g = base + k * T + int(threadIdx.x);
        uint4 b = make_uint4(
            __shfl_down_sync(0xffffffffu, a[k].x, 1), __shfl_down_sync(0xffffffffu, a[k].y, 1),
            __shfl_down_sync(0xffffffffu, a[k].z, 1), __shfl_down_sync(0xffffffffu, a[k].w, 1));
        const bool inside = g >= lo && g + 1 < hi;
        // (a neighbour from v1 on belongs to the next part and was not read)
        if (inside && (lane == 31 || g + 1 >= v1) && g < v1) b = __ldg(p + g + 1);
        // bytes skew .. skew + 15 of (a, b): whole words by selection, the rest by shifts
        const uint32_t w0[8] = {a[k].x, a[k].y, a[k].z, a[k].w, b.x, b.y, b.z, b.w};
        uint32_t w1[7], w2[5];
#pragma unroll
        for (int i = 0; i < 7; ++i) w1[i] = one ? w0[i + 1] : w0[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) w2[i] = two ? w1[i + 2] : w1[i];
        const uint4 r = make_uint4(
            __funnelshift_r(w2[0], w2[1], bits), __funnelshift_r(w2[1], w2[2], bits),
            __funnelshift_r(w2[2], w2[3], bits), __funnelshift_r(w2[3], w2[4], bits));
        if (inside)
            a[k] = r;
        else if (g < v1)
            a[k] = load_vec<DT>(row, false, g, n);
        else
            a[k] = none;
    }
}

// Its elements.
template <int DT>
__device__ __forceinline__ void widen(const uint4& a, float (&v)[16 / kSize<DT>]) {
    constexpr int VE = 16 / kSize<DT>;
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < VE; ++k) {
        v[k] = DT == BI_F32 ? __uint_as_float(w[k & 3])
                            : widen16(uint16_t(w[(k >> 1) & 3] >> (16 * (k & 1))), DT == BI_F16);
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

template <int T>
__device__ __forceinline__ unsigned long long block_max(unsigned long long v,
                                                        unsigned long long* scratch) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const unsigned long long o = __shfl_xor_sync(~0u, v, off);
        v = o > v ? o : v;
    }
    __syncthreads();  // scratch may still be read from the last one
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = scratch[0];
    for (int w = 1; w < T / 32; ++w) v = scratch[w] > v ? scratch[w] : v;
    return v;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {  // at most 2 ulp from 2^x; 0 below 2^-126
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// e^d, d <= 0 (the argument of 2^ is rounded once)
__device__ __forceinline__ float exp_of(float d) { return ex2(d * kLog2e); }

// Two fp32 operations in one instruction, each rounded as its scalar form.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// The largest of a whole vector's elements (NaN ignored beside a number; a max is exact in the
// element's own type).
template <int DT>
__device__ __forceinline__ float vec_max(const uint4& a) {
    if (DT == BI_F32)
        return fmaxf(fmax3(__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z)),
                     __uint_as_float(a.w));
    if (DT == BI_BF16) {
        auto h = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
        const __nv_bfloat162 m = __hmax2(__hmax2(h(a.x), h(a.y)), __hmax2(h(a.z), h(a.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
    auto h = [](uint32_t w) { return *reinterpret_cast<const __half2*>(&w); };
    const __half2 m = __hmax2(__hmax2(h(a.x), h(a.y)), __hmax2(h(a.z), h(a.w)));
    return fmaxf(__low2float(m), __high2float(m));
}

__device__ __forceinline__ void st_cluster_b64(uint32_t addr, unsigned long long v) {
    asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// The sums of a set of entries, in powers of two: m their maximum, s = sum 2^u and
// w = sum 2^u u over u = (x - m) log2 e.  s is NaN where an entry is.
struct Stats {
    float m, s, w;
};
__device__ __forceinline__ float ref_of(float m) { return m == -INFINITY ? 0.f : m; }

// Two sets together; m = -inf, s = w = 0 is none.  A set of nothing but NaN and -inf has m = -inf
// and s = NaN, which stays.
__device__ __forceinline__ void join(Stats& a, const Stats& b) {
    const float M = fmaxf(a.m, b.m), c = ref_of(M);
    // (2^u is 0 long before -1e4; 0 * -inf is not, nor is 0 * +inf: none beside the lowest value)
    const float da = a.m == -INFINITY ? 0.f : fmaxf((a.m - c) * kLog2e, -1e4f);
    const float db = b.m == -INFINITY ? 0.f : fmaxf((b.m - c) * kLog2e, -1e4f);
    const float fa = a.m == -INFINITY ? a.s : ex2(da), fb = b.m == -INFINITY ? b.s : ex2(db);
    a.w = fmaf(fa, fmaf(a.s, da, a.w), fb * fmaf(b.s, db, b.w));
    a.s = fmaf(a.s, fa, b.s * fb);
    a.m = M;
}

constexpr int kGroups = 64;  // groups of threads whose maxima bound the top entries

// `ctas` CTAs (one cluster) per row, each over parts / ctas parts of `part` vectors.
// CTAs per multiprocessor: seven of 128 threads (1024 x 100001 bf16, unaligned, 63 us; six 69,
// where 1024 rows are two waves), four of 256; three where unaligned, or registers spill (fp32 96
// us, 106 with four).
// LONG: a part has more than kFold batches.
template <int DT, int T, bool ALIGNED, bool LONG>
__global__ void __launch_bounds__(T, T == 128 ? 7 : ALIGNED ? 4 : 3)
token_logprobs_kernel(const void* __restrict__ x, int64_t ldx, const int32_t* __restrict__ tokens,
                      int n, int part, int parts, int ctas, float* logp, float* entropy,
                      float* lse_out, int top, float* top_logp, int32_t* top_ids,
                      unsigned int* err) {
    constexpr int ES = kSize<DT>, VE = 16 / ES;
    __shared__ Stats stats[kMaxParts];
    __shared__ float tm[kMaxParts][T], ts[kMaxParts][T], tw[kMaxParts][T];
    __shared__ unsigned long long list[kList];
    __shared__ unsigned long long best[kMaxParts * BI_LOGPROBS_MAX_TOP];
    __shared__ unsigned long long redk[T / 32];
    __shared__ uint32_t gmax[kGroups];
    __shared__ uint32_t floor_order;
    __shared__ int found, holding;
    __shared__ uint16_t holders[kMaxParts * T];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.x / ctas, rank = blockIdx.x - row * ctas;
    const int mine = parts / ctas, p0 = rank * mine;
    const char* xr = static_cast<const char*>(x) + int64_t(row) * ldx * ES;
    const uint32_t skew = ALIGNED ? 0u : uint32_t(reinterpret_cast<uintptr_t>(xr) & 15u);
    const int vecs = (n + VE - 1) / VE;
    pdl_wait();
    pdl_trigger();
    if (tid == 0) found = holding = 0;
    __syncthreads();
    const int whole = n / VE;  // vectors that hold no padding
    auto sums = [&](auto clamp) {
        bool again = false;
        for (int p = 0; p < mine; ++p) {
            const int v0 = (p0 + p) * part, v1 = min(vecs, v0 + part);
            float m = -INFINITY, s = 0.f, w = 0.f;
            Stats level[LONG ? kLevels : 1];  // sums of 2^l groups, for each bit l of `groups`
            uint32_t groups = 0;
            int batch = 0;
            for (int g = v0; g < v1; g += T * kBatch) {
                // every thread's vectors are there, and whole
                const bool full = g + kBatch * T <= min(v1, whole);
                uint4 a[kBatch];
                if (ALIGNED && full) {
#pragma unroll
                    for (int k = 0; k < kBatch; ++k)
                        a[k] = __ldg(reinterpret_cast<const uint4*>(xr) + g + k * T + tid);
                } else {
                    load_batch<DT, T, ALIGNED>(a, xr, skew, g, v1, n);
                }
                float bm = vec_max<DT>(a[0]);
#pragma unroll
                for (int k = 1; k < kBatch; ++k) bm = fmaxf(bm, vec_max<DT>(a[k]));
                if (bm > m) {
                    const float d = m == -INFINITY ? 0.f : fmaxf((m - bm) * kLog2e, -1e4f);
                    const float f = m == -INFINITY ? s : ex2(d);  // (s is 0 or NaN there)
                    w = f * fmaf(s, d, w);
                    s *= f;
                    m = bm;
                }
                const float c = -ref_of(m);
                // two running sums each, of the even and the odd elements: one instruction for both
                float2 s2 = make_float2(s, 0.f), w2 = make_float2(w, 0.f);
                auto take = [&](float x0, float x1, bool held) {
                    const float2 u = mul2(add2(make_float2(x0, x1), make_float2(c, c)),
                                          make_float2(kLog2e, kLog2e));
                    const float2 e = make_float2(ex2(u.x), ex2(u.y));
                    s2 = add2(s2, e);
                    w2 = fma2(e, held ? make_float2(fmaxf(u.x, -1e4f), fmaxf(u.y, -1e4f)) : u, w2);
                };
                if (full && !decltype(clamp)::value) {
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        float v[VE];
                        widen<DT>(a[k], v);
#pragma unroll
                        for (int q = 0; q < VE; q += 2) take(v[q], v[q + 1], false);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        if (g + k * T >= v1) break;  // (no thread has a vector here)
                        float v[VE];
                        widen<DT>(a[k], v);
#pragma unroll
                        for (int q = 0; q < VE; q += 2) take(v[q], v[q + 1], true);
                    }
                }
                s = s2.x + s2.y;
                w = w2.x + w2.y;
                if (LONG && (++batch % kFold == 0 || g + T * kBatch >= v1)) {
                    Stats a{m, s, w};
                    int l = 0;
                    for (; (groups >> l) & 1u; ++l) join(a, level[l]);
                    level[l] = a;
                    ++groups;
                    m = -INFINITY;
                    s = w = 0.f;
                }
            }
            if (LONG) {
                Stats a{m, s, w};  // (none, and that of a part without vectors)
                for (int l = 0; l < kLevels; ++l)
                    if ((groups >> l) & 1u) join(a, level[l]);
                m = a.m;
                s = a.s;
                w = a.w;
            }
            tm[p][tid] = m;
            ts[p][tid] = s;
            tw[p][tid] = w;
            again |= isnan(w) && !isnan(s);
        }
        return again;
    };
    // 0 * -inf makes w NaN where an entry is -inf: then the CTA goes over its parts again with u
    // held above -1e4 in w (2^u is 0 long before), which changes no other term
    if (__syncthreads_or(sums(std::false_type()))) {
        sums(std::true_type());
        __syncthreads();
    }
    // the parts' sums, a warp each
    for (int p = warp; p < mine; p += T / 32) {
        Stats a{tm[p][lane], ts[p][lane], tw[p][lane]};
#pragma unroll
        for (int i = 1; i < T / 32; ++i)
            join(a, Stats{tm[p][lane + 32 * i], ts[p][lane + 32 * i], tw[p][lane + 32 * i]});
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const Stats b{__shfl_xor_sync(~0u, a.m, off), __shfl_xor_sync(~0u, a.s, off),
                          __shfl_xor_sync(~0u, a.w, off)};
            join(a, b);
        }
        if (lane == 0) stats[p0 + p] = a;
    }
    if (top > 0) {
        // this CTA's first `top` entries in order, as keys (0 where it has fewer)
        const int cnt = max(0, min(n, (p0 + mine) * part * VE) - p0 * part * VE);
        const int want = min(top, cnt);
        float m = -INFINITY;
        for (int p = 0; p < mine; ++p) m = fmaxf(m, tm[p][tid]);
        const uint32_t own = order(m);
        uint32_t gm = own;
#pragma unroll
        for (int off = 1; off < T / kGroups; off <<= 1)
            gm = max(gm, __shfl_xor_sync(~0u, gm, off));
        if (tid % (T / kGroups) == 0) gmax[tid / (T / kGroups)] = gm;
        for (int i = tid; i < BI_LOGPROBS_MAX_TOP; i += T) best[i] = 0ull;
        __syncthreads();
        if (tid < kGroups) {  // the group maximum that want - 1 others exceed
            const uint32_t g = gmax[tid];
            int above = 0;
#pragma unroll 16
            for (int i = 0; i < kGroups; ++i)
                above += gmax[i] > g || (gmax[i] == g && i < tid) ? 1 : 0;
            if (above == max(want, 1) - 1) floor_order = g;
        }
        __syncthreads();
        const uint32_t fl = floor_order;
        // the threads, by part, whose maximum reaches the floor; all threads look at their vectors
        for (int p = 0; p < mine; ++p)
            if (order(tm[p][tid]) >= fl) holders[atomicAdd(&holding, 1)] = uint16_t(p * T + tid);
        __syncthreads();
        const int each = (part + T - 1) / T, looks = holding * each;
        for (int base = tid; base < looks; base += T * kBatch) {
            uint4 a[kBatch];
            int at[kBatch];  // the vectors, -1: none
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = base + k * T, h = i / each;
                at[k] = -1;
                if (i < looks) {
                    const int p = holders[h] / T;
                    const int g = (p0 + p) * part + holders[h] % T + (i - h * each) * T;
                    if (g < min(vecs, (p0 + p + 1) * part)) {
                        at[k] = g;
                        a[k] = load_vec<DT>(xr, skew == 0, g, n);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (at[k] < 0) continue;
                float v[VE];
                widen<DT>(a[k], v);
                float vm = v[0];
#pragma unroll
                for (int q = 1; q < VE; ++q) vm = fmaxf(vm, v[q]);
                if (order(vm) < fl) continue;
#pragma unroll
                for (int q = 0; q < VE; ++q) {
                    const int i = at[k] * VE + q;
                    if (i < n && order(v[q]) >= fl) {
                        const int to = atomicAdd(&found, 1);
                        if (to < kList) list[to] = order_key(v[q], i);
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
                for (int g = p0 * part + tid; g < min(vecs, (p0 + mine) * part); g += T) {
                    float v[VE];
                    widen<DT>(load_vec<DT>(xr, skew == 0, g, n), v);
#pragma unroll
                    for (int q = 0; q < VE; ++q) {
                        const unsigned long long key = order_key(v[q], g * VE + q);
                        if (g * VE + q < n && key < last && key > b) b = key;
                    }
                }
                last = block_max<T>(b, redk);
                if (tid == 0) best[k] = last;
            }
        }
    }
    __syncthreads();

    // the CTAs of a row meet in rank 0
    if (ctas > 1) {
        cluster_sync_all();  // (rank 0 has started, and its own entries are written)
        if (rank != 0) {
            if (tid < mine) {
                const uint32_t a = cluster_map(smem_addr(&stats[p0 + tid]), 0);
                st_cluster_f32(a, stats[p0 + tid].m);
                st_cluster_f32(a + 4, stats[p0 + tid].s);
                st_cluster_f32(a + 8, stats[p0 + tid].w);
            }
            if (tid < top)
                st_cluster_b64(cluster_map(smem_addr(&best[rank * top]), 0) + tid * 8, best[tid]);
        }
        cluster_sync_all();
        if (rank != 0) return;
    }
    Stats a = stats[0];
    for (int p = 1; p < parts; ++p) join(a, stats[p]);
    const bool bad = isnan(a.s) || !isfinite(a.m);
    const float ls = bad ? kNaN : logf(a.s);
    if (tid == 0) {
        const int t = tokens[row];
        if (t >= 0 && t < n) {
            logp[row] = (load1<DT>(xr, t) - a.m) - ls;
        } else if (t == -1) {
            logp[row] = 0.f;
        } else {
            latch_error(err, kErrDeviceArg);
            logp[row] = kNaN;
        }
        if (entropy) entropy[row] = ls - a.w / a.s * kLn2;
        if (lse_out) lse_out[row] = a.m + ls;
    }
    if (top > 0) {
        const int total = ctas * top;  // rank r's keys at best[r * top]
        for (int i = tid; i < total; i += T) {
            const unsigned long long key = best[i];
            int r = key ? 0 : top;
            for (int j = 0; j < total && r < top; ++j) r += best[j] > key ? 1 : 0;
            if (r < top) {
                top_ids[int64_t(row) * top + r] = 0x7fffffff - int(uint32_t(key));
                top_logp[int64_t(row) * top + r] =
                    (ordered_value(uint32_t(key >> 32)) - a.m) - ls;
            }
        }
    }
}

// How a row of n elements is cut: parts, and 16-byte vectors of each.
struct RowCut {
    int parts, part;
};
RowCut row_cut(int64_t n, int ve) {
    RowCut c;
    c.parts = int(std::min<int64_t>(kMaxParts, (n + kPart - 1) / kPart));
    const int64_t vecs = (n + ve - 1) / ve;
    c.part = int((vecs + c.parts - 1) / c.parts);
    return c;
}

template <int DT, int T, bool ALIGNED>
cudaError_t launch_forward(const DeviceInfo& dev, const void* x, int64_t ldx,
                           const int32_t* tokens, int64_t rows, int64_t n, float* logp,
                           float* entropy, float* lse, int top, float* top_logp,
                           int32_t* top_ids, cudaStream_t stream) {
    const RowCut c = row_cut(n, 16 / kSize<DT>);
    // CTAs per row: one, once the rows give every multiprocessor two; with fewer rows, as many
    // as do that (up to one per part).  Splitting more rows than that costs more in the cluster's
    // meeting than a last wave that is not full: 1024 x 128256 fp32 83 us with one CTA a row, 166
    // with four.
    int ctas = 1;
    while (ctas < c.parts && rows * ctas < 2 * int64_t(dev.num_sms)) {
        do ++ctas; while (c.parts % ctas != 0);
    }
    auto kern = token_logprobs_kernel<DT, T, ALIGNED, false>;
    if constexpr (DT != BI_F32 || T == 256) {  // (fp32 rows for 128 threads are short)
        if (c.part > kFold * T * kBatch) kern = token_logprobs_kernel<DT, T, ALIGNED, true>;
    }
    return launch_pdl_cluster(kern, dim3(unsigned(rows * ctas)), dim3(T), 0, stream,
                              unsigned(ctas), x, ldx, tokens, int(n), c.part, c.parts, ctas, logp,
                              entropy, lse, top, top_logp, top_ids, dev.err_word);
}

// ------------------------------------------------------------------------- backward

constexpr int GT = 256;  // threads of a gradient CTA
constexpr int GV = 4;    // 16-byte vectors per thread

// zero: 0, or the largest bit pattern where no gradient comes in and none goes out, from a NaN
// either (p is a number from 0 up, or NaN).
template <int DT>
__device__ __forceinline__ float gradient_of(float x, int i, int t, float gl, float ge, float ls,
                                             float H, uint32_t zero) {
    const float lp = x - ls;
    const float p = exp_of(lp);
    const float d = __float_as_uint(p) <= zero ? 0.f : -p * fmaf(ge, lp + H, gl);
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
    const uint32_t zero = gl == 0.f && ge == 0.f ? ~0u : 0u;
    auto one = [&](int i) {
        const float d = gradient_of<DT>(load1<DT>(xr, i), i, t, gl, ge, ls, H, zero);
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
                    gradient_of<DT>(__uint_as_float(w[q]), i + q, t, gl, ge, ls, H, zero));
            } else {
                constexpr bool F16 = DT == BI_F16;
                o[q] = pack16x2(
                    gradient_of<DT>(widen16(uint16_t(w[q]), F16), i + 2 * q, t, gl, ge, ls, H,
                                    zero),
                    gradient_of<DT>(widen16(uint16_t(w[q] >> 16), F16), i + 2 * q + 1, t, gl, ge,
                                    ls, H, zero),
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
    // (indices of a row's padded last vectors stay within 32 bits)
    if (rows < 0 || n < 1 || n > BI_LOGPROBS_MAX_N)
        return fail(BI_ERR_INVALID_ARG, "%s: need rows >= 0 and 1 <= n <= %d", fn,
                    BI_LOGPROBS_MAX_N);
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
    auto run = [&](auto f) {
        return launched(f(*dev, x, ldx, tokens, rows, n, logp, entropy, lse, int(top), top_logp,
                          top_ids, reinterpret_cast<cudaStream_t>(stream)),
                        fn);
    };
    const bool al = aligned(x, 16) && ldx * (x_dtype == BI_F32 ? 4 : 2) % 16 == 0;
    if (x_dtype == BI_F32 && n > 8192)
        return run(al ? launch_forward<BI_F32, 256, true> : launch_forward<BI_F32, 256, false>);
    if (x_dtype == BI_F32)
        return run(al ? launch_forward<BI_F32, 128, true> : launch_forward<BI_F32, 128, false>);
    if (x_dtype == BI_F16)
        return run(al ? launch_forward<BI_F16, 128, true> : launch_forward<BI_F16, 128, false>);
    return run(al ? launch_forward<BI_BF16, 128, true> : launch_forward<BI_BF16, 128, false>);
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
