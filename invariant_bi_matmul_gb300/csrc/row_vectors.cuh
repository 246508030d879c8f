// row_vectors.cuh -- what the kernels that read rows of logits share: 16-byte vectors of rows of
// any alignment, their elements and their order.
#pragma once

#include "bi.h"
#include "common.cuh"

namespace bi {

constexpr int kBatch = 8;              // vectors that a thread requests at a time
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

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {  // at most 2 ulp from 2^x; 0 below 2^-126
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// e^d, d <= 0 (the argument of 2^ is rounded once)
__device__ __forceinline__ float exp_of(float d) { return ex2(d * kLog2e); }

// What a maximum is taken off: the maximum, or 0 where there is none.
__device__ __forceinline__ float ref_of(float m) { return m == -INFINITY ? 0.f : m; }

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

}  // namespace bi
