// attn_common.cuh -- what the split-KV attention kernels (decode / verify in attention.cu,
// chunked prefill in prefill.cu) share: the page and invariant chunk lengths, the lazy
// rescale threshold, the swizzled tile addressing and the per-sequence block geometry.
// The per-query reduction both kernels implement is described at the top of
// attention.cu; prefill.cu reproduces it row by row.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "tmap.h"
#include "bi.h"

namespace bi {

constexpr int PAGE = 64;
constexpr int CHUNK_LOG2 = 9;  // the invariant chunk length: 512 keys
constexpr int CHUNK = 1 << CHUNK_LOG2;
constexpr float kRescaleLog2 = 8.0f;  // rescale O only when the row max grows by > 2^8
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 2^x by the hardware's approximation (PTX ex2.approx.ftz.f32: at most 2 ulp from 2^x;
// results below 2^-126 flush to +0; 2^-inf = +0).  The softmax of every split-KV kernel
// takes P and the rescale factors from this one function, so they agree bit for bit.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// byte offset of (row, 16-byte chunk) in a 128-byte-swizzled box (the TMA SWIZZLE_128B
// pattern: chunk index XOR row mod 8)
__device__ __forceinline__ uint32_t swz(int row, int chunk) {
    return uint32_t(row) * 128u + (uint32_t((chunk ^ (row & 7)) & 7) << 4);
}

// sequence b's block: length L (new tokens included), block width qb, first token t0
struct SeqInfo {
    int L, qb, t0;
};

__device__ __forceinline__ SeqInfo seq_info(const int32_t* seq_lens, const int32_t* cu_q, int b) {
    SeqInfo s;
    s.L = seq_lens[b];
    if (cu_q) {
        s.t0 = cu_q[b];
        s.qb = int(uint32_t(cu_q[b + 1]) - uint32_t(s.t0));  // (wraps: seq_ok takes any value)
    } else {
        s.t0 = b;
        s.qb = 1;
    }
    return s;
}

__device__ __forceinline__ bool seq_ok(const SeqInfo& s, int max_q, int max_seq_len, int total_q) {
    // (no sum of two offsets, which could pass 2^31: a block that ends in total_q or before)
    return s.L >= 1 && s.L <= max_seq_len && s.qb >= 1 && s.qb <= max_q && s.qb <= s.L &&
           s.t0 >= 0 && s.t0 <= total_q - s.qb;
}

// ------------------------------------------------------------------------ shaped scores
// A call may shape its scores before the softmax: x = scale q.k, then
//   x := softcap tanh(x / softcap),  x := x + slope[h] (j - pos),
// and restrict the keys that a token sees to max(first_key[t], pos - window + 1, 0) .. pos.  The
// kernels are compiled for the combinations of kCap and kBias; kRange stands with every shaped
// call.  Shaped scores are held in units of log2 (times log2 e), as the exponents of 2^x.
enum : int { kRange = 1, kCap = 2, kBias = 4 };

struct Shape {
    float cap_in = 0.f;                 // scale / softcap
    float cap_log2 = 0.f;               // softcap * log2 e
    const float* slopes = nullptr;      // [num_q_heads]
    const int32_t* first_key = nullptr; // [total_q]
    int window = 0;                     // 0: none
    int mode = 0;                       // kRange, kCap, kBias; 0: a call that shapes nothing
};

// The first key that the window leaves to position pos.
__device__ __forceinline__ int window_low(const Shape& sh, int pos) {
    return sh.window > 0 ? max(pos - sh.window + 1, 0) : 0;
}

// The first key that token t at position pos sees; past pos where it sees none.
__device__ __forceinline__ int row_low(const Shape& sh, int t, int pos) {
    const int low = window_low(sh, pos);
    return sh.first_key ? max(low, sh.first_key[t]) : low;
}

// The first key that any of the tokens t .. t + n - 1 (positions pos ..) sees; a token that sees
// none counts as if it saw itself, so that every block has a chunk and a page.
__device__ __forceinline__ int block_low(const Shape& sh, int t, int pos, int n) {
    if (!sh.first_key) return window_low(sh, pos);  // (it rises with the position)
    int low = pos + n - 1;
    for (int j = 0; j < n; ++j) low = min(low, row_low(sh, t + j, pos + j));
    return low;
}

// Which of 16 consecutive keys lie in low .. last (both counted from the first of them).
__device__ __forceinline__ uint32_t keys_between(int low, int last) {
    low = max(low, 0);
    last = min(last, 15);
    return last >= low ? ((2u << last) - 1u) & ~((1u << low) - 1u) : 0u;
}

// Zeroes those of the 16 value rows from row r0 on of a page in shared memory (BOXES boxes of 64
// columns, BOX_BYTES apart) that no query sees: a weight of 0 times a value that is not finite
// would be NaN.  A warp calls it together; the caller orders it before the product.
template <int BOXES, int BOX_BYTES>
__device__ __forceinline__ void zero_unseen(uint8_t* v, int r0, uint32_t seen) {
#pragma unroll 1
    for (int idx = int(threadIdx.x) & 31; idx < BOXES * 128; idx += 32) {
        const int row = (idx >> 3) & 15;
        if (!((seen >> row) & 1u))
            *reinterpret_cast<uint4*>(v + (idx >> 7) * BOX_BYTES + (r0 + row) * 128 +
                                      (idx & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
}

// cap_log2 * tanh(s * cap_in) of a warp's scores.  Up to |y| = 1 an odd polynomial (2^-24 off;
// with its fp32 evaluation 2^-22.5), which needs neither of the two special functions of the other
// branch, 1 - 2 / (1 + e^2y), and goes two scores to an instruction; a warp takes the other one for
// all its scores when one of them is beyond, and each score keeps the value of its own range, so a
// value does not depend on its neighbours.  (tanh.approx, off by 2^-11, would move a score near a
// cap of 50 by 0.02.)  Every operation is one that the compiler joins with no other: the kernels
// that call this have the same bits.
__device__ __forceinline__ float far_tanh(float y) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.f, ex2(__fmul_rn(y, 2.f * kLog2e)))));
    return fmaf(-2.f, r, 1.f);
}
template <int N>
__device__ __forceinline__ void cap_scores(float (&v)[N], float cap_in, float cap_log2) {
    static_assert(N % 2 == 0, "pairs");
    constexpr float c1 = -0.333329856f, c2 = 0.133264095f, c3 = -0.0534987077f,
                    c4 = 0.0203597602f, c5 = -0.0062593394f, c6 = 0.00105826475f;
    auto both = [](float x) { return make_float2(x, x); };
    float2 t[N / 2];
    float most = 0.f;
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
        const float2 y = mul2(make_float2(v[2 * k], v[2 * k + 1]), both(cap_in));
        v[2 * k] = y.x;
        v[2 * k + 1] = y.y;
        most = fmax3(most, fabsf(y.x), fabsf(y.y));
        const float2 z = mul2(y, y);
        float2 p = fma2(z, both(c6), both(c5));
        p = fma2(z, p, both(c4));
        p = fma2(z, p, both(c3));
        p = fma2(z, p, both(c2));
        p = fma2(z, p, both(c1));
        t[k] = fma2(mul2(z, p), y, y);
    }
    if (__builtin_expect(__any_sync(0xffffffffu, most > 1.f), 0)) {  // (out of the common line)
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
            if (fabsf(v[2 * k]) > 1.f) t[k].x = far_tanh(v[2 * k]);
            if (fabsf(v[2 * k + 1]) > 1.f) t[k].y = far_tanh(v[2 * k + 1]);
        }
    }
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
        const float2 x = mul2(both(cap_log2), t[k]);
        v[2 * k] = x.x;
        v[2 * k + 1] = x.y;
    }
}
__device__ __forceinline__ float cap_score(float s, float cap_in, float cap_log2) {
    float v[2] = {s, s};
    cap_scores(v, cap_in, cap_log2);
    return v[0];
}

// Scores of N consecutive keys, in log2 units; slope: the row's, times log2 e, and dist: how far
// the first key is from the row's position (j - pos; whole numbers below 2^24 are exact, and so is
// their sum with k: a bias at a short distance is not the difference of two long ones).
template <int MODE, int N>
__device__ __forceinline__ void shape_scores(float (&v)[N], const Shape& sh, float scale_log2,
                                             float slope, float dist) {
    if (MODE & kCap) cap_scores(v, sh.cap_in, sh.cap_log2);
    if (MODE & kBias) {
        auto both = [](float x) { return make_float2(x, x); };
#pragma unroll
        for (int k = 0; k < N; k += 2) {
            float2 s = make_float2(v[k], v[k + 1]);
            if (!(MODE & kCap)) s = mul2(s, both(scale_log2));
            s = fma2(both(slope), add2(both(dist), make_float2(float(k), float(k + 1))), s);
            v[k] = s.x;
            v[k + 1] = s.y;
        }
    }
}

// The running reference of a row's softmax (log2 units) and its raises: by a page's largest score
// where that exceeds it by more than 2^8.  With a cap the reference is the capped score of the
// largest one at its last raise, and a raise is judged by the scores before the cap, of which it
// takes no more than their difference: so a page that raises nothing forms no capped maximum.
template <int MODE>
struct Reference {
    float m = -INFINITY;    // scores are taken relative to it
    float seen = -INFINITY; // what raises are judged by
    // page: the page's largest score as the MMA left it, or shaped with a bias; returns whether
    // the reference was raised, and by which factor sums and O shrink
    __device__ __forceinline__ bool raise(float page, const Shape& sh, float scale_log2,
                                          float& factor) {
        const float now = (MODE & kBias) ? page : __fmul_rn(page, scale_log2);
        const bool up = now > __fadd_rn(seen, kRescaleLog2) || (seen == -INFINITY && now != -INFINITY);
        factor = 1.f;
        if (__any_sync(0xffffffffu, up)) {
            const float to = ((MODE & kCap) && !(MODE & kBias))
                                 ? cap_score(page, sh.cap_in, sh.cap_log2)
                                 : now;
            if (up) {
                factor = ex2(__fadd_rn(m, -to));
                m = to;
                seen = now;
            }
        }
        return up;
    }
};

}  // namespace bi
