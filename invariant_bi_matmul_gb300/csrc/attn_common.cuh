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

// The first key that token t at position pos sees; past pos where it sees none.
__device__ __forceinline__ int row_low(const Shape& sh, int t, int pos) {
    int low = sh.window > 0 ? pos - sh.window + 1 : 0;
    if (sh.first_key) low = max(low, sh.first_key[t]);
    return max(low, 0);
}

// The first key that any of the tokens t .. t + n - 1 (positions pos ..) sees; a token that sees
// none counts as if it saw itself, so that every block has a chunk and a page.
__device__ __forceinline__ int block_low(const Shape& sh, int t, int pos, int n) {
    if (!sh.first_key) return min(row_low(sh, t, pos), pos);  // (the window's rises with t)
    int low = pos + n - 1;
    for (int j = 0; j < n; ++j) low = min(low, row_low(sh, t + j, pos + j));
    return low;
}

// v := cap_log2 * tanh(v * cap_in).  Up to |y| = 1 an odd polynomial (2^-24 off; with its fp32
// evaluation 2^-22.5), which needs neither of the two special functions of the other branch,
// 1 - 2 / (1 + e^2y); a warp takes that one for all its scores when one of them is beyond, and
// each score keeps the value of its own range, so a value does not depend on its neighbours.
// tanh.approx, off by 2^-11, would move a score near a cap of 50 by 0.02.
template <int N>
__device__ __forceinline__ void cap_scores(float (&v)[N], float cap_in, float cap_log2) {
    float most = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] *= cap_in;
        most = fmaxf(most, fabsf(v[k]));
    }
    const bool far = __any_sync(0xffffffffu, most > 1.f);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const float y = v[k], z = y * y;
        float p = fmaf(z, 0.00105826475f, -0.0062593394f);
        p = fmaf(z, p, 0.0203597602f);
        p = fmaf(z, p, -0.0534987077f);
        p = fmaf(z, p, 0.133264095f);
        p = fmaf(z, p, -0.333329856f);
        float t = fmaf(z * p, y, y);
        if (far) {
            float r;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(y * (2.f * kLog2e))));
            t = fabsf(y) > 1.f ? fmaf(-2.f, r, 1.f) : t;
        }
        v[k] = __fmul_rn(cap_log2, t);  // (not joined with what the caller adds: one value)
    }
}

// Scores of N consecutive keys of a row, the first at distance `dist` (j - pos), in log2 units.
template <int MODE, int N>
__device__ __forceinline__ void shape_scores(float (&v)[N], const Shape& sh, float scale_log2,
                                             float slope_log2, float dist) {
    if (MODE & kCap) {
        cap_scores(v, sh.cap_in, sh.cap_log2);
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = __fmul_rn(v[k], scale_log2);
    }
    if (MODE & kBias) {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = fmaf(slope_log2, dist + float(k), v[k]);
    }
}

}  // namespace bi
