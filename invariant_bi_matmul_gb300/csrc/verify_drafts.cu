// verify_drafts.cu -- verification of drafted tokens against the target's probabilities from
// given uniform numbers (include/bi_rowwise.h, bi_verify_drafts).
//
// With p = softmax(x / T) of a target row and q the draft's probabilities, draft j is kept while
// u q(token) < p(token); the block's last token is drawn by inverting the cumulative sums of
// D_i = max(p_i - q_i, 0) (behind a refused draft) or of p_i.  Two launches:
//
// Statistics.  A warp takes one part of a row (kBatch vectors a lane, all requested before any is
// used) and leaves the part's maximum, sum of 2^((x - m) log2 e / T) in fp32 and, for a sequence
// at temperature 0, its largest entry.  Every target row and every draft row is read once, which
// is what the call cannot do without.  (Persistent warps that request the next part before they
// use this one had fewer loads under way: 32 sequences of up to 5 rows 43 us, 29 as it is.)
//
// Decision and draw.  A cluster of CTAs per sequence joins the parts (lanes over the parts, a
// butterfly), finds the first refused draft, and goes over that row, and the draft's, once more.
// A drawn token must not depend on how sums round, or it would depend on the order in which they
// are taken: near equal entries of 2^-17 of the mass, fp32 sums would choose a neighbour in one
// row of a few hundred.  So each weight is a whole number, 2^60 p_i, from a product x c in two
// floats and 2^(j/32) (fixed_exp), off by at most 2^-29 of itself, and sums of whole
// numbers are exact in any order: the token is the same whatever the split, in one row in 10^5 or
// so another than the definition's.  The fp32 statistics only scale the weights to sums near
// 2^60; what the sums come to, sp and sq, corrects that: D_i is proportional to
// max(p_i sq/sp - q_i, 0), and with e = sq/sp - 1 = sum (q_i - p_i) / 2^60 (1e-6 at most) the sum
// of D over a block is sum max(p_i - q_i, 0) + e * sum of p_i where p_i > q_i, but for entries
// whose p and q agree to within e, which weigh e times as much.  One pass so gives the totals,
// the correction and the sums of each block of 512; the block that holds the drawn share is taken
// again, entry by entry.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <type_traits>

#include "bi.h"
#include "bi_rowwise.h"
#include "launch.h"
#include "row_vectors.cuh"

#define BI_EXPORT extern "C" __attribute__((visibility("default")))

namespace bi {

void set_last_error_message(const char* msg);

namespace {

constexpr int kStats = 128;                             // threads of a statistics CTA
constexpr int kThreads = 256;                           // ... and of the others
constexpr int kBlock = 512;                             // entries of a block: 16 for each lane
constexpr int kMaxCtas = 8;                             // of a sequence's cluster
constexpr int kMaxBlocks = (BI_DRAFTS_MAX_N + kBlock - 1) / kBlock;
constexpr float kHot = 0x1p-64f;                        // temperatures below it are 0

template <int DT>
constexpr int kPartLen = 32 * kBatch * (16 / kSize<DT>);  // entries of a part

struct PartStats {
    float m, s;
    unsigned long long best;  // order_key of the largest entry (temperature 0 alone)
};

struct DraftArgs {
    const void* x;            // target rows [total_q, n]
    const void* y;            // draft rows [num_drafts, n], or null: q = 1 at the token
    int64_t ldx, ldy;
    const int32_t* draft_tokens;
    const float* uniforms;
    const float* temperatures;  // null: `temperature` for all
    const int32_t* cu_q;
    PartStats* parts;         // [total_q + num_drafts][nparts]
    int32_t* tokens;
    int32_t* accepted;
    float* logprobs;
    unsigned int* err;
    float temperature;
    int B, total_q, num_drafts, max_q, n, nparts, items;  // items: parts of all rows
    int ahead;                // parts to fetch ahead in the statistics' own launch, or 0
};

__device__ __forceinline__ float temperature_of(const DraftArgs& a, int b) {
    const float t = a.temperatures ? a.temperatures[b] : a.temperature;
    return t < kHot ? (t >= 0.f ? 0.f : kNaN) : isfinite(t) ? t : kNaN;  // NaN: refused
}

// log2 e / T in two floats, to 2^-46 of itself.
struct Rate {
    float hi, lo;
};
__device__ __noinline__ Rate rate_of(float T) {
    if (T == 0.f) T = 1.f;
    Rate c;
    c.hi = kLog2e / T;
    c.lo = (fmaf(-c.hi, T, kLog2e) + 1.925963033500e-8f) / T;  // (log2 e - float(log2 e))
    return c;
}

// --------------------------------------------------------------------------- statistics

// The statistics of one part, by a warp; temperature(): the row's, asked for once the loads are
// under way (NaN: nothing to do for this row).
template <int DT, bool ALIGNED, class Temperature>
__device__ __forceinline__ void part_stats(const DraftArgs& a, int row, int part,
                                           Temperature temperature) {
    constexpr int VE = 16 / kSize<DT>, kLen = 32 * kBatch;  // vectors of a part
    const int lane = threadIdx.x & 31, warp0 = threadIdx.x & ~31;
    const bool draft = row >= a.total_q;
    const int r = draft ? row - a.total_q : row;
    const char* xr = static_cast<const char*>(draft ? a.y : a.x) +
                     int64_t(r) * (draft ? a.ldy : a.ldx) * kSize<DT>;
    const uint32_t skew = ALIGNED ? 0u : uint32_t(reinterpret_cast<uintptr_t>(xr) & 15u);
    uint4 v[kBatch];
    // (load_batch counts a CTA's threads: this warp's are 0 .. 31)
    load_batch<DT, 32, ALIGNED>(v, xr, skew, part * kLen - warp0,
                                min((a.n + VE - 1) / VE, (part + 1) * kLen), a.n);
    const float T = temperature();
    const bool greedy = T == 0.f;
    if (isnan(T) || (greedy && draft)) return;
    const float c = rate_of(T).hi;

    float m = vec_max<DT>(v[0]);
#pragma unroll
    for (int k = 1; k < kBatch; ++k) m = fmaxf(m, vec_max<DT>(v[k]));
    const float ref = -ref_of(m);
    float2 s2 = make_float2(0.f, 0.f);      // (entries past the row are -inf: they add 0)
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        float e[VE];
        widen<DT>(v[k], e);
#pragma unroll
        for (int q = 0; q < VE; q += 2) {
            const float2 t = mul2(add2(make_float2(e[q], e[q + 1]), make_float2(ref, ref)),
                                  make_float2(c, c));
            s2 = add2(s2, make_float2(ex2(t.x), ex2(t.y)));
        }
    }
    float s = s2.x + s2.y;
    unsigned long long best = 0;
    if (greedy) {  // (read again, one vector after the other: unrolled, this doubled the kernel)
#pragma unroll 1
        for (int k = 0; k < kBatch; ++k) {
            const int g = part * kLen + k * 32 + lane;
            float e[VE];
            widen<DT>(load_vec<DT>(xr, skew == 0, g, a.n), e);
#pragma unroll
            for (int q = 0; q < VE; ++q) {
                if (g * VE + q < a.n) {
                    const unsigned long long key = order_key(e[q], g * VE + q);
                    best = key > best ? key : best;
                }
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const unsigned long long o = __shfl_xor_sync(~0u, best, off);
            best = o > best ? o : best;
        }
    }
    float M = m;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, off));
    if (m != -INFINITY) s *= ex2((m - M) * c);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(~0u, s, off);
    if (lane == 0) a.parts[int64_t(row) * a.nparts + part] = PartStats{M, s, best};
}

// A part into L2 (its whole 16-byte pieces), by a warp's first lane: the one that a warp of the
// next wave will take, so that the memory is not idle while this wave computes.  Worth it while
// there are few waves (32 sequences of up to 5 rows of 128,256 fp32, four waves, 49.8 us with it and
// 53.3 without; 128 of 8 in bf16, 22 waves that are long out of step, 169 and 164).
template <int DT>
__device__ __forceinline__ void prefetch_part(const DraftArgs& a, int item) {
    if ((threadIdx.x & 31) != 0 || item >= a.items) return;
    const int row = int(unsigned(item) / unsigned(a.nparts)), part = item - row * a.nparts;
    const bool draft = row >= a.total_q;
    const uintptr_t from = reinterpret_cast<uintptr_t>(draft ? a.y : a.x) +
                           uintptr_t(int64_t(draft ? row - a.total_q : row) *
                                     (draft ? a.ldy : a.ldx)) * kSize<DT>;
    const uintptr_t end = (from + uintptr_t(a.n) * kSize<DT>) & ~uintptr_t(15);
    constexpr uintptr_t kBytes = 32 * kBatch * 16;
    const uintptr_t at = (from + part * kBytes + 15) & ~uintptr_t(15);
    if (at >= end) return;
    const uint32_t bytes = uint32_t(end - at < kBytes ? end - at : kBytes);
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(bytes) : "memory");
}

template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kStats, !ALIGNED ? 6 : DT == BI_F32 ? 9 : 8)
draft_stats_kernel(const DraftArgs a) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int item = int(blockIdx.x) * (kStats / 32) + int(threadIdx.x >> 5);
    if (item >= a.items) return;
    const int row = int(unsigned(item) / unsigned(a.nparts)), part = item - row * a.nparts;
    part_stats<DT, ALIGNED>(a, row, part, [&]() {
        if (a.ahead) prefetch_part<DT>(a, item + a.ahead);
        // the row's sequence: target rows of b are cu_q[b] .., draft rows cu_q[b] - b ..  (By
        // counting, a lane's loads all at once: a binary search waits for one after the other.)
        const bool draft = row >= a.total_q;
        const int r = draft ? row - a.total_q : row;
        int b = 0;
        for (int i = lane; i < a.B; i += 32) b += a.cu_q[i] - (draft ? i : 0) <= r ? 1 : 0;
        b = max(__reduce_add_sync(~0u, b) - 1, 0);
        const float T = temperature_of(a, b);
        return r < a.cu_q[b + 1] - (draft ? b + 1 : 0) ? T : kNaN;
    });
}

// ---------------------------------------------------------------- weights in whole numbers

// Lane j's register holds 2^31 * 2^(j/32), rounded; a lane takes the one it needs by a shuffle.
// (A table of 512 in shared memory, with a shorter series, cost twelve cycles of its pipe for each
// look-up of a warp, and bound the kernel.)
__constant__ uint32_t kPowers[32] = {
    0x80000000u, 0x82cd8699u, 0x85aac368u, 0x88980e81u, 0x8b95c1e4u, 0x8ea4398bu,
    0x91c3d374u, 0x94f4efa9u, 0x9837f052u, 0x9b8d39bau, 0x9ef53261u, 0xa2704303u,
    0xa5fed6aau, 0xa9a15ab5u, 0xad583eeau, 0xb123f582u, 0xb504f334u, 0xb8fbaf47u,
    0xbd08a39fu, 0xc12c4ccau, 0xc5672a11u, 0xc9b9bd86u, 0xce248c15u, 0xd2a81d92u,
    0xd744fccbu, 0xdbfbb798u, 0xe0ccdeecu, 0xe5b906e7u, 0xeac0c6e8u, 0xefe4b99cu,
    0xf5257d15u, 0xfa83b2dbu,
};

// How a row's entries become weights 2^60 * 2^(x c - K), K = m c + log2 s (about), as
// 2^((x - m0) c - i - f / 2^30): c in two floats, and m0 = 0, so that x needs no subtraction, or m
// where m c is large, when x - m is exact for every x near enough to m to have a weight.
struct RowScale {
    float m0, ch, cl, alive;  // alive: what (x - m0) c exceeds in an entry with a weight
    int i, f;
};

// All lanes of a warp call it together; power: the lane's entry of kPowers.
__device__ __forceinline__ unsigned long long fixed_exp(float x, const RowScale& r,
                                                        uint32_t power) {
    constexpr float kMagic = 12582912.f;    // 1.5 * 2^23: adding it rounds to a whole number
    constexpr uint32_t kMagicBits = 0x4b400000u;
    // t + tl = (x - m0) c to 2^-46 of itself, |t| < 2^14
    const float d = x - r.m0;
    const float t = d * r.ch;
    const float tl = fmaf(d, r.cl, fmaf(d, r.ch, -t));
    // whole part and fraction, in 2^-30: each of three terms is rounded to that
    const float whole = t + kMagic;
    const uint32_t us = uint32_t(__float2int_rn((t - (whole - kMagic)) * 0x1p30f)) +
                        (uint32_t(__float_as_int(fmaf(tl, 0x1p30f, kMagic))) - kMagicBits) -
                        uint32_t(r.f);
    const int s = int(us);
    const int N = int(uint32_t(__float_as_int(whole)) - kMagicBits - uint32_t(r.i) +
                      uint32_t(s >> 30));
    // 2^(fraction): kPowers at its first five bits; of the other 25, z = (s mod 2^25) / 2^30, the
    // linear term of 2^z - 1 in whole numbers (2^-32) and the rest, at most 2^-12, in fp32, as the
    // low bits of 2^23 + ...
    const uint32_t hi = __shfl_sync(~0u, power, s >> 25);
    const uint32_t z = us << 7;
    constexpr float kZ = 0.6931471805599453f / 32.f;  // y = 32 z
    constexpr float b2 = 0x1p32f * kZ * kZ / 2.f, b3 = 0x1p32f * kZ * kZ * kZ / 6.f,
                    b4 = 0x1p32f * kZ * kZ * kZ * kZ / 24.f;
    const float y = __uint_as_float((z >> 9) | 0x3f800000u) - 1.f;
    const float g = fmaf(y * y, fmaf(y, fmaf(y, b4, b3), b2), 8388608.f);
    const uint32_t G = __umulhi(z, 93032640u) + (__float_as_uint(g) - 0x4b000000u);  // ln 2 * 2^27
    // (t is -inf or NaN where an entry is -inf, or far below the maximum: no weight)
    const uint32_t w = t > r.alive ? hi + __umulhi(hi, G) : 0u;
    return (static_cast<unsigned long long>(w) << 32) >> min(uint32_t(3 - N) & 0xffu, 63u);
}

// A sum of max(p - q, 0), with p raised by e of itself (e in 2^-46); p: the sum of the upper words
// of p where p > q.
__device__ __forceinline__ unsigned long long corrected(unsigned long long d, uint32_t p, int e) {
    return d + static_cast<unsigned long long>((static_cast<long long>(p) * e) >> 14);
}

// ------------------------------------------------------------------------ decision and draw

struct RowStats {
    float m, s;
    unsigned long long best;
};

// The parts of a row together, the same in every lane of a warp: each lane's in ascending order,
// four of them requested at a time, then a butterfly.
__device__ __noinline__ RowStats join_parts(const PartStats* p, int nparts, float c) {
    const int lane = threadIdx.x & 31;
    RowStats r{-INFINITY, 0.f, 0ull};
    auto add = [&](float m, float s) {      // (a part of nothing but -inf and NaN has s = 0 or NaN)
        const float M = fmaxf(r.m, m);
        if (M != -INFINITY) {
            r.s = r.m == -INFINITY ? r.s : r.s * ex2((r.m - M) * c);
            s = m == -INFINITY ? s : s * ex2((m - M) * c);
        }
        r.s += s;
        r.m = M;
    };
#pragma unroll 1
    for (int i0 = 0; i0 < nparts; i0 += 128) {
        PartStats q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + 32 * k + lane;
            q[k] = PartStats{-INFINITY, 0.f, 0ull};
            if (i < nparts) q[k] = p[i];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            add(q[k].m, q[k].s);
            r.best = q[k].best > r.best ? q[k].best : r.best;
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        add(__shfl_xor_sync(~0u, r.m, off), __shfl_xor_sync(~0u, r.s, off));
        const unsigned long long o = __shfl_xor_sync(~0u, r.best, off);
        r.best = o > r.best ? o : r.best;
    }
    return r;
}

__device__ __forceinline__ bool has_distribution(const RowStats& r) {
    return isfinite(r.m) && isfinite(r.s);  // (a NaN or +inf in the row makes s NaN)
}

__device__ __noinline__ RowScale scale_of(const RowStats& r, const Rate& c) {
    RowScale k;
    k.ch = c.hi;
    k.cl = c.lo;
    k.m0 = fabsf(r.m) * c.hi < 8192.f ? 0.f : r.m;
    const float d = r.m - k.m0, t = d * c.hi, tl = fmaf(d, c.lo, fmaf(d, c.hi, -t));
    const float L = log2f(r.s), i = rintf(L), whole = rintf(t);
    const int f = __float2int_rn((t - whole) * 0x1p30f) + __float2int_rn(tl * 0x1p30f) +
                  __float2int_rn((L - i) * 0x1p30f);
    k.i = int(whole) + int(i) + (f >> 30);
    k.f = f & 0x3fffffff;
    k.alive = float(k.i - 62);
    return k;
}

// (x - m) c in two floats.
__device__ __forceinline__ float2 exponent_of(float x, const RowStats& r, const Rate& c) {
    const float d = x - r.m, xs = d + r.m, dl = (x - xs) + ((xs - d) - r.m), t = d * c.hi;
    return make_float2(t, fmaf(dl, c.hi, fmaf(d, c.lo, fmaf(d, c.hi, -t))));
}

// (not inlined: it stands at several places of a kernel that runs from a cold cache)
__device__ __noinline__ float logp_of(float x, const RowStats& r, const Rate& c) {
    const float2 t = exponent_of(x, r, c);
    // (the type's lowest value: times log2 e it is past fp32's range, by itself it need not be)
    if (t.x == -INFINITY) return (x - r.m) * (c.hi * kLn2);
    return fmaf(t.x, kLn2, t.y * kLn2) - logf(r.s);
}

// floor(u * Z) for 0 <= u < 1.
__device__ __forceinline__ unsigned long long share_of(float u, unsigned long long Z) {
    const uint32_t bits = __float_as_uint(u);
    const int e = int(bits >> 23);
    const unsigned long long m = e ? (bits & 0x7fffffu) | 0x800000u : bits;  // u = m / 2^(150 - e)
    const int shift = 150 - max(e, 1);                                       // 24 .. 149
    const unsigned long long lo = m * Z, hi = __umul64hi(m, Z);
    return shift >= 128 ? 0ull : shift >= 64 ? hi >> (shift - 64)
                                             : (hi << (64 - shift)) | (lo >> shift);
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(~0u, v, off);
    return v;
}
__device__ __forceinline__ unsigned long long warp_scan(unsigned long long v) {  // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned long long o = __shfl_up_sync(~0u, v, off);
        if (lane >= off) v += o;
    }
    return v;
}

struct Sums {
    unsigned long long d;  // of max(p - q, 0)
    uint32_t p;            // of p's upper words where p > q
};

// AHEAD: iterations whose entries are under way.  With one CTA or two on a multiprocessor a warp
// waits for its own loads (a row of 128,256 entries over eight CTAs, the whole call 17.5 us with
// one iteration, 15.3 with four); with three CTAs the others fill the time, and the registers are
// better spent on them.
// OWN: the cluster takes its sequence's statistics itself (1: rows aligned, 2: not), for blocks of
// few parts: one launch less.
template <int DT, int AHEAD, int OWN>
__global__ void __launch_bounds__(kThreads, AHEAD > 1 ? 2 : 3)
draft_draw_kernel(const DraftArgs a, int ctas) {
    constexpr int kWarps = kThreads / 32, kGroups = kBlock / 32;
    constexpr int kAtOnce = 4, kSteps = kGroups / kAtOnce;  // entries of a block per lane
    __shared__ Sums block_sums[kMaxBlocks];
    __shared__ unsigned long long warp_sums[kWarps][3];
    __shared__ unsigned long long cta_sums[kMaxCtas][3];  // every CTA's: p - q, and Sums
    __shared__ RowStats last[2];                          // of the row that ends the block: p, q
    __shared__ int first_refused, the_block;
    __shared__ Sums the_start;
    __shared__ unsigned long long weights[kGroups][32], group_sums[kGroups];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = int(blockIdx.x / unsigned(ctas)), rank = int(blockIdx.x - unsigned(b) * ctas);
    const uint32_t power = kPowers[lane];
    if (tid == 0) first_refused = 0x7fffffff;
    pdl_wait();
    pdl_trigger();
    // the offsets of the whole batch: a call with malformed ones decides nothing
    bool bad = tid == 0 && (a.cu_q[0] != 0 || a.cu_q[a.B] > a.total_q ||
                            a.cu_q[a.B] - a.B > a.num_drafts);
#pragma unroll 1
    for (int i = tid; i < a.B; i += kThreads) {
        const int w = int(uint32_t(a.cu_q[i + 1]) - uint32_t(a.cu_q[i]));
        bad |= w < 1 || w > a.max_q || a.cu_q[i + 1] < 0;  // (so they rise: none wraps)
    }
    const float T0 = temperature_of(a, b);
    const int t0 = a.cu_q[b], drafts = a.cu_q[b + 1] - t0 - 1;
    bad = __syncthreads_or(bad) != 0;
    const float T = bad ? kNaN : T0;
    int32_t* out = a.tokens + int64_t(b) * a.max_q;
    float* out_logp = a.logprobs ? a.logprobs + int64_t(b) * a.max_q : nullptr;
    if (isnan(T)) {
        if (rank == 0) {
#pragma unroll 1
            for (int j = tid; j < a.max_q; j += kThreads) {
                out[j] = -1;
                if (out_logp) out_logp[j] = 0.f;
            }
            if (tid == 0) {
                a.accepted[b] = 0;
                latch_error(a.err, kErrDeviceArg);
            }
        }
        return;
    }
    const bool greedy = T == 0.f;
    const Rate c = rate_of(T);
    const int d0 = t0 - b;                  // the sequence's first draft
    const int64_t es = kSize<DT>;
    auto target_row = [&](int j) {
        return static_cast<const char*>(a.x) + int64_t(t0 + j) * a.ldx * es;
    };
    auto draft_row = [&](int j) {
        return static_cast<const char*>(a.y) + int64_t(d0 + j) * a.ldy * es;
    };

    if (OWN) {
        const int rows = drafts + 1 + (a.y && !greedy ? drafts : 0);
#pragma unroll 1
        for (int i = rank * kWarps + warp; i < rows * a.nparts; i += ctas * kWarps) {
            const int r = i / a.nparts;
            part_stats<DT, OWN == 1>(a, r <= drafts ? t0 + r : a.total_q + d0 + r - drafts - 1,
                                     i - r * a.nparts, [&]() { return T; });
        }
        // (the barriers order the parts in global memory, too)
        if (ctas > 1) cluster_sync_all(); else __syncthreads();
    }
    // a warp per draft, and one for the row behind the last; a warp stops at its first refusal,
    // since no later row of its own ends the block
    RowStats P{0.f, 1.f, 0ull}, Q{0.f, 1.f, 0ull};
    int mine = -1;
#pragma unroll 1
    for (int j = warp; j <= drafts && mine < 0; j += kWarps) {
        const int token = j < drafts ? a.draft_tokens[d0 + j] : -1;
        const bool inside = token >= 0 && token < a.n;
        const bool with_q = inside && a.y && !greedy;
        float x = 0.f, y = 0.f, u = 0.f;
        if (inside) x = load1<DT>(target_row(j), token);
        if (with_q) y = load1<DT>(draft_row(j), token);
        if (inside) u = a.uniforms[t0 + j];
        const PartStats* const qp = a.parts + (int64_t(a.total_q) + d0 + j) * a.nparts;
        if (with_q && lane * 8 < a.nparts)  // (on their way while the target's parts are joined)
            asm volatile("prefetch.global.L1 [%0];" ::"l"(qp + lane * 8));
        P = join_parts(a.parts + int64_t(t0 + j) * a.nparts, a.nparts, c.hi);
        if (with_q) Q = join_parts(qp, a.nparts, c.hi);
        bool take = false;
        if (inside && greedy) {
            take = has_distribution(P) && 0x7fffffff - int(uint32_t(P.best)) == token;
        } else if (inside && has_distribution(P) && x != -INFINITY) {
            // u 2^tq / sq < 2^tp / sp
            const float2 tp = exponent_of(x, P, c);
            float2 tq = make_float2(0.f, 0.f);
            bool fine = true;
            if (with_q) {
                fine = has_distribution(Q);
                tq = exponent_of(y, Q, c);
            }
            const float t = tq.x - tp.x, back = t + tp.x;
            const float tl = ((tq.x - back) + ((back - t) - tp.x)) + (tq.y - tp.y);
            const float e = exp2f(t) * (isfinite(t) ? fmaf(tl, kLn2, 1.f) : 1.f);
            take = fine && (u == 0.f || u * e * P.s < (with_q ? Q.s : 1.f));
        } else if (!inside && token != -1 && lane == 0 && rank == 0) {
            latch_error(a.err, kErrDeviceArg);
        }
        if (!take) {
            mine = j;
            if (lane == 0) atomicMin(&first_refused, j);
        } else if (rank == 0 && lane == 0) {
            out[j] = token;
            if (out_logp) out_logp[j] = logp_of(x, P, c);
        }
    }
    __syncthreads();
    const int kept = first_refused;         // (at most `drafts`)
    if (mine == kept && lane == 0) {
        last[0] = P;
        last[1] = Q;
    }
    const int refused = kept < drafts ? a.draft_tokens[d0 + kept] : -1;  // -1: drawn from p
    const bool behind = refused >= 0 && refused < a.n;
    const float u_last = a.uniforms[t0 + drafts];
    if (rank == 0) {
#pragma unroll 1
        for (int j = kept + 1 + tid; j < a.max_q; j += kThreads) {
            out[j] = -1;
            if (out_logp) out_logp[j] = 0.f;
        }
        if (tid == 0) a.accepted[b] = kept;
    }
    __syncthreads();
    P = last[0];
    const char* xr = target_row(kept);
    auto emit = [&](int token) {
        out[kept] = token;
        if (out_logp) out_logp[kept] = token < 0 ? kNaN : logp_of(load1<DT>(xr, token), P, c);
    };
    if (greedy) {
        if (rank == 0 && tid == 0)
            emit(has_distribution(P) ? 0x7fffffff - int(uint32_t(P.best)) : -1);
        return;
    }
    bool both = behind && a.y;              // subtract the draft's probabilities
    Q = last[1];
    if (!has_distribution(P) || (both && !has_distribution(Q))) {
        if (rank == 0 && tid == 0) emit(-1);
        return;
    }
    int without = behind && !a.y ? refused : -1;  // q = 1 there: that entry has no weight
    const char* yr = both ? draft_row(kept) : nullptr;
    const RowScale kp = scale_of(P, c), kq = both ? scale_of(Q, c) : kp;
    const int blocks = (a.n + kBlock - 1) / kBlock;
    // (at most 2^11 blocks and 8 CTAs)
    const int k0 = rank * blocks / ctas, k1 = (rank + 1) * blocks / ctas;

    if (!OWN && ctas > 1) cluster_sync_all();  // (the others have started)
    unsigned long long Z = 0;
    int e = 0;
    Sums before{0, 0};                      // of the CTAs in front of the one that holds the share
    int holder = 0;
    unsigned long long share = 0;
    for (;;) {
        unsigned long long diff = 0, sd = 0;
        uint32_t sp = 0;
        // (rolled loops: the code runs from a cold instruction cache, and unrolled over a block
        // it was 180 KB, which took longer to fetch than to run)
        auto pass = [&](auto subtracts) {
            constexpr bool BOTH = decltype(subtracts)::value;
            constexpr int N = BOTH ? 2 * kAtOnce : kAtOnce;  // target entries, then draft's
            float x[AHEAD][N];                               // of this iteration and the next ones
            auto fetch = [&](float (&to)[N], int it) {
                const int i0 = (k0 + warp + it / kSteps * kWarps) * kBlock +
                               it % kSteps * (kAtOnce * 32) + lane;
                const bool all = i0 - lane + kAtOnce * 32 <= a.n;
#pragma unroll
                for (int q = 0; q < N; ++q) {
                    const int i = i0 + q % kAtOnce * 32;
                    to[q] = -INFINITY;
                    if (all || i < a.n) to[q] = load1<DT>(q < kAtOnce ? xr : yr, i);
                }
            };
            const int its = (max(0, k1 - k0 - warp) + kWarps - 1) / kWarps * kSteps;
#pragma unroll
            for (int f = 0; f < AHEAD; ++f)
                if (f < its) fetch(x[f], f);
            Sums s{0, 0};
#pragma unroll 1
            for (int it = 0; it < its; ++it) {
                float now[N];
#pragma unroll
                for (int q = 0; q < N; ++q) {
                    now[q] = x[0][q];
#pragma unroll
                    for (int f = 1; f < AHEAD; ++f) x[f - 1][q] = x[f][q];
                }
                if (it + AHEAD < its) fetch(x[AHEAD - 1], it + AHEAD);
#pragma unroll
                for (int q = 0; q < kAtOnce; ++q) {
                    const unsigned long long p = fixed_exp(now[q], kp, power);
                    if (BOTH) {
                        const unsigned long long over =
                            p - fixed_exp(now[(q + kAtOnce) % N], kq, power);
                        diff += over;
                        if (static_cast<long long>(over) > 0) {
                            s.d += over;
                            s.p += uint32_t(p >> 32);
                        }
                    } else {
                        s.d += p;
                    }
                }
                if (it % kSteps == kSteps - 1) {
                    const int k = warp + it / kSteps * kWarps;
                    s.d = warp_sum(s.d);
                    if (BOTH) s.p = __reduce_add_sync(~0u, s.p);
                    if (!BOTH && without >= 0 && without / kBlock == k0 + k)
                        s.d -= fixed_exp(load1<DT>(xr, without), kp, power);
                    if (lane == 0) block_sums[k] = s;
                    sd += s.d;
                    sp += s.p;
                    s = Sums{0, 0};
                }
            }
            if (BOTH) diff = warp_sum(diff);
        };
        if (both) pass(std::true_type()); else pass(std::false_type());
        if (lane == 0) {
            warp_sums[warp][0] = diff;
            warp_sums[warp][1] = sd;
            warp_sums[warp][2] = sp;
        }
        __syncthreads();
        if (tid < 4 * ctas && (tid & 3) < 3) {  // a thread per sum and CTA to tell it to
            const int i = tid & 3, to = tid >> 2;
            unsigned long long v = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += warp_sums[w][i];
            if (to == rank)
                cta_sums[rank][i] = v;
            else
                st_cluster_b64(cluster_map(smem_addr(&cta_sums[rank][i]), to), v);
        }
        if (ctas > 1) cluster_sync_all(); else __syncthreads();
        // every thread of the cluster comes to the same numbers
        unsigned long long all[3] = {0, 0, 0};
#pragma unroll 1
        for (int r = 0; r < ctas; ++r)
#pragma unroll
            for (int i = 0; i < 3; ++i) all[i] += cta_sums[r][i];
        // e = sum (q - p) / 2^60, in 2^-46
        if (both)
            e = int(max(-(1ll << 30), min(1ll << 30, -static_cast<long long>(all[0]) >> 14)));
        Z = corrected(all[1], uint32_t(all[2]), e);
        if (static_cast<long long>(Z) > 0) break;
        if (!both && without < 0) break;    // (p has a sum near 2^60: not reached)
        // nothing is left of p: the two distributions are one.  Drawn from p.
        both = false;
        without = -1;
        e = 0;
        if (ctas > 1) cluster_sync_all(); else __syncthreads();
    }
    share = min(share_of(u_last >= 0.f ? fminf(u_last, 0.99999994f) : 0.f, Z), Z - 1);
    // the first CTA whose sums reach past the share
#pragma unroll 1
    for (holder = 0; holder < ctas - 1; ++holder) {
        const Sums next{before.d + cta_sums[holder][1],
                        before.p + uint32_t(cta_sums[holder][2])};
        if (static_cast<long long>(corrected(next.d, next.p, e)) > static_cast<long long>(share))
            break;
        before = next;
    }
    if (rank != holder) return;

    // the first block that does (a warp's lanes take 32 blocks at a time)
    if (warp == 0) {
        int block = k1 - 1;
#pragma unroll 1
        for (int k = k0; k < k1; k += 32) {
            const Sums s = k + lane < k1 ? block_sums[k - k0 + lane] : Sums{0, 0};
            const Sums to{before.d + warp_scan(s.d), before.p + uint32_t(warp_scan(s.p))};
            const bool past = k + lane < k1 && static_cast<long long>(corrected(to.d, to.p, e)) >
                                                   static_cast<long long>(share);
            const uint32_t who = __ballot_sync(~0u, past);
            if (who || k + 32 >= k1) {
                const int at = who ? __ffs(who) - 1 : min(31, k1 - 1 - k);
                block = k + at;
                before.d = __shfl_sync(~0u, to.d - s.d, at);
                before.p = __shfl_sync(~0u, to.p - s.p, at);
                break;
            }
            before.d = __shfl_sync(~0u, to.d, 31);
            before.p = __shfl_sync(~0u, to.p, 31);
        }
        if (lane == 0) {
            the_block = block;
            the_start = before;
        }
    }
    __syncthreads();
    // ... its entries' weights, 32 at a time
#pragma unroll 1
    for (int g = warp; g < kGroups; g += kWarps) {
        const int i = the_block * kBlock + g * 32 + lane;
        const float x = i < a.n && i != without ? load1<DT>(xr, i) : -INFINITY;
        const float y = both && i < a.n ? load1<DT>(yr, i) : -INFINITY;
        const unsigned long long p = fixed_exp(x, kp, power);
        long long w = static_cast<long long>(corrected(p, uint32_t(p >> 32), e));
        if (both) w = max(0ll, w - static_cast<long long>(fixed_exp(y, kq, power)));
        weights[g][lane] = static_cast<unsigned long long>(w);
        const unsigned long long s = warp_sum(static_cast<unsigned long long>(w));
        if (lane == 0) group_sums[g] = s;
    }
    __syncthreads();
    if (warp != 0) return;
    // ... and the first that reaches past the share (the last one with a weight, should the sums
    // of rounded corrections end below it).  (The sum in front may be below 0 by such roundings.)
    const long long over = static_cast<long long>(share) -
                           static_cast<long long>(corrected(the_start.d, the_start.p, e));
    const unsigned long long s = lane < kGroups ? group_sums[lane] : 0ull, to = warp_scan(s);
    uint32_t who = __ballot_sync(~0u, s > 0 && static_cast<long long>(to) > over);
    const uint32_t any = __ballot_sync(~0u, s > 0);
    if (!any) {  // (not reached: a block is chosen for its sum)
        if (lane == 0) emit(-1);
        return;
    }
    const int g = who ? __ffs(who) - 1 : 31 - __clz(any);
    const unsigned long long w = weights[g][lane];
    const long long reach = static_cast<long long>(__shfl_sync(~0u, to - s, g) + warp_scan(w));
    who = __ballot_sync(~0u, w > 0 && reach > over);
    const uint32_t some = __ballot_sync(~0u, w > 0);
    if (lane == 0)
        emit(the_block * kBlock + g * 32 + (who ? __ffs(who) - 1 : 31 - __clz(some)));
}

// ------------------------------------------------------------------------ host side

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

template <int DT>
cudaError_t launch(const DeviceInfo& dev, DraftArgs& a, bool rows_aligned, cudaStream_t stream) {
    a.nparts = (a.n + kPartLen<DT> - 1) / kPartLen<DT>;
    const int64_t items = (int64_t(a.total_q) + (a.y ? a.num_drafts : 0)) * a.nparts;
    if (items > kI32Max) return cudaErrorNotSupported;
    a.items = int(items);
    const int64_t wave = 9 * (kStats / 32) * int64_t(dev.num_sms);
    a.ahead = items <= 8 * wave ? int(wave) : 0;
    // CTAs of a sequence: one for every eight blocks (a block for each warp), while the
    // multiprocessors hold them all at once (three each).  The batch is spread over them: left to
    // itself the hardware puts the clusters of a small one on half of them.  Six where seven would
    // fit: clusters of seven do not all find room at once (64 sequences of 128,256 bf16 82.9 us with
    // seven, 72.4 with six).  Two where one each leaves three eighths of the room empty and rows
    // are long (230 sequences of 2 rows of 128,256 bf16 211 us with one, 175 with two, 256 of 50,257
    // 94.6 and 88.8; 300 of 2 fp32 rows 156 and 165, 300 of 32,000 63.9 and 65.6).
    const int blocks = (a.n + kBlock - 1) / kBlock;
    const int64_t sms = dev.num_sms, room = 3 * sms;
    int64_t fit = room / a.B;
    if (fit == 7) fit = 6;
    if (fit == 1 && 8 * int64_t(a.B) <= 5 * room && blocks >= 64) fit = 2;
    const int ctas = int(std::max<int64_t>(
        1, std::min<int64_t>({int64_t(kMaxCtas), (blocks + 7) / 8, fit})));
    const int64_t total = int64_t(a.B) * ctas;
    const size_t apart = total <= sms ? 120 * 1024 : total <= 2 * sms ? 48 * 1024 : 0;
    // statistics in the same launch where a warp gets no more than two parts of its sequence (7
    // sequences of 999 entries 12.4 us on the GPU, 22 to 25 with the host's time; 15.2 and 26 in two
    // launches; 4 rows of 128,256, eight parts for each warp, 29 and 25)
    const int64_t rows = a.y ? 2 * int64_t(a.max_q) - 1 : a.max_q;
    const bool own = total <= 2 * sms && rows * a.nparts <= 2 * ctas * (kThreads / 32);
    if (!own) {
        auto stats = rows_aligned ? draft_stats_kernel<DT, true> : draft_stats_kernel<DT, false>;
        const int64_t grid = (items + kStats / 32 - 1) / (kStats / 32);
        cudaError_t e = launch_pdl(stats, dim3(unsigned(grid)), dim3(kStats), 0, stream, a);
        if (e != cudaSuccess) return e;
    }
    auto draw = total > 2 * sms ? draft_draw_kernel<DT, 1, 0>
                : !own          ? draft_draw_kernel<DT, 4, 0>
                : rows_aligned  ? draft_draw_kernel<DT, 4, 1>
                                : draft_draw_kernel<DT, 4, 2>;
    static bool attr_done[64] = {};
    if (dev.device >= 0 && dev.device < 64 && !attr_done[dev.device]) {
        for (auto k : {draft_draw_kernel<DT, 4, 0>, draft_draw_kernel<DT, 4, 1>,
                       draft_draw_kernel<DT, 4, 2>}) {
            cudaError_t e =
                cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 120 * 1024);
            if (e != cudaSuccess) return e;
        }
        attr_done[dev.device] = true;
    }
    return launch_pdl_cluster(draw, dim3(unsigned(total)), dim3(kThreads), apart, stream,
                              unsigned(ctas), a, ctas);
}

}  // namespace
}  // namespace bi

using namespace bi;

BI_EXPORT size_t bi_verify_drafts_workspace_size(int64_t total_q, int64_t num_drafts, int64_t n) {
    if (total_q < 0 || num_drafts < 0 || total_q > kI32Max || num_drafts > kI32Max || n < 1 ||
        n > BI_DRAFTS_MAX_N)
        return 0;
    const size_t parts = size_t((n + kPartLen<BI_F32> - 1) / kPartLen<BI_F32>);
    return size_t(total_q + num_drafts) * parts * sizeof(PartStats);
}

BI_EXPORT bi_status bi_verify_drafts(const void* logits, int64_t ldl, const void* draft_logits,
                                     int64_t ldd, int dtype, const int32_t* draft_tokens,
                                     int64_t num_drafts, const float* uniforms,
                                     const float* temperatures, float temperature,
                                     const int32_t* cu_q, int64_t batch, int64_t total_q,
                                     int64_t max_q, int64_t n, int32_t* tokens, int32_t* accepted,
                                     float* logprobs, void* workspace, size_t workspace_bytes,
                                     bi_stream_t stream) {
    const char* fn = "bi_verify_drafts";
    if (dtype != BI_BF16 && dtype != BI_F16 && dtype != BI_F32)
        return fail(BI_ERR_INVALID_ARG, "%s: dtype must be BI_BF16, BI_F16 or BI_F32", fn);
    if (batch < 0 || total_q < 0 || num_drafts < 0 || max_q < 1 || n < 1)
        return fail(BI_ERR_INVALID_ARG,
                    "%s: need batch, total_q, num_drafts >= 0 and max_q, n >= 1", fn);
    if (n > BI_DRAFTS_MAX_N)
        return fail(BI_ERR_UNSUPPORTED, "%s: n must be at most %d", fn, BI_DRAFTS_MAX_N);
    if (total_q > kI32Max / 2 || num_drafts > kI32Max / 2 || max_q > kI32Max / 2 ||
        batch > kI32Max / kMaxCtas)
        return fail(BI_ERR_UNSUPPORTED, "%s: a size is too large", fn);
    if (ldl < n || (draft_logits && ldd < n))
        return fail(BI_ERR_INVALID_ARG, "%s: a row stride is below n", fn);
    if (batch == 0) return BI_OK;
    if (total_q < batch) return fail(BI_ERR_INVALID_ARG, "%s: total_q < batch", fn);
    if (!temperatures && !(temperature >= 0.f && std::isfinite(temperature)))
        return fail(BI_ERR_INVALID_ARG, "%s: temperature must be finite and >= 0", fn);
    if (!logits || !uniforms || !cu_q || !tokens || !accepted || !workspace ||
        (num_drafts > 0 && !draft_tokens))
        return fail(BI_ERR_INVALID_ARG, "%s: null pointer", fn);
    const size_t es = dtype == BI_F32 ? 4 : 2;
    if (!aligned(logits, es) || !aligned(draft_logits, es) || !aligned(draft_tokens, 4) ||
        !aligned(uniforms, 4) || !aligned(temperatures, 4) || !aligned(cu_q, 4) ||
        !aligned(tokens, 4) || !aligned(accepted, 4) || !aligned(logprobs, 4))
        return fail(BI_ERR_INVALID_ARG, "%s: pointers not element-aligned", fn);
    if (!aligned(workspace, 16))
        return fail(BI_ERR_UNSUPPORTED, "%s: workspace must be 16-byte aligned", fn);
    const size_t need = bi_verify_drafts_workspace_size(total_q, draft_logits ? num_drafts : 0, n);
    if (workspace_bytes < need)
        return fail(BI_ERR_INVALID_ARG, "%s: workspace too small (%zu < %zu bytes)", fn,
                    workspace_bytes, need);
    cudaError_t why = cudaSuccess;
    const DeviceInfo* dev = current_device_info(&why);
    if (!dev) return launched(why, fn);
    DraftArgs a{};
    a.x = logits;
    a.y = num_drafts > 0 ? draft_logits : nullptr;
    a.ldx = ldl;
    a.ldy = ldd;
    a.draft_tokens = draft_tokens;
    a.uniforms = uniforms;
    a.temperatures = temperatures;
    a.temperature = temperature;
    a.cu_q = cu_q;
    a.parts = static_cast<PartStats*>(workspace);
    a.tokens = tokens;
    a.accepted = accepted;
    a.logprobs = logprobs;
    a.err = dev->err_word;
    a.B = int(batch);
    a.total_q = int(total_q);
    a.num_drafts = int(num_drafts);
    a.max_q = int(max_q);
    a.n = int(n);
    const bool al = aligned(logits, 16) && ldl * int64_t(es) % 16 == 0 &&
                    (!a.y || (aligned(a.y, 16) && ldd * int64_t(es) % 16 == 0));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = dtype == BI_F32   ? launch<BI_F32>(*dev, a, al, st)
                    : dtype == BI_F16 ? launch<BI_F16>(*dev, a, al, st)
                                      : launch<BI_BF16>(*dev, a, al, st);
    if (e == cudaErrorNotSupported) return fail(BI_ERR_UNSUPPORTED, "%s: too many rows", fn);
    return launched(e, fn);
}
