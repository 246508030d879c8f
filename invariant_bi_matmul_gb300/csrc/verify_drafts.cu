// verify_drafts.cu -- verification of drafted tokens against the target's probabilities from
// given uniform numbers (include/bi_rowwise.h, bi_verify_drafts).
//
// With p = softmax(x / T) of a target row and q the draft's probabilities, draft j is kept while
// u q(token) < p(token); the block's last token is drawn by inverting the cumulative sums of
// D_i = max(p_i - q_i, 0) (behind a refused draft) or of p_i.  Two launches:
//
// Statistics.  A CTA takes one part of one row (kBatch vectors a thread, all requested before
// any is used) and leaves the part's maximum, sum of 2^((x - m) log2 e / T) in fp32 and, for a
// sequence at temperature 0, its largest entry.  Every target row and every draft row is read
// once, which is what the call cannot do without.
//
// Decision and draw.  A cluster of CTAs per sequence joins the parts (lanes over the parts, a
// butterfly), finds the first refused draft, and goes over that row, and the draft's, once more.
// A drawn token must not depend on how sums round, or it would depend on the order in which they
// are taken: near equal entries of 2^-17 of the mass, fp32 sums would choose a neighbour in one
// row of a few hundred.  So each weight is a whole number, 2^60 p_i, from a product x c in two
// floats and a table of 2^(j/512), off by at most 2^-30 of itself (fixed_exp), and sums of whole
// numbers are exact in any order: the token is the same whatever the split, in one row in 10^5 or
// so another than the definition's.  The fp32 statistics only scale the weights to a sum near
// 2^60; what the sums come to, sp and sq, corrects that: D_i is proportional to
// max(p_i sq/sp - q_i, 0), and with e = sq/sp - 1 (1e-6 at most) the sum of D over a block is
// sum max(p_i - q_i, 0) + e * sum of p_i where p_i > q_i, but for entries whose p and q agree to
// within e, which weigh e times as much.  One pass so gives the totals, the correction and the
// sums of each block of 512; the block that holds the drawn share is taken again, entry by entry.
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

constexpr int kThreads = 256;
constexpr int kBlock = 512;                             // entries of a block: 16 for each lane
constexpr int kMaxCtas = 8;                             // of a sequence's cluster
constexpr int kMaxBlocks = (BI_DRAFTS_MAX_N + kBlock - 1) / kBlock;
constexpr float kHot = 0x1p-64f;                        // temperatures below it are 0

template <int DT>
constexpr int kPartLen = kThreads * kBatch * (16 / kSize<DT>);  // entries of a part

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
    int B, total_q, num_drafts, max_q, n, nparts;
};

__device__ __forceinline__ float temperature_of(const DraftArgs& a, int b) {
    const float t = a.temperatures ? a.temperatures[b] : a.temperature;
    return t < kHot ? (t >= 0.f ? 0.f : kNaN) : t <= 3.4e38f ? t : kNaN;  // NaN: refused
}

// --------------------------------------------------------------------------- statistics

template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) draft_stats_kernel(const DraftArgs a) {
    constexpr int VE = 16 / kSize<DT>;
    __shared__ float sm[kThreads / 32], ss[kThreads / 32];
    __shared__ unsigned long long sk[kThreads / 32];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = int(blockIdx.x / unsigned(a.nparts));
    const int part = int(blockIdx.x - unsigned(row) * unsigned(a.nparts));
    const bool draft = row >= a.total_q;
    const int r = draft ? row - a.total_q : row;
    const char* xr = static_cast<const char*>(draft ? a.y : a.x) +
                     int64_t(r) * (draft ? a.ldy : a.ldx) * kSize<DT>;
    const uint32_t skew = ALIGNED ? 0u : uint32_t(reinterpret_cast<uintptr_t>(xr) & 15u);
    const int v0 = part * (kThreads * kBatch);
    uint4 v[kBatch];
    load_batch<DT, kThreads, ALIGNED>(v, xr, skew, v0,
                                      min((a.n + VE - 1) / VE, v0 + kThreads * kBatch), a.n);
    // the row's sequence, found while the loads are under way: target rows of b are
    // cu_q[b] .., draft rows cu_q[b] - b ..
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_q[mid] - (draft ? mid : 0) <= r) lo = mid; else hi = mid;
    }
    const int end = a.cu_q[lo + 1] - (draft ? lo + 1 : 0);
    if (r >= end) return;                   // a row of no sequence
    const float T = temperature_of(a, lo);
    const bool greedy = T == 0.f;
    if (isnan(T) || (greedy && draft)) return;
    const float c = kLog2e / (greedy ? 1.f : T);

    float m = vec_max<DT>(v[0]);
#pragma unroll
    for (int k = 1; k < kBatch; ++k) m = fmaxf(m, vec_max<DT>(v[k]));
    const float ref = ref_of(m);
    float s0 = 0.f, s1 = 0.f;               // (entries past the row are -inf: they add 0)
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        float e[VE];
        widen<DT>(v[k], e);
#pragma unroll
        for (int q = 0; q < VE; q += 2) {
            s0 += ex2((e[q] - ref) * c);
            s1 += ex2((e[q + 1] - ref) * c);
        }
    }
    float s = s0 + s1;
    unsigned long long best = 0;
    if (greedy) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            float e[VE];
            widen<DT>(v[k], e);
            const int64_t i0 = int64_t(v0 + k * kThreads + tid) * VE;
#pragma unroll
            for (int q = 0; q < VE; ++q) {
                if (i0 + q < a.n) {
                    const unsigned long long key = order_key(e[q], int(i0) + q);
                    best = key > best ? key : best;
                }
            }
        }
    }
    float M = m;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        M = fmaxf(M, __shfl_xor_sync(~0u, M, off));
        const unsigned long long o = __shfl_xor_sync(~0u, best, off);
        best = o > best ? o : best;
    }
    if (m != -INFINITY) s *= ex2((m - M) * c);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(~0u, s, off);
    if (lane == 0) {
        sm[warp] = M;
        ss[warp] = s;
        sk[warp] = best;
    }
    __syncthreads();
    if (tid == 0) {
        float top = sm[0];
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) top = fmaxf(top, sm[w]);
        PartStats p{top, 0.f, 0ull};
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            p.s += sm[w] == -INFINITY ? ss[w] : ss[w] * ex2((sm[w] - top) * c);
            p.best = sk[w] > p.best ? sk[w] : p.best;
        }
        a.parts[int64_t(row) * a.nparts + part] = p;
    }
}

// ---------------------------------------------------------------- weights in whole numbers

// Entry j stands for v = 2^62 * 2^(j/512): hi = v / 2^32, and adj = v - hi * 0x4b000000, so that
// hi * (0x4b000000 + G) + adj = v (1 + G / 2^32).
struct Power {
    uint32_t hi, pad;
    unsigned long long adj;
};
struct Powers {
    Power at[512];
};
constexpr unsigned long long mul62(unsigned long long x, unsigned long long y) {
    const unsigned long long xh = x >> 32, xl = x & 0xffffffffull, yh = y >> 32,
                             yl = y & 0xffffffffull;
    const unsigned long long mid = xh * yl + ((xl * yl) >> 32), mid2 = xl * yh + (mid & 0xffffffffull);
    const unsigned long long h = xh * yh + (mid >> 32) + (mid2 >> 32), l = mid2 & 0xffffffffull;
    return (h << 2) | (l >> 30);
}
constexpr Powers powers() {
    // 2^62 * 2^(1/2), 2^(1/4), ..., 2^(1/512)
    const unsigned long long root[9] = {
        0x5a827999fcef3242ull, 0x4c1bf828c6dc54b8ull, 0x45cae0f1f545eb73ull,
        0x42d561b3e6243d8aull, 0x4166c34c5615d0ecull, 0x40b268f9de0183baull,
        0x4058f6a7ecccd5b6ull, 0x402c6be96af2fb58ull, 0x4016321b687027a8ull};
    Powers p{};
    for (int j = 0; j < 512; ++j) {
        unsigned long long v = 1ull << 62;
        for (int k = 0; k < 9; ++k)
            if ((j >> (8 - k)) & 1) v = mul62(v, root[k]);
        p.at[j].hi = uint32_t(v >> 32);
        p.at[j].adj = v - (v >> 32) * 0x4b000000ull;
    }
    return p;
}
__device__ const Powers kPowers = powers();

// How a row's entries become weights 2^60 * 2^((x - m) c - L): c in two floats, L = i + f / 2^30.
struct RowScale {
    float m, ch, cl;
    int i, f;
};

__device__ __forceinline__ unsigned long long fixed_exp(float x, const RowScale& r,
                                                        const Power* table) {
    constexpr float kMagic = 12582912.f;    // 1.5 * 2^23: adding it rounds to a whole number
    constexpr int kMagicBits = 0x4b400000;
    constexpr float kZ = 0.6931471805599453f / 512.f;
    // d + dl = x - m exactly; t + tl = (x - m) c to 2^-46 of itself
    const float d = x - r.m;
    const float xs = d + r.m;
    const float dl = (x - xs) + ((xs - d) - r.m);
    const float t = d * r.ch;
    const float tl = fmaf(dl, r.ch, fmaf(d, r.cl, fmaf(d, r.ch, -t)));
    // whole part and fraction, in 2^-30: each of three terms is rounded to that
    const float whole = t + kMagic;
    const int s = __float2int_rn((t - (whole - kMagic)) * 0x1p30f) +
                  (__float_as_int(fmaf(tl, 0x1p30f, kMagic)) - kMagicBits) - r.f;
    const int N = (__float_as_int(whole) - kMagicBits) - r.i + (s >> 30);
    // 2^(fraction): the table at its first nine bits, a cubic of the other 21 (off by 2^-43), in
    // units of 2^-32 as the low bits of 2^23 + ...
    const float z = __uint_as_float((uint32_t(s) << 2 & 0x7fffffu) | 0x3f800000u) - 1.f;
    constexpr float a1 = 0x1p32f * kZ, a2 = 0x1p32f * kZ * kZ / 2.f,
                    a3 = 0x1p32f * kZ * kZ * kZ / 6.f;
    const float g = fmaf(z, fmaf(z, fmaf(z, a3, a2), a1), 8388608.f);
    const uint4 e = *reinterpret_cast<const uint4*>(&table[(s >> 21) & 511]);
    const unsigned long long v =
        static_cast<unsigned long long>(e.x) * __float_as_uint(g) +
        ((static_cast<unsigned long long>(e.w) << 32) | e.z);
    // (t is -inf or NaN where an entry is -inf, or far below the maximum: no weight)
    return t > -64.f ? v >> min(max(2 - N, 0), 63) : 0ull;
}

// 2^60 p_i (1 + e): what a weight is after the correction, e in 2^-46.
__device__ __forceinline__ unsigned long long corrected(unsigned long long d, unsigned long long p,
                                                        long long e) {
    return d + static_cast<unsigned long long>((static_cast<long long>(p >> 28) * e) >> 18);
}

// ------------------------------------------------------------------------ decision and draw

struct RowStats {
    float m, s;
    unsigned long long best;
};

// The parts of a row together, the same in every lane of a warp.
__device__ __forceinline__ RowStats join_parts(const PartStats* p, int nparts, float c) {
    const int lane = threadIdx.x & 31;
    RowStats r{-INFINITY, 0.f, 0ull};
    for (int i = lane; i < nparts; i += 32) r.m = fmaxf(r.m, p[i].m);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) r.m = fmaxf(r.m, __shfl_xor_sync(~0u, r.m, off));
    for (int i = lane; i < nparts; i += 32) {
        r.s += p[i].m == -INFINITY ? p[i].s : p[i].s * ex2((p[i].m - r.m) * c);
        r.best = p[i].best > r.best ? p[i].best : r.best;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        r.s += __shfl_xor_sync(~0u, r.s, off);
        const unsigned long long o = __shfl_xor_sync(~0u, r.best, off);
        r.best = o > r.best ? o : r.best;
    }
    return r;
}

__device__ __forceinline__ bool has_distribution(const RowStats& r) {
    return isfinite(r.m) && isfinite(r.s);  // (a NaN or +inf in the row makes s NaN)
}

__device__ __forceinline__ RowScale scale_of(const RowStats& r, double c) {
    RowScale k;
    k.m = r.m;
    k.ch = float(c);
    k.cl = float(c - double(k.ch));
    const float L = log2f(r.s), i = rintf(L);
    k.i = int(i);
    k.f = __float2int_rn((L - i) * 0x1p30f);
    return k;
}

// log p of an entry: (x - m) c is formed in fp64, once per emitted token.
__device__ __forceinline__ float logp_of(float x, const RowStats& r, double c) {
    return float((double(x) - double(r.m)) * c * 0.6931471805599453 - double(logf(r.s)));
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
    unsigned long long d, p;  // of max(p - q, 0), and of p where p > q
};

template <int DT>
__global__ void __launch_bounds__(kThreads)
draft_draw_kernel(const DraftArgs a, int ctas) {
    constexpr int kWarps = kThreads / 32;
    __shared__ __align__(16) Power table[512];
    __shared__ Sums block_sums[kMaxBlocks / kMaxCtas];
    __shared__ unsigned long long warp_sums[kWarps][4];
    __shared__ unsigned long long cta_sums[kMaxCtas][4];  // every CTA's: p, q, d, p where p > q
    __shared__ int first_refused;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = int(blockIdx.x / unsigned(ctas)), rank = int(blockIdx.x - unsigned(b) * ctas);
    for (int i = tid; i < 512; i += kThreads)
        *reinterpret_cast<uint4*>(&table[i]) = *reinterpret_cast<const uint4*>(&kPowers.at[i]);
    if (tid == 0) first_refused = 0x7fffffff;
    pdl_wait();
    pdl_trigger();
    // the offsets of the whole batch: a call with malformed ones decides nothing
    bool bad = tid == 0 && (a.cu_q[0] != 0 || a.cu_q[a.B] > a.total_q ||
                            a.cu_q[a.B] - a.B > a.num_drafts);
    for (int i = tid; i < a.B; i += kThreads) {
        const int w = int(uint32_t(a.cu_q[i + 1]) - uint32_t(a.cu_q[i]));
        bad |= w < 1 || w > a.max_q || a.cu_q[i] < 0;
    }
    bad = __syncthreads_or(bad) != 0;
    const float T = bad ? kNaN : temperature_of(a, b);
    int32_t* out = a.tokens + int64_t(b) * a.max_q;
    float* out_logp = a.logprobs ? a.logprobs + int64_t(b) * a.max_q : nullptr;
    if (isnan(T)) {
        if (rank == 0) {
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
    const double c = greedy ? 1.4426950408889634 : 1.4426950408889634 / double(T);
    const int t0 = a.cu_q[b], drafts = a.cu_q[b + 1] - t0 - 1;
    const int d0 = t0 - b;                  // the sequence's first draft
    auto target = [&](int j) {
        return join_parts(a.parts + int64_t(t0 + j) * a.nparts, a.nparts, float(c));
    };
    auto drafted = [&](int j) {
        return join_parts(a.parts + (int64_t(a.total_q) + d0 + j) * a.nparts, a.nparts, float(c));
    };
    const int64_t xs = kSize<DT>;
    auto target_row = [&](int j) {
        return static_cast<const char*>(a.x) + int64_t(t0 + j) * a.ldx * xs;
    };
    auto draft_row = [&](int j) {
        return static_cast<const char*>(a.y) + int64_t(d0 + j) * a.ldy * xs;
    };

    // a warp per draft; the row of a warp's lanes is the same
    for (int j = warp; j < drafts; j += kWarps) {
        const RowStats p = target(j);
        const int token = a.draft_tokens[d0 + j];
        bool take = false;
        float x = 0.f;
        if (token >= 0 && token < a.n) {
            x = load1<DT>(target_row(j), token);
            if (greedy) {
                take = p.best != 0ull && 0x7fffffff - int(uint32_t(p.best)) == token;
            } else if (has_distribution(p) && x != -INFINITY) {
                // u 2^tq / sq < 2^tp / sp
                double t = -(double(x) - double(p.m)) * c;
                float sq = 1.f;
                bool fine = true;
                if (a.y) {
                    const RowStats q = drafted(j);
                    fine = has_distribution(q);
                    sq = q.s;
                    t += (double(load1<DT>(draft_row(j), token)) - double(q.m)) * c;
                }
                const float th = float(t);
                const float e =
                    isfinite(th) ? exp2f(th) * fmaf(float(t - double(th)), kLn2, 1.f) : exp2f(th);
                const float u = a.uniforms[t0 + j];
                take = fine && (u == 0.f || double(u) * double(e) * double(p.s) < double(sq));
            }
        } else if (token != -1 && lane == 0 && rank == 0) {
            latch_error(a.err, kErrDeviceArg);
        }
        if (lane == 0) {
            if (!take) atomicMin(&first_refused, j);
            if (rank == 0 && take) {
                out[j] = token;
                if (out_logp) out_logp[j] = logp_of(x, p, c);
            }
        }
    }
    __syncthreads();
    const int kept = min(drafts, first_refused);
    const int refused = kept < drafts ? a.draft_tokens[d0 + kept] : -1;  // -1: drawn from p
    const bool behind = refused >= 0 && refused < a.n;
    if (rank == 0) {
        for (int j = kept + 1 + tid; j < a.max_q; j += kThreads) {
            out[j] = -1;
            if (out_logp) out_logp[j] = 0.f;
        }
        if (tid == 0) a.accepted[b] = kept;
    }
    const RowStats P = target(kept);
    const char* xr = target_row(kept);
    auto emit = [&](int token) {
        out[kept] = token;
        if (out_logp) out_logp[kept] = token < 0 ? kNaN : logp_of(load1<DT>(xr, token), P, c);
    };
    if (greedy) {
        if (rank == 0 && tid == 0) emit(0x7fffffff - int(uint32_t(P.best)));
        return;
    }
    bool both = behind && a.y;              // subtract the draft's probabilities
    RowStats Q{0.f, 1.f, 0ull};
    if (both) Q = drafted(kept);
    if (!has_distribution(P) || (both && !has_distribution(Q))) {
        if (rank == 0 && tid == 0) emit(-1);
        return;
    }
    int without = behind && !a.y ? refused : -1;  // q = 1 there: that entry has no weight
    const char* yr = both ? draft_row(kept) : nullptr;
    const RowScale kp = scale_of(P, c), kq = both ? scale_of(Q, c) : kp;
    const int blocks = (a.n + kBlock - 1) / kBlock;
    const int k0 = int(int64_t(rank) * blocks / ctas), k1 = int(int64_t(rank + 1) * blocks / ctas);

    if (ctas > 1) cluster_sync_all();       // (the others have started)
    unsigned long long Z = 0;
    long long e = 0;
    Sums before{0, 0};                      // of the CTAs in front of the one that holds the share
    int holder = 0;
    unsigned long long share = 0;
    for (;;) {
        unsigned long long sp = 0, sq = 0, sd = 0, sdp = 0;
        auto pass = [&](auto subtracts) {
            constexpr bool BOTH = decltype(subtracts)::value;
            for (int k = k0 + warp; k < k1; k += kWarps) {
                Sums s{0, 0};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x[8], y[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const int i = k * kBlock + (8 * h + q) * 32 + lane;
                        x[q] = i < a.n && i != without ? load1<DT>(xr, i) : -INFINITY;
                        if (BOTH) y[q] = i < a.n ? load1<DT>(yr, i) : -INFINITY;
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const unsigned long long p = fixed_exp(x[q], kp, table);
                        if (BOTH) {
                            const unsigned long long w = fixed_exp(y[q], kq, table);
                            sp += p;
                            sq += w;
                            if (p > w) {
                                s.d += p - w;
                                s.p += p;
                            }
                        } else {
                            s.d += p;
                        }
                    }
                }
                s.d = warp_sum(s.d);
                if (BOTH) s.p = warp_sum(s.p);
                if (lane == 0) block_sums[k - k0] = s;
                sd += s.d;
                sdp += s.p;
            }
            if (BOTH) {
                sp = warp_sum(sp);
                sq = warp_sum(sq);
            }
        };
        if (both) pass(std::true_type()); else pass(std::false_type());
        if (lane == 0) {
            warp_sums[warp][0] = sp;
            warp_sums[warp][1] = sq;
            warp_sums[warp][2] = sd;
            warp_sums[warp][3] = sdp;
        }
        __syncthreads();
        if (tid < 4) {
            unsigned long long v = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += warp_sums[w][tid];
            cta_sums[rank][tid] = v;
            for (int r = 0; r < ctas; ++r)
                if (r != rank) st_cluster_b64(cluster_map(smem_addr(&cta_sums[rank][tid]), r), v);
        }
        if (ctas > 1) cluster_sync_all(); else __syncthreads();
        // every thread of the cluster comes to the same numbers
        unsigned long long all[4] = {0, 0, 0, 0};
        for (int r = 0; r < ctas; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) all[i] += cta_sums[r][i];
        e = both ? __double2ll_rn((double(all[1]) / double(all[0]) - 1.0) * 0x1p46) : 0;
        e = max(-(1ll << 30), min(1ll << 30, e));
        Z = corrected(all[2], all[3], e);
        if (static_cast<long long>(Z) <= 0) {
            if (!both && without < 0) break;  // (p has a sum near 2^60: not reached)
            // nothing is left of p: the two distributions are one.  Drawn from p.
            both = false;
            without = -1;
            if (ctas > 1) cluster_sync_all(); else __syncthreads();
            continue;
        }
        const float u = a.uniforms[t0 + drafts];
        const double part = double(u >= 0.f ? fminf(u, 0.99999994f) : 0.f) * double(Z);
        share = min(static_cast<unsigned long long>(part), Z - 1);
        // the first CTA whose sums reach past the share
        for (holder = 0; holder < ctas - 1; ++holder) {
            const Sums next{before.d + cta_sums[holder][2], before.p + cta_sums[holder][3]};
            const unsigned long long F = corrected(next.d, next.p, e);
            if (static_cast<long long>(F) > static_cast<long long>(share)) break;
            before = next;
        }
        break;
    }
    if (rank != holder || warp != 0) return;

    // the first block that does (a warp's lanes take 32 blocks at a time)
    int block = k1 - 1;
    for (int k = k0; k < k1; k += 32) {
        const Sums s = k + lane < k1 ? block_sums[k - k0 + lane] : Sums{0, 0};
        const Sums to{before.d + warp_scan(s.d), before.p + warp_scan(s.p)};
        const bool past = k + lane < k1 && static_cast<long long>(corrected(to.d, to.p, e)) >
                                               static_cast<long long>(share);
        const uint32_t who = __ballot_sync(~0u, past);
        const int at = who ? __ffs(who) - 1 : 31;
        if (who || k + 32 >= k1) {
            const int last = who ? at : min(31, k1 - 1 - k);
            block = k + last;
            before.d = __shfl_sync(~0u, to.d - s.d, last);
            before.p = __shfl_sync(~0u, to.p - s.p, last);
            break;
        }
        before.d = __shfl_sync(~0u, to.d, 31);
        before.p = __shfl_sync(~0u, to.p, 31);
    }
    // ... and its first entry (the last one with a weight, should the sums of rounded
    // corrections end below the share)
    long long sum = static_cast<long long>(corrected(before.d, before.p, e));
    int token = -1;
    for (int q = 0; q < kBlock / 32; ++q) {
        const int i = block * kBlock + q * 32 + lane;
        long long w = 0;
        if (i < a.n && i != without) {
            const unsigned long long p = fixed_exp(load1<DT>(xr, i), kp, table);
            w = static_cast<long long>(corrected(p, p, e));
            if (both) w -= static_cast<long long>(fixed_exp(load1<DT>(yr, i), kq, table));
            w = max(w, 0ll);
        }
        const long long to =
            sum + static_cast<long long>(warp_scan(static_cast<unsigned long long>(w)));
        const uint32_t some = __ballot_sync(~0u, w > 0);
        const uint32_t past = __ballot_sync(~0u, w > 0 && to > static_cast<long long>(share));
        if (some) token = block * kBlock + q * 32 + (past ? __ffs(past) - 1 : 31 - __clz(some));
        if (past) break;
        sum = __shfl_sync(~0u, to, 31);
    }
    if (lane == 0) emit(token);
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
cudaError_t launch(DraftArgs& a, bool rows_aligned, cudaStream_t stream) {
    a.nparts = (a.n + kPartLen<DT> - 1) / kPartLen<DT>;
    const int64_t rows = int64_t(a.total_q) + (a.y ? a.num_drafts : 0);
    if (rows * a.nparts > kI32Max) return cudaErrorNotSupported;
    auto stats = rows_aligned ? draft_stats_kernel<DT, true> : draft_stats_kernel<DT, false>;
    cudaError_t e = launch_pdl(stats, dim3(unsigned(rows * a.nparts)), dim3(kThreads), 0, stream, a);
    if (e != cudaSuccess) return e;
    // eight blocks (one for each warp) are worth a CTA
    const int blocks = (a.n + kBlock - 1) / kBlock;
    int ctas = 1;
    while (ctas < kMaxCtas && blocks > ctas * 8) ctas *= 2;
    return launch_pdl_cluster(draft_draw_kernel<DT>, dim3(unsigned(a.B) * unsigned(ctas)),
                              dim3(kThreads), 0, stream, unsigned(ctas), a, ctas);
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
    if (total_q > kI32Max / 2 || num_drafts > kI32Max / 2 || max_q > kI32Max ||
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
    cudaError_t e = dtype == BI_F32   ? launch<BI_F32>(a, al, st)
                    : dtype == BI_F16 ? launch<BI_F16>(a, al, st)
                                      : launch<BI_BF16>(a, al, st);
    if (e == cudaErrorNotSupported) return fail(BI_ERR_UNSUPPORTED, "%s: too many rows", fn);
    return launched(e, fn);
}
