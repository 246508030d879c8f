// rope_append.cu -- rotary embedding of a block's queries and keys together with the append of
// its keys and values to a bf16 or 8-bit paged cache (include/bi.h, bi_rope_kv_append*): one
// launch in place of bi_rope twice and an append.
//
// Pair i (i < R/2, R the rotary dimension) joins elements i and i + R/2 of a head and turns by
// a = pos * w_i:  y_i = x_i cos a - x_{i+R/2} sin a,  y_{i+R/2} = x_{i+R/2} cos a + x_i sin a.
// pos is the token's place in its sequence or, with several axes, the position on the axis whose
// section holds pair i.
//
// Angles.  The host turns each w_i into f_i = w_i / 2 pi mod 1 as a 64-bit fixed-point fraction
// of a turn; pos * f_i in wrapping 64-bit arithmetic is then the angle modulo a turn, off by at
// most |pos| * 2^-65 turns besides the double's own 2^-53 of pos * w_i.  (A float product
// pos * w_i is off by 2^-24 of itself: 0.004 rad at position 65,536, half a bf16 step.)  The
// signed fraction is rounded once to fp32, relative to itself, and sincospif takes it: full
// accuracy at any position, without its argument reduction or fp64 instructions.
//
// One thread per two 16-byte pieces of a head: pieces g and R/16 + g, the halves of eight pairs
// (behind R: two neighbouring pieces, copied).  The D/16 threads of a head are neighbours in a
// warp; each keeps its eight sines and cosines for the HPT heads that it takes of its token.
// The 8-bit cache's row maxima go by shuffles among them.  Bound by memory: every q row is read
// and written, every k and v row read and written (2 bytes an element, or 1 + 1/D).  8,192 tokens
// of 32 + 8 heads of 128 take 31.9 us into an 8-bit cache (5.8 TB/s) and 33.5 into a bf16 one (6.0),
// 32 tokens 3.4 us.  CTAs of 64 threads, so that the last ones of a call do not wait for large
// ones: 512 tokens 4.6 us, 6.9 with 256 threads.  Two heads a thread were slower on long blocks
// (40.7 us), eight too (37.0); streaming loads changed nothing.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "attn_common.cuh"
#include "kv_q8.cuh"

#define BI_EXPORT extern "C" __attribute__((visibility("default")))

namespace bi {

void set_last_error_message(const char* msg);

namespace {

constexpr int kThreads = 64;
constexpr int kMaxPairs = 64;  // head_dim 128

// What the rotation of a call needs beside the tensors.
struct Rotary {
    unsigned long long turn[kMaxPairs];  // 2^64 * (w_i / 2 pi mod 1)
    uint8_t axis[kMaxPairs];
    int pieces;                          // R / 16: threads of a head that turn pairs
    int axes;                            // 0: positions follow the cache
};

struct AppendArgs {
    const uint4* q;
    const uint4* k;
    const uint4* v;
    uint4* out;
    int64_t ldq, ldk, ldv, ldo;          // row strides in 16-byte pieces
    const int32_t* positions;
    int64_t ldp;
    void* k_cache;
    void* v_cache;
    uint8_t* k_scale;
    uint8_t* v_scale;
    const int32_t* block_table;
    const int32_t* seq_lens;
    const int32_t* cu_q;
    unsigned int* err;
    int num_pages, max_pages, B, total_q, hq, hkv;
};

__device__ __forceinline__ void unpack8(const uint4& raw, float (&v)[8]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}

template <int D, bool Q8, int HPT>
__global__ void __launch_bounds__(kThreads)
rope_kv_append_kernel(const AppendArgs a, const __grid_constant__ Rotary rot) {
    constexpr int LPH = D / 16;             // threads of a head
    constexpr int TPC = kThreads / LPH;     // tokens of a CTA
    pdl_wait();
    pdl_trigger();
    const int heads = a.hq + 2 * a.hkv;     // q heads, then k heads, then v heads
    const int groups = (heads + HPT - 1) / HPT;
    const int tile = int(blockIdx.x / unsigned(groups));
    const int h0 = int(blockIdx.x - unsigned(tile) * unsigned(groups)) * HPT;
    const int t = tile * TPC + int(threadIdx.x) / LPH;
    const int g = int(threadIdx.x) & (LPH - 1);
    const bool live = t < a.total_q;        // (the others take part in the shuffles)
    const bool turns = g < rot.pieces;
    const int p0 = turns ? g : 2 * g;
    const int p1 = turns ? rot.pieces + g : p0 + 1;

    uint4 x[HPT][2];
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
        const int h = h0 + i;
        x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
        if (live && h < heads) {
            const uint4* row = h < a.hq ? a.q + t * a.ldq + int64_t(h) * (D / 8)
                               : h < a.hq + a.hkv
                                   ? a.k + t * a.ldk + int64_t(h - a.hq) * (D / 8)
                                   : a.v + t * a.ldv + int64_t(h - a.hq - a.hkv) * (D / 8);
            x[i][0] = row[p0];
            x[i][1] = row[p1];
        }
    }

    // the token's place, found while the loads are under way
    bool in = false;
    int pos = 0;
    int64_t slot = -1;                      // (page * hkv) * PAGE + place in the page; -1: nowhere
    if (live) {
        int lo = 0, hi = a.B;               // sequence of token t: largest b with cu_q[b] <= t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu_q[mid] <= t) lo = mid; else hi = mid;
        }
        const int L = a.seq_lens[lo], t0 = a.cu_q[lo], t1 = a.cu_q[lo + 1];
        if (t >= t0 && t < t1) {            // (else a token of no sequence: left alone)
            // (t0 <= t < t1: their difference passes 2^31 where t0 is negative only)
            const int qb = int(uint32_t(t1) - uint32_t(t0));
            if (t0 < 0 || qb > L || int64_t(L) > int64_t(a.max_pages) * PAGE || t1 > a.total_q) {
                latch_error(a.err, kErrDeviceArg);
            } else {
                in = true;
                pos = L - qb + (t - t0);
                const int phys = a.block_table[int64_t(lo) * a.max_pages + pos / PAGE];
                if (phys >= 0 && phys < a.num_pages)
                    slot = int64_t(phys) * a.hkv * PAGE + pos % PAGE;
                else
                    latch_error(a.err, kErrDeviceArg);
            }
        }
    }

    float c[8], s[8];
    if (in && turns && h0 < a.hq + a.hkv) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = 8 * g + e;
            const long long at =
                rot.axes ? a.positions[rot.axis[i] * a.ldp + t] : pos;
            // the angle modulo a turn, in [-1/2, 1/2) turns * 2^64
            const long long f =
                static_cast<long long>(static_cast<unsigned long long>(at) * rot.turn[i]);
            sincospif(__ll2float_rn(f) * 0x1p-63f, &s[e], &c[e]);
        }
    }

#pragma unroll
    for (int i = 0; i < HPT; ++i) {
        const int h = h0 + i;
        if (h >= heads) break;              // (the whole CTA)
        if (in && turns && h < a.hq + a.hkv) {
            float u[8], w[8], yu[8], yw[8];
            unpack8(x[i][0], u);
            unpack8(x[i][1], w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                yu[e] = u[e] * c[e] - w[e] * s[e];
                yw[e] = w[e] * c[e] + u[e] * s[e];
            }
            x[i][0] = pack8(yu);
            x[i][1] = pack8(yw);
        }
        if (h < a.hq) {
            if (in) {
                uint4* row = a.out + t * a.ldo + int64_t(h) * (D / 8);
                row[p0] = x[i][0];
                row[p1] = x[i][1];
            }
            continue;
        }
        const bool key = h < a.hq + a.hkv;
        const int64_t row = slot + int64_t(key ? h - a.hq : h - a.hq - a.hkv) * PAGE;
        void* cache = key ? a.k_cache : a.v_cache;
        if (!Q8) {
            if (slot >= 0) {
                uint4* dst = static_cast<uint4*>(cache) + row * (D / 8);
                dst[p0] = x[i][0];
                dst[p1] = x[i][1];
            }
            continue;
        }
        uint32_t m = max(amax_bits(x[i][0]), amax_bits(x[i][1]));
#pragma unroll
        for (int off = LPH / 2; off > 0; off >>= 1)
            m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (slot >= 0) {
            const bool bad = m >= 0x7f80u;
            const int e = scale_exp(bad ? 0u : m);
            const float inv = __uint_as_float(uint32_t(127 - e) << 23);
            uint2* dst = static_cast<uint2*>(cache) + row * (D / 8);
            dst[p0] = bad ? make_uint2(0, 0) : codes8(x[i][0], inv);
            dst[p1] = bad ? make_uint2(0, 0) : codes8(x[i][1], inv);
            if (g == 0) (key ? a.k_scale : a.v_scale)[row] = bad ? 255 : uint8_t(e + 127);
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

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

constexpr int64_t kI32Max = 0x7fffffffLL;

// 2^64 * (w / 2 pi mod 1), rounded to nearest.  (A negative one from its magnitude: 1 - |w| / 2 pi
// has no bits of a small |w| left, an angle of 1e-14 a token was 2% off.)
unsigned long long turn_of(double w) {
    if (w < 0) return 0ull - turn_of(-w);
    const double f = std::fmod(w * 0.15915494309189533577, 1.0);
    const double hi = std::floor(std::ldexp(f, 32));       // (exact: f has 53 bits)
    const double lo = std::ldexp(f, 64) - std::ldexp(hi, 32);
    return (static_cast<unsigned long long>(hi) << 32) + static_cast<unsigned long long>(lo + 0.5);
}

// The frequencies theta^(-2i/R) as turns; the last ones of this thread are kept, since 64 powers
// take longer on the host than a launch.
void turns_of(Rotary& rot, double theta, int rotary_dim) {
    thread_local double last_theta = 0.0;
    thread_local int last_dim = 0;
    thread_local unsigned long long last[kMaxPairs];
    if (theta != last_theta || rotary_dim != last_dim) {
        for (int i = 0; i < rotary_dim / 2; ++i)
            last[i] = turn_of(std::pow(theta, -2.0 * i / rotary_dim));
        last_theta = theta;
        last_dim = rotary_dim;
    }
    std::copy(last, last + rotary_dim / 2, rot.turn);
}

template <bool Q8>
bi_status run(const char* fn, const void* q, int64_t ldq, const void* k_new, int64_t ldk,
              const void* v_new, int64_t ldv, void* q_out, int64_t ldo, void* k_cache,
              void* v_cache, void* k_scale, void* v_scale, int64_t num_pages,
              const int32_t* block_table, int64_t max_pages, const int32_t* seq_lens,
              const int32_t* cu_q, int64_t batch, int64_t total_q, int64_t hq, int64_t hkv,
              int64_t head_dim, int64_t page_size, double theta, const double* inv_freq,
              int64_t rotary_dim, const int32_t* positions, int64_t ldp, int64_t num_axes,
              const int64_t* sections, bi_stream_t stream) {
    if (batch < 0 || total_q < 0)
        return fail(BI_ERR_INVALID_ARG, "%s: negative batch or total_q", fn);
    if (head_dim != 64 && head_dim != 128)
        return fail(BI_ERR_UNSUPPORTED, "%s: head_dim must be 64 or 128", fn);
    if (page_size != BI_PAGE_SIZE)
        return fail(BI_ERR_UNSUPPORTED, "%s: page_size must be %d", fn, BI_PAGE_SIZE);
    if (hq < 1 || hkv < 1 || num_pages < 1 || max_pages < 1)
        return fail(BI_ERR_INVALID_ARG,
                    "%s: num_q_heads, num_kv_heads, num_pages, max_pages >= 1", fn);
    if (rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16 != 0)
        return fail(BI_ERR_UNSUPPORTED, "%s: rotary_dim must be a multiple of 16 in [16, head_dim]",
                    fn);
    // (the powers of a subnormal one may be infinite)
    if (!inv_freq && (!(theta > 0.0) || !std::isnormal(theta)))
        return fail(BI_ERR_INVALID_ARG, "%s: theta must be finite, > 0 and no subnormal", fn);
    if (num_axes < 0 || num_axes > rotary_dim / 2 || (num_axes > 0 && !sections))
        return fail(BI_ERR_INVALID_ARG, "%s: need 0 <= num_axes <= rotary_dim / 2, and sections",
                    fn);
    Rotary rot;
    rot.pieces = int(rotary_dim / 16);
    rot.axes = int(num_axes);
    int64_t pairs = 0;
    for (int64_t i = 0; i < num_axes; ++i) {
        if (sections[i] < 0 || sections[i] > rotary_dim / 2 - pairs)
            return fail(BI_ERR_INVALID_ARG, "%s: sections must be >= 0 and sum to rotary_dim / 2",
                        fn);
        for (int64_t n = 0; n < sections[i]; ++n) rot.axis[pairs++] = uint8_t(i);
    }
    if (num_axes > 0 && pairs != rotary_dim / 2)
        return fail(BI_ERR_INVALID_ARG, "%s: sections must be >= 0 and sum to rotary_dim / 2", fn);
    if (inv_freq) {
        for (int64_t i = 0; i < rotary_dim / 2; ++i) {
            if (!std::isfinite(inv_freq[i]))
                return fail(BI_ERR_INVALID_ARG, "%s: inv_freq must be finite", fn);
            rot.turn[i] = turn_of(inv_freq[i]);
        }
    } else {
        turns_of(rot, theta, int(rotary_dim));
    }
    if (ldq < hq * head_dim || ldo < hq * head_dim || ldk < hkv * head_dim || ldv < hkv * head_dim)
        return fail(BI_ERR_INVALID_ARG, "%s: a row stride is too small", fn);
    if (ldq % 8 || ldk % 8 || ldv % 8 || ldo % 8)
        return fail(BI_ERR_UNSUPPORTED, "%s: row strides must be multiples of 8", fn);
    if (num_axes > 0 && ldp < total_q)
        return fail(BI_ERR_INVALID_ARG, "%s: ldp < total_q", fn);
    if (num_pages > kI32Max || max_pages > kI32Max || batch > kI32Max || hq > kI32Max / 4 ||
        hkv > kI32Max / 4)
        return fail(BI_ERR_UNSUPPORTED, "%s: a size is 2^31 or more", fn);
    const int64_t heads = hq + 2 * hkv, per_cta = kThreads / (head_dim / 16);
    const int64_t tiles = (total_q + per_cta - 1) / per_cta;
    if (total_q > kI32Max || tiles > kI32Max / heads)
        return fail(BI_ERR_UNSUPPORTED, "%s: block too large", fn);
    if (batch == 0 || total_q == 0) return BI_OK;
    if (!q || !k_new || !v_new || !q_out || !k_cache || !v_cache || !block_table || !seq_lens ||
        !cu_q || (Q8 && (!k_scale || !v_scale)) || (num_axes > 0 && !positions))
        return fail(BI_ERR_INVALID_ARG, "%s: null pointer", fn);
    for (const void* p : {q, k_new, v_new, static_cast<const void*>(q_out),
                          static_cast<const void*>(k_cache), static_cast<const void*>(v_cache)})
        if (!aligned(p, 16))
            return fail(BI_ERR_UNSUPPORTED, "%s: tensors must be 16-byte aligned", fn);
    if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_q, 4) ||
        !aligned(positions, 4))
        return fail(BI_ERR_UNSUPPORTED, "%s: index tensors not element-aligned", fn);
    if (q_out == q && ldo != ldq)
        return fail(BI_ERR_INVALID_ARG, "%s: in place, ldo must be ldq", fn);
    cudaError_t why = cudaSuccess;
    const DeviceInfo* dev = current_device_info(&why);
    if (!dev) return launched(why, fn);

    // four heads a thread once that leaves every multiprocessor a CTA (300 tokens of 32 + 8 heads
    // 3.5 us, 6.1 with one head; 8 tokens 4.0 and 3.3)
    const bool wide = tiles * ((heads + 3) / 4) >= int64_t(dev->num_sms);
    const int64_t groups = wide ? (heads + 3) / 4 : heads;
    const AppendArgs a{static_cast<const uint4*>(q), static_cast<const uint4*>(k_new),
                       static_cast<const uint4*>(v_new), static_cast<uint4*>(q_out), ldq / 8,
                       ldk / 8, ldv / 8, ldo / 8, positions, ldp, k_cache, v_cache,
                       static_cast<uint8_t*>(k_scale), static_cast<uint8_t*>(v_scale), block_table,
                       seq_lens, cu_q, dev->err_word, int(num_pages), int(max_pages), int(batch),
                       int(total_q), int(hq), int(hkv)};
    auto kern = head_dim == 64 ? (wide ? rope_kv_append_kernel<64, Q8, 4>
                                       : rope_kv_append_kernel<64, Q8, 1>)
                               : (wide ? rope_kv_append_kernel<128, Q8, 4>
                                       : rope_kv_append_kernel<128, Q8, 1>);
    return launched(launch_pdl(kern, dim3(unsigned(tiles * groups)), dim3(kThreads), 0,
                               reinterpret_cast<cudaStream_t>(stream), a, rot),
                    fn);
}

}  // namespace
}  // namespace bi

using namespace bi;

BI_EXPORT bi_status bi_rope_kv_append(const void* q, int64_t ldq, const void* k_new, int64_t ldk,
                                      const void* v_new, int64_t ldv, void* q_out, int64_t ldo,
                                      void* k_cache, void* v_cache, int64_t num_pages,
                                      const int32_t* block_table, int64_t max_pages,
                                      const int32_t* seq_lens, const int32_t* cu_q, int64_t batch,
                                      int64_t total_q, int64_t num_q_heads, int64_t num_kv_heads,
                                      int64_t head_dim, int64_t page_size, double theta,
                                      const double* inv_freq, int64_t rotary_dim,
                                      const int32_t* positions, int64_t ldp, int64_t num_axes,
                                      const int64_t* sections, bi_stream_t stream) {
    return run<false>("bi_rope_kv_append", q, ldq, k_new, ldk, v_new, ldv, q_out, ldo, k_cache,
                      v_cache, nullptr, nullptr, num_pages, block_table, max_pages, seq_lens, cu_q,
                      batch, total_q, num_q_heads, num_kv_heads, head_dim, page_size, theta,
                      inv_freq, rotary_dim, positions, ldp, num_axes, sections, stream);
}

BI_EXPORT bi_status bi_rope_kv_append_q8(const void* q, int64_t ldq, const void* k_new,
                                         int64_t ldk, const void* v_new, int64_t ldv, void* q_out,
                                         int64_t ldo, void* k_cache, void* v_cache, void* k_scale,
                                         void* v_scale, int64_t num_pages,
                                         const int32_t* block_table, int64_t max_pages,
                                         const int32_t* seq_lens, const int32_t* cu_q,
                                         int64_t batch, int64_t total_q, int64_t num_q_heads,
                                         int64_t num_kv_heads, int64_t head_dim, int64_t page_size,
                                         double theta, const double* inv_freq, int64_t rotary_dim,
                                         const int32_t* positions, int64_t ldp, int64_t num_axes,
                                         const int64_t* sections, bi_stream_t stream) {
    return run<true>("bi_rope_kv_append_q8", q, ldq, k_new, ldk, v_new, ldv, q_out, ldo, k_cache,
                     v_cache, k_scale, v_scale, num_pages, block_table, max_pages, seq_lens, cu_q,
                     batch, total_q, num_q_heads, num_kv_heads, head_dim, page_size, theta,
                     inv_freq, rotary_dim, positions, ldp, num_axes, sections, stream);
}
