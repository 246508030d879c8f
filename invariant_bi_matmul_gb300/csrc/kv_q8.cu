// kv_q8.cu -- the 8-bit paged KV cache: the quantising append.
//
// Format of a cache row (one token, one KV head, D values): D e4m3 codes c and one E8M0
// byte s, standing for c * 2^(s-127).  With amax the row's largest magnitude,
//   e = the smallest integer >= -64 with amax <= 448 * 2^e,  s = e + 127,
//   c_i = e4m3(x_i * 2^-e), round to nearest even (448 is e4m3's largest finite value).
// A power-of-two scale makes x * 2^-e exact, so the only rounding is e4m3's own: at most
// half a step, 2^-4 of a value in e4m3's normal range and 2^(e-10) below it.  The scale
// block is one token of one head because anything longer would make a token's stored bits
// depend on its neighbours -- on how a prompt was cut into calls, and on drafts that were
// rejected.  A row that holds a NaN or an infinity gets s = 255 (E8M0's NaN) and zero codes:
// it reads as NaN throughout, and a query that does not see it stays untouched.
//
// One thread per 16-byte piece of a K row and of the V row beside it; the D/8 threads of a
// row are neighbours in a warp and combine their maxima by shuffles; a CTA takes consecutive
// tokens of one head, so the codes and scale bytes it writes lie together in the page.  Reads 4
// bytes and writes 2 + 2/D per element pair: 8,192 tokens of 8 heads of 128 take 10.9 us (4.6
// TB/s; 2.2 us of it are what the smallest call takes).  The rows are read once, with streaming
// loads, which leave the L2 to the codes (12.2 us without them).  Slower before that: the heads of
// a token together (12.9 to 12.3, scattered single scale bytes), two and four rows per thread
// (13.4 and 14.2), CTAs of 512 (12.7).
#include "attn_common.cuh"

#include <cuda_fp8.h>

namespace bi {
namespace {

constexpr int APPEND_THREADS = 128;
constexpr int kMinExp = -64;  // the smallest scale exponent (a row of zeros has it)

// Largest magnitude of eight bf16 values, as a bf16 bit pattern (magnitudes order as their
// bits; infinities and NaN are the patterns from 0x7f80 on).
__device__ __forceinline__ uint32_t amax_bits(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    return m;
}

// The scale exponent of a row from its largest magnitude (a finite bf16 pattern):
// amax = 1.f * 2^E; 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exp(uint32_t amax) {
    const int E = int(amax >> 7) - 127;
    return max(kMinExp, E - 8 + ((amax & 0x7fu) > 0x60u ? 1 : 0));
}

__device__ __forceinline__ uint2 codes8(const uint4& v, float inv) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(w[i] << 16) * inv,
                                                    __uint_as_float(w[i] & 0xffff0000u) * inv),
                                        __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

template <int D>
__global__ void __launch_bounds__(APPEND_THREADS)
kv_append_q8_kernel(const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
                    uint2* __restrict__ k_cache, uint2* __restrict__ v_cache,
                    uint8_t* __restrict__ k_scale, uint8_t* __restrict__ v_scale, int num_pages,
                    const int32_t* __restrict__ block_table, int max_pages,
                    const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ cu_q, int B,
                    int total_q, int Hkv, unsigned int* err) {
    constexpr int LPR = D / 8;  // threads per row
    pdl_wait();
    pdl_trigger();
    const int h = int(blockIdx.x % unsigned(Hkv));
    const int t = int(blockIdx.x / unsigned(Hkv)) * (APPEND_THREADS / LPR) + int(threadIdx.x) / LPR;
    const int ch = int(threadIdx.x) & (LPR - 1);
    const bool live = t < total_q;  // (the others take part in the shuffles)
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    if (live) {
        const int64_t src = (int64_t(t) * Hkv + h) * LPR + ch;
        k = __ldcs(k_new + src);
        v = __ldcs(v_new + src);
    }
    // the row's place, found while the loads are under way; -1: nowhere
    int64_t dst = -1;
    int lo = 0, hi = B;  // sequence of token t: largest b with cu_q[b] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu_q[mid] <= t) lo = mid; else hi = mid;
    }
    const int b = lo;
    const int L = seq_lens[b];
    const int t0 = cu_q[b];
    const int t1 = cu_q[b + 1];
    if (live && t >= t0 && t < t1) {  // (else a token of no sequence: padding)
        // (t0 <= t < t1: their difference passes 2^31 where t0 is negative only)
        const int qb = int(uint32_t(t1) - uint32_t(t0));
        if (t0 < 0 || qb > L || int64_t(L) > int64_t(max_pages) * PAGE || t1 > total_q) {
            latch_error(err, kErrDeviceArg);
        } else {
            const int pos = L - qb + (t - t0);
            const int phys = block_table[int64_t(b) * max_pages + pos / PAGE];
            if (phys < 0 || phys >= num_pages)
                latch_error(err, kErrDeviceArg);
            else
                dst = (int64_t(phys) * Hkv + h) * PAGE + pos % PAGE;
        }
    }
    uint32_t mk = amax_bits(k), mv = amax_bits(v);
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) {
        mk = max(mk, __shfl_xor_sync(0xffffffffu, mk, off));
        mv = max(mv, __shfl_xor_sync(0xffffffffu, mv, off));
    }
    if (dst < 0) return;
    auto put = [&](const uint4& x, uint32_t m, uint2* cache, uint8_t* scale) {
        const bool bad = m >= 0x7f80u;
        const int e = scale_exp(m);
        cache[dst * LPR + ch] =
            bad ? make_uint2(0, 0) : codes8(x, __uint_as_float(uint32_t(127 - e) << 23));
        if (ch == 0) scale[dst] = bad ? 255 : uint8_t(e + 127);
    };
    put(k, mk, k_cache, k_scale);
    put(v, mv, v_cache, v_scale);
}

}  // namespace

cudaError_t launch_kv_append_q8(const DeviceInfo& dev, const void* k_new, const void* v_new,
                                void* k_cache, void* v_cache, void* k_scale, void* v_scale,
                                const PagedArgs& a, cudaStream_t stream) {
    const int64_t per = APPEND_THREADS / (a.head_dim / 8);  // tokens of a CTA
    auto kern = a.head_dim == 64 ? kv_append_q8_kernel<64> : kv_append_q8_kernel<128>;
    return launch_pdl(kern, dim3(unsigned((a.total_q + per - 1) / per * a.hkv)),
                      dim3(APPEND_THREADS), 0, stream, static_cast<const uint4*>(k_new),
                      static_cast<const uint4*>(v_new), static_cast<uint2*>(k_cache),
                      static_cast<uint2*>(v_cache), static_cast<uint8_t*>(k_scale),
                      static_cast<uint8_t*>(v_scale), int(a.num_pages), a.block_table,
                      int(a.max_pages), a.seq_lens, a.cu_q, int(a.batch), int(a.total_q),
                      int(a.hkv), dev.err_word);
}

}  // namespace bi
