// attention_q8.cu -- decode / verify / prefill attention over the 8-bit paged KV cache
// (kv_q8.cu has its format).
//
// Simple form: one CTA per (sequence, query tile, KV head, 512-key chunk); each row's scores,
// weights and weighted values on the CUDA cores, into the chunk partials that the merge of
// attention.cu combines.
#include "attn_common.cuh"

#include <cuda_fp8.h>

namespace bi {
namespace {

constexpr int QR = 32;  // query rows of a tile: QR / G tokens times the G heads of a KV head
constexpr int THREADS = 128;

__device__ __forceinline__ float e4m3_value(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}
__device__ __forceinline__ float e8m0_value(uint8_t s) {
    return s == 255 ? __int_as_float(0x7fc00000) : exp2f(float(int(s) - 127));
}

template <int D>
__global__ void __launch_bounds__(THREADS)
attn_q8_kernel(const __nv_bfloat16* __restrict__ q, const uint8_t* __restrict__ k_cache,
               const uint8_t* __restrict__ v_cache, const uint8_t* __restrict__ k_scale,
               const uint8_t* __restrict__ v_scale, const int32_t* __restrict__ block_table,
               int max_pages, int num_pages, const int32_t* __restrict__ seq_lens,
               const int32_t* __restrict__ cu_q, int total_q, int max_q, int max_seq_len, int Hq,
               int Hkv, int tiles, float scale_log2, float* __restrict__ ws_o,
               float* __restrict__ ws_ml, int maxC, unsigned int* err) {
    __shared__ float p[CHUNK];
    __shared__ float sq[D];
    __shared__ float red[THREADS / 32];
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x, h = blockIdx.y / tiles, u = blockIdx.y % tiles, b = blockIdx.z;
    const int tid = threadIdx.x, G = Hq / Hkv, TQ = QR / G;
    const SeqInfo si = seq_info(seq_lens, cu_q, b);
    if (!seq_ok(si, max_q, max_seq_len, total_q)) {
        if (tid == 0) latch_error(err, kErrDeviceArg);
        return;
    }
    for (int r = 0; r < TQ * G; ++r) {
        const int j = u * TQ + r / G, hq = h * G + r % G;
        if (j >= si.qb) break;
        const int pos = si.L - si.qb + j;
        if (pos < c * CHUNK) continue;
        const int n = min(CHUNK, pos + 1 - c * CHUNK);
        const int64_t row = int64_t(si.t0 + j) * Hq + hq;
        __syncthreads();
        for (int d = tid; d < D; d += THREADS) sq[d] = __bfloat162float(q[row * D + d]);
        __syncthreads();
        float m = -INFINITY;
        for (int i = tid; i < n; i += THREADS) {
            const int key = c * CHUNK + i;
            const int phys = block_table[int64_t(b) * max_pages + key / PAGE];
            float s = -INFINITY;
            if (phys >= 0 && phys < num_pages) {
                const int64_t at = (int64_t(phys) * Hkv + h) * PAGE + key % PAGE;
                float dot = 0.f;
                for (int d = 0; d < D; ++d) dot = fmaf(sq[d], e4m3_value(k_cache[at * D + d]), dot);
                s = dot * e8m0_value(k_scale[at]) * scale_log2;
            } else {
                latch_error(err, kErrDeviceArg);
            }
            p[i] = s;
            m = fmaxf(m, s);
        }
        for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, off));
        if ((tid & 31) == 0) red[tid >> 5] = m;
        __syncthreads();
        m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        const float use = m == -INFINITY ? 0.f : m;
        __syncthreads();
        float l = 0.f;
        for (int i = tid; i < n; i += THREADS) {
            p[i] = exp2f(p[i] - use);
            l += p[i];
        }
        for (int off = 16; off; off >>= 1) l += __shfl_xor_sync(~0u, l, off);
        if ((tid & 31) == 0) red[tid >> 5] = l;
        __syncthreads();
        l = (red[0] + red[1]) + (red[2] + red[3]);
        const int64_t idx = row * maxC + c;
        for (int d = tid; d < D; d += THREADS) {
            float o = 0.f;
            for (int i = 0; i < n; ++i) {
                const int key = c * CHUNK + i;
                const int phys = block_table[int64_t(b) * max_pages + key / PAGE];
                if (phys < 0 || phys >= num_pages) continue;
                const int64_t at = (int64_t(phys) * Hkv + h) * PAGE + key % PAGE;
                o = fmaf(p[i] * e8m0_value(v_scale[at]), e4m3_value(v_cache[at * D + d]), o);
            }
            ws_o[idx * D + d] = o;
        }
        if (tid == 0) {
            ws_ml[idx * 2] = m;
            ws_ml[idx * 2 + 1] = l;
        }
    }
}

template <int D>
cudaError_t launch_q8_t(const DeviceInfo& dev, const void* q, const PagedArgs& a,
                        const void* k_scale, const void* v_scale, float scale, void* out,
                        float* lse, void* workspace, cudaStream_t stream) {
    const int maxC = int((a.max_seq_len + CHUNK - 1) / CHUNK);
    float* ws_o = static_cast<float*>(workspace);
    float* ws_ml = ws_o + a.total_q * a.hq * int64_t(maxC) * D;
    const int TQ = QR / int(a.hq / a.hkv);
    const int tiles = int((a.max_q + TQ - 1) / TQ);
    if (int64_t(tiles) * a.hkv > 65535) return cudaErrorNotSupported;
    cudaError_t e = launch_pdl(
        attn_q8_kernel<D>, dim3(maxC, unsigned(tiles * a.hkv), unsigned(a.batch)), dim3(THREADS),
        0, stream, static_cast<const __nv_bfloat16*>(q), static_cast<const uint8_t*>(a.k_cache),
        static_cast<const uint8_t*>(a.v_cache), static_cast<const uint8_t*>(k_scale),
        static_cast<const uint8_t*>(v_scale), a.block_table, int(a.max_pages), int(a.num_pages),
        a.seq_lens, a.cu_q, int(a.total_q), int(a.max_q), int(a.max_seq_len), int(a.hq),
        int(a.hkv), tiles, scale * kLog2e, ws_o, ws_ml, maxC, dev.err_word);
    if (e != cudaSuccess) return e;
    return launch_attn_merge(a, workspace, CHUNK_LOG2, out, lse, nullptr, dev.err_word, stream);
}

}  // namespace

cudaError_t launch_attention_q8(const DeviceInfo& dev, const void* q, const PagedArgs& a,
                                const void* k_scale, const void* v_scale, float scale, void* out,
                                float* lse, void* workspace, cudaStream_t stream) {
    if (a.head_dim == 64)
        return launch_q8_t<64>(dev, q, a, k_scale, v_scale, scale, out, lse, workspace, stream);
    return launch_q8_t<128>(dev, q, a, k_scale, v_scale, scale, out, lse, workspace, stream);
}

}  // namespace bi
